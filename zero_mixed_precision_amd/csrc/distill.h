// distill.h -- distillation from a teacher's top logits, and the mean over
// rows that the losses here end with.  Included by dszero.hip inside its
// namespace.
//
// A block has a row of the student's logits.  It loads the row into registers
// once, forms the softmax's maximum and sum from there and writes the gradient
// from there, so a call with the gradient moves each logit once in and once
// out.  Rows too long for the registers are read twice.
//   p_v = exp2((z_v - max) c - log2 sum),  c = log2(e) / temperature
//   dz_v = S coef temperature / T' (p_v - q_v)
// The difference comes before the factor c, so that logits at the type's
// lowest value neither overflow nor lose a row that holds nothing else.

constexpr int kMeanBlock = 1024;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

// coef / used * the sum of the block's rows' losses (fp64, fixed order), for
// thread 0 of a block of BLOCK lanes.
template <int BLOCK>
__device__ __forceinline__ float rows_mean(const float* token_loss, int64_t tokens, int32_t used, float coef)
{
    __shared__ double part[BLOCK / 64];
    double sum = 0.0;
    for (int64_t t = threadIdx.x; t < tokens; t += BLOCK)
        sum += static_cast<double>(token_loss[t]);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        sum += __shfl_xor(sum, off);
    if (__lane_id() == 0)
        part[threadIdx.x / 64] = sum;
    __syncthreads();
    sum = 0.0;
    for (int w = 0; w < BLOCK / 64; ++w)
        sum += part[w];
    return used > 0 ? static_cast<float>(static_cast<double>(coef) * sum / used) : 0.0f;
}

// `count` is left at zero for the next call, if asked.
__global__ __launch_bounds__(kMeanBlock) void rows_mean_kernel(const float* __restrict__ token_loss, int64_t tokens,
                                                              int32_t* __restrict__ count, float coef,
                                                              float* __restrict__ loss, int32_t* __restrict__ used_out,
                                                              int32_t clear)
{
    const int32_t used = *count;
    const float mean = rows_mean<kMeanBlock>(token_loss, tokens, used, coef);
    if (threadIdx.x == 0) {
        *loss = mean;
        *used_out = used;
        if (clear)
            *count = 0;
    }
}

struct Distill {
    const unsigned char* logits;
    int64_t tokens, vocab, stride;
    const void *teacher, *index;
    int64_t ts, is;                        // strides of teacher and index
    int32_t k, tfmt, wide;                 // wide: indices of 64 bits
    int32_t search;                        // the blocks find the used rows themselves
    const uint8_t* mask;
    float c, tau, per_tau;                 // log2(e) / temperature, temperature, 1 / temperature
    float coef;
    float* token_loss;
    unsigned char* grad;
    int64_t gs;
    int32_t* count;                        // used rows; behind it the blocks that are done (zero between calls)
    uint8_t* flag;                         // [tokens]: the row is used
    const ds_scaler* st;
    float* loss;
    int32_t* used;
};

__device__ __forceinline__ int64_t distill_index(const Distill& s, int64_t t, int j)
{
    const int64_t at = t * s.is + j;
    return s.wide ? static_cast<const int64_t*>(s.index)[at] : static_cast<const int32_t*>(s.index)[at];
}

// Whether row t is used (mask, a teacher's entry above -infinity, a logit above
// -infinity), for the lane's own t (below s.tokens, or the lane has none).  A
// row's first entry and first logit nearly always say so; the rows where they do
// not are searched by the wave together, one after another (4096 x 32000 in bf16,
// 64 entries: 134 us, 202 if no row has a first logit, 219 without first entries,
// 3.9 ms with a fourth of the rows nothing but -infinity: leave such out by mask).
template <int ZF>
__device__ __forceinline__ bool distill_used(const Distill& s, int64_t t, int lane)
{
    bool on = t < s.tokens && (s.mask == nullptr || s.mask[t] != 0), open = false;
    if (on)
        open = distill_index(s, t, 0) < 0 || load_gate(s.teacher, s.tfmt, t * s.ts) == kNegInf ||
               load_elem<ZF>(s.logits, t * s.stride) == kNegInf;
    for (uint64_t left = __ballot(open); left != 0ull; left &= left - 1) {
        const int of = __ffsll(static_cast<long long>(left)) - 1;
        const int64_t u = t - lane + of;
        bool any = false;
        for (int j = lane; j < s.k; j += 64)
            any = any || (distill_index(s, u, j) >= 0 && !(load_gate(s.teacher, s.tfmt, u * s.ts + j) == kNegInf));
        bool found = false;
        if (__ballot(any) != 0ull)
            for (int64_t v = lane; v - lane < s.vocab && !found; v += 64)
                found = __ballot(v < s.vocab && !(load_elem<ZF>(s.logits, u * s.stride + v) == kNegInf)) != 0ull;
        if (lane == of)
            on = found;
    }
    return on;
}

constexpr int kUsedBlock = 256;
template <int ZF>
__global__ __launch_bounds__(kUsedBlock) void distill_used_kernel(Distill s)
{
    __shared__ int32_t part[kUsedBlock / 64];
    const int lane = static_cast<int>(__lane_id()), wave = threadIdx.x / 64;
    int32_t used = 0;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kUsedBlock;
    for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kUsedBlock; t0 < s.tokens; t0 += step) {
        const int64_t t = t0 + threadIdx.x;
        const bool on = distill_used<ZF>(s, t, lane);
        if (t < s.tokens)
            s.flag[t] = on;
        used += __popcll(__ballot(on));
    }
    if (lane == 0)
        part[wave] = used;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kUsedBlock / 64; ++w)
            used += part[w];
        if (used != 0)
            atomicAdd(s.count, used);
    }
}

// A maximum and a sum of exp2((x - max) c) beside it.
struct TopSum {
    float top, sum;
};

__device__ __forceinline__ float finite_top(float top) { return top == kNegInf ? 0.0f : top; }

__device__ __forceinline__ TopSum join(TopSum a, TopSum b, float c)
{
    const float top = fmaxf(a.top, b.top), ref = finite_top(top);
    // a side that holds nothing (sum 0 under -infinity) gives nothing; NaN and infinities stay
    const float x = a.top == kNegInf ? a.sum : a.sum * __builtin_amdgcn_exp2f((a.top - ref) * c);
    const float y = b.top == kNegInf ? b.sum : b.sum * __builtin_amdgcn_exp2f((b.top - ref) * c);
    return {top, x + y};
}

__device__ __forceinline__ TopSum wave_join(TopSum a, float c)
{
#pragma unroll
    for (int off = 1; off < 64; off <<= 1)
        a = join(a, TopSum{__shfl_xor(a.top, off), __shfl_xor(a.sum, off)}, c);
    return a;
}

template <int ZF>
__device__ __forceinline__ float top_of(u32x4 v)
{
    float x[ZF == kF32 ? 4 : 8], top = kNegInf;
    widen_vec<ZF>(v, x);
#pragma unroll
    for (int i = 0; i < (ZF == kF32 ? 4 : 8); ++i)
        top = fmaxf(top, x[i]);
    return top;
}

__device__ __forceinline__ float wave_max(float x)
{
#pragma unroll
    for (int off = 1; off < 64; off <<= 1)
        x = fmaxf(x, __shfl_xor(x, off));
    return x;
}

__device__ __forceinline__ float wave_sum(float x)
{
#pragma unroll
    for (int off = 1; off < 64; off <<= 1)
        x += __shfl_xor(x, off);
    return x;
}

// A row's softmax as the gradient needs it: p = 2^((x - top) c - log2 sum).
// `by` is the gradient's factor, NaN where the teacher's entries hold one.
struct DistillRow {
    float top, c, log_sum, by;
};

__device__ __forceinline__ float distill_p(float x, const DistillRow& r)
{
    return __builtin_amdgcn_exp2f(__builtin_fmaf(x - r.top, r.c, -r.log_sum));
}

// Vector i from `at` on: a base that is the same for the wave and an offset of 32 bits.
__device__ __forceinline__ u32x4 vector_at(const unsigned char* at, uint32_t i)
{
    return reinterpret_cast<const u32x4_any*>(at)[i];
}

template <int ZF, bool ACC>
__device__ __forceinline__ void distill_write(unsigned char* out, uint32_t i, u32x4 v, const DistillRow& r, bool on)
{
    constexpr int kVec = ZF == kF32 ? 4 : 8;
    float x[kVec], o[kVec] = {};
    widen_vec<ZF>(v, x);
    if constexpr (ACC)
        widen_vec<ZF>(vector_at(out, i), o);
#pragma unroll
    for (int m = 0; m < kVec; ++m)
        x[m] = ACC ? __builtin_fmaf(r.by, distill_p(x[m], r), o[m]) : r.by * distill_p(x[m], r);
    v = narrow_vec<ZF>(x);
#pragma unroll
    for (int m = 0; m < 4; ++m)
        v[m] = on ? v[m] : 0u;                                 // a row that is not used
    reinterpret_cast<u32x4_any*>(out)[i] = v;
}

constexpr int kTwice = 0;                  // NV of the form that reads its row twice
constexpr int kTwiceHold = 4;

// Up to so many rows one kernel does the whole call: every block finds all used
// rows itself, and the last block to end forms the mean.  Where the gradient takes
// the logits' place a row's logits are gone once its block has written, and a row
// of nothing but -infinity, zeroed, would look used to a block that searches it
// then: the used rows come from a kernel before, unless one block has the only row
// (32 x 32000 in bf16 17.6 us, 15.2 with the gradient elsewhere).
constexpr int kFewRows = 256;

// NV vectors a lane hold a row, as they came: what is widened from them is formed
// again where it is used, or it would need twice the registers, and the scheduler
// is held to one vector at a time for the same reason.  A block goes from row to
// row; while it writes a row's gradient it loads the next row into the registers
// that this frees, so loads and stores are on their way together, and sums the
// first vectors while the last are still coming.  For that, the wait for a vector
// must be able to count the loads behind it: none of them is conditional, lanes
// past the row's end read and write its last vector with the others.
//
// The sum needs no maximum, only a reference that no logit exceeds by far: a
// wave takes the largest of its first vectors.  With ref = c top rounded, 2^(c x
// - ref) is one fused operation and an exponential, and as exact as from the
// difference (the gradient takes the difference itself, which cannot overflow).
// Where the sum says that the reference was none (nothing but
// -infinity in the first vectors, a logit 2^64 times as likely as the reference,
// values near the type's range, NaN), the row is summed again from its maximum,
// differences first.
template <int ZF, int BLOCK, int NV, bool GRAD, bool ACC>
__global__ __launch_bounds__(BLOCK) void distill_kernel(Distill s)
{
    constexpr int ES = ZF == kF32 ? 4 : 2, kVec = 16 / ES, kWaves = BLOCK / 64;
    constexpr int kHold = NV == kTwice ? kTwiceHold : NV;
        __shared__ TopSum of_row[kWaves], of_teacher[kWaves];
    __shared__ float part[kWaves];
    // the entries' places (-1: absent) and their shares, of two used rows in turn (a
    // wave may read the last row's while another writes this one's; the row after
    // writes behind this one's barriers, which a row that is not used does not have);
    // a lane's own: the student's logit there, and what the gradient held there
    __shared__ __attribute__((aligned(16))) int32_t places[2][DS_MAX_TEACHER_LOGITS];
    __shared__ float shares[2][DS_MAX_TEACHER_LOGITS];
    __shared__ float of_logit[DS_MAX_TEACHER_LOGITS];
    __shared__ float old[ACC ? DS_MAX_TEACHER_LOGITS : 1];
    __shared__ uint8_t few[kFewRows];
    __shared__ int32_t few_used[kWaves];
    const bool is_few = s.tokens <= kFewRows, search = s.search != 0;
    const int tid = static_cast<int>(threadIdx.x), lane = static_cast<int>(__lane_id());
    const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
    const int vecs = static_cast<int>(s.vocab / kVec);
    const int64_t rest = static_cast<int64_t>(vecs) * kVec;
    const int rest_lanes = static_cast<int>(s.vocab - rest);
    const float c = s.c;
    u32x4 v[kHold];
    // where the lane's vector n starts, from a row's first byte: the wave's part and the lane's vectors behind it
    auto part_of = [&](int n) { return min(n * BLOCK, vecs - 1); };
    auto lane_of = [&](int n) {
        int own = tid;
        asm volatile("" : "+v"(own));                          // formed where it is used: NV of them take too many registers
        return min(own, vecs - 1 - part_of(n));
    };
    auto load_one = [&](int64_t t, int n) { v[n] = vector_at(s.logits + t * s.stride * ES + part_of(n) * 16, lane_of(n)); };
    // what comes before a row's vectors: the lane's first entry (its place, past the vocabulary as it is, and the
    // teacher's logit), its one value past the vectors, whether the row is used
    int64_t place = -1;
    float theirs_here = kNegInf, last = kNegInf;
    uint32_t flag = 0;
    auto load_entry = [&](int64_t t) {
        place = -1;
        if (tid < s.k) {
            place = distill_index(s, t, tid);
            theirs_here = load_gate(s.teacher, s.tfmt, t * s.ts + tid);
        }
        if (tid < rest_lanes)
            last = load_elem<ZF>(s.logits, t * s.stride + rest + tid);
        if (!search)
            flag = s.flag[t];
    };
    load_entry(min(static_cast<int64_t>(blockIdx.x), s.tokens - 1));
    if constexpr (NV != kTwice) {
#pragma unroll
        for (int n = 0; n < NV; ++n)
            load_one(min(static_cast<int64_t>(blockIdx.x), s.tokens - 1), n);
    }
    int32_t used = 0;
    if (search) {
        int32_t mine = 0;
        for (int64_t t0 = 0; t0 < s.tokens; t0 += BLOCK) {
            const bool on = distill_used<ZF>(s, t0 + tid, lane);
            if (t0 + tid < s.tokens)
                few[t0 + tid] = on;
            mine += __popcll(__ballot(on));
        }
        if (lane == 0)
            few_used[wave] = mine;
        __syncthreads();
        for (int w = 0; w < kWaves; ++w)
            used += few_used[w];
    } else {
        used = *s.count;
    }
    const float scale = s.st != nullptr ? s.st->scale : 1.0f;
    const float factor = used > 0 ? static_cast<float>(static_cast<double>(scale) * static_cast<double>(s.coef) *
                                                       static_cast<double>(s.tau) / used)
                                  : 0.0f;
    int turn = 0;
    for (int64_t t = blockIdx.x; t < s.tokens; t += gridDim.x) {
        const unsigned char* in = s.logits + t * s.stride * ES;
        unsigned char* out = GRAD ? s.grad + t * s.gs * ES : nullptr;
        const int64_t next = min(t + gridDim.x, s.tokens - 1);
        // the same for the whole block
        const bool on = __builtin_amdgcn_readfirstlane(search ? few[t & (kFewRows - 1)] : flag) != 0;
        const float mine = last;
        DistillRow row{0.0f, c, 0.0f, 0.0f};
        float loss = 0.0f, fine = 1.0f;
        int here = -1;                                         // the first entry's place, and the rest that is the lane's
        float logit_here = 0.0f, old_here = 0.0f, share_here = 0.0f;
        bool first = true, alone = true;                       // of its place: the first entry, the only one
        int32_t* at = places[turn];
        float* share = shares[turn];
        if (on) {
            turn ^= 1;                                         // for the next used row
            TopSum theirs{kNegInf, 0.0f};
            auto add_entry = [&](int64_t& p, float& x) {       // an absent one is -infinity, one past the vocabulary NaN
                if (p < 0)
                    x = kNegInf;
                if (p >= s.vocab) {
                    p = -1;
                    x = __builtin_nanf("");
                }
                if (!(x == kNegInf))
                    theirs = join(theirs, TopSum{x, __builtin_amdgcn_exp2f((x - x) * c)}, c);
            };
            if (tid < s.k) {
                add_entry(place, theirs_here);
                here = static_cast<int>(place);
                at[tid] = here;
                if (here >= 0) {                               // used after the row's sums: no wait for it here
                    logit_here = load_elem<ZF>(in, here);
                    if constexpr (GRAD && ACC)
                        old_here = load_elem<ZF>(out, here);
                }
            }
            for (int j = tid + BLOCK; j < s.k; j += BLOCK) {
                int64_t p = distill_index(s, t, j);
                float x = load_gate(s.teacher, s.tfmt, t * s.ts + j);
                add_entry(p, x);
                at[j] = static_cast<int32_t>(p);
                share[j] = x;
                of_logit[j] = p >= 0 ? load_elem<ZF>(in, p) : 0.0f;
                if constexpr (GRAD && ACC)
                    old[j] = p >= 0 ? load_elem<ZF>(out, p) : 0.0f;
            }
            // f(vector, whether the lane has it) for every vector
            auto each = [&](auto f) {
                if constexpr (NV == kTwice) {
                    for (int i0 = tid; i0 < vecs; i0 += kHold * BLOCK) {
#pragma unroll
                        for (int n = 0; n < kHold; ++n)
                            v[n] = vector_at(in, min(i0 + n * BLOCK, vecs - 1));
#pragma unroll
                        for (int n = 0; n < kHold; ++n)
                            f(v[n], i0 + n * BLOCK < vecs);
                    }
                } else {
#pragma unroll
                    for (int n = 0; n < NV; ++n) {
                        int own = tid;
                        asm volatile("" : "+v"(own));
                        f(v[n], own < vecs - n * BLOCK);
                        asm("" : "+v"(v[n]));
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            };
            float top = mine;
            if constexpr (NV == kTwice) {
                if (tid < vecs)
                    top = fmaxf(top, top_of<ZF>(vector_at(in, tid)));
            } else {
                top = fmaxf(top, tid < vecs ? top_of<ZF>(v[0]) : kNegInf);
            }
            top = wave_max(top);
            const float ref = top * c;
            float sum = __builtin_amdgcn_exp2f(__builtin_fmaf(mine, c, -ref));
            each([&](u32x4 vec, bool has) {
                float x[kVec], of_vec = 0.0f;
                widen_vec<ZF>(vec, x);
#pragma unroll
                for (int i = 0; i < kVec; ++i)
                    of_vec = of_vec + __builtin_amdgcn_exp2f(__builtin_fmaf(x[i], c, -ref));
                sum = sum + (has ? of_vec : 0.0f);
            });
            sum = wave_sum(sum);
            if (wave * 64 < s.k)
                theirs = wave_join(theirs, c);
            if (lane == 0) {
                const bool some = wave * 64 < vecs || wave * 64 < rest_lanes;
                of_row[wave] = some ? TopSum{top, sum} : TopSum{kNegInf, 0.0f};
                of_teacher[wave] = theirs;
            }
            __syncthreads();
            row.top = of_row[0].top;
#pragma unroll
            for (int w = 1; w < kWaves; ++w)
                row.top = fmaxf(row.top, of_row[w].top);
            const float row_ref = row.top * c;
            float total_sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w)
                total_sum += of_row[w].top == kNegInf ? of_row[w].sum
                                                      : of_row[w].sum * __builtin_amdgcn_exp2f(of_row[w].top * c - row_ref);
            const bool fits = total_sum >= 0.5f && total_sum <= 0x1p64f && fabsf(row_ref) <= 0x1p126f;
            theirs = of_teacher[0];
            for (int w = 1; w < kWaves && w * 64 < s.k; ++w)
                theirs = join(theirs, of_teacher[w], c);
            if (!fits) {                                       // seldom: from memory, in short code
                float most = mine;
#pragma unroll 1
                for (int i = tid; i < vecs; i += BLOCK)
                    most = fmaxf(most, top_of<ZF>(vector_at(in, i)));
                most = wave_max(most);
                __syncthreads();                               // the sums above have been read
                if (lane == 0)
                    of_row[wave].top = most;
                __syncthreads();
                for (int w = 0; w < kWaves; ++w)
                    most = fmaxf(most, of_row[w].top);
                sum = __builtin_amdgcn_exp2f((mine - most) * c);
#pragma unroll 1
                for (int i = tid; i < vecs; i += BLOCK) {
                    float x[kVec];
                    widen_vec<ZF>(vector_at(in, i), x);
#pragma unroll
                    for (int m = 0; m < kVec; ++m)
                        sum = sum + __builtin_amdgcn_exp2f((x[m] - most) * c);
                }
                sum = wave_sum(sum);
                if (lane == 0)
                    of_row[wave].sum = sum;
                __syncthreads();
                total_sum = 0.0f;
                for (int w = 0; w < kWaves; ++w)
                    total_sum += of_row[w].sum;
                row.top = most;
            }
            row.log_sum = __builtin_amdgcn_logf(total_sum);
            const float log_theirs = __builtin_amdgcn_logf(theirs.sum);
            // 1, or NaN where the teacher's entries hold a NaN or +infinity
            fine = theirs.sum * __builtin_amdgcn_rcpf(theirs.sum) > 0.0f ? 1.0f : __builtin_nanf("");
            row.by = factor * fine;
            // what the reference's rounding has added to the sum's logarithm
            if (fits)
                row.log_sum -= __builtin_fmaf(row.top, c, -row_ref);
            auto take_share = [&](float x, int p, float z) {
                const float q = x == kNegInf ? 0.0f : __builtin_amdgcn_exp2f((x - theirs.top) * c - log_theirs);
                // in natural logarithms: a difference near the type's range does not fit times log2(e)
                if (q != 0.0f && p >= 0)
                    loss = loss + q * (((x - theirs.top) * s.per_tau - log_theirs * kLn2) -
                                       ((z - row.top) * s.per_tau - row.log_sum * kLn2));
                return q;
            };
            if (wave * 64 < s.k) {
                if (tid < s.k) {
                    share_here = take_share(theirs_here, here, logit_here);
                    share[tid] = share_here;
                    if (GRAD && here >= 0) {
                        for (int i = 0; i < s.k; ++i) {
                            const bool same = at[i] == here && i != tid;
                            first = first && !(same && i < tid);
                            alone = alone && !same;
                        }
                    }
                }
                for (int j = tid + BLOCK; j < s.k; j += BLOCK)
                    share[j] = take_share(share[j], at[j], of_logit[j]);
#pragma unroll
                for (int off = 1; off < 64; off <<= 1)
                    loss += __shfl_xor(loss, off);
            }
            if (lane == 0)
                part[wave] = loss;
        }
        load_entry(next);
        if constexpr (NV == kTwice) {
            if (GRAD && (on || !ACC))
#pragma unroll 4
                for (int i = tid; i < vecs; i += BLOCK)
                    distill_write<ZF, ACC>(out, i, vector_at(in, i), row, on);
        } else {
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                if constexpr (GRAD && ACC) {                   // added to: by one lane only
                    if (on && n * BLOCK + tid < vecs)
                        distill_write<ZF, ACC>(out + n * BLOCK * 16, tid, v[n], row, on);
                } else if constexpr (GRAD) {
                    distill_write<ZF, ACC>(out + part_of(n) * 16, lane_of(n), v[n], row, on);
                }
                load_one(next, n);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if (GRAD && (on || !ACC) && tid < rest_lanes) {
            const float was = ACC ? load_elem<ZF>(out, rest + tid) : 0.0f;
            store_elem<ZF>(out, rest + tid, on ? __builtin_fmaf(row.by, distill_p(mine, row), was) : 0.0f);
        }
        if (on)
            __syncthreads();
        if (tid == 0) {
            for (int w = 1; w < kWaves && on; ++w)
                loss += part[w];
            s.token_loss[t] = s.tau * s.tau * loss * fine;
        }
        if (GRAD && on && tid < s.k) {
            // where the teacher has entries: written again with their shares, by the first entry of each place
            auto rewrite = [&](int p, float q, float z, float was) {
                store_elem<ZF>(out, p, __builtin_fmaf(row.by, distill_p(z, row) - q, was));
            };
            auto total = [&](int p) {
                float q = 0.0f;
                for (int i = 0; i < s.k; ++i)
                    q = at[i] == p ? q + share[i] : q;
                return q;
            };
            if (here >= 0 && first)
                rewrite(here, alone ? share_here : total(here), logit_here, old_here);
            for (int j = tid + BLOCK; j < s.k; j += BLOCK) {
                const int p = at[j];
                bool lead = p >= 0;
                for (int i = 0; i < j && lead; ++i)
                    lead = at[i] != p;
                if (lead)
                    rewrite(p, total(p), of_logit[j], ACC ? old[j] : 0.0f);
            }
        }
    }
    if (is_few) {
        __shared__ uint32_t ticket;
        uint32_t* done = reinterpret_cast<uint32_t*>(s.count) + 1;
        if (gridDim.x > 1) {
            __threadfence();
            __syncthreads();
            if (tid == 0)
                ticket = atomicAdd(done, 1u);
            __syncthreads();
            if (ticket != gridDim.x - 1)
                return;
            __threadfence();
        } else {
            __syncthreads();
        }
        const float mean = rows_mean<BLOCK>(s.token_loss, s.tokens, used, s.coef);
        if (tid == 0) {
            *s.loss = mean;
            *s.used = used;
            *done = 0;
            if (!search)
                *s.count = 0;                                  // all blocks have read it
        }
    }
}

// ---- host side ----

constexpr int64_t kDistillMaxVocab = int64_t(1) << 30;

uint64_t distill_ws_bytes(int64_t tokens) { return 8 + static_cast<uint64_t>(tokens); }

bool distill_tokens_ok(int64_t tokens) { return tokens >= 0 && tokens <= kBalMaxTokens; }

// As many blocks as rows, or per_cu for each of the 256 CUs with about as many
// rows each.  That many a CU holds at once, but for two forms, whose last blocks
// start when others end: of 64 lanes seven fit (20.8 KB of LDS each; six where the
// gradient is added), not twelve, and of 256 lanes with the gradient five (82
// registers), not six.
template <int ZF, int BLOCK, int NV>
void launch_distill2(int per_cu, hipStream_t st, const Distill& s, bool accumulate)
{
    const int64_t most = 256 * static_cast<int64_t>(per_cu), turns = (s.tokens + most - 1) / most;
    // no more blocks than rows: none but a row's own may search it
    const unsigned b = static_cast<unsigned>(std::min<int64_t>(grid_blocks((s.tokens + turns - 1) / turns, BLOCK), s.tokens));
    if (s.grad == nullptr) distill_kernel<ZF, BLOCK, NV, false, false><<<b, BLOCK, 0, st>>>(s);
    else if (accumulate)   distill_kernel<ZF, BLOCK, NV, true, true><<<b, BLOCK, 0, st>>>(s);
    else                   distill_kernel<ZF, BLOCK, NV, true, false><<<b, BLOCK, 0, st>>>(s);
}

template <int ZF>
void launch_distill(hipStream_t st, const Distill& s, bool accumulate)
{
    const int64_t vecs = s.vocab / (ZF == kF32 ? 4 : 8);
    if (vecs < 1)           launch_distill2<ZF, 1024, kTwice>(1, st, s, accumulate);
    else if (vecs <= 256)   launch_distill2<ZF, 64, 4>(12, st, s, accumulate);
    else if (vecs <= 1024)  launch_distill2<ZF, 256, 4>(6, st, s, accumulate);
    else if (vecs <= 4096)  launch_distill2<ZF, 512, 8>(2, st, s, accumulate);
    else if (vecs <= 8192)  launch_distill2<ZF, 1024, 8>(1, st, s, accumulate);
    else if (vecs <= 16384) launch_distill2<ZF, 1024, 16>(1, st, s, accumulate);
    else                    launch_distill2<ZF, 1024, kTwice>(1, st, s, accumulate);
}

ds_status distill_loss(const ds_scaler* st, const void* logits, ds_dtype dt, int64_t tokens, int64_t vocab, int64_t stride,
                       const void* teacher, ds_dtype tdt, int64_t ts, const void* index, int32_t index_bytes, int64_t is,
                       int32_t k, const uint8_t* mask, float temperature, float coef, float* token_loss, float* loss,
                       int32_t* used, void* grad, int64_t gs, bool accumulate, void* ws, size_t ws_bytes, hipStream_t stream)
{
    if (!distill_tokens_ok(tokens) || vocab < 1 || vocab > kDistillMaxVocab || k < 1 || k > DS_MAX_TEACHER_LOGITS ||
        !rows_ok(tokens, vocab, stride) || !rows_ok(tokens, k, ts) || !rows_ok(tokens, k, is) ||
        (grad != nullptr && !rows_ok(tokens, vocab, gs)))
        return DS_ERR_SIZE;
    if (!known(dt) || !known(tdt) || (index_bytes != 4 && index_bytes != 8))
        return DS_ERR_DTYPE;
    if (!finite_ge0(coef) || !(temperature >= 1.0f / 1024.0f && temperature <= 1024.0f) ||
        (accumulate && grad == nullptr))
        return DS_ERR_HPARAM;
    if (loss == nullptr || used == nullptr || ws == nullptr ||
        (tokens > 0 && (logits == nullptr || teacher == nullptr || index == nullptr || token_loss == nullptr)))
        return DS_ERR_NULL;
    const uint64_t es = esize(dt), ib = static_cast<uint64_t>(index_bytes);
    if (!aligned(logits, es) || !aligned(teacher, esize(tdt)) || !aligned(index, ib) || !aligned(token_loss, 4) ||
        !aligned(loss, 4) || !aligned(used, 4) || !aligned(grad, es) || !aligned(ws, 8) || !aligned(st, 8))
        return DS_ERR_ALIGN;
    const uint64_t need = distill_ws_bytes(tokens);
    if (ws_bytes < need)
        return DS_ERR_SIZE;
    // the gradient may take the logits' place
    const bool in_place = grad == logits && gs == stride && !accumulate;
    const void* p[10] = {logits, teacher, index, mask, st, token_loss, loss, used, ws, in_place ? nullptr : grad};
    const uint64_t span = disp_span(tokens, vocab, stride, dt);
    const uint64_t bytes[10] = {span, disp_span(tokens, k, ts, tdt), bal_span(tokens, k, is, ib),
                                static_cast<uint64_t>(tokens), sizeof(ds_scaler), 4 * static_cast<uint64_t>(tokens), 4, 4,
                                need, grad == nullptr ? 0 : disp_span(tokens, vocab, gs, dt)};
    if (bal_alias(p, bytes, 10, 5))
        return DS_ERR_ALIAS;
    if (in_place)
        for (int i = 1; i < 5; ++i)
            if (overlap(grad, span, p[i], bytes[i]))
                return DS_ERR_ALIAS;
    const bool search = tokens <= kFewRows && (!in_place || tokens == 1);
    const Distill s{static_cast<const unsigned char*>(logits), tokens, vocab, stride, teacher, index, ts, is, k, fmt_of(tdt),
                    index_bytes == 8, search, mask, static_cast<float>(1.44269504088896340736 / static_cast<double>(temperature)),
                    temperature, 1.0f / temperature, coef, token_loss, static_cast<unsigned char*>(grad), gs, static_cast<int32_t*>(ws),
                    static_cast<uint8_t*>(ws) + 8, st, loss, used};
    if (tokens > 0 && !search) {
        const unsigned b = grid_blocks((tokens + kUsedBlock - 1) / kUsedBlock, kUsedBlock);
        if (dt == DS_FP16)      distill_used_kernel<kF16><<<b, kUsedBlock, 0, stream>>>(s);
        else if (dt == DS_BF16) distill_used_kernel<kBF16><<<b, kUsedBlock, 0, stream>>>(s);
        else                    distill_used_kernel<kF32><<<b, kUsedBlock, 0, stream>>>(s);
        if (launched() != DS_OK)
            return DS_ERR_HIP;
    }
    if (tokens > 0) {
        if (dt == DS_FP16)      launch_distill<kF16>(stream, s, accumulate);
        else if (dt == DS_BF16) launch_distill<kBF16>(stream, s, accumulate);
        else                    launch_distill<kF32>(stream, s, accumulate);
        if (launched() != DS_OK)
            return DS_ERR_HIP;
        if (tokens <= kFewRows)
            return DS_OK;
    }
    rows_mean_kernel<<<1, kMeanBlock, 0, stream>>>(token_loss, tokens, s.count, coef, loss, used, 1);
    return launched();
}
