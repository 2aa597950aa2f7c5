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

// loss = coef / used * sum of token_loss (fp64, fixed order), *used_out = used.
// `count` is left at zero for the next call.
__global__ __launch_bounds__(kMeanBlock) void rows_mean_kernel(const float* __restrict__ token_loss, int64_t tokens,
                                                              int32_t* __restrict__ count, float coef,
                                                              float* __restrict__ loss, int32_t* __restrict__ used_out,
                                                              int32_t clear)
{
    __shared__ double part[kMeanBlock / 64];
    double sum = 0.0;
    for (int64_t t = threadIdx.x; t < tokens; t += kMeanBlock)
        sum += static_cast<double>(token_loss[t]);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        sum += __shfl_xor(sum, off);
    if (__lane_id() == 0)
        part[threadIdx.x / 64] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        sum = 0.0;
        for (int w = 0; w < kMeanBlock / 64; ++w)
            sum += part[w];
        const int32_t used = *count;
        *loss = used > 0 ? static_cast<float>(static_cast<double>(coef) * sum / used) : 0.0f;
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
    const uint8_t* mask;
    float c, tau, per_tau;                 // log2(e) / temperature, temperature, 1 / temperature
    float coef;
    float* token_loss;
    unsigned char* grad;
    int64_t gs;
    int32_t* count;                        // used rows
    uint8_t* flag;                         // [tokens]: the row is used
    const ds_scaler* st;
};

__device__ __forceinline__ int64_t distill_index(const Distill& s, int64_t t, int j)
{
    const int64_t at = t * s.is + j;
    return s.wide ? static_cast<const int64_t*>(s.index)[at] : static_cast<const int32_t*>(s.index)[at];
}

// Which rows are used, and how many: mask, a teacher's entry above -infinity, a
// logit above -infinity.  A wave has a row and reads on only while it has seen
// nothing else than -infinity.
constexpr int kUsedBlock = 256;
template <int ZF>
__global__ __launch_bounds__(kUsedBlock) void distill_used_kernel(Distill s)
{
    __shared__ int32_t part[kUsedBlock / 64];
    const int lane = static_cast<int>(__lane_id()), wave = threadIdx.x / 64;
    int32_t used = 0;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kUsedBlock / 64);
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * (kUsedBlock / 64) + wave; t < s.tokens; t += step) {
        bool on = s.mask == nullptr || s.mask[t] != 0;
        if (on) {
            bool any = false;
            for (int j = lane; j < s.k; j += 64)
                any = any || (distill_index(s, t, j) >= 0 && !(load_gate(s.teacher, s.tfmt, t * s.ts + j) == kNegInf));
            on = __ballot(any) != 0ull;
        }
        if (on) {
            on = false;
            for (int64_t v = lane; v - lane < s.vocab && !on; v += 64)
                on = __ballot(v < s.vocab && !(load_elem<ZF>(s.logits, t * s.stride + v) == kNegInf)) != 0ull;
        }
        if (lane == 0)
            s.flag[t] = on;
        used += on;
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

constexpr int kNoVectors = 0;              // NV of the form that reads its row twice
constexpr int kTwiceUnroll = 4;

template <int ZF, int BLOCK, int NV, bool GRAD, bool ACC>
__global__ __launch_bounds__(BLOCK) void distill_kernel(Distill s)
{
    constexpr int ES = ZF == kF32 ? 4 : 2, kVec = 16 / ES, kWaves = BLOCK / 64;
    constexpr int kTeacher = (DS_MAX_TEACHER_LOGITS + BLOCK - 1) / BLOCK;   // entries per lane, at most
    constexpr int kHold = NV == kNoVectors ? kTwiceUnroll : NV;
    __shared__ TopSum of_row[kWaves], of_teacher[kWaves];
    __shared__ float part[kWaves];
    __shared__ int32_t at[DS_MAX_TEACHER_LOGITS];
    __shared__ float share[DS_MAX_TEACHER_LOGITS];
    const int tid = static_cast<int>(threadIdx.x), wave = tid / 64, lane = static_cast<int>(__lane_id());
    const int64_t vecs = s.vocab / kVec, rest = vecs * kVec;
    const float c = s.c;
    const int32_t used = *s.count;
    const float scale = s.st != nullptr ? s.st->scale : 1.0f;
    const float factor = used > 0 ? static_cast<float>(static_cast<double>(scale) * static_cast<double>(s.coef) *
                                                       static_cast<double>(s.tau) / used)
                                  : 0.0f;
    for (int64_t t = blockIdx.x; t < s.tokens; t += gridDim.x) {
        const unsigned char* row = s.logits + t * s.stride * ES;
        unsigned char* out = GRAD ? s.grad + t * s.gs * ES : nullptr;
        const u32x4_any* in = reinterpret_cast<const u32x4_any*>(row);
        if (s.flag[t] == 0) {                                  // the same for the whole block
            if (tid == 0)
                s.token_loss[t] = 0.0f;
            if constexpr (GRAD && !ACC) {
                for (int64_t i = tid; i < vecs; i += BLOCK)
                    reinterpret_cast<u32x4_any*>(out)[i] = u32x4{0, 0, 0, 0};
                if (rest + tid < s.vocab)
                    store_elem<ZF>(out, rest + tid, 0.0f);
            }
            continue;
        }
        u32x4 v[kHold];
        TopSum mine{kNegInf, 0.0f};
        constexpr uint32_t kNone = ZF == kF32 ? 0xFF800000u : ZF == kBF16 ? 0xFF80FF80u : 0xFC00FC00u;
        float last = kNegInf;                                  // the lane's one value past the vectors
        if (rest + tid < s.vocab)
            last = load_elem<ZF>(row, rest + tid);
        for (int64_t i0 = tid; i0 < vecs; i0 += static_cast<int64_t>(kHold) * BLOCK) {
#pragma unroll
            for (int n = 0; n < kHold; ++n) {
                v[n] = u32x4{kNone, kNone, kNone, kNone};
                if (i0 + n * BLOCK < vecs)
                    v[n] = in[i0 + n * BLOCK];
            }
            float top = kNegInf;
#pragma unroll
            for (int n = 0; n < kHold; ++n) {
                float x[kVec];
                widen_vec<ZF>(v[n], x);
#pragma unroll
                for (int i = 0; i < kVec; ++i)
                    top = fmaxf(top, x[i]);
            }
            const float ref = finite_top(top);
            float sum = 0.0f;
#pragma unroll
            for (int n = 0; n < kHold; ++n) {
                float x[kVec];
                widen_vec<ZF>(v[n], x);
#pragma unroll
                for (int i = 0; i < kVec; ++i)
                    sum = sum + __builtin_amdgcn_exp2f((x[i] - ref) * c);
            }
            mine = NV == kNoVectors ? join(mine, TopSum{top, sum}, c) : TopSum{top, sum};
        }
        if (rest + tid < s.vocab)
            mine = join(mine, TopSum{last, __builtin_amdgcn_exp2f((last - finite_top(last)) * c)}, c);
        // the teacher's entries: an absent one is -infinity, one past the vocabulary NaN
        float entry[kTeacher], of_logit[kTeacher], old[kTeacher];
        int64_t place[kTeacher];
        TopSum theirs{kNegInf, 0.0f};
#pragma unroll
        for (int n = 0; n < kTeacher; ++n) {
            const int j = tid + n * BLOCK;
            entry[n] = kNegInf;
            of_logit[n] = old[n] = 0.0f;
            place[n] = -1;
            if (j < s.k) {
                place[n] = distill_index(s, t, j);
                if (place[n] >= 0)
                    entry[n] = load_gate(s.teacher, s.tfmt, t * s.ts + j);
                if (place[n] >= s.vocab) {
                    place[n] = -1;
                    entry[n] = __builtin_nanf("");
                }
                if (place[n] >= 0) {
                    of_logit[n] = load_elem<ZF>(row, place[n]);
                    if constexpr (GRAD && ACC)
                        old[n] = load_elem<ZF>(out, place[n]);
                }
                if (!(entry[n] == kNegInf))
                    theirs = join(theirs, TopSum{entry[n], __builtin_amdgcn_exp2f((entry[n] - entry[n]) * c)}, c);
                at[j] = static_cast<int32_t>(place[n]);
            }
        }
        mine = wave_join(mine, c);
        theirs = wave_join(theirs, c);
        if (lane == 0) {
            of_row[wave] = mine;
            of_teacher[wave] = theirs;
        }
        __syncthreads();
        mine = of_row[0];
        theirs = of_teacher[0];
        for (int w = 1; w < kWaves; ++w) {
            mine = join(mine, of_row[w], c);
            theirs = join(theirs, of_teacher[w], c);
        }
        const float log_sum = __builtin_amdgcn_logf(mine.sum), log_theirs = __builtin_amdgcn_logf(theirs.sum);
        // 1, or NaN where the teacher's entries hold a NaN or +infinity
        const float fine = theirs.sum / theirs.sum;
        float loss = 0.0f;
#pragma unroll
        for (int n = 0; n < kTeacher; ++n) {
            const int j = tid + n * BLOCK;
            if (j < s.k) {
                const float q = entry[n] == kNegInf
                                    ? 0.0f
                                    : __builtin_amdgcn_exp2f((entry[n] - theirs.top) * c - log_theirs);
                share[j] = q;
                // in natural logarithms: a difference near the type's range does not fit times log2(e)
                if (q != 0.0f && place[n] >= 0)
                    loss = loss + q * (((entry[n] - theirs.top) * s.per_tau - log_theirs * kLn2) -
                                       ((of_logit[n] - mine.top) * s.per_tau - log_sum * kLn2));
            }
        }
#pragma unroll
        for (int off = 1; off < 64; off <<= 1)
            loss += __shfl_xor(loss, off);
        if (lane == 0)
            part[wave] = loss;
        if constexpr (GRAD) {
            const float by = factor * fine;
            for (int64_t i0 = tid; i0 < vecs; i0 += static_cast<int64_t>(kHold) * BLOCK) {
#pragma unroll
                for (int n = 0; n < kHold; ++n) {
                    const int64_t i = i0 + n * BLOCK;
                    if (i < vecs) {
                        if constexpr (NV == kNoVectors)
                            v[n] = in[i];
                        float x[kVec], o[kVec] = {};
                        widen_vec<ZF>(v[n], x);
                        if constexpr (ACC)
                            widen_vec<ZF>(reinterpret_cast<const u32x4_any*>(out)[i], o);
#pragma unroll
                        for (int m = 0; m < kVec; ++m)
                            x[m] = o[m] + by * __builtin_amdgcn_exp2f((x[m] - mine.top) * c - log_sum);
                        reinterpret_cast<u32x4_any*>(out)[i] = narrow_vec<ZF>(x);
                    }
                }
            }
            if (rest + tid < s.vocab) {
                const float was = ACC ? load_elem<ZF>(out, rest + tid) : 0.0f;
                store_elem<ZF>(out, rest + tid,
                               was + by * __builtin_amdgcn_exp2f((last - mine.top) * c - log_sum));
            }
        }
        __syncthreads();
        if (tid == 0) {
            for (int w = 1; w < kWaves; ++w)
                loss += part[w];
            s.token_loss[t] = s.tau * s.tau * loss * fine;
        }
        if constexpr (GRAD) {
            // where the teacher has entries: written again with their shares, by the first entry of each place
            const float by = factor * fine;
#pragma unroll
            for (int n = 0; n < kTeacher; ++n) {
                const int j = tid + n * BLOCK;
                if (j < s.k && place[n] >= 0) {
                    float q = 0.0f;
                    bool first = true;
                    for (int i = 0; i < s.k; ++i)
                        if (at[i] == static_cast<int32_t>(place[n])) {
                            first = first && i >= j;
                            q = q + share[i];
                        }
                    if (first) {
                        const float p = __builtin_amdgcn_exp2f((of_logit[n] - mine.top) * c - log_sum);
                        store_elem<ZF>(out, place[n], old[n] + by * (p - q));
                    }
                }
            }
        }
        __syncthreads();                                       // the next row's entries
    }
}

// ---- host side ----

constexpr int64_t kDistillMaxVocab = int64_t(1) << 30;

uint64_t distill_ws_bytes(int64_t tokens) { return 8 + static_cast<uint64_t>(tokens); }

bool distill_tokens_ok(int64_t tokens) { return tokens >= 0 && tokens <= kBalMaxTokens; }

template <int ZF, int BLOCK, int NV>
void launch_distill2(unsigned b, hipStream_t st, const Distill& s, bool accumulate)
{
    if (s.grad == nullptr) distill_kernel<ZF, BLOCK, NV, false, false><<<b, BLOCK, 0, st>>>(s);
    else if (accumulate)   distill_kernel<ZF, BLOCK, NV, true, true><<<b, BLOCK, 0, st>>>(s);
    else                   distill_kernel<ZF, BLOCK, NV, true, false><<<b, BLOCK, 0, st>>>(s);
}

template <int ZF>
void launch_distill(hipStream_t st, const Distill& s, bool accumulate)
{
    const int64_t vecs = s.vocab / (ZF == kF32 ? 4 : 8);
    const unsigned b = grid_blocks(s.tokens, 1024);
    if (vecs <= 256)        launch_distill2<ZF, 256, 1>(b, st, s, accumulate);
    else if (vecs <= 1024)  launch_distill2<ZF, 256, 4>(b, st, s, accumulate);
    else if (vecs <= 4096)  launch_distill2<ZF, 512, 8>(b, st, s, accumulate);
    else if (vecs <= 8192)  launch_distill2<ZF, 1024, 8>(b, st, s, accumulate);
    else if (vecs <= 16384) launch_distill2<ZF, 1024, 16>(b, st, s, accumulate);
    else                    launch_distill2<ZF, 1024, kNoVectors>(b, st, s, accumulate);
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
    const Distill s{static_cast<const unsigned char*>(logits), tokens, vocab, stride, teacher, index, ts, is, k, fmt_of(tdt),
                    index_bytes == 8, mask, static_cast<float>(1.44269504088896340736 / static_cast<double>(temperature)),
                    temperature, 1.0f / temperature, coef, token_loss, static_cast<unsigned char*>(grad), gs, static_cast<int32_t*>(ws),
                    static_cast<uint8_t*>(ws) + 8, st};
    if (tokens > 0) {
        const unsigned b = grid_blocks((tokens + kUsedBlock / 64 - 1) / (kUsedBlock / 64), kUsedBlock);
        if (dt == DS_FP16)      distill_used_kernel<kF16><<<b, kUsedBlock, 0, stream>>>(s);
        else if (dt == DS_BF16) distill_used_kernel<kBF16><<<b, kUsedBlock, 0, stream>>>(s);
        else                    distill_used_kernel<kF32><<<b, kUsedBlock, 0, stream>>>(s);
        if (launched() != DS_OK)
            return DS_ERR_HIP;
        if (dt == DS_FP16)      launch_distill<kF16>(stream, s, accumulate);
        else if (dt == DS_BF16) launch_distill<kBF16>(stream, s, accumulate);
        else                    launch_distill<kF32>(stream, s, accumulate);
        if (launched() != DS_OK)
            return DS_ERR_HIP;
    }
    rows_mean_kernel<<<1, kMeanBlock, 0, stream>>>(token_loss, tokens, s.count, coef, loss, used, 1);
    return launched();
}
