// balance.h -- a mixture-of-experts router's balance loss, counts per expert,
// and the gradient.  Included by dszero.hip inside its namespace.
//
// A token's row is held by G lanes of a wave, 64 / G tokens per wave at a
// time.  Lane g holds the experts 4 (c G + g) + j, j = 0..3, for its chunks
// c = 0 .. V/4 - 1, in registers: loads are vectors of four, the softmax's
// maximum and sum and the k largest are reductions over G lanes, and since a
// lane meets the same experts in every row, the counts and the probability
// sums stay in its registers until the block has done all its rows.
//
// 131072 x 256 in bf16, the 8 largest: forward 40.6 us, bound by vector
// instructions (95 % of the busy cycles; about a third of them keep and merge the
// lists of the largest), the sums of its partial rows 9.7 us, bound by the
// latency of reading them, gradient 29.6 us (134 MB): neither memory (4.5 TB/s,
// two thirds of a copy's rate) nor the vector units (77 % of the busy cycles)
// bound it alone, since a wave loads its next row when it has done with one.
// Loads that do not wait for the mask, or 512 blocks instead of 1024, made the
// forward kernel 44 and 45 us.

constexpr int kBalBlock = 256;
constexpr int kBalMaxBlocks = 1024;        // rows of partial sums: four blocks per CU
constexpr int kBalFinishBlock = 1024, kBalFinishCols = 16;   // finishing kernel: lanes, experts per block
// Up to so many blocks (and 64 experts) the last block of the forward kernel
// ends the call, instead of a second kernel.  That saves a launch, which is what
// a call from a program costs, and takes the GPU longer, a ticket and a fence
// for each block.  Loss and gradient of 64 experts, called one after another,
// with the meeting and with the second kernel: 32 blocks 11.4 and 14.6 us, 64
// 12.4 and 14.6, 128 14.1 and 14.5, 160 15.4 and 14.5, 256 18.2 and 14.7 (8
// experts: 128 12.8 and 14.6, 192 14.6 and 14.6, 256 16.6 and 14.6).  Inside a
// graph, where launches are cheap, the second kernel is ahead from 32 blocks on
// (the loss alone at 128 blocks: 10.1 and 7.0).
constexpr int64_t kBalMeet = 128;
// A lane sums the probabilities of so many turns in fp32, the block then in
// fp64: however many tokens there are, a partial sum has some 80 roundings (one
// fp32 sum over all turns is off by 1e-4 of itself at 2^28 tokens).
constexpr int kBalTurns = 64;
constexpr int64_t kBalGradBlocks = 2048;   // gradient: eight blocks per CU
constexpr int64_t kBalMaxTokens = int64_t(1) << 30;
static_assert(DS_MAX_EXPERTS == 512 && DS_MAX_EXPERT_CHOICES == 16, "the instances below");

struct BalShape {
    int64_t tokens, stride;                // rows, elements from row to row
    int32_t experts, k, vec;               // vec: rows allow vectors of four
};

// Workspace: parts of the loss (fp64), the ticket, counts, probability sums
// and used rows per block.
struct BalWork {
    double* loss;
    uint32_t* ticket;
    int32_t *used, *count;
    float* prob;
};

constexpr float kNegInf = -__builtin_huge_valf();

// The lane's V logits of one row (a row that is off, and absent experts:
// -infinity).  Either kind of access is one run of loads, converted once they
// are all on their way.
template <int GF, int G, int V>
__device__ __forceinline__ void bal_load(const void* row, const BalShape& s, int g, bool on, float (&z)[V])
{
    if (s.vec) {
        if constexpr (GF == kF32) {
            f32x4 x[V / 4];
#pragma unroll
            for (int c = 0; c < V / 4; ++c) {
                x[c] = f32x4{kNegInf, kNegInf, kNegInf, kNegInf};
                if (on && 4 * (c * G + g) < s.experts)
                    x[c] = static_cast<const f32x4*>(row)[c * G + g];
            }
#pragma unroll
            for (int v = 0; v < V; ++v)
                z[v] = x[v / 4][v % 4];
        } else {
            u32x2 x[V / 4];
#pragma unroll
            for (int c = 0; c < V / 4; ++c) {
                constexpr uint32_t kNone = GF == kBF16 ? 0xFF80FF80u : 0xFC00FC00u;
                x[c] = u32x2{kNone, kNone};
                if (on && 4 * (c * G + g) < s.experts)
                    x[c] = static_cast<const u32x2*>(row)[c * G + g];
            }
#pragma unroll
            for (int c = 0; c < V / 4; ++c) {
                const f32x4 y = widen4<GF>(x[c]);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    z[4 * c + j] = y[j];
            }
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = 4 * ((v / 4) * G + g) + v % 4;
            z[v] = kNegInf;
            if (on && e < s.experts)
                z[v] = load_grad1<GF>(row, e);
        }
    }
}

// z becomes exp(z - max); returns 1 / sum.  The exponential is the hardware's, of
// 2, of z - max times log2 e: off by some 2 units and 2 |z - max| 2^-24 of itself,
// as the tests count it (the accurate one: 131072 x 256 with its gradient 91.6 us,
// 78.2 with this).  `top` is the row's maximum (NaN
// left out); a NaN or +infinity in the row makes the sum, so 1 / sum, NaN.
// A row that is not used passes top 0 and comes back as zeros.
template <int G, int V>
__device__ __forceinline__ float bal_softmax(float (&z)[V], float top)
{
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        z[v] = __expf(z[v] - top);
        sum = sum + z[v];
    }
    return 1.0f / row_sum<G>(sum);
}

template <int G, int V>
__device__ __forceinline__ float bal_top(const float (&z)[V])
{
    float top = z[0];
#pragma unroll
    for (int v = 1; v < V; ++v)
        top = fmaxf(top, z[v]);
    return row_max<G>(top);
}

// Whether the row counts as used: some logit is not -infinity (a NaN is not).
template <int G, int V>
__device__ __forceinline__ bool bal_used(const float (&z)[V], float top)
{
    uint32_t any = 0u;
#pragma unroll
    for (int v = 0; v < V; ++v)
        any |= z[v] != kNegInf ? 1u : 0u;
    return top > kNegInf || row_sum_int<G>(any) != 0;
}

// The KK largest of two lanes' falling lists: rising then falling, and sorted
// if SORT.
template <int OFF, int KK, bool SORT>
__device__ __forceinline__ void bal_merge(float (&best)[KK])
{
    float other[KK];
#pragma unroll
    for (int i = 0; i < KK; ++i)
        other[i] = row_other<OFF>(best[i]);
#pragma unroll
    for (int i = 0; i < KK; ++i)
        best[i] = fmaxf(best[i], other[KK - 1 - i]);
    if constexpr (SORT) {
#pragma unroll
        for (int d = KK / 2; d > 0; d >>= 1)
#pragma unroll
            for (int i = 0; i < KK; ++i)
                if ((i & d) == 0) {
                    const float hi = fmaxf(best[i], best[i + d]), lo = fminf(best[i], best[i + d]);
                    best[i] = hi;
                    best[i + d] = lo;
                }
    }
}

// The k-th largest of the row, the same in each of its G lanes.  Every lane
// keeps the KK largest of its own values in falling order (insertion, one
// median per place), the lists of lanes 1, 2, 4 .. apart are merged, and the
// smallest of the last merge is it: the row's first lane starts with KK - k
// infinities, so that the KK-th largest is the k-th of the row.
template <int G, int V, int KK>
__device__ __forceinline__ float bal_cut(const float (&z)[V], int k, int g)
{
    float best[KK];
#pragma unroll
    for (int i = 0; i < KK; ++i)
        best[i] = g == 0 && i < KK - k ? -kNegInf : kNegInf;
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int i = KK - 1; i > 0; --i)
            best[i] = __builtin_amdgcn_fmed3f(best[i - 1], best[i], z[v]);
        best[0] = fmaxf(best[0], z[v]);
    }
    bal_merge<1, KK, true>(best);
    bal_merge<2, KK, true>(best);
    bal_merge<4, KK, (G > 8)>(best);
    if constexpr (G > 8)
        bal_merge<8, KK, (G > 16)>(best);
    if constexpr (G > 16)
        bal_merge<16, KK, false>(best);
    float cut = best[0];
#pragma unroll
    for (int i = 1; i < KK; ++i)
        cut = fminf(cut, best[i]);
    return cut;
}

// What the forward pass leaves, and what it is scaled by.
struct BalOut {
    int32_t* counts;
    float* mean_prob;
    float* loss;
    int32_t* used;
    float coef;
};

// Expert e of E: its count n and probability sum p become outputs; returns its
// part of the loss, f_e mean_prob_e.
__device__ __forceinline__ double bal_expert(const BalOut& o, int32_t k, int rows, int e, int n, double p)
{
    const double some = rows > 0 ? static_cast<double>(rows) : 1.0;
    const double mean = p / some;
    o.counts[e] = n;
    o.mean_prob[e] = static_cast<float>(mean);
    return mean * (static_cast<double>(n) / (some * static_cast<double>(k)));
}

__device__ __forceinline__ void bal_end(const BalOut& o, int32_t experts, int rows, double sum)
{
    *o.loss = static_cast<float>(static_cast<double>(o.coef) * static_cast<double>(experts) * sum);
    *o.used = rows;
}

// Lanes whose sums share a row of the block's shared arrays.
constexpr int bal_span_lanes(int G) { return G > 16 ? G : 16; }

// The lanes' sums x by expert into the shared array: lanes of the same experts
// in a row of 16 by a rotation, the others a row each.
template <int G, int V, typename T>
__device__ __forceinline__ void bal_rows(T (&lds)[kBalBlock / bal_span_lanes(G)][G * V], T (&x)[V])
{
    const int lane = static_cast<int>(__lane_id()), g = lane % G;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if constexpr (G == 8)
            x[v] = x[v] + row_half(x[v]);
        if (G > 8 || lane % 16 < 8)
            lds[threadIdx.x / bal_span_lanes(G)][4 * ((v / 4) * G + g) + v % 4] = x[v];
    }
}

// Expert e over the shared array's rows, in their order.
template <int G, int V, typename T>
__device__ __forceinline__ T bal_row_sum(const T (&lds)[kBalBlock / bal_span_lanes(G)][G * V], int e)
{
    T x = 0;
#pragma unroll
    for (int i = 0; i < kBalBlock / bal_span_lanes(G); ++i)
        x = x + lds[i][e];
    return x;
}

// Forward: counts and probability sums of this block's rows into row
// blockIdx.x of the partial arrays, used rows into used[blockIdx.x].  A grid
// of one block ends the call itself, and of up to kBalMeet the last block.
template <int GF, int G, int V, int KK>
__global__ __launch_bounds__(kBalBlock) void balance_kernel(const void* __restrict__ logits, BalShape s,
                                                            const uint8_t* __restrict__ mask, BalWork w, BalOut o)
{
    constexpr int kRows = 64 / G;          // rows of a wave
    constexpr int kWaves = kBalBlock / 64;
    __shared__ int32_t lds_count[kBalBlock / bal_span_lanes(G)][G * V];
    __shared__ float lds_prob[kBalBlock / bal_span_lanes(G)][G * V];
    __shared__ double lds_sum[G * V];
    __shared__ int32_t lds_used[kWaves];
    __shared__ double lds_loss[2 * kWaves];
    const int lane = static_cast<int>(__lane_id()), wave = threadIdx.x / 64, g = lane % G;
    int cnt[V];
    float prob[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        cnt[v] = 0;
        prob[v] = 0.0f;
    }
    int used = 0;
    constexpr int es = GF == kF32 ? 4 : 2;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWaves * kRows;
    int turns = 0;
    bool folded = false;
    for (int64_t b0 = static_cast<int64_t>(blockIdx.x) * kWaves * kRows; b0 < s.tokens; b0 += step) {
        if (turns == kBalTurns) {          // the same for all of the block
            bal_rows<G, V>(lds_prob, prob);
            __syncthreads();
            for (int e = threadIdx.x; e < s.experts; e += kBalBlock)
                lds_sum[e] = (folded ? lds_sum[e] : 0.0) + static_cast<double>(bal_row_sum<G, V>(lds_prob, e));
            __syncthreads();
#pragma unroll
            for (int v = 0; v < V; ++v)
                prob[v] = 0.0f;
            turns = 0;
            folded = true;
        }
        ++turns;
        const int64_t t = b0 + wave * kRows + lane / G;
        bool on = t < s.tokens;
        if (on && mask != nullptr)
            on = mask[t] != 0;
        float z[V];
        bal_load<GF, G, V>(static_cast<const unsigned char*>(logits) + t * s.stride * es, s, g, on, z);
        float top = bal_top<G, V>(z);
        if (__ballot(on && !(top > kNegInf)) != 0ull)
            on = on && bal_used<G, V>(z, top);
        float cut = bal_cut<G, V, KK>(z, s.k, g);
        cut = fmaxf(cut, -3.402823466e+38f);   // -infinity is never chosen
        uint32_t chosen = 0u;              // bit V - 1 - v: the lane's value v
#pragma unroll
        for (int v = 0; v < V; ++v)
            chosen = chosen + chosen + (z[v] >= cut ? 1u : 0u);
        // more than k of them: of those equal to the cut the highest indices go
        int over = on ? row_sum_int<G>(__popc(chosen)) - s.k : 0;
        if (__ballot(over > 0) != 0ull) {
            uint32_t equal = 0u;
#pragma unroll
            for (int v = 0; v < V; ++v)
                equal = equal + equal + (z[v] == cut ? 1u : 0u);
            if (__ballot(over > 3) == 0ull) {
                while (__ballot(over > 0) != 0ull) {   // at most three turns
                    const int v = V - __ffs(static_cast<int>(equal));
                    const int e = equal != 0u ? 4 * ((v / 4) * G + g) + v % 4 : -1;
                    if (over > 0 && e == row_max_int<G>(e)) {
                        chosen &= ~(equal & -equal);
                        equal &= equal - 1u;
                    }
                    over -= 1;
                }
            } else {
                // by ranks: chunk by chunk, the number of equal ones before a lane's own
                int left = row_sum_int<G>(__popc(equal)) - (over > 0 ? over : 0);
#pragma unroll
                for (int c = 0; c < V / 4; ++c) {
                    const uint32_t mine = (equal >> (V - 4 - 4 * c)) & 15u;
                    int before = __popc(mine);         // inclusive prefix over the row's lanes
#pragma unroll
                    for (int off = 1; off < G; off <<= 1) {
                        const int x = __shfl_up(before, off, G);
                        before += g >= off ? x : 0;
                    }
                    const int all = __shfl(before, G - 1, G);
                    int rank = before - __popc(mine);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t bit = 8u >> j;
                        if ((mine & bit) != 0u && rank >= left)
                            chosen &= ~(bit << (V - 4 - 4 * c));
                        rank += (mine & bit) != 0u ? 1 : 0;
                    }
                    left -= all;
                }
            }
        }
        float inv = bal_softmax<G, V>(z, on ? top : 0.0f);
        if (!on)
            inv = 0.0f;
        if (!on || inv != inv)             // a row with a NaN or +infinity counts nothing
            chosen = 0u;
        used += on ? 1 : 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            prob[v] = __builtin_fmaf(z[v], inv, prob[v]);
            cnt[v] += static_cast<int>((chosen >> (V - 1 - v)) & 1u);
        }
    }
    bal_rows<G, V>(lds_count, cnt);
    bal_rows<G, V>(lds_prob, prob);
#pragma unroll
    for (int off = G; off < 64; off <<= 1)
        used += __shfl_xor(used, off);
    if (lane == 0)
        lds_used[wave] = used;
    __syncthreads();
    int rows = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i)
        rows += lds_used[i];
    double part = 0.0;
    for (int e = threadIdx.x; e < s.experts; e += kBalBlock) {
        const int n = bal_row_sum<G, V>(lds_count, e);
        const double p = (folded ? lds_sum[e] : 0.0) + static_cast<double>(bal_row_sum<G, V>(lds_prob, e));
        if (gridDim.x > 1) {
            w.count[blockIdx.x * s.experts + e] = n;
            w.prob[blockIdx.x * s.experts + e] = static_cast<float>(p);
        } else {
            part = part + bal_expert(o, s.k, rows, e, n, p);
        }
    }
    if (gridDim.x == 1) {
        part = block_sum_fixed<kBalBlock>(part, lds_loss, 0);
        if (threadIdx.x == 0)
            bal_end(o, s.experts, rows, part);
        return;
    }
    if (threadIdx.x == 0)
        w.used[blockIdx.x] = rows;
    if constexpr (G * V <= 64) {
        if (gridDim.x > kBalMeet)
            return;
        // the last block to come here ends the call
        __syncthreads();
        if (threadIdx.x == 0) {
            __threadfence();
            lds_used[0] = atomicAdd(w.ticket, 1u) == gridDim.x - 1u ? 1 : 0;
        }
        __syncthreads();
        if (lds_used[0] == 0)
            return;
        __threadfence();
        const int parts = static_cast<int>(gridDim.x), col = lane, e = col < s.experts ? col : 0;
        int n = 0;
        double p = 0.0;
        for (int i0 = wave; i0 < parts; i0 += 16 * kWaves) {
            int32_t c[16];
            float q[16];
#pragma unroll
            for (int u = 0; u < 16; ++u) {
                const int i = i0 + u * kWaves < parts ? i0 + u * kWaves : 0;
                c[u] = w.count[i * s.experts + e];
                q[u] = w.prob[i * s.experts + e];
            }
#pragma unroll
            for (int u = 0; u < 16; ++u) {
                const bool in = i0 + u * kWaves < parts;
                n += in ? c[u] : 0;
                p = p + static_cast<double>(in ? q[u] : 0.0f);
            }
        }
        rows = 0;
        for (int i = threadIdx.x; i < parts; i += kBalBlock)
            rows += w.used[i];
#pragma unroll
        for (int off = 1; off < 64; off <<= 1)
            rows += __shfl_xor(rows, off);
        __shared__ double sum[kWaves][64];
        __shared__ int32_t count[kWaves][64], some[kWaves];
        sum[wave][col] = p;
        count[wave][col] = n;
        if (lane == 0)
            some[wave] = rows;
        __syncthreads();
        if (wave != 0)
            return;
        rows = 0;
        n = 0;
        p = 0.0;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
            rows += some[i];
            n += count[i][col];
            p = p + sum[i][col];
        }
        part = col < s.experts ? bal_expert(o, s.k, rows, col, n, p) : 0.0;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1)
            part = part + __shfl_xor(part, off);
        if (lane == 0) {
            bal_end(o, s.experts, rows, part);
            *w.ticket = 0u;
        }
    }
}

// Sums the partial rows: COLS experts per block, 1024 / COLS groups of rows,
// fp64.  The block that finishes last adds the blocks' parts of the loss in
// order; one block of 64 columns, without that meeting, does up to 64 experts
// (128 partial rows of 64: 5.8 us by four blocks of 16).
template <int COLS>
__global__ __launch_bounds__(kBalFinishBlock) void balance_finish_kernel(int32_t parts, int32_t experts, int32_t k,
                                                                         BalWork w, BalOut o)
{
    constexpr int kGroups = kBalFinishBlock / COLS, kWaves = kBalFinishBlock / 64;
    constexpr int kDeep = 10;              // rows on their way a lane: 131072 x 256 takes the same with 4, 6 or 16 (1 %)
    __shared__ double lds_prob[kWaves][COLS];
    __shared__ int32_t lds_count[kWaves][COLS];
    __shared__ int32_t lds_used[kWaves];
    const int col = threadIdx.x % COLS, group = threadIdx.x / COLS;
    const int lane = static_cast<int>(__lane_id()), wave = threadIdx.x / 64;
    const int e = blockIdx.x * COLS + col, column = e < experts ? e : 0;
    int rows = 0;
    for (int i = threadIdx.x; i < parts; i += kBalFinishBlock)
        rows += w.used[i];
    int n = 0;
    double p = 0.0;
    for (int i0 = group; i0 < parts; i0 += kGroups * kDeep) {
        int32_t c[kDeep];
        float q[kDeep];
#pragma unroll
        for (int u = 0; u < kDeep; ++u) {
            // past the end: the first row again, left out below (no branch between the loads)
            const int i = i0 + u * kGroups < parts ? i0 + u * kGroups : 0;
            c[u] = w.count[i * experts + column];
            q[u] = w.prob[i * experts + column];
        }
#pragma unroll
        for (int u = 0; u < kDeep; ++u) {
            const bool in = i0 + u * kGroups < parts;
            n += in ? c[u] : 0;
            p = p + static_cast<double>(in ? q[u] : 0.0f);
        }
    }
#pragma unroll
    for (int off = COLS; off < 64; off <<= 1) {
        n += __shfl_xor(n, off);
        p = p + __shfl_xor(p, off);
    }
#pragma unroll
    for (int off = 1; off < 64; off <<= 1)
        rows += __shfl_xor(rows, off);
    if (lane < COLS) {
        lds_count[wave][col] = n;
        lds_prob[wave][col] = p;
    }
    if (lane == 0)
        lds_used[wave] = rows;
    __syncthreads();
    if (wave != 0)
        return;
    rows = 0;
    n = 0;
    p = 0.0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
        rows += lds_used[i];
        n += lds_count[i][col];
        p = p + lds_prob[i][col];
    }
    double part = lane < COLS && e < experts ? bal_expert(o, k, rows, e, n, p) : 0.0;
#pragma unroll
    for (int off = 1; off < COLS; off <<= 1)
        part = part + __shfl_xor(part, off);
    if (gridDim.x > 1) {
        uint32_t before = 0u;
        if (lane == 0) {
            w.loss[blockIdx.x] = part;
            __threadfence();
            before = atomicAdd(w.ticket, 1u);
        }
        if (__builtin_amdgcn_readfirstlane(before) != gridDim.x - 1u)
            return;
        if (lane == 0)
            *w.ticket = 0u;
        __threadfence();
        part = lane < static_cast<int>(gridDim.x) ? __builtin_nontemporal_load(w.loss + lane) : 0.0;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1)
            part = part + __shfl_xor(part, off);
    }
    if (lane == 0)
        bal_end(o, experts, rows, part);
}

// The lane's V values into (or, with ACC, added to) one row.
template <int GF, int G, int V, bool ACC>
__device__ __forceinline__ void bal_store(void* row, int experts, int32_t vec, int g, const float (&d)[V])
{
    if (vec) {
#pragma unroll
        for (int c = 0; c < V / 4; ++c) {
            if (4 * (c * G + g) < experts) {
                f32x4 x = {d[4 * c], d[4 * c + 1], d[4 * c + 2], d[4 * c + 3]};
                if constexpr (GF == kF32) {
                    f32x4* p = static_cast<f32x4*>(row) + c * G + g;
                    *p = ACC ? *p + x : x;
                } else {
                    u32x2* p = static_cast<u32x2*>(row) + c * G + g;
                    *p = narrow4<GF>(ACC ? widen4<GF>(*p) + x : x);
                }
            }
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = 4 * ((v / 4) * G + g) + v % 4;
            if (e < experts) {
                if constexpr (GF == kF32) {
                    float* p = static_cast<float*>(row) + e;
                    *p = ACC ? *p + d[v] : d[v];
                } else {
                    uint16_t* p = static_cast<uint16_t*>(row) + e;
                    *p = static_cast<uint16_t>(enc1<GF>(ACC ? dec1<GF>(*p) + d[v] : d[v]));
                }
            }
        }
    }
}

// Gradient: d_j = S coef E / T' p_j (f_j - sum_e f_e p_e).  Since the p of a
// row add up to 1, f may be taken off by a constant: f_e - 1/E-th of their
// sum, formed from the counts exactly, so that the difference loses nothing
// where the counts are nearly even.
template <int GF, int G, int V, bool ACC>
__global__ __launch_bounds__(kBalBlock) void balance_grad_kernel(const ds_scaler* __restrict__ st,
                                                                 const void* __restrict__ logits, BalShape s,
                                                                 const uint8_t* __restrict__ mask, float coef,
                                                                 const int32_t* __restrict__ counts,
                                                                 const int32_t* __restrict__ used,
                                                                 void* __restrict__ dlogits, int64_t dstride,
                                                                 int32_t dvec)
{
    constexpr int kRows = 64 / G, kWaves = kBalBlock / 64;
    constexpr int es = GF == kF32 ? 4 : 2;
    const int lane = static_cast<int>(__lane_id()), wave = threadIdx.x / 64, g = lane % G;
    const int rows = *used;
    const double scale = st != nullptr ? static_cast<double>(st->scale) : 1.0;
    const double some = rows > 0 ? static_cast<double>(rows) : 1.0;
    const float factor =
        rows > 0 ? static_cast<float>(scale * static_cast<double>(coef) * static_cast<double>(s.experts) / some) : 0.0f;
    // f less its mean: (E c_e - sum c) / (E k T'), the difference exact
    float f[V];
    double total = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = 4 * ((v / 4) * G + g) + v % 4;
        f[v] = __int_as_float(e < s.experts ? counts[e] : 0);
        total = total + static_cast<double>(__float_as_int(f[v]));
    }
#pragma unroll
    for (int off = G / 2; off > 0; off >>= 1)
        total = total + __shfl_xor(total, off);
    const double unit = 1.0 / (static_cast<double>(s.experts) * some * static_cast<double>(s.k));
#pragma unroll
    for (int v = 0; v < V; ++v)
        f[v] = static_cast<float>(
            __builtin_fma(static_cast<double>(__float_as_int(f[v])), static_cast<double>(s.experts), -total) * unit);
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWaves * kRows;
    for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kWaves + wave) * kRows; t0 < s.tokens; t0 += step) {
        const int64_t t = t0 + lane / G;
        const bool in = t < s.tokens;
        bool on = in;
        if (on && mask != nullptr)
            on = mask[t] != 0;
        float z[V];
        bal_load<GF, G, V>(static_cast<const unsigned char*>(logits) + t * s.stride * es, s, g, on, z);
        const float top = bal_top<G, V>(z);
        if (__ballot(on && !(top > kNegInf)) != 0ull)
            on = on && bal_used<G, V>(z, top);
        float inv = bal_softmax<G, V>(z, on ? top : 0.0f);
        if (!on)
            inv = 0.0f;
        float dot = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            z[v] = z[v] * inv;
            dot = __builtin_fmaf(z[v], f[v], dot);
        }
        dot = row_sum<G>(dot);
        const float by = on ? factor : 0.0f;       // the factor itself may be infinite
#pragma unroll
        for (int v = 0; v < V; ++v)
            z[v] = by * (z[v] * (f[v] - dot));
        if (ACC ? on : in)
            bal_store<GF, G, V, ACC>(static_cast<unsigned char*>(dlogits) + t * dstride * es, s.experts, dvec, g, z);
    }
}

// ---- host side ----

// Blocks of the forward pass: one per 4 waves' rows, at most kBalMaxBlocks.
int bal_lanes(int32_t experts) { return experts <= 128 ? 8 : experts <= 256 ? 16 : 32; }

int64_t bal_blocks(int64_t tokens, int32_t experts)
{
    const int64_t rows = static_cast<int64_t>(kBalBlock) / bal_lanes(experts);
    const int64_t b = (tokens + rows - 1) / rows;
    return b < 1 ? 1 : (b > kBalMaxBlocks ? kBalMaxBlocks : b);
}

constexpr int kBalLossParts = DS_MAX_EXPERTS / kBalFinishCols;
static_assert(kBalLossParts <= 64, "one wave adds them");

uint64_t bal_ws_bytes(int64_t blocks, int32_t experts)
{
    return 8 * kBalLossParts + 8 + 4 * static_cast<uint64_t>(blocks) * (1 + 2 * static_cast<uint64_t>(experts));
}

BalWork bal_work(void* ws, int64_t blocks, int32_t experts)
{
    BalWork w;
    w.loss = static_cast<double*>(ws);
    w.ticket = reinterpret_cast<uint32_t*>(w.loss + kBalLossParts);
    w.used = reinterpret_cast<int32_t*>(w.ticket + 2);
    w.count = w.used + blocks;
    w.prob = reinterpret_cast<float*>(w.count + blocks * experts);
    return w;
}

bool bal_sizes_ok(int64_t tokens, int32_t experts)
{
    return tokens >= 0 && tokens <= kBalMaxTokens && experts >= 1 && experts <= DS_MAX_EXPERTS;
}

// Bytes from the first to the last element of the rows.
uint64_t bal_span(int64_t tokens, int32_t experts, int64_t stride, uint64_t es)
{
    return tokens == 0 ? 0 : es * (static_cast<uint64_t>(tokens - 1) * static_cast<uint64_t>(stride) + experts);
}

bool bal_vec(const void* p, int64_t stride, int32_t experts, uint64_t es)
{
    return aligned(p, 4 * es) && stride % 4 == 0 && experts % 4 == 0;
}

ds_status bal_check(const void* logits, ds_dtype dt, int64_t tokens, int32_t experts, int64_t stride, int32_t k,
                    float coef)
{
    if (!bal_sizes_ok(tokens, experts) || k < 1 || k > experts || k > DS_MAX_EXPERT_CHOICES || stride < experts ||
        stride > kMaxElems || (tokens > 0 && stride > kMaxElems / tokens))
        return DS_ERR_SIZE;
    if (!known(dt))
        return DS_ERR_DTYPE;
    if (!finite_ge0(coef))
        return DS_ERR_HPARAM;
    if (tokens > 0 && logits == nullptr)
        return DS_ERR_NULL;
    if (!aligned(logits, esize(dt)))
        return DS_ERR_ALIGN;
    return DS_OK;
}

// Whether any two of the ranges overlap, `reads` first ones aside.
bool bal_alias(const void* const* p, const uint64_t* bytes, int n, int reads)
{
    for (int i = 0; i < n; ++i)
        for (int j = i + 1; j < n; ++j)
            if (j >= reads && overlap(p[i], bytes[i], p[j], bytes[j]))
                return true;
    return false;
}

template <int GF, int G, int V>
void launch_balance3(int64_t blocks, hipStream_t st, const void* z, const BalShape& s, const uint8_t* mask,
                     const BalWork& w, const BalOut& o)
{
    const unsigned b = static_cast<unsigned>(blocks);
    if (s.k <= 2)      balance_kernel<GF, G, V, 2><<<b, kBalBlock, 0, st>>>(z, s, mask, w, o);
    else if (s.k <= 4) balance_kernel<GF, G, V, 4><<<b, kBalBlock, 0, st>>>(z, s, mask, w, o);
    else if (s.k <= 8) balance_kernel<GF, G, V, 8><<<b, kBalBlock, 0, st>>>(z, s, mask, w, o);
    else               balance_kernel<GF, G, V, 16><<<b, kBalBlock, 0, st>>>(z, s, mask, w, o);
}

template <int GF>
void launch_balance2(int64_t blocks, hipStream_t st, const void* z, const BalShape& s, const uint8_t* mask,
                     const BalWork& w, const BalOut& o)
{
    if (s.experts <= 32)       launch_balance3<GF, 8, 4>(blocks, st, z, s, mask, w, o);
    else if (s.experts <= 64)  launch_balance3<GF, 8, 8>(blocks, st, z, s, mask, w, o);
    else if (s.experts <= 128) launch_balance3<GF, 8, 16>(blocks, st, z, s, mask, w, o);
    else if (s.experts <= 256) launch_balance3<GF, 16, 16>(blocks, st, z, s, mask, w, o);
    else                       launch_balance3<GF, 32, 16>(blocks, st, z, s, mask, w, o);
}

ds_status balance_loss(const void* logits, ds_dtype dt, int64_t tokens, int32_t experts, int64_t stride,
                       const uint8_t* mask, int32_t k, float coef, int32_t* counts, float* mean_prob, float* loss,
                       int32_t* used, void* ws, size_t ws_bytes, hipStream_t s)
{
    if (const ds_status rc = bal_check(logits, dt, tokens, experts, stride, k, coef); rc != DS_OK)
        return rc;
    if (counts == nullptr || mean_prob == nullptr || loss == nullptr || used == nullptr || ws == nullptr)
        return DS_ERR_NULL;
    if (!aligned(counts, 4) || !aligned(mean_prob, 4) || !aligned(loss, 4) || !aligned(used, 4) || !aligned(ws, 8))
        return DS_ERR_ALIGN;
    const int64_t blocks = bal_blocks(tokens, experts);
    const uint64_t need = bal_ws_bytes(blocks, experts), ue = static_cast<uint64_t>(experts);
    if (ws_bytes < need)
        return DS_ERR_SIZE;
    const uint64_t es = esize(dt);
    const void* p[7] = {logits, mask, counts, mean_prob, loss, used, ws};
    const uint64_t bytes[7] = {bal_span(tokens, experts, stride, es), static_cast<uint64_t>(tokens), 4 * ue, 4 * ue, 4,
                               4, need};
    if (bal_alias(p, bytes, 7, 2))
        return DS_ERR_ALIAS;
    const BalShape shape{tokens, stride, experts, k, bal_vec(logits, stride, experts, es) ? 1 : 0};
    const BalWork w = bal_work(ws, blocks, experts);
    const BalOut o{counts, mean_prob, loss, used, coef};
    if (dt == DS_FP16)      launch_balance2<kF16>(blocks, s, logits, shape, mask, w, o);
    else if (dt == DS_BF16) launch_balance2<kBF16>(blocks, s, logits, shape, mask, w, o);
    else                    launch_balance2<kF32>(blocks, s, logits, shape, mask, w, o);
    if (launched() != DS_OK)
        return DS_ERR_HIP;
    if (blocks == 1 || (experts <= 64 && blocks <= kBalMeet))
        return DS_OK;
    const int32_t parts = static_cast<int32_t>(blocks);
    if (experts <= 64) {
        balance_finish_kernel<64><<<1, kBalFinishBlock, 0, s>>>(parts, experts, k, w, o);
    } else {
        const unsigned fb = static_cast<unsigned>((experts + kBalFinishCols - 1) / kBalFinishCols);
        balance_finish_kernel<kBalFinishCols><<<fb, kBalFinishBlock, 0, s>>>(parts, experts, k, w, o);
    }
    return launched();
}

template <int GF, bool ACC>
void launch_balance_grad(unsigned b, hipStream_t s, const ds_scaler* st, const void* z, const BalShape& sh,
                         const uint8_t* mask, float coef, const int32_t* counts, const int32_t* used, void* d,
                         int64_t ds, int32_t dv)
{
    if (sh.experts <= 32)       balance_grad_kernel<GF, 8, 4, ACC><<<b, kBalBlock, 0, s>>>(st, z, sh, mask, coef, counts, used, d, ds, dv);
    else if (sh.experts <= 64)  balance_grad_kernel<GF, 8, 8, ACC><<<b, kBalBlock, 0, s>>>(st, z, sh, mask, coef, counts, used, d, ds, dv);
    else if (sh.experts <= 128) balance_grad_kernel<GF, 8, 16, ACC><<<b, kBalBlock, 0, s>>>(st, z, sh, mask, coef, counts, used, d, ds, dv);
    else if (sh.experts <= 256) balance_grad_kernel<GF, 16, 16, ACC><<<b, kBalBlock, 0, s>>>(st, z, sh, mask, coef, counts, used, d, ds, dv);
    else                        balance_grad_kernel<GF, 32, 16, ACC><<<b, kBalBlock, 0, s>>>(st, z, sh, mask, coef, counts, used, d, ds, dv);
}

ds_status balance_grad(const ds_scaler* st, const void* logits, ds_dtype dt, int64_t tokens, int32_t experts,
                       int64_t stride, const uint8_t* mask, int32_t k, float coef, const int32_t* counts,
                       const int32_t* used, void* dlogits, int64_t dstride, bool accumulate, hipStream_t s)
{
    if (const ds_status rc = bal_check(logits, dt, tokens, experts, stride, k, coef); rc != DS_OK)
        return rc;
    if (dstride < experts || dstride > kMaxElems || (tokens > 0 && dstride > kMaxElems / tokens))
        return DS_ERR_SIZE;
    if (counts == nullptr || used == nullptr || (tokens > 0 && dlogits == nullptr))
        return DS_ERR_NULL;
    const uint64_t es = esize(dt);
    if (!aligned(st, 8) || !aligned(counts, 4) || !aligned(used, 4) || !aligned(dlogits, es))
        return DS_ERR_ALIGN;
    const void* p[6] = {logits, mask, counts, used, st, dlogits};
    const uint64_t bytes[6] = {bal_span(tokens, experts, stride, es), static_cast<uint64_t>(tokens),
                               4 * static_cast<uint64_t>(experts), 4, sizeof(ds_scaler),
                               bal_span(tokens, experts, dstride, es)};
    if (bal_alias(p, bytes, 6, 5))
        return DS_ERR_ALIAS;
    if (tokens == 0)
        return DS_OK;
    const BalShape sh{tokens, stride, experts, k, bal_vec(logits, stride, experts, es) ? 1 : 0};
    const int32_t dv = bal_vec(dlogits, dstride, experts, es) ? 1 : 0;
    const int64_t rows = static_cast<int64_t>(kBalBlock) / bal_lanes(experts);
    const int64_t turns = (tokens + rows - 1) / rows;
    const unsigned b = grid_blocks(turns < kBalGradBlocks ? turns : kBalGradBlocks, kBalBlock);
    const int gf = fmt_of(dt);
    if (accumulate) {
        if (gf == kF16)       launch_balance_grad<kF16, true>(b, s, st, logits, sh, mask, coef, counts, used, dlogits, dstride, dv);
        else if (gf == kBF16) launch_balance_grad<kBF16, true>(b, s, st, logits, sh, mask, coef, counts, used, dlogits, dstride, dv);
        else                  launch_balance_grad<kF32, true>(b, s, st, logits, sh, mask, coef, counts, used, dlogits, dstride, dv);
    } else {
        if (gf == kF16)       launch_balance_grad<kF16, false>(b, s, st, logits, sh, mask, coef, counts, used, dlogits, dstride, dv);
        else if (gf == kBF16) launch_balance_grad<kBF16, false>(b, s, st, logits, sh, mask, coef, counts, used, dlogits, dstride, dv);
        else                  launch_balance_grad<kF32, false>(b, s, st, logits, sh, mask, coef, counts, used, dlogits, dstride, dv);
    }
    return launched();
}
