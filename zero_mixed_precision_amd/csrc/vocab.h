// vocab.h -- softmax cross entropy over a large vocabulary from hidden states
// and the head's weight, without keeping the logits, with its gradient.
// Included by dszero.hip inside its namespace.
//
//   z = X W^T,  l_t = lse_t - z_t,y,  dz = S coef / T' (softmax(z) - onehot(y))
//   dX = dz W,  dW = dz^T X
//
// The used rows are packed first (compact, padded with zeros to tiles of 64 k),
// so rows that are left out cost nothing and what they hold reaches nothing.
// The first product goes over the whole vocabulary and leaves a maximum and a
// sum per row and tile, joined per row afterwards.  The gradient goes over
// pieces of the vocabulary: the logits of a piece are formed again and become
// dz in 16 bits at the product's end, then two products take it to dX (summed
// over the pieces in fp32) and to the piece's rows of dW.  8 T V D operations
// instead of the 6 that keeping the logits would take.
//
// dz in 16 bits: each value is off by half a unit of its own, as much as the
// result's own rounding; in fp16 it is held times 2^15, so that probabilities
// down to 2^-29 have all their bits.

constexpr int kVocabTile = 256;            // rows of packed arrays are a multiple of it
constexpr int64_t kVocabMaxTokens = int64_t(1) << 24;
constexpr int64_t kVocabMaxVocab = int64_t(1) << 24;
constexpr int64_t kVocabMaxWidth = 65536;
constexpr int64_t kVocabMaxStride = int64_t(1) << 22;   // of W read in place: offsets in a tile have 32 bits
constexpr uint64_t kVocabPiece = uint64_t(1) << 29;     // bytes of a piece's dz
constexpr int64_t kVocabMinPiece = 2048, kVocabWidePiece = 32768;   // a piece of at least so much, or
constexpr int64_t kVocabWeights = int64_t(1) << 27;     // so many values of W
constexpr int64_t kVocabSmallTokens = 8192;             // up to so many, tiles of 64 x 64
// Tiles of the two gradients that are to be there at once: where there are fewer,
// a tile's sum is split over k and joined afterwards.
constexpr int64_t kVocabBlocks = 512;
constexpr uint64_t kVocabParts = static_cast<uint64_t>(kVocabBlocks) * 128 * 128 * 4;   // bytes of the parts

struct VocabSizes {
    int64_t tokens, vocab, width;
    int64_t tp, dp, vc;                    // padded tokens and width, vocabulary of a piece
    int64_t vmax;                          // the largest piece of any number of tokens
    int64_t tiles;                         // partial sums per row
    int32_t xs, ws;                        // parts of the sums for dX and dW
};

struct VocabWork {
    int32_t *used, *slot, *list, *target;  // [1], [tokens], [tp], [tp]
    uint32_t* ticket;                      // blocks of the join that are done
    float* of_target;                      // [tp] the target's logit
    TopSum* part;                          // [tiles][tp]
    TopSum* row;                           // [tp] maximum, log2 of the sum
    uint16_t* x;                           // [tp][dp]
    uint16_t* w;                           // [vc][dp], where W cannot be read in place
    uint16_t* dz;                          // [tp][vc]
    float* dx;                             // [xs][tokens][dp], where there are several pieces or parts
    float* dw;                             // [ws][vc][dp], where there are several parts
};

// Compact numbers of the used rows (t ascending), by one block.
constexpr int kVocabListBlock = 1024;
template <typename I>
__global__ __launch_bounds__(kVocabListBlock) void vocab_list_kernel(const I* __restrict__ targets,
                                                                const uint8_t* __restrict__ mask, VocabSizes s,
                                                                VocabWork w, float* __restrict__ token_loss)
{
    __shared__ int32_t part[kVocabListBlock / 64];
    const int lane = static_cast<int>(__lane_id()), wave = threadIdx.x / 64;
    int32_t before = 0;
    for (int64_t t0 = 0; t0 < s.tokens; t0 += kVocabListBlock) {
        const int64_t t = t0 + threadIdx.x;
        int64_t y = -1;
        if (t < s.tokens && (mask == nullptr || mask[t] != 0))
            y = targets[t];
        const uint64_t on = __ballot(y >= 0);
        if (lane == 0)
            part[wave] = __popcll(on);
        __syncthreads();
        int32_t at = before + __popcll(on & ((1ull << lane) - 1));
        for (int v = 0; v < kVocabListBlock / 64; ++v) {
            at += v < wave ? part[v] : 0;
            before += part[v];
        }
        if (t < s.tokens) {
            w.slot[t] = y >= 0 ? at : -1;
            if (y >= 0) {
                w.list[at] = static_cast<int32_t>(t);
                w.target[at] = y < s.vocab ? static_cast<int32_t>(y) : -1;
            } else {
                token_loss[t] = 0.0f;
            }
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        *w.used = before;
        *w.ticket = 0;
    }
}

// A row of `width` 16-bit values, padded with zeros to dp, by one wave.
__device__ __forceinline__ void pack_row(const uint16_t* from, int64_t width, uint16_t* to, int64_t dp, int lane)
{
    for (int64_t c = lane; c < dp / 8; c += 64) {
        u32x4 v = {0, 0, 0, 0};
        if (from != nullptr) {
            if (8 * c + 8 <= width) {
                v = *reinterpret_cast<const u32x4_any*>(from + 8 * c);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (8 * c + i < width)
                        v[i / 2] |= static_cast<uint32_t>(from[8 * c + i]) << (16 * (i % 2));
            }
        }
        reinterpret_cast<u32x4*>(to)[c] = v;
    }
}

constexpr int kPackBlock = 256;

// The row of wave-number t: row t of X to its place, or zeros to its gradient;
// behind the last: zero rows up to the next 64.
__device__ __forceinline__ void pack_token(const uint16_t* hidden, int64_t hs, uint16_t* dhidden, int64_t dhs,
                                           const VocabSizes& s, const VocabWork& w, int64_t t, int slot, int used, int lane)
{
    if (t >= s.tokens) {
        const int64_t row = used + (t - s.tokens);
        if (row < (used + kBK - 1) / kBK * kBK)
            pack_row(nullptr, 0, w.x + row * s.dp, s.dp, lane);
    } else if (slot >= 0) {
        pack_row(hidden + t * hs, s.width, w.x + slot * s.dp, s.dp, lane);
    } else if (dhidden != nullptr) {
        for (int64_t i = lane; i < s.width; i += 64)
            dhidden[t * dhs + i] = 0;
    }
}

__global__ __launch_bounds__(kPackBlock) void vocab_pack_kernel(const uint16_t* __restrict__ hidden, int64_t hs,
                                                                uint16_t* __restrict__ dhidden, int64_t dhs,
                                                                VocabSizes s, VocabWork w)
{
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kPackBlock / 64);
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * (kPackBlock / 64) + threadIdx.x / 64; t < s.tokens + kBK; t += step)
        pack_token(hidden, hs, dhidden, dhs, s, w, t, t < s.tokens ? w.slot[t] : -1, *w.used,
                   static_cast<int>(__lane_id()));
}

// Both in one kernel for few tokens: every block numbers all rows itself.
constexpr int kFewTokens = 2048;
template <typename I>
__global__ __launch_bounds__(kPackBlock) void vocab_list_pack_kernel(const I* __restrict__ targets,
                                                                     const uint8_t* __restrict__ mask,
                                                                     const uint16_t* __restrict__ hidden, int64_t hs,
                                                                     uint16_t* __restrict__ dhidden, int64_t dhs, VocabSizes s,
                                                                     VocabWork w, float* __restrict__ token_loss)
{
    constexpr int kWaves = kPackBlock / 64;
    __shared__ uint64_t on[kFewTokens / 64];                   // a bit for each row
    const int lane = static_cast<int>(__lane_id()), wave = threadIdx.x / 64;
    const int tokens = static_cast<int>(s.tokens), words = (tokens + 63) / 64;
    for (int v = wave; v < words; v += kWaves) {
        const int t = v * 64 + lane;
        int64_t y = -1;
        if (t < tokens && (mask == nullptr || mask[t] != 0))
            y = targets[t];
        const uint64_t bits = __ballot(y >= 0);
        if (lane == 0)
            on[v] = bits;
    }
    __syncthreads();
    auto before = [&](int t) {                                 // used rows below t
        int n = 0;
        for (int v = lane; v * 64 < t; v += 64)
            n += __popcll(v * 64 + 64 <= t ? on[v] : on[v] & ((1ull << (t - v * 64)) - 1));
#pragma unroll
        for (int off = 1; off < 64; off <<= 1)
            n += __shfl_xor(n, off);
        return n;
    };
    const int used = before(tokens);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        *w.used = used;
        *w.ticket = 0;
    }
    const int step = static_cast<int>(gridDim.x) * kWaves;
    for (int t = static_cast<int>(blockIdx.x) * kWaves + wave; t < tokens + kBK; t += step) {
        int slot = -1;
        if (t < tokens && (on[t / 64] >> (t % 64) & 1)) {
            slot = before(t);
            if (lane == 0) {
                const int64_t y = targets[t];
                w.list[slot] = t;
                w.target[slot] = y < s.vocab ? static_cast<int32_t>(y) : -1;
            }
        } else if (t < tokens && lane == 0) {
            token_loss[t] = 0.0f;
        }
        pack_token(hidden, hs, dhidden, dhs, s, w, t, slot, used, lane);
    }
}

// Rows v0 .. v0 + rows - 1 of W.
__global__ __launch_bounds__(kPackBlock) void vocab_pack_weight_kernel(const uint16_t* __restrict__ weight, int64_t ws,
                                                                       int64_t rows, VocabSizes s, uint16_t* __restrict__ to)
{
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kPackBlock / 64);
    for (int64_t v = static_cast<int64_t>(blockIdx.x) * (kPackBlock / 64) + threadIdx.x / 64; v < rows; v += step)
        pack_row(weight + v * ws, s.width, to + v * s.dp, s.dp, static_cast<int>(__lane_id()));
}

// A piece of the vocabulary: W's rows from v0 on.
struct VocabPiece {
    const uint16_t* w;
    int64_t stride, v0, rows;
};

// A row's maximum and sum over the whole vocabulary from its partial ones, a
// share of them (`first`, `step`).  Rows are always joined from kJoinWaves
// shares, so that a loss has the same bits with and without the gradient.
constexpr int kJoinWaves = 4;
// JOIN of the logits kernel: its rows, and partial sums that a lane goes through
// in the time of a launch.
constexpr int kVocabJoinTokens = 128, kVocabJoinTiles = 32;
__device__ __forceinline__ TopSum vocab_join(const VocabSizes& s, const VocabWork& w, int64_t n, int first, int step)
{
    TopSum sum{kNegInf, 0.0f};
    for (int64_t i = first; i < s.tiles; i += 8 * step) {      // eight loads on their way
        TopSum v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int64_t at = i + u * step;
            v[u] = at < s.tiles ? w.part[at * s.tp + n] : TopSum{kNegInf, 0.0f};
        }
#pragma unroll
        for (int u = 0; u < 8; ++u)
            sum = join(sum, v[u], kLog2e);
    }
    return sum;
}

// What a row's joined sums say: maximum and log2 of the sum, NaN for a target
// past the vocabulary, and the row's loss.
__device__ __forceinline__ TopSum vocab_row(const VocabWork& w, int64_t n, TopSum sum, float& loss)
{
    const bool known = w.target[n] >= 0;
    const float log_sum = __builtin_amdgcn_logf(sum.sum);
    loss = known ? (sum.top - w.of_target[n]) + log_sum * kLn2 : __builtin_nanf("");
    return {known ? sum.top : __builtin_nanf(""), log_sum};
}

struct VocabLoss {
    float coef;
    float *token_loss, *loss;
    int32_t* used;
};

// Logits of a piece and, at the end, (DZ) dz or else each row's maximum and sum
// over the tile.  m: vocabulary, n: tokens.  JOIN (with DZ, for few tokens and a
// small vocabulary): every block joins all rows' partial sums itself, the last
// one ends the loss, which saves a launch.
template <int FMT, bool DZ, bool JOIN, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64) void vocab_logits_kernel(VocabPiece p, VocabSizes s, VocabWork w,
                                                                                VocabLoss l)
{
    using P = Product<FMT, false, false, BM, BN, WM, WN>;
    __shared__ __attribute__((aligned(1024))) unsigned char lds[P::kLds];
    __shared__ TopSum joined[JOIN ? kVocabJoinTokens : 1];
    const int used = *w.used;
    int tm, tn;
    tile_of(static_cast<int>(blockIdx.x), static_cast<int>((p.rows + BM - 1) / BM), static_cast<int>((s.tokens + BN - 1) / BN),
            tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    if constexpr (JOIN) {
        static_assert(DZ && P::kThreads >= kVocabJoinTokens, "a lane for each row");
        const int n = static_cast<int>(threadIdx.x);
        if (n < used && n < kVocabJoinTokens) {
            float loss;
            TopSum sum = vocab_join(s, w, n, 0, kJoinWaves);
#pragma unroll
            for (int i = 1; i < kJoinWaves; ++i)
                sum = join(sum, vocab_join(s, w, n, i, kJoinWaves), kLog2e);
            joined[n] = vocab_row(w, n, sum, loss);
            if (blockIdx.x + 1 == gridDim.x)
                l.token_loss[w.list[n]] = loss;
        }
        __syncthreads();
        if (blockIdx.x + 1 == gridDim.x) {                     // the last one: a short tile, or none
            const float mean = rows_mean<P::kThreads>(l.token_loss, s.tokens, used, l.coef);
            if (threadIdx.x == 0) {
                *l.loss = mean;
                *l.used = used;
            }
        }
    }
    if (n0 >= used)
        return;
    P c;
    c.run(lds, Operand{p.w + m0 * p.stride, p.stride, static_cast<int32_t>(p.rows) - m0, 0},
          Operand{w.x + n0 * s.dp, s.dp, static_cast<int32_t>(s.tp) - n0, 0}, static_cast<int>(s.dp / kBK));
    const int rows = static_cast<int>(p.rows) - m0;            // of the tile that exist
#pragma unroll
    for (int j = 0; j < P::NI; ++j) {
        const int n = n0 + c.col(j);
        const bool on = n < used;
        const int y = on ? w.target[n] : -1;
        const int hit = y < 0 ? -1 : static_cast<int>(y - p.v0) - m0;
        if constexpr (DZ) {
            const TopSum row = !on ? TopSum{0.0f, 0.0f} : JOIN ? joined[JOIN ? n : 0] : w.row[n];
            constexpr float unit = FMT == kF16 ? 32768.0f : 1.0f;
#pragma unroll
            for (int i = 0; i < P::MI; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    f32x4 d;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int m = c.row(i, 4 * q + r);
                        float z = __builtin_amdgcn_exp2f(
                            __builtin_fmaf(c.acc[i][j][4 * q + r] - row.top, kLog2e, -row.sum));
                        z = m == hit ? z - 1.0f : z;
                        d[r] = on && m < rows ? z * unit : 0.0f;
                    }
                    const int m = m0 + c.row(i, 4 * q);
                    if (m < s.vc && n < s.tp)
                        *reinterpret_cast<u32x2*>(w.dz + static_cast<int64_t>(n) * s.vc + m) = narrow4<FMT>(d);
                }
        } else {
            float top = kNegInf;
#pragma unroll
            for (int i = 0; i < P::MI; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int m = c.row(i, r);
                    if (m == hit)
                        w.of_target[n] = c.acc[i][j][r];
                    if (m < rows)
                        top = fmaxf(top, c.acc[i][j][r]);
                }
            const float ref = finite_top(top);
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < P::MI; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (c.row(i, r) < rows)
                        sum = sum + __builtin_amdgcn_exp2f((c.acc[i][j][r] - ref) * kLog2e);
            TopSum part = join(TopSum{top, sum}, TopSum{__shfl_xor(top, 32), __shfl_xor(sum, 32)}, kLog2e);
            if (c.lane < 32)
                reinterpret_cast<TopSum*>(lds)[c.wm / WM * BN + c.col(j)] = part;
        }
    }
    if constexpr (!DZ) {
        __syncthreads();
        for (int n = threadIdx.x; n < BN; n += P::kThreads)
            if (n0 + n < used) {
                TopSum part = reinterpret_cast<TopSum*>(lds)[n];
                for (int i = 1; i < P::kWavesM; ++i)
                    part = join(part, reinterpret_cast<TopSum*>(lds)[i * BN + n], kLog2e);
                w.part[(p.v0 / BM + tm) * s.tp + n0 + n] = part;
            }
    }
}

// Joins each row's partial sums: 64 rows a block, its waves share the tiles.
// MEAN: the last block to end forms the mean.
constexpr int kJoinBlock = 64 * kJoinWaves;
constexpr int64_t kJoinMean = 16384;       // up to so many tokens; past that the sum wants more lanes
template <bool MEAN>
__global__ __launch_bounds__(kJoinBlock) void vocab_join_kernel(VocabSizes s, VocabWork w, VocabLoss l)
{
    __shared__ TopSum part[kJoinWaves][64];
    __shared__ uint32_t ticket;
    const int lane = static_cast<int>(__lane_id()), wave = threadIdx.x / 64;
    const int used = *w.used;
    for (int64_t n0 = static_cast<int64_t>(blockIdx.x) * 64; n0 < used; n0 += static_cast<int64_t>(gridDim.x) * 64) {
        const int64_t n = n0 + lane;
        TopSum sum{kNegInf, 0.0f};
        if (n < used)
            sum = vocab_join(s, w, n, wave, kJoinWaves);
        part[wave][lane] = sum;
        __syncthreads();
        if (wave == 0 && n < used) {
            for (int i = 1; i < kJoinWaves; ++i)
                sum = join(sum, part[i][lane], kLog2e);
            float loss_here;
            w.row[n] = vocab_row(w, n, sum, loss_here);
            l.token_loss[w.list[n]] = loss_here;
        }
        __syncthreads();
    }
    if constexpr (MEAN) {
        if (gridDim.x > 1) {
            __threadfence();
            __syncthreads();
            if (threadIdx.x == 0)
                ticket = atomicAdd(w.ticket, 1u);
            __syncthreads();
            if (ticket != gridDim.x - 1)
                return;
            __threadfence();
        }
        const float mean = rows_mean<kJoinBlock>(l.token_loss, s.tokens, used, l.coef);
        if (threadIdx.x == 0) {
            *l.loss = mean;
            *l.used = used;
        }
    }
}

struct VocabGrad {
    const ds_scaler* st;
    float coef;
    uint16_t* dhidden;
    int64_t dhs;
    void* dweight;
    int64_t dws;
    int32_t dw32, accumulate;              // dW in fp32; added to
    int32_t first, last;                   // of the pieces
};

template <int FMT>
__device__ __forceinline__ float vocab_factor(const VocabGrad& g, int used)
{
    const double scale = g.st != nullptr ? static_cast<double>(g.st->scale) : 1.0;
    return used > 0 ? static_cast<float>(scale * static_cast<double>(g.coef) / used * (FMT == kF16 ? 1.0 / 32768.0 : 1.0))
                    : 0.0f;
}

// Four values at column d of a row of `width`, the row's last ones one by one.
template <int FMT>
__device__ __forceinline__ void store4(void* row, int64_t d, int64_t width, f32x4 x)
{
    typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
    typedef uint32_t u32x4_4 __attribute__((ext_vector_type(4), aligned(4)));
    if (d + 4 <= width) {
        if constexpr (FMT == kF32)
            *reinterpret_cast<u32x4_4*>(static_cast<float*>(row) + d) = __builtin_bit_cast(u32x4, x);
        else
            *reinterpret_cast<u32x2_any*>(static_cast<uint16_t*>(row) + d) = narrow4<FMT>(x);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (d + i < width)
                store_elem<FMT>(row, d + i, x[i]);
    }
}

template <int FMT>
__device__ __forceinline__ f32x4 load4(const void* row, int64_t d, int64_t width)
{
    f32x4 x = {};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (d + i < width)
            x[i] = load_elem<FMT>(row, d + i);
    return x;
}

template <int FMT>
__device__ __forceinline__ void store_dw(const VocabGrad& g, int64_t v, int64_t d, int64_t width, f32x4 x)
{
    unsigned char* row = static_cast<unsigned char*>(g.dweight) + v * g.dws * (g.dw32 ? 4 : 2);
    if (g.dw32)
        store4<kF32>(row, d, width, g.accumulate ? x + load4<kF32>(row, d, width) : x);
    else
        store4<FMT>(row, d, width, g.accumulate ? x + load4<FMT>(row, d, width) : x);
}

// The k tiles of part `of` of `parts`.
__device__ __forceinline__ void part_of_k(int ktiles, int of, int parts, int& first, int& count)
{
    const int each = (ktiles + parts - 1) / parts;
    first = min(of * each, ktiles);
    count = min(each, ktiles - first);
}

// dX of a piece (m: width, n: tokens, k: the piece's vocabulary) by the first
// `tx` blocks, dW of its rows (m: width, n: the piece's vocabulary, k: tokens) by
// the others.
template <int FMT, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64) void vocab_grads_kernel(VocabPiece p, VocabSizes s, VocabWork w,
                                                                               VocabGrad g, int32_t tx)
{
    using PX = Product<FMT, true, false, BM, BN, WM, WN>;
    using PW = Product<FMT, true, true, BM, BN, WM, WN>;
    __shared__ __attribute__((aligned(1024))) unsigned char lds[PX::kLds];
    const int used = *w.used;
    const float factor = vocab_factor<FMT>(g, used);
    const int tiles_m = static_cast<int>((s.dp + BM - 1) / BM);
    int tm, tn, first, count;
    if (static_cast<int>(blockIdx.x) < tx) {
        const int tiles = tx / s.xs, of = static_cast<int>(blockIdx.x) / tiles;
        tile_of(static_cast<int>(blockIdx.x) % tiles, tiles_m, tiles / tiles_m, tm, tn);
        const int m0 = tm * BM, n0 = tn * BN;
        if (n0 >= used)
            return;
        part_of_k(static_cast<int>((p.rows + kBK - 1) / kBK), of, s.xs, first, count);
        const int64_t k0 = static_cast<int64_t>(first) * kBK;
        PX c;
        c.run(lds, Operand{p.w + k0 * p.stride + m0, p.stride, static_cast<int32_t>(s.dp) - m0, static_cast<int32_t>(p.rows - k0)},
              Operand{w.dz + n0 * s.vc + k0, s.vc, static_cast<int32_t>(s.tp) - n0, 0}, count);
        const bool out = g.last && s.xs == 1;
#pragma unroll
        for (int j = 0; j < PX::NI; ++j) {
            const int n = n0 + c.col(j);
            if (n >= used)
                continue;
            const int64_t t = out ? w.list[n] : 0;
#pragma unroll
            for (int i = 0; i < PX::MI; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int d = m0 + c.row(i, 4 * q);
                    if (d >= s.dp)
                        continue;
                    f32x4 x = {c.acc[i][j][4 * q], c.acc[i][j][4 * q + 1], c.acc[i][j][4 * q + 2], c.acc[i][j][4 * q + 3]};
                    f32x4* sum = reinterpret_cast<f32x4*>(w.dx + (of * s.tokens + n) * s.dp + d);
                    if (!g.first)
                        x = x + *sum;
                    if (out)
                        store4<FMT>(g.dhidden + t * g.dhs, d, s.width, x * factor);
                    else
                        *sum = x;
                }
        }
    } else {
        const int block = static_cast<int>(blockIdx.x) - tx, tiles = (static_cast<int>(gridDim.x) - tx) / s.ws;
        const int of = block / tiles;
        tile_of(block % tiles, tiles_m, tiles / tiles_m, tm, tn);
        const int m0 = tm * BM, n0 = tn * BN;
        part_of_k((used + kBK - 1) / kBK, of, s.ws, first, count);
        const int64_t k0 = static_cast<int64_t>(first) * kBK;
        const int k_rows = static_cast<int>(s.tp - k0);
        PW c;
        c.run(lds, Operand{w.x + k0 * s.dp + m0, s.dp, static_cast<int32_t>(s.dp) - m0, k_rows},
              Operand{w.dz + k0 * s.vc + n0, s.vc, static_cast<int32_t>(s.vc) - n0, k_rows}, count);
#pragma unroll
        for (int j = 0; j < PW::NI; ++j) {
            const int n = n0 + c.col(j);
            if (n >= p.rows)
                continue;
#pragma unroll
            for (int i = 0; i < PW::MI; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int d = m0 + c.row(i, 4 * q);
                    if (d >= s.dp)
                        continue;
                    const f32x4 x = {c.acc[i][j][4 * q], c.acc[i][j][4 * q + 1], c.acc[i][j][4 * q + 2],
                                     c.acc[i][j][4 * q + 3]};
                    if (s.ws > 1)
                        *reinterpret_cast<f32x4*>(w.dw + (of * p.rows + n) * s.dp + d) = x;
                    else if (d < s.width)
                        store_dw<FMT>(g, p.v0 + n, d, s.width, x * factor);
                }
        }
    }
}

// Adds the parts: rows of dX (behind the last piece) by the first rows, rows of
// dW by the others; a wave has a row.
template <int FMT>
__global__ __launch_bounds__(kPackBlock) void vocab_parts_kernel(VocabPiece p, VocabSizes s, VocabWork w, VocabGrad g,
                                                                 int64_t xrows, int64_t wrows)
{
    const int lane = static_cast<int>(__lane_id());
    const int used = *w.used;
    const float factor = vocab_factor<FMT>(g, used);
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kPackBlock / 64);
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * (kPackBlock / 64) + threadIdx.x / 64; r < xrows + wrows; r += step) {
        const bool x_side = r < xrows;
        if (x_side && r >= used)
            continue;
        const int64_t row = x_side ? r : r - xrows, all = x_side ? s.tokens : p.rows;
        const float* part = x_side ? w.dx : w.dw;
        const int parts = x_side ? s.xs : s.ws;
        for (int64_t d = 4 * lane; d < s.width; d += 256) {
            f32x4 sum = *reinterpret_cast<const f32x4*>(part + row * s.dp + d);
            for (int i = 1; i < parts; ++i)
                sum = sum + *reinterpret_cast<const f32x4*>(part + (i * all + row) * s.dp + d);
            sum = sum * factor;
            if (x_side)
                store4<FMT>(g.dhidden + w.list[row] * g.dhs, d, s.width, sum);
            else
                store_dw<FMT>(g, p.v0 + row, d, s.width, sum);
        }
    }
}

// ---- host side ----

int64_t up_to(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

// Parts that a product over `ktiles` tiles of k is split into, for `tiles` tiles
// of 128 x 128: as many as fill the GPU, with four tiles of k each at least.
int32_t vocab_split(int64_t tiles, int64_t ktiles)
{
    int64_t n = kVocabBlocks / tiles;
    n = n < ktiles / 4 ? n : ktiles / 4;
    return static_cast<int32_t>(n < 1 ? 1 : n);
}

bool vocab_sizes(int64_t tokens, int64_t vocab, int64_t width, VocabSizes* s)
{
    if (tokens < 0 || tokens > kVocabMaxTokens || vocab < 1 || vocab > kVocabMaxVocab || width < 1 || width > kVocabMaxWidth)
        return false;
    s->tokens = tokens;
    s->vocab = vocab;
    s->width = width;
    s->tp = up_to(tokens > 0 ? tokens : 1, kVocabTile);
    s->dp = up_to(width, kBK);
    const int64_t whole = up_to(vocab, kVocabTile);
    s->vmax = std::min(whole, std::max(kVocabWidePiece, kVocabWeights / s->dp / kVocabTile * kVocabTile));
    int64_t vc = static_cast<int64_t>(kVocabPiece / (2 * static_cast<uint64_t>(s->tp))) / kVocabTile * kVocabTile;
    vc = std::min(std::max(vc, kVocabMinPiece), s->vmax);
    const int64_t pieces = (vocab + vc - 1) / vc;           // of about the same size
    s->vc = up_to((vocab + pieces - 1) / pieces, kVocabTile);
    s->tiles = 0;
    const int64_t dt = (s->dp + 127) / 128;
    s->xs = vocab_split(dt * ((s->tp + 127) / 128), s->vc / kBK);
    s->ws = vocab_split(dt * ((s->vc + 127) / 128), s->tp / kBK);
    return true;
}

// The workspace's arrays from `base` on, each 256-byte aligned; returns the
// bytes, which are no fewer than those for fewer tokens (with larger pieces).
uint64_t vocab_work(const VocabSizes& s, void* base, VocabWork* w)
{
    uint64_t at = 0;
    auto take = [&](uint64_t bytes) {
        void* p = reinterpret_cast<void*>(reinterpret_cast<uintptr_t>(base) + at);
        at += (bytes + 255) / 256 * 256;
        return p;
    };
    const uint64_t tp = static_cast<uint64_t>(s.tp), dp = static_cast<uint64_t>(s.dp), vmax = static_cast<uint64_t>(s.vmax);
    const uint64_t v64 = (static_cast<uint64_t>(s.vocab) + 63) / 64;   // tiles of 64 up to kVocabSmallTokens, else of 128
    const uint64_t parts = std::max((v64 + 1) / 2 * tp, v64 * std::min(tp, static_cast<uint64_t>(kVocabSmallTokens)));
    const uint64_t piece = 2 * tp * static_cast<uint64_t>(s.vc), most = std::min(2 * tp * vmax, kVocabPiece);
    w->used = static_cast<int32_t*>(take(4));
    w->ticket = static_cast<uint32_t*>(take(4));
    w->slot = static_cast<int32_t*>(take(4 * tp));
    w->list = static_cast<int32_t*>(take(4 * tp));
    w->target = static_cast<int32_t*>(take(4 * tp));
    w->of_target = static_cast<float*>(take(4 * tp));
    w->part = static_cast<TopSum*>(take(sizeof(TopSum) * parts));
    w->row = static_cast<TopSum*>(take(sizeof(TopSum) * tp));
    w->x = static_cast<uint16_t*>(take(2 * tp * dp));
    w->w = static_cast<uint16_t*>(take(2 * vmax * dp));
    w->dz = static_cast<uint16_t*>(take(std::max(piece, most)));
    w->dx = static_cast<float*>(take(std::max(kVocabParts, s.vc < s.vocab ? 4 * tp * dp : 0)));
    w->dw = static_cast<float*>(take(kVocabParts));
    return at;
}

struct VocabCall {
    const uint16_t* weight;
    int64_t ws;
    bool in_place;                         // W is read where it lies
};

VocabPiece vocab_piece(const VocabSizes& s, const VocabWork& w, const VocabCall& c, int64_t v0, hipStream_t st)
{
    const int64_t rows = s.vocab - v0 < s.vc ? s.vocab - v0 : s.vc;
    if (c.in_place)
        return {c.weight + v0 * c.ws, c.ws, v0, rows};
    vocab_pack_weight_kernel<<<grid_blocks((rows + 3) / 4, kPackBlock), kPackBlock, 0, st>>>(c.weight + v0 * c.ws, c.ws,
                                                                                           rows, s, w.w);
    return {w.w, s.dp, v0, rows};
}

int64_t vocab_tiles(int64_t m, int64_t n, int tile) { return ((m + tile - 1) / tile) * ((n + tile - 1) / tile); }

// The side of a product's tiles, from how many there would be.  Up to 256 tiles
// of 128 x 128 (a CU each) take tiles of 64 x 64: the blocks go through their k in
// the same number of turns, each shorter, and have a quarter of the code to fetch
// at the end.  Else 256 x 256 (one block a CU) or 128 x 128 (two), by the rounds
// of the GPU, a tile of 128 costing 1 / 0.85 of a quarter of one of 256.
int vocab_side(const VocabSizes& s, int64_t n128, int64_t n256)
{
    if (n128 <= 256 && s.tokens <= kVocabSmallTokens)
        return 64;
    return 4.0 * static_cast<double>((n256 + 255) / 256) <= 2.0 / 0.85 * static_cast<double>((n128 + 511) / 512) ? 256 : 128;
}

int vocab_logits_side(const VocabSizes& s, int64_t rows)
{
    return vocab_side(s, vocab_tiles(rows, s.tokens, 128), vocab_tiles(rows, s.tokens, 256));
}

template <int FMT, bool DZ>
void vocab_logits(const VocabPiece& p, const VocabSizes& s, const VocabWork& w, const VocabLoss& l, int side, bool join,
                  hipStream_t st)
{
    const unsigned b = static_cast<unsigned>(vocab_tiles(p.rows, s.tokens, side));
    if (DZ && join)       vocab_logits_kernel<FMT, true, true, 64, 64, 32, 32><<<b, 256, 0, st>>>(p, s, w, l);
    else if (side == 64)  vocab_logits_kernel<FMT, DZ, false, 64, 64, 32, 32><<<b, 256, 0, st>>>(p, s, w, l);
    else if (side == 128) vocab_logits_kernel<FMT, DZ, false, 128, 128, 64, 64><<<b, 256, 0, st>>>(p, s, w, l);
    else                  vocab_logits_kernel<FMT, DZ, false, 256, 256, 64, 128><<<b, 512, 0, st>>>(p, s, w, l);
}

template <int FMT>
ds_status vocab_run(VocabSizes s, const VocabWork& w, const VocabCall& c, const VocabGrad& g, const VocabLoss& l, hipStream_t st)
{
    const bool with_grad = g.dhidden != nullptr || g.dweight != nullptr;
    bool join = false;
    if (s.tokens > 0) {
        const int64_t piece = s.vc < s.vocab ? s.vc : s.vocab;
        const int side = vocab_logits_side(s, piece);
        s.tiles = (s.vocab + side - 1) / side;
        join = with_grad && s.tokens <= kVocabJoinTokens && s.tiles <= kVocabJoinTiles && side == 64;
        for (int64_t v0 = 0; v0 < s.vocab; v0 += s.vc)
            vocab_logits<FMT, false>(vocab_piece(s, w, c, v0, st), s, w, l, side, false, st);
        const unsigned b = grid_blocks((s.tokens + 63) / 64, kJoinBlock);
        if (!join && s.tokens <= kJoinMean)
            vocab_join_kernel<true><<<b, kJoinBlock, 0, st>>>(s, w, l);
        else if (!join)
            vocab_join_kernel<false><<<b, kJoinBlock, 0, st>>>(s, w, l);
    }
    if (s.tokens == 0 || s.tokens > kJoinMean)
        rows_mean_kernel<<<1, kMeanBlock, 0, st>>>(l.token_loss, s.tokens, w.used, l.coef, l.loss, l.used, 0);
    if (launched() != DS_OK)
        return DS_ERR_HIP;
    if (!with_grad)
        return DS_OK;
    for (int64_t v0 = 0; v0 < s.vocab; v0 += s.vc) {
        const VocabPiece p = vocab_piece(s, w, c, v0, st);
        VocabGrad h = g;
        h.first = v0 == 0;
        h.last = v0 + p.rows == s.vocab;
        if (s.tokens > 0)
            vocab_logits<FMT, true>(p, s, w, l, vocab_logits_side(s, p.rows), join, st);
        // both gradients in one launch: the second fills what the first leaves free
        const bool dx = g.dhidden != nullptr && s.tokens > 0, dw = g.dweight != nullptr;
        auto tiles = [&](int tile, int64_t& x, int64_t& all) {
            x = dx ? vocab_tiles(s.dp, s.tokens, tile) * s.xs : 0;
            all = x + (dw ? vocab_tiles(s.dp, p.rows, tile) * s.ws : 0);
        };
        int64_t x, n128, n256;
        tiles(256, x, n256);
        tiles(128, x, n128);
        if (n128 == 0)
            continue;
        const int side = vocab_side(s, n128, n256);
        int64_t all;
        tiles(side, x, all);
        const unsigned b = static_cast<unsigned>(all);
        const int32_t tx = static_cast<int32_t>(x);
        if (side == 64)       vocab_grads_kernel<FMT, 64, 64, 32, 32><<<b, 256, 0, st>>>(p, s, w, h, tx);
        else if (side == 128) vocab_grads_kernel<FMT, 128, 128, 64, 64><<<b, 256, 0, st>>>(p, s, w, h, tx);
        else                  vocab_grads_kernel<FMT, 256, 256, 64, 128><<<b, 512, 0, st>>>(p, s, w, h, tx);
        const int64_t xrows = dx && h.last && s.xs > 1 ? s.tokens : 0, wrows = dw && s.ws > 1 ? p.rows : 0;
        if (xrows + wrows > 0)
            vocab_parts_kernel<FMT><<<grid_blocks((xrows + wrows + 3) / 4, kPackBlock), kPackBlock, 0, st>>>(p, s, w, h, xrows,
                                                                                                         wrows);
        if (launched() != DS_OK)
            return DS_ERR_HIP;
    }
    return DS_OK;
}

ds_status vocab_ce(const ds_scaler* scaler, const void* hidden, int64_t hs, const void* weight, int64_t ws, ds_dtype dt,
                   const void* targets, int32_t index_bytes, int64_t tokens, int64_t vocab, int64_t width,
                   const uint8_t* mask, float coef, float* token_loss, float* loss, int32_t* used, void* dhidden, int64_t dhs,
                   void* dweight, ds_dtype dwt, int64_t dws, bool accumulate, void* workspace, size_t bytes, hipStream_t st)
{
    VocabSizes s;
    if (!vocab_sizes(tokens, vocab, width, &s) || !rows_ok(tokens, width, hs) || !rows_ok(vocab, width, ws) ||
        (dhidden != nullptr && !rows_ok(tokens, width, dhs)) || (dweight != nullptr && !rows_ok(vocab, width, dws)))
        return DS_ERR_SIZE;
    if (!is16(dt) || (index_bytes != 4 && index_bytes != 8) || (dweight != nullptr && dwt != dt && dwt != DS_FP32))
        return DS_ERR_DTYPE;
    if (!finite_ge0(coef) || (accumulate && dweight == nullptr))
        return DS_ERR_HPARAM;
    if (weight == nullptr || loss == nullptr || used == nullptr || workspace == nullptr ||
        (tokens > 0 && (hidden == nullptr || targets == nullptr || token_loss == nullptr)))
        return DS_ERR_NULL;
    const uint64_t ib = static_cast<uint64_t>(index_bytes);
    if (!aligned(hidden, 2) || !aligned(weight, 2) || !aligned(targets, ib) || !aligned(token_loss, 4) || !aligned(loss, 4) ||
        !aligned(used, 4) || !aligned(dhidden, 2) || !aligned(dweight, dwt == DS_FP32 ? 4 : 2) || !aligned(scaler, 8) ||
        !aligned(workspace, 256))
        return DS_ERR_ALIGN;
    VocabWork w;
    const uint64_t need = vocab_work(s, workspace, &w);
    if (bytes < need)
        return DS_ERR_SIZE;
    const uint64_t ut = static_cast<uint64_t>(tokens);
    const void* p[11] = {hidden, weight, targets, mask, scaler, token_loss, loss, used, dhidden, dweight, workspace};
    const uint64_t span[11] = {disp_span(tokens, width, hs, dt), disp_span(vocab, width, ws, dt), ib * ut, ut,
                               sizeof(ds_scaler), 4 * ut, 4, 4,
                               dhidden == nullptr ? 0 : disp_span(tokens, width, dhs, dt),
                               dweight == nullptr ? 0 : disp_span(vocab, width, dws, dwt), need};
    if (bal_alias(p, span, 11, 5))
        return DS_ERR_ALIAS;
    const VocabCall c{static_cast<const uint16_t*>(weight), ws,
                      aligned(weight, 16) && ws % 8 == 0 && width % kBK == 0 && ws <= kVocabMaxStride};
    const VocabGrad g{scaler, coef, static_cast<uint16_t*>(dhidden), dhs, dweight, dws, dwt == DS_FP32, accumulate, 0, 0};
    const uint16_t* x = static_cast<const uint16_t*>(hidden);
    const unsigned pack = grid_blocks((tokens + kBK + 3) / 4, kPackBlock);
    if (tokens <= kFewTokens) {
        if (index_bytes == 4)
            vocab_list_pack_kernel<int32_t><<<pack, kPackBlock, 0, st>>>(static_cast<const int32_t*>(targets), mask, x, hs,
                                                                        g.dhidden, dhs, s, w, token_loss);
        else
            vocab_list_pack_kernel<int64_t><<<pack, kPackBlock, 0, st>>>(static_cast<const int64_t*>(targets), mask, x, hs,
                                                                        g.dhidden, dhs, s, w, token_loss);
    } else {
        if (index_bytes == 4)
            vocab_list_kernel<int32_t><<<1, kVocabListBlock, 0, st>>>(static_cast<const int32_t*>(targets), mask, s, w, token_loss);
        else
            vocab_list_kernel<int64_t><<<1, kVocabListBlock, 0, st>>>(static_cast<const int64_t*>(targets), mask, s, w, token_loss);
        vocab_pack_kernel<<<pack, kPackBlock, 0, st>>>(x, hs, g.dhidden, dhs, s, w);
    }
    if (launched() != DS_OK)
        return DS_ERR_HIP;
    const VocabLoss l{coef, token_loss, loss, used};
    return dt == DS_FP16 ? vocab_run<kF16>(s, w, c, g, l, st) : vocab_run<kBF16>(s, w, c, g, l, st);
}
