// dispatch.h -- tokens sorted by expert, moved there and back.
// Included by dszero.hip inside its namespace.
//
// The pairs p = t k + j (token, choice) are sorted by expert with a stable
// counting sort.  A block has a chunk of consecutive pairs, a wave a quarter of
// it; a lane's rank among the 64 pairs of a turn is the number of lower lanes
// with the same expert, found by ballots over the bits of the expert's number.
// Nothing depends on the order in which blocks or atomics run.
//
// The moves go by token: its row of x is read once and written to its k slots
// (gather), its k rows are read and summed (combine, and the gradient of
// gather), or its row of dy is read once beside the k rows (gradient of
// combine).  Each is bound by memory; a token's choices are held by the lanes
// of one wave, so no atomics are needed and the sums have a fixed order.

constexpr int kDispBlock = 256, kDispWaves = kDispBlock / 64;
constexpr int64_t kDispChunk = 1024;       // pairs per block, at least
constexpr int64_t kDispMaxBlocks = 256;    // blocks of the sort: each reads the counts of all
constexpr int kDispSpan = 4;               // vectors of a row that a lane has at once
// Non-temporal stores of the sorted side above so many bytes of it, and
// non-temporal loads of it: what is written there otherwise stays in the Infinity
// Cache and is written back under the next kernel.  All moves of 10007 x 1001 by 4
// in fp32 (160 MB) 216 -> 201 us with the stores, 223 with the loads too; 4096 x
// 4096 by 8 (268 MB) 333 -> 307 and 306; 65536 x 2048 by 8 (2.1 GB) 2386 -> 2359
// and 2302.
constexpr uint64_t kDispStoreBytes = uint64_t(64) << 20, kDispLoadBytes = uint64_t(512) << 20;
constexpr int64_t kDispMaxPairs = (int64_t(1) << 31) - 1;
constexpr int64_t kDispMaxWidth = int64_t(1) << 24;
static_assert(DS_MAX_EXPERTS <= 2 * kDispBlock, "the scan has two experts a lane");

struct DispSort {
    const void* chosen;
    int64_t stride;            // elements from a token's choices to the next one's
    int64_t pairs, chunk;
    int32_t k, experts, blocks;
    int32_t* hist;             // [blocks][experts]
    int32_t *offsets, *place, *source;
};

// The expert of pair p, or -1.
template <typename I>
__device__ __forceinline__ int disp_expert(const DispSort& s, uint32_t p)
{
    const uint32_t t = p / static_cast<uint32_t>(s.k), j = p - t * static_cast<uint32_t>(s.k);
    const int64_t e = static_cast<const I*>(s.chosen)[static_cast<int64_t>(t) * s.stride + j];
    return e >= 0 && e < s.experts ? static_cast<int>(e) : -1;
}

template <typename I>
__global__ __launch_bounds__(kDispBlock) void dispatch_count_kernel(DispSort s)
{
    __shared__ int32_t count[DS_MAX_EXPERTS];
    for (int e = threadIdx.x; e < s.experts; e += kDispBlock)
        count[e] = 0;
    __syncthreads();
    const int64_t lo = blockIdx.x * s.chunk, hi = min(lo + s.chunk, s.pairs);
    for (int64_t p = lo + threadIdx.x; p < hi; p += kDispBlock) {
        const int e = disp_expert<I>(s, static_cast<uint32_t>(p));
        if (e >= 0)
            atomicAdd(&count[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < s.experts; e += kDispBlock)
        s.hist[static_cast<int64_t>(blockIdx.x) * s.experts + e] = count[e];
}

template <typename I>
__global__ __launch_bounds__(kDispBlock) void dispatch_place_kernel(DispSort s)
{
    __shared__ int32_t next[kDispWaves][DS_MAX_EXPERTS];   // counts, then the next slot, per wave
    __shared__ int32_t wave_total[kDispWaves];
    const int lane = static_cast<int>(__lane_id()), wave = threadIdx.x / 64;
    for (int e = threadIdx.x; e < kDispWaves * DS_MAX_EXPERTS; e += kDispBlock)
        (&next[0][0])[e] = 0;
    __syncthreads();
    const int64_t part = s.chunk / kDispWaves;
    const int64_t lo = min(blockIdx.x * s.chunk + wave * part, s.pairs), hi = min(lo + part, s.pairs);
    for (int64_t p = lo + lane; p < hi; p += 64) {
        const int e = disp_expert<I>(s, static_cast<uint32_t>(p));
        if (e >= 0)
            atomicAdd(&next[wave][e], 1);
    }
    __syncthreads();
    // two neighbouring experts per lane: pairs in earlier blocks, pairs in all
    int32_t before[2] = {0, 0}, all[2] = {0, 0};
    const int e0 = 2 * static_cast<int>(threadIdx.x);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int e = e0 + i;
        if (e >= s.experts)
            continue;
        if (s.blocks == 1) {
            for (int w = 0; w < kDispWaves; ++w)
                all[i] += next[w][e];
        } else {
#pragma unroll 8
            for (int b = 0; b < s.blocks; ++b) {
                const int32_t c = s.hist[static_cast<int64_t>(b) * s.experts + e];
                all[i] += c;
                before[i] += b < static_cast<int>(blockIdx.x) ? c : 0;
            }
        }
    }
    int32_t sum = all[0] + all[1];
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int32_t below = __shfl_up(sum, off);
        sum += lane >= off ? below : 0;
    }
    if (lane == 63)
        wave_total[wave] = sum;
    __syncthreads();
    int32_t start = sum - all[0] - all[1], total = 0;
    for (int w = 0; w < kDispWaves; ++w) {
        start += w < wave ? wave_total[w] : 0;
        total += wave_total[w];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int e = e0 + i;
        if (e < s.experts) {
            if (blockIdx.x == 0)
                s.offsets[e] = start;
            int32_t slot = start + before[i];
            for (int w = 0; w < kDispWaves; ++w) {
                const int32_t c = next[w][e];
                next[w][e] = slot;
                slot += c;
            }
            start += all[i];
        }
    }
    if (blockIdx.x == 0 && threadIdx.x == 0)
        s.offsets[s.experts] = total;
    __syncthreads();
    for (int64_t p0 = lo; p0 < hi; p0 += 64) {
        const int64_t p = p0 + lane;
        const int e = p < hi ? disp_expert<I>(s, static_cast<uint32_t>(p)) : -1;
        uint64_t same = __ballot(e >= 0);
        for (int bit = 0; (1 << bit) < s.experts; ++bit) {
            const uint64_t set = __ballot((e >> bit) & 1);
            same &= (e >> bit) & 1 ? set : ~set;
        }
        if (e >= 0) {
            const int32_t slot = next[wave][e] + __popcll(same & ((1ull << lane) - 1));
            s.place[p] = slot;
            s.source[slot] = static_cast<int32_t>(p);
        } else if (p < hi) {
            s.place[p] = -1;
        }
        __builtin_amdgcn_wave_barrier();
        if (e >= 0 && lane == 63 - __clzll(static_cast<long long>(same)))
            next[wave][e] += __popcll(same);
        __builtin_amdgcn_wave_barrier();
    }
    const int64_t step = static_cast<int64_t>(gridDim.x) * kDispBlock;
    for (int64_t q = total + static_cast<int64_t>(blockIdx.x) * kDispBlock + threadIdx.x; q < s.pairs; q += step)
        s.source[q] = -1;
}

// ---- moves ----

// Rows start anywhere that their type allows: a 16-byte access needs no more
// than that here, so that every width has vectors and a short tail.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

struct DispMove {
    int64_t tokens, width, rows;          // rows: slots that the sorted side holds
    int32_t k;
    const int32_t* place;
};

template <int FMT>
__device__ __forceinline__ void widen_vec(u32x4 w, float (&x)[FMT == kF32 ? 4 : 8])
{
    if constexpr (FMT == kF32) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = __uint_as_float(w[i]);
    } else {
        const f32x4 a = widen4<FMT>(u32x2{w.x, w.y}), b = widen4<FMT>(u32x2{w.z, w.w});
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = a[i];
            x[4 + i] = b[i];
        }
    }
}

template <int FMT>
__device__ __forceinline__ u32x4 narrow_vec(const float (&x)[FMT == kF32 ? 4 : 8])
{
    if constexpr (FMT == kF32) {
        return u32x4{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
    } else {
        const u32x2 a = narrow4<FMT>(f32x4{x[0], x[1], x[2], x[3]}), b = narrow4<FMT>(f32x4{x[4], x[5], x[6], x[7]});
        return u32x4{a.x, a.y, b.x, b.y};
    }
}

template <int FMT>
__device__ __forceinline__ float load_elem(const void* p, int64_t i)
{
    if constexpr (FMT == kF32)
        return static_cast<const float*>(p)[i];
    else
        return dec1<FMT>(static_cast<const uint16_t*>(p)[i]);
}

template <int FMT>
__device__ __forceinline__ void store_elem(void* p, int64_t i, float x)
{
    if constexpr (FMT == kF32)
        static_cast<float*>(p)[i] = x;
    else
        static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(enc1<FMT>(x));
}

__device__ __forceinline__ float load_gate(const void* p, int fmt, int64_t i)
{
    return fmt == kF32 ? load_elem<kF32>(p, i) : fmt == kBF16 ? load_elem<kBF16>(p, i) : load_elem<kF16>(p, i);
}

__device__ __forceinline__ void store_gate(void* p, int fmt, int64_t i, float x)
{
    if (fmt == kF32)       store_elem<kF32>(p, i, x);
    else if (fmt == kBF16) store_elem<kBF16>(p, i, x);
    else                   store_elem<kF16>(p, i, x);
}

// The first token of the calling lane's group of G lanes, and the groups of
// the grid.
template <int G>
__device__ __forceinline__ int64_t disp_first(int64_t& groups)
{
    groups = static_cast<int64_t>(gridDim.x) * (kDispBlock / G);
    int first = static_cast<int>(threadIdx.x) / G;
    if constexpr (G >= 64)
        first = __builtin_amdgcn_readfirstlane(first);
    return static_cast<int64_t>(blockIdx.x) * (kDispBlock / G) + first;
}

template <int G>
__device__ __forceinline__ int disp_slot(const DispMove& s, int64_t t, int j)
{
    int slot = s.place[t * s.k + j];
    if constexpr (G >= 64)
        slot = __builtin_amdgcn_readfirstlane(slot);
    return static_cast<uint32_t>(slot) < static_cast<uint64_t>(s.rows) ? slot : -1;
}

// A group goes over a row in spans of U vectors a lane, and takes a span of one
// row whole before the next row's, so that what it reads and writes of a row lies
// together.  Lanes past a row's last vector repeat it, and rows of dropped choices
// are read as the first row's: no load is conditional, so that a wait for one
// row's span can leave the next one's on its way.
template <int G, int U>
struct DispSpan {
    int at[U];                             // the lane's vectors
    bool has[U];

    __device__ __forceinline__ DispSpan(int base, int vecs, int lane)
    {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = base + u * G + lane;
            has[u] = c < vecs;
            at[u] = min(c, vecs - 1);
        }
    }

    template <bool NT = false>
    __device__ __forceinline__ void load(u32x4 (&v)[U], const unsigned char* row) const
    {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const u32x4_any* p = reinterpret_cast<const u32x4_any*>(row) + static_cast<uint32_t>(at[u]);
            if constexpr (NT)
                v[u] = __builtin_nontemporal_load(p);
            else
                v[u] = *p;
        }
    }

    template <bool NT = false>
    __device__ __forceinline__ void store(unsigned char* row, int u, u32x4 v) const
    {
        u32x4_any* p = reinterpret_cast<u32x4_any*>(row) + static_cast<uint32_t>(at[u]);
        if (has[u]) {
            if constexpr (NT)
                __builtin_nontemporal_store(v, p);
            else
                *p = v;
        }
    }
};

template <int ES, int G, int U, bool NT>
__global__ __launch_bounds__(kDispBlock) void dispatch_gather_kernel(DispMove s, const unsigned char* __restrict__ x,
                                                                     int64_t xs, unsigned char* __restrict__ out,
                                                                     int64_t os)
{
    constexpr int kVec = 16 / ES;
    const int lane = static_cast<int>(threadIdx.x) % G;
    const int vecs = static_cast<int>(s.width / kVec);
    int64_t groups;
    for (int64_t t = disp_first<G>(groups); t < s.tokens; t += groups) {
        const unsigned char* from = x + t * xs * ES;
        for (int base = 0; base < vecs; base += U * G) {
            const DispSpan<G, U> span(base, vecs, lane);
            u32x4 v[U];
            span.load(v, from);
            for (int j = 0; j < s.k; ++j) {
                const int slot = disp_slot<G>(s, t, j);
                if (slot >= 0) {
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        span.template store<NT>(out + slot * os * ES, u, v[u]);
                }
            }
        }
        for (int64_t i = static_cast<int64_t>(vecs) * kVec + lane; i < s.width; i += G)
            for (int j = 0; j < s.k; ++j) {
                const int slot = disp_slot<G>(s, t, j);
                if (slot >= 0) {
                    if constexpr (ES == 4)
                        reinterpret_cast<uint32_t*>(out)[slot * os + i] = reinterpret_cast<const uint32_t*>(from)[i];
                    else
                        reinterpret_cast<uint16_t*>(out)[slot * os + i] = reinterpret_cast<const uint16_t*>(from)[i];
                }
            }
    }
}

// out[t] = sum_j gate_tj rows[place_tj] (without gates: of the rows), in fp32,
// j ascending, rounded once.
template <int FMT, int G, int KM, int U, bool NT>
__global__ __launch_bounds__(kDispBlock) void dispatch_combine_kernel(DispMove s, const unsigned char* __restrict__ rows,
                                                                      int64_t rs, const void* __restrict__ gates,
                                                                      int gfmt, int64_t gs,
                                                                      unsigned char* __restrict__ out, int64_t os)
{
    constexpr int ES = FMT == kF32 ? 4 : 2, kVec = 16 / ES;
    const int lane = static_cast<int>(threadIdx.x) % G;
    const int vecs = static_cast<int>(s.width / kVec);
    int64_t groups;
    for (int64_t t = disp_first<G>(groups); t < s.tokens; t += groups) {
        int slot[KM];
        float gate[KM];
#pragma unroll
        for (int j = 0; j < KM; ++j) {
            slot[j] = j < s.k ? disp_slot<G>(s, t, j) : -1;
            gate[j] = 1.0f;
            if (slot[j] >= 0 && gates != nullptr)
                gate[j] = load_gate(gates, gfmt, t * gs + j);
        }
        for (int base = 0; base < vecs; base += U * G) {
            const DispSpan<G, U> span(base, vecs, lane);
            float sum[U][kVec] = {};
            if (s.rows > 0) {
                u32x4 v[2][U];
                span.template load<NT>(v[0], rows + max(slot[0], 0) * rs * ES);
#pragma unroll
                for (int j = 0; j < KM; ++j) {
                    if (j + 1 < KM)
                        span.template load<NT>(v[(j + 1) % 2], rows + max(slot[j + 1], 0) * rs * ES);
                    if (slot[j] >= 0) {
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            float r[kVec];
                            widen_vec<FMT>(v[j % 2][u], r);
#pragma unroll
                            for (int i = 0; i < kVec; ++i)
                                sum[u][i] = __builtin_fmaf(gate[j], r[i], sum[u][i]);
                        }
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                span.store(out + t * os * ES, u, narrow_vec<FMT>(sum[u]));
        }
        for (int64_t i = static_cast<int64_t>(vecs) * kVec + lane; i < s.width; i += G) {
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < KM; ++j)
                if (slot[j] >= 0)
                    sum = __builtin_fmaf(gate[j], load_elem<FMT>(rows, slot[j] * rs + i), sum);
            store_elem<FMT>(out, t * os + i, sum);
        }
    }
}

// drows[place_tj] = gate_tj dy[t], dgate_tj = sum_d dy[t] rows[place_tj] in
// fp32 (a choice that was dropped: 0).  One wave (or block) has a whole row.
template <int FMT, int G, int KM, int U, bool NT>
__global__ __launch_bounds__(kDispBlock) void dispatch_combine_grad_kernel(
    DispMove s, const unsigned char* __restrict__ dy, int64_t ds, const unsigned char* __restrict__ rows, int64_t rs,
    const void* __restrict__ gates, int gfmt, int64_t gs, unsigned char* __restrict__ drows, int64_t drs,
    void* __restrict__ dgates, int64_t dgs)
{
    constexpr int ES = FMT == kF32 ? 4 : 2, kVec = 16 / ES;
    static_assert(G <= 64 || G == kDispBlock, "a wave or a block has a token");
    __shared__ float part[G > 64 ? kDispWaves : 1][KM];
    const int lane = static_cast<int>(threadIdx.x) % G;
    const int vecs = static_cast<int>(s.width / kVec);
    int64_t groups;
    for (int64_t t = disp_first<G>(groups); t < s.tokens; t += groups) {
        int slot[KM];
        float gate[KM], dot[KM];
#pragma unroll
        for (int j = 0; j < KM; ++j) {
            slot[j] = j < s.k ? disp_slot<G>(s, t, j) : -1;
            dot[j] = 0.0f;
            gate[j] = slot[j] >= 0 ? load_gate(gates, gfmt, t * gs + j) : 0.0f;
        }
        for (int base = 0; s.rows > 0 && base < vecs; base += U * G) {
            const DispSpan<G, U> span(base, vecs, lane);
            u32x4 own[U], v[2][U];
            span.load(own, dy + t * ds * ES);
            span.load(v[0], rows + max(slot[0], 0) * rs * ES);
#pragma unroll
            for (int j = 0; j < KM; ++j) {
                if (j + 1 < KM)
                    span.load(v[(j + 1) % 2], rows + max(slot[j + 1], 0) * rs * ES);
                if (slot[j] >= 0) {
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        float d[kVec], r[kVec], sum = 0.0f;
                        widen_vec<FMT>(own[u], d);
                        widen_vec<FMT>(v[j % 2][u], r);
#pragma unroll
                        for (int i = 0; i < kVec; ++i) {
                            sum = __builtin_fmaf(d[i], r[i], sum);
                            r[i] = gate[j] * d[i];
                        }
                        dot[j] = dot[j] + (span.has[u] ? sum : 0.0f);
                        span.template store<NT>(drows + slot[j] * drs * ES, u, narrow_vec<FMT>(r));
                    }
                }
            }
        }
        for (int64_t i = static_cast<int64_t>(vecs) * kVec + lane; i < s.width; i += G) {
            const float d = load_elem<FMT>(dy, t * ds + i);
#pragma unroll
            for (int j = 0; j < KM; ++j)
                if (slot[j] >= 0) {
                    dot[j] = __builtin_fmaf(d, load_elem<FMT>(rows, slot[j] * rs + i), dot[j]);
                    store_elem<FMT>(drows, slot[j] * drs + i, gate[j] * d);
                }
        }
#pragma unroll
        for (int j = 0; j < KM; ++j) {
#pragma unroll
            for (int off = 1; off < (G < 64 ? G : 64); off <<= 1)
                dot[j] += __shfl_xor(dot[j], off);
        }
        if constexpr (G > 64) {
            __syncthreads();                       // the sums of the token before have been read
#pragma unroll
            for (int j = 0; j < KM; ++j)
                if (__lane_id() == 0)
                    part[threadIdx.x / 64][j] = dot[j];
            __syncthreads();
#pragma unroll
            for (int j = 0; j < KM; ++j) {
                dot[j] = part[0][j];
                for (int w = 1; w < kDispWaves; ++w)
                    dot[j] += part[w][j];
            }
        }
        if (lane == 0) {
#pragma unroll
            for (int j = 0; j < KM; ++j)
                if (j < s.k)
                    store_gate(dgates, gfmt, t * dgs + j, dot[j]);
        }
    }
}

// ---- host side ----

bool disp_sizes_ok(int64_t tokens, int32_t experts, int32_t k)
{
    return tokens >= 0 && experts >= 1 && experts <= DS_MAX_EXPERTS && k >= 1 && k <= DS_MAX_EXPERT_CHOICES &&
           tokens <= kDispMaxPairs / k;
}

int64_t disp_chunk(int64_t pairs)
{
    const int64_t least = (pairs + kDispMaxBlocks - 1) / kDispMaxBlocks;
    const int64_t c = least > kDispChunk ? least : kDispChunk;
    return (c + kDispBlock - 1) / kDispBlock * kDispBlock;
}

int64_t disp_blocks(int64_t pairs)
{
    const int64_t c = disp_chunk(pairs), b = (pairs + c - 1) / c;
    return b < 1 ? 1 : b;
}

// No fewer than for fewer pairs, and never short: past kDispMaxBlocks chunks of
// kDispChunk a longer chunk's rounding leaves fewer blocks than that.
uint64_t disp_ws_bytes(int64_t pairs, int32_t experts)
{
    const int64_t chunks = (pairs + kDispChunk - 1) / kDispChunk;
    return 4 * static_cast<uint64_t>(std::clamp(chunks, int64_t(1), kDispMaxBlocks)) * static_cast<uint64_t>(experts);
}

// Rows of `width` values, `stride` apart: sizes that the byte counts can hold.
bool rows_ok(int64_t rows, int64_t width, int64_t stride)
{
    return stride >= width && stride <= kMaxElems && (rows == 0 || stride <= kMaxElems / rows);
}

ds_status dispatch_sort(const void* chosen, int32_t index_bytes, int64_t tokens, int32_t experts, int32_t k,
                        int64_t stride, int32_t* offsets, int32_t* place, int32_t* source, void* ws, size_t ws_bytes,
                        hipStream_t st)
{
    if (!disp_sizes_ok(tokens, experts, k) || !rows_ok(tokens, k, stride))
        return DS_ERR_SIZE;
    if (index_bytes != 4 && index_bytes != 8)
        return DS_ERR_DTYPE;
    const int64_t pairs = tokens * k;
    if (offsets == nullptr || ws == nullptr ||
        (pairs > 0 && (chosen == nullptr || place == nullptr || source == nullptr)))
        return DS_ERR_NULL;
    if (!aligned(chosen, static_cast<uintptr_t>(index_bytes)) || !aligned(offsets, 4) || !aligned(place, 4) ||
        !aligned(source, 4) || !aligned(ws, 4))
        return DS_ERR_ALIGN;
    const uint64_t need = disp_ws_bytes(pairs, experts), up = static_cast<uint64_t>(pairs);
    if (ws_bytes < need)
        return DS_ERR_SIZE;
    const void* p[5] = {chosen, offsets, place, source, ws};
    const uint64_t bytes[5] = {bal_span(tokens, k, stride, static_cast<uint64_t>(index_bytes)),
                               4 * (static_cast<uint64_t>(experts) + 1), 4 * up, 4 * up, need};
    if (bal_alias(p, bytes, 5, 1))
        return DS_ERR_ALIAS;
    const unsigned blocks = static_cast<unsigned>(disp_blocks(pairs));
    const DispSort s{chosen, stride, pairs, disp_chunk(pairs), k, experts, static_cast<int32_t>(blocks),
                     static_cast<int32_t*>(ws), offsets, place, source};
    if (blocks > 1) {
        if (index_bytes == 4) dispatch_count_kernel<int32_t><<<blocks, kDispBlock, 0, st>>>(s);
        else                  dispatch_count_kernel<int64_t><<<blocks, kDispBlock, 0, st>>>(s);
        if (launched() != DS_OK)
            return DS_ERR_HIP;
    }
    if (index_bytes == 4) dispatch_place_kernel<int32_t><<<blocks, kDispBlock, 0, st>>>(s);
    else                  dispatch_place_kernel<int64_t><<<blocks, kDispBlock, 0, st>>>(s);
    return launched();
}

// What the four moves share.  a: the tokens' side [tokens][width], b: the
// sorted side [rows][width].
ds_status disp_move_check(const DispMove& s, ds_dtype dt, const void* a, int64_t as, const void* b, int64_t bs)
{
    if (s.k < 1 || s.k > DS_MAX_EXPERT_CHOICES || s.tokens < 0 || s.tokens > kDispMaxPairs / s.k || s.width < 1 ||
        s.width > kDispMaxWidth || s.rows < 0 || s.rows > kDispMaxPairs || !rows_ok(s.tokens, s.width, as) ||
        !rows_ok(s.rows, s.width, bs))
        return DS_ERR_SIZE;
    if (!known(dt))
        return DS_ERR_DTYPE;
    if ((s.tokens > 0 && (a == nullptr || s.place == nullptr)) || (s.rows > 0 && b == nullptr))
        return DS_ERR_NULL;
    if (!aligned(a, esize(dt)) || !aligned(b, esize(dt)) || !aligned(s.place, 4))
        return DS_ERR_ALIGN;
    return DS_OK;
}

uint64_t disp_place_bytes(const DispMove& s)
{
    return 4 * static_cast<uint64_t>(s.tokens) * static_cast<uint64_t>(s.k);
}

uint64_t disp_span(int64_t rows, int64_t width, int64_t stride, ds_dtype dt)
{
    return rows == 0 ? 0
                     : esize(dt) * (static_cast<uint64_t>(rows - 1) * static_cast<uint64_t>(stride) +
                                    static_cast<uint64_t>(width));
}

// Lanes per token: 16 where a row is a few vectors, a block where there are
// too few tokens to fill the GPU with a wave each.
int disp_lanes(const DispMove& s, ds_dtype dt)
{
    const int64_t vecs = s.width * static_cast<int64_t>(esize(dt)) / 16;
    if (vecs <= 16)
        return 16;
    return vecs > 64 && s.tokens <= 2048 ? 256 : 64;
}

unsigned disp_grid(const DispMove& s, int lanes)
{
    const int64_t per = kDispBlock / lanes;
    return grid_blocks((s.tokens + per - 1) / per, kDispBlock);
}

ds_status dispatch_gather(const DispMove& s, ds_dtype dt, const void* x, int64_t xs, void* out, int64_t os,
                          hipStream_t st)
{
    if (const ds_status rc = disp_move_check(s, dt, x, xs, out, os); rc != DS_OK)
        return rc;
    const void* p[3] = {x, s.place, out};
    const uint64_t bytes[3] = {disp_span(s.tokens, s.width, xs, dt), disp_place_bytes(s),
                               disp_span(s.rows, s.width, os, dt)};
    if (bal_alias(p, bytes, 3, 2))
        return DS_ERR_ALIAS;
    if (s.tokens == 0 || s.rows == 0)
        return DS_OK;
    const int lanes = disp_lanes(s, dt);
    const bool nt = lanes == 64 && bytes[2] > kDispStoreBytes;
    const unsigned b = disp_grid(s, lanes);
    const unsigned char* from = static_cast<const unsigned char*>(x);
    unsigned char* to = static_cast<unsigned char*>(out);
    if (dt == DS_FP32) {
        if (lanes == 16)      dispatch_gather_kernel<4, 16, 1, false><<<b, kDispBlock, 0, st>>>(s, from, xs, to, os);
        else if (nt)          dispatch_gather_kernel<4, 64, kDispSpan, true><<<b, kDispBlock, 0, st>>>(s, from, xs, to, os);
        else if (lanes == 64) dispatch_gather_kernel<4, 64, kDispSpan, false><<<b, kDispBlock, 0, st>>>(s, from, xs, to, os);
        else                  dispatch_gather_kernel<4, 256, kDispSpan, false><<<b, kDispBlock, 0, st>>>(s, from, xs, to, os);
    } else {
        if (lanes == 16)      dispatch_gather_kernel<2, 16, 1, false><<<b, kDispBlock, 0, st>>>(s, from, xs, to, os);
        else if (nt)          dispatch_gather_kernel<2, 64, kDispSpan, true><<<b, kDispBlock, 0, st>>>(s, from, xs, to, os);
        else if (lanes == 64) dispatch_gather_kernel<2, 64, kDispSpan, false><<<b, kDispBlock, 0, st>>>(s, from, xs, to, os);
        else                  dispatch_gather_kernel<2, 256, kDispSpan, false><<<b, kDispBlock, 0, st>>>(s, from, xs, to, os);
    }
    return launched();
}

struct DispCombine {
    const unsigned char* rows;
    int64_t rs;
    const void* gates;
    int gfmt;
    int64_t gs;
    unsigned char* out;
    int64_t os;
};

template <int FMT, int G, bool NT>
void launch_combine2(unsigned b, hipStream_t st, const DispMove& s, const DispCombine& a)
{
    if (s.k <= 2)      dispatch_combine_kernel<FMT, G, 2, (G == 16 ? 1 : kDispSpan), NT><<<b, kDispBlock, 0, st>>>(s, a.rows, a.rs, a.gates, a.gfmt, a.gs, a.out, a.os);
    else if (s.k <= 4) dispatch_combine_kernel<FMT, G, 4, (G == 16 ? 1 : kDispSpan), NT><<<b, kDispBlock, 0, st>>>(s, a.rows, a.rs, a.gates, a.gfmt, a.gs, a.out, a.os);
    else if (s.k <= 8) dispatch_combine_kernel<FMT, G, 8, (G == 16 ? 1 : kDispSpan), NT><<<b, kDispBlock, 0, st>>>(s, a.rows, a.rs, a.gates, a.gfmt, a.gs, a.out, a.os);
    else               dispatch_combine_kernel<FMT, G, 16, (G == 16 ? 1 : kDispSpan), NT><<<b, kDispBlock, 0, st>>>(s, a.rows, a.rs, a.gates, a.gfmt, a.gs, a.out, a.os);
}

template <int FMT>
void launch_combine(int lanes, bool nt, unsigned b, hipStream_t st, const DispMove& s, const DispCombine& a)
{
    if (lanes == 16)      launch_combine2<FMT, 16, false>(b, st, s, a);
    else if (lanes != 64) launch_combine2<FMT, 256, false>(b, st, s, a);
    else if (nt)          launch_combine2<FMT, 64, true>(b, st, s, a);
    else                  launch_combine2<FMT, 64, false>(b, st, s, a);
}

// gates NULL: the plain sum (the gradient of the gather).
ds_status dispatch_combine(const DispMove& s, ds_dtype dt, const void* rows, int64_t rs, const void* gates, ds_dtype gdt,
                           int64_t gs, bool with_gates, void* out, int64_t os, hipStream_t st)
{
    if (const ds_status rc = disp_move_check(s, dt, out, os, rows, rs); rc != DS_OK)
        return rc;
    if (with_gates) {
        if (!rows_ok(s.tokens, s.k, gs))
            return DS_ERR_SIZE;
        if (!known(gdt))
            return DS_ERR_DTYPE;
        if (s.tokens > 0 && gates == nullptr)
            return DS_ERR_NULL;
        if (!aligned(gates, esize(gdt)))
            return DS_ERR_ALIGN;
    }
    const void* p[4] = {rows, s.place, with_gates ? gates : nullptr, out};
    const uint64_t bytes[4] = {disp_span(s.rows, s.width, rs, dt), disp_place_bytes(s),
                               with_gates ? disp_span(s.tokens, s.k, gs, gdt) : 0, disp_span(s.tokens, s.width, os, dt)};
    if (bal_alias(p, bytes, 4, 3))
        return DS_ERR_ALIAS;
    if (s.tokens == 0)
        return DS_OK;
    const int lanes = disp_lanes(s, dt);
    const DispCombine a{static_cast<const unsigned char*>(rows), rs, with_gates ? gates : nullptr,
                        with_gates ? fmt_of(gdt) : kF32, gs, static_cast<unsigned char*>(out), os};
    const bool nt = bytes[0] > kDispLoadBytes;
    const unsigned b = disp_grid(s, lanes);
    if (dt == DS_FP16)      launch_combine<kF16>(lanes, nt, b, st, s, a);
    else if (dt == DS_BF16) launch_combine<kBF16>(lanes, nt, b, st, s, a);
    else                    launch_combine<kF32>(lanes, nt, b, st, s, a);
    return launched();
}

struct DispCombineGrad {
    const unsigned char* dy;
    int64_t ds;
    const unsigned char* rows;
    int64_t rs;
    const void* gates;
    int gfmt;
    int64_t gs;
    unsigned char* drows;
    int64_t drs;
    void* dgates;
    int64_t dgs;
};

template <int FMT, int G, int KM, bool NT>
void launch_combine_grad3(unsigned b, hipStream_t st, const DispMove& s, const DispCombineGrad& a)
{
    dispatch_combine_grad_kernel<FMT, G, KM, (G == 16 ? 1 : kDispSpan), NT><<<b, kDispBlock, 0, st>>>(s, a.dy, a.ds, a.rows, a.rs, a.gates, a.gfmt, a.gs,
                                                                      a.drows, a.drs, a.dgates, a.dgs);
}

template <int FMT, int G, bool NT>
void launch_combine_grad2(unsigned b, hipStream_t st, const DispMove& s, const DispCombineGrad& a)
{
    if (s.k <= 2)      launch_combine_grad3<FMT, G, 2, NT>(b, st, s, a);
    else if (s.k <= 4) launch_combine_grad3<FMT, G, 4, NT>(b, st, s, a);
    else if (s.k <= 8) launch_combine_grad3<FMT, G, 8, NT>(b, st, s, a);
    else               launch_combine_grad3<FMT, G, 16, NT>(b, st, s, a);
}

template <int FMT>
void launch_combine_grad(int lanes, bool nt, unsigned b, hipStream_t st, const DispMove& s, const DispCombineGrad& a)
{
    if (lanes == 16)      launch_combine_grad2<FMT, 16, false>(b, st, s, a);
    else if (lanes != 64) launch_combine_grad2<FMT, 256, false>(b, st, s, a);
    else if (nt)          launch_combine_grad2<FMT, 64, true>(b, st, s, a);
    else                  launch_combine_grad2<FMT, 64, false>(b, st, s, a);
}

ds_status dispatch_combine_grad(const DispMove& s, ds_dtype dt, const void* dy, int64_t ds, const void* rows, int64_t rs,
                                const void* gates, ds_dtype gdt, int64_t gs, void* drows, int64_t drs, void* dgates,
                                int64_t dgs, hipStream_t st)
{
    if (const ds_status rc = disp_move_check(s, dt, dy, ds, rows, rs); rc != DS_OK)
        return rc;
    if (!rows_ok(s.rows, s.width, drs) || !rows_ok(s.tokens, s.k, gs) || !rows_ok(s.tokens, s.k, dgs))
        return DS_ERR_SIZE;
    if (!known(gdt))
        return DS_ERR_DTYPE;
    if ((s.tokens > 0 && (gates == nullptr || dgates == nullptr)) || (s.rows > 0 && drows == nullptr))
        return DS_ERR_NULL;
    if (!aligned(drows, esize(dt)) || !aligned(gates, esize(gdt)) || !aligned(dgates, esize(gdt)))
        return DS_ERR_ALIGN;
    const void* p[6] = {dy, rows, s.place, gates, drows, dgates};
    const uint64_t bytes[6] = {disp_span(s.tokens, s.width, ds, dt), disp_span(s.rows, s.width, rs, dt),
                               disp_place_bytes(s), disp_span(s.tokens, s.k, gs, gdt),
                               disp_span(s.rows, s.width, drs, dt), disp_span(s.tokens, s.k, dgs, gdt)};
    if (bal_alias(p, bytes, 6, 4))
        return DS_ERR_ALIAS;
    if (s.tokens == 0)
        return DS_OK;
    const int lanes = disp_lanes(s, dt);
    const DispCombineGrad a{static_cast<const unsigned char*>(dy), ds, static_cast<const unsigned char*>(rows), rs, gates,
                            fmt_of(gdt), gs, static_cast<unsigned char*>(drows), drs, dgates, dgs};
    const bool nt = bytes[4] > kDispStoreBytes;
    const unsigned b = disp_grid(s, lanes);
    if (dt == DS_FP16)      launch_combine_grad<kF16>(lanes, nt, b, st, s, a);
    else if (dt == DS_BF16) launch_combine_grad<kBF16>(lanes, nt, b, st, s, a);
    else                    launch_combine_grad<kF32>(lanes, nt, b, st, s, a);
    return launched();
}
