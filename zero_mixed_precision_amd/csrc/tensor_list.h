// tensor_list.h -- the optimizer step over a list of tensors: device table,
// overflow check with the sum of squares, Adam with 32-bit or 8-bit states.
// Included by dszero.hip inside its namespace, after its helpers.
//
// Tensors are cut into tiles of 4096 elements, numbered through the list; a
// block finds the tensor of its tile in the table's first-tile numbers, 64 at
// a time (one load for up to 64 tensors, two for up to 4096).

constexpr int64_t kListTile = 4096;
constexpr int kListBlock = 256;                    // lanes: 4 quads each per tile
constexpr int kListQuads = 4;
static_assert(kListTile == 4 * kListBlock * kListQuads, "one tile per block");
static_assert(DS_STATE_BLOCK == 4 * 64, "one quad per lane of a wave is one block of an 8-bit state");
constexpr int32_t kMaxTensors = 1 << 20;

// One tensor in the device table.
struct ListEntry {
    float* master;
    uint16_t* p16;
    void *m, *v;
    float *m_scale, *v_scale;
    const void* grad;
    int64_t n;
    float weight_decay, lr_scale;
    int16_t pf, gf;         // kF16, kBF16, kF32
    int32_t vec;            // every array aligned for vector access
    int32_t tile0;          // first tile
    int32_t pad[3];
};
static_assert(sizeof(ListEntry) == 96, "table entry");

// The table: first-tile numbers (count of them, padded to 16 bytes), then the entries.
__host__ __device__ inline int64_t list_entries_at(int32_t count) { return (4 * int64_t(count) + 15) / 16 * 16; }

// Entries that one table-writing kernel carries in its arguments (3.8 KB).
constexpr int kListChunk = 40;
struct ListChunk {
    ListEntry e[kListChunk];
};

__global__ void list_write_kernel(unsigned char* table, int32_t count, int32_t first, int32_t n, ListChunk c)
{
    int32_t* tile0 = reinterpret_cast<int32_t*>(table);
    ListEntry* entries = reinterpret_cast<ListEntry*>(table + list_entries_at(count));
    const int i = threadIdx.x;
    if (i < n) {
        tile0[first + i] = c.e[i].tile0;
        entries[first + i] = c.e[i];
    }
}

// The tensor that holds `tile`: the last with tile0 <= tile (a tensor without
// tiles is never it, the next one has the same tile0).  Uniform over the wave.
__device__ __forceinline__ int list_find(const int32_t* __restrict__ tile0, int count, int tile)
{
    const int lane = static_cast<int>(__lane_id());
    int lo = 0, hi = count;
    while (hi - lo > 1) {
        const int stride = (hi - lo + 63) / 64;
        const int i = lo + lane * stride;
        const bool le = i < hi && tile0[i] <= tile;
        const int k = __popcll(__ballot(le)) - 1;   // lane 0 holds always
        lo = lo + k * stride;
        hi = lo + stride < hi ? lo + stride : hi;
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

__device__ __forceinline__ float list_grad1(int gf, const void* grad, int64_t i)
{
    if (gf == kF32)
        return load_grad1<kF32>(grad, i);
    return gf == kBF16 ? load_grad1<kBF16>(grad, i) : load_grad1<kF16>(grad, i);
}

// ---- overflow check and sum of squares ----

template <int GF, bool SUMSQ>
__device__ __forceinline__ void list_check_tile(const void* grad, uint32_t& bad, double& s)
{
    constexpr int kPer = GF == kF32 ? 4 : 8;
    constexpr int kVecs = static_cast<int>(kListTile) / (kListBlock * kPer);
    const u32x4* G = static_cast<const u32x4*>(grad) + threadIdx.x;
    u32x4 w[kVecs];
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
        w[j] = G[j * kListBlock];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
        if constexpr (SUMSQ)
            check_sq_vec<GF>(w[j], bad, s);
        else if constexpr (GF == kF32)
            bad |= nonfinite_f32(w[j].x) | nonfinite_f32(w[j].y) | nonfinite_f32(w[j].z) | nonfinite_f32(w[j].w);
        else
            bad |= nonfinite16x2<GF>(w[j].x) | nonfinite16x2<GF>(w[j].y) | nonfinite16x2<GF>(w[j].z) |
                   nonfinite16x2<GF>(w[j].w);
    }
}

// One tile per block and loop turn; with SUMSQ its sum goes to part[tile].
template <bool SUMSQ>
__global__ __launch_bounds__(kListBlock) void list_check_kernel(ds_scaler* __restrict__ st,
                                                                const unsigned char* __restrict__ table,
                                                                int32_t count, int32_t tiles,
                                                                double* __restrict__ part)
{
    __shared__ double lds[2 * (kListBlock / 64)];
    const int32_t* tile0 = reinterpret_cast<const int32_t*>(table);
    const ListEntry* entries = reinterpret_cast<const ListEntry*>(table + list_entries_at(count));
    uint32_t bad = 0u;
    int parity = 0;
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const ListEntry e = entries[list_find(tile0, count, tile)];
        const int64_t base = static_cast<int64_t>(tile - e.tile0) * kListTile;
        const unsigned char* g = static_cast<const unsigned char*>(e.grad) + base * (e.gf == kF32 ? 4 : 2);
        const int64_t left = e.n - base;
        double s = 0.0;
        if (left >= kListTile && (reinterpret_cast<uintptr_t>(g) & 15) == 0) {
            if (e.gf == kF32)
                list_check_tile<kF32, SUMSQ>(g, bad, s);
            else if (e.gf == kBF16)
                list_check_tile<kBF16, SUMSQ>(g, bad, s);
            else
                list_check_tile<kF16, SUMSQ>(g, bad, s);
        } else {
            for (int64_t i = threadIdx.x; i < left && i < kListTile; i += kListBlock) {
                const float x = list_grad1(e.gf, g, i);
                bad |= nonfinite_f32(__float_as_uint(x));
                if constexpr (SUMSQ)
                    s = s + sq(x);
            }
        }
        if constexpr (SUMSQ) {
            const double ts = block_sum_fixed<kListBlock>(s, lds, parity);
            parity ^= 1;
            if (threadIdx.x == 0)
                part[tile] = ts;
        }
    }
    raise_flag(st, bad);
}

// ---- 8-bit states ----

constexpr uint32_t kGold = 0x9E3779B9u, kMixA = 0x6A09E667u, kMixB = 0xBB67AE85u;

__host__ __device__ inline uint32_t dither_mix(uint32_t x)
{
    x ^= x >> 16;
    x *= kMixA;
    x ^= x >> 15;
    x *= kMixB;
    return x ^ (x >> 16);
}

constexpr float kMaxM = 448.0f, kMaxV = 57344.0f;
constexpr float kTopMin = 0x1p-110f;      // below: max / top would overflow; stored as zeros
constexpr float kTopMax = 0x1p126f;       // above: 1 / top would be subnormal, the largest code's value overflow

// Codes come from fp32 bit patterns.  Times 2^-120 (m) or 2^-112 (v) the
// formats' exponents become fp32's lowest ones, subnormals with subnormals, so
// that a step is 2^20 (2^21) units of the pattern everywhere: adding u of
// those units and dropping as many bits is floor(a / ulp + u).  A NaN keeps
// its code.
__device__ __forceinline__ uint32_t code_m(float x, float inv, uint32_t u)
{
    const float a = fabsf(x) * inv;
    const uint32_t c = (__float_as_uint(fminf(a, kMaxM) * 0x1p-120f) + u) >> 20;
    return (a == a ? c : 0x7Fu) | ((__float_as_uint(x) >> 24) & 0x80u);
}

__device__ __forceinline__ uint32_t code_v(float x, float inv, uint32_t u)
{
    const float a = x * inv;
    uint32_t c = (__float_as_uint(fminf(a, kMaxV) * 0x1p-112f) + u) >> 21;
    c = x > 0.0f && c == 0u ? 1u : c;
    return a == a ? c : 0x7Fu;
}

__device__ __forceinline__ f32x4 decode_m(uint32_t w)
{
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), true);
    return f32x4{lo[0], lo[1], hi[0], hi[1]};
}

__device__ __forceinline__ f32x4 decode_v(uint32_t w)
{
    const auto lo = __builtin_amdgcn_cvt_pk_f32_bf8(static_cast<int>(w), false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_bf8(static_cast<int>(w), true);
    return f32x4{lo[0], lo[1], hi[0], hi[1]};
}

// Largest of the lanes' non-negative values over the wave (NaN is left out by
// the maxNum of the lanes' own maxima).
__device__ __forceinline__ float wave_top(float x)
{
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        x = fmaxf(x, __shfl_xor(x, off));
    return x;
}

// ---- Adam ----

struct ListHyper {
    AdamHyper h;            // lr, eps, clipping, accumulation, schedule (weight_decay unused, betas rounded)
    double beta1, beta2;
    uint32_t seed;          // mix(mix(seed >> 32) ^ seed)
};

// What a block needs of the step, for any tensor of it.
struct ListStep {
    AdamConsts c;           // step_size and lrwd of the tensor at hand
    float lr;
    uint32_t key;           // dither key of the step
};

__device__ __forceinline__ void list_tensor_consts(const ds_scaler* st, const ListHyper& hp, const ListEntry& e,
                                                   ListStep& q)
{
    const float lr = q.lr * e.lr_scale;
    bias_scalars(st->step + 1, lr, hp.beta1, hp.beta2, &q.c.step_size, &q.c.rbc2);
    q.c.lrwd = lr * e.weight_decay;
}

__device__ __forceinline__ void list_update(const f32x4& g, f32x4& p, f32x4& m, f32x4& v, bool wd, const AdamConsts& c)
{
    if (wd)
        adam4<true>(g, p, m, v, c);
    else
        adam4<false>(g, p, m, v, c);
}

// Scales and codes of one quad per lane of a wave: one block of the states.
// The scales are uniform over the wave.
template <bool DITHER>
__device__ __forceinline__ void list_encode(const f32x4& m, const f32x4& v, uint32_t key, float& s_m, float& s_v,
                                            uint32_t& cm, uint32_t& cv)
{
    float tm = fmaxf(fmaxf(fabsf(m.x), fabsf(m.y)), fmaxf(fabsf(m.z), fabsf(m.w)));
    float tv = fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w));
    tm = fminf(wave_top(fmaxf(tm, 0.0f)), kTopMax);
    tv = fminf(wave_top(fmaxf(tv, 0.0f)), kTopMax);
    const float im = tm >= kTopMin ? kMaxM * (1.0f / tm) : 0.0f;
    const float iv = tv >= kTopMin ? kMaxV * (1.0f / tv) : 0.0f;
    s_m = tm >= kTopMin ? tm * (1.0f / kMaxM) : 0.0f;
    s_v = tv >= kTopMin ? tv * (1.0f / kMaxV) : 0.0f;
    const uint32_t lane = 4u * __lane_id() * kGold;
    const uint32_t a = key + lane, b = dither_mix(key ^ kMixB) + lane;
    cm = cv = 0u;
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k) {
        const uint32_t um = DITHER ? (a + k * kGold) >> 12 : 1u << 19;
        const uint32_t uv = DITHER ? (b + k * kGold) >> 11 : 1u << 20;
        cm |= code_m(m[k], im, um) << (8 * k);
        cv |= code_v(v[k], iv, uv) << (8 * k);
    }
}

// A whole, aligned tile: vectors of four, every load before the arithmetic.
template <bool E8, bool DITHER, bool NT>
__device__ __forceinline__ void list_tile(const ListEntry& e, int64_t base, const AdamConsts& c, uint32_t key)
{
    constexpr int U = kListQuads;
    const int64_t q0 = base / 4 + threadIdx.x;
    f32x4* P = reinterpret_cast<f32x4*>(e.master) + q0;
    f32x4 g[U], p[U], m[U], v[U];
    uint32_t mc[U], vc[U];
    float ms[U], vs[U];
    const int64_t blk0 = base / DS_STATE_BLOCK + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        p[u] = load<NT>(P + u * kListBlock);
        if constexpr (E8) {
            mc[u] = load<NT>(static_cast<const uint32_t*>(e.m) + q0 + u * kListBlock);
            vc[u] = load<NT>(static_cast<const uint32_t*>(e.v) + q0 + u * kListBlock);
            ms[u] = e.m_scale[blk0 + u * (kListBlock / 64)];
            vs[u] = e.v_scale[blk0 + u * (kListBlock / 64)];
        } else {
            m[u] = load<NT>(static_cast<const f32x4*>(e.m) + q0 + u * kListBlock);
            v[u] = load<NT>(static_cast<const f32x4*>(e.v) + q0 + u * kListBlock);
        }
    }
    if (e.gf == kF32) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            g[u] = load_grad4<kF32, NT>(e.grad, q0 + u * kListBlock);
    } else {
        u32x2 w[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            w[u] = load<NT>(static_cast<const u32x2*>(e.grad) + q0 + u * kListBlock);
        if (e.gf == kBF16) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                g[u] = widen4<kBF16>(w[u]);
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u)
                g[u] = widen4<kF16>(w[u]);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if constexpr (E8) {
            m[u] = decode_m(mc[u]) * ms[u];
            v[u] = decode_v(vc[u]) * vs[u];
        }
        list_update(g[u], p[u], m[u], v[u], c.lrwd != 0.0f, c);
        store<NT>(P + u * kListBlock, p[u]);
        if constexpr (E8) {
            const int64_t blk = blk0 + u * (kListBlock / 64);
            float sm, sv;
            uint32_t cm, cv;
            const uint32_t bk = DITHER ? dither_mix(key + static_cast<uint32_t>(blk) * kGold) : 0u;
            list_encode<DITHER>(m[u], v[u], bk, sm, sv, cm, cv);
            store<NT>(static_cast<uint32_t*>(e.m) + q0 + u * kListBlock, cm);
            store<NT>(static_cast<uint32_t*>(e.v) + q0 + u * kListBlock, cv);
            if (__lane_id() == 0u) {
                e.m_scale[blk] = sm;
                e.v_scale[blk] = sv;
            }
        } else {
            store<NT>(static_cast<f32x4*>(e.m) + q0 + u * kListBlock, m[u]);
            store<NT>(static_cast<f32x4*>(e.v) + q0 + u * kListBlock, v[u]);
        }
        if (e.pf == kBF16)
            store<NT>(reinterpret_cast<u32x2*>(e.p16) + q0 + u * kListBlock, narrow4<kBF16>(p[u]));
        else if (e.pf == kF16)
            store<NT>(reinterpret_cast<u32x2*>(e.p16) + q0 + u * kListBlock, narrow4<kF16>(p[u]));
    }
}

// A short or unaligned tile: element by element, the same arithmetic.
template <bool E8, bool DITHER>
__device__ __forceinline__ void list_tile_edge(const ListEntry& e, int64_t base, const AdamConsts& c, uint32_t key)
{
    for (int u = 0; u < kListQuads; ++u) {
        const int64_t i0 = base + 4 * (static_cast<int64_t>(u) * kListBlock + threadIdx.x);
        const int64_t blk = base / DS_STATE_BLOCK + u * (kListBlock / 64) +
                            __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
        if (blk * DS_STATE_BLOCK >= e.n)   // uniform over the wave
            break;
        f32x4 g = {0, 0, 0, 0}, p = {0, 0, 0, 0}, m = {0, 0, 0, 0}, v = {0, 0, 0, 0};
        float ms = 0.0f, vs = 0.0f;
        if constexpr (E8) {
            ms = e.m_scale[blk];
            vs = e.v_scale[blk];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t i = i0 + k;
            if (i < e.n) {
                g[k] = list_grad1(e.gf, e.grad, i);
                p[k] = e.master[i];
                if constexpr (E8) {
                    m[k] = decode_m(static_cast<const uint8_t*>(e.m)[i]).x * ms;
                    v[k] = decode_v(static_cast<const uint8_t*>(e.v)[i]).x * vs;
                } else {
                    m[k] = static_cast<const float*>(e.m)[i];
                    v[k] = static_cast<const float*>(e.v)[i];
                }
            }
        }
        list_update(g, p, m, v, c.lrwd != 0.0f, c);
        float sm = 0.0f, sv = 0.0f;
        uint32_t cm = 0u, cv = 0u;
        if constexpr (E8) {   // elements past the end are zero: they raise no top
            const uint32_t bk = DITHER ? dither_mix(key + static_cast<uint32_t>(blk) * kGold) : 0u;
            list_encode<DITHER>(m, v, bk, sm, sv, cm, cv);
            if (__lane_id() == 0u) {
                e.m_scale[blk] = sm;
                e.v_scale[blk] = sv;
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t i = i0 + k;
            if (i < e.n) {
                e.master[i] = p[k];
                if constexpr (E8) {
                    static_cast<uint8_t*>(e.m)[i] = static_cast<uint8_t>(cm >> (8 * k));
                    static_cast<uint8_t*>(e.v)[i] = static_cast<uint8_t>(cv >> (8 * k));
                } else {
                    static_cast<float*>(e.m)[i] = m[k];
                    static_cast<float*>(e.v)[i] = v[k];
                }
                if (e.pf == kBF16)
                    e.p16[i] = static_cast<uint16_t>(enc1<kBF16>(p[k]));
                else if (e.pf == kF16)
                    e.p16[i] = static_cast<uint16_t>(enc1<kF16>(p[k]));
            }
        }
    }
}

template <bool E8, bool DITHER, bool NT, bool FUSE>
__global__ __launch_bounds__(kListBlock) void list_adam_kernel(ds_scaler* __restrict__ st,
                                                               const unsigned char* __restrict__ table,
                                                               int32_t count, int32_t tiles, ListHyper hp)
{
    if (st->overflow == 0u) {
        const int32_t* tile0 = reinterpret_cast<const int32_t*>(table);
        const ListEntry* entries = reinterpret_cast<const ListEntry*>(table + list_entries_at(count));
        ListStep q;
        q.c = make_consts(st, hp.h);
        q.c.omb1 = static_cast<float>(1.0 - hp.beta1);
        q.c.omb2 = static_cast<float>(1.0 - hp.beta2);
        q.lr = step_lr(st, hp.h);
        q.key = dither_mix(hp.seed + static_cast<uint32_t>(st->step + 1) * kGold);
        for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
            const int j = list_find(tile0, count, tile);
            const ListEntry e = entries[j];
            list_tensor_consts(st, hp, e, q);
            const uint32_t key = DITHER ? dither_mix(q.key + static_cast<uint32_t>(j) * kGold) : 0u;
            const int64_t base = static_cast<int64_t>(tile - e.tile0) * kListTile;
            if (e.vec && e.n - base >= kListTile)
                list_tile<E8, DITHER, NT>(e, base, q.c, key);
            else
                list_tile_edge<E8, DITHER>(e, base, q.c, key);
        }
    }
    if constexpr (FUSE) {
        __syncthreads();   // every lane of this block has read the scaler state
        if (threadIdx.x == 0 && atomicAdd(&st->blocks_done, 1u) == gridDim.x - 1u) {
            st->blocks_done = 0u;
            advance_scaler(st);
        }
    }
}

// ---- host side ----

struct ListRange {
    uintptr_t at, end;
    bool written;
};

// Validates one tensor and adds its arrays to `r` (room for 7); returns how many.
ds_status list_check_tensor(const ds_tensor& t, ds_dtype sdt, ListRange* r, int* ranges, ListEntry* e)
{
    const bool e8 = sdt == DS_FP8;
    if (!known(t.pdt) || !known(t.gdt))
        return DS_ERR_DTYPE;
    if (!finite_ge0(t.weight_decay) || !finite_ge0(t.lr_scale) || (t.pdt == DS_FP32 && t.p16 != nullptr) ||
        (!e8 && (t.m_scale != nullptr || t.v_scale != nullptr)))
        return DS_ERR_HPARAM;
    *ranges = 0;
    *e = ListEntry{t.master, t.p16, t.m, t.v, t.m_scale, t.v_scale, t.grad, t.n, t.weight_decay, t.lr_scale,
                   static_cast<int16_t>(fmt_of(t.pdt)), static_cast<int16_t>(fmt_of(t.gdt)), 0, 0, {0, 0, 0}};
    if (t.n == 0)
        return DS_OK;
    const bool copy = t.pdt != DS_FP32;
    if (t.master == nullptr || t.m == nullptr || t.v == nullptr || t.grad == nullptr || (copy && t.p16 == nullptr) ||
        (e8 && (t.m_scale == nullptr || t.v_scale == nullptr)))
        return DS_ERR_NULL;
    const uintptr_t gs = static_cast<uintptr_t>(esize(t.gdt));
    if (!aligned(t.master, 4) || !aligned(t.p16, 2) || !aligned(t.grad, gs) || !aligned(t.m_scale, 4) ||
        !aligned(t.v_scale, 4) || (!e8 && (!aligned(t.m, 4) || !aligned(t.v, 4))))
        return DS_ERR_ALIGN;
    e->vec = aligned(t.master, 16) && aligned(t.p16, 8) && aligned(t.grad, 4 * gs) &&
             aligned(t.m, e8 ? 4 : 16) && aligned(t.v, e8 ? 4 : 16);
    const uint64_t n = static_cast<uint64_t>(t.n), sb = (n + DS_STATE_BLOCK - 1) / DS_STATE_BLOCK * 4;
    auto add = [&](const void* p, uint64_t bytes, bool written) {
        if (p != nullptr) {
            const uintptr_t a = reinterpret_cast<uintptr_t>(p);
            r[(*ranges)++] = ListRange{a, a + bytes, written};
        }
    };
    add(t.master, 4 * n, true);
    add(t.p16, 2 * n, true);
    add(t.m, e8 ? n : 4 * n, true);
    add(t.v, e8 ? n : 4 * n, true);
    add(t.m_scale, sb, true);
    add(t.v_scale, sb, true);
    add(t.grad, gs * n, false);
    return DS_OK;
}

// Whether a written range overlaps any other (sorts them).
bool list_alias(ListRange* r, int64_t n)
{
    std::sort(r, r + n, [](const ListRange& a, const ListRange& b) { return a.at < b.at; });
    uintptr_t any = 0, written = 0;   // ends of the ranges before this one
    for (int64_t i = 0; i < n; ++i) {
        if (r[i].at < written || (r[i].written && r[i].at < any))
            return true;
        if (r[i].end > any)
            any = r[i].end;
        if (r[i].written && r[i].end > written)
            written = r[i].end;
    }
    return false;
}

size_t list_bytes(int32_t count)
{
    return count < 0 ? 0 : static_cast<size_t>(list_entries_at(count)) + sizeof(ListEntry) * static_cast<size_t>(count);
}

// A list that ds_tensor_list_write can have filled.
ds_status list_ok(const ds_tensor_list* l)
{
    if (l == nullptr)
        return DS_ERR_NULL;
    if (l->sdt != DS_FP32 && l->sdt != DS_FP8)
        return DS_ERR_DTYPE;
    if (l->count < 0 || l->count > kMaxTensors || l->tiles < 0 || l->elems < 0 || l->elems > kMaxElems ||
        l->tiles > l->elems / kListTile + l->count || (l->tiles == 0) != (l->elems == 0))
        return DS_ERR_SIZE;
    if (l->tiles > 0 && l->table == nullptr)
        return DS_ERR_NULL;
    return DS_OK;
}

uint64_t list_ws_bytes(int64_t tiles) { return 8 * static_cast<uint64_t>(tiles + finish_groups(tiles)); }

ds_status list_write(ds_tensor_list* list, void* table, size_t table_bytes, const ds_tensor* tensors, int32_t count,
                     ds_dtype sdt, hipStream_t s)
{
    if (list == nullptr)
        return DS_ERR_NULL;
    if (count < 0 || count > kMaxTensors)
        return DS_ERR_SIZE;
    if (sdt != DS_FP32 && sdt != DS_FP8)
        return DS_ERR_DTYPE;
    if (count > 0 && (tensors == nullptr || table == nullptr))
        return DS_ERR_NULL;
    if (table_bytes < list_bytes(count))
        return DS_ERR_SIZE;
    if (!aligned(table, 16))
        return DS_ERR_ALIGN;
    ds_tensor_list out{count > 0 ? table : nullptr, 0, 0, count, sdt};
    if (count > 0) {
        // host scratch of the call: the entries, and the byte ranges of all arrays
        ListEntry* e = static_cast<ListEntry*>(std::malloc(sizeof(ListEntry) * static_cast<size_t>(count)));
        ListRange* r = static_cast<ListRange*>(std::malloc(sizeof(ListRange) * (7 * static_cast<size_t>(count) + 1)));
        ds_status rc = e == nullptr || r == nullptr ? DS_ERR_SIZE : DS_OK;
        int64_t ranges = 0;
        for (int32_t i = 0; rc == DS_OK && i < count; ++i) {
            if (!size_ok(tensors[i].n) || out.elems + tensors[i].n > kMaxElems) {
                rc = DS_ERR_SIZE;
                break;
            }
            int got = 0;
            rc = list_check_tensor(tensors[i], sdt, r + ranges, &got, e + i);
            e[i].tile0 = static_cast<int32_t>(out.tiles);
            ranges += got;
            out.elems += tensors[i].n;
            out.tiles += (tensors[i].n + kListTile - 1) / kListTile;
        }
        if (rc == DS_OK) {
            const uintptr_t a = reinterpret_cast<uintptr_t>(table);
            r[ranges++] = ListRange{a, a + list_bytes(count), true};
            if (list_alias(r, ranges))
                rc = DS_ERR_ALIAS;
        }
        for (int32_t first = 0; rc == DS_OK && first < count; first += kListChunk) {
            const int32_t n = count - first < kListChunk ? count - first : kListChunk;
            ListChunk c{};
            std::memcpy(c.e, e + first, sizeof(ListEntry) * static_cast<size_t>(n));
            list_write_kernel<<<1, 64, 0, s>>>(static_cast<unsigned char*>(table), count, first, n, c);
            rc = launched();
        }
        std::free(e);
        std::free(r);
        if (rc != DS_OK)
            return rc;
    }
    *list = out;
    return DS_OK;
}

ds_status list_check(ds_scaler* st, const ds_tensor_list* l, void* ws, size_t ws_bytes, hipStream_t s)
{
    if (const ds_status rc = list_ok(l); rc != DS_OK)
        return rc;
    if (st == nullptr)
        return DS_ERR_NULL;
    if (!aligned(st, 8) || !aligned(ws, 8) || !aligned(l->table, 16))
        return DS_ERR_ALIGN;
    if (l->tiles == 0)
        return DS_OK;
    if (ws != nullptr && ws_bytes < list_ws_bytes(l->tiles))
        return DS_ERR_SIZE;
    const size_t tb = list_bytes(l->count);
    if (overlap(st, sizeof(ds_scaler), l->table, tb) || overlap(ws, list_ws_bytes(l->tiles), l->table, tb) ||
        overlap(ws, list_ws_bytes(l->tiles), st, sizeof(ds_scaler)))
        return DS_ERR_ALIAS;
    const unsigned blocks = grid_blocks(l->tiles, kListBlock);
    const unsigned char* table = static_cast<const unsigned char*>(l->table);
    const int32_t tiles = static_cast<int32_t>(l->tiles);
    double* part = static_cast<double*>(ws);
    if (part == nullptr) {
        list_check_kernel<false><<<blocks, kListBlock, 0, s>>>(st, table, l->count, tiles, nullptr);
        return launched();
    }
    list_check_kernel<true><<<blocks, kListBlock, 0, s>>>(st, table, l->count, tiles, part);
    if (launched() != DS_OK)
        return DS_ERR_HIP;
    return launch_finish(st, part, l->tiles, s);
}

template <bool E8, bool DITHER, bool NT>
void launch_list_adam2(bool fuse, unsigned blocks, hipStream_t s, ds_scaler* st, const ds_tensor_list* l,
                       const ListHyper& hp)
{
    const unsigned char* table = static_cast<const unsigned char*>(l->table);
    const int32_t tiles = static_cast<int32_t>(l->tiles);
    if (fuse) list_adam_kernel<E8, DITHER, NT, true><<<blocks, kListBlock, 0, s>>>(st, table, l->count, tiles, hp);
    else      list_adam_kernel<E8, DITHER, NT, false><<<blocks, kListBlock, 0, s>>>(st, table, l->count, tiles, hp);
}

template <bool E8, bool DITHER>
void launch_list_adam(bool nt, bool fuse, unsigned blocks, hipStream_t s, ds_scaler* st, const ds_tensor_list* l,
                      const ListHyper& hp)
{
    if (nt) launch_list_adam2<E8, DITHER, true>(fuse, blocks, s, st, l, hp);
    else    launch_list_adam2<E8, DITHER, false>(fuse, blocks, s, st, l, hp);
}

ds_status list_adam(ds_scaler* st, const ds_tensor_list* l, const AdamHyper& h, double beta1, double beta2,
                    ds_rounding rounding, uint64_t seed, bool end_step, hipStream_t s)
{
    if (const ds_status rc = list_ok(l); rc != DS_OK)
        return rc;
    if (!finite_ge0(h.lr) || !(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !std::isfinite(h.eps) || h.eps <= 0.0f ||
        !finite_ge0(h.max_grad_norm) || h.accum_steps < 1 ||
        (rounding != DS_ROUND_NEAREST && rounding != DS_ROUND_DITHER))
        return DS_ERR_HPARAM;
    if (st == nullptr)
        return DS_ERR_NULL;
    if (!aligned(st, 8) || !aligned(l->table, 16))
        return DS_ERR_ALIGN;
    if (l->tiles == 0) {
        if (!end_step)
            return DS_OK;
        update_scale_kernel<<<1, 1, 0, s>>>(st);
        return launched();
    }
    if (overlap(st, sizeof(ds_scaler), l->table, list_bytes(l->count)))
        return DS_ERR_ALIAS;
    const ListHyper hp{h, beta1, beta2, dither_mix(dither_mix(static_cast<uint32_t>(seed >> 32)) ^ static_cast<uint32_t>(seed))};
    const bool nt = variant_nt(l->elems);
    const unsigned blocks = grid_blocks(l->tiles, kListBlock);
    if (l->sdt == DS_FP32)
        launch_list_adam<false, false>(nt, end_step, blocks, s, st, l, hp);
    else if (rounding == DS_ROUND_DITHER)
        launch_list_adam<true, true>(nt, end_step, blocks, s, st, l, hp);
    else
        launch_list_adam<true, false>(nt, end_step, blocks, s, st, l, hp);
    return launched();
}
