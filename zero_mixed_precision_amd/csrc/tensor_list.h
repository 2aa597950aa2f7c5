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
// Tiles that share one partial sum of squares, and a block's turn: four keep
// enough loads on their way on a long list, a short one is over as soon one by
// one.  Check and sum of a bf16 list, one by one and by fours: 256 tiles 6.4 and
// 6.6 us, 512 6.7 and 6.9, 1024 7.4 and 6.9, 2048 8.9 and 7.4, 4096 12.9 and
// 9.6, four layers (197,636) 433 and 272.  Up to kCheckFew one by one, though
// fours are ahead from some 700 on: ds_step_list's update adds up these sums,
// one per tile, up to as many tiles (kStepParts).
constexpr int kCheckTiles = 4;
constexpr int32_t kCheckFew = 2048;                // tiles
// Tickets of the blocks of one step: taken from one address they cost about
// 13 ns each, one after another (2.5 ms for four layers' 197,636 blocks, more
// than the 8-bit step itself), so block b takes one from counter b % 64 (of 16
// up to 1024 blocks), each counter on a line of its own, and the last of each
// from the scaler's.  Taken before the update they cost it little even where a
// block's time is short (8-bit states, one layer: 570 us a step, 576 with a
// kernel of its own that advances the scaler; taken at the end they made the
// update alone 561 us instead of 522).
constexpr unsigned kTicketLines = 64, kTicketBytes = 128;
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

// The table: ticket counters (0 between steps), first-tile numbers (count of
// them, padded to 16 bytes), the entries.
constexpr int64_t kTile0At = kTicketLines * kTicketBytes;
__host__ __device__ inline int64_t list_entries_at(int32_t count)
{
    return kTile0At + (4 * int64_t(count) + 15) / 16 * 16;
}

// Entries that one table-writing kernel carries in its arguments (3.8 KB).
constexpr int kListChunk = 40;
struct ListChunk {
    ListEntry e[kListChunk];
};

static_assert(kTicketLines == 64, "list_write_kernel clears one per lane of its wave");
__global__ __launch_bounds__(64) void list_write_kernel(unsigned char* table, int32_t count, int32_t first, int32_t n, ListChunk c)
{
    int32_t* tile0 = reinterpret_cast<int32_t*>(table + kTile0At);
    ListEntry* entries = reinterpret_cast<ListEntry*>(table + list_entries_at(count));
    const int i = threadIdx.x;
    if (first == 0)
        *reinterpret_cast<uint32_t*>(table + i * kTicketBytes) = 0u;
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

// list_find of two tiles (at once where one load serves both).
__device__ __forceinline__ void list_find2(const int32_t* __restrict__ tile0, int count, int a, int b, int& of_a, int& of_b)
{
    if (count > 64) {
        of_a = list_find(tile0, count, a);
        of_b = list_find(tile0, count, b);
        return;
    }
    const int lane = static_cast<int>(__lane_id());
    const int first = lane < count ? tile0[lane] : 0x7FFFFFFF;
    of_a = __popcll(__ballot(first <= a)) - 1;
    of_b = __popcll(__ballot(first <= b)) - 1;
}

// Loads and stores through pointers that come from the table: they are known
// to be global memory, not the generic pointers that the compiler must take
// them for (whose accesses also occupy the shared memory's counters).
#define DS_GLOBAL __attribute__((address_space(1)))

template <bool NT = false, typename T>
__device__ __forceinline__ T gload(const T* p)
{
    const DS_GLOBAL T* q = (const DS_GLOBAL T*)p;
    if constexpr (NT)
        return __builtin_nontemporal_load(q);
    else
        return *q;
}

template <bool NT = false, typename T>
__device__ __forceinline__ void gstore(T* p, T x)
{
    DS_GLOBAL T* q = (DS_GLOBAL T*)p;
    if constexpr (NT)
        __builtin_nontemporal_store(x, q);
    else
        *q = x;
}

__device__ __forceinline__ float list_grad1(int gf, const void* grad, int64_t i)
{
    if (gf == kF32)
        return gload(static_cast<const float*>(grad) + i);
    const uint32_t w = gload(static_cast<const uint16_t*>(grad) + i);
    return gf == kBF16 ? dec1<kBF16>(w) : dec1<kF16>(w);
}

// ---- overflow check and sum of squares ----

template <int GF, bool SUMSQ>
__device__ __forceinline__ void list_check_vec(const u32x4& w, uint32_t& bad, double& s)
{
    if constexpr (SUMSQ)
        check_sq_vec<GF>(w, bad, s);
    else if constexpr (GF == kF32)
        bad |= nonfinite_f32(w.x) | nonfinite_f32(w.y) | nonfinite_f32(w.z) | nonfinite_f32(w.w);
    else
        bad |= nonfinite16x2<GF>(w.x) | nonfinite16x2<GF>(w.y) | nonfinite16x2<GF>(w.z) | nonfinite16x2<GF>(w.w);
}

// TILES whole, aligned tiles at `grad`: every load before the arithmetic.
template <int GF, bool SUMSQ, int TILES>
__device__ __forceinline__ void list_check_tiles(const void* grad, uint32_t& bad, double& s)
{
    constexpr int kPer = GF == kF32 ? 4 : 8;
    constexpr int kVecs = TILES * static_cast<int>(kListTile) / (kListBlock * kPer);
    const u32x4* G = static_cast<const u32x4*>(grad) + threadIdx.x;
    u32x4 w[kVecs];
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
        w[j] = gload(G + j * kListBlock);
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
        list_check_vec<GF, SUMSQ>(w[j], bad, s);
}

template <bool SUMSQ>
__device__ __forceinline__ void list_check_any(int gf, const u32x4& w, uint32_t& bad, double& s)
{
    if (gf == kF32)
        list_check_vec<kF32, SUMSQ>(w, bad, s);
    else if (gf == kBF16)
        list_check_vec<kBF16, SUMSQ>(w, bad, s);
    else
        list_check_vec<kF16, SUMSQ>(w, bad, s);
}

template <bool SUMSQ>
__device__ __forceinline__ void list_check1(float x, uint32_t& bad, double& s)
{
    bad |= nonfinite_f32(__float_as_uint(x));
    if constexpr (SUMSQ)
        s = s + sq(x);
}

// Tile `left` elements from its tensor's end.  Aligned: whole vectors, vector
// j * kListBlock + l by lane l in j order, then the elements left over, one a
// lane; else element j * kListBlock + l by lane l.
template <bool SUMSQ>
__device__ __forceinline__ void list_check_tile(const unsigned char* g, int gf, int64_t left, uint32_t& bad, double& s)
{
    const bool fast = (reinterpret_cast<uintptr_t>(g) & 15) == 0;
    if (fast && left >= kListTile) {
        if (gf == kF32)
            list_check_tiles<kF32, SUMSQ, 1>(g, bad, s);
        else if (gf == kBF16)
            list_check_tiles<kBF16, SUMSQ, 1>(g, bad, s);
        else
            list_check_tiles<kF16, SUMSQ, 1>(g, bad, s);
        return;
    }
    const int n = static_cast<int>(left < kListTile ? left : kListTile), per = gf == kF32 ? 4 : 8, me = threadIdx.x;
    int done = 0;
    if (fast) {
        for (int v = me; v < n / per; v += kListBlock)
            list_check_any<SUMSQ>(gf, gload(reinterpret_cast<const u32x4*>(g) + v), bad, s);
        done = n / per * per;
    }
    for (int i = done + me; i < n; i += kListBlock)
        list_check1<SUMSQ>(list_grad1(gf, g, i), bad, s);
}

__host__ __device__ inline int list_turn(int64_t tiles) { return tiles <= kCheckFew ? 1 : kCheckTiles; }

// A group of tiles per block and loop turn; with SUMSQ its sum goes to
// part[group].  Four whole tiles of one 16-bit tensor go at once.
template <bool SUMSQ>
__global__ __launch_bounds__(kListBlock) void list_check_kernel(ds_scaler* __restrict__ st,
                                                                const unsigned char* __restrict__ table,
                                                                int32_t count, int32_t tiles,
                                                                double* __restrict__ part)
{
    __shared__ double lds[2 * (kListBlock / 64)];
    const int32_t* tile0 = reinterpret_cast<const int32_t*>(table + kTile0At);
    const ListEntry* entries = reinterpret_cast<const ListEntry*>(table + list_entries_at(count));
    const int turn = list_turn(tiles), groups = (tiles + turn - 1) / turn;
    uint32_t bad = 0u;
    int parity = 0;
    for (int group = blockIdx.x; group < groups; group += gridDim.x) {
        int tile = group * turn;
        const int end = tile + turn < tiles ? tile + turn : tiles;
        double s = 0.0;
        while (tile < end) {
            const ListEntry e = entries[list_find(tile0, count, tile)];
            int64_t base = static_cast<int64_t>(tile - e.tile0) * kListTile;
            const unsigned char* g = static_cast<const unsigned char*>(e.grad) + base * (e.gf == kF32 ? 4 : 2);
            if (e.gf != kF32 && tile + kCheckTiles == end && e.n - base >= kCheckTiles * kListTile &&
                (reinterpret_cast<uintptr_t>(g) & 15) == 0) {
                if (e.gf == kBF16)
                    list_check_tiles<kBF16, SUMSQ, kCheckTiles>(g, bad, s);
                else
                    list_check_tiles<kF16, SUMSQ, kCheckTiles>(g, bad, s);
                break;
            }
            for (; tile < end && base < e.n; ++tile, base += kListTile, g += kListTile * (e.gf == kF32 ? 4 : 2))
                list_check_tile<SUMSQ>(g, e.gf, e.n - base, bad, s);
        }
        if constexpr (SUMSQ) {
            const double ts = block_sum_fixed<kListBlock>(s, lds, parity);
            parity ^= 1;
            if (threadIdx.x == 0)
                part[group] = ts;
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
// its code; blocks without one (`nan` false) skip the test.
__device__ __forceinline__ uint32_t code_m(float x, float inv, uint32_t u, bool nan)
{
    const float a = fabsf(x) * inv;
    const uint32_t c = (__float_as_uint(fminf(a, kMaxM) * 0x1p-120f) + u) >> 20;
    return nan && a != a ? 0x7Fu : c;    // the sign joins in list_encode
}

__device__ __forceinline__ uint32_t code_v(float x, float inv, uint32_t u, bool nan)
{
    const float a = x * inv;
    uint32_t c = (__float_as_uint(fminf(a, kMaxV) * 0x1p-112f) + u) >> 21;
    c = x > 0.0f && c == 0u ? 1u : c;
    return nan && a != a ? 0x7Fu : c;
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
    x = row_max<16>(x);
    const int b = __float_as_int(x);     // rows of 16 lanes; non-negative floats order as integers
    const int r01 = max(__builtin_amdgcn_readlane(b, 0), __builtin_amdgcn_readlane(b, 16));
    const int r23 = max(__builtin_amdgcn_readlane(b, 32), __builtin_amdgcn_readlane(b, 48));
    return __int_as_float(max(r01, r23));
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
    double om1;             // 1 - beta1^t
    uint32_t key;           // dither key of the step
};

__device__ __forceinline__ ListStep list_step(const ds_scaler* st, const ListHyper& hp)
{
    ListStep q;
    q.c = make_consts(st, hp.h);
    q.c.omb1 = static_cast<float>(1.0 - hp.beta1);
    q.c.omb2 = static_cast<float>(1.0 - hp.beta2);
    q.lr = step_lr(st, hp.h);
    double om2;
    bias_powers(st->step + 1, hp.beta1, hp.beta2, &q.om1, &om2);
    q.c.rbc2 = static_cast<float>(1.0 / sqrt(om2));
    q.key = dither_mix(hp.seed + static_cast<uint32_t>(st->step + 1) * kGold);
    return q;
}

__device__ __forceinline__ void list_tensor_consts(const ListEntry& e, ListStep& q)
{
    const float lr = q.lr * e.lr_scale;
    q.c.step_size = static_cast<float>(static_cast<double>(lr) / q.om1);
    q.c.lrwd = lr * e.weight_decay;
}

// The constants in scalar registers (they are the same in every lane, which
// the compiler cannot know of a value that it formed in vector registers).
__device__ __forceinline__ float list_scalar(float x)
{
    return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(x)));
}

__device__ __forceinline__ AdamConsts list_scalars(const AdamConsts& c)
{
    return AdamConsts{list_scalar(c.inv),  c.b1, c.b2, list_scalar(c.omb1), list_scalar(c.omb2), list_scalar(c.lrwd),
                      list_scalar(c.step_size), list_scalar(c.rbc2), c.eps};
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
    // a NaN anywhere shows in the sum (as may infinities of both signs)
    const float sum = ((m.x + m.y) + (m.z + m.w)) + ((v.x + v.y) + (v.z + v.w));
    const bool nan = __ballot(sum != sum) != 0ull;
    uint32_t c[4], d[4];
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k) {
        c[k] = code_m(m[k], im, DITHER ? (a + k * kGold) >> 12 : 1u << 19, false);
        d[k] = code_v(v[k], iv, DITHER ? (b + k * kGold) >> 11 : 1u << 20, false);
    }
    if (nan) {
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) {
            c[k] = code_m(m[k], im, DITHER ? (a + k * kGold) >> 12 : 1u << 19, true);
            d[k] = code_v(v[k], iv, DITHER ? (b + k * kGold) >> 11 : 1u << 20, true);
        }
    }
    cm = c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24;
    cv = d[0] | d[1] << 8 | d[2] << 16 | d[3] << 24;
    // signs: the top bits of the values' top bytes
    const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(m.y), __float_as_uint(m.x), 0x0C0C0703u);
    const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(m.w), __float_as_uint(m.z), 0x07030C0Cu);
    cm |= (lo | hi) & 0x80808080u;
}

// The hardware's square root takes a subnormal v for zero.  Its true root is
// below 2^-63: where rbc2 times that is below 2^-26 of eps, as at any usual eps,
// it is lost in the denominator's rounding; else (the same for a whole block)
// such a v is scaled first.
__device__ __forceinline__ bool list_tiny(const AdamConsts& c) { return c.rbc2 * 0x1p-37f > c.eps; }

__device__ __forceinline__ float list_small_root(float v, float root)
{
    return v < 0x1p-126f ? __builtin_amdgcn_sqrtf(v * 0x1p64f) * 0x1p-32f : root;
}

// Four elements with 8-bit states: adam1 with the hardware's square root and
// reciprocal (each within 1 unit) and fused multiply-adds in the parameter's
// part.  Its states' arithmetic is adam1's, rounding by rounding.  The IEEE
// forms are 24 more vector instructions an element beside 79 (one layer: 606 us
// a step, 573 with these; 363 odd tiles 17.1 and 15.9; four tiles 6.0 and 5.8).
__device__ __forceinline__ void adam4_fp8(const f32x4& graw, f32x4& p, f32x4& m, f32x4& v, const AdamConsts& c,
                                          bool tiny)
{
    float root[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float g = graw[k] * c.inv;
        const float m1 = c.b1 * m[k], m2 = c.omb1 * g;
        m[k] = m1 + m2;
        const float gg = g * g, v1 = c.b2 * v[k], v2 = c.omb2 * gg;
        v[k] = v1 + v2;
        root[k] = __builtin_amdgcn_sqrtf(v[k]);
    }
    if (__builtin_expect(tiny, 0)) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            root[k] = list_small_root(v[k], root[k]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        // at least the smallest normal number: the reciprocal of a smaller one is infinite
        const float den = fmaxf(__builtin_fmaf(root[k], c.rbc2, c.eps), 0x1p-126f);
        const float q = __builtin_fmaf(-c.lrwd, p[k], p[k]);
        p[k] = __builtin_fmaf(-c.step_size, m[k] * __builtin_amdgcn_rcpf(den), q);
    }
}

// A tile's quads in registers, four per lane.
template <bool E8>
struct ListRegs {
    u32x2 g[kListQuads], g2[kListQuads];
    f32x4 p[kListQuads], m[kListQuads], v[kListQuads];
};

template <>
struct ListRegs<true> {
    u32x2 g[kListQuads], g2[kListQuads];
    f32x4 p[kListQuads];
    uint32_t m[kListQuads], v[kListQuads];
    float m_scale[kListQuads], v_scale[kListQuads];
};

// Scale block of the wave's quad u from element `base` on.
__device__ __forceinline__ int64_t list_block(int64_t base, int u)
{
    return base / DS_STATE_BLOCK + u * (kListBlock / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
}

// A state's scale, uniform over the wave, by a scalar load.  The wave that reads
// it is the one that writes it, afterwards.
__device__ __forceinline__ float list_scale(const float* p)
{
    return *(const __attribute__((address_space(4))) float*)p;
}

// Loads of U quads per lane, into the first U, from element `base` on.  FULL: whole and aligned,
// vectors of four throughout.  Else a vector where the tensor is aligned and
// the quad whole, single elements otherwise, zeros past the end (so that a
// short block's top is right).
template <bool E8, bool NT, bool FULL, int U>
__device__ __forceinline__ void list_load(const ListEntry& e, int64_t base, ListRegs<E8>& r)
{
    const int64_t q0 = base / 4 + threadIdx.x;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t q = q0 + u * kListBlock;
        if constexpr (E8) {
            const int64_t blk = list_block(base, u);
            const bool in = FULL || blk * DS_STATE_BLOCK < e.n;
            r.m_scale[u] = in ? list_scale(e.m_scale + blk) : 0.0f;
            r.v_scale[u] = in ? list_scale(e.v_scale + blk) : 0.0f;
        }
        if (FULL || (e.vec && 4 * q + 4 <= e.n)) {
            r.p[u] = gload<NT>(reinterpret_cast<const f32x4*>(e.master) + q);
            if constexpr (E8) {
                r.m[u] = gload<NT>(static_cast<const uint32_t*>(e.m) + q);
                r.v[u] = gload<NT>(static_cast<const uint32_t*>(e.v) + q);
            } else {
                r.m[u] = gload<NT>(static_cast<const f32x4*>(e.m) + q);
                r.v[u] = gload<NT>(static_cast<const f32x4*>(e.v) + q);
            }
        } else {
            f32x4 p = {0, 0, 0, 0};
            decltype(r.m[0] + r.m[0]) m = {}, v = {};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t i = 4 * q + k;
                if (i < e.n) {
                    p[k] = gload(e.master + i);
                    if constexpr (E8) {
                        m |= static_cast<uint32_t>(gload(static_cast<const uint8_t*>(e.m) + i)) << (8 * k);
                        v |= static_cast<uint32_t>(gload(static_cast<const uint8_t*>(e.v) + i)) << (8 * k);
                    } else {
                        m[k] = gload(static_cast<const float*>(e.m) + i);
                        v[k] = gload(static_cast<const float*>(e.v) + i);
                    }
                }
            }
            r.p[u] = p;
            r.m[u] = m;
            r.v[u] = v;
        }
    }
    // The gradient's bits: the first two words hold a 16-bit quad, and all four
    // an fp32 one (two loads: with one of four words for fp32 alone, merging
    // the two kinds of registers would wait here for every load).  Widened by
    // list_widen, once all loads are on their way and the constants formed.
    const bool wide = e.gf == kF32;
    const unsigned char* grad = static_cast<const unsigned char*>(e.grad);
    if (FULL || (e.vec && 4 * (q0 + (U - 1) * kListBlock) + 4 <= e.n)) {
        const int64_t size = wide ? 16 : 8;
#pragma unroll
        for (int u = 0; u < U; ++u)
            r.g[u] = gload<NT>(reinterpret_cast<const u32x2*>(grad + (q0 + u * kListBlock) * size));
        if (wide) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                r.g2[u] = gload<NT>(reinterpret_cast<const u32x2*>(grad + (q0 + u * kListBlock) * 16 + 8));
        }
    } else {
        static_assert(FULL || U == 1, "one quad");
        uint32_t x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t i = 4 * q0 + k;
            x[k] = 0u;
            if (i < e.n) {
                if (wide)
                    x[k] = gload(reinterpret_cast<const uint32_t*>(grad) + i);
                else
                    x[k] = gload(reinterpret_cast<const uint16_t*>(grad) + i);
            }
        }
        r.g[0] = wide ? u32x2{x[0], x[1]} : u32x2{x[0] | x[1] << 16, x[2] | x[3] << 16};
        r.g2[0] = u32x2{x[2], x[3]};
    }
}

__device__ __forceinline__ f32x4 list_widen(int gf, const u32x2& a, const u32x2& b)
{
    if (gf == kF32)
        return f32x4{__uint_as_float(a.x), __uint_as_float(a.y), __uint_as_float(b.x), __uint_as_float(b.y)};
    return gf == kBF16 ? widen4<kBF16>(a) : widen4<kF16>(a);
}

// Update and stores of the U quads loaded by list_load.
template <bool E8, bool DITHER, bool NT, bool FULL, int U>
__device__ __forceinline__ void list_finish(const ListEntry& e, int64_t base, ListRegs<E8>& r, const AdamConsts& c,
                                            uint32_t key)
{
    const int64_t q0 = base / 4 + threadIdx.x;
    float scale_m = 0.0f, scale_v = 0.0f;
    const bool tiny = E8 && list_tiny(c);
    f32x4 g[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const u32x2 lo = r.g[u], hi = r.g2[u];
        g[u] = list_widen(e.gf, lo, hi);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t q = q0 + u * kListBlock, blk = list_block(base, u);
        if (!FULL && blk * DS_STATE_BLOCK >= e.n)   // uniform over the wave
            return;
        f32x4 m, v;
        if constexpr (E8) {
            m = decode_m(r.m[u]) * r.m_scale[u];
            v = decode_v(r.v[u]) * r.v_scale[u];
        } else {
            m = r.m[u];
            v = r.v[u];
        }
        f32x4 p = r.p[u];
        uint32_t cm = 0u, cv = 0u;
        if constexpr (E8) {
            adam4_fp8(g[u], p, m, v, c, tiny);
        } else {
            list_update(g[u], p, m, v, c.lrwd != 0.0f, c);
        }
        if constexpr (E8) {
            float sm, sv;
            list_encode<DITHER>(m, v, DITHER ? dither_mix(key + static_cast<uint32_t>(blk) * kGold) : 0u, sm, sv, cm,
                                cv);
            if (__lane_id() == static_cast<unsigned>(u)) {
                scale_m = sm;
                scale_v = sv;
            }
            if (u == U - 1) {                      // the wave's scales together, one a lane
                const int64_t mine = list_block(base, 0) + __lane_id() * (kListBlock / 64);
                if (__lane_id() < U) {
                    gstore(e.m_scale + mine, scale_m);
                    gstore(e.v_scale + mine, scale_v);
                }
            }
        }
        if (FULL || (e.vec && 4 * q + 4 <= e.n)) {
            gstore<NT>(reinterpret_cast<f32x4*>(e.master) + q, p);
            if constexpr (E8) {
                gstore<NT>(static_cast<uint32_t*>(e.m) + q, cm);
                gstore<NT>(static_cast<uint32_t*>(e.v) + q, cv);
            } else {
                gstore<NT>(static_cast<f32x4*>(e.m) + q, m);
                gstore<NT>(static_cast<f32x4*>(e.v) + q, v);
            }
            if (e.pf == kBF16)
                gstore<NT>(reinterpret_cast<u32x2*>(e.p16) + q, narrow4<kBF16>(p));
            else if (e.pf == kF16)
                gstore<NT>(reinterpret_cast<u32x2*>(e.p16) + q, narrow4<kF16>(p));
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t i = 4 * q + k;
                if (i < e.n) {
                    gstore(e.master + i, float(p[k]));
                    if constexpr (E8) {
                        gstore(static_cast<uint8_t*>(e.m) + i, static_cast<uint8_t>(cm >> (8 * k)));
                        gstore(static_cast<uint8_t*>(e.v) + i, static_cast<uint8_t>(cv >> (8 * k)));
                    } else {
                        gstore(static_cast<float*>(e.m) + i, float(m[k]));
                        gstore(static_cast<float*>(e.v) + i, float(v[k]));
                    }
                    if (e.pf == kBF16)
                        gstore(e.p16 + i, static_cast<uint16_t>(enc1<kBF16>(p[k])));
                    else if (e.pf == kF16)
                        gstore(e.p16 + i, static_cast<uint16_t>(enc1<kF16>(p[k])));
                }
            }
        }
    }
}

// What one block has in flight: a tile, or with U = 1 a quarter of one (a quad
// per lane).  A whole aligned tile is loaded at once; any other goes one quad
// per lane after another when its turn comes (its code once, not four times: a
// short list's time is in part the fetching of code that no block has run
// before).
template <bool E8, bool DITHER, bool NT, int U>
struct ListTile {
    static_assert(U == 1 || U == kListQuads, "a quarter or a whole tile");
    ListEntry e;
    int64_t base;
    bool full;
    int index;
    ListRegs<E8> r;

    // `part` of kListQuads / U of the tile
    __device__ __forceinline__ void set(const ListEntry* entries, int tile, int part)
    {
        e = entries[index];
        base = static_cast<int64_t>(tile - e.tile0) * kListTile + part * (U * 4 * kListBlock);
        full = U == kListQuads && e.vec && e.n - base >= kListTile;
    }

    __device__ __forceinline__ void load()
    {
        if constexpr (U == 1)
            list_load<E8, false, false, 1>(e, base, r);
        else if (full)
            list_load<E8, NT, true, U>(e, base, r);
    }

    __device__ __forceinline__ void finish(ListStep& q)
    {
        list_tensor_consts(e, q);
        const AdamConsts c = list_scalars(q.c);
        const uint32_t key = DITHER ? dither_mix(q.key + static_cast<uint32_t>(index) * kGold) : 0u;
        if constexpr (U == 1) {
            list_finish<E8, DITHER, false, false, 1>(e, base, r, c, key);
            return;
        }
        if (full) {
            list_finish<E8, DITHER, NT, true, U>(e, base, r, c, key);
            return;
        }
        const int64_t end = e.n - base < kListTile ? e.n : base + kListTile;
#pragma unroll 1
        for (int64_t at = base; at < end; at += 4 * kListBlock) {
            list_load<E8, false, false, 1>(e, at, r);
            list_finish<E8, DITHER, false, false, 1>(e, at, r, c, key);
        }
    }
};

// The part of the scaler that a step's end changes or goes by: all before the
// counters.  Read by scalar loads at a kernel's start and held in scalar
// registers; the compiler would move the loads of what only the last block
// needs behind the tickets and make them vector loads there, and such a load
// per wave of the line that tickets are taken from made the kernel 4.6 times
// slower.
constexpr int kScalerWords = offsetof(ds_scaler, blocks_done) / 4;
static_assert(kScalerWords == 20, "whole 16-byte vectors");

__device__ __forceinline__ ds_scaler list_scaler(const ds_scaler* st)
{
    const auto* w = (const __attribute__((address_space(4))) uint32_t*)reinterpret_cast<const uint32_t*>(st);
    uint32_t x[kScalerWords];
#pragma unroll
    for (int i = 0; i < kScalerWords; ++i)
        x[i] = w[i];
#pragma unroll
    for (int i = 0; i < kScalerWords; ++i)
        asm volatile("" : "+s"(x[i]));
    ds_scaler s{};
    __builtin_memcpy(&s, x, sizeof(x));
    return s;
}

// A block's ticket: taken by thread 0 once all of the block has read the scaler
// (and found the step's flag and norm), so early that the update hides the
// atomic; the last block then advances the scaler from `now`, what it has read.
// Up to kTicketLines blocks take theirs from the scaler's counter at once.
__device__ __forceinline__ unsigned list_lines() { return gridDim.x <= 1024 ? 16 : kTicketLines; }

__device__ __forceinline__ uint32_t list_ticket(ds_scaler* st, uint32_t* tickets)
{
    if (gridDim.x <= kTicketLines)
        return atomicAdd(&st->blocks_done, 1u);
    return atomicAdd(tickets + blockIdx.x % list_lines() * (kTicketBytes / 4), 1u);
}

__device__ __forceinline__ void list_end_step(ds_scaler* st, const ds_scaler& now, uint32_t* tickets, uint32_t before)
{
    if (gridDim.x > kTicketLines) {
        const unsigned lines = list_lines(), line = blockIdx.x % lines;
        if (before != (gridDim.x - line + lines - 1) / lines - 1u)
            return;
        tickets[line * (kTicketBytes / 4)] = 0u;
        if (atomicAdd(&st->blocks_done, 1u) != lines - 1u)
            return;
    } else if (before != gridDim.x - 1u) {
        return;
    }
    const ds_scaler s = advanced(now, now.overflow);
    u32x4 x[kScalerWords / 4];
    __builtin_memcpy(x, &s, sizeof(x));
#pragma unroll
    for (int i = 0; i < kScalerWords / 4; ++i)
        reinterpret_cast<u32x4*>(st)[i] = x[i];
    st->blocks_done = 0u;
}

// A tile per block and loop turn: for a pinned grid (DSZERO_GRID), and past the
// largest one.
template <bool E8, bool DITHER, bool FUSE>
__global__ __launch_bounds__(kListBlock, 4) void list_adam_kernel(ds_scaler* __restrict__ st,
                                                               const unsigned char* __restrict__ table,
                                                               uint32_t* __restrict__ tickets, int32_t count,
                                                               int32_t tiles, ListHyper hp)
{
    const int32_t* tile0 = reinterpret_cast<const int32_t*>(table + kTile0At);
    const ListEntry* entries = reinterpret_cast<const ListEntry*>(table + list_entries_at(count));
    const ds_scaler now = list_scaler(st);
    uint32_t before = 0u;
    if constexpr (FUSE) {
        __syncthreads();   // every wave of this block has read the scaler
        if (threadIdx.x == 0)
            before = list_ticket(st, tickets);
    }
    if (now.overflow == 0u) {
        ListStep q = list_step(&now, hp);
        for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
            ListTile<E8, DITHER, false, kListQuads> t;
            t.index = list_find(tile0, count, tile);
            t.set(entries, tile, 0);
            t.load();
            t.finish(q);
        }
    }
    if constexpr (FUSE)
        if (threadIdx.x == 0)
            list_end_step(st, now, tickets, before);
}

// ---- a block per tile; a whole step over a short list ----

// Up to kStepParts tiles every block adds the check's partial sums itself,
// instead of a kernel between the check and the update (363 tiles: 14.0 us a
// step, 17.3); up to kStepCheck tiles every block also checks the whole list
// itself, instead of a kernel before (four tiles: 5.3 us, 8.8; eight with the
// norm: 8.7, 9.1).  Up to kStepQuarter tiles a block does a quarter of one:
// the code that a block runs for the first time is then a third as long, and
// fetching it is most of so short a kernel's time (64 tiles with the norm:
// 9.1 us, 10.6 with a tile a block; 256: 13.0, 12.6).
constexpr int kStepParts = 2048, kStepQuarter = 128, kStepCheck = 8;
static_assert(kStepParts <= kCheckFew && kStepParts <= kGroup && kFinishBlock == kListBlock,
              "one group of one tile's sums each: the order of sumsq_finish_kernel");
enum ListFront { kFrontNone, kFrontParts, kFrontCheck, kFrontCheckSum };
constexpr bool list_checks(int front) { return front == kFrontCheck || front == kFrontCheckSum; }

// This lane's share of the sum over part[0 .. parts), in sumsq_finish_kernel's order.
struct ListParts {
    double x[kStepParts / kListBlock];

    __device__ __forceinline__ void load(const double* part, int parts)
    {
#pragma unroll
        for (int j = 0; j < kStepParts / kListBlock; ++j) {
            const int i = j * kListBlock + static_cast<int>(threadIdx.x);
            x[j] = part[i < parts ? i : 0];     // past the end: left out below (no branch between the loads)
        }
    }

    __device__ __forceinline__ double lane_sum(int parts) const
    {
        double s = 0.0;
#pragma unroll
        for (int j = 0; j < kStepParts / kListBlock; ++j)
            s = s + (j * kListBlock + static_cast<int>(threadIdx.x) < parts ? x[j] : 0.0);
        return s;
    }
};

// One tile checked by one wave, lane by lane as the four waves of
// list_check_kernel's block do it (list_check_tile): s[w] is what lane `lane`
// of its wave w sums.  512 vectors are in registers at a time, half an fp32
// tile or a whole one of 16 bits.
template <bool SUMSQ>
struct ListWaveCheck {
    static constexpr int kWaves = kListBlock / 64;
    const unsigned char* g;
    int gf, n;
    bool fast;
    u32x4 x[2][kWaves];

    __device__ __forceinline__ void set(const ListEntry& e, int tile)
    {
        const int64_t base = static_cast<int64_t>(tile - e.tile0) * kListTile, left = e.n - base;
        gf = e.gf;
        g = static_cast<const unsigned char*>(e.grad) + base * (gf == kF32 ? 4 : 2);
        n = static_cast<int>(left < kListTile ? left : kListTile);
        fast = (reinterpret_cast<uintptr_t>(g) & 15) == 0;
    }

    __device__ __forceinline__ void load(int first)
    {
        const int vecs = fast ? n / (gf == kF32 ? 4 : 8) : 0;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const int v = first + j * kListBlock + w * 64 + static_cast<int>(__lane_id());
                x[j][w] = u32x4{0u, 0u, 0u, 0u};     // adds nothing
                if (v < vecs)
                    x[j][w] = gload(reinterpret_cast<const u32x4*>(g) + v);
            }
    }

    template <int GF>
    __device__ __forceinline__ void add(uint32_t& bad, double (&s)[kWaves]) const
    {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int w = 0; w < kWaves; ++w)
                list_check_vec<GF, SUMSQ>(x[j][w], bad, s[w]);
    }

    // The check of the tile whose first 512 vectors are loaded; its sum, in every lane.
    __device__ __forceinline__ double finish(uint32_t& bad)
    {
        const int lane = static_cast<int>(__lane_id());
        double s[kWaves] = {};
        if (fast) {
            if (gf == kBF16) {
                add<kBF16>(bad, s);
            } else if (gf == kF16) {
                add<kF16>(bad, s);
            } else {
                add<kF32>(bad, s);
                if (n > static_cast<int>(kListTile) / 2) {
                    load(2 * kListBlock);
                    add<kF32>(bad, s);
                }
            }
            const int left = n % (gf == kF32 ? 4 : 8);
            if (left != 0 && lane < left)
                list_check1<SUMSQ>(list_grad1(gf, g, n - left + lane), bad, s[0]);
        } else {
#pragma unroll 1
            for (int at = 0; at < n; at += 2 * kListBlock) {
                float y[2][kWaves];
                if (gf == kF32) {
#pragma unroll
                    for (int i = 0; i < 2 * kWaves; ++i) {
                        const int e = at + i * 64 + lane;
                        y[i / kWaves][i % kWaves] = e < n ? gload(reinterpret_cast<const float*>(g) + e) : 0.0f;
                    }
                } else {
                    uint32_t h[2 * kWaves];
#pragma unroll
                    for (int i = 0; i < 2 * kWaves; ++i) {
                        const int e = at + i * 64 + lane;
                        h[i] = e < n ? gload(reinterpret_cast<const uint16_t*>(g) + e) : 0u;
                    }
#pragma unroll
                    for (int i = 0; i < 2 * kWaves; ++i)
                        y[i / kWaves][i % kWaves] = gf == kBF16 ? dec1<kBF16>(h[i]) : dec1<kF16>(h[i]);
                }
#pragma unroll
                for (int i = 0; i < 2 * kWaves; ++i)
                    list_check1<SUMSQ>(y[i / kWaves][i % kWaves], bad, s[i % kWaves]);
            }
        }
        if constexpr (!SUMSQ)
            return 0.0;
        static_assert(kWaves == 4, "the butterfly of block_sum_fixed over the waves");
#pragma unroll
        for (int off = 32; off > 0; off >>= 1)
#pragma unroll
            for (int w = 0; w < kWaves; ++w)
                s[w] = s[w] + __shfl_xor(s[w], off);
        return (s[0] + s[2]) + (s[1] + s[3]);
    }
};

// A block per tile, or four: the update, with FUSE the step's end, and with
// kFrontCheck and kFrontCheckSum its check.  The gradients are only read, so
// the blocks need not meet: each comes to the same flag and sum.  The step's
// constants (fp64 powers and divisions) are formed while the loads are on
// their way.  One layer of 202,383,360 parameters in bf16: 938 us with 32-bit
// states (6.04 TB/s of 28 bytes an element), 508 us with 8-bit ones (6.40 TB/s
// of 16.06; a plain copy reaches 6.65): memory bounds both, and in 8 bits the
// vector units are as busy (79 instructions an element; forming the constants
// in one wave alone took 8 % of them and no time).  Blocks that loop over tiles
// are slower (1024 to 16384 of them: 10 to 14 % in 32 bits, 20 to 30 % in 8).
template <bool E8, bool DITHER, bool NT, bool FUSE, int FRONT, int U>
__global__ __launch_bounds__(kListBlock, list_checks(FRONT) ? 2 : 4) void list_step_kernel(
    ds_scaler* __restrict__ st, const unsigned char* __restrict__ table, uint32_t* __restrict__ tickets, int32_t count,
    int32_t tiles, ListHyper hp, const double* __restrict__ part)
{
    __shared__ double lds[FRONT == kFrontParts ? kListBlock / 64 + 1 : kStepCheck];
    const int32_t* tile0 = reinterpret_cast<const int32_t*>(table + kTile0At);
    const ListEntry* entries = reinterpret_cast<const ListEntry*>(table + list_entries_at(count));
    ds_scaler now = list_scaler(st);
    if constexpr (FRONT == kFrontNone) {
        if (now.overflow != 0u) {              // nothing to update
            __syncthreads();
            if (FUSE && threadIdx.x == 0)
                list_end_step(st, now, tickets, list_ticket(st, tickets));
            return;
        }
    }
    constexpr int kSplit = kListQuads / U;
    const int own = blockIdx.x / kSplit, part_of = blockIdx.x % kSplit;
    ListTile<E8, DITHER, NT, U> t;
    double mine = 0.0;
    if constexpr (FRONT == kFrontParts) {
        // beside the table's loads; what adds them later would wait for the tile's
        ListParts parts;
        parts.load(part, tiles);
        t.index = list_find(tile0, count, own);
        t.set(entries, own, part_of);
        mine = parts.lane_sum(tiles);
    } else if constexpr (FRONT == kFrontNone) {
        t.index = list_find(tile0, count, own);
        t.set(entries, own, part_of);
    }
    // the whole list's check: a tile per wave in turn, the first one's loads before the block's own
    constexpr int kWaves = kListBlock / 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = static_cast<int>(__lane_id());
    ListWaveCheck<FRONT == kFrontCheckSum> check;
    if constexpr (list_checks(FRONT)) {
        int other;
        list_find2(tile0, count, own, wave < tiles ? wave : 0, t.index, other);
        t.set(entries, own, part_of);
        check.set(entries[other], wave < tiles ? wave : 0);
        check.load(0);
    }
    t.load();
    ListStep q = list_step(&now, hp);      // while the loads are on their way
    if constexpr (FRONT == kFrontParts) {
        mine = block_sum_fixed<kListBlock>(mine, lds, 0);
        if (threadIdx.x == 0)
            lds[kListBlock / 64] = mine;
        __syncthreads();
        now.grad_sumsq = now.grad_sumsq + lds[kListBlock / 64];
    } else if constexpr (FRONT == kFrontNone) {
        if constexpr (FUSE)
            __syncthreads();
    } else {
        uint32_t bad = 0u;
        static_assert(kStepCheck <= 64, "one lane per tile below");
#pragma unroll 1
        for (int tile = wave; tile < tiles; tile += kWaves) {
            if (tile != wave) {
                check.set(entries[list_find(tile0, count, tile)], tile);
                check.load(0);
            }
            const double sum = check.finish(bad);
            if (FRONT == kFrontCheckSum && lane == 0)
                lds[tile] = sum;
        }
        now.overflow |= static_cast<uint32_t>(__syncthreads_or(static_cast<int>(bad)));
        if constexpr (FRONT == kFrontCheckSum) {
            double sum = lane < tiles ? lds[lane] : 0.0;
#pragma unroll
            for (int off = 32; off > 0; off >>= 1)
                sum = sum + __shfl_xor(sum, off);
            now.grad_sumsq = now.grad_sumsq + sum;
        }
    }
    uint32_t before = 0u;
    if (FUSE && threadIdx.x == 0)          // behind a barrier that every wave reached with the scaler read
        before = list_ticket(st, tickets);
    if (now.overflow == 0u) {
        if constexpr (FRONT == kFrontParts || FRONT == kFrontCheckSum)
            q.c.inv = make_consts(&now, hp.h).inv;   // by the norm
        t.finish(q);
    }
    if (FUSE && threadIdx.x == 0)
        list_end_step(st, now, tickets, before);
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
    return count <= 0 ? 0 : static_cast<size_t>(list_entries_at(count)) + sizeof(ListEntry) * static_cast<size_t>(count);
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

// Partial sums of squares of a list: one per group of tiles.
int64_t list_parts(int64_t tiles) { return (tiles + list_turn(tiles) - 1) / list_turn(tiles); }

uint64_t list_ws_bytes(int64_t tiles)
{
    const int64_t parts = list_parts(tiles);
    return 8 * static_cast<uint64_t>(parts + finish_groups(parts));
}

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

ds_status list_check_args(const ds_scaler* st, const ds_tensor_list* l, const void* ws, size_t ws_bytes)
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
    return DS_OK;
}

// The check's first kernel: the flag, and the partial sums where `part` is given.
ds_status launch_list_check(ds_scaler* st, const ds_tensor_list* l, double* part, hipStream_t s)
{
    const unsigned blocks = grid_blocks(list_parts(l->tiles), kListBlock);
    const unsigned char* table = static_cast<const unsigned char*>(l->table);
    const int32_t tiles = static_cast<int32_t>(l->tiles);
    if (part == nullptr) list_check_kernel<false><<<blocks, kListBlock, 0, s>>>(st, table, l->count, tiles, nullptr);
    else                 list_check_kernel<true><<<blocks, kListBlock, 0, s>>>(st, table, l->count, tiles, part);
    return launched();
}

ds_status list_check(ds_scaler* st, const ds_tensor_list* l, void* ws, size_t ws_bytes, hipStream_t s)
{
    if (const ds_status rc = list_check_args(st, l, ws, ws_bytes); rc != DS_OK)
        return rc;
    if (l->tiles == 0)
        return DS_OK;
    double* part = static_cast<double*>(ws);
    if (const ds_status rc = launch_list_check(st, l, part, s); rc != DS_OK || part == nullptr)
        return rc;
    return launch_finish(st, part, list_parts(l->tiles), s);
}

// What the kernels of one step take.
struct ListLaunch {
    ds_scaler* st;
    const ds_tensor_list* l;
    ListHyper hp;
    const double* part;
    hipStream_t s;
};

template <bool E8, bool DITHER, bool NT, bool FUSE, int FRONT, int U>
void launch_list_step2(const ListLaunch& a)
{
    const unsigned char* table = static_cast<const unsigned char*>(a.l->table);
    uint32_t* tickets = static_cast<uint32_t*>(a.l->table);
    const int32_t tiles = static_cast<int32_t>(a.l->tiles), count = a.l->count;
    const unsigned b = static_cast<unsigned>(tiles) * (kListQuads / U);
    list_step_kernel<E8, DITHER, NT, FUSE, FRONT, U><<<b, kListBlock, 0, a.s>>>(a.st, table, tickets, count, tiles, a.hp, a.part);
}

template <bool NT, bool FUSE, int FRONT, int U>
void launch_list_step(const ListLaunch& a, bool dither)
{
    if (a.l->sdt == DS_FP32) launch_list_step2<false, false, NT, FUSE, FRONT, U>(a);
    else if (dither)         launch_list_step2<true, true, NT, FUSE, FRONT, U>(a);
    else                     launch_list_step2<true, false, NT, FUSE, FRONT, U>(a);
}

template <bool E8, bool DITHER>
void launch_list_adam(const ListLaunch& a, bool end_step, unsigned blocks)
{
    const unsigned char* table = static_cast<const unsigned char*>(a.l->table);
    uint32_t* tickets = static_cast<uint32_t*>(a.l->table);
    const int32_t tiles = static_cast<int32_t>(a.l->tiles), count = a.l->count;
    if (end_step) list_adam_kernel<E8, DITHER, true><<<blocks, kListBlock, 0, a.s>>>(a.st, table, tickets, count, tiles, a.hp);
    else          list_adam_kernel<E8, DITHER, false><<<blocks, kListBlock, 0, a.s>>>(a.st, table, tickets, count, tiles, a.hp);
}

// The kernels' hyperparameters from a call's; false: a schedule that is not one.
bool list_adam_hyper(float lr, const ds_lr_schedule* sched, double beta1, double beta2, float eps, float max_grad_norm,
                     int32_t accum_steps, AdamHyper* hp)
{
    *hp = AdamHyper{lr, static_cast<float>(beta1), static_cast<float>(beta2), eps, 0.0f, max_grad_norm, accum_steps,
                    0, 0.0f, 0, 0};
    if (sched == nullptr)
        return true;
    if (!schedule_ok(*sched))
        return false;
    hp->lr = sched->warmup_max_lr;
    hp->lr_kind = sched->kind;
    hp->lr_min = sched->warmup_min_lr;
    hp->lr_warmup = sched->warmup_num_steps;
    hp->lr_total = sched->total_num_steps;
    return true;
}

bool list_hyper_ok(const AdamHyper& h, double beta1, double beta2, ds_rounding rounding)
{
    return finite_ge0(h.lr) && beta1 >= 0.0 && beta1 < 1.0 && beta2 >= 0.0 && beta2 < 1.0 && std::isfinite(h.eps) &&
           h.eps > 0.0f && finite_ge0(h.max_grad_norm) && h.accum_steps >= 1 &&
           (rounding == DS_ROUND_NEAREST || rounding == DS_ROUND_DITHER);
}

ListHyper list_hyper(const AdamHyper& h, double beta1, double beta2, uint64_t seed)
{
    return ListHyper{h, beta1, beta2, dither_mix(dither_mix(static_cast<uint32_t>(seed >> 32)) ^ static_cast<uint32_t>(seed))};
}

ds_status list_adam(ds_scaler* st, const ds_tensor_list* l, const AdamHyper& h, double beta1, double beta2,
                    ds_rounding rounding, uint64_t seed, bool end_step, hipStream_t s)
{
    if (const ds_status rc = list_ok(l); rc != DS_OK)
        return rc;
    if (!list_hyper_ok(h, beta1, beta2, rounding))
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
    const ListLaunch a{st, l, list_hyper(h, beta1, beta2, seed), nullptr, s};
    const unsigned blocks = grid_blocks(l->tiles, kListBlock);
    const bool e8 = l->sdt != DS_FP32, dither = rounding == DS_ROUND_DITHER;
    if (blocks != l->tiles) {
        if (!e8)         launch_list_adam<false, false>(a, end_step, blocks);
        else if (dither) launch_list_adam<true, true>(a, end_step, blocks);
        else             launch_list_adam<true, false>(a, end_step, blocks);
    } else if (variant_nt(l->elems)) {
        if (end_step) launch_list_step<true, true, kFrontNone, kListQuads>(a, dither);
        else          launch_list_step<true, false, kFrontNone, kListQuads>(a, dither);
    } else {
        if (end_step) launch_list_step<false, true, kFrontNone, kListQuads>(a, dither);
        else          launch_list_step<false, false, kFrontNone, kListQuads>(a, dither);
    }
    return launched();
}

ds_status list_step_all(ds_scaler* st, const ds_tensor_list* l, void* ws, size_t ws_bytes, const AdamHyper& h,
                        double beta1, double beta2, ds_rounding rounding, uint64_t seed, hipStream_t s)
{
    if (const ds_status rc = list_ok(l); rc != DS_OK)
        return rc;
    if (!list_hyper_ok(h, beta1, beta2, rounding))
        return DS_ERR_HPARAM;
    // a pinned grid (DSZERO_GRID) is for the kernels that loop over their tiles
    if (l->tiles < 1 || l->tiles > (ws != nullptr ? kStepParts : kStepQuarter) || env_long("DSZERO_GRID", 0) > 0) {
        if (const ds_status rc = list_check(st, l, ws, ws_bytes, s); rc != DS_OK)
            return rc;
        return list_adam(st, l, h, beta1, beta2, rounding, seed, true, s);
    }
    const bool alone = l->tiles <= kStepCheck;
    if (const ds_status rc = list_check_args(st, l, ws, ws_bytes); rc != DS_OK)
        return rc;
    const bool dither = rounding == DS_ROUND_DITHER;
    const ListLaunch a{st, l, list_hyper(h, beta1, beta2, seed), static_cast<double*>(ws), s};
    if (alone) {
        if (ws == nullptr) launch_list_step<false, true, kFrontCheck, 1>(a, dither);
        else               launch_list_step<false, true, kFrontCheckSum, 1>(a, dither);
        return launched();
    }
    if (const ds_status rc = launch_list_check(st, l, static_cast<double*>(ws), s); rc != DS_OK)
        return rc;
    if (ws == nullptr)                     launch_list_step<false, true, kFrontNone, 1>(a, dither);
    else if (l->tiles <= kStepQuarter)     launch_list_step<false, true, kFrontParts, 1>(a, dither);
    else                                   launch_list_step<false, true, kFrontParts, kListQuads>(a, dither);
    return launched();
}
