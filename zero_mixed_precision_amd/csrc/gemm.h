// gemm.h -- 16-bit matrix products with fp32 sums on the matrix cores, for the
// kernels that fuse something into the product's end.  Included by dszero.hip
// inside its namespace.
//
//   C[m][n] = sum_k A(m, k) B(n, k)
//
// A block has a tile of BM x BN, a wave WM x WN of it, in 32x32x16 products.
// Either operand lies in memory with k inside a row ("by rows": row m, k
// adjacent) or with k as the row ("by columns": row k, m adjacent).  Tiles of 64
// k go to LDS as they lie in memory, by loads that write there directly (16
// bytes a lane, two tiles in turn).  Fragments by rows are read as 16 bytes, 8 k
// of a row; those by columns with the transposing read, 4 k of 16 columns at a
// time.  LDS holds 16-byte pieces at places permuted within their row, so that
// the lanes of one read meet different banks.
//
// Callers keep every access in bounds by clamping: rows and columns past the
// operand's end repeat its last ones (their results are not stored), and k past
// its end meets zeros in the other operand.

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t lds_u32 __attribute__((address_space(3)));

constexpr int kBK = 64;

// One operand of a tile.  By rows: `base` is row 0 of the tile, `limit` the rows
// that exist from there.  By columns: `base` is the tile's first column of k row
// 0, `limit` the columns that exist from there (a multiple of 8), `k_rows` the k
// rows that exist.
struct Operand {
    const uint16_t* base;
    int64_t stride;
    int32_t limit, k_rows;
};

// 16 bytes a lane from base + voff to LDS at lds_at + 16 lane.  The wait state
// after m0 is what loads to LDS ask for.  Written in assembly because the
// compiler would have every LDS read behind such a load wait for it, the reads of
// the other tile too; m0 is set here each time and kept for nothing else.
__device__ __forceinline__ void load_to_lds(uint32_t lds_at, uint32_t voff, const void* base)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(lds_at), "v"(voff), "s"(base)
                 : "memory");
}

__device__ __forceinline__ void loads_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

template <int FMT>
__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c)
{
    if constexpr (FMT == kBF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// The part of an operand's tile that one wave loads and reads.  BR: rows of the
// tile (by rows) or columns (by columns).
template <int BR, bool COLS, int WAVES>
struct TileOf {
    static constexpr int kBytes = BR * kBK * 2;
    static constexpr int kLoads = kBytes / (1024 * WAVES);     // of 1 KiB, per wave
    static_assert(kLoads * 1024 * WAVES == kBytes, "whole loads");
    static constexpr int kRowBytes = COLS ? BR * 2 : kBK * 2;
    static constexpr int kPieces = kRowBytes / 16;             // per row in LDS

    // The permutation of a row's pieces: 16 lanes that read one after another
    // meet all 64 banks (no conflict counted in either form).
    static __device__ __forceinline__ int mix(int row)
    {
        static_assert(kPieces >= 8, "what the permutations move");
        return !COLS ? (row >> 1) & 7 : kPieces >= 16 ? (row & 3) << 2 : (row & 3) << 1;
    }

    uint32_t voff[kLoads];

    // Offsets of this lane's pieces from the tile's first byte; rows: the k rows
    // left (by columns), so that the last tile of k repeats its last row.
    __device__ __forceinline__ void place(const Operand& o, int wave, int lane, int rows)
    {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int at = (i * WAVES + wave) * 64 + lane;     // piece of the tile
            int row = at / kPieces;
            int piece = (at % kPieces) ^ mix(row);
            if constexpr (COLS) {
                row = min(row, rows - 1);
                piece = min(piece, o.limit / 8 - 1);
            } else {
                row = min(row, o.limit - 1);
            }
            voff[i] = static_cast<uint32_t>(row * o.stride * 2 + piece * 16);
        }
    }

    __device__ __forceinline__ void load(uint32_t lds, const uint16_t* base, int wave) const
    {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            load_to_lds(lds + (i * WAVES + wave) * 1024, voff[i], base);
    }

    // Fragment `i` (32 rows from `first`) of k step kk: rows lane % 32, k 8 (lane / 32) .. + 7.
    static __device__ __forceinline__ u32x4 frag(const unsigned char* lds, int first, int i, int kk, int lane)
    {
        if constexpr (COLS) {
            const int k = kk * 16 + 8 * (lane / 32) + (lane % 16) / 4;
            const int col = first + i * 32 + 16 * ((lane / 16) % 2) + 4 * (lane % 4);
            const int at = k * kRowBytes + (((col >> 3) ^ mix(k)) << 4) + (col & 4) * 2;
            auto* p = (__attribute__((address_space(3))) s16x4*)(lds + at);
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(p);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) s16x4*)(lds + at + 4 * kRowBytes));
            const u32x2 a = __builtin_bit_cast(u32x2, lo), b = __builtin_bit_cast(u32x2, hi);
            return u32x4{a.x, a.y, b.x, b.y};
        } else {
            const int row = first + i * 32 + lane % 32;
            const int piece = (kk * 2 + lane / 32) ^ mix(row);
            return *reinterpret_cast<const u32x4*>(lds + row * kRowBytes + piece * 16);
        }
    }
};

template <int FMT, bool AC, bool BC, int BM_, int BN_, int WM_, int WN_>
struct Product {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
    static constexpr int kWavesM = BM / WM, kWavesN = BN / WN, kWaves = kWavesM * kWavesN, kThreads = kWaves * 64;
    static constexpr int MI = WM / 32, NI = WN / 32;
    using TA = TileOf<BM, AC, kWaves>;
    using TB = TileOf<BN, BC, kWaves>;
    static constexpr int kStage = TA::kBytes + TB::kBytes, kLds = 2 * kStage;

    int lane, wave, wm, wn;                // this wave's first row and column in the tile
    f32x16 acc[MI][NI];

    __device__ __forceinline__ Product()
    {
        lane = static_cast<int>(__lane_id());
        wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / 64);
        wm = wave % kWavesM * WM;
        wn = wave / kWavesM * WN;
    }

    // Row m of the wave's accumulator register r of fragment i.
    __device__ __forceinline__ int row(int i, int r) const { return wm + 32 * i + 8 * (r / 4) + 4 * (lane / 32) + r % 4; }
    __device__ __forceinline__ int col(int j) const { return wn + 32 * j + lane % 32; }

    // k: the length of the sum, in tiles of 64.
    __device__ __forceinline__ void run(unsigned char* lds, Operand a, Operand b, int ktiles)
    {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j)
                acc[i][j] = f32x16{};
        const uint32_t at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
            (__attribute__((address_space(3))) unsigned char*)lds));
        TA ta;
        TB tb;
        ta.place(a, wave, lane, min(kBK, a.k_rows));
        tb.place(b, wave, lane, min(kBK, b.k_rows));
        const uint16_t *pa = a.base, *pb = b.base;
        auto load = [&](int kt, uint32_t stage) {
            if constexpr (AC)
                if (kt > 0 && (kt + 1) * kBK > a.k_rows)
                    ta.place(a, wave, lane, a.k_rows - kt * kBK);
            if constexpr (BC)
                if (kt > 0 && (kt + 1) * kBK > b.k_rows)
                    tb.place(b, wave, lane, b.k_rows - kt * kBK);
            ta.load(at + stage, pa, wave);
            tb.load(at + stage + TA::kBytes, pb, wave);
            pa += AC ? kBK * a.stride : kBK;
            pb += BC ? kBK * b.stride : kBK;
        };
        if (ktiles <= 0)
            return;
        load(0, 0);
        loads_done();
        __syncthreads();
        if constexpr (kWaves == 8)
            in_turns(lds, load, ktiles);
        else
            in_step(lds, load, ktiles);
        __syncthreads();
    }

    // A SIMD has two waves, one of either half.  The halves take turns: one reads
    // its fragments of 32 k (and sends off the next tile's loads), the other
    // multiplies; all meet behind each turn, the second half one turn behind.  A
    // tile's place is free once the second half has read its last fragments, in the
    // turn before the first half sends off the loads that go there; at that turn's
    // end either half has also waited for its own loads of the next tile, so that
    // both may read it.  Rows and rows 32768 x 4096 x 4096 / columns and rows 4096 x
    // 8192 x 16384 / columns 4096 x 16384 x 8192 reach 1110 / 1260 / 1230 TFLOP/s,
    // 1075 / 1180 / 1190 with all waves in step, 1300 to 1490 with the loads of all
    // tiles but the first left out; the cross entropy of 8192 x 131072 x 4096 takes
    // 28.4 ms, 29.5 in step.  Turns of 16 k gain nothing over in step.
    template <typename Load>
    __device__ __forceinline__ void in_turns(const unsigned char* lds, Load load, int ktiles)
    {
        constexpr int kSteps = 2;                              // of 16 k, in a turn
        const bool second = wave >= kWaves / 2;
        auto meet = [] {
            __builtin_amdgcn_sched_barrier(0);
            asm volatile("s_barrier" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
        };
        if (second)
            meet();
        uint32_t now = 0;
        for (int kt = 0; kt < ktiles; ++kt) {
            const unsigned char* la = lds + now;
            const unsigned char* lb = la + TA::kBytes;
#pragma unroll
            for (int kk = 0; kk < kBK / 16; kk += kSteps) {
                constexpr int kLast = kBK / 16 - kSteps;
                u32x4 fa[kSteps][MI], fb[kSteps][NI];
#pragma unroll
                for (int h = 0; h < kSteps; ++h) {
#pragma unroll
                    for (int i = 0; i < MI; ++i)
                        fa[h][i] = TA::frag(la, wm, i, kk + h, lane);
#pragma unroll
                    for (int j = 0; j < NI; ++j)
                        fb[h][j] = TB::frag(lb, wn, j, kk + h, lane);
                }
                if (kk == 0 && kt + 1 < ktiles)
                    load(kt + 1, now ^ kStage);
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                if (kk == kLast && second)
                    loads_done();
                meet();
                __builtin_amdgcn_s_setprio(1);
#pragma unroll
                for (int h = 0; h < kSteps; ++h)
#pragma unroll
                    for (int i = 0; i < MI; ++i)
#pragma unroll
                        for (int j = 0; j < NI; ++j)
                            acc[i][j] = mfma32<FMT>(fa[h][i], fb[h][j], acc[i][j]);
                __builtin_amdgcn_s_setprio(0);
                if (kk == kLast && !second)
                    loads_done();
                meet();
            }
            now ^= kStage;
        }
        if (!second)
            meet();
    }

    // One wave of the block on a SIMD, which has nobody to take turns with: it reads
    // the next fragments while the matrix cores have the last ones.
    template <typename Load>
    __device__ __forceinline__ void in_step(const unsigned char* lds, Load load, int ktiles)
    {
        if (ktiles > 1)
            load(1, kStage);
        u32x4 fa[2][MI], fb[2][NI];
        auto read = [&](uint32_t stage, int kk, int to) {
            const unsigned char* la = lds + stage;
            const unsigned char* lb = la + TA::kBytes;
#pragma unroll
            for (int i = 0; i < MI; ++i)
                fa[to][i] = TA::frag(la, wm, i, kk, lane);
#pragma unroll
            for (int j = 0; j < NI; ++j)
                fb[to][j] = TB::frag(lb, wn, j, kk, lane);
        };
        read(0, 0, 0);
        uint32_t now = 0;
        for (int kt = 0; kt < ktiles; ++kt) {
#pragma unroll
            for (int kk = 0; kk < kBK / 16; ++kk) {
                // the next fragments, while the matrix cores have the last ones; behind a tile's last, all waves
                // have read it, and its place takes the tile after the next
                if (kk + 1 < kBK / 16) {
                    read(now, kk + 1, (kk + 1) & 1);
                } else if (kt + 1 < ktiles) {
                    loads_done();
                    __syncthreads();
                    if (kt + 2 < ktiles)
                        load(kt + 2, now);
                    read(now ^ kStage, 0, 0);
                }
#pragma unroll
                for (int i = 0; i < MI; ++i)
#pragma unroll
                    for (int j = 0; j < NI; ++j)
                        acc[i][j] = mfma32<FMT>(fa[kk & 1][i], fb[kk & 1][j], acc[i][j]);
            }
            now ^= kStage;
        }
    }
};

// Tile of the block: consecutive blocks go to the 8 XCDs in turn, so each XCD
// gets a run of tiles of its own; runs go through groups of kGroupM tiles of m
// for every tile of n, so that what they share stays in the XCD's L2.
constexpr int kXcds = 8, kGroupM = 8;
__device__ __forceinline__ void tile_of(int block, int tm, int tn, int& m, int& n)
{
    const int total = tm * tn, each = total / kXcds, more = total % kXcds;
    const int xcd = block % kXcds, nth = block / kXcds;
    const int id = xcd * each + min(xcd, more) + nth;
    const int group = id / (kGroupM * tn), first = group * kGroupM;
    const int height = min(kGroupM, tm - first), in = id - first * tn;
    m = first + in % height;
    n = in / height;
}
