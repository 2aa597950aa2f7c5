// lanes.h -- reductions over rows of 8, 16 or 32 lanes.
// Included by dszero.hip inside its namespace.

// x of the lane 1, 2, 4, 8 or 16 lanes apart by xor; for 4 and 8 of a mirrored
// one, which holds the same where every four (eight) lanes hold the same, as
// after the smaller steps of the reductions below.  Every lane is active.
template <int OFF>
__device__ __forceinline__ uint32_t row_other(uint32_t x)
{
    static_assert(OFF == 1 || OFF == 2 || OFF == 4 || OFF == 8 || OFF == 16, "inside 32 lanes");
    if constexpr (OFF == 16) {
        return __shfl_xor(x, 16);
    } else {
        constexpr int kCtrl = OFF == 1 ? 0xB1 : OFF == 2 ? 0x4E : OFF == 4 ? 0x141 : 0x140;
        return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), kCtrl, 0xF, 0xF, true));
    }
}

template <int OFF>
__device__ __forceinline__ float row_other(float x)
{
    return __uint_as_float(row_other<OFF>(__float_as_uint(x)));
}

template <int G>
__device__ __forceinline__ float row_max(float x)
{
    x = fmaxf(x, row_other<1>(x));
    x = fmaxf(x, row_other<2>(x));
    x = fmaxf(x, row_other<4>(x));
    if constexpr (G > 8)
        x = fmaxf(x, row_other<8>(x));
    if constexpr (G > 16)
        x = fmaxf(x, row_other<16>(x));
    return x;
}

template <int G>
__device__ __forceinline__ float row_sum(float x)
{
    x = x + row_other<1>(x);
    x = x + row_other<2>(x);
    x = x + row_other<4>(x);
    if constexpr (G > 8)
        x = x + row_other<8>(x);
    if constexpr (G > 16)
        x = x + row_other<16>(x);
    return x;
}

template <int G>
__device__ __forceinline__ int row_sum_int(uint32_t x)
{
    x = x + row_other<1>(x);
    x = x + row_other<2>(x);
    x = x + row_other<4>(x);
    if constexpr (G > 8)
        x = x + row_other<8>(x);
    if constexpr (G > 16)
        x = x + row_other<16>(x);
    return static_cast<int>(x);
}

template <int G>
__device__ __forceinline__ int row_max_int(int x)
{
    x = max(x, static_cast<int>(row_other<1>(static_cast<uint32_t>(x))));
    x = max(x, static_cast<int>(row_other<2>(static_cast<uint32_t>(x))));
    x = max(x, static_cast<int>(row_other<4>(static_cast<uint32_t>(x))));
    if constexpr (G > 8)
        x = max(x, static_cast<int>(row_other<8>(static_cast<uint32_t>(x))));
    if constexpr (G > 16)
        x = max(x, static_cast<int>(row_other<16>(static_cast<uint32_t>(x))));
    return x;
}

// x of the lane 8 away in the row of 16 lanes (a rotation by 8).
__device__ __forceinline__ uint32_t row_half(uint32_t x)
{
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0x128, 0xF, 0xF, true));
}

__device__ __forceinline__ float row_half(float x) { return __uint_as_float(row_half(__float_as_uint(x))); }

__device__ __forceinline__ int row_half(int x) { return static_cast<int>(row_half(static_cast<uint32_t>(x))); }
