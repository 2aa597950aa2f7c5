// lanes.h -- reductions over rows of 8 or 16 lanes without shared memory.
// Included by dszero.hip inside its namespace.

// x of the lane 1, 2, 4 or 8 lanes apart by xor; for 4 and 8 of a mirrored
// one, which holds the same where every four (eight) lanes hold the same, as
// after the smaller steps of the reductions below.  Every lane is active.
template <int OFF>
__device__ __forceinline__ uint32_t row_other(uint32_t x)
{
    constexpr int kCtrl = OFF == 1 ? 0xB1 : OFF == 2 ? 0x4E : OFF == 4 ? 0x141 : 0x140;
    static_assert(OFF == 1 || OFF == 2 || OFF == 4 || OFF == 8, "inside 16 lanes");
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), kCtrl, 0xF, 0xF, true));
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
    if constexpr (G == 16)
        x = fmaxf(x, row_other<8>(x));
    return x;
}

template <int G>
__device__ __forceinline__ float row_sum(float x)
{
    x = x + row_other<1>(x);
    x = x + row_other<2>(x);
    x = x + row_other<4>(x);
    if constexpr (G == 16)
        x = x + row_other<8>(x);
    return x;
}

template <int G>
__device__ __forceinline__ int row_sum_int(uint32_t x)
{
    x = x + row_other<1>(x);
    x = x + row_other<2>(x);
    x = x + row_other<4>(x);
    if constexpr (G == 16)
        x = x + row_other<8>(x);
    return static_cast<int>(x);
}
