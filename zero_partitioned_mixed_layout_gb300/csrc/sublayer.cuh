// Pieces shared by the feed-forward sub-block's translation units
// (norm.cu, ffn.cu): element access at any alignment and the argument
// checks of row-strided matrices.
#pragma once

#include "common.cuh"

// Returns the code of a check or a launch that is not ZERO_OK.
#define ZERO_TRY(call)          \
    do {                        \
        const int rc_ = (call); \
        if (rc_ != ZERO_OK)     \
            return rc_;         \
    } while (0)

namespace zpml {
namespace {

// One element of any type from / to binary32.
template <int DT>
__device__ __forceinline__ float load1(const void *p, int64_t i)
{
    return Elem<DT>::scalar(p, i);
}

template <int DT>
__device__ __forceinline__ void store1(void *p, int64_t i, float v)
{
    if constexpr (DT == ZERO_F32)
        static_cast<float *>(p)[i] = v;
    else
        LowP<DT>::store(p, i, v);
}

// The same with the type known at run time only (weight gradients, whose type
// may differ from the activations').
__device__ __forceinline__ void store1_as(int32_t dt, void *p, int64_t i, float v)
{
    if (dt == ZERO_F32)
        store1<ZERO_F32>(p, i, v);
    else if (dt == ZERO_F16)
        store1<ZERO_F16>(p, i, v);
    else
        store1<ZERO_BF16>(p, i, v);
}

// Division of n < 2^31 by a divisor known at launch: a product and a shift
// (Granlund and Montgomery 1994).
struct FastDiv {
    uint32_t magic, shift;
};

constexpr int64_t kFastDivMost = (int64_t)1 << 31;

inline FastDiv fast_divisor(uint32_t d)
{
    FastDiv f{0, 0};
    while (((uint64_t)1 << f.shift) < d)
        ++f.shift;
    f.magic = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << f.shift) - d)) / d + 1);
    return f;
}

__device__ __forceinline__ uint32_t fast_div(uint32_t n, FastDiv f)
{
    return (uint32_t)(((uint64_t)__umulhi(n, f.magic) + n) >> f.shift);
}

inline int elem_bytes(int32_t dt) { return dt == ZERO_F32 ? 4 : 2; }

// Checks of one array that a call reads or writes: n elements from p on
// (none if n == 0), element-aligned, in device memory.
inline int check_array(const void *p, int64_t n, int32_t dt)
{
    if (n == 0)
        return ZERO_OK;
    if (!p)
        return ZERO_EINVAL;
    if ((reinterpret_cast<uintptr_t>(p) & (uintptr_t)(elem_bytes(dt) - 1)) != 0)
        return ZERO_EALIGN;
    return device_ptr(p) ? ZERO_OK : ZERO_EINVAL;
}

// Checks of a rows x cols matrix with row stride ld.
inline int check_matrix(const void *p, int64_t ld, int64_t rows, int64_t cols, int32_t dt)
{
    if (rows == 0 || cols == 0)
        return ZERO_OK;
    if (ld < cols || ld > ((int64_t)1 << 60) / rows)
        return ZERO_ESIZE;
    return check_array(p, 1, dt);
}

inline int check_workspace(const void *ws, size_t ws_bytes, size_t need)
{
    if (!ws)
        return ZERO_EWORKSPACE;
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
        return ZERO_EALIGN;
    if (ws_bytes < need)
        return ZERO_EWORKSPACE;
    return device_ptr(ws) ? ZERO_OK : ZERO_EINVAL;
}

}  // namespace
}  // namespace zpml
