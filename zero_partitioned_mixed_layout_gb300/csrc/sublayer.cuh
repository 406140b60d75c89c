// Pieces shared by the sub-blocks' translation units (norm.cu, ffn.cu;
// qk_norm.cu, attention.cu): element access at any alignment and the argument
// checks of row-strided matrices and of arrays of heads.
#pragma once

#include <cuda.h>

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

// Two binary32 in one instruction.
struct F2 {
    float x, y;
};

__device__ __forceinline__ unsigned long long bits(F2 a)
{
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
    return r;
}

__device__ __forceinline__ F2 pair(unsigned long long a)
{
    F2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
    return r;
}

__device__ __forceinline__ F2 operator*(F2 a, F2 b)
{
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
    return pair(r);
}

__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
    return pair(r);
}

__device__ __forceinline__ F2 operator+(F2 a, F2 b)
{
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
    return pair(r);
}

__device__ __forceinline__ F2 twice(float a) { return {a, a}; }

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

// The device memory that one call's pointers lie in.  The arrays of a call
// are often slices of one allocation, and the driver takes 0.4 us to say
// what a pointer is, so it is asked for the allocation too, and not again
// for what lies in it.  (Of no longer life than the call.)
class Reach {
public:
    bool has(const void *p)
    {
        const uintptr_t x = reinterpret_cast<uintptr_t>(p);
        for (int i = 0; i < kRanges; ++i)
            if (x - from_[i] < size_[i])
                return true;
        void *from = nullptr;
        size_t size = 0;
        unsigned type = 0;
        CUpointer_attribute what[3] = {CU_POINTER_ATTRIBUTE_MEMORY_TYPE, CU_POINTER_ATTRIBUTE_RANGE_START_ADDR,
                                       CU_POINTER_ATTRIBUTE_RANGE_SIZE};
        void *to[3] = {&type, &from, &size};
        const Query query = driver();
        if (!query || query(3, what, to, (CUdeviceptr)x) != CUDA_SUCCESS || type != CU_MEMORYTYPE_DEVICE ||
            x - reinterpret_cast<uintptr_t>(from) >= size)
            return device_ptr(p);
        from_[next_] = reinterpret_cast<uintptr_t>(from), size_[next_] = size;
        next_ = (next_ + 1) % kRanges;
        return true;
    }

private:
    using Query = CUresult (*)(unsigned, CUpointer_attribute *, void **, CUdeviceptr);
    static Query driver()
    {
        static Query fn = [] {
            void *p = nullptr;
            cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
            if (cudaGetDriverEntryPointByVersion("cuPointerGetAttributes", &p, 12000, cudaEnableDefault, &found) !=
                    cudaSuccess ||
                found != cudaDriverEntryPointSuccess) {
                cudaGetLastError();
                p = nullptr;
            }
            return reinterpret_cast<Query>(p);
        }();
        return fn;
    }
    static constexpr int kRanges = 4;
    uintptr_t from_[kRanges] = {}, size_[kRanges] = {};
    int next_ = 0;
};

// Checks of one array that a call reads or writes: n elements from p on
// (none if n == 0), element-aligned, in device memory.
inline int check_array(const void *p, int64_t n, int32_t dt, Reach *reach = nullptr)
{
    if (n == 0)
        return ZERO_OK;
    if (!p)
        return ZERO_EINVAL;
    if ((reinterpret_cast<uintptr_t>(p) & (uintptr_t)(elem_bytes(dt) - 1)) != 0)
        return ZERO_EALIGN;
    return (reach ? reach->has(p) : device_ptr(p)) ? ZERO_OK : ZERO_EINVAL;
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

// An array of heads: tokens x heads x head_dim, the elements of a head
// contiguous.
struct Heads {
    const void *p;
    int64_t ld, hd;  // elements from a token, from a head, to the next
};

// Checks of one; the strides that no two rows need become 0.
inline int check_heads(Heads *a, int64_t tokens, int64_t heads, int64_t dim, int32_t dt, Reach *reach)
{
    if (tokens == 0 || heads == 0 || dim == 0)
        return ZERO_OK;
    if (tokens == 1)
        a->ld = 0;
    if (heads == 1)
        a->hd = 0;
    if (a->ld < 0 || a->hd < 0)
        return ZERO_EINVAL;
    // offsets stay below 2^61, and a tensor map's strides below 2^40 bytes
    const int64_t most = (int64_t)1 << 38, all = (int64_t)1 << 60;
    if (a->ld >= most || a->hd >= most || a->ld > all / tokens || a->hd > all / heads)
        return ZERO_ESIZE;
    return check_array(a->p, 1, dt, reach);
}

inline int check_workspace(const void *ws, size_t ws_bytes, size_t need, Reach *reach = nullptr)
{
    if (!ws)
        return ZERO_EWORKSPACE;
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
        return ZERO_EALIGN;
    if (ws_bytes < need)
        return ZERO_EWORKSPACE;
    return (reach ? reach->has(ws) : device_ptr(ws)) ? ZERO_OK : ZERO_EINVAL;
}

}  // namespace
}  // namespace zpml
