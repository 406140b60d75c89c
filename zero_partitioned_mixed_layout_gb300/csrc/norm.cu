// Dropout with the residual sum, and layer norm (alone or with that sum in
// front of it), forward and backward.
#include <cmath>

#include "sublayer.cuh"

namespace zpml {
namespace {

// ------------------------------------------------------------- the mask

// Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", 2011): ten rounds of two 32 x 32 -> 64 bit products on a
// 128-bit counter, the key moved on by a constant per round.
__device__ __forceinline__ uint4 philox4x32_10(uint4 c, uint32_t k0, uint32_t k1)
{
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)0xD2511F53u * c.x, b = (uint64_t)0xCD9E8D57u * c.z;
        c = make_uint4((uint32_t)(b >> 32) ^ c.y ^ k0, (uint32_t)b, (uint32_t)(a >> 32) ^ c.w ^ k1, (uint32_t)a);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return c;
}

// A dropout as the kernels take it.
struct Drop {
    const uint64_t *d_offset;
    uint64_t offset;
    uint32_t k0, k1;
    uint32_t threshold;  // kept iff the word is at least this ...
    uint32_t all;        // ... and not everything is dropped (p = 1)
    float scale;
};

__device__ __forceinline__ uint64_t drop_offset(const Drop &d)
{
    return d.d_offset ? d.offset + *d.d_offset : d.offset;
}

// Whether word w of a counter keeps its element.
__device__ __forceinline__ bool kept(const Drop &d, uint32_t w) { return w >= d.threshold && !d.all; }

__device__ __forceinline__ uint4 drop_words(const Drop &d, uint64_t off, int64_t row, int64_t col)
{
    return philox4x32_10(make_uint4((uint32_t)(col >> 2), (uint32_t)row, (uint32_t)off, (uint32_t)(off >> 32)), d.k0,
                         d.k1);
}

__device__ __forceinline__ uint32_t word_of(const uint4 &w, int k)
{
    return k == 0 ? w.x : k == 1 ? w.y : k == 2 ? w.z : w.w;
}

// ------------------------------------------------------------- kernels

struct Matrix {
    void *p;
    int64_t ld;
};

// One thread per four columns (one counter).
template <int DT>
__global__ void __launch_bounds__(kThreads) k_dropout_add(Matrix x, Matrix res, Matrix out, int64_t rows, int64_t cols,
                                                          Drop d)
{
    const int64_t quads = (cols + 3) >> 2, n = rows * quads;
    const uint64_t off = drop_offset(d);
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
        const int64_t r = i / quads, c = (i - r * quads) * 4;
        const uint4 w = drop_words(d, off, r, c);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (c + k < cols) {
                float v = kept(d, word_of(w, k)) ? load1<DT>(x.p, r * x.ld + c + k) * d.scale : 0.0f;
                if (res.p)
                    v += load1<DT>(res.p, r * res.ld + c + k);
                store1<DT>(out.p, r * out.ld + c + k, v);
            }
    }
}

__device__ __forceinline__ float block_sum(float v)
{
    __shared__ float s[kWarps];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k)
        v += s[k];
    return v;
}

struct NormArgs {
    Matrix x, res, sum, y;
    const void *weight, *bias;
    int32_t wdtype;
    float *mean, *rstd;
    int64_t rows, cols;
    float eps;
    int32_t dropping;
    Drop d;
};

// The value of element (r, c) of the normed matrix, before its rounding.
template <int DT>
__device__ __forceinline__ float norm_input(const NormArgs &a, uint64_t off, int64_t r, int64_t c)
{
    float v = load1<DT>(a.x.p, r * a.x.ld + c);
    if (a.dropping)
        v = kept(a.d, word_of(drop_words(a.d, off, r, c), c & 3)) ? v * a.d.scale : 0.0f;
    if (a.res.p)
        v += load1<DT>(a.res.p, r * a.res.ld + c);
    return v;
}

// One block per row, three passes over it.
template <int DT>
__global__ void __launch_bounds__(kThreads) k_norm_fwd(NormArgs a)
{
    const uint64_t off = a.dropping ? drop_offset(a.d) : 0;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        float s = 0.0f;
        for (int64_t c = threadIdx.x; c < a.cols; c += kThreads)
            s += norm_input<DT>(a, off, r, c);
        const float mean = block_sum(s) / (float)a.cols;
        s = 0.0f;
        for (int64_t c = threadIdx.x; c < a.cols; c += kThreads) {
            const float t = norm_input<DT>(a, off, r, c) - mean;
            s += t * t;
        }
        const float rstd = 1.0f / sqrtf(block_sum(s) / (float)a.cols + a.eps);
        for (int64_t c = threadIdx.x; c < a.cols; c += kThreads) {
            const float t = norm_input<DT>(a, off, r, c);
            float y = (t - mean) * rstd;
            if (a.weight)
                y *= load1_as(a.wdtype, a.weight, c);
            if (a.bias)
                y += load1_as(a.wdtype, a.bias, c);
            if (a.sum.p)
                store1<DT>(a.sum.p, r * a.sum.ld + c, t);
            store1<DT>(a.y.p, r * a.y.ld + c, y);
        }
        if (threadIdx.x == 0) {
            if (a.mean)
                a.mean[r] = mean;
            if (a.rstd)
                a.rstd[r] = rstd;
        }
    }
}

struct NormBwdArgs {
    Matrix dy, x, dres, dx, dropped;
    const void *weight;
    int32_t wdtype, gdtype;
    const float *mean, *rstd;
    void *dweight, *dbias;
    int64_t rows, cols;
    int32_t dropping;
    Drop d;
};

template <int DT>
__global__ void __launch_bounds__(kThreads) k_norm_bwd_rows(NormBwdArgs a)
{
    const uint64_t off = a.dropping ? drop_offset(a.d) : 0;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const float mean = a.mean[r], rstd = a.rstd[r];
        float s0 = 0.0f, s1 = 0.0f;
        for (int64_t c = threadIdx.x; c < a.cols; c += kThreads) {
            float g = load1<DT>(a.dy.p, r * a.dy.ld + c);
            if (a.weight)
                g *= load1_as(a.wdtype, a.weight, c);
            s0 += g;
            s1 += g * ((load1<DT>(a.x.p, r * a.x.ld + c) - mean) * rstd);
        }
        s0 = block_sum(s0) / (float)a.cols;
        s1 = block_sum(s1) / (float)a.cols;
        for (int64_t c = threadIdx.x; c < a.cols; c += kThreads) {
            float g = load1<DT>(a.dy.p, r * a.dy.ld + c);
            if (a.weight)
                g *= load1_as(a.wdtype, a.weight, c);
            const float xh = (load1<DT>(a.x.p, r * a.x.ld + c) - mean) * rstd;
            float v = rstd * (g - s0 - xh * s1);
            if (a.dres.p)
                v += load1<DT>(a.dres.p, r * a.dres.ld + c);
            store1<DT>(a.dx.p, r * a.dx.ld + c, v);
            if (a.dropping)
                store1<DT>(a.dropped.p, r * a.dropped.ld + c,
                           kept(a.d, word_of(drop_words(a.d, off, r, c), c & 3)) ? v * a.d.scale : 0.0f);
        }
    }
}

// dweight and dbias: a block takes 32 columns, its 8 warps the rows in turn.
template <int DT>
__global__ void __launch_bounds__(kThreads) k_norm_bwd_cols(NormBwdArgs a)
{
    __shared__ float sw[kWarps][32], sb[kWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float w = 0.0f, b = 0.0f;
    if (c < a.cols)
        for (int64_t r = warp; r < a.rows; r += kWarps) {
            const float dy = load1<DT>(a.dy.p, r * a.dy.ld + c);
            w += dy * ((load1<DT>(a.x.p, r * a.x.ld + c) - a.mean[r]) * a.rstd[r]);
            b += dy;
        }
    sw[warp][lane] = w;
    sb[warp][lane] = b;
    __syncthreads();
    if (warp == 0 && c < a.cols) {
#pragma unroll
        for (int k = 1; k < kWarps; ++k) {
            w += sw[k][lane];
            b += sb[k][lane];
        }
        if (a.dweight)
            store1_as(a.gdtype, a.dweight, c, w);
        if (a.dbias)
            store1_as(a.gdtype, a.dbias, c, b);
    }
}

// ------------------------------------------------------------- host side

// The kernels' form of a dropout (NULL: none).
int drop_args(const zero_dropout_t *drop, Drop *d)
{
    *d = Drop{};
    if (!drop)
        return ZERO_OK;
    if (!(drop->p >= 0.0 && drop->p <= 1.0))
        return ZERO_EINVAL;
    if (drop->d_offset) {
        if ((reinterpret_cast<uintptr_t>(drop->d_offset) & 7u) != 0)
            return ZERO_EALIGN;
        if (!device_ptr(drop->d_offset))
            return ZERO_EINVAL;
    }
    const uint64_t t = (uint64_t)std::floor(drop->p * 4294967296.0 + 0.5);
    d->d_offset = drop->d_offset;
    d->offset = drop->offset;
    d->k0 = (uint32_t)drop->seed;
    d->k1 = (uint32_t)(drop->seed >> 32);
    d->all = t > 0xffffffffu;
    d->threshold = (uint32_t)t;
    d->scale = drop->p < 1.0 ? (float)(1.0 / (1.0 - drop->p)) : 0.0f;
    return ZERO_OK;
}

int check_sizes(int64_t rows, int64_t cols)
{
    if (rows < 0 || cols < 0)
        return ZERO_EINVAL;
    if (rows >= ((int64_t)1 << 32) || cols > ((int64_t)1 << 34))
        return ZERO_ESIZE;
    return ZERO_OK;
}

Matrix matrix(const void *p, int64_t ld) { return {const_cast<void *>(p), ld}; }

unsigned grid_rows(int64_t rows) { return (unsigned)(rows < 65535 * 16 ? rows : 65535 * 16); }

}  // namespace
}  // namespace zpml

using namespace zpml;

extern "C" int zero_dropout_add(const void *x, int64_t x_ld, const void *residual, int64_t residual_ld, void *out,
                                int64_t out_ld, int64_t rows, int64_t cols, int32_t dtype, const zero_dropout_t *drop,
                                void *stream)
{
    if (!drop)
        return ZERO_EINVAL;
    if (!grad_dtype_ok(dtype))
        return ZERO_EDTYPE;
    ZERO_TRY(check_sizes(rows, cols));
    Drop d;
    ZERO_TRY(drop_args(drop, &d));
    ZERO_TRY(check_matrix(x, x_ld, rows, cols, dtype));
    if (residual)
        ZERO_TRY(check_matrix(residual, residual_ld, rows, cols, dtype));
    ZERO_TRY(check_matrix(out, out_ld, rows, cols, dtype));
    if (rows == 0 || cols == 0)
        return ZERO_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int64_t n = rows * ((cols + 3) / 4), blocks = (n + kThreads - 1) / kThreads, most = (int64_t)sm_count() * 8;
    const unsigned grid = (unsigned)(blocks < most ? blocks : most);
    const Matrix mx = matrix(x, x_ld), mr = matrix(residual, residual_ld), mo = matrix(out, out_ld);
    if (dtype == ZERO_F16)
        k_dropout_add<ZERO_F16><<<grid, kThreads, 0, st>>>(mx, mr, mo, rows, cols, d);
    else if (dtype == ZERO_BF16)
        k_dropout_add<ZERO_BF16><<<grid, kThreads, 0, st>>>(mx, mr, mo, rows, cols, d);
    else
        k_dropout_add<ZERO_F32><<<grid, kThreads, 0, st>>>(mx, mr, mo, rows, cols, d);
    return check_launch("k_dropout_add");
}

extern "C" int zero_layer_norm(const void *x, int64_t x_ld, const void *residual, int64_t residual_ld,
                               const zero_dropout_t *drop, void *sum, int64_t sum_ld, const void *weight,
                               const void *bias, int32_t wdtype, void *y, int64_t y_ld, float *mean, float *rstd,
                               int64_t rows, int64_t cols, double eps, int32_t dtype, void *stream)
{
    if (!grad_dtype_ok(dtype) || ((weight || bias) && wdtype != dtype && wdtype != ZERO_F32))
        return ZERO_EDTYPE;
    ZERO_TRY(check_sizes(rows, cols));
    if (!(eps >= 0.0) || ((residual || drop) && !sum && rows > 0 && cols > 0) || (sum && !residual && !drop))
        return ZERO_EINVAL;
    NormArgs a{};
    ZERO_TRY(drop_args(drop, &a.d));
    ZERO_TRY(check_matrix(x, x_ld, rows, cols, dtype));
    if (residual)
        ZERO_TRY(check_matrix(residual, residual_ld, rows, cols, dtype));
    if (sum)
        ZERO_TRY(check_matrix(sum, sum_ld, rows, cols, dtype));
    ZERO_TRY(check_matrix(y, y_ld, rows, cols, dtype));
    if (weight)
        ZERO_TRY(check_array(weight, cols, wdtype));
    if (bias)
        ZERO_TRY(check_array(bias, cols, wdtype));
    if (mean)
        ZERO_TRY(check_array(mean, rows, ZERO_F32));
    if (rstd)
        ZERO_TRY(check_array(rstd, rows, ZERO_F32));
    if (rows == 0 || cols == 0)
        return ZERO_OK;
    a.x = matrix(x, x_ld), a.res = matrix(residual, residual_ld), a.sum = matrix(sum, sum_ld), a.y = matrix(y, y_ld);
    a.weight = weight, a.bias = bias, a.wdtype = wdtype, a.mean = mean, a.rstd = rstd;
    a.rows = rows, a.cols = cols, a.eps = (float)eps, a.dropping = drop != nullptr;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const unsigned grid = grid_rows(rows);
    if (dtype == ZERO_F16)
        k_norm_fwd<ZERO_F16><<<grid, kThreads, 0, st>>>(a);
    else if (dtype == ZERO_BF16)
        k_norm_fwd<ZERO_BF16><<<grid, kThreads, 0, st>>>(a);
    else
        k_norm_fwd<ZERO_F32><<<grid, kThreads, 0, st>>>(a);
    return check_launch("k_norm_fwd");
}

extern "C" size_t zero_layer_norm_workspace_bytes(int64_t rows, int64_t cols)
{
    (void)rows;
    (void)cols;
    return 256;
}

extern "C" int zero_layer_norm_backward(const void *dy, int64_t dy_ld, const void *x, int64_t x_ld,
                                        const void *weight, int32_t wdtype, const float *mean, const float *rstd,
                                        const void *dresidual, int64_t dresidual_ld, void *dx, int64_t dx_ld,
                                        const zero_dropout_t *drop, void *dropped, int64_t dropped_ld, void *dweight,
                                        void *dbias, int32_t gdtype, int64_t rows, int64_t cols, int32_t dtype,
                                        void *ws, size_t ws_bytes, void *stream)
{
    if (!grad_dtype_ok(dtype) || (weight && wdtype != dtype && wdtype != ZERO_F32) ||
        ((dweight || dbias) && gdtype != dtype && gdtype != ZERO_F32))
        return ZERO_EDTYPE;
    ZERO_TRY(check_sizes(rows, cols));
    if (rows > 0 && cols > 0 && (drop != nullptr) != (dropped != nullptr))
        return ZERO_EINVAL;
    NormBwdArgs a{};
    ZERO_TRY(drop_args(drop, &a.d));
    ZERO_TRY(check_matrix(dy, dy_ld, rows, cols, dtype));
    ZERO_TRY(check_matrix(x, x_ld, rows, cols, dtype));
    if (dresidual)
        ZERO_TRY(check_matrix(dresidual, dresidual_ld, rows, cols, dtype));
    ZERO_TRY(check_matrix(dx, dx_ld, rows, cols, dtype));
    if (drop)
        ZERO_TRY(check_matrix(dropped, dropped_ld, rows, cols, dtype));
    if (weight)
        ZERO_TRY(check_array(weight, cols, wdtype));
    if (cols > 0) {
        ZERO_TRY(check_array(mean, rows, ZERO_F32));
        ZERO_TRY(check_array(rstd, rows, ZERO_F32));
    }
    if (dweight)
        ZERO_TRY(check_array(dweight, cols, gdtype));
    if (dbias)
        ZERO_TRY(check_array(dbias, cols, gdtype));
    ZERO_TRY(check_workspace(ws, ws_bytes, zero_layer_norm_workspace_bytes(rows, cols)));
    if (cols == 0)
        return ZERO_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    a.dy = matrix(dy, dy_ld), a.x = matrix(x, x_ld), a.dres = matrix(dresidual, dresidual_ld);
    a.dx = matrix(dx, dx_ld), a.dropped = matrix(dropped, dropped_ld);
    a.weight = weight, a.wdtype = wdtype, a.gdtype = gdtype, a.mean = mean, a.rstd = rstd;
    a.dweight = dweight, a.dbias = dbias, a.rows = rows, a.cols = cols, a.dropping = drop != nullptr;
    const unsigned grid = grid_rows(rows), cgrid = (unsigned)((cols + 31) / 32);
    if (rows > 0) {
        if (dtype == ZERO_F16)
            k_norm_bwd_rows<ZERO_F16><<<grid, kThreads, 0, st>>>(a);
        else if (dtype == ZERO_BF16)
            k_norm_bwd_rows<ZERO_BF16><<<grid, kThreads, 0, st>>>(a);
        else
            k_norm_bwd_rows<ZERO_F32><<<grid, kThreads, 0, st>>>(a);
        ZERO_TRY(check_launch("k_norm_bwd_rows"));
    }
    if (!dweight && !dbias)
        return ZERO_OK;
    if (dtype == ZERO_F16)
        k_norm_bwd_cols<ZERO_F16><<<cgrid, kThreads, 0, st>>>(a);
    else if (dtype == ZERO_BF16)
        k_norm_bwd_cols<ZERO_BF16><<<cgrid, kThreads, 0, st>>>(a);
    else
        k_norm_bwd_cols<ZERO_F32><<<cgrid, kThreads, 0, st>>>(a);
    return check_launch("k_norm_bwd_cols");
}
