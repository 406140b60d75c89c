// Dropout with the residual sum, and layer norm (alone or with that sum in
// front of it), forward and backward.
#include <cmath>
#include <initializer_list>

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

// ------------------------------------------------------------- groups of eight columns

struct Matrix {
    void *p;
    int64_t ld;
};

// The unit of access is a group of eight columns that starts on a 16-byte
// boundary of memory: columns 8 i - s .. 8 i - s + 7 of a row that starts s
// elements past such a boundary.  Three cases (Rows::kind, by the host):
//   kWhole    every row starts on 16 bytes and is whole groups: plain 16-byte
//             accesses, nothing to check but a group's first column;
//   kShifted  all matrices share one s per row (it depends on the row for odd
//             strides): 16-byte accesses inside the row, its two ends element
//             by element;
//   kLoose    the matrices' starts differ: s = 0, all element by element.
// The kernels are compiled for kWhole and for the other two together.
enum { kWhole, kShifted, kLoose };

struct Rows {
    int64_t rows, cols;
    int32_t kind;
    uint32_t s0, s_step, s_mask;  // s of row r: (s0 + r * s_step) & s_mask
};

template <bool kW>
__device__ __forceinline__ int row_shift(const Rows &a, int64_t r)
{
    return kW ? 0 : (int)((a.s0 + (uint32_t)r * a.s_step) & a.s_mask);
}

template <int DT>
__device__ __forceinline__ char *row_ptr(const Matrix &m, int64_t r)
{
    return static_cast<char *>(m.p) + r * m.ld * Elem<DT>::kBytes;
}

// Whether element e of the group at c0 lies in the row; for a whole row a
// group does or does not as one.
template <bool kW, class I>
__device__ __forceinline__ bool inside(I c0, int e, I cols)
{
    return kW ? c0 < cols : c0 + e >= 0 && c0 + e < cols;
}

template <int DT>
struct Group {
    uint4 w[Elem<DT>::kWords];

    __device__ __forceinline__ void to_float(float (&f)[8]) const { Elem<DT>::to_float(w, f); }
};

// The group at column c0 (< cols) of a row; zeros outside the row.  kRead:
// the matrix is not written by this kernel.
template <int DT, bool kW, bool kRead = true, class I>
__device__ __forceinline__ Group<DT> load_group(const char *row, I c0, I cols, bool vec)
{
    Group<DT> g;
    const char *q = row + (int64_t)c0 * Elem<DT>::kBytes;
    if (kW || (vec && c0 >= 0 && c0 + 8 <= cols)) {
#pragma unroll
        for (int k = 0; k < Elem<DT>::kWords; ++k)
            g.w[k] = kRead ? __ldg(reinterpret_cast<const uint4 *>(q) + k) : reinterpret_cast<const uint4 *>(q)[k];
        return g;
    }
    uint32_t w[4 * Elem<DT>::kWords] = {};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (inside<kW>(c0, e, cols)) {
            if (DT == ZERO_F32)
                w[e] = reinterpret_cast<const uint32_t *>(q)[e];
            else
                w[e >> 1] |= (uint32_t) reinterpret_cast<const uint16_t *>(q)[e] << (16 * (e & 1));
        }
#pragma unroll
    for (int k = 0; k < Elem<DT>::kWords; ++k)
        g.w[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
    return g;
}

template <int DT, bool kW, class I>
__device__ __forceinline__ void store_group(char *row, I c0, I cols, bool vec, const float (&f)[8])
{
    char *q = row + (int64_t)c0 * Elem<DT>::kBytes;
    if (kW || (vec && c0 >= 0 && c0 + 8 <= cols)) {
        if constexpr (DT == ZERO_F32) {
            reinterpret_cast<float4 *>(q)[0] = make_float4(f[0], f[1], f[2], f[3]);
            reinterpret_cast<float4 *>(q)[1] = make_float4(f[4], f[5], f[6], f[7]);
        } else {
            *reinterpret_cast<uint4 *>(q) = LowP<DT>::pack(f);
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (inside<kW>(c0, e, cols))
            store1<DT>(q, e, f[e]);
}

// The mask words of the eight columns from c0 on.  c0 is 0 mod 4 unless the
// rows are shifted: then a group spans three counters.
template <bool kW>
__device__ __forceinline__ void group_words(const Drop &d, uint64_t off, int64_t row, int64_t c0, uint32_t (&w)[8])
{
    const int64_t base = kW ? c0 : c0 & ~(int64_t)3;
    const uint4 a = drop_words(d, off, row, base), b = drop_words(d, off, row, base + 4);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    const int o = kW ? 0 : (int)(c0 & 3);
    if (o != 0) {
        const uint4 e = drop_words(d, off, row, base + 8);
        if (o == 1) {
#pragma unroll
            for (int k = 0; k < 7; ++k)
                w[k] = w[k + 1];
            w[7] = e.x;
        } else if (o == 2) {
#pragma unroll
            for (int k = 0; k < 6; ++k)
                w[k] = w[k + 2];
            w[6] = e.x, w[7] = e.y;
        } else {
#pragma unroll
            for (int k = 0; k < 5; ++k)
                w[k] = w[k + 3];
            w[5] = e.x, w[6] = e.y, w[7] = e.z;
        }
    }
}

template <bool kW>
__device__ __forceinline__ void drop_group(const Drop &d, uint64_t off, int64_t row, int64_t c0, float (&f)[8])
{
    uint32_t w[8];
    group_words<kW>(d, off, row, c0, w);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        f[e] = kept(d, w[e]) ? f[e] * d.scale : 0.0f;
}

// A weight or bias vector's eight columns, as binary32 (`none` without one).
template <int DT, bool kW, class I>
__device__ __forceinline__ void load_vector(const void *p, bool f32, I c0, I cols, bool vec, float none, float (&f)[8])
{
    const char *q = static_cast<const char *>(p);
    if (!p) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            f[e] = none;
    } else if (DT == ZERO_F32 || f32) {
        if (vec)
            load_group<ZERO_F32, kW>(q, c0, cols, true).to_float(f);
        else
            load_group<ZERO_F32, false>(q, c0, cols, false).to_float(f);
    } else {
        if (vec)
            load_group<DT, kW>(q, c0, cols, true).to_float(f);
        else
            load_group<DT, false>(q, c0, cols, false).to_float(f);
    }
}

// ------------------------------------------------------------- dropout

struct DropoutArgs {
    Matrix x, res, out;
    Rows rows;
    uint32_t groups;               // per row
    uint32_t step_rows, step_groups;  // what the whole grid advances by
    Drop d;
};

// One thread per group, the grid striding over all groups.
template <int DT, bool kW>
__global__ void __launch_bounds__(kThreads) k_dropout_add(const __grid_constant__ DropoutArgs a)
{
    const uint32_t flat = blockIdx.x * kThreads + threadIdx.x;
    int64_t r = flat / a.groups;
    uint32_t g = flat - (uint32_t)r * a.groups;
    const uint64_t off = drop_offset(a.d);
    const int64_t cols = a.rows.cols;
    const bool vec = a.rows.kind != kLoose;
    while (r < a.rows.rows) {
        const int64_t c0 = (int64_t)g * 8 - row_shift<kW>(a.rows, r);
        float f[8], t[8];
        const Group<DT> x = load_group<DT, kW, false>(row_ptr<DT>(a.x, r), c0, cols, vec);
        Group<DT> y{};
        if (a.res.p)
            y = load_group<DT, kW, false>(row_ptr<DT>(a.res, r), c0, cols, vec);
        x.to_float(f);
        drop_group<kW>(a.d, off, r, c0, f);
        if (a.res.p) {
            y.to_float(t);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                f[e] += t[e];
        }
        store_group<DT, kW>(row_ptr<DT>(a.out, r), c0, cols, vec, f);
        r += a.step_rows;
        g += a.step_groups;
        if (g >= a.groups) {
            g -= a.groups;
            ++r;
        }
    }
}

// ------------------------------------------------------------- layer norm

__device__ __forceinline__ float warp_sum_f(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over the threads of a row: one warp, or a whole block of `warps` warps
// (s: 33 floats; one barrier before s is used again).
template <bool kWarp>
__device__ __forceinline__ float row_sum(float v, float *s)
{
    v = warp_sum_f(v);
    if (kWarp)
        return v;
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0)
        s[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum_f(lane < warps ? s[lane] : 0.0f);
}

struct NormArgs {
    Matrix x, res, sum, y;
    const void *weight, *bias;
    int32_t w_f32, w_vec;  // weight and bias are binary32; their groups are whole 16 bytes
    float *mean, *rstd;
    Rows rows;
    float eps, inv_cols;
    int32_t dropping;
    Drop d;
};

// Forward: a row in registers, NV groups per thread, read once; mean, then
// the squared deviations from it, then the output.  kWarp: a warp per row
// (no barriers), else a block per row.
template <int DT, int NV, bool kWarp, bool kFused, bool kW>
__global__ void __launch_bounds__(kWarp ? 256 : 512, !kWarp ? 1 : NV <= 2 ? 4 : NV <= 4 ? 3 : 2)
    k_norm_fwd(const __grid_constant__ NormArgs a)
{
    __shared__ float s_red[2][32];
    const int lane = kWarp ? (int)(threadIdx.x & 31) : (int)threadIdx.x;
    const int tpr = kWarp ? 32 : (int)blockDim.x;
    const int64_t first = kWarp ? (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
    const int64_t step = kWarp ? (int64_t)gridDim.x * 8 : (int64_t)gridDim.x;
    const uint64_t off = kFused && a.dropping ? drop_offset(a.d) : 0;
    const int cols = (int)a.rows.cols;
    const bool vec = a.rows.kind != kLoose;
    for (int64_t r = first; r < a.rows.rows; r += step) {
        const int at = lane * 8 - row_shift<kW>(a.rows, r);
        Group<DT> raw[NV], add[kFused ? NV : 1];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c0 = at + v * tpr * 8;
            if (c0 < cols)
                raw[v] = load_group<DT, kW>(row_ptr<DT>(a.x, r), c0, cols, vec);
            else
                raw[v] = Group<DT>{};
        }
        if (kFused && a.res.p) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c0 = at + v * tpr * 8;
                if (c0 < cols)
                    add[kFused ? v : 0] = load_group<DT, kW>(row_ptr<DT>(a.res, r), c0, cols, vec);
                else
                    add[kFused ? v : 0] = Group<DT>{};
            }
        }
        float t[NV][8], s = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c0 = at + v * tpr * 8;
            raw[v].to_float(t[v]);
            if (kFused && c0 < cols) {
                if (a.dropping)
                    drop_group<kW>(a.d, off, r, c0, t[v]);
                if (a.res.p) {
                    float x[8];
                    add[kFused ? v : 0].to_float(x);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        t[v][e] += x[e];
                }
                store_group<DT, kW>(row_ptr<DT>(a.sum, r), c0, cols, vec, t[v]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
                s += t[v][e];
        }
        const float mean = row_sum<kWarp>(s, s_red[0]) * a.inv_cols;
        s = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c0 = at + v * tpr * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                t[v][e] = inside<kW>(c0, e, cols) ? t[v][e] - mean : 0.0f;
                s += t[v][e] * t[v][e];
            }
        }
        const float rstd = 1.0f / sqrtf(row_sum<kWarp>(s, s_red[1]) * a.inv_cols + a.eps);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c0 = at + v * tpr * 8;
            if (c0 < cols) {
                float w[8], b[8];
                load_vector<DT, kW>(a.weight, a.w_f32, c0, cols, a.w_vec, 1.0f, w);
                load_vector<DT, kW>(a.bias, a.w_f32, c0, cols, a.w_vec, 0.0f, b);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    t[v][e] = t[v][e] * rstd * w[e] + b[e];
                store_group<DT, kW>(row_ptr<DT>(a.y, r), c0, cols, vec, t[v]);
            }
        }
        if (lane == 0) {
            if (a.mean)
                a.mean[r] = mean;
            if (a.rstd)
                a.rstd[r] = rstd;
        }
    }
}

// Forward of rows too wide for the registers of a block: three passes over
// the row (the later two from L2).
template <int DT>
__global__ void __launch_bounds__(512) k_norm_fwd_wide(const __grid_constant__ NormArgs a)
{
    __shared__ float s_red[2][32];
    const uint64_t off = a.dropping ? drop_offset(a.d) : 0;
    const int64_t cols = a.rows.cols, step = (int64_t)blockDim.x * 8;
    const bool vec = a.rows.kind != kLoose;
    for (int64_t r = blockIdx.x; r < a.rows.rows; r += gridDim.x) {
        const int64_t at = (int64_t)threadIdx.x * 8 - row_shift<false>(a.rows, r);
        auto value = [&](int64_t c0, float(&t)[8]) {
            load_group<DT, false>(row_ptr<DT>(a.x, r), c0, cols, vec).to_float(t);
            if (a.dropping)
                drop_group<false>(a.d, off, r, c0, t);
            if (a.res.p) {
                float x[8];
                load_group<DT, false>(row_ptr<DT>(a.res, r), c0, cols, vec).to_float(x);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    t[e] += x[e];
            }
        };
        float s = 0.0f, t[8];
        for (int64_t c0 = at; c0 < cols; c0 += step) {
            value(c0, t);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                s += t[e];
        }
        const float mean = row_sum<false>(s, s_red[0]) * a.inv_cols;
        s = 0.0f;
        for (int64_t c0 = at; c0 < cols; c0 += step) {
            value(c0, t);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c0 + e >= 0 && c0 + e < cols)
                    s += (t[e] - mean) * (t[e] - mean);
        }
        const float rstd = 1.0f / sqrtf(row_sum<false>(s, s_red[1]) * a.inv_cols + a.eps);
        for (int64_t c0 = at; c0 < cols; c0 += step) {
            float w[8], b[8];
            value(c0, t);
            if (a.sum.p)
                store_group<DT, false>(row_ptr<DT>(a.sum, r), c0, cols, vec, t);
            load_vector<DT, false>(a.weight, a.w_f32, c0, cols, a.w_vec, 1.0f, w);
            load_vector<DT, false>(a.bias, a.w_f32, c0, cols, a.w_vec, 0.0f, b);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                t[e] = (t[e] - mean) * rstd * w[e] + b[e];
            store_group<DT, false>(row_ptr<DT>(a.y, r), c0, cols, vec, t);
        }
        if (threadIdx.x == 0) {
            if (a.mean)
                a.mean[r] = mean;
            if (a.rstd)
                a.rstd[r] = rstd;
        }
        __syncthreads();
    }
}

struct NormBwdArgs {
    Matrix dy, x, dres, dx, dropped;
    const void *weight;
    int32_t w_f32, w_vec;
    const float *mean, *rstd;
    float *partials;  // [block][dweight, dbias][cols]; NULL: neither is wanted
    Rows rows;
    float inv_cols;
    int32_t dropping;
    int32_t tpr;  // threads per row
    Drop d;
};

// Two sums over the threads of a row group (tpr threads of the block, its
// own named barrier), in a buffer that alternates from row to row.
__device__ __forceinline__ float2 group_sum2(float2 v, float2 *s, int tpr, int group, int t)
{
    v.x = warp_sum_f(v.x);
    v.y = warp_sum_f(v.y);
    if (tpr == 32)
        return v;
    if ((t & 31) == 0)
        s[t >> 5] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(tpr) : "memory");
    v = (t & 31) < (tpr >> 5) ? s[t & 31] : make_float2(0.0f, 0.0f);
    v.x = warp_sum_f(v.x);
    v.y = warp_sum_f(v.y);
    return v;
}

// Backward: a block of several row groups of tpr threads, each thread with NV
// groups of columns, which stay its own from row to row, so that dweight and
// dbias build up in its registers.  Rows are taken NG = gridDim * (groups per
// block) apart; NG is a multiple of 8 when a group takes more than one row,
// so that its rows all have the same shift.  The next row is loaded before
// the sums of this one are exchanged; a row is held as it came (16-bit) and
// converted again after the exchange.
template <int DT, int NV, bool kW>
__global__ void __launch_bounds__(NV == 1 ? 768 : 512) k_norm_bwd(const __grid_constant__ NormBwdArgs a)
{
    extern __shared__ float s_cols[];
    __shared__ float2 s_red[2][32];
    const int tpr = a.tpr, group = threadIdx.x / tpr, t = threadIdx.x - group * tpr, groups = blockDim.x / tpr;
    const int cols = (int)a.rows.cols;
    const int64_t step = (int64_t)gridDim.x * groups;
    const uint64_t off = a.dropping ? drop_offset(a.d) : 0;
    const bool vec = a.rows.kind != kLoose;
    int64_t r = (int64_t)blockIdx.x * groups + group;
    const int at = t * 8 - row_shift<kW>(a.rows, r);
    float dw[NV][8], db[NV][8], w[NV][8];
    Group<DT> ndy[NV], nx[NV], nres[NV];
    float nmean = 0.0f, nrstd = 0.0f;
    auto fetch = [&](int64_t row) {
        if (row >= a.rows.rows)
            return;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c0 = at + v * tpr * 8;
            if (c0 < cols) {
                ndy[v] = load_group<DT, kW>(row_ptr<DT>(a.dy, row), c0, cols, vec);
                nx[v] = load_group<DT, kW>(row_ptr<DT>(a.x, row), c0, cols, vec);
                if (a.dres.p)
                    nres[v] = load_group<DT, kW>(row_ptr<DT>(a.dres, row), c0, cols, vec);
            }
        }
        nmean = __ldg(a.mean + row);
        nrstd = __ldg(a.rstd + row);
    };
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c0 = at + v * tpr * 8;
        ndy[v] = nx[v] = nres[v] = Group<DT>{};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            dw[v][e] = db[v][e] = w[v][e] = 0.0f;
        if (c0 < cols)
            load_vector<DT, kW>(a.weight, a.w_f32, c0, cols, a.w_vec, 1.0f, w[v]);
    }
    fetch(r);
    for (int buf = 0; r < a.rows.rows; r += step, buf ^= 1) {
        const float mean = nmean, rstd = nrstd;
        Group<DT> cdy[NV], cx[NV], cres[NV];
        float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c0 = at + v * tpr * 8;
            float dy[8], x[8];
            cdy[v] = ndy[v], cx[v] = nx[v], cres[v] = nres[v];
            cdy[v].to_float(dy);
            cx[v].to_float(x);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // outside the row dy is 0, and 0 - mean must not be seen
                const float xh = inside<kW>(c0, e, cols) ? (x[e] - mean) * rstd : 0.0f, g = dy[e] * w[v][e];
                dw[v][e] += dy[e] * xh;
                db[v][e] += dy[e];
                s.x += g;
                s.y += g * xh;
            }
        }
        fetch(r + step);
        s = group_sum2(s, s_red[buf] + group * (tpr >> 5), tpr, group, t);
        s.x *= a.inv_cols;
        s.y *= a.inv_cols;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c0 = at + v * tpr * 8;
            if (c0 >= cols)
                continue;
            float dy[8], x[8];
            cdy[v].to_float(dy);
            cx[v].to_float(x);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                dy[e] = rstd * (dy[e] * w[v][e] - s.x - (x[e] - mean) * rstd * s.y);
            if (a.dres.p) {
                cres[v].to_float(x);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    dy[e] += x[e];
            }
            store_group<DT, kW>(row_ptr<DT>(a.dx, r), c0, cols, vec, dy);
            if (a.dropping) {
                drop_group<kW>(a.d, off, r, c0, dy);
                store_group<DT, kW>(row_ptr<DT>(a.dropped, r), c0, cols, vec, dy);
            }
        }
    }
    if (!a.partials)
        return;
    // the block's row groups, in order, column by column
    const int width = tpr * NV * 8;
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                s_cols[group * width + (v * tpr + t) * 8 + e] = which ? db[v][e] : dw[v][e];
        __syncthreads();
        for (int c = threadIdx.x; c < cols; c += blockDim.x) {
            float sum = 0.0f;
            for (int q = 0; q < groups; ++q) {
                const int64_t row = (int64_t)blockIdx.x * groups + q;
                if (row < a.rows.rows)
                    sum += s_cols[q * width + c + row_shift<kW>(a.rows, row)];
            }
            a.partials[((int64_t)blockIdx.x * 2 + which) * cols + c] = sum;
        }
    }
}

// dx of rows too wide for k_norm_bwd: a block per row, two passes.
template <int DT>
__global__ void __launch_bounds__(512) k_norm_bwd_wide(const __grid_constant__ NormBwdArgs a)
{
    __shared__ float2 s_red[2][32];
    const uint64_t off = a.dropping ? drop_offset(a.d) : 0;
    const int64_t cols = a.rows.cols, step = (int64_t)blockDim.x * 8;
    const bool vec = a.rows.kind != kLoose;
    int buf = 0;
    for (int64_t r = blockIdx.x; r < a.rows.rows; r += gridDim.x, buf ^= 1) {
        const int64_t at = (int64_t)threadIdx.x * 8 - row_shift<false>(a.rows, r);
        const float mean = a.mean[r], rstd = a.rstd[r];
        auto value = [&](int64_t c0, float(&g)[8], float(&xh)[8]) {
            float w[8];
            load_group<DT, false>(row_ptr<DT>(a.dy, r), c0, cols, vec).to_float(g);
            load_group<DT, false>(row_ptr<DT>(a.x, r), c0, cols, vec).to_float(xh);
            load_vector<DT, false>(a.weight, a.w_f32, c0, cols, a.w_vec, 1.0f, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                g[e] *= w[e];
                xh[e] = (xh[e] - mean) * rstd;
            }
        };
        float2 s = make_float2(0.0f, 0.0f);
        for (int64_t c0 = at; c0 < cols; c0 += step) {
            float g[8], xh[8];
            value(c0, g, xh);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c0 + e >= 0 && c0 + e < cols) {
                    s.x += g[e];
                    s.y += g[e] * xh[e];
                }
        }
        s = group_sum2(s, s_red[buf], blockDim.x, 0, threadIdx.x);
        s.x *= a.inv_cols;
        s.y *= a.inv_cols;
        for (int64_t c0 = at; c0 < cols; c0 += step) {
            float g[8], xh[8];
            value(c0, g, xh);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                g[e] = rstd * (g[e] - s.x - xh[e] * s.y);
            if (a.dres.p) {
                float x[8];
                load_group<DT, false>(row_ptr<DT>(a.dres, r), c0, cols, vec).to_float(x);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    g[e] += x[e];
            }
            store_group<DT, false>(row_ptr<DT>(a.dx, r), c0, cols, vec, g);
            if (a.dropping) {
                drop_group<false>(a.d, off, r, c0, g);
                store_group<DT, false>(row_ptr<DT>(a.dropped, r), c0, cols, vec, g);
            }
        }
    }
}

// Partial dweight and dbias of those rows: block (x, y) takes 256 columns
// (a thread: eight) and every (8 gridDim.y)-th eight rows, a warp per row.
template <int DT>
__global__ void __launch_bounds__(kThreads) k_norm_bwd_wide_cols(const __grid_constant__ NormBwdArgs a)
{
    __shared__ float s_cols[kWarps][256];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t cols = a.rows.cols, col = (int64_t)blockIdx.x * 256;
    const int64_t c0 = col + lane * 8;
    float dw[8] = {}, db[8] = {};
    const bool vec = a.rows.kind != kLoose && a.rows.s_mask == 0;
    if (c0 < cols)
        for (int64_t r = (int64_t)blockIdx.y * kWarps + warp; r < a.rows.rows; r += (int64_t)gridDim.y * kWarps) {
            float dy[8], x[8];
            load_group<DT, false>(row_ptr<DT>(a.dy, r), c0, cols, vec).to_float(dy);
            load_group<DT, false>(row_ptr<DT>(a.x, r), c0, cols, vec).to_float(x);
            const float mean = __ldg(a.mean + r), rstd = __ldg(a.rstd + r);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                dw[e] += dy[e] * ((x[e] - mean) * rstd);
                db[e] += dy[e];
            }
        }
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e)
            s_cols[warp][lane * 8 + e] = which ? db[e] : dw[e];
        __syncthreads();
        float sum = 0.0f;
#pragma unroll
        for (int q = 0; q < kWarps; ++q)
            sum += s_cols[q][threadIdx.x];
        if (col + threadIdx.x < cols)
            a.partials[((int64_t)blockIdx.y * 2 + which) * cols + col + threadIdx.x] = sum;
    }
}

// dweight (blockIdx.y 0) and dbias (1): `n` partials of each column added in
// a fixed order, a block per 32 columns, eight warps taking every eighth.
__global__ void __launch_bounds__(kThreads) k_norm_bwd_sum(const float *partials, int n, int64_t cols, void *dweight,
                                                           void *dbias, int32_t gdtype)
{
    __shared__ float s[kWarps][32];
    void *out = blockIdx.y ? dbias : dweight;
    if (!out)
        return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    pdl_wait();
    float sum = 0.0f;
    if (c < cols)
#pragma unroll 8
        for (int q = warp; q < n; q += kWarps)
            sum += __ldcg(partials + ((int64_t)q * 2 + blockIdx.y) * cols + c);
    s[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && c < cols) {
#pragma unroll
        for (int k = 1; k < kWarps; ++k)
            sum += s[k][lane];
        store1_as(gdtype, out, c, sum);
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

// How the groups of a call's matrices lie (see Rows): one shift for all of
// them, or element by element.
Rows row_groups(int64_t rows, int64_t cols, int32_t dtype, std::initializer_list<Matrix> mats)
{
    const uint32_t es = elem_bytes(dtype), per = 16 / es;
    Rows g{};
    g.rows = rows, g.cols = cols, g.kind = kShifted;
    bool first = true;
    for (const Matrix &m : mats) {
        if (!m.p)
            continue;
        const uint32_t s0 = (uint32_t)(reinterpret_cast<uintptr_t>(m.p) / es) & (per - 1);
        const uint32_t step = rows > 1 ? (uint32_t)m.ld & (per - 1) : 0;
        if (first)
            g.s0 = s0, g.s_step = step;
        else if (g.s0 != s0 || g.s_step != step)
            g.kind = kLoose;
        first = false;
    }
    if (g.kind == kLoose)
        g.s0 = g.s_step = 0;
    else if (g.s0 == 0 && g.s_step == 0 && (cols & 7) == 0)
        g.kind = kWhole;
    g.s_mask = g.s0 || g.s_step ? per - 1 : 0;
    return g;
}

// Groups that cover a row at any of its shifts.
int64_t groups_per_row(const Rows &g) { return (g.cols + g.s_mask + 7) / 8; }

int vector_groups(const Rows &g, const void *a, const void *b) { return g.s_mask == 0 && aligned16(a) && aligned16(b); }

// Rows wider than this go through the three-pass kernels (registers hold NV
// <= 8 groups for each of at most 512 threads).
constexpr int64_t kMostGroups = 512 * 8;

template <int DT, int NV, bool kFused, bool kW>
int norm_fwd_nv(const NormArgs &a, bool warp, int block, cudaStream_t st)
{
    const int64_t most = (int64_t)sm_count() * 32;
    if (warp) {
        const int64_t g = (a.rows.rows + 7) / 8;
        k_norm_fwd<DT, NV, true, kFused, kW><<<(unsigned)(g < most ? g : most), 256, 0, st>>>(a);
    } else {
        k_norm_fwd<DT, NV, false, kFused, kW><<<(unsigned)(a.rows.rows < most ? a.rows.rows : most), block, 0, st>>>(a);
    }
    return check_launch("k_norm_fwd");
}

template <int DT, bool kFused, bool kW>
int norm_fwd(const NormArgs &a, cudaStream_t st)
{
    const int64_t groups = groups_per_row(a.rows);
    if (groups > kMostGroups) {
        const int64_t most = (int64_t)sm_count() * 4;
        k_norm_fwd_wide<DT><<<(unsigned)(a.rows.rows < most ? a.rows.rows : most), 512, 0, st>>>(a);
        return check_launch("k_norm_fwd_wide");
    }
    // A warp per row where that fills the GPU (16 warps per SM) and a lane's
    // share fits its registers; else a block per row, one or two groups per
    // thread while rows are few (latency), up to eight for wide rows.
    const bool warp = groups <= 32 || (groups <= 32 * 8 && a.rows.rows >= 16 * (int64_t)sm_count());
    int block = 32;
    if (!warp)
        block = groups >= 512 ? 512 : (int)((groups + 31) / 32 * 32);
    const int64_t nv = (groups + block - 1) / block;
    if (nv <= 1)
        return norm_fwd_nv<DT, 1, kFused, kW>(a, warp, block, st);
    if (nv <= 2)
        return norm_fwd_nv<DT, 2, kFused, kW>(a, warp, block, st);
    if (nv <= 4)
        return norm_fwd_nv<DT, 4, kFused, kW>(a, warp, block, st);
    return norm_fwd_nv<DT, 8, kFused, kW>(a, warp, block, st);
}

template <int DT>
int norm_fwd_of(const NormArgs &a, cudaStream_t st)
{
    const bool whole = a.rows.kind == kWhole;
    if (a.sum.p)
        return whole ? norm_fwd<DT, true, true>(a, st) : norm_fwd<DT, true, false>(a, st);
    return whole ? norm_fwd<DT, false, true>(a, st) : norm_fwd<DT, false, false>(a, st);
}

// The backward pass's blocks: threads per row, row groups per block, blocks,
// and partials of dweight and dbias that they leave.
struct BwdPlan {
    bool wide;
    int nv, tpr, groups;
    int64_t blocks, partials;
};

constexpr int kBwdBlocks = 152;  // a multiple of 8 (see k_norm_bwd); one block per SM

BwdPlan bwd_plan(int64_t rows, int64_t groups_row)
{
    BwdPlan p{};
    p.wide = groups_row > 1024;
    if (p.wide) {
        p.partials = rows < kWarps * 64 ? (rows + kWarps - 1) / kWarps : 64;
        return p;
    }
    p.nv = groups_row <= 768 ? 1 : 2;
    p.tpr = (int)(((groups_row + p.nv - 1) / p.nv + 31) / 32 * 32);
    p.groups = (p.nv == 1 ? 768 : 512) / p.tpr;
    if (p.tpr > 32 && p.groups > 15)
        p.groups = 15;  // named barriers
    const int64_t need = (rows + p.groups - 1) / p.groups;
    if (need < kBwdBlocks) {  // few rows: spread them over the SMs
        const int64_t per = (rows + kBwdBlocks - 1) / kBwdBlocks;
        if (per < p.groups)
            p.groups = (int)(per < 1 ? 1 : per);
    }
    const int64_t n = (rows + p.groups - 1) / p.groups;
    p.blocks = n < kBwdBlocks ? n : kBwdBlocks;
    p.partials = p.blocks;
    return p;
}

template <int DT>
int norm_bwd(NormBwdArgs &a, const BwdPlan &p, cudaStream_t st)
{
    if (p.wide) {
        const int64_t most = (int64_t)sm_count() * 4;
        k_norm_bwd_wide<DT><<<(unsigned)(a.rows.rows < most ? a.rows.rows : most), 512, 0, st>>>(a);
        ZERO_TRY(check_launch("k_norm_bwd_wide"));
        if (!a.partials)
            return ZERO_OK;
        const dim3 grid((unsigned)((a.rows.cols + 255) / 256), (unsigned)p.partials);
        k_norm_bwd_wide_cols<DT><<<grid, kThreads, 0, st>>>(a);
        return check_launch("k_norm_bwd_wide_cols");
    }
    a.tpr = p.tpr;
    const int smem = p.groups * p.tpr * p.nv * 8 * 4;
    const unsigned grid = (unsigned)p.blocks, block = (unsigned)(p.groups * p.tpr);
    const bool whole = a.rows.kind == kWhole;
    if (p.nv == 1 && whole)
        k_norm_bwd<DT, 1, true><<<grid, block, smem, st>>>(a);
    else if (p.nv == 1)
        k_norm_bwd<DT, 1, false><<<grid, block, smem, st>>>(a);
    else if (whole)
        k_norm_bwd<DT, 2, true><<<grid, block, smem, st>>>(a);
    else
        k_norm_bwd<DT, 2, false><<<grid, block, smem, st>>>(a);
    return check_launch("k_norm_bwd");
}

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
    DropoutArgs a{};
    a.x = matrix(x, x_ld), a.res = matrix(residual, residual_ld), a.out = matrix(out, out_ld);
    a.rows = row_groups(rows, cols, dtype, {a.x, a.res, a.out});
    a.groups = (uint32_t)groups_per_row(a.rows);
    a.d = d;
    const int64_t blocks = (rows * (int64_t)a.groups + kThreads - 1) / kThreads, most = (int64_t)sm_count() * 8;
    const unsigned grid = (unsigned)(blocks < most ? blocks : most);
    a.step_rows = grid * kThreads / a.groups, a.step_groups = grid * kThreads % a.groups;
    const bool whole = a.rows.kind == kWhole;
    if (dtype == ZERO_F16)
        (whole ? k_dropout_add<ZERO_F16, true> : k_dropout_add<ZERO_F16, false>)<<<grid, kThreads, 0, st>>>(a);
    else if (dtype == ZERO_BF16)
        (whole ? k_dropout_add<ZERO_BF16, true> : k_dropout_add<ZERO_BF16, false>)<<<grid, kThreads, 0, st>>>(a);
    else
        (whole ? k_dropout_add<ZERO_F32, true> : k_dropout_add<ZERO_F32, false>)<<<grid, kThreads, 0, st>>>(a);
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
    a.rows = row_groups(rows, cols, dtype, {a.x, a.res, a.sum, a.y});
    a.weight = weight, a.bias = bias, a.w_f32 = wdtype == ZERO_F32, a.w_vec = vector_groups(a.rows, weight, bias);
    a.mean = mean, a.rstd = rstd, a.eps = (float)eps, a.inv_cols = 1.0f / (float)cols, a.dropping = drop != nullptr;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == ZERO_F16)
        return norm_fwd_of<ZERO_F16>(a, st);
    if (dtype == ZERO_BF16)
        return norm_fwd_of<ZERO_BF16>(a, st);
    return norm_fwd_of<ZERO_F32>(a, st);
}

extern "C" size_t zero_layer_norm_workspace_bytes(int64_t rows, int64_t cols)
{
    if (rows < 0 || cols < 0 || check_sizes(rows, cols) != ZERO_OK)
        return 0;
    // rows may start off 16 bytes: up to a group more
    const BwdPlan a = bwd_plan(rows, (cols + 7) / 8), b = bwd_plan(rows, (cols + 7) / 8 + 1);
    const int64_t n = a.partials > b.partials ? a.partials : b.partials;
    return 256 + align256((size_t)n * 2 * (size_t)cols * 4);
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
    a.rows = row_groups(rows, cols, dtype, {a.dy, a.x, a.dres, a.dx, a.dropped});
    a.weight = weight, a.w_f32 = wdtype == ZERO_F32, a.w_vec = vector_groups(a.rows, weight, nullptr);
    a.mean = mean, a.rstd = rstd, a.inv_cols = 1.0f / (float)cols, a.dropping = drop != nullptr;
    if (rows == 0) {
        for (void *p : {dweight, dbias})
            if (p && cudaMemsetAsync(p, 0, (size_t)cols * elem_bytes(gdtype), st) != cudaSuccess)
                return check_launch("cudaMemsetAsync");
        return ZERO_OK;
    }
    if (dweight || dbias)
        a.partials = reinterpret_cast<float *>(static_cast<char *>(ws) + 256);
    const BwdPlan plan = bwd_plan(rows, groups_per_row(a.rows));
    if (dtype == ZERO_F16)
        ZERO_TRY(norm_bwd<ZERO_F16>(a, plan, st));
    else if (dtype == ZERO_BF16)
        ZERO_TRY(norm_bwd<ZERO_BF16>(a, plan, st));
    else
        ZERO_TRY(norm_bwd<ZERO_F32>(a, plan, st));
    if (!a.partials)
        return ZERO_OK;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((cols + 31) / 32), 2);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, k_norm_bwd_sum, (const float *)a.partials, (int)plan.partials, cols, dweight, dbias, gdtype);
    return check_launch("k_norm_bwd_sum");
}
