// Norms of queries and keys for each head with the position rotation in the
// same pass, forward and backward.
#include <cmath>

#include "sublayer.cuh"

namespace zpml {
namespace {

constexpr int kMostDim = 256;               // of a head
constexpr int kMostPairs = kMostDim / 2;    // of the rotation
constexpr int64_t kMostHeads = (int64_t)1 << 20;

struct QkArgs {
    Heads x[2], y[2], dx[2];  // q, k: the inputs; the outputs (or their gradients); the inputs' gradients
    const void *w[2];
    const uint64_t *turns;
    const int64_t *positions;
    int64_t tokens, units;          // a unit: `per` heads of one token
    int32_t heads[2], per, chunks;  // units of a token
    int32_t dim, rot, interleaved, w_f32;
    int32_t lanes;  // per row, a power of two
    float eps, inv_dim;
    float *partial;  // of the weights' gradients: [block][2][dim]
};

// ------------------------------------------------------------- pieces of a row

// V elements of a row, 2 to 16 bytes.
template <int DT, int V>
struct Piece {
    static constexpr int kBytes = V * (DT == ZERO_F32 ? 4 : 2), kWords = (kBytes + 3) / 4;
    uint32_t w[kWords];

    __device__ __forceinline__ void load(const void *p, int64_t i)
    {
        const char *at = static_cast<const char *>(p) + i * (kBytes / V);
        if constexpr (kBytes == 16) {
            const uint4 v = *reinterpret_cast<const uint4 *>(at);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else if constexpr (kBytes == 8) {
            const uint2 v = *reinterpret_cast<const uint2 *>(at);
            w[0] = v.x, w[1] = v.y;
        } else if constexpr (kBytes == 4) {
            w[0] = *reinterpret_cast<const uint32_t *>(at);
        } else {
            w[0] = *reinterpret_cast<const uint16_t *>(at);
        }
    }

    __device__ __forceinline__ void store(void *p, int64_t i) const
    {
        char *at = static_cast<char *>(p) + i * (kBytes / V);
        if constexpr (kBytes == 16)
            *reinterpret_cast<uint4 *>(at) = make_uint4(w[0], w[1], w[2], w[3]);
        else if constexpr (kBytes == 8)
            *reinterpret_cast<uint2 *>(at) = make_uint2(w[0], w[1]);
        else if constexpr (kBytes == 4)
            *reinterpret_cast<uint32_t *>(at) = w[0];
        else
            *reinterpret_cast<uint16_t *>(at) = (uint16_t)w[0];
    }

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int k = 0; k < kWords; ++k)
            w[k] = 0;
    }

    __device__ __forceinline__ void get(float (&f)[V]) const
    {
        if constexpr (DT == ZERO_F32) {
#pragma unroll
            for (int e = 0; e < V; ++e)
                f[e] = __uint_as_float(w[e]);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const uint32_t h = (e & 1) ? w[e / 2] >> 16 : w[e / 2] & 0xffffu;
                if constexpr (DT == ZERO_F16)
                    f[e] = __half2float(__ushort_as_half((unsigned short)h));
                else
                    f[e] = (e & 1) ? __uint_as_float(w[e / 2] & 0xffff0000u) : __uint_as_float(w[e / 2] << 16);
            }
        }
    }

    __device__ __forceinline__ void put(const float (&f)[V])
    {
        if constexpr (DT == ZERO_F32) {
#pragma unroll
            for (int e = 0; e < V; ++e)
                w[e] = __float_as_uint(f[e]);
        } else if constexpr (V == 1) {
            w[0] = DT == ZERO_F16 ? __half_as_ushort(__float2half_rn(f[0])) : __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
        } else {
#pragma unroll
            for (int e = 0; e < V; e += 2) {
                if constexpr (DT == ZERO_F16) {
                    const __half2 h = __floats2half2_rn(f[e], f[e + 1]);
                    w[e / 2] = *reinterpret_cast<const uint32_t *>(&h);
                } else {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(f[e], f[e + 1]);
                    w[e / 2] = *reinterpret_cast<const uint32_t *>(&h);
                }
            }
        }
    }
};

// V consecutive binary32 of shared memory (V a multiple of 4: on 16 bytes).
template <int V>
__device__ __forceinline__ void shared_floats(const float *p, float (&f)[V])
{
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int e = 0; e < V; e += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(p + e);
            f[e] = v.x, f[e + 1] = v.y, f[e + 2] = v.z, f[e + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
            f[e] = p[e];
    }
}

// ------------------------------------------------------------- the rotation

// The angle of a position and a frequency: phase = position * turns modulo
// 2^64 is the angle's fraction of a turn, exactly.  Its nearest quarter turn
// is taken off in integers too, so that what becomes binary32 is an angle of
// at most pi / 4 with a relative error of 2^-24 (2.4e-8 of a radian and a half
// in the worst case); a binary32 angle of position 10^6 would be off by 0.03.
__device__ __forceinline__ float2 cos_sin(uint64_t phase)
{
    const uint32_t quarter = (uint32_t)((phase + ((uint64_t)1 << 61)) >> 62);
    const int64_t rest = (int64_t)(phase - ((uint64_t)quarter << 62));
    float s, c;
    sincospif((float)rest * 0x1p-63f, &s, &c);
    if (quarter & 1) {
        const float t = c;
        c = -s, s = t;
    }
    return quarter & 2 ? make_float2(-c, -s) : make_float2(c, s);
}

struct QkShared {
    float w[2][kMostDim];                            // both weights in binary32 (1 without one)
    float cos[kWarps][kMostPairs], sin[kWarps][kMostPairs];  // of each warp's token
};

__device__ __forceinline__ void load_weights(const QkArgs &a, QkShared &sh, int dt)
{
    for (int i = threadIdx.x; i < 2 * a.dim; i += kThreads) {
        const int kind = i >= a.dim, e = i - kind * a.dim;
        const void *w = a.w[kind];
        float v = 1.0f;
        if (w)
            v = a.w_f32 ? load1<ZERO_F32>(w, e) : dt == ZERO_F16 ? load1<ZERO_F16>(w, e)
                                              : dt == ZERO_BF16 ? load1<ZERO_BF16>(w, e) : load1<ZERO_F32>(w, e);
        sh.w[kind][e] = v;
    }
    __syncthreads();
}

__device__ __forceinline__ void token_angles(const QkArgs &a, QkShared &sh, int warp, int lane, int64_t token)
{
    const uint64_t pos = (uint64_t)(a.positions ? a.positions[token] : token);
    __syncwarp();  // the token before is done with the tables
    for (int i = lane; i < a.rot / 2; i += 32) {
        const float2 cs = cos_sin(pos * a.turns[i]);
        sh.cos[warp][i] = cs.x;
        sh.sin[warp][i] = cs.y;
    }
    __syncwarp();
}

// What a lane's pieces need of the rotation: cos and +-sin for each element
// (forward: of the sum x cos + partner sin), and where a piece's partners are.
// A piece lies wholly before, in the first or in the second half of the
// rotated elements (the host picks V so); interleaved pairs lie in one piece
// unless V is 1.
template <int V, int N>
struct Turn {
    float c[N][V], s[N][V];
    int partner[N];  // piece (element of a piece, for w)
};

template <int V>
__device__ __forceinline__ int partner_piece(const QkArgs &a, int piece)
{
    const int e = piece * V, half = a.rot / 2;
    if (e >= a.rot)
        return piece;
    if (a.interleaved)
        return V == 1 ? piece ^ 1 : piece;
    return e < half ? piece + half / V : piece - half / V;
}

template <int V, int N>
__device__ __forceinline__ void load_turn(const QkArgs &a, const QkShared &sh, int warp, int at, Turn<V, N> &t)
{
    const int half = a.rot / 2;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int piece = at + n * a.lanes, e0 = piece * V;
        t.partner[n] = partner_piece<V>(a, piece);
        if (e0 >= a.rot || e0 >= a.dim) {
#pragma unroll
            for (int e = 0; e < V; ++e)
                t.c[n][e] = 1.0f, t.s[n][e] = 0.0f;
        } else if (a.interleaved) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const bool in = V == 1 || e0 + e < a.rot;
                const int pair = in ? (e0 + e) / 2 : 0;
                const float s = sh.sin[warp][pair];
                t.c[n][e] = in ? sh.cos[warp][pair] : 1.0f;
                t.s[n][e] = !in ? 0.0f : ((e0 + e) & 1) ? s : -s;
            }
        } else {
            const bool first = e0 < half;
            shared_floats<V>(&sh.cos[warp][first ? e0 : e0 - half], t.c[n]);
            shared_floats<V>(&sh.sin[warp][first ? e0 : e0 - half], t.s[n]);
#pragma unroll
            for (int e = 0; e < V; ++e)
                t.s[n][e] = first ? -t.s[n][e] : t.s[n][e];
        }
    }
}

// The partners of a lane's elements: from its own piece (interleaved), or
// from another lane of the row.
template <int DT, int V, int N>
__device__ __forceinline__ void partners(const QkArgs &a, const Turn<V, N> &t, const Piece<DT, V> (&x)[N], int lane,
                                         float (&f)[N][V])
{
    if (V > 1 && a.interleaved) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float own[V];
            x[n].get(own);
#pragma unroll
            for (int e = 0; e < V; ++e)
                f[n][e] = own[V > 1 ? e ^ 1 : e];
        }
        return;
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int from = (lane & ~(a.lanes - 1)) | (t.partner[n] & (a.lanes - 1));
        Piece<DT, V> p{};
#pragma unroll
        for (int m = 0; m < N; ++m)
#pragma unroll
            for (int k = 0; k < Piece<DT, V>::kWords; ++k) {
                const uint32_t v = __shfl_sync(0xffffffffu, x[m].w[k], from);
                if (N == 1 || t.partner[n] / a.lanes == m)
                    p.w[k] = v;
            }
        p.get(f[n]);
    }
}

__device__ __forceinline__ float row_sum(float v, int lanes)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (o < lanes)
            v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// ------------------------------------------------------------- kernels

// A warp takes a token's heads (or, of few tokens, `per` of them): its lanes
// work out the token's angles once, one pair each, and share them through
// shared memory; then rows of `lanes` lanes, V elements to a lane and
// U * 32 / lanes rows on their way at once.  With A = weight cos and B =
// +-(partner's weight) sin, which the heads of a token share,
//     out = (x A + partner B) / sqrt(mean(x^2) + eps).
template <int DT, int V, int N, int U>
__global__ void __launch_bounds__(kThreads) k_qk_norm(const __grid_constant__ QkArgs a)
{
    __shared__ __align__(16) QkShared sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows = 32 / a.lanes, sub = lane / a.lanes, at = lane & (a.lanes - 1);
    load_weights(a, sh, DT);
    for (int64_t u = (int64_t)blockIdx.x * kWarps + warp; u < a.units; u += (int64_t)gridDim.x * kWarps) {
        const int64_t token = u / a.chunks;
        const int first = (int)(u - token * a.chunks) * a.per, all = a.heads[0] + a.heads[1];
        const int last = first + a.per < all ? first + a.per : all;
        if (a.rot)
            token_angles(a, sh, warp, lane, token);
        Turn<V, N> t;
        load_turn(a, sh, warp, at, t);
#pragma unroll
        for (int kind = 0; kind < 2; ++kind) {
            const int base = kind ? a.heads[0] : 0;
            const int lo = first > base ? first - base : 0;
            const int hi = last - base < a.heads[kind] ? last - base : a.heads[kind];
            if (lo >= hi)
                continue;
            float A[N][V], B[N][V];
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const int e0 = (at + n * a.lanes) * V;
                float w[V] = {}, wp[V] = {};
                if (e0 < a.dim) {
                    shared_floats<V>(&sh.w[kind][e0], w);
                    shared_floats<V>(&sh.w[kind][t.partner[n] * V], wp);
                }
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    A[n][e] = w[e] * t.c[n][e];
                    B[n][e] = (V > 1 && a.interleaved ? w[V > 1 ? e ^ 1 : e] : wp[e]) * t.s[n][e];
                }
            }
            const int es = DT == ZERO_F32 ? 4 : 2;
            const char *x = static_cast<const char *>(a.x[kind].p) + token * a.x[kind].ld * es;
            char *y = static_cast<char *>(const_cast<void *>(a.y[kind].p)) + token * a.y[kind].ld * es;
            for (int h0 = lo + sub; h0 - sub < hi; h0 += rows * U) {
                Piece<DT, V> p[U][N];
#pragma unroll
                for (int k = 0; k < U; ++k)
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        const int h = h0 + k * rows, e0 = (at + n * a.lanes) * V;
                        p[k][n].clear();
                        if (h < hi && e0 < a.dim)
                            p[k][n].load(x + h * a.x[kind].hd * es, e0);
                    }
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    if (h0 - sub + k * rows >= hi)
                        break;
                    float f[N][V], g[N][V] = {}, sq = 0.0f;
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        p[k][n].get(f[n]);
#pragma unroll
                        for (int e = 0; e < V; ++e)
                            sq += f[n][e] * f[n][e];
                    }
                    if (a.rot)
                        partners<DT, V, N>(a, t, p[k], lane, g);
                    const float r = rsqrtf(row_sum(sq, a.lanes) * a.inv_dim + a.eps);
                    const int h = h0 + k * rows;
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        const int e0 = (at + n * a.lanes) * V;
                        float o[V];
#pragma unroll
                        for (int e = 0; e < V; ++e)
                            o[e] = (f[n][e] * A[n][e] + g[n][e] * B[n][e]) * r;
                        Piece<DT, V> out;
                        out.put(o);
                        if (h < hi && e0 < a.dim)
                            out.store(y + h * a.y[kind].hd * es, e0);
                    }
                }
            }
        }
    }
}

// The backward pass in the same shape, over persistent warps: a lane holds
// its columns of both weights' gradients from its first row to its last, and
// a block leaves one partial sum per column.
template <int DT, int V, int N, int U>
__global__ void __launch_bounds__(kThreads) k_qk_norm_bwd(const __grid_constant__ QkArgs a)
{
    __shared__ __align__(16) QkShared sh;
    __shared__ float s_dw[kWarps][2][kMostDim];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows = 32 / a.lanes, sub = lane / a.lanes, at = lane & (a.lanes - 1);
    pdl_launch_next();
    load_weights(a, sh, DT);
    float dw[2][N][V] = {};
    for (int64_t u = (int64_t)blockIdx.x * kWarps + warp; u < a.units; u += (int64_t)gridDim.x * kWarps) {
        const int64_t token = u / a.chunks;
        const int first = (int)(u - token * a.chunks) * a.per, all = a.heads[0] + a.heads[1];
        const int last = first + a.per < all ? first + a.per : all;
        if (a.rot)
            token_angles(a, sh, warp, lane, token);
        Turn<V, N> t;  // turned back: the sines' signs the other way
        load_turn(a, sh, warp, at, t);
#pragma unroll
        for (int kind = 0; kind < 2; ++kind) {
            const int base = kind ? a.heads[0] : 0;
            const int lo = first > base ? first - base : 0;
            const int hi = last - base < a.heads[kind] ? last - base : a.heads[kind];
            if (lo >= hi)
                continue;
            float w[N][V] = {};
#pragma unroll
            for (int n = 0; n < N; ++n)
                if ((at + n * a.lanes) * V < a.dim)
                    shared_floats<V>(&sh.w[kind][(at + n * a.lanes) * V], w[n]);
            const int es = DT == ZERO_F32 ? 4 : 2;
            const char *x = static_cast<const char *>(a.x[kind].p) + token * a.x[kind].ld * es;
            const char *y = static_cast<const char *>(a.y[kind].p) + token * a.y[kind].ld * es;
            char *dx = static_cast<char *>(const_cast<void *>(a.dx[kind].p)) + token * a.dx[kind].ld * es;
            for (int h0 = lo + sub; h0 - sub < hi; h0 += rows * U) {
                Piece<DT, V> px[U][N], py[U][N];
#pragma unroll
                for (int k = 0; k < U; ++k)
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        const int h = h0 + k * rows, e0 = (at + n * a.lanes) * V;
                        px[k][n].clear();
                        py[k][n].clear();
                        if (h < hi && e0 < a.dim) {
                            px[k][n].load(x + h * a.x[kind].hd * es, e0);
                            py[k][n].load(y + h * a.y[kind].hd * es, e0);
                        }
                    }
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    if (h0 - sub + k * rows >= hi)
                        break;
                    float f[N][V], dz[N][V], g[N][V] = {}, sq = 0.0f, dot = 0.0f;
                    if (a.rot)
                        partners<DT, V, N>(a, t, py[k], lane, g);
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        px[k][n].get(f[n]);
                        py[k][n].get(dz[n]);
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            dz[n][e] = dz[n][e] * t.c[n][e] - g[n][e] * t.s[n][e];
                            sq += f[n][e] * f[n][e];
                            dot += dz[n][e] * w[n][e] * f[n][e];
                        }
                    }
                    sq = row_sum(sq, a.lanes);
                    dot = row_sum(dot, a.lanes);
                    const float r = rsqrtf(sq * a.inv_dim + a.eps), m = dot * a.inv_dim * r * r;
                    const int h = h0 + k * rows;
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        const int e0 = (at + n * a.lanes) * V;
                        float o[V];
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            dw[kind][n][e] += dz[n][e] * (f[n][e] * r);
                            o[e] = r * (dz[n][e] * w[n][e] - f[n][e] * m);
                        }
                        Piece<DT, V> out;
                        out.put(o);
                        if (h < hi && e0 < a.dim)
                            out.store(dx + h * a.dx[kind].hd * es, e0);
                    }
                }
            }
        }
    }
    if (!a.partial)
        return;
#pragma unroll
    for (int kind = 0; kind < 2; ++kind)
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float v = dw[kind][n][e];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    if (o >= a.lanes)
                        v += __shfl_xor_sync(0xffffffffu, v, o);
                const int col = (at + n * a.lanes) * V + e;
                if (sub == 0 && col < a.dim)
                    s_dw[warp][kind][col] = v;
            }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.dim; i += kThreads) {
        const int kind = i >= a.dim, e = i - kind * a.dim;
        float v = s_dw[0][kind][e];
#pragma unroll
        for (int k = 1; k < kWarps; ++k)
            v += s_dw[k][kind][e];
        a.partial[(int64_t)blockIdx.x * 2 * a.dim + i] = v;
    }
}

// The weights' gradients from the blocks' partial sums: a block takes 32
// columns, its warps every 32nd partial, in a fixed order.
struct SumArgs {
    const float *partial;
    int32_t blocks, dim, dt;
    void *dw[2];
};

constexpr int kSumWarps = 32;

__global__ void __launch_bounds__(kSumWarps * 32) k_qk_norm_sum(const __grid_constant__ SumArgs a)
{
    __shared__ float s[kSumWarps][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int col = blockIdx.x * 32 + lane;
    pdl_wait();
    float v = 0.0f;
    if (col < 2 * a.dim)
#pragma unroll 8
        for (int b = warp; b < a.blocks; b += kSumWarps)
            v += a.partial[(int64_t)b * 2 * a.dim + col];
    s[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && col < 2 * a.dim) {
#pragma unroll
        for (int k = 1; k < kSumWarps; ++k)
            v += s[k][lane];
        const int kind = col >= a.dim;
        if (a.dw[kind])
            store1_as(a.dt, a.dw[kind], col - kind * a.dim, v);
    }
}

// ------------------------------------------------------------- host side

constexpr int64_t kMostTokens = ((int64_t)1 << 31) - 1;
constexpr int kMostSumBlocks = 152 * 8;

int check_qk(Heads *h[2], int n, int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t dim, int32_t dtype)
{
    for (int i = 0; i < n; ++i) {
        ZERO_TRY(check_heads(&h[0][i], tokens, q_heads, dim, dtype));
        ZERO_TRY(check_heads(&h[1][i], tokens, k_heads, dim, dtype));
    }
    return ZERO_OK;
}

int check_qk_sizes(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t dim, double eps, int32_t dtype,
                   int32_t wdtype, const zero_rotary_t *rotary)
{
    if (!grad_dtype_ok(dtype) || (wdtype != dtype && wdtype != ZERO_F32))
        return ZERO_EDTYPE;
    if (tokens < 0 || q_heads < 0 || k_heads < 0 || dim < 0 || !(eps >= 0))
        return ZERO_EINVAL;
    if (tokens > kMostTokens || q_heads > kMostHeads || k_heads > kMostHeads || q_heads + k_heads > kMostHeads ||
        dim > kMostDim)
        return ZERO_ESIZE;
    if (rotary && (rotary->rot_dim < 0 || rotary->rot_dim > dim || (rotary->rot_dim & 1) != 0))
        return ZERO_ESIZE;
    return ZERO_OK;
}

// Pointers to 8-byte words on the device.
int check_words(const void *p)
{
    if (!p)
        return ZERO_EINVAL;
    if ((reinterpret_cast<uintptr_t>(p) & 7u) != 0)
        return ZERO_EALIGN;
    return device_ptr(p) ? ZERO_OK : ZERO_EINVAL;
}

int check_rotary(const zero_rotary_t *rotary, const int64_t *positions, int64_t tokens)
{
    if (tokens == 0 || !rotary || rotary->rot_dim == 0)
        return ZERO_OK;
    ZERO_TRY(check_words(rotary->turns));
    return positions ? check_words(positions) : ZERO_OK;
}

// The widest piece that rows and halves of the rotation are whole numbers of
// and every row starts on.
int piece_elems(const QkArgs &a, bool backward, int es)
{
    int v = 16 / es;
    auto fits = [&](int n) {
        const int bytes = n * es;
        if (a.dim % n != 0 || (a.rot && !a.interleaved && a.rot / 2 % n != 0))
            return false;
        const Heads *all[3] = {a.x, a.y, a.dx};
        for (int i = 0; i < (backward ? 3 : 2); ++i)
            for (int k = 0; k < 2; ++k) {
                if (a.heads[k] == 0)
                    continue;
                const Heads &h = all[i][k];
                if ((reinterpret_cast<uintptr_t>(h.p) | (uintptr_t)(h.ld * es) | (uintptr_t)(h.hd * es)) & (bytes - 1))
                    return false;
            }
        return true;
    };
    while (v > 1 && !fits(v))
        v /= 2;
    return v;
}

struct QkPlan {
    int v, n;
};

// Few tokens: a token's heads are dealt out to several warps, down to one
// set of rows each, until every SM has 16 warps.
QkPlan plan_qk(QkArgs &a, bool backward, int es, int unroll)
{
    QkPlan p;
    p.v = piece_elems(a, backward, es);
    const int pieces = (a.dim + p.v - 1) / p.v;
    a.lanes = 1;
    while (a.lanes < 32 && a.lanes < pieces)
        a.lanes *= 2;
    p.n = (pieces + a.lanes - 1) / a.lanes > 1 ? 2 : 1;
    const int all = a.heads[0] + a.heads[1], rows = 32 / a.lanes;
    const int64_t want = ((int64_t)152 * 16 + a.tokens - 1) / a.tokens;
    int64_t per = (all + want - 1) / want;
    per = (per + rows - 1) / rows * rows;
    if (per < (int64_t)rows)
        per = rows;
    (void)unroll;
    a.per = (int)(per < all ? per : all);
    a.chunks = (all + a.per - 1) / a.per;
    a.units = a.tokens * a.chunks;
    return p;
}

void fill_qk(QkArgs &a, const Heads (&q)[3], const Heads (&k)[3], const void *qw, const void *kw, int32_t wdtype,
             const zero_rotary_t *rotary, const int64_t *positions, int64_t tokens, int64_t q_heads, int64_t k_heads,
             int64_t dim, double eps)
{
    a.x[0] = q[0], a.y[0] = q[1], a.dx[0] = q[2];
    a.x[1] = k[0], a.y[1] = k[1], a.dx[1] = k[2];
    a.w[0] = qw, a.w[1] = kw, a.w_f32 = wdtype == ZERO_F32;
    a.rot = rotary ? rotary->rot_dim : 0;
    a.turns = rotary ? rotary->turns : nullptr;
    a.interleaved = rotary ? rotary->interleaved != 0 : 0;
    a.positions = positions;
    a.tokens = tokens, a.heads[0] = (int32_t)q_heads, a.heads[1] = (int32_t)k_heads, a.dim = (int32_t)dim;
    a.eps = (float)eps, a.inv_dim = (float)(1.0 / (double)dim);
}

template <int DT, int V, int N>
int launch_forward(const QkArgs &a, cudaStream_t st)
{
    auto kernel = k_qk_norm<DT, V, N, N == 1 ? 4 : 1>;
    const int64_t blocks = (a.units + kWarps - 1) / kWarps;
    kernel<<<grid_for(reinterpret_cast<const void *>(kernel), blocks, 1 << 30), kThreads, 0, st>>>(a);
    return check_launch("k_qk_norm");
}

template <int DT, int V, int N>
int launch_backward(const QkArgs &a, cudaStream_t st, int *grid)
{
    auto kernel = k_qk_norm_bwd<DT, V, N, N == 1 ? 2 : 1>;
    const int64_t blocks = (a.units + kWarps - 1) / kWarps;
    *grid = grid_for(reinterpret_cast<const void *>(kernel), blocks, kMostSumBlocks);
    kernel<<<*grid, kThreads, 0, st>>>(a);
    return check_launch("k_qk_norm_bwd");
}

#define ZERO_PIECES(CALL)                                             \
    do {                                                              \
        if (dtype == ZERO_F32) {                                      \
            ZERO_WIDTHS(ZERO_F32, 4, CALL)                            \
        } else if (dtype == ZERO_F16) {                               \
            if (p.v == 8)                                             \
                return CALL(ZERO_F16, 8, 1);                          \
            ZERO_WIDTHS(ZERO_F16, 4, CALL)                            \
        } else {                                                      \
            if (p.v == 8)                                             \
                return CALL(ZERO_BF16, 8, 1);                         \
            ZERO_WIDTHS(ZERO_BF16, 4, CALL)                           \
        }                                                             \
    } while (0)
#define ZERO_WIDTHS(DT, V, CALL)                                      \
    if (p.v == V)                                                     \
        return p.n == 1 ? CALL(DT, V, 1) : CALL(DT, V, 2);            \
    if (p.v == 2)                                                     \
        return p.n == 1 ? CALL(DT, 2, 1) : CALL(DT, 2, 4);            \
    return p.n == 1 ? CALL(DT, 1, 1) : CALL(DT, 1, 8);

int forward_any(const QkArgs &a, QkPlan p, int32_t dtype, cudaStream_t st)
{
#define ZERO_FWD(DT, V, N) launch_forward<DT, V, N>(a, st)
    ZERO_PIECES(ZERO_FWD);
#undef ZERO_FWD
}

int backward_any(const QkArgs &a, QkPlan p, int32_t dtype, cudaStream_t st, int *grid)
{
#define ZERO_BWD(DT, V, N) launch_backward<DT, V, N>(a, st, grid)
    ZERO_PIECES(ZERO_BWD);
#undef ZERO_BWD
}

size_t qk_ws_bytes(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t dim)
{
    (void)tokens, (void)q_heads, (void)k_heads;
    return 256 + align256((size_t)kMostSumBlocks * 2 * (size_t)dim * sizeof(float));
}

}  // namespace
}  // namespace zpml

using namespace zpml;

extern "C" int zero_rotary_turns(const double *inv_freq, int64_t n, uint64_t *turns)
{
    if (n < 0 || (n > 0 && (!inv_freq || !turns)))
        return ZERO_EINVAL;
    for (int64_t i = 0; i < n; ++i)
        if (!(std::fabs(inv_freq[i]) <= 0x1p20))
            return ZERO_EINVAL;
    // 2 pi to 106 bits; the quotient's remainder gives its next 53
    const double hi = 6.283185307179586, lo = 2.4492935982947064e-16;
    for (int64_t i = 0; i < n; ++i) {
        const double f = std::fabs(inv_freq[i]), q = f / hi;
        const double more = (std::fma(-q, hi, f) - q * lo) / hi;
        // the whole turns go, exactly; the rest is at least 0 in units of 2^-64
        const double part = std::ldexp(q - std::floor(q), 64), lead = std::floor(part);
        const uint64_t t = (uint64_t)lead + (uint64_t)(int64_t)std::nearbyint(part - lead + std::ldexp(more, 64));
        turns[i] = inv_freq[i] < 0 ? 0 - t : t;
    }
    return ZERO_OK;
}

extern "C" int zero_qk_norm(const void *q, int64_t q_ld, int64_t q_hd, const void *k, int64_t k_ld, int64_t k_hd,
                            const void *q_weight, const void *k_weight, int32_t wdtype, const zero_rotary_t *rotary,
                            const int64_t *positions, void *q_out, int64_t q_out_ld, int64_t q_out_hd, void *k_out,
                            int64_t k_out_ld, int64_t k_out_hd, int64_t tokens, int64_t q_heads, int64_t k_heads,
                            int64_t head_dim, double eps, int32_t dtype, void *stream)
{
    ZERO_TRY(check_qk_sizes(tokens, q_heads, k_heads, head_dim, eps, dtype, wdtype, rotary));
    Heads qs[3] = {{q, q_ld, q_hd}, {q_out, q_out_ld, q_out_hd}, {}};
    Heads ks[3] = {{k, k_ld, k_hd}, {k_out, k_out_ld, k_out_hd}, {}};
    Heads *both[2] = {qs, ks};
    ZERO_TRY(check_qk(both, 2, tokens, q_heads, k_heads, head_dim, dtype));
    if (q_weight)
        ZERO_TRY(check_array(q_weight, head_dim, wdtype));
    if (k_weight)
        ZERO_TRY(check_array(k_weight, head_dim, wdtype));
    ZERO_TRY(check_rotary(rotary, positions, tokens));
    if (tokens == 0 || q_heads + k_heads == 0 || head_dim == 0)
        return ZERO_OK;
    QkArgs a{};
    fill_qk(a, qs, ks, q_weight, k_weight, wdtype, rotary, positions, tokens, q_heads, k_heads, head_dim, eps);
    return forward_any(a, plan_qk(a, false, elem_bytes(dtype), 4), dtype, static_cast<cudaStream_t>(stream));
}

extern "C" size_t zero_qk_norm_workspace_bytes(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t head_dim)
{
    if (tokens < 0 || q_heads < 0 || k_heads < 0 || head_dim < 0 || tokens > kMostTokens || q_heads > kMostHeads ||
        k_heads > kMostHeads || head_dim > kMostDim)
        return 0;
    return qk_ws_bytes(tokens, q_heads, k_heads, head_dim);
}

extern "C" int zero_qk_norm_backward(const void *dq_out, int64_t dq_out_ld, int64_t dq_out_hd, const void *dk_out,
                                     int64_t dk_out_ld, int64_t dk_out_hd, const void *q, int64_t q_ld, int64_t q_hd,
                                     const void *k, int64_t k_ld, int64_t k_hd, const void *q_weight,
                                     const void *k_weight, int32_t wdtype, const zero_rotary_t *rotary,
                                     const int64_t *positions, void *dq, int64_t dq_ld, int64_t dq_hd, void *dk,
                                     int64_t dk_ld, int64_t dk_hd, void *dq_weight, void *dk_weight, int32_t gdtype,
                                     int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t head_dim, double eps,
                                     int32_t dtype, void *ws, size_t ws_bytes, void *stream)
{
    ZERO_TRY(check_qk_sizes(tokens, q_heads, k_heads, head_dim, eps, dtype, wdtype, rotary));
    if (gdtype != dtype && gdtype != ZERO_F32)
        return ZERO_EDTYPE;
    Heads qs[3] = {{q, q_ld, q_hd}, {dq_out, dq_out_ld, dq_out_hd}, {dq, dq_ld, dq_hd}};
    Heads ks[3] = {{k, k_ld, k_hd}, {dk_out, dk_out_ld, dk_out_hd}, {dk, dk_ld, dk_hd}};
    Heads *both[2] = {qs, ks};
    ZERO_TRY(check_qk(both, 3, tokens, q_heads, k_heads, head_dim, dtype));
    if (q_weight)
        ZERO_TRY(check_array(q_weight, head_dim, wdtype));
    if (k_weight)
        ZERO_TRY(check_array(k_weight, head_dim, wdtype));
    if (dq_weight)
        ZERO_TRY(check_array(dq_weight, head_dim, gdtype));
    if (dk_weight)
        ZERO_TRY(check_array(dk_weight, head_dim, gdtype));
    ZERO_TRY(check_rotary(rotary, positions, tokens));
    ZERO_TRY(check_workspace(ws, ws_bytes, qk_ws_bytes(tokens, q_heads, k_heads, head_dim)));
    if (head_dim == 0)
        return ZERO_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    QkArgs a{};
    fill_qk(a, qs, ks, q_weight, k_weight, wdtype, rotary, positions, tokens, q_heads, k_heads, head_dim, eps);
    SumArgs s{};
    if (dq_weight || dk_weight) {
        a.partial = reinterpret_cast<float *>(static_cast<char *>(ws) + 256);
        s = {a.partial, 0, a.dim, gdtype, {dq_weight, dk_weight}};
    }
    if (tokens > 0 && q_heads + k_heads > 0)
        ZERO_TRY(backward_any(a, plan_qk(a, true, elem_bytes(dtype), 2), dtype, st, &s.blocks));
    if (!s.partial)
        return ZERO_OK;
    const cudaError_t e = launch_k(k_qk_norm_sum, (2 * a.dim + 31) / 32, kSumWarps * 32, st, s.blocks > 0, s);
    if (e != cudaSuccess) {
        cudaGetLastError();
        set_cuda_error("k_qk_norm_sum", (int)e, cudaGetErrorString(e));
        return ZERO_ECUDA;
    }
    return ZERO_OK;
}
