// Attention with a sliding window and a few first keys that stay visible,
// forward and backward, over packed sequences and caches.
#include <cmath>
#include <initializer_list>

#include "sublayer.cuh"

namespace zpml {
namespace {

constexpr int kMostDim = 128;  // of a head

// What every kernel of a call knows.
struct Attn {
    const int64_t *q_offsets, *k_offsets, *k_lengths;
    int64_t q_tokens, k_tokens;
    int32_t sequences, q_heads, k_heads, group, dim;
    int32_t window, sinks;  // at most 2^31 - 1: more than any sequence has keys
    float scale;
};

struct Seq {
    int64_t q0, k0;  // the first rows
    int32_t lq, lk;
};

__device__ __forceinline__ int64_t cut(int64_t x, int64_t lo, int64_t hi) { return x < lo ? lo : x > hi ? hi : x; }

// Sequence s, cut to the rows that there are, whatever the arrays hold.
__device__ __forceinline__ Seq sequence(const Attn &a, int32_t s)
{
    Seq q;
    q.q0 = a.q_offsets ? cut(a.q_offsets[s], 0, a.q_tokens) : 0;
    q.lq = (int32_t)((a.q_offsets ? cut(a.q_offsets[s + 1], q.q0, a.q_tokens) : a.q_tokens) - q.q0);
    if (!a.k_offsets) {
        q.k0 = q.q0, q.lk = q.lq;
        return q;
    }
    q.k0 = cut(a.k_offsets[s], 0, a.k_tokens);
    const int64_t room = cut(a.k_offsets[s + 1], q.k0, a.k_tokens) - q.k0;
    q.lk = (int32_t)(a.k_lengths ? cut(a.k_lengths[s], 0, room) : room);
    return q;
}

// The sequence that holds row `row` of `offsets`: the last that starts at or
// before it (-1: none).
__device__ __forceinline__ int32_t sequence_of(const int64_t *offsets, int32_t n, int64_t row)
{
    if (!offsets)
        return 0;
    int32_t lo = -1, hi = n;  // offsets[lo] <= row < offsets[hi]
    while (hi - lo > 1) {
        const int32_t mid = lo + (hi - lo) / 2;
        if (offsets[mid] <= row)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

struct Fwd {
    Attn a;
    Heads q, k, v, out;
    float *lse;
};

// A warp per query and head, key by key.
template <int DT>
__global__ void __launch_bounds__(kThreads) k_attn_rows(const __grid_constant__ Fwd f)
{
    const Attn &a = f.a;
    const int lane = threadIdx.x & 31;
    for (int64_t u = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5; u < a.q_tokens * a.q_heads;
         u += (int64_t)gridDim.x * kWarps) {
        const int64_t row = u / a.q_heads;
        const int32_t h = (int32_t)(u - row * a.q_heads), g = h / a.group;
        const int32_t s = sequence_of(a.q_offsets, a.sequences, row);
        if (s < 0)
            continue;
        const Seq sq = sequence(a, s);
        if (row - sq.q0 >= sq.lq)
            continue;
        const int32_t p = (int32_t)(row - sq.q0) + sq.lk - sq.lq;
        float q[4] = {}, o[4] = {}, m = -INFINITY, l = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (lane + 32 * e < a.dim)
                q[e] = load1<DT>(f.q.p, row * f.q.ld + h * f.q.hd + lane + 32 * e) * a.scale;
        for (int32_t j = 0; j <= p; ++j) {
            if (j >= a.sinks && j <= p - a.window) {
                j = p - a.window;
                continue;
            }
            const int64_t key = sq.k0 + j;
            float t = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (lane + 32 * e < a.dim)
                    t += q[e] * load1<DT>(f.k.p, key * f.k.ld + g * f.k.hd + lane + 32 * e);
#pragma unroll
            for (int x = 16; x > 0; x >>= 1)
                t += __shfl_xor_sync(0xffffffffu, t, x);
            const float top = fmaxf(m, t), keep = m == -INFINITY ? 0.0f : __expf(m - top), w = __expf(t - top);
            m = top;
            l = l * keep + w;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (lane + 32 * e < a.dim)
                    o[e] = o[e] * keep + w * load1<DT>(f.v.p, key * f.v.ld + g * f.v.hd + lane + 32 * e);
        }
        const float inv = p < 0 ? 0.0f : 1.0f / l;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (lane + 32 * e < a.dim)
                store1<DT>(const_cast<void *>(f.out.p), row * f.out.ld + h * f.out.hd + lane + 32 * e, o[e] * inv);
        if (lane == 0 && f.lse)
            f.lse[(int64_t)h * a.q_tokens + row] = p < 0 ? -INFINITY : m + logf(l);
    }
}

struct Bwd {
    Attn a;
    Heads dout, q, k, v, out, dq, dk, dv;
    const float *lse;
    float *delta;  // q_heads x q_tokens
};

__device__ __forceinline__ float warp_add(float t)
{
#pragma unroll
    for (int x = 16; x > 0; x >>= 1)
        t += __shfl_xor_sync(0xffffffffu, t, x);
    return t;
}

template <int DT>
__device__ __forceinline__ void load_row(const Heads &h, int64_t row, int64_t head, int lane, int dim, float (&f)[4])
{
#pragma unroll
    for (int e = 0; e < 4; ++e)
        f[e] = lane + 32 * e < dim ? load1<DT>(h.p, row * h.ld + head * h.hd + lane + 32 * e) : 0.0f;
}

template <int DT>
__device__ __forceinline__ void store_row(const Heads &h, int64_t row, int64_t head, int lane, int dim, const float (&f)[4])
{
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (lane + 32 * e < dim)
            store1<DT>(const_cast<void *>(h.p), row * h.ld + head * h.hd + lane + 32 * e, f[e]);
}

__device__ __forceinline__ float dot4(const float (&x)[4], const float (&y)[4])
{
    return warp_add(x[0] * y[0] + x[1] * y[1] + x[2] * y[2] + x[3] * y[3]);
}

// delta and dq: a warp per query and head.
template <int DT>
__global__ void __launch_bounds__(kThreads) k_attn_dq(const __grid_constant__ Bwd b)
{
    const Attn &a = b.a;
    const int lane = threadIdx.x & 31;
    for (int64_t u = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5; u < a.q_tokens * a.q_heads;
         u += (int64_t)gridDim.x * kWarps) {
        const int64_t row = u / a.q_heads;
        const int32_t h = (int32_t)(u - row * a.q_heads), g = h / a.group;
        const int32_t s = sequence_of(a.q_offsets, a.sequences, row);
        if (s < 0)
            continue;
        const Seq sq = sequence(a, s);
        if (row - sq.q0 >= sq.lq)
            continue;
        const int32_t p = (int32_t)(row - sq.q0) + sq.lk - sq.lq;
        float q[4], dout[4], out[4], dq[4] = {};
        load_row<DT>(b.q, row, h, lane, a.dim, q);
        load_row<DT>(b.dout, row, h, lane, a.dim, dout);
        load_row<DT>(b.out, row, h, lane, a.dim, out);
        const float delta = dot4(dout, out), lse = b.lse[(int64_t)h * a.q_tokens + row];
        if (lane == 0)
            b.delta[(int64_t)h * a.q_tokens + row] = delta;
        for (int32_t j = 0; j <= p; ++j) {
            if (j >= a.sinks && j <= p - a.window) {
                j = p - a.window;
                continue;
            }
            float k[4], v[4];
            load_row<DT>(b.k, sq.k0 + j, g, lane, a.dim, k);
            load_row<DT>(b.v, sq.k0 + j, g, lane, a.dim, v);
            const float w = __expf(dot4(q, k) * a.scale - lse), ds = w * (dot4(dout, v) - delta) * a.scale;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                dq[e] += ds * k[e];
        }
        store_row<DT>(b.dq, row, h, lane, a.dim, dq);
    }
}

// dk and dv: a warp per key and key head.
template <int DT>
__global__ void __launch_bounds__(kThreads) k_attn_dkv(const __grid_constant__ Bwd b)
{
    const Attn &a = b.a;
    const int lane = threadIdx.x & 31;
    for (int64_t u = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5; u < a.k_tokens * a.k_heads;
         u += (int64_t)gridDim.x * kWarps) {
        const int64_t key = u / a.k_heads;
        const int32_t g = (int32_t)(u - key * a.k_heads);
        const int32_t s = sequence_of(a.k_offsets ? a.k_offsets : a.q_offsets, a.sequences, key);
        if (s < 0 || s >= a.sequences)
            continue;
        const Seq sq = sequence(a, s);
        const int64_t j = key - sq.k0;
        if (j >= sq.lk)
            continue;
        float k[4], v[4], dk[4] = {}, dv[4] = {};
        load_row<DT>(b.k, key, g, lane, a.dim, k);
        load_row<DT>(b.v, key, g, lane, a.dim, v);
        const int64_t shift = sq.lk - sq.lq;
        const int64_t first = j > shift ? j : shift;
        const int64_t last = j < a.sinks || j + a.window > sq.lk ? sq.lk : j + a.window;
        for (int32_t h = g * a.group; h < (g + 1) * a.group; ++h)
            for (int64_t p = first; p < last; ++p) {
                const int64_t row = sq.q0 + p - shift;
                float q[4], dout[4];
                load_row<DT>(b.q, row, h, lane, a.dim, q);
                load_row<DT>(b.dout, row, h, lane, a.dim, dout);
                const float w = __expf(dot4(q, k) * a.scale - b.lse[(int64_t)h * a.q_tokens + row]);
                const float ds = w * (dot4(dout, v) - b.delta[(int64_t)h * a.q_tokens + row]) * a.scale;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    dk[e] += ds * q[e], dv[e] += w * dout[e];
            }
        store_row<DT>(b.dk, key, g, lane, a.dim, dk);
        store_row<DT>(b.dv, key, g, lane, a.dim, dv);
    }
}

// ------------------------------------------------------------- host side

constexpr int64_t kMostRows = ((int64_t)1 << 31) - 512;
constexpr int32_t kMostHeads = 1 << 15;

int check_attention(const zero_attention_t *a)
{
    if (!a)
        return ZERO_EINVAL;
    if (!lp_dtype_ok(a->dtype))
        return ZERO_EDTYPE;
    if (a->q_tokens < 0 || a->k_tokens < 0 || a->sequences < 0 || a->q_heads < 1 || a->k_heads < 1 ||
        a->head_dim < 1 || a->window < 1 || a->sinks < 0 || !(a->scale > 0) || !std::isfinite((float)a->scale))
        return ZERO_EINVAL;
    if (a->q_tokens > kMostRows || a->k_tokens > kMostRows || a->sequences > kMostRows || a->q_heads > kMostHeads ||
        a->q_heads % a->k_heads != 0 || a->head_dim % 8 != 0 || a->head_dim > kMostDim)
        return ZERO_ESIZE;
    return ZERO_OK;
}

// The arrays of lengths: checked by a call, not by the workspace's size.
int check_offsets(const zero_attention_t *a)
{
    if ((a->k_lengths && !a->k_offsets) || (!a->q_offsets && a->sequences != 1))
        return ZERO_EINVAL;
    if (!a->k_offsets && a->k_tokens != a->q_tokens)
        return ZERO_ESIZE;
    for (const int64_t *p : {a->q_offsets, a->k_offsets, a->k_lengths}) {
        if (!p)
            continue;
        if ((reinterpret_cast<uintptr_t>(p) & 7u) != 0)
            return ZERO_EALIGN;
        if (!device_ptr(p))
            return ZERO_EINVAL;
    }
    return ZERO_OK;
}

// An array of heads whose rows are whole 16 bytes.
int check_rows(Heads *h, int64_t tokens, int64_t heads, int64_t dim, int32_t dtype)
{
    if (tokens == 0)
        return ZERO_OK;
    ZERO_TRY(check_heads(h, tokens, heads, dim, dtype));
    return aligned16(h->p) && ((h->ld | h->hd) & 7) == 0 ? ZERO_OK : ZERO_EALIGN;
}

Attn attn_of(const zero_attention_t *a)
{
    Attn r{};
    const int64_t most = ((int64_t)1 << 31) - 1;
    r.q_offsets = a->q_offsets, r.k_offsets = a->k_offsets, r.k_lengths = a->k_lengths;
    r.q_tokens = a->q_tokens, r.k_tokens = a->k_tokens, r.sequences = (int32_t)a->sequences;
    r.q_heads = a->q_heads, r.k_heads = a->k_heads, r.group = a->q_heads / a->k_heads, r.dim = a->head_dim;
    r.window = (int32_t)(a->window < most ? a->window : most);
    r.sinks = (int32_t)(a->sinks < most ? a->sinks : most);
    r.scale = (float)a->scale;
    return r;
}

struct AttnSpace {
    size_t delta, total;
};

AttnSpace attn_space(const zero_attention_t *a, bool backward)
{
    AttnSpace s{};
    s.delta = 256;
    s.total = s.delta + (backward ? align256((size_t)a->q_heads * (size_t)a->q_tokens * 4) : 0);
    return s;
}

}  // namespace
}  // namespace zpml

using namespace zpml;

extern "C" size_t zero_window_attention_workspace_bytes(const zero_attention_t *a, int32_t backward)
{
    return check_attention(a) == ZERO_OK ? attn_space(a, backward != 0).total : 0;
}

extern "C" int zero_window_attention(const zero_attention_t *a, const void *q, int64_t q_ld, int64_t q_hd,
                                     const void *k, int64_t k_ld, int64_t k_hd, const void *v, int64_t v_ld,
                                     int64_t v_hd, void *out, int64_t out_ld, int64_t out_hd, float *lse, void *ws,
                                     size_t ws_bytes, void *stream)
{
    ZERO_TRY(check_attention(a));
    ZERO_TRY(check_offsets(a));
    Fwd f{attn_of(a), {q, q_ld, q_hd}, {k, k_ld, k_hd}, {v, v_ld, v_hd}, {out, out_ld, out_hd}, lse};
    ZERO_TRY(check_rows(&f.q, a->q_tokens, a->q_heads, a->head_dim, a->dtype));
    ZERO_TRY(check_rows(&f.k, a->k_tokens, a->k_heads, a->head_dim, a->dtype));
    ZERO_TRY(check_rows(&f.v, a->k_tokens, a->k_heads, a->head_dim, a->dtype));
    ZERO_TRY(check_rows(&f.out, a->q_tokens, a->q_heads, a->head_dim, a->dtype));
    if (lse)
        ZERO_TRY(check_array(lse, a->q_tokens, ZERO_F32));
    ZERO_TRY(check_workspace(ws, ws_bytes, attn_space(a, false).total));
    if (a->q_tokens == 0 || a->sequences == 0)
        return ZERO_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto kernel = a->dtype == ZERO_F16 ? k_attn_rows<ZERO_F16> : k_attn_rows<ZERO_BF16>;
    const int64_t blocks = (a->q_tokens * a->q_heads + kWarps - 1) / kWarps;
    kernel<<<grid_for(reinterpret_cast<const void *>(kernel), blocks, 1 << 30), kThreads, 0, st>>>(f);
    return check_launch("k_attn_rows");
}

extern "C" int zero_window_attention_backward(const zero_attention_t *a, const void *dout, int64_t dout_ld,
                                              int64_t dout_hd, const void *q, int64_t q_ld, int64_t q_hd,
                                              const void *k, int64_t k_ld, int64_t k_hd, const void *v, int64_t v_ld,
                                              int64_t v_hd, const void *out, int64_t out_ld, int64_t out_hd,
                                              const float *lse, void *dq, int64_t dq_ld, int64_t dq_hd, void *dk,
                                              int64_t dk_ld, int64_t dk_hd, void *dv, int64_t dv_ld, int64_t dv_hd,
                                              void *ws, size_t ws_bytes, void *stream)
{
    ZERO_TRY(check_attention(a));
    ZERO_TRY(check_offsets(a));
    Bwd b{attn_of(a), {dout, dout_ld, dout_hd}, {q, q_ld, q_hd}, {k, k_ld, k_hd}, {v, v_ld, v_hd},
          {out, out_ld, out_hd}, {dq, dq_ld, dq_hd}, {dk, dk_ld, dk_hd}, {dv, dv_ld, dv_hd}, lse, nullptr};
    for (Heads *h : {&b.dout, &b.q, &b.out, &b.dq})
        ZERO_TRY(check_rows(h, a->q_tokens, a->q_heads, a->head_dim, a->dtype));
    for (Heads *h : {&b.k, &b.v, &b.dk, &b.dv})
        ZERO_TRY(check_rows(h, a->k_tokens, a->k_heads, a->head_dim, a->dtype));
    ZERO_TRY(check_array(lse, a->q_tokens, ZERO_F32));
    ZERO_TRY(check_workspace(ws, ws_bytes, attn_space(a, true).total));
    b.delta = reinterpret_cast<float *>(static_cast<char *>(ws) + attn_space(a, true).delta);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (a->sequences == 0)
        return ZERO_OK;
    if (a->q_tokens > 0) {
        auto kernel = a->dtype == ZERO_F16 ? k_attn_dq<ZERO_F16> : k_attn_dq<ZERO_BF16>;
        const int64_t blocks = (a->q_tokens * a->q_heads + kWarps - 1) / kWarps;
        kernel<<<grid_for(reinterpret_cast<const void *>(kernel), blocks, 1 << 30), kThreads, 0, st>>>(b);
        ZERO_TRY(check_launch("k_attn_dq"));
    }
    if (a->k_tokens > 0) {
        auto kernel = a->dtype == ZERO_F16 ? k_attn_dkv<ZERO_F16> : k_attn_dkv<ZERO_BF16>;
        const int64_t blocks = (a->k_tokens * a->k_heads + kWarps - 1) / kWarps;
        kernel<<<grid_for(reinterpret_cast<const void *>(kernel), blocks, 1 << 30), kThreads, 0, st>>>(b);
        ZERO_TRY(check_launch("k_attn_dkv"));
    }
    return ZERO_OK;
}
