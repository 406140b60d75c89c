// The gated feed-forward block, forward and backward.
#include "sublayer.cuh"

namespace zpml {
namespace {

// ------------------------------------------------------------- the activation

// act(g) and act'(g), both through s = sigmoid(k(g)): SiLU has k(g) = g, the
// tanh form of GELU k(g) = 2 sqrt(2/pi) (g + 0.044715 g^3), because
// (1 + tanh(z)) / 2 = sigmoid(2 z).  d/dg [g s] = s + g s (1 - s) k'(g).
struct Act {
    float value, slope;
};

__device__ __forceinline__ Act activate(int32_t act, float g)
{
    constexpr float kA = 1.5957691216057308f, kB = 0.044715f;
    const float k = act == ZERO_ACT_SILU ? g : kA * (g + kB * g * g * g);
    const float dk = act == ZERO_ACT_SILU ? 1.0f : kA * (1.0f + 3.0f * kB * g * g);
    const float s = 1.0f / (1.0f + expf(-k));
    return {g * s, s + g * s * (1.0f - s) * dk};
}

// ------------------------------------------------------------- kernels

// C[m, n] = sum over the pairs p and over k of A_p[m, k] B_p[n, k], every
// operand with its own two strides.
struct Operand {
    const void *p;
    int64_t s_mn, s_k;
};

enum Epilogue {
    kStore,   // C as it is
    kGate,    // two products (the pairs are not summed): act(C0) * C1, and C0, C1 kept
    kGateBwd  // from dh = C and the kept gate and up: dgate, dup, act(gate) * up
};

struct GemmArgs {
    Operand a[2], b[2];
    int64_t k;
    int32_t pairs;
    int64_t m, n;
    int32_t act, odtype;
    void *out;  // kStore: C; kGate: act(gate) * up; kGateBwd: the same, formed again
    int64_t out_ld;
    void *o1, *o2;            // kGate: gate, up (or NULL); kGateBwd: dgate, dup
    const void *gate, *up;    // kGateBwd
    int64_t n_ld;             // row stride of o1, o2, gate, up
};

template <int DT, int EPI>
__device__ __forceinline__ void finish_element(const GemmArgs &a, int64_t m, int64_t n, float c0, float c1)
{
    if (EPI == kStore) {
        store1_as(a.odtype, a.out, m * a.out_ld + n, c0);
    } else if (EPI == kGate) {
        store1<DT>(a.out, m * a.out_ld + n, activate(a.act, c0).value * c1);
        if (a.o1) {
            store1<DT>(a.o1, m * a.n_ld + n, c0);
            store1<DT>(a.o2, m * a.n_ld + n, c1);
        }
    } else {
        const float u = load1<DT>(a.up, m * a.n_ld + n);
        const Act t = activate(a.act, load1<DT>(a.gate, m * a.n_ld + n));
        store1<DT>(a.o1, m * a.n_ld + n, c0 * u * t.slope);
        store1<DT>(a.o2, m * a.n_ld + n, c0 * t.value);
        store1<DT>(a.out, m * a.out_ld + n, t.value * u);
    }
}

// 64 x 64 tiles, 16 columns of k at a time through shared memory, 4 x 4
// elements per thread in binary32.
template <int DT, int EPI>
__global__ void __launch_bounds__(kThreads) k_ffn_product(GemmArgs a)
{
    __shared__ float sa[16][65], sb[2][16][65];
    const int64_t tiles_n = (a.n + 63) / 64;
    const int64_t m0 = (int64_t)blockIdx.x / tiles_n * 64, n0 = (int64_t)blockIdx.x % tiles_n * 64;
    const int tm = threadIdx.x >> 4, tn = threadIdx.x & 15;
    float c[2][4][4] = {};
    constexpr int kB = EPI == kGate ? 2 : 1;
    for (int p = 0; p < a.pairs; ++p)
        for (int64_t k0 = 0; k0 < a.k; k0 += 16) {
            __syncthreads();
            for (int e = threadIdx.x; e < 64 * 16; e += kThreads) {
                const int k = e & 15, i = e >> 4;
                const bool kin = k0 + k < a.k;
                sa[k][i] = kin && m0 + i < a.m ? load1<DT>(a.a[p].p, (m0 + i) * a.a[p].s_mn + (k0 + k) * a.a[p].s_k) : 0.0f;
#pragma unroll
                for (int q = 0; q < kB; ++q) {
                    const Operand &b = a.b[kB == 2 ? q : p];
                    sb[q][k][i] = kin && n0 + i < a.n ? load1<DT>(b.p, (n0 + i) * b.s_mn + (k0 + k) * b.s_k) : 0.0f;
                }
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < 16; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int q = 0; q < kB; ++q)
                            c[q][i][j] += sa[k][tm * 4 + i] * sb[q][k][tn * 4 + j];
        }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j)
            if (m0 + tm * 4 + i < a.m && n0 + tn * 4 + j < a.n)
                finish_element<DT, EPI>(a, m0 + tm * 4 + i, n0 + tn * 4 + j, c[0][i][j], c[1][i][j]);
}

template <int EPI>
int product(const GemmArgs &a, int32_t dtype, cudaStream_t st)
{
    const int64_t tiles = ((a.m + 63) / 64) * ((a.n + 63) / 64);
    if (tiles == 0)
        return ZERO_OK;
    if (tiles > 0x7fffffff)
        return ZERO_ESIZE;
    if (dtype == ZERO_F16)
        k_ffn_product<ZERO_F16, EPI><<<(unsigned)tiles, kThreads, 0, st>>>(a);
    else
        k_ffn_product<ZERO_BF16, EPI><<<(unsigned)tiles, kThreads, 0, st>>>(a);
    return check_launch("k_ffn_product");
}

// ------------------------------------------------------------- host side

constexpr int64_t kMostSize = ((int64_t)1 << 31) - 512;

int check_ffn(int64_t tokens, int64_t dim, int64_t inner, int32_t act, int32_t dtype)
{
    if (!lp_dtype_ok(dtype))
        return ZERO_EDTYPE;
    if (tokens < 0 || dim < 0 || inner < 0 || (act != ZERO_ACT_SILU && act != ZERO_ACT_GELU_TANH))
        return ZERO_EINVAL;
    if (tokens > kMostSize || dim > kMostSize || inner > kMostSize)
        return ZERO_ESIZE;
    return ZERO_OK;
}

// An operand of a product: a row-strided matrix, on 16 bytes when the widths
// are multiples of 8.
int check_operand(const void *p, int64_t ld, int64_t rows, int64_t cols, int32_t dtype, bool whole)
{
    const int rc = check_matrix(p, ld, rows, cols, dtype);
    if (rc != ZERO_OK || rows == 0 || cols == 0)
        return rc;
    return whole && (!aligned16(p) || (ld & 7) != 0) ? ZERO_EALIGN : ZERO_OK;
}

}  // namespace
}  // namespace zpml

using namespace zpml;

extern "C" size_t zero_gated_ffn_workspace_bytes(int64_t tokens, int64_t dim, int64_t inner, int32_t backward)
{
    (void)dim;
    if (tokens < 0 || inner < 0)
        return 0;
    return 256 + (backward ? 3 : 1) * align256((size_t)tokens * (size_t)inner * 2);
}

extern "C" int zero_gated_ffn(const void *x, int64_t x_ld, const void *w_gate, const void *w_up, const void *w_down,
                              void *y, int64_t y_ld, void *gate, void *up, int64_t tokens, int64_t dim, int64_t inner,
                              int32_t act, int32_t dtype, void *ws, size_t ws_bytes, void *stream)
{
    ZERO_TRY(check_ffn(tokens, dim, inner, act, dtype));
    if ((gate != nullptr) != (up != nullptr))
        return ZERO_EINVAL;
    const bool whole = ((dim | inner) & 7) == 0;
    ZERO_TRY(check_operand(x, x_ld, tokens, dim, dtype, whole));
    ZERO_TRY(check_operand(w_gate, dim, inner, dim, dtype, whole));
    ZERO_TRY(check_operand(w_up, dim, inner, dim, dtype, whole));
    ZERO_TRY(check_operand(w_down, inner, dim, inner, dtype, whole));
    ZERO_TRY(check_matrix(y, y_ld, tokens, dim, dtype));
    if (gate) {
        ZERO_TRY(check_matrix(gate, inner, tokens, inner, dtype));
        ZERO_TRY(check_matrix(up, inner, tokens, inner, dtype));
    }
    ZERO_TRY(check_workspace(ws, ws_bytes, zero_gated_ffn_workspace_bytes(tokens, dim, inner, 0)));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    void *h = static_cast<char *>(ws) + 256;
    GemmArgs g{};
    g.a[0] = {x, x_ld, 1};
    g.b[0] = {w_gate, dim, 1}, g.b[1] = {w_up, dim, 1};
    g.k = dim, g.pairs = 1, g.m = tokens, g.n = inner, g.act = act;
    g.out = h, g.out_ld = inner, g.o1 = gate, g.o2 = up, g.n_ld = inner;
    ZERO_TRY(product<kGate>(g, dtype, st));
    GemmArgs d{};
    d.a[0] = {h, inner, 1};
    d.b[0] = {w_down, inner, 1};
    d.k = inner, d.pairs = 1, d.m = tokens, d.n = dim;
    d.out = y, d.out_ld = y_ld, d.odtype = dtype;
    return product<kStore>(d, dtype, st);
}

extern "C" int zero_gated_ffn_backward(const void *dy, int64_t dy_ld, const void *x, int64_t x_ld, const void *w_gate,
                                       const void *w_up, const void *w_down, const void *gate, const void *up,
                                       void *dx, int64_t dx_ld, void *dw_gate, void *dw_up, void *dw_down,
                                       int32_t gdtype, int64_t tokens, int64_t dim, int64_t inner, int32_t act,
                                       int32_t dtype, void *ws, size_t ws_bytes, void *stream)
{
    ZERO_TRY(check_ffn(tokens, dim, inner, act, dtype));
    if (gdtype != dtype && gdtype != ZERO_F32)
        return ZERO_EDTYPE;
    const bool whole = ((dim | inner) & 7) == 0;
    ZERO_TRY(check_operand(dy, dy_ld, tokens, dim, dtype, whole));
    ZERO_TRY(check_operand(x, x_ld, tokens, dim, dtype, whole));
    ZERO_TRY(check_operand(w_gate, dim, inner, dim, dtype, whole));
    ZERO_TRY(check_operand(w_up, dim, inner, dim, dtype, whole));
    ZERO_TRY(check_operand(w_down, inner, dim, inner, dtype, whole));
    ZERO_TRY(check_matrix(gate, inner, tokens, inner, dtype));
    ZERO_TRY(check_matrix(up, inner, tokens, inner, dtype));
    ZERO_TRY(check_matrix(dx, dx_ld, tokens, dim, dtype));
    ZERO_TRY(check_matrix(dw_gate, dim, inner, dim, gdtype));
    ZERO_TRY(check_matrix(dw_up, dim, inner, dim, gdtype));
    ZERO_TRY(check_matrix(dw_down, inner, dim, inner, gdtype));
    ZERO_TRY(check_workspace(ws, ws_bytes, zero_gated_ffn_workspace_bytes(tokens, dim, inner, 1)));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const size_t mf = align256((size_t)tokens * (size_t)inner * 2);
    char *dg = static_cast<char *>(ws) + 256, *du = dg + mf, *h = du + mf;
    GemmArgs g{};  // dh, and from it dgate, dup and h
    g.a[0] = {dy, dy_ld, 1};
    g.b[0] = {w_down, 1, inner};
    g.k = dim, g.pairs = 1, g.m = tokens, g.n = inner, g.act = act;
    g.out = h, g.out_ld = inner, g.o1 = dg, g.o2 = du, g.gate = gate, g.up = up, g.n_ld = inner;
    ZERO_TRY(product<kGateBwd>(g, dtype, st));
    GemmArgs d{};  // dx
    d.a[0] = {dg, inner, 1}, d.a[1] = {du, inner, 1};
    d.b[0] = {w_gate, 1, dim}, d.b[1] = {w_up, 1, dim};
    d.k = inner, d.pairs = 2, d.m = tokens, d.n = dim, d.out = dx, d.out_ld = dx_ld, d.odtype = dtype;
    ZERO_TRY(product<kStore>(d, dtype, st));
    GemmArgs w{};  // the weight gradients
    w.k = tokens, w.pairs = 1, w.odtype = gdtype;
    w.m = inner, w.n = dim, w.out_ld = dim;
    w.b[0] = {x, 1, x_ld};
    w.a[0] = {dg, 1, inner}, w.out = dw_gate;
    ZERO_TRY(product<kStore>(w, dtype, st));
    w.a[0] = {du, 1, inner}, w.out = dw_up;
    ZERO_TRY(product<kStore>(w, dtype, st));
    w.m = dim, w.n = inner, w.out_ld = inner;
    w.a[0] = {dy, 1, dy_ld}, w.b[0] = {h, 1, inner}, w.out = dw_down;
    return product<kStore>(w, dtype, st);
}
