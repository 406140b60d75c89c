// Dropout with the residual sum, and layer norm (alone or with that sum in
// front of it), forward and backward.
#include <cmath>
#include <initializer_list>
#include <type_traits>

#include "sublayer.cuh"

namespace zpml {
namespace {

// ------------------------------------------------------------- the mask

// Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", 2011): ten rounds of two 32 x 32 -> 64 bit products on a
// 128-bit counter, the key moved on by a constant per round.  Here word 0 of
// the counter is the column's quad, word 1 the row and words 2 and 3 the
// offset, so one product of each of the first two rounds is the row's alone
// (RowMask), and the keys of all rounds come as launch constants: 38
// instructions per four elements instead of 60, which is what bounds the
// kernels below after memory.
constexpr uint32_t kPhilox0 = 0xD2511F53u, kPhilox1 = 0xCD9E8D57u;

// The 64-bit product as one instruction (written as a C product whose halves
// are used apart, it became two).
__device__ __forceinline__ uint64_t wide(uint32_t a, uint32_t b)
{
    uint64_t r;
    asm("mul.wide.u32 %0, %1, %2;" : "=l"(r) : "r"(a), "r"(b));
    return r;
}

// A dropout as the kernels take it.
struct Drop {
    const uint64_t *d_offset;
    uint64_t offset;
    uint32_t key[10][2];  // of each round
    uint32_t threshold;   // kept iff the word is at least this ...
    uint32_t all;         // ... and not everything is dropped (p = 1)
    float scale;
};

__device__ __forceinline__ uint64_t drop_offset(const Drop &d)
{
    return d.d_offset ? d.offset + *d.d_offset : d.offset;
}

struct RowMask {
    uint32_t w0, w2, w3;  // what a row and an offset put into the state after two rounds
    uint32_t first;       // and into word 2 after the first
};

__device__ __forceinline__ RowMask row_mask(const Drop &d, uint64_t off, int64_t row)
{
    const uint64_t b = wide(kPhilox1, (uint32_t)off);
    const uint64_t a = wide(kPhilox0, (uint32_t)(b >> 32) ^ (uint32_t)row ^ d.key[0][0]);
    return {(uint32_t)b ^ d.key[1][0], (uint32_t)(a >> 32) ^ d.key[1][1], (uint32_t)a, (uint32_t)(off >> 32) ^ d.key[0][1]};
}

// The four words of the columns 4 quad .. 4 quad + 3.
__device__ __forceinline__ uint4 mask_words(const Drop &d, const RowMask &m, uint32_t quad)
{
    const uint64_t a1 = wide(kPhilox0, quad);
    const uint64_t b2 = wide(kPhilox1, (uint32_t)(a1 >> 32) ^ m.first);
    uint4 c = make_uint4((uint32_t)(b2 >> 32) ^ m.w0, (uint32_t)b2, m.w2 ^ (uint32_t)a1, m.w3);
#pragma unroll
    for (int r = 2; r < 10; ++r) {
        const uint64_t a = wide(kPhilox0, c.x), b = wide(kPhilox1, c.z);
        c = make_uint4((uint32_t)(b >> 32) ^ c.y ^ d.key[r][0], (uint32_t)b, (uint32_t)(a >> 32) ^ c.w ^ d.key[r][1],
                       (uint32_t)a);
    }
    return c;
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

// (rows are fewer than 2^32)
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

    // as pairs, for the two-element binary32 instructions
    __device__ __forceinline__ void to_pairs(float2 (&f)[4]) const
    {
        float t[8];
        Elem<DT>::to_float(w, t);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            f[k] = make_float2(t[2 * k], t[2 * k + 1]);
    }
};

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

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

// Zeros what the words drop (kAll: everything may be).
template <bool kAll>
__device__ __forceinline__ void drop_words(const Drop &d, const uint32_t (&w)[8], float (&f)[8])
{
    if (kAll && d.all) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            f[e] = 0.0f;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            f[e] = w[e] >= d.threshold ? f[e] : 0.0f;
    }
}

// Zeros the dropped ones of the eight columns from c0 on (the scale is left to
// the caller).  c0 is 0 mod 4 unless the rows are shifted: then a group spans
// three counters, and the third is the first of the next lane's group.  So
// the kernels give a warp 31 groups of a row that is not whole (lane_group),
// its last lane works out masks for its neighbour alone, and all lanes of a
// warp come here together.
template <bool kW, bool kAll = true>
__device__ __forceinline__ void keep_group(const Drop &d, const RowMask &m, int64_t c0, float (&f)[8])
{
    uint32_t w[8];
    const uint32_t quad = (uint32_t)(c0 >> 2);
    const uint4 a = mask_words(d, m, quad), b = mask_words(d, m, quad + 1);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    if (!kW) {
        const int o = (int)(c0 & 3);
        const uint32_t n0 = __shfl_down_sync(0xffffffffu, a.x, 1), n1 = __shfl_down_sync(0xffffffffu, a.y, 1),
                       n2 = __shfl_down_sync(0xffffffffu, a.z, 1);
        if (o & 1) {
#pragma unroll
            for (int k = 0; k < 7; ++k)
                w[k] = w[k + 1];
            w[7] = n0;
        }
        if (o & 2) {
#pragma unroll
            for (int k = 0; k < 6; ++k)
                w[k] = w[k + 2];
            w[6] = o & 1 ? n1 : n0;
            w[7] = o & 1 ? n2 : n1;
        }
    }
    drop_words<kAll>(d, w, f);
}

// The group of thread t of a row's threads, and whether it is the thread's
// own (see keep_group).
template <bool kW>
__device__ __forceinline__ int lane_group(int t)
{
    return kW ? t : (t >> 5) * 31 + (t & 31);
}

template <bool kW>
__device__ __forceinline__ bool owns_group()
{
    return kW || (threadIdx.x & 31) != 31;
}

template <bool kW, bool kAll = true>
__device__ __forceinline__ void keep_pairs(const Drop &d, const RowMask &m, int64_t c0, float2 (&f)[4])
{
    float t[8];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        t[2 * k] = f[k].x, t[2 * k + 1] = f[k].y;
    keep_group<kW, kAll>(d, m, c0, t);
#pragma unroll
    for (int k = 0; k < 4; ++k)
        f[k] = make_float2(t[2 * k], t[2 * k + 1]);
}

template <int DT, bool kW, class I>
__device__ __forceinline__ void store_pairs(char *row, I c0, I cols, bool vec, const float2 (&f)[4])
{
    float t[8];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        t[2 * k] = f[k].x, t[2 * k + 1] = f[k].y;
    store_group<DT, kW>(row, c0, cols, vec, t);
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

template <int DT, bool kW, class I>
__device__ __forceinline__ void load_vector(const void *p, bool f32, I c0, I cols, bool vec, float none,
                                            float2 (&f)[4])
{
    float t[8];
    load_vector<DT, kW>(p, f32, c0, cols, vec, none, t);
#pragma unroll
    for (int k = 0; k < 4; ++k)
        f[k] = make_float2(t[2 * k], t[2 * k + 1]);
}

// ------------------------------------------------------------- dropout

struct DropoutArgs {
    Matrix x, res, out;
    Rows rows;
    uint32_t groups;  // per row
    FastDiv per_row;
    uint32_t step_rows, step_groups;  // what the whole grid advances by
    Drop d;
};

// One thread per group, the grid striding over all groups.  32 blocks per SM
// (four waves of them) leave no SM idle at the end: 16384 x 8192 bfloat16
// with a residual takes 122 us (6.6 TB/s), one wave of eight blocks 130.
// Without a residual the masks' wide multiplications, four cycles of a
// scheduler's pipe each, are the limit (109 us).  Two groups at a time per
// thread, for more loads in flight, took 148 us.
template <int DT, bool kW>
__global__ void __launch_bounds__(kThreads) k_dropout_add(const __grid_constant__ DropoutArgs a)
{
    const uint32_t flat = kW ? blockIdx.x * kThreads + threadIdx.x
                             : (blockIdx.x * kWarps + (threadIdx.x >> 5)) * 31 + (threadIdx.x & 31);
    const uint32_t row = fast_div(flat, a.per_row);
    int64_t r = row;
    uint32_t g = flat - row * a.groups;
    const uint64_t off = drop_offset(a.d);
    const int64_t cols = a.rows.cols;
    const bool vec = a.rows.kind != kLoose, mine = owns_group<kW>();
    // (rows that are not whole: until the whole warp has left the matrix)
    while (kW ? r < a.rows.rows : __any_sync(0xffffffffu, r < a.rows.rows)) {
        const int64_t c0 = (int64_t)g * 8 - row_shift<kW>(a.rows, r);
        const bool in = kW || (mine && r < a.rows.rows && c0 < cols);
        float f[8] = {}, t[8];
        Group<DT> y{};
        if (in) {
            load_group<DT, kW, false>(row_ptr<DT>(a.x, r), c0, cols, vec).to_float(f);
            if (a.res.p)
                y = load_group<DT, kW, false>(row_ptr<DT>(a.res, r), c0, cols, vec);
        }
        keep_group<kW>(a.d, row_mask(a.d, off, r), c0, f);
        y.to_float(t);  // zeros without a residual
#pragma unroll
        for (int e = 0; e < 8; ++e)
            f[e] = f[e] * a.d.scale + t[e];
        if (in)
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

// Sum over the threads of a row: a team of `tpr` threads (whole warps) with
// its own named barrier; s: a slot per warp of the team.
__device__ __forceinline__ float team_sum(float v, float *s, int tpr, int team, int t)
{
    v = warp_sum_f(v);
    if (tpr == 32)
        return v;
    if ((t & 31) == 0)
        s[t >> 5] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(tpr) : "memory");
    v = (t & 31) < (tpr >> 5) ? s[t & 31] : 0.0f;
    for (int o = 1; o < (tpr >> 5); o <<= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return __shfl_sync(0xffffffffu, v, 0);
}

struct NormArgs {
    Matrix x, res, sum, y;
    const void *weight, *bias;
    int32_t w_f32, w_vec;  // weight and bias are binary32; their groups are whole 16 bytes
    float *mean, *rstd;
    Rows rows;
    float eps, cols, inv_cols;
    int32_t dropping;
    int32_t tpr;  // threads per row
    Drop d;
};

// sum / cols, correctly rounded: the product with the rounded reciprocal, put
// right by what it leaves of the sum (Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990).  The product alone
// is a unit in the last place off at times, which a row of equal values shows:
// 1601 values of 1000 gave y = -0.02, a deviation of 2^-14 at an rstd of 316,
// where it is 0.  (An infinite sum has an infinite mean, and leaves nothing.)
__device__ __forceinline__ float row_mean(float sum, const NormArgs &a)
{
    const float q = sum * a.inv_cols, left = fmaf(-q, a.cols, sum);
    return left == left ? fmaf(left, a.inv_cols, q) : q;
}

// Forward: a row in the registers of a team of tpr threads, NV groups of
// columns each, read once; mean, then the squared deviations from it, then
// the output.  A thread keeps its columns (the rows of a team are a multiple
// of 8 apart, so their shift is the same), and with up to two groups also
// their weight and bias, and has the next row on its way while it works on
// this one (four groups of binary32 leave no registers for that; of 16 bits,
// 4096 x 16384: 73 us with it, 98 without).  One row of 1600 takes 2.3 us,
// which is a launch and two trips to memory; 8192 x 1600 binary32 23.0
// (4.6 TB/s), bounded by the instructions of a row's two sums and its ends.
template <int DT, int NV, bool kFused, bool kW, int THREADS>
__global__ void __launch_bounds__(THREADS) k_norm_fwd(const __grid_constant__ NormArgs a)
{
    constexpr bool kKeep = NV <= 2, kAhead = NV <= 2 || DT != ZERO_F32;
    __shared__ float s_red[2][32];
    const int tpr = a.tpr, team = threadIdx.x / tpr, t0 = threadIdx.x - team * tpr, teams = blockDim.x / tpr;
    float *const red0 = s_red[0] + team * (tpr >> 5), *const red1 = s_red[1] + team * (tpr >> 5);
    const uint64_t off = kFused && a.dropping ? drop_offset(a.d) : 0;
    const int cols = (int)a.rows.cols;
    const bool vec = a.rows.kind != kLoose;
    const int64_t step = (int64_t)gridDim.x * teams;
    int64_t r = (int64_t)blockIdx.x * teams + team;
    const int at = lane_group<kW>(t0) * 8 - row_shift<kW>(a.rows, r);
    const int wide = kW ? tpr * 8 : (tpr >> 5) * 31 * 8;  // columns from one of a thread's groups to the next
    const bool mine = owns_group<kW>();
    float2 w[kKeep ? NV : 1][4], b[kKeep ? NV : 1][4];
    const float2 scale = both(kFused && a.dropping ? a.d.scale : 1.0f);
    if (kKeep) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c0 = at + v * wide;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                w[kKeep ? v : 0][k] = b[kKeep ? v : 0][k] = both(0.0f);
            if (mine && c0 < cols) {
                load_vector<DT, kW>(a.weight, a.w_f32, c0, cols, a.w_vec, 1.0f, w[kKeep ? v : 0]);
                load_vector<DT, kW>(a.bias, a.w_f32, c0, cols, a.w_vec, 0.0f, b[kKeep ? v : 0]);
            }
        }
    }
    Group<DT> raw[NV], add[kFused ? NV : 1];
    auto fetch = [&](int64_t row) {
        if (row >= a.rows.rows)
            return;
        const char *px = row_ptr<DT>(a.x, row), *pr = row_ptr<DT>(a.res, row);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c0 = at + v * wide;
            if (mine && c0 < cols) {
                raw[v] = load_group<DT, kW>(px, c0, cols, vec);
                if (kFused && a.res.p)
                    add[kFused ? v : 0] = load_group<DT, kW>(pr, c0, cols, vec);
            }
        }
    };
#pragma unroll
    for (int v = 0; v < NV; ++v)
        raw[v] = add[kFused ? v : 0] = Group<DT>{};
    if (kAhead)
        fetch(r);
    for (; r < a.rows.rows; r += step) {
        if (!kAhead)
            fetch(r);
        RowMask mask{};
        if (kFused && a.dropping)
            mask = row_mask(a.d, off, r);
        char *const ps = row_ptr<DT>(a.sum, r), *const py = row_ptr<DT>(a.y, r);
        float2 t[NV][4], s = both(0.0f);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c0 = at + v * wide;
            raw[v].to_pairs(t[v]);
            // (a warp stays together unless its rows are whole)
            if (kFused && a.dropping && (kW ? c0 : c0 - (int)(threadIdx.x & 31) * 8) < cols)
                keep_pairs<kW>(a.d, mask, c0, t[v]);
            if (kFused && mine && c0 < cols) {
                float2 x[4];
                add[kFused ? v : 0].to_pairs(x);  // zeros without a residual
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    t[v][k] = __ffma2_rn(t[v][k], scale, x[k]);
                store_pairs<DT, kW>(ps, c0, cols, vec, t[v]);
            }
            // elements outside the row are 0 here
#pragma unroll
            for (int k = 0; k < 4; ++k)
                s = __fadd2_rn(s, t[v][k]);
        }
        if (kAhead)
            fetch(r + step);
        const float mean = row_mean(team_sum(s.x + s.y, red0, tpr, team, t0), a);
        s = both(0.0f);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c0 = at + v * wide;
            if (mine && c0 < cols) {
                const bool full = kW || (c0 >= 0 && c0 + 8 <= cols);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    t[v][k] = __fadd2_rn(t[v][k], both(-mean));
                    if (!full) {
                        t[v][k].x = inside<kW>(c0, 2 * k, cols) ? t[v][k].x : 0.0f;
                        t[v][k].y = inside<kW>(c0, 2 * k + 1, cols) ? t[v][k].y : 0.0f;
                    }
                    s = __ffma2_rn(t[v][k], t[v][k], s);
                }
            }
        }
        const float rstd = __frsqrt_rn(team_sum(s.x + s.y, red1, tpr, team, t0) * a.inv_cols + a.eps);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c0 = at + v * wide;
            if (mine && c0 < cols) {
                if (!kKeep) {
                    load_vector<DT, kW>(a.weight, a.w_f32, c0, cols, a.w_vec, 1.0f, w[0]);
                    load_vector<DT, kW>(a.bias, a.w_f32, c0, cols, a.w_vec, 0.0f, b[0]);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    t[v][k] = __ffma2_rn(__fmul2_rn(t[v][k], both(rstd)), w[kKeep ? v : 0][k], b[kKeep ? v : 0][k]);
                store_pairs<DT, kW>(py, c0, cols, vec, t[v]);
            }
        }
        if (t0 == 0) {
            if (a.mean)
                a.mean[r] = mean;
            if (a.rstd)
                a.rstd[r] = rstd;
        }
    }
}

// Sixteen bytes of memory to shared memory without registers between, or as
// many zeros if not `there` (memory is then not read); each thread waits for
// its own copies alone and reads them alone.
__device__ __forceinline__ void copy16(void *to, const void *from, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from),
                 "r"(there ? 16 : 0)
                 : "memory");
}

__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Threads of a block of the kernel below: the registers of NV groups decide.
constexpr int norm_rows_threads(int nv) { return nv <= 3 ? 1024 : nv <= 4 ? 896 : nv <= 6 ? 768 : nv == 7 ? 640 : 512; }

// Forward of whole rows of 16-bit elements, for many rows: teams of T warps
// that take a row each, one warp where the row fits its registers (no barrier
// then, and no idle lanes but in the last group).  A lane keeps its NV groups
// in binary32, weight and bias lie in shared memory in binary32, and a group's
// copy of the next row is under way as soon as this row's has been read, so
// registers hold no row ahead and an SM more rows at once.  Straight-line code
// over the groups: 208 instructions per group with sum and mask, where
// k_norm_fwd takes 290 and a barrier.  8192 x 1600 float16: 12.1 us (4.3 TB/s)
// where k_norm_fwd takes 15.5; with sum and mask 24.4 (4.3 TB/s) and 31.9;
// 16384 x 8192: 100 (5.4 TB/s) and 122.  The issue of the mask's multiplications
// and the start and end of the launch are what is left over the copy's time.
// Rows of binary32 stay with k_norm_fwd: staged they are twice as long, so half
// the warps fit (8192 x 1600: 28.7 us staged, 23.0 there).
template <int DT, int NV, int T, bool kFused>
__global__ void __launch_bounds__(norm_rows_threads(NV)) k_norm_fwd_rows(const __grid_constant__ NormArgs a)
{
    constexpr int kNext = T * 32;  // groups from one of a lane's to the next
    // No copy is under way when the block gives its memory back.  Of a row that
    // is not there, copies are either zeros, which the end waits for, or not
    // issued: one warp per row with the sum has no registers for the branch
    // (8192 x 1600: 24.3 us with zeros, 24.7 without), the others none for the
    // wait (8192 x 2560 without the sum 21.7 and 17.8, 16384 x 8192 with it 191
    // and 179).
    constexpr bool kZeros = kFused && T == 1;
    extern __shared__ float4 s_rows[];
    __shared__ float s_red[2][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, team = warp / T, teams = blockDim.x / kNext;
    const int cols = (int)a.rows.cols, groups = cols >> 3, g0 = warp % T * 32 + lane;
    // weight, then bias: the first and the last four columns of each group apart
    float4 *const vec = s_rows;
    uint4 *const in = reinterpret_cast<uint4 *>(s_rows + 4 * groups) + warp * (kFused ? 2 : 1) * NV * 32 + lane;
    const int64_t step = (int64_t)gridDim.x * teams;
    int64_t r = (int64_t)blockIdx.x * teams + team;
    // (T = 1: only the last group may be outside the row; else the last two)
    auto has = [&](int v) { return v < NV - (T == 1 ? 1 : 2) || g0 + v * kNext < groups; };
    auto fetch = [&](int64_t row, int v) {
        const bool there = row < a.rows.rows;
        if (!kZeros && !there)
            return;
        copy16(in + v * 32, row_ptr<DT>(a.x, row) + (g0 + v * kNext) * 16, there);
        if (kFused)
            copy16(in + (NV + v) * 32, row_ptr<DT>(a.res, row) + (g0 + v * kNext) * 16, there && a.res.p);
    };
    auto sum_of = [&](float2 s, int which) {
        const float v = warp_sum_f(s.x + s.y);
        if (T == 1)
            return v;
        float *const red = s_red[which] + team * T;
        if (lane == 0)
            red[warp % T] = v;
        asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(kNext) : "memory");
        float sum = red[0];
#pragma unroll
        for (int q = 1; q < T; ++q)
            sum += red[q];
        return sum;
    };
#pragma unroll
    for (int v = 0; v < NV; ++v)
        if (has(v))
            fetch(r, v);
    for (int i = threadIdx.x; i < cols; i += blockDim.x) {
        float *const to = reinterpret_cast<float *>(vec + (i >> 2 & 1) * groups + (i >> 3)) + (i & 3);
        to[0] = !a.weight ? 1.0f : a.w_f32 ? load1<ZERO_F32>(a.weight, i) : load1<DT>(a.weight, i);
        to[8 * groups] = !a.bias ? 0.0f : a.w_f32 ? load1<ZERO_F32>(a.bias, i) : load1<DT>(a.bias, i);
    }
    __syncthreads();
    const uint64_t off = kFused && a.dropping ? drop_offset(a.d) : 0;
    const float2 scale = both(kFused && a.dropping ? a.d.scale : 1.0f);
    for (; r < a.rows.rows; r += step) {
        RowMask mask{};
        if (kFused && a.dropping)
            mask = row_mask(a.d, off, r);
        char *const ps = row_ptr<DT>(a.sum, r) + g0 * 16, *const py = row_ptr<DT>(a.y, r) + g0 * 16;
        float2 t[NV][4], s = both(0.0f);
        copies_done();
        auto first = [&](auto dropping) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    t[v][k] = both(0.0f);
                if (has(v)) {
                    Group<DT> g;
                    g.w[0] = in[v * 32];
                    g.to_pairs(t[v]);
                    if (kFused) {
                        if (dropping)
                            keep_pairs<true, false>(a.d, mask, (g0 + kNext * v) * 8, t[v]);
                        float2 x[4];
                        g.w[0] = in[(NV + v) * 32];
                        g.to_pairs(x);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            t[v][k] = __ffma2_rn(t[v][k], scale, x[k]);
                        store_pairs<DT, true>(ps, v * kNext * 8, cols, true, t[v]);
                    }
                    fetch(r + step, v);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    s = __fadd2_rn(s, t[v][k]);
            }
        };
        if (kFused && a.dropping)
            first(std::true_type{});
        else
            first(std::false_type{});
        const float mean = row_mean(sum_of(s, 0), a);
        s = both(0.0f);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float2 q = both(0.0f);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                t[v][k] = __fadd2_rn(t[v][k], both(-mean));
                q = __ffma2_rn(t[v][k], t[v][k], q);
            }
            if (has(v))
                s = __fadd2_rn(s, q);
        }
        const float rstd = __frsqrt_rn(sum_of(s, 1) * a.inv_cols + a.eps);
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (has(v)) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float4 w = vec[h * groups + g0 + kNext * v], b = vec[(2 + h) * groups + g0 + kNext * v];
                    float2 &t0 = t[v][2 * h], &t1 = t[v][2 * h + 1];
                    t0 = __ffma2_rn(__fmul2_rn(t0, both(rstd)), make_float2(w.x, w.y), make_float2(b.x, b.y));
                    t1 = __ffma2_rn(__fmul2_rn(t1, both(rstd)), make_float2(w.z, w.w), make_float2(b.z, b.w));
                }
                store_pairs<DT, true>(py, v * kNext * 8, cols, true, t[v]);
            }
        if (g0 == 0) {
            if (a.mean)
                a.mean[r] = mean;
            if (a.rstd)
                a.rstd[r] = rstd;
        }
    }
    if (kZeros)
        copies_done();
}

// Forward of rows too wide for the registers of a block: three passes over
// the row (the later two from L2), bounded by their latency, one after the
// other.
template <int DT>
__global__ void __launch_bounds__(512) k_norm_fwd_wide(const __grid_constant__ NormArgs a)
{
    __shared__ float s_red[2][32];
    const uint64_t off = a.dropping ? drop_offset(a.d) : 0;
    const int64_t cols = a.rows.cols, step = (int64_t)(blockDim.x >> 5) * 31 * 8;
    const bool mine = owns_group<false>();
    const bool vec = a.rows.kind != kLoose;
    for (int64_t r = blockIdx.x; r < a.rows.rows; r += gridDim.x) {
        const int64_t first = -(int64_t)row_shift<false>(a.rows, r), at = lane_group<false>(threadIdx.x) * 8;
        const RowMask mask = row_mask(a.d, off, r);
        // the whole warp together, for keep_group
        auto value = [&](int64_t c0, float(&t)[8]) {
            const bool in = mine && c0 < cols;
            Group<DT> x{}, y{};
            if (in) {
                x = load_group<DT, false>(row_ptr<DT>(a.x, r), c0, cols, vec);
                if (a.res.p)
                    y = load_group<DT, false>(row_ptr<DT>(a.res, r), c0, cols, vec);
            }
            x.to_float(t);
            if (a.dropping) {
                keep_group<false>(a.d, mask, c0, t);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    t[e] *= a.d.scale;
            }
            float z[8];
            y.to_float(z);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                t[e] += z[e];
        };
        float s = 0.0f, t[8];
        for (int64_t pass = first; pass < cols; pass += step) {
            const int64_t c0 = pass + at;
            value(c0, t);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                s += t[e];
        }
        const float mean = row_mean(team_sum(s, s_red[0], 512, 0, threadIdx.x), a);
        s = 0.0f;
        for (int64_t pass = first; pass < cols; pass += step) {
            const int64_t c0 = pass + at;
            value(c0, t);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (mine && c0 + e >= 0 && c0 + e < cols)
                    s += (t[e] - mean) * (t[e] - mean);
        }
        const float rstd = __frsqrt_rn(team_sum(s, s_red[1], 512, 0, threadIdx.x) * a.inv_cols + a.eps);
        for (int64_t pass = first; pass < cols; pass += step) {
            const int64_t c0 = pass + at;
            float w[8], b[8];
            value(c0, t);
            if (!mine || c0 >= cols)
                continue;
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

// Two sums over a warp: the halves exchange one of the two, then each half
// adds up its own (five shuffles, one more to share the results).  Lanes below
// 16 end with the sum of x, the others with that of y.
__device__ __forceinline__ float half_sums(float2 v)
{
    const bool hi = (threadIdx.x & 16) != 0;
    float k = hi ? v.y : v.x;
    k += __shfl_xor_sync(0xffffffffu, hi ? v.x : v.y, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
        k += __shfl_xor_sync(0xffffffffu, k, o);
    return k;
}

__device__ __forceinline__ float2 both_sums(float k)
{
    const float other = __shfl_xor_sync(0xffffffffu, k, 16);
    return (threadIdx.x & 16) != 0 ? make_float2(other, k) : make_float2(k, other);
}

// Two sums over the threads of a row group (tpr threads of the block, its
// own named barrier), in a buffer that alternates from row to row.
__device__ __forceinline__ float2 group_sum2(float2 v, float2 *s, int tpr, int group, int t)
{
    const float k = half_sums(v);
    if (tpr == 32)
        return both_sums(k);
    if ((t & 15) == 0)
        (t & 16 ? s[t >> 5].y : s[t >> 5].x) = k;
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(tpr) : "memory");
    return both_sums(half_sums((t & 31) < (tpr >> 5) ? s[t & 31] : make_float2(0.0f, 0.0f)));
}

// Backward: a block of several row groups of tpr threads, each thread with NV
// groups of columns, which stay its own from row to row, so that dweight and
// dbias build up in its registers.  Rows are taken NG = gridDim * (groups per
// block) apart; NG is a multiple of 8 when a group takes more than one row,
// so that its rows all have the same shift.  The next row is loaded before
// the sums of this one are exchanged; a row is held as it came (16-bit) and
// converted again after the exchange.  3001 x 2049 binary32: 23.4 us
// (3.2 TB/s); 8192 x 1600 binary32 with sum and mask 51 (5.1 TB/s): bounded by
// instructions (a row's address, ends and two sums are each warp's own) and by
// the barrier that the sums cross.
template <int DT, int NV, bool kW, int THREADS>
__global__ void __launch_bounds__(THREADS) k_norm_bwd(const __grid_constant__ NormBwdArgs a)
{
    extern __shared__ float s_cols[];
    __shared__ float2 s_red[2][32];
    const int tpr = a.tpr, group = threadIdx.x / tpr, t = threadIdx.x - group * tpr, groups = blockDim.x / tpr;
    const int cols = (int)a.rows.cols;
    const int64_t step = (int64_t)gridDim.x * groups;
    const uint64_t off = a.dropping ? drop_offset(a.d) : 0;
    const bool vec = a.rows.kind != kLoose;
    pdl_launch_next();
    int64_t r = (int64_t)blockIdx.x * groups + group;
    const int at = lane_group<kW>(t) * 8 - row_shift<kW>(a.rows, r);
    const int wide = kW ? tpr * 8 : (tpr >> 5) * 31 * 8;  // columns from one of a thread's groups to the next
    const bool mine = owns_group<kW>();
    float dw[NV][8], db[NV][8], w[NV][8];
    Group<DT> ndy[NV], nx[NV], nres[NV];
    float nmean = 0.0f, nrstd = 0.0f;
    auto fetch = [&](int64_t row) {
        if (row >= a.rows.rows)
            return;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c0 = at + v * wide;
            if (mine && c0 < cols) {
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
        const int c0 = at + v * wide;
        ndy[v] = nx[v] = nres[v] = Group<DT>{};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            dw[v][e] = db[v][e] = w[v][e] = 0.0f;
        if (mine && c0 < cols)
            load_vector<DT, kW>(a.weight, a.w_f32, c0, cols, a.w_vec, 1.0f, w[v]);
    }
    fetch(r);
    for (int buf = 0; r < a.rows.rows; r += step, buf ^= 1) {
        const float mean = nmean, rstd = nrstd;
        Group<DT> cdy[NV], cx[NV], cres[NV];
        float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float dy[8], x[8];
            cdy[v] = ndy[v], cx[v] = nx[v], cres[v] = nres[v];
            cdy[v].to_float(dy);
            cx[v].to_float(x);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // outside the row dy and w are 0: its terms vanish
                const float xh = (x[e] - mean) * rstd, g = dy[e] * w[v][e];
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
            const int c0 = at + v * wide;
            if (kW && c0 >= cols)
                continue;
            const bool in = kW || (mine && c0 < cols);
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
            if (in)
                store_group<DT, kW>(row_ptr<DT>(a.dx, r), c0, cols, vec, dy);
            // (a warp stays together unless its rows are whole)
            if (a.dropping && (kW || c0 - (int)(threadIdx.x & 31) * 8 < cols)) {
                keep_group<kW>(a.d, row_mask(a.d, off, r), c0, dy);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    dy[e] *= a.d.scale;
                if (in)
                    store_group<DT, kW>(row_ptr<DT>(a.dropped, r), c0, cols, vec, dy);
            }
        }
    }
    if (!a.partials)
        return;
    // the block's row groups, in order, column by column
    const int width = wide * NV;
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
        if (mine) {
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    s_cols[group * width + v * wide + lane_group<kW>(t) * 8 + e] = which ? db[v][e] : dw[v][e];
        }
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

constexpr int kBwdRowsThreads = 512;

// Backward of whole rows of 16-bit elements, for many rows: teams of T warps
// that take a row each, NV groups per lane, whose dweight and dbias build up
// in registers; the row stays in shared memory between the sums over it and
// dx, and a group's copy of the next row is under way as soon as this row's
// has been read for dx.  T is the least that leaves four groups to a lane: with
// one warp for seven groups the sums' registers left 11 warps to an SM (36.4 us
// for 8192 x 1600 with sum and mask; two warps of four groups 36.2, 3.6 TB/s;
// k_norm_bwd 39.6).  16384 x 1600: 61 us where k_norm_bwd takes 71; 8192 x 16384
// 294 (5.4 TB/s) where the two passes take 580.  9 us of each call are its start,
// its partials and their sum; the rest runs at 5.2 TB/s.
template <int DT, int NV, int T>
__global__ void __launch_bounds__(kBwdRowsThreads) k_norm_bwd_rows(const __grid_constant__ NormBwdArgs a)
{
    constexpr int kPieces = NV * 32;  // of a warp's part of a row, in shared memory
    constexpr int kNext = T * 32;  // groups from one of a lane's to the next
    extern __shared__ float4 s_rows[];
    __shared__ float2 s_red[2][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, teams = blockDim.x / (T * 32), team = warp / T;
    const int cols = (int)a.rows.cols, groups = cols >> 3, g0 = warp % T * 32 + lane;
    const int64_t step = (int64_t)gridDim.x * teams;
    const uint64_t off = a.dropping ? drop_offset(a.d) : 0;
    float4 *const vec = s_rows;  // weight: the first and the last four columns of each group apart
    uint4 *const in = reinterpret_cast<uint4 *>(s_rows + 2 * groups) + warp * 3 * kPieces + lane;
    pdl_launch_next();
    int64_t r = (int64_t)blockIdx.x * teams + team;
    // (T = 16: only the last two groups may be outside the row; else the last)
    auto has = [&](int v) { return v < NV - (T == 16 ? 2 : 1) || g0 + v * kNext < groups; };
    auto fetch = [&](int64_t row, int v) {
        const int at = (g0 + v * kNext) * 16;
        const bool there = row < a.rows.rows;
        copy16(in + v * 32, row_ptr<DT>(a.dy, row) + at, there);
        copy16(in + kPieces + v * 32, row_ptr<DT>(a.x, row) + at, there);
        copy16(in + 2 * kPieces + v * 32, row_ptr<DT>(a.dres, row) + at, there && a.dres.p);
    };
    auto take = [&](int which, int v, float2 (&f)[4]) {
        Group<DT> g;
        g.w[0] = in[which * kPieces + v * 32];
        g.to_pairs(f);
    };
#pragma unroll
    for (int v = 0; v < NV; ++v)
        if (has(v))
            fetch(r, v);
    float nmean = 0.0f, nrstd = 0.0f;  // of the next row
    auto statistics = [&](int64_t row) {
        if (row < a.rows.rows)
            nmean = __ldg(a.mean + row), nrstd = __ldg(a.rstd + row);
    };
    statistics(r);
    for (int i = threadIdx.x; i < cols; i += blockDim.x) {
        float *const to = reinterpret_cast<float *>(vec + (i >> 2 & 1) * groups + (i >> 3)) + (i & 3);
        *to = !a.weight ? 1.0f : a.w_f32 ? load1<ZERO_F32>(a.weight, i) : load1<DT>(a.weight, i);
    }
    float2 dw[NV][4], db[NV][4];
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            dw[v][k] = db[v][k] = both(0.0f);
    __syncthreads();
    auto weights = [&](int v, float2 (&w)[4]) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 q = vec[h * groups + g0 + kNext * v];
            w[2 * h] = make_float2(q.x, q.y), w[2 * h + 1] = make_float2(q.z, q.w);
        }
    };
    for (int buf = 0; r < a.rows.rows; r += step, buf ^= 1) {
        const float mean = nmean, rstd = nrstd;
        statistics(r + step);
        float2 sx = both(0.0f), sy = both(0.0f);
        copies_done();
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (has(v)) {
                float2 g[4], xh[4], w[4];
                take(0, v, g);
                take(1, v, xh);
                weights(v, w);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    xh[k] = __fmul2_rn(__fadd2_rn(xh[k], both(-mean)), both(rstd));
                    dw[v][k] = __ffma2_rn(g[k], xh[k], dw[v][k]);
                    db[v][k] = __fadd2_rn(db[v][k], g[k]);
                    g[k] = __fmul2_rn(g[k], w[k]);
                    sx = __fadd2_rn(sx, g[k]);
                    sy = __ffma2_rn(g[k], xh[k], sy);
                }
            }
        const float half = half_sums(make_float2(sx.x + sx.y, sy.x + sy.y));
        float2 s;
        if (T == 1) {
            s = both_sums(half);
        } else {
            float2 *const red = s_red[buf] + team * T;
            if ((lane & 15) == 0)
                (lane ? red[warp % T].y : red[warp % T].x) = half;
            asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(T * 32) : "memory");
            s = red[0];
#pragma unroll
            for (int q = 1; q < T; ++q)
                s = __fadd2_rn(s, red[q]);
        }
        // rstd (g - mean(g) - xh mean(g xh))
        const float2 c1 = both(-s.x * a.inv_cols * rstd), c2 = both(-s.y * a.inv_cols * rstd);
        RowMask mask{};
        if (a.dropping)
            mask = row_mask(a.d, off, r);
        char *const px = row_ptr<DT>(a.dx, r) + g0 * 16, *const pd = row_ptr<DT>(a.dropped, r) + g0 * 16;
        auto second = [&](auto dropping) {
#pragma unroll
            for (int v = 0; v < NV; ++v)
                if (has(v)) {
                    float2 g[4], xh[4], w[4], add[4];
                    take(0, v, g);
                    take(1, v, xh);
                    take(2, v, add);
                    weights(v, w);
                    fetch(r + step, v);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        xh[k] = __fmul2_rn(__fadd2_rn(xh[k], both(-mean)), both(rstd));
                        g[k] = __fmul2_rn(g[k], w[k]);
                        g[k] = __ffma2_rn(xh[k], c2, __ffma2_rn(g[k], both(rstd), __fadd2_rn(add[k], c1)));
                    }
                    store_pairs<DT, true>(px, v * kNext * 8, cols, true, g);
                    if (dropping) {
                        keep_pairs<true, false>(a.d, mask, (g0 + kNext * v) * 8, g);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            g[k] = __fmul2_rn(g[k], both(a.d.scale));
                        store_pairs<DT, true>(pd, v * kNext * 8, cols, true, g);
                    }
                }
        };
        if (a.dropping)
            second(std::true_type{});
        else
            second(std::false_type{});
    }
    // the last turn's copies, of rows that are not there, write zeros where the
    // rows lay at any time until their thread has waited for them
    copies_done();
    if (!a.partials)
        return;
    // the block's teams, in order, column by column (the first and the last
    // four of each group apart again)
    __syncthreads();
    constexpr int width = NV * kNext;  // groups
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        float4 *const to = s_rows + team * 4 * width + g0 + kNext * v;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            to[h * width] = make_float4(dw[v][2 * h].x, dw[v][2 * h].y, dw[v][2 * h + 1].x, dw[v][2 * h + 1].y);
            to[(2 + h) * width] = make_float4(db[v][2 * h].x, db[v][2 * h].y, db[v][2 * h + 1].x, db[v][2 * h + 1].y);
        }
    }
    __syncthreads();
    float4 *const out = reinterpret_cast<float4 *>(a.partials + (int64_t)blockIdx.x * 2 * cols);
    for (int i = threadIdx.x; i < 4 * groups; i += blockDim.x) {
        const int which = i >= 2 * groups, q = i - which * 2 * groups;
        const float4 *from = s_rows + (2 * which + (q & 1)) * width + (q >> 1);
        float4 sum = from[0];
#pragma unroll 4
        for (int k = 1; k < teams; ++k) {
            const float4 x = from[k * 4 * width];
            sum.x += x.x, sum.y += x.y, sum.z += x.z, sum.w += x.w;
        }
        out[i] = sum;
    }
}

// dx of rows too wide for k_norm_bwd: a block per row, two passes.
template <int DT>
__global__ void __launch_bounds__(512) k_norm_bwd_wide(const __grid_constant__ NormBwdArgs a)
{
    __shared__ float2 s_red[2][32];
    const uint64_t off = a.dropping ? drop_offset(a.d) : 0;
    const int64_t cols = a.rows.cols, step = (int64_t)(blockDim.x >> 5) * 31 * 8;
    const bool mine = owns_group<false>();
    const bool vec = a.rows.kind != kLoose;
    int buf = 0;
    for (int64_t r = blockIdx.x; r < a.rows.rows; r += gridDim.x, buf ^= 1) {
        const int64_t first = -(int64_t)row_shift<false>(a.rows, r), at = lane_group<false>(threadIdx.x) * 8;
        const float mean = a.mean[r], rstd = a.rstd[r];
        const RowMask mask = row_mask(a.d, off, r);
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
        for (int64_t pass = first; pass < cols; pass += step) {
            const int64_t c0 = pass + at;
            const bool in = mine && c0 < cols;
            if (!in)
                continue;
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
        for (int64_t pass = first; pass < cols; pass += step) {
            const int64_t c0 = pass + at;
            const bool in = mine && c0 < cols;
            float g[8] = {}, xh[8];
            if (in) {
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
            }
            if (a.dropping) {
                keep_group<false>(a.d, mask, c0, g);  // the whole warp together
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    g[e] *= a.d.scale;
                if (in)
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
// a fixed order, a block per 16 columns, 32 threads of a column taking every
// 32nd.  It is launched ahead and waits; what it adds to a call is 2 to 3 us of
// start and of two trips to L2 (8 columns per block were 0.1 us faster for 1600
// columns and 2 us slower for 8192).
constexpr int kSumThreads = 512, kSumCols = 16;

__global__ void __launch_bounds__(kSumThreads) k_norm_bwd_sum(const float *partials, int n, int64_t cols, void *dweight,
                                                       void *dbias, int32_t gdtype)
{
    constexpr int kSlots = kSumThreads / kSumCols;
    __shared__ float s[kSlots][kSumCols];
    void *out = blockIdx.y ? dbias : dweight;
    if (!out)
        return;
    const int at = threadIdx.x % kSumCols, slot = threadIdx.x / kSumCols;
    const int64_t c = (int64_t)blockIdx.x * kSumCols + at;
    pdl_wait();
    float sum = 0.0f;
    if (c < cols)
#pragma unroll 5
        for (int q = slot; q < n; q += kSlots)
            sum += __ldcg(partials + ((int64_t)q * 2 + blockIdx.y) * cols + c);
    s[slot][at] = sum;
    __syncthreads();
    if (slot == 0 && c < cols) {
#pragma unroll
        for (int q = 1; q < kSlots; ++q)
            sum += s[q][at];
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
    for (uint32_t r = 0; r < 10; ++r) {
        d->key[r][0] = (uint32_t)drop->seed + r * 0x9E3779B9u;
        d->key[r][1] = (uint32_t)(drop->seed >> 32) + r * 0xBB67AE85u;
    }
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

// Whole warps for a row's groups, per_thread of them each (see keep_group).
int row_threads(int64_t groups, int per_thread, bool whole)
{
    const int64_t lanes = (groups + per_thread - 1) / per_thread;
    return (int)((whole ? (lanes + 31) / 32 : (lanes + 30) / 31) * 32);
}

int vector_groups(const Rows &g, const void *a, const void *b) { return g.s_mask == 0 && aligned16(a) && aligned16(b); }

// Threads of a row with four groups each; wider rows go through the
// three-pass kernels.
constexpr int kMostThreads = 512;

// Blocks of the kernels that go from row to row: one per SM, and a multiple
// of 8, so that a thread's rows all have the same shift.
constexpr int kRowBlocks = 152;

// From how many rows on the kernels that stage their rows are taken, for a
// team of so many warps: a start and an end of theirs cost one to two us more
// than the others', a row less (forward of 1600 columns: 4.2 us against 3.9
// for 700 rows, 4.1 against 4.9 for 1500).  Sixteen warps stand against the
// kernels of two passes (backward of 16384 columns: 31 us against 20 for 160
// rows, 42 against 51 for 700).
constexpr int64_t many_rows(int team) { return (team == 16 ? 2 : team > 2 ? 16 : 8) * kRowBlocks; }
constexpr int kMostShared = 232448 - 1024;  // of a block, less what the row kernels have besides

// Teams of `size` warps for a block's share of the rows: as few rows after one
// another as `most` warps allow, and as few teams as do that.
int64_t row_teams(int64_t rows, int most, int size)
{
    const int64_t all = (int64_t)kRowBlocks * (most / size), waves = (rows + all - 1) / all;
    return (rows + waves * kRowBlocks - 1) / (waves * kRowBlocks);
}

template <int DT, int NV, int T, bool kFused>
int norm_fwd_rows(NormArgs &a, cudaStream_t st)
{
    const int64_t warps = row_teams(a.rows.rows, norm_rows_threads(NV) / 32, T) * T;
    const int smem = (int)(a.rows.cols * 8 + warps * (kFused ? 2 : 1) * NV * 512);
    auto kernel = k_norm_fwd_rows<DT, NV, T, kFused>;
    // (the most there is, whatever this call needs: other threads' calls set it too)
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostShared) == cudaSuccess)
        kernel<<<kRowBlocks, (unsigned)warps * 32, smem, st>>>(a);
    return check_launch("k_norm_fwd_rows");
}

template <int DT, bool kFused, bool kW>
int norm_fwd(NormArgs &a, cudaStream_t st)
{
    const int64_t groups = groups_per_row(a.rows), rows = a.rows.rows;
    if (row_threads(groups, 4, kW) > kMostThreads) {
        const int64_t most = (int64_t)sm_count() * 4;
        k_norm_fwd_wide<DT><<<(unsigned)(rows < most ? rows : most), 512, 0, st>>>(a);
        return check_launch("k_norm_fwd_wide");
    }
    // Two groups per thread, one while rows are few (latency); teams fill a
    // block (what the registers of one block per SM allow), few rows are
    // spread over all SMs first.
    const bool few = rows <= 4 * kRowBlocks;
    // Binary32 with the sum spills in the registers of 640 threads: 512 there
    // (8192 x 1600 37.7 us to 34.0, 8192 x 1601 52 to 37), and 384 where four
    // groups leave them.
    constexpr bool kSpills = DT == ZERO_F32 && kFused;
    constexpr int kTwo = kSpills ? 512 : 640, kFour = kSpills ? 384 : 512;
    int nv = 4;
    if constexpr (kW && DT != ZERO_F32) {
        // (p = 1 drops what no word says)
        if (rows >= many_rows(groups <= 512 ? 1 : 4) && groups > 64 && groups <= 1024 && !a.d.all) {
            switch ((groups + 31) / 32) {
            case 3: return norm_fwd_rows<DT, 3, 1, kFused>(a, st);
            case 4: return norm_fwd_rows<DT, 4, 1, kFused>(a, st);
            case 5: return norm_fwd_rows<DT, 5, 1, kFused>(a, st);
            case 6: return norm_fwd_rows<DT, 6, 1, kFused>(a, st);
            case 7: return norm_fwd_rows<DT, 7, 1, kFused>(a, st);
            case 8: return norm_fwd_rows<DT, 8, 1, kFused>(a, st);
            }
            if (groups <= 6 * 64)
                return norm_fwd_rows<DT, 6, 2, kFused>(a, st);
            if (groups <= 8 * 64)
                return norm_fwd_rows<DT, 8, 2, kFused>(a, st);
            if (groups <= 6 * 128)
                return norm_fwd_rows<DT, 6, 4, kFused>(a, st);
            return norm_fwd_rows<DT, 8, 4, kFused>(a, st);
        }
    }
    if (groups <= 32 || (few && row_threads(groups, 1, kW) <= 768))
        nv = 1;
    else if (row_threads(groups, 2, kW) <= kTwo)
        nv = 2;
    const int tpr = row_threads(groups, nv, kW), most = nv == 1 ? 768 : nv == 2 ? kTwo : 512;
    int64_t teams = most / tpr;
    if (tpr > 32 && teams > 15)
        teams = 15;  // named barriers
    if (rows < teams * kRowBlocks)
        teams = rows < kRowBlocks ? 1 : (rows + kRowBlocks - 1) / kRowBlocks;
    a.tpr = tpr;
    const int64_t need = (rows + teams - 1) / teams;
    const unsigned grid = (unsigned)(need < kRowBlocks ? need : kRowBlocks), block = (unsigned)(teams * tpr);
    if (nv == 1)
        k_norm_fwd<DT, 1, kFused, kW, 768><<<grid, block, 0, st>>>(a);
    else if (nv == 2)
        k_norm_fwd<DT, 2, kFused, kW, kTwo><<<grid, block, 0, st>>>(a);
    else if (block <= kFour)
        k_norm_fwd<DT, 4, kFused, kW, kFour><<<grid, block, 0, st>>>(a);
    else
        k_norm_fwd<DT, 4, kFused, kW, 512><<<grid, block, 0, st>>>(a);
    return check_launch("k_norm_fwd");
}

template <int DT>
int norm_fwd_of(NormArgs &a, cudaStream_t st)
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
    int rows_team;  // k_norm_bwd_rows' warps per row, or 0
    int nv, tpr, groups;
    int64_t blocks, partials;
};

// `staged`: rows that k_norm_bwd_rows may take.
BwdPlan bwd_plan(int64_t rows, int64_t groups_row, bool whole, bool staged, bool f32)
{
    BwdPlan p{};
    int team = 1;
    while (team < 16 && groups_row > 128 * team)
        team *= 2;
    if (staged && rows >= many_rows(team) && groups_row > (team == 1 || team == 16 ? 64 : 96) * team &&
        groups_row <= 128 * team) {
        p.rows_team = team;
        p.nv = groups_row <= 96 ? 3 : 4;
        p.blocks = p.partials = kRowBlocks;
        return p;
    }
    p.nv = row_threads(groups_row, 1, whole) <= 768 ? 1 : 2;
    p.tpr = row_threads(groups_row, p.nv, whole);
    p.wide = p.tpr > 512 && p.nv == 2;
    if (p.wide) {
        p.partials = rows < kWarps * 64 ? (rows + kWarps - 1) / kWarps : 64;
        return p;
    }
    p.groups = (p.nv == 2 ? 512 : f32 && p.tpr <= 640 ? 640 : 768) / p.tpr;
    if (p.tpr > 32 && p.groups > 15)
        p.groups = 15;  // named barriers
    const int64_t need = (rows + p.groups - 1) / p.groups;
    if (need < kRowBlocks) {  // few rows: spread them over the SMs
        const int64_t per = (rows + kRowBlocks - 1) / kRowBlocks;
        if (per < p.groups)
            p.groups = (int)(per < 1 ? 1 : per);
    }
    const int64_t n = (rows + p.groups - 1) / p.groups;
    p.blocks = n < kRowBlocks ? n : kRowBlocks;
    p.partials = p.blocks;
    return p;
}

template <int DT, int NV, int T>
int norm_bwd_rows(NormBwdArgs &a, cudaStream_t st)
{
    const int64_t warps = row_teams(a.rows.rows, kBwdRowsThreads / 32, T) * T;
    const int64_t rows = a.rows.cols * 4 + warps * 3 * NV * 512, sums = warps * NV * 2048;
    auto kernel = k_norm_bwd_rows<DT, NV, T>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostShared) == cudaSuccess)
        kernel<<<kRowBlocks, (unsigned)warps * 32, rows > sums ? rows : sums, st>>>(a);
    return check_launch("k_norm_bwd_rows");
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
    if (p.rows_team) {
        if constexpr (DT != ZERO_F32) {
            if (p.rows_team == 1)
                return p.nv == 3 ? norm_bwd_rows<DT, 3, 1>(a, st) : norm_bwd_rows<DT, 4, 1>(a, st);
            if (p.rows_team <= 4)
                return p.rows_team == 2 ? norm_bwd_rows<DT, 4, 2>(a, st) : norm_bwd_rows<DT, 4, 4>(a, st);
            return p.rows_team == 8 ? norm_bwd_rows<DT, 4, 8>(a, st) : norm_bwd_rows<DT, 4, 16>(a, st);
        }
    }
    // (binary32 spills in the registers of 768 threads: 3001 x 2049 27.9 us to 23.1, 8192 x 1601 45 to 40)
    constexpr int kMost = DT == ZERO_F32 ? 640 : 768;
    if (p.nv == 2)
        (whole ? k_norm_bwd<DT, 2, true, 512> : k_norm_bwd<DT, 2, false, 512>)<<<grid, block, smem, st>>>(a);
    else if (block <= kMost)
        (whole ? k_norm_bwd<DT, 1, true, kMost> : k_norm_bwd<DT, 1, false, kMost>)<<<grid, block, smem, st>>>(a);
    else
        (whole ? k_norm_bwd<DT, 1, true, 768> : k_norm_bwd<DT, 1, false, 768>)<<<grid, block, smem, st>>>(a);
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
    const bool whole = a.rows.kind == kWhole;
    // (one more group in rows that are not whole: each then has a neighbour)
    a.groups = (uint32_t)groups_per_row(a.rows) + (whole ? 0 : 1);
    a.d = d;
    a.per_row = fast_divisor(a.groups);
    const int64_t per_block = whole ? kThreads : kWarps * 31;
    const int64_t blocks = (rows * (int64_t)a.groups + per_block - 1) / per_block, most = (int64_t)sm_count() * 32;
    const unsigned grid = (unsigned)(blocks < most ? blocks : most);
    a.step_rows = (uint32_t)(grid * per_block / a.groups), a.step_groups = (uint32_t)(grid * per_block % a.groups);
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
    a.mean = mean, a.rstd = rstd, a.eps = (float)eps, a.cols = (float)cols, a.inv_cols = 1.0f / (float)cols, a.dropping = drop != nullptr;
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
    // No plan leaves more partials than blocks, or blocks than rows.  (Not the
    // plan's own count: that falls as a row more gives a block another team,
    // and a workspace for many rows is to serve fewer as well.)
    const int64_t most = rows < kRowBlocks ? rows : kRowBlocks;
    return 256 + align256((size_t)most * 2 * (size_t)cols * 4);
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
    const bool whole = a.rows.kind == kWhole;
    const BwdPlan plan = bwd_plan(rows, groups_per_row(a.rows), whole, whole && dtype != ZERO_F32 && !a.d.all, dtype == ZERO_F32);
    if (dtype == ZERO_F16)
        ZERO_TRY(norm_bwd<ZERO_F16>(a, plan, st));
    else if (dtype == ZERO_BF16)
        ZERO_TRY(norm_bwd<ZERO_BF16>(a, plan, st));
    else
        ZERO_TRY(norm_bwd<ZERO_F32>(a, plan, st));
    if (!a.partials)
        return ZERO_OK;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((cols + kSumCols - 1) / kSumCols), 2);
    cfg.blockDim = dim3(kSumThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, k_norm_bwd_sum, (const float *)a.partials, (int)plan.partials, cols, dweight, dbias, gdtype);
    return check_launch("k_norm_bwd_sum");
}
