// Norms of queries and keys for each head with the position rotation in the
// same pass, forward and backward.
#include <cmath>

#include "sublayer.cuh"

namespace zpml {
namespace {

constexpr int kMostDim = 256;               // of a head
constexpr int kMostPairs = kMostDim / 2;    // of the rotation
constexpr int64_t kMostHeads = (int64_t)1 << 20;

// A set of rows: the 32 / lanes heads, of the queries or of the keys of one
// token, that a warp works on at once.  The sets of all tokens stand in a row
// and are dealt out to the warps in stretches of one length.
struct QkArgs {
    Heads x[2], y[2], dx[2];  // q, k: the inputs; the outputs (or their gradients); the inputs' gradients
    const void *w[2];
    const uint64_t *turns;
    const int64_t *positions;
    int64_t tokens, sets;
    int32_t heads[2], q_sets, token_sets;  // sets of a token: of its queries, and all
    int32_t dim, rot, interleaved, w_f32;
    float eps, inv_dim;
    float *partial;  // of the weights' gradients: [block][2][dim]
};

// ------------------------------------------------------------- elements of a row

// A lane's share of a row is V elements in V / 2 pairs, of which the first are
// lo and the second hi.  Split (the rotation's pairs lie half of it apart):
// V / 2 elements and as many half of the rotated, or of the other, elements
// further on; else V in a row, neighbours in pairs.  So a rotation stays in
// its lane.  C and D are where the two runs of elements start.
enum Share { kSplit, kRun, kOne };  // kOne: V = 2 single elements, at any place

template <int DT>
__device__ __forceinline__ F2 unpack(uint32_t w)
{
    if constexpr (DT == ZERO_F16) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
        return {f.x, f.y};
    } else {
        return {__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)};
    }
}

template <int DT>
__device__ __forceinline__ uint32_t pack(F2 a)
{
    if constexpr (DT == ZERO_F16) {
        const __half2 h = __floats2half2_rn(a.x, a.y);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a.x, a.y);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

template <int DT, int V, int SH>
struct Raw {
    static constexpr int kBytes = V * (DT == ZERO_F32 ? 4 : 2), kWords = kBytes / 4 > 1 ? kBytes / 4 : 2;
    uint32_t w[kWords];

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int k = 0; k < kWords; ++k)
            w[k] = 0;
    }

    // (kOne: the second element may not be there)
    __device__ __forceinline__ void load(const char *row, int c, int d, bool second)
    {
        constexpr int es = DT == ZERO_F32 ? 4 : 2;
        if constexpr (SH == kOne) {
            w[0] = es == 4 ? *reinterpret_cast<const uint32_t *>(row + c * es) : *reinterpret_cast<const uint16_t *>(row + c * es);
            w[1] = 0;
            if (second)
                w[1] = es == 4 ? *reinterpret_cast<const uint32_t *>(row + d * es) : *reinterpret_cast<const uint16_t *>(row + d * es);
        } else if constexpr (SH == kSplit) {
            const uint2 x = *reinterpret_cast<const uint2 *>(row + c * es), y = *reinterpret_cast<const uint2 *>(row + d * es);
            w[0] = x.x, w[1] = x.y, w[2] = y.x, w[3] = y.y;
        } else {
            const uint4 x = *reinterpret_cast<const uint4 *>(row + c * es);
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
        }
    }

    __device__ __forceinline__ void store(char *row, int c, int d, bool second) const
    {
        constexpr int es = DT == ZERO_F32 ? 4 : 2;
        if constexpr (SH == kOne) {
            if (es == 4) {
                *reinterpret_cast<uint32_t *>(row + c * es) = w[0];
                if (second)
                    *reinterpret_cast<uint32_t *>(row + d * es) = w[1];
            } else {
                *reinterpret_cast<uint16_t *>(row + c * es) = (uint16_t)w[0];
                if (second)
                    *reinterpret_cast<uint16_t *>(row + d * es) = (uint16_t)w[1];
            }
        } else if constexpr (SH == kSplit) {
            *reinterpret_cast<uint2 *>(row + c * es) = make_uint2(w[0], w[1]);
            *reinterpret_cast<uint2 *>(row + d * es) = make_uint2(w[2], w[3]);
        } else {
            *reinterpret_cast<uint4 *>(row + c * es) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
};

// The pairs, two at a time (V = 2: one, and a zero beside it).
template <int V>
struct Pairs {
    static constexpr int N = V >= 4 ? V / 4 : 1;
    F2 lo[N], hi[N];
};

template <int DT, int V, int SH>
__device__ __forceinline__ void get(const Raw<DT, V, SH> &r, Pairs<V> &p)
{
    if constexpr (SH == kOne) {
        p.lo[0] = {DT == ZERO_F32 ? __uint_as_float(r.w[0]) : unpack<DT>(r.w[0]).x, 0.0f};
        p.hi[0] = {DT == ZERO_F32 ? __uint_as_float(r.w[1]) : unpack<DT>(r.w[1]).x, 0.0f};
    } else if constexpr (DT == ZERO_F32) {
        const float a = __uint_as_float(r.w[0]), b = __uint_as_float(r.w[1]), c = __uint_as_float(r.w[2]), d = __uint_as_float(r.w[3]);
        if (SH == kSplit)
            p.lo[0] = {a, b}, p.hi[0] = {c, d};
        else
            p.lo[0] = {a, c}, p.hi[0] = {b, d};
    } else {
        const F2 a = unpack<DT>(r.w[0]), b = unpack<DT>(r.w[1]), c = unpack<DT>(r.w[2]), d = unpack<DT>(r.w[3]);
        if (SH == kSplit)
            p.lo[0] = a, p.lo[1] = b, p.hi[0] = c, p.hi[1] = d;
        else
            p.lo[0] = {a.x, b.x}, p.hi[0] = {a.y, b.y}, p.lo[1] = {c.x, d.x}, p.hi[1] = {c.y, d.y};
    }
}

template <int DT, int V, int SH>
__device__ __forceinline__ void put(Raw<DT, V, SH> &r, const Pairs<V> &p)
{
    if constexpr (SH == kOne) {
        r.w[0] = DT == ZERO_F32 ? __float_as_uint(p.lo[0].x) : pack<DT>(p.lo[0]);
        r.w[1] = DT == ZERO_F32 ? __float_as_uint(p.hi[0].x) : pack<DT>(p.hi[0]);
    } else if constexpr (DT == ZERO_F32) {
        const F2 a = p.lo[0], b = p.hi[0];
        r.w[0] = __float_as_uint(a.x), r.w[3] = __float_as_uint(b.y);
        r.w[1] = __float_as_uint(SH == kSplit ? a.y : b.x), r.w[2] = __float_as_uint(SH == kSplit ? b.x : a.y);
    } else if (SH == kSplit) {
        r.w[0] = pack<DT>(p.lo[0]), r.w[1] = pack<DT>(p.lo[1]), r.w[2] = pack<DT>(p.hi[0]), r.w[3] = pack<DT>(p.hi[1]);
    } else {
        r.w[0] = pack<DT>(F2{p.lo[0].x, p.hi[0].x}), r.w[1] = pack<DT>(F2{p.lo[0].y, p.hi[0].y});
        r.w[2] = pack<DT>(F2{p.lo[1].x, p.hi[1].x}), r.w[3] = pack<DT>(F2{p.lo[1].y, p.hi[1].y});
    }
}

// Where a lane's share i starts, and the rotation's pair that its first pair
// is (-1: not rotated).
struct Place {
    int c, d, turn;
    bool in, second;
};

template <int V, int SH>
__device__ __forceinline__ Place place(const QkArgs &a, int i)
{
    Place p;
    const int half = a.rot / 2;
    if (SH == kRun) {
        p.c = p.d = i * V;
        p.turn = p.c < a.rot ? i * (V / 2) : -1;
        p.in = p.c < a.dim;
        p.second = true;
        return p;
    }
    const int e = i * (V / 2);  // of the first runs
    if (e < half) {
        p.turn = e;
        p.c = SH == kOne && a.interleaved ? 2 * e : e;
        p.d = SH == kOne && a.interleaved ? 2 * e + 1 : e + half;
        p.in = p.second = true;
        return p;
    }
    const int rest = (a.dim - a.rot + 1) / 2, j = e - half;
    p.turn = -1;
    p.c = a.rot + j;
    p.d = p.c + rest;
    p.in = j < rest;
    p.second = p.d < a.dim;
    return p;
}

// ------------------------------------------------------------- the rotation

// The angle of a position and a frequency: phase = position * turns modulo
// 2^64 is the angle's fraction of a turn, exactly.  Its nearest quarter turn
// is taken off in integers too, so that what becomes binary32 is an angle of
// at most pi / 4, off by 2^-24 of itself; a binary32 angle of position 10^6
// would be off by 0.03.
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
    float w[2][kMostDim];                                    // both weights in binary32 (1 without one)
    float cos[kWarps][kMostPairs], sin[kWarps][kMostPairs];  // of each warp's token
};

__device__ __forceinline__ void load_weights(const QkArgs &a, QkShared &sh, int dt)
{
    for (int i = threadIdx.x; i < 2 * a.dim; i += kThreads) {
        const int kind = i >= a.dim, e = i - kind * a.dim;
        const void *w = a.w[kind];
        float v = 1.0f;
        if (w)
            v = a.w_f32 || dt == ZERO_F32 ? load1<ZERO_F32>(w, e) : dt == ZERO_F16 ? load1<ZERO_F16>(w, e) : load1<ZERO_BF16>(w, e);
        sh.w[kind][e] = v;
    }
    __syncthreads();
}

// A token's angles: one pair per lane, shared through shared memory.
__device__ __forceinline__ void token_angles(const QkArgs &a, QkShared &sh, int warp, int lane, uint64_t position)
{
    __syncwarp();  // the token before is done with the tables
    for (int i = lane; i < a.rot / 2; i += 32) {
        const float2 cs = cos_sin(position * a.turns[i]);
        sh.cos[warp][i] = cs.x;
        sh.sin[warp][i] = cs.y;
    }
    __syncwarp();
}

// cos and sin of a share's pairs.
template <int V, int SH>
__device__ __forceinline__ void load_turn(const QkArgs &a, const QkShared &sh, int warp, const Place &p, F2 (&c)[Pairs<V>::N], F2 (&s)[Pairs<V>::N])
{
#pragma unroll
    for (int k = 0; k < Pairs<V>::N; ++k) {
        c[k] = {1.0f, 1.0f};
        s[k] = {0.0f, 0.0f};
        // (a run of neighbours may end its rotation at any pair)
        if (p.in && p.turn >= 0 && p.turn + 2 * k < a.rot / 2)
            c[k].x = sh.cos[warp][p.turn + 2 * k], s[k].x = sh.sin[warp][p.turn + 2 * k];
        if (V > 2 && p.in && p.turn >= 0 && p.turn + 2 * k + 1 < a.rot / 2)
            c[k].y = sh.cos[warp][p.turn + 2 * k + 1], s[k].y = sh.sin[warp][p.turn + 2 * k + 1];
    }
}

// A weight's elements of a share.
template <int V, int SH>
__device__ __forceinline__ void load_weight(const float *w, const Place &p, Pairs<V> &out)
{
#pragma unroll
    for (int k = 0; k < Pairs<V>::N; ++k) {
        out.lo[k] = out.hi[k] = {0.0f, 0.0f};
        if (!p.in)
            continue;
        if (SH == kRun) {
            out.lo[k] = {w[p.c + 4 * k], w[p.c + 4 * k + 2]};
            out.hi[k] = {w[p.c + 4 * k + 1], w[p.c + 4 * k + 3]};
        } else if (SH == kSplit) {
            out.lo[k] = {w[p.c + 2 * k], w[p.c + 2 * k + 1]};
            out.hi[k] = {w[p.d + 2 * k], w[p.d + 2 * k + 1]};
        } else {
            out.lo[k].x = w[p.c];
            out.hi[k].x = p.second ? w[p.d] : 0.0f;
        }
    }
}

template <int L>
__device__ __forceinline__ float row_sum(float v)
{
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Two sums at a time.
template <int L>
__device__ __forceinline__ F2 row_sum(F2 v)
{
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1)
        v = v + F2{__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)};
    return v;
}

// ------------------------------------------------------------- kernels

// Where a warp is among its sets, with a pointer to this lane's row in each of
// ARRAYS arrays of heads (0: x, 1: y, 2: dx of the kernel's arguments).
template <int ES, int L, int... ARRAYS>
struct Cursor {
    static constexpr int kRows = 32 / L, kArrays = sizeof...(ARRAYS);
    int64_t token;
    int32_t left;  // sets, this one among them
    int32_t of;    // set of the token
    int32_t head;  // of this lane
    char *row[kArrays];
    int64_t step[kArrays];

    __device__ __forceinline__ int kind(const QkArgs &a) const { return of >= a.q_sets; }
    __device__ __forceinline__ bool there(const QkArgs &a) const { return head < (of < a.q_sets ? a.heads[0] : a.heads[1]); }

    // to the first set of a token's queries or keys, or any other
    __device__ __forceinline__ void place(const QkArgs &a, int sub)
    {
        const bool keys = of >= a.q_sets;
        head = (of - (keys ? a.q_sets : 0)) * kRows + sub;
        int i = 0;
        auto set = [&](const Heads &h) {
            row[i] = static_cast<char *>(const_cast<void *>(h.p)) + (token * h.ld + head * h.hd) * ES;
            step[i] = h.hd * (kRows * ES);
            ++i;
        };
        auto pick = [&](const Heads &q, const Heads &k) { set(Heads{keys ? k.p : q.p, keys ? k.ld : q.ld, keys ? k.hd : q.hd}); };
        ((ARRAYS == 0 ? pick(a.x[0], a.x[1]) : ARRAYS == 1 ? pick(a.y[0], a.y[1]) : pick(a.dx[0], a.dx[1])), ...);
    }
    __device__ __forceinline__ void start(const QkArgs &a, int64_t first, int64_t end, int sub)
    {
        left = end > first ? (int32_t)(end - first) : 0;
        token = first / a.token_sets;
        of = (int32_t)(first - token * a.token_sets);
        place(a, sub);
    }
    __device__ __forceinline__ void next(const QkArgs &a, int sub)
    {
        --left;
        ++of;
        if (of == a.q_sets || of == a.token_sets) {
            if (of == a.token_sets)
                of = 0, ++token;
            place(a, sub);
            return;
        }
        head += kRows;
#pragma unroll
        for (int i = 0; i < kArrays; ++i)
            row[i] += step[i];
    }
};

// Rows on their way from memory: every lane copies its own shares of the next
// DEPTH sets into its own slots of shared memory, asynchronously, and waits
// for its own copies alone.  (Held in registers, two sets ahead at most, they
// left a warp waiting for memory most of the time: 8192 tokens of 25 + 25
// heads of 64, backward 58 us.)  Single elements are loaded when they are used.
template <int DT, int V, int SH, int N, int DEPTH, int ARRAYS>
struct Stream {
    static constexpr int kSlots = SH == kOne ? 1 : kWarps * DEPTH * ARRAYS * N * 32;
    static constexpr int kSet = ARRAYS * N * 32;  // 16-byte slots of a set
    uint4 *first, *in, *out;                      // this lane's: the first, the next to fill, the next to take

    __device__ __forceinline__ void start(uint4 *slots, int warp, int lane)
    {
        first = in = out = slots + (SH == kOne ? 0 : warp * DEPTH * kSet + lane);
    }
    __device__ __forceinline__ void after(uint4 *&at) const { at = at + kSet == first + DEPTH * kSet ? first : at + kSet; }

    __device__ __forceinline__ void fetch(int array, const char *row, const Place (&pl)[N], bool there) const
    {
        constexpr int es = DT == ZERO_F32 ? 4 : 2;
        if constexpr (SH != kOne) {
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const uint32_t to = smem_addr(in + (array * N + k) * 32);
                if (there && pl[k].in) {
                    if constexpr (SH == kRun) {
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(row + pl[k].c * es) : "memory");
                    } else {
                        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(row + pl[k].c * es) : "memory");
                        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to + 8), "l"(row + pl[k].d * es)
                                     : "memory");
                    }
                }
            }
        }
    }

    __device__ __forceinline__ static void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    template <int LEFT>
    __device__ __forceinline__ static void arrived()
    {
        asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
    }

    // Zeros where there is no row.
    __device__ __forceinline__ void take(int array, const char *row, const Place (&pl)[N], bool there, Raw<DT, V, SH> (&raw)[N]) const
    {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            raw[k].clear();
            if (there && pl[k].in) {
                if constexpr (SH == kOne) {
                    raw[k].load(row, pl[k].c, pl[k].d, pl[k].second);
                } else {
                    const uint4 v = out[(array * N + k) * 32];
                    raw[k].w[0] = v.x, raw[k].w[1] = v.y, raw[k].w[2] = v.z, raw[k].w[3] = v.w;
                }
            }
        }
    }
};

// With what the heads of a token share,
//     lo' = (lo (w_lo cos) - hi (w_hi sin)) r,  hi' = (hi (w_hi cos) + lo (w_lo sin)) r,
// r = 1 / sqrt(mean(x^2) + eps).
// Every byte is read once and written once; a token's angles cost its warp as
// much as a few rows, so a warp takes rows of one token after another.  Rows of
// 128 are bound by bytes: 16384 tokens of 64 + 8 heads bf16 (604 MB) 102 us,
// 5.9 TB/s, 0.87 of the copy; rows of 64 by issue (72 % of the slots): 8192
// tokens of 25 + 25 heads f16 (105 MB) 23.2 us from and to L2, 29.8 from HBM.
// One token: 3 us.
template <int DT, int V, int SH, int N, int L, int DEPTH>
__global__ void __launch_bounds__(kThreads, SH == kOne ? 1 : 4) k_qk_norm(const __grid_constant__ QkArgs a)
{
    constexpr int M = Pairs<V>::N, es = DT == ZERO_F32 ? 4 : 2;
    using Rows = Stream<DT, V, SH, N, DEPTH, 1>;
    __shared__ __align__(16) QkShared sh;
    __shared__ uint4 s_rows[Rows::kSlots];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = lane / L, at = lane & (L - 1);
    const int64_t me = (int64_t)blockIdx.x * kWarps + warp, warps = (int64_t)gridDim.x * kWarps;
    const int64_t begin = a.sets * me / warps, end = a.sets * (me + 1) / warps;
    Place pl[N];
#pragma unroll
    for (int n = 0; n < N; ++n)
        pl[n] = place<V, SH>(a, at + n * L);
    Rows in;
    in.start(s_rows, warp, lane);
    Cursor<es, L, 0> ahead;
    Cursor<es, L, 0, 1> now;
    ahead.start(a, begin, end, sub);
    now.start(a, begin, end, sub);
    auto fetch = [&] {
        if (SH != kOne) {
            if (ahead.left > 0) {
                in.fetch(0, ahead.row[0], pl, ahead.there(a));
                in.after(in.in);
                ahead.next(a, sub);
            }
            Rows::commit();
        }
    };
#pragma unroll
    for (int k = 0; k < DEPTH - 1; ++k)
        fetch();
    load_weights(a, sh, DT);
    Pairs<V> A[N], B[N];
    int64_t token = -1;
    int kind = -1;
    for (; now.left > 0; now.next(a, sub)) {
        const int new_kind = now.kind(a);
        if (now.token != token || new_kind != kind) {
            if (a.rot && now.token != token)
                token_angles(a, sh, warp, lane, (uint64_t)(a.positions ? a.positions[now.token] : now.token));
            token = now.token, kind = new_kind;
#pragma unroll
            for (int n = 0; n < N; ++n) {
                Pairs<V> w;
                F2 c[M], s[M];
                load_weight<V, SH>(sh.w[kind], pl[n], w);
                load_turn<V, SH>(a, sh, warp, pl[n], c, s);
#pragma unroll
                for (int k = 0; k < M; ++k) {
                    A[n].lo[k] = w.lo[k] * c[k], A[n].hi[k] = w.hi[k] * c[k];
                    B[n].lo[k] = w.hi[k] * s[k] * twice(-1.0f), B[n].hi[k] = w.lo[k] * s[k];
                }
            }
        }
        const bool there = now.there(a);
        Raw<DT, V, SH> raw[N];
        Rows::template arrived<DEPTH - 2>();
        in.take(0, now.row[0], pl, there, raw);
        in.after(in.out);
        fetch();
        __syncwarp();  // (a row may be written where it was read)
        Pairs<V> f[N];
        F2 sq = {0.0f, 0.0f};
#pragma unroll
        for (int n = 0; n < N; ++n) {
            get<DT, V, SH>(raw[n], f[n]);
#pragma unroll
            for (int e = 0; e < M; ++e)
                sq = fma2(f[n].hi[e], f[n].hi[e], fma2(f[n].lo[e], f[n].lo[e], sq));
        }
        const F2 r = twice(rsqrtf(row_sum<L>(sq.x + sq.y) * a.inv_dim + a.eps));
#pragma unroll
        for (int n = 0; n < N; ++n) {
            Pairs<V> o;
#pragma unroll
            for (int e = 0; e < M; ++e) {
                o.lo[e] = fma2(f[n].lo[e], A[n].lo[e], f[n].hi[e] * B[n].lo[e]) * r;
                o.hi[e] = fma2(f[n].hi[e], A[n].hi[e], f[n].lo[e] * B[n].hi[e]) * r;
            }
            put<DT, V, SH>(raw[n], o);
            if (there && pl[n].in)
                raw[n].store(now.row[1], pl[n].c, pl[n].d, pl[n].second);
        }
    }
}

// The backward pass in the same shape: a lane holds its columns of both
// weights' gradients from its first row to its last, and a block leaves one
// partial sum per column:
//     dz = dy turned back, g = dz w, dx = r (g - x r mean(g x r)), dw += dz x r.
// Bound by its bytes and, at 64 elements to a row, by the shuffles and
// arithmetic of a row: 8192 tokens of 25 + 25 heads of 64 f16 (157 MB): 36.3
// us with the weights' second launch, 4.3 TB/s.
template <int DT, int V, int SH, int N, int L, int DEPTH>
__global__ void __launch_bounds__(kThreads, SH == kOne ? 1 : 2) k_qk_norm_bwd(const __grid_constant__ QkArgs a)
{
    constexpr int M = Pairs<V>::N, es = DT == ZERO_F32 ? 4 : 2;
    using Rows = Stream<DT, V, SH, N, DEPTH, 2>;
    constexpr int kSums = kWarps * 2 * kMostDim / 4;  // the slots become the warps' sums
    __shared__ __align__(16) QkShared sh;
    __shared__ uint4 s_rows[Rows::kSlots > kSums ? Rows::kSlots : kSums];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = lane / L, at = lane & (L - 1);
    const int64_t me = (int64_t)blockIdx.x * kWarps + warp, warps = (int64_t)gridDim.x * kWarps;
    const int64_t begin = a.sets * me / warps, end = a.sets * (me + 1) / warps;
    pdl_launch_next();
    Place pl[N];
    Pairs<V> dw[2][N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        pl[n] = place<V, SH>(a, at + n * L);
#pragma unroll
        for (int e = 0; e < M; ++e)
            dw[0][n].lo[e] = dw[0][n].hi[e] = dw[1][n].lo[e] = dw[1][n].hi[e] = {0.0f, 0.0f};
    }
    Rows in;
    in.start(s_rows, warp, lane);
    Cursor<es, L, 0, 1> ahead;
    ahead.start(a, begin, end, sub);
    auto fetch = [&] {
        if (ahead.left > 0) {
            const bool there = ahead.there(a);
            in.fetch(0, ahead.row[0], pl, there);
            in.fetch(1, ahead.row[1], pl, there);
            in.after(in.in);
            ahead.next(a, sub);
        }
        Rows::commit();
    };
    if (SH != kOne)
#pragma unroll
        for (int k = 0; k < DEPTH - 1; ++k)
            fetch();
    Cursor<es, L, 2> now;
    now.start(a, begin, end, sub);
    load_weights(a, sh, DT);
    Pairs<V> w[N];
    F2 c[N][M], s[N][M], back[N][M];  // back: -sin
    int64_t token = -1;
    int kind = -1;
    for (; now.left > 0; now.next(a, sub)) {
        const int new_kind = now.kind(a);
        if (now.token != token) {
            if (a.rot)
                token_angles(a, sh, warp, lane, (uint64_t)(a.positions ? a.positions[now.token] : now.token));
#pragma unroll
            for (int n = 0; n < N; ++n) {
                load_turn<V, SH>(a, sh, warp, pl[n], c[n], s[n]);
#pragma unroll
                for (int e = 0; e < M; ++e)
                    back[n][e] = s[n][e] * twice(-1.0f);
            }
        }
        if (new_kind != kind)
#pragma unroll
            for (int n = 0; n < N; ++n)
                load_weight<V, SH>(sh.w[new_kind], pl[n], w[n]);
        token = now.token, kind = new_kind;
        const bool there = now.there(a);
        Raw<DT, V, SH> rx[N], ry[N];
        if (SH != kOne)
            Rows::template arrived<DEPTH - 2>();
        in.take(0, ahead.row[0], pl, there, rx);
        in.take(1, ahead.row[1], pl, there, ry);
        if (SH != kOne) {
            in.after(in.out);
            fetch();
        } else {
            ahead.next(a, sub);
        }
        __syncwarp();  // (a row may be written where it was read)
        Pairs<V> f[N], dz[N], g[N];
        F2 sq = {0.0f, 0.0f}, dot = {0.0f, 0.0f};
#pragma unroll
        for (int n = 0; n < N; ++n) {
            Pairs<V> dy;
            get<DT, V, SH>(rx[n], f[n]);
            get<DT, V, SH>(ry[n], dy);
#pragma unroll
            for (int e = 0; e < M; ++e) {
                dz[n].lo[e] = fma2(dy.lo[e], c[n][e], dy.hi[e] * s[n][e]);
                dz[n].hi[e] = fma2(dy.hi[e], c[n][e], dy.lo[e] * back[n][e]);
                g[n].lo[e] = dz[n].lo[e] * w[n].lo[e];
                g[n].hi[e] = dz[n].hi[e] * w[n].hi[e];
                sq = fma2(f[n].hi[e], f[n].hi[e], fma2(f[n].lo[e], f[n].lo[e], sq));
                dot = fma2(g[n].hi[e], f[n].hi[e], fma2(g[n].lo[e], f[n].lo[e], dot));
            }
        }
        const F2 sums = row_sum<L>(F2{sq.x + sq.y, dot.x + dot.y});
        const float r = rsqrtf(sums.x * a.inv_dim + a.eps);
        const float m = sums.y * a.inv_dim * r * r;
        const F2 r2 = twice(r), m2 = twice(-m * r);
        auto add = [&](Pairs<V> (&sum)[N]) {
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int e = 0; e < M; ++e) {
                    sum[n].lo[e] = fma2(dz[n].lo[e], f[n].lo[e] * r2, sum[n].lo[e]);
                    sum[n].hi[e] = fma2(dz[n].hi[e], f[n].hi[e] * r2, sum[n].hi[e]);
                }
        };
        if (there) {  // (a row that is not there may have r = 1 / 0)
            if (kind == 0)
                add(dw[0]);
            else
                add(dw[1]);
        }
#pragma unroll
        for (int n = 0; n < N; ++n) {
            Pairs<V> o;
#pragma unroll
            for (int e = 0; e < M; ++e) {
                o.lo[e] = fma2(g[n].lo[e], r2, f[n].lo[e] * m2);
                o.hi[e] = fma2(g[n].hi[e], r2, f[n].hi[e] * m2);
            }
            put<DT, V, SH>(rx[n], o);
            if (there && pl[n].in)
                rx[n].store(now.row[0], pl[n].c, pl[n].d, pl[n].second);
        }
    }
    if (!a.partial)
        return;
    __syncthreads();  // every warp is done with its slots
    float *const s_dw = reinterpret_cast<float *>(s_rows);
    auto leave = [&](int kind, int col, float v, bool in) {
#pragma unroll
        for (int o = 16; o >= L; o >>= 1)
            v += __shfl_xor_sync(0xffffffffu, v, o);
        if (sub == 0 && in)
            s_dw[(warp * 2 + kind) * kMostDim + col] = v;
    };
#pragma unroll
    for (int kind = 0; kind < 2; ++kind)
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int e = 0; e < M; ++e) {
                const Place &p = pl[n];
                const Pairs<V> &d = dw[kind][n];
                if (SH == kRun) {
                    leave(kind, p.c + 4 * e, d.lo[e].x, p.in);
                    leave(kind, p.c + 4 * e + 1, d.hi[e].x, p.in);
                    leave(kind, p.c + 4 * e + 2, d.lo[e].y, p.in);
                    leave(kind, p.c + 4 * e + 3, d.hi[e].y, p.in);
                } else {
                    leave(kind, p.c + 2 * e, d.lo[e].x, p.in);
                    leave(kind, p.d + 2 * e, d.hi[e].x, p.in && p.second);
                    if (V > 2) {
                        leave(kind, p.c + 2 * e + 1, d.lo[e].y, p.in);
                        leave(kind, p.d + 2 * e + 1, d.hi[e].y, p.in);
                    }
                }
            }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.dim; i += kThreads) {
        const int kind = i >= a.dim, e = i - kind * a.dim;
        float v = s_dw[kind * kMostDim + e];
#pragma unroll
        for (int k = 1; k < kWarps; ++k)
            v += s_dw[(k * 2 + kind) * kMostDim + e];
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

int check_qk(Heads *h[2], int n, int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t dim, int32_t dtype, Reach *reach)
{
    for (int i = 0; i < n; ++i) {
        ZERO_TRY(check_heads(&h[0][i], tokens, q_heads, dim, dtype, reach));
        ZERO_TRY(check_heads(&h[1][i], tokens, k_heads, dim, dtype, reach));
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
int check_words(const void *p, Reach *reach)
{
    if (!p)
        return ZERO_EINVAL;
    if ((reinterpret_cast<uintptr_t>(p) & 7u) != 0)
        return ZERO_EALIGN;
    return reach->has(p) ? ZERO_OK : ZERO_EINVAL;
}

int check_rotary(const zero_rotary_t *rotary, const int64_t *positions, int64_t tokens, Reach *reach)
{
    if (tokens == 0 || !rotary || rotary->rot_dim == 0)
        return ZERO_OK;
    ZERO_TRY(check_words(rotary->turns, reach));
    return positions ? check_words(positions, reach) : ZERO_OK;
}

// Whether every row's V elements (in runs of `run`) start on whole loads.
bool rows_fit(const QkArgs &a, bool backward, int es, int V, int run)
{
    if (a.dim % V != 0)
        return false;
    const Heads *all[3] = {a.x, a.y, a.dx};
    for (int i = 0; i < (backward ? 3 : 2); ++i)
        for (int k = 0; k < 2; ++k) {
            if (a.heads[k] == 0)
                continue;
            const Heads &h = all[i][k];
            if ((reinterpret_cast<uintptr_t>(h.p) | (uintptr_t)(h.ld * es) | (uintptr_t)(h.hd * es)) & (uintptr_t)(run * es - 1))
                return false;
        }
    return true;
}

struct QkPlan {
    int share, n, lanes;  // lanes to a row, n shares to each
};

// 16 bytes to a lane where rows and the rotation's halves are whole numbers of
// them (in two runs of 8 where the pairs lie half of the rotation apart), else
// single elements.  8192 tokens of 25 + 25 heads of 64, both ways: bf16 23 and
// 165 us, binary32 37 and 149.
QkPlan plan_qk(QkArgs &a, bool backward, int es)
{
    QkPlan p{kOne, 1, 8};
    int V = 16 / es;
    if (a.rot == 0 || a.interleaved) {
        if (rows_fit(a, backward, es, V, V))
            p.share = kRun;
    } else if (a.rot % V == 0 && rows_fit(a, backward, es, V, V / 2)) {
        p.share = kSplit;
    }
    V = p.share == kOne ? 2 : V;
    const int pairs = a.rot / 2 + (a.dim - a.rot + 1) / 2, shares = (pairs + V / 2 - 1) / (V / 2);
    while (p.lanes < 32 && (p.lanes < shares || p.share == kOne))
        p.lanes *= 2;
    p.n = (shares + p.lanes - 1) / p.lanes;
    const int rows = 32 / p.lanes;
    a.q_sets = (a.heads[0] + rows - 1) / rows;
    a.token_sets = a.q_sets + (a.heads[1] + rows - 1) / rows;
    a.sets = a.tokens * a.token_sets;
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

template <int DT, int V, int SH, int N, int L>
int launch_forward(const QkArgs &a, cudaStream_t st)
{
    auto kernel = k_qk_norm<DT, V, SH, N, L, N == 1 ? 6 : 3>;
    const int64_t blocks = (a.sets + kWarps - 1) / kWarps;
    kernel<<<grid_for(reinterpret_cast<const void *>(kernel), blocks, 1 << 30), kThreads, 0, st>>>(a);
    return check_launch("k_qk_norm");
}

template <int DT, int V, int SH, int N, int L>
int launch_backward(const QkArgs &a, cudaStream_t st, int *grid)
{
    auto kernel = k_qk_norm_bwd<DT, V, SH, N, L, N == 1 ? 4 : 2>;
    const int64_t blocks = (a.sets + kWarps - 1) / kWarps;
    *grid = grid_for(reinterpret_cast<const void *>(kernel), blocks, kMostSumBlocks);
    kernel<<<*grid, kThreads, 0, st>>>(a);
    return check_launch("k_qk_norm_bwd");
}

// (binary32: up to two 16-byte shares to a lane; single pairs: up to four)
#define ZERO_LANES(CALL, DT, V, SH)                                          \
    do {                                                                      \
        if (DT == ZERO_F32 && p.n == 2)                                       \
            return CALL(DT, V, SH, (DT == ZERO_F32 ? 2 : 1), 32);             \
        return p.lanes == 8    ? CALL(DT, V, SH, 1, 8)                        \
               : p.lanes == 16 ? CALL(DT, V, SH, 1, 16)                       \
                               : CALL(DT, V, SH, 1, 32);                      \
    } while (0)
#define ZERO_SHARES(CALL)                                                     \
    if (dtype == ZERO_F32) {                                                  \
        if (p.share == kSplit)                                                \
            ZERO_LANES(CALL, ZERO_F32, 4, kSplit);                            \
        if (p.share == kRun)                                                  \
            ZERO_LANES(CALL, ZERO_F32, 4, kRun);                              \
        return CALL(ZERO_F32, 2, kOne, 4, 32);                                \
    }                                                                         \
    if (dtype == ZERO_F16) {                                                  \
        if (p.share == kSplit)                                                \
            ZERO_LANES(CALL, ZERO_F16, 8, kSplit);                            \
        if (p.share == kRun)                                                  \
            ZERO_LANES(CALL, ZERO_F16, 8, kRun);                              \
        return CALL(ZERO_F16, 2, kOne, 4, 32);                                \
    }                                                                         \
    if (p.share == kSplit)                                                    \
        ZERO_LANES(CALL, ZERO_BF16, 8, kSplit);                               \
    if (p.share == kRun)                                                      \
        ZERO_LANES(CALL, ZERO_BF16, 8, kRun);                                 \
    return CALL(ZERO_BF16, 2, kOne, 4, 32);

int forward_any(const QkArgs &a, QkPlan p, int32_t dtype, cudaStream_t st)
{
#define ZERO_FWD(DT, V, SH, N, L) launch_forward<DT, V, SH, N, L>(a, st)
    ZERO_SHARES(ZERO_FWD)
#undef ZERO_FWD
}

int backward_any(const QkArgs &a, QkPlan p, int32_t dtype, cudaStream_t st, int *grid)
{
#define ZERO_BWD(DT, V, SH, N, L) launch_backward<DT, V, SH, N, L>(a, st, grid)
    ZERO_SHARES(ZERO_BWD)
#undef ZERO_BWD
}

// The partial sums of the weights' gradients: as many blocks as there may be,
// whatever the tokens.
size_t qk_ws_bytes(int64_t dim)
{
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
    Reach reach;
    ZERO_TRY(check_qk(both, 2, tokens, q_heads, k_heads, head_dim, dtype, &reach));
    if (q_weight)
        ZERO_TRY(check_array(q_weight, head_dim, wdtype, &reach));
    if (k_weight)
        ZERO_TRY(check_array(k_weight, head_dim, wdtype, &reach));
    ZERO_TRY(check_rotary(rotary, positions, tokens, &reach));
    if (tokens == 0 || q_heads + k_heads == 0 || head_dim == 0)
        return ZERO_OK;
    QkArgs a{};
    fill_qk(a, qs, ks, q_weight, k_weight, wdtype, rotary, positions, tokens, q_heads, k_heads, head_dim, eps);
    return forward_any(a, plan_qk(a, false, elem_bytes(dtype)), dtype, static_cast<cudaStream_t>(stream));
}

extern "C" size_t zero_qk_norm_workspace_bytes(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t head_dim)
{
    if (tokens < 0 || q_heads < 0 || k_heads < 0 || head_dim < 0 || tokens > kMostTokens || q_heads > kMostHeads ||
        k_heads > kMostHeads || head_dim > kMostDim)
        return 0;
    return qk_ws_bytes(head_dim);
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
    Reach reach;
    ZERO_TRY(check_qk(both, 3, tokens, q_heads, k_heads, head_dim, dtype, &reach));
    if (q_weight)
        ZERO_TRY(check_array(q_weight, head_dim, wdtype, &reach));
    if (k_weight)
        ZERO_TRY(check_array(k_weight, head_dim, wdtype, &reach));
    if (dq_weight)
        ZERO_TRY(check_array(dq_weight, head_dim, gdtype, &reach));
    if (dk_weight)
        ZERO_TRY(check_array(dk_weight, head_dim, gdtype, &reach));
    ZERO_TRY(check_rotary(rotary, positions, tokens, &reach));
    ZERO_TRY(check_workspace(ws, ws_bytes, qk_ws_bytes(head_dim), &reach));
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
        ZERO_TRY(backward_any(a, plan_qk(a, true, elem_bytes(dtype)), dtype, st, &s.blocks));
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
