// Attention with a sliding window and a few first keys that stay visible,
// forward and backward, over packed sequences and caches.
#include <cmath>
#include <initializer_list>

#include "sublayer.cuh"
#include "tensor.cuh"

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

// ------------------------------------------------------------- tiles

// Arrays of heads as the kernels load them: boxes of 64 elements of 128
// tokens of one head.
struct HeadsMap {
    CUtensorMap map;
    int32_t heads_last;  // the map's dimensions are (element, token, head), else (element, head, token)
};

__device__ __forceinline__ void load_box(uint32_t dst, const HeadsMap &m, int32_t x, int32_t token, int32_t head,
                                         uint32_t bar)
{
    tma_load3(dst, &m.map, x, m.heads_last ? token : head, m.heads_last ? head : token, bar);
}

// Tiles of the rows of all sequences, T rows each.  Sequence s has the tile
// numbers from floor(its first row / T) + s on: at least as many as it needs,
// whatever its length, so a tile's sequence is found in the offsets alone.
// (Numbers that are left over, one per sequence at most, are skipped.)
__host__ __device__ inline int64_t tile_numbers(int64_t rows, int64_t sequences, bool one, int32_t T)
{
    return one ? (rows + T - 1) / T : rows / T + sequences;
}

struct TileAt {
    Seq s;
    int32_t first;  // row of its sequence
    bool any;
};

// By a whole warp: 32 offsets at a time.
__device__ __forceinline__ TileAt find_tile(const Attn &a, const int64_t *offsets, int64_t rows, int64_t number, int32_t T,
                                            bool keys, int lane)
{
    TileAt t{};
    int32_t s = 0;
    int64_t first = number * T;
    if (offsets) {
        int32_t lo = -1, hi = a.sequences;
        while (hi - lo > 1) {
            const int32_t step = (hi - lo - 1 + 31) / 32, at = lo + (lane + 1) * step;
            const bool before = at < hi && cut(offsets[at], 0, rows) / T + at <= number;
            const int32_t n = __popc(__ballot_sync(0xffffffffu, before));
            hi = hi < lo + (n + 1) * step ? hi : lo + (n + 1) * step;
            lo += n * step;
        }
        if (lo < 0)
            return t;
        s = lo;
        first = (number - (cut(offsets[s], 0, rows) / T + s)) * T;
    }
    t.s = sequence(a, s);
    t.any = first >= 0 && first < (keys ? t.s.lk : t.s.lq);
    t.first = t.any ? (int32_t)first : 0;
    return t;
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    if constexpr (DT == ZERO_F16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

// Bits c of 0 .. 31 with c <= x.
__device__ __forceinline__ uint32_t bits_up_to(int32_t x) { return x >= 31 ? ~0u : x < 0 ? 0u : (2u << x) - 1u; }

// Of 32 keys from key `first` on: those that a query at position p sees.
__device__ __forceinline__ uint32_t seen_bits(int32_t p, int32_t window, int32_t sinks, int32_t first)
{
    const int32_t low = p >= window ? p - window + 1 : 0;
    return bits_up_to(p - first) & (~bits_up_to(low - first - 1) | bits_up_to(sinks - first - 1));
}

// The key tiles of 128 queries, and of two such tiles.
struct KeyTiles {
    int32_t low, high;  // of the window
    int32_t sinks;      // first tiles that are seen outside it
    bool any;
};

__device__ __forceinline__ KeyTiles key_tiles(const Attn &a, int32_t first, int32_t lq, int32_t lk)
{
    KeyTiles t{0, -1, 0, false};
    const int32_t last = first + 127 < lq ? first + 127 : lq - 1;
    const int32_t p0 = first + lk - lq, p1 = last + lk - lq;
    if (first >= lq || p1 < 0)
        return t;
    const int32_t sinks = a.sinks < p1 + 1 ? a.sinks : p1 + 1;
    t.any = true;
    t.low = p0 >= a.window ? (p0 - a.window + 1) / 128 : 0;
    t.high = p1 / 128;
    t.sinks = (sinks + 127) / 128;
    return t;
}

__device__ __forceinline__ bool needs(const KeyTiles &t, int32_t kt)
{
    return t.any && kt <= t.high && (kt >= t.low || kt < t.sinks);
}

// The tiles of a pair, from the last to the first: every query that sees a
// key sees one of its first tile.
struct TileList {
    int32_t high, low, sinks, n;
    __device__ __forceinline__ int32_t at(int32_t i) const
    {
        const int32_t kt = high - i;
        return kt >= low ? kt : sinks - 1 - (low - 1 - kt);
    }
};

__device__ __forceinline__ TileList tile_list(const KeyTiles &x, const KeyTiles &y)
{
    TileList l;
    l.low = !x.any ? y.low : !y.any ? x.low : x.low < y.low ? x.low : y.low;
    l.high = x.high > y.high ? x.high : y.high;
    const int32_t sinks = x.sinks > y.sinks ? x.sinks : y.sinks;
    l.sinks = sinks < l.low ? sinks : l.low;
    l.n = x.any || y.any ? l.high - l.low + 1 + l.sinks : 0;
    return l;
}

struct Unit {
    int32_t q_row, k_row;  // of the unit's first query, and the sequence's first key
    int32_t first, lq, lk, head;
    int32_t end;
};

struct FwdTiles {
    HeadsMap q, k, v;
    Attn a;
    Heads out;
    float *lse;
    int64_t tiles;
    float scale_log2;
    WsHeader *hdr;
    uint64_t limit_ns;
};

constexpr int kUnitRing = 4;

template <int DP>
struct FwdShape {
    static constexpr int BOXES = DP / 64, TILE = BOXES * 16384;  // bytes of 128 rows
    static constexpr int STAGES = DP == 64 ? 4 : 2;
    static constexpr int THREADS = 320;  // eight warps of rows, one that loads, one that issues
    static constexpr int SMEM = 1024 + (2 + 2 * STAGES) * TILE;
};

struct FwdShared {
    uint64_t q_full[2], q_empty[2], k_full[4], k_empty[4], v_full[4], v_empty[4], s_full[2], p_full[2], o_full[2];
    uint64_t unit_full[kUnitRing], unit_empty[kUnitRing];
    Unit units[kUnitRing];
    uint32_t tmem, gave_up;
};

// Two tiles of 128 queries of one head at a time (one CTA per SM, persistent).
template <int DT, int DP>
__global__ void __launch_bounds__(FwdShape<DP>::THREADS, 1) k_attn_tiles(const __grid_constant__ FwdTiles f)
{
    using S = FwdShape<DP>;
    extern __shared__ unsigned char smem_raw[];
    __shared__ FwdShared sh;
    unsigned char *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023u)) & 1023u);
    unsigned char *const s_q = smem, *const s_k = smem + 2 * S::TILE, *const s_v = s_k + S::STAGES * S::TILE;
    const Attn &a = f.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kTma = 8, kMma = 9;

    if (threadIdx.x == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init_count(&sh.q_full[t], 1);
            mbar_init_count(&sh.q_empty[t], 1);
            mbar_init_count(&sh.s_full[t], 1);
            mbar_init_count(&sh.p_full[t], 4);
            mbar_init_count(&sh.o_full[t], 1);
        }
        for (int s = 0; s < S::STAGES; ++s) {
            mbar_init_count(&sh.k_full[s], 1);
            mbar_init_count(&sh.k_empty[s], 1);
            mbar_init_count(&sh.v_full[s], 1);
            mbar_init_count(&sh.v_empty[s], 1);
        }
        for (int s = 0; s < kUnitRing; ++s) {
            mbar_init_count(&sh.unit_full[s], 1);
            mbar_init_count(&sh.unit_empty[s], 9);
        }
        sh.gave_up = 0;
        mbar_init_done();
    }
    if (warp == kMma)
        tmem_alloc<1>(&sh.tmem, 512);
    if (warp == kTma && lane < 3)
        tma_prefetch_map(lane == 0 ? &f.q.map : lane == 1 ? &f.k.map : &f.v.map);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = sh.tmem;
    auto wait = [&](uint64_t *bar, uint32_t parity) { return mbar_wait_warp(bar, parity, f.limit_ns, &sh.gave_up); };
    // the next unit, from the loading warp
    uint32_t units = 0;
    auto next = [&](Unit &u) {
        const uint32_t slot = units % kUnitRing;
        if (!wait(&sh.unit_full[slot], (units / kUnitRing) & 1))
            return false;
        u = sh.units[slot];
        __syncwarp();
        if (lane == 0)
            mbar_arrive_cluster(smem_addr(&sh.unit_empty[slot]));
        ++units;
        return u.end == 0;
    };

    if (warp == kTma) {
        uint32_t kn = 0, vn = 0, qn[2] = {0, 0};
        bool ok = true;
        auto publish = [&](const Unit &u) {
            const uint32_t slot = units % kUnitRing;
            if (!wait(&sh.unit_empty[slot], ((units / kUnitRing) & 1) ^ 1))
                return false;
            if (lane == 0) {
                sh.units[slot] = u;
                mbar_arrive_cluster(smem_addr(&sh.unit_full[slot]));
            }
            __syncwarp();
            ++units;
            return true;
        };
        auto load = [&](unsigned char *to, const HeadsMap &m, int32_t row, int32_t head, uint64_t *bar) {
            if (elect_one()) {
                mbar_expect(bar, S::TILE);
#pragma unroll
                for (int x = 0; x < S::BOXES; ++x)
                    load_box(smem_addr(to) + x * 16384, m, 64 * x, row, head, smem_addr(bar));
            }
            __syncwarp();
        };
        const int64_t all = f.tiles * a.q_heads;
        for (int64_t i = blockIdx.x; ok && i < all; i += gridDim.x) {
            // long ones first: a sequence's later queries see more keys
            const int64_t number = f.tiles - 1 - i / a.q_heads;
            const TileAt at = find_tile(a, a.q_offsets, a.q_tokens, number, 256, false, lane);
            if (!at.any)
                continue;
            const Unit u{(int32_t)at.s.q0 + at.first, (int32_t)at.s.k0, at.first, at.s.lq, at.s.lk, (int32_t)(i % a.q_heads), 0};
            if (!publish(u)) {
                ok = false;
                break;
            }
            const KeyTiles x = key_tiles(a, u.first, u.lq, u.lk), y = key_tiles(a, u.first + 128, u.lq, u.lk);
            const TileList list = tile_list(x, y);
            const int32_t g = u.head / a.group;
            for (int32_t n = 0; ok && n < list.n; ++n) {
                const int32_t kt = list.at(n);
                if (n == 0)
                    for (int t = 0; ok && t < 2; ++t) {
                        if (!(t ? y.any : x.any))
                            continue;
                        ok = wait(&sh.q_empty[t], (qn[t] & 1) ^ 1);
                        if (ok)
                            load(s_q + t * S::TILE, f.q, u.q_row + 128 * t, u.head, &sh.q_full[t]);
                        ++qn[t];
                    }
                const uint32_t ks = kn % S::STAGES;
                ok = ok && wait(&sh.k_empty[ks], ((kn / S::STAGES) & 1) ^ 1);
                if (!ok)
                    break;
                load(s_k + ks * S::TILE, f.k, u.k_row + kt * 128, g, &sh.k_full[ks]);
                ++kn;
                const uint32_t vs = vn % S::STAGES;
                ok = wait(&sh.v_empty[vs], ((vn / S::STAGES) & 1) ^ 1);
                if (!ok)
                    break;
                load(s_v + vs * S::TILE, f.v, u.k_row + kt * 128, g, &sh.v_full[vs]);
                ++vn;
            }
        }
        if (ok)
            publish(Unit{0, 0, 0, 0, 0, 0, 1});
    } else if (warp == kMma) {
        constexpr uint32_t kBf16 = DT == ZERO_BF16;
        const uint32_t desc_s = product_desc(kBf16, false, false, 128, 128);
        const int wide = (a.dim + 15) & ~15, steps = wide / 16;
        const uint32_t desc_o = product_desc(kBf16, false, true, 128, wide);
        const uint64_t q0 = operand_desc(smem_addr(s_q), 16, 1024), k0 = operand_desc(smem_addr(s_k), 16, 1024);
        const uint64_t v0 = operand_desc(smem_addr(s_v), 16384, 1024);
        uint32_t kn = 0, vn = 0, qn[2] = {0, 0}, pn[2] = {0, 0};
        bool ok = true;
        Unit u;
        while (ok && next(u)) {
            const KeyTiles kt2[2] = {key_tiles(a, u.first, u.lq, u.lk), key_tiles(a, u.first + 128, u.lq, u.lk)};
            const TileList list = tile_list(kt2[0], kt2[1]);
            // S_t = Q_t K^T of the n-th tile
            auto scores = [&](int t, uint32_t stage) {
                if (elect_one()) {
                    const uint64_t dq = q0 + ((t * S::TILE) >> 4), dk = k0 + ((stage * S::TILE) >> 4);
                    for (int s = 0; s < steps; ++s) {
                        const uint32_t off = (s >> 2) * (16384 >> 4) + (s & 3) * 2;
                        tensor_product<1>(tmem + t * 128, dq + off, dk + off, desc_s, s != 0);
                    }
                    tensor_commit<1>(&sh.s_full[t]);
                }
                __syncwarp();
            };
            bool first[2] = {true, true};
            for (int32_t n = 0; ok && n <= list.n; ++n) {
                const int32_t kt = n < list.n ? list.at(n) : -1, before = n > 0 ? list.at(n - 1) : -1;
                const uint32_t ks = kn % S::STAGES, vs = vn % S::STAGES;
                bool k_here = false, v_here = false;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (n > 0 && needs(kt2[t], before)) {
                        if (!v_here)
                            ok = ok && wait(&sh.v_full[vs], (vn / S::STAGES) & 1);
                        v_here = true;
                        ok = ok && wait(&sh.p_full[t], pn[t] & 1);
                        ++pn[t];
                        if (!ok)
                            break;
                        tmem_fence_after();
                        if (elect_one()) {
                            const uint64_t dv = v0 + ((vs * S::TILE) >> 4);
#pragma unroll
                            for (int s = 0; s < 8; ++s)
                                tensor_product_tmem(tmem + 256 + t * 128, tmem + t * 128 + s * 8, dv + s * 128, desc_o,
                                                    !first[t] || s != 0);
                            // the last product of this tile of queries?
                            bool more = false;
                            for (int32_t m = n; m < list.n && !more; ++m)
                                more = needs(kt2[t], list.at(m));
                            if (!more)
                                tensor_commit<1>(&sh.o_full[t]);
                        }
                        __syncwarp();
                        first[t] = false;
                    }
                    if (kt >= 0 && needs(kt2[t], kt)) {
                        if (!k_here)
                            ok = ok && wait(&sh.k_full[ks], (kn / S::STAGES) & 1);
                        k_here = true;
                        if (first[t])  // these queries' first scores
                            ok = ok && wait(&sh.q_full[t], qn[t] & 1);
                        if (!ok)
                            break;
                        tmem_fence_after();
                        scores(t, ks);
                    }
                }
                if (!ok)
                    break;
                if (elect_one()) {
                    if (n > 0)
                        tensor_commit<1>(&sh.v_empty[vs]);
                    if (kt >= 0)
                        tensor_commit<1>(&sh.k_empty[ks]);
                    if (n + 1 == list.n) {
                        if (kt2[0].any)
                            tensor_commit<1>(&sh.q_empty[0]);
                        if (kt2[1].any)
                            tensor_commit<1>(&sh.q_empty[1]);
                    }
                }
                __syncwarp();
                vn += n > 0;
                kn += kt >= 0;
            }
            qn[0] += kt2[0].any;
            qn[1] += kt2[1].any;
        }
    } else {
        const int t = warp >> 2, quarter = warp & 3;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const uint32_t at_s = tmem + lanes + t * 128, at_o = tmem + lanes + 256 + t * 128;
        const float sl = f.scale_log2;
        uint32_t sn = 0, on = 0, vn = 0;
        bool ok = true;
        Unit u;
        while (ok && next(u)) {
            const KeyTiles x = key_tiles(a, u.first, u.lq, u.lk), y = key_tiles(a, u.first + 128, u.lq, u.lk);
            const KeyTiles mine = t ? y : x;
            const TileList list = tile_list(x, y);
            const int32_t row = u.first + 128 * t + quarter * 32 + lane, p = row + u.lk - u.lq;
            const int32_t p_first = u.first + 128 * t + u.lk - u.lq;
            const int32_t p_last = (u.first + 128 * t + 127 < u.lq ? u.first + 128 * t + 127 : u.lq - 1) + u.lk - u.lq;
            float m = -INFINITY, l = 0.0f;
            for (int32_t n = 0; n < list.n; ++n) {
                const int32_t kt = list.at(n);
                if (!needs(mine, kt))
                    continue;
                ok = ok && wait(&sh.s_full[t], sn & 1);
                ++sn;
                if (!ok)
                    break;
                tmem_fence_after();
                const int32_t k_first = kt * 128;
                const bool whole = k_first + 127 <= p_first &&
                                   (k_first > p_last - a.window || k_first + 127 < a.sinks);
                uint32_t r[2][32];
                auto load = [&](int c) {  // 64 scores from column 64 c on
                    tmem_load32(at_s + 64 * c, r[0]);
                    tmem_load32(at_s + 64 * c + 32, r[1]);
                    tmem_wait_loads(r[0]);
                    tmem_wait_loads(r[1]);
                    if (!whole) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t bits = seen_bits(p, a.window, a.sinks, k_first + 64 * c + 32 * h);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                r[h][e] = bits & (1u << e) ? r[h][e] : 0xff800000u;
                        }
                    }
                };
                float top = -INFINITY;
#pragma unroll
                for (int c = 1; c >= 0; --c) {
                    load(c);
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            top = fmaxf(top, __uint_as_float(r[h][e]));
                }
                // The weights' reference is the largest score so far, or up to
                // 2^8 below it: the weights stay below 2^8, and sums are
                // rarely multiplied anew.
                const bool far = top > m && (m == -INFINITY || (top - m) * sl > 8.0f);
                if (__any_sync(0xffffffffu, far)) {
                    const float to = far ? top : m;
                    const float keep = m == -INFINITY ? 0.0f : exp2_fast((m - to) * sl);
                    if (__any_sync(0xffffffffu, l != 0.0f)) {
                        for (int c = 0; c < a.dim; c += 32) {
                            uint32_t o[32];
                            tmem_load32(at_o + c, o);
                            tmem_wait_loads(o);
                            uint32_t lo[16], hi[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                lo[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
                                hi[e] = __float_as_uint(__uint_as_float(o[16 + e]) * keep);
                            }
                            tmem_store16(at_o + c, lo);
                            tmem_store16(at_o + c + 16, hi);
                        }
                    }
                    l *= keep;
                    m = to;
                }
                const float base = m == -INFINITY ? 0.0f : m * sl;
                float sum[4] = {};
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    if (c)  // the others again: all 128 do not fit the registers
                        load(c);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float w0 = exp2_fast(__uint_as_float(r[h][2 * e]) * sl - base);
                            const float w1 = exp2_fast(__uint_as_float(r[h][2 * e + 1]) * sl - base);
                            sum[e & 1] += w0;
                            sum[2 + (e & 1)] += w1;
                            w[e] = pack2<DT>(w0, w1);
                        }
                        tmem_store16(at_s + 32 * c + 16 * h, w);
                    }
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                if (k_first + 128 > u.lk) {
                    // rows behind the last key: zeros, since 0 times what they hold may not be 0
                    const uint32_t now = vn + n, vs = now % S::STAGES;
                    ok = wait(&sh.v_full[vs], (now / S::STAGES) & 1);
                    if (!ok)
                        break;
                    const int32_t from = u.lk - k_first;
                    const int id = threadIdx.x & 127;
                    for (int i = from * 8 + id; i < 1024; i += 128)
#pragma unroll
                        for (int b = 0; b < S::BOXES; ++b)
                            *reinterpret_cast<uint4 *>(s_v + vs * S::TILE + b * 16384 + i * 16) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async();
                }
                tmem_wait_stores();
                tmem_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_cluster(smem_addr(&sh.p_full[t]));
            }
            vn += list.n;
            if (!ok)
                break;
            if (u.first + 128 * t >= u.lq)
                continue;  // no such tile
            if (mine.any) {
                ok = wait(&sh.o_full[t], on & 1);
                ++on;
                tmem_fence_after();
                if (!ok)
                    break;
            }
            const bool live = row < u.lq;
            const int64_t out_row = (int64_t)u.q_row + 128 * t + quarter * 32 + lane;
            if (live && f.lse)
                f.lse[(int64_t)u.head * a.q_tokens + out_row] =
                    l == 0.0f ? -INFINITY : m * a.scale + logf(l);
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            char *out = static_cast<char *>(const_cast<void *>(f.out.p)) + (out_row * f.out.ld + u.head * f.out.hd) * 2;
            for (int c = 0; c < a.dim; c += 32) {
                uint32_t o[32];
                if (mine.any) {
                    tmem_load32(at_o + c, o);
                    tmem_wait_loads(o);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o[e] = 0;
                }
                if (live) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        if (c + e >= a.dim)
                            break;
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float f0 = l == 0.0f ? 0.0f : __uint_as_float(o[e + 2 * i]) * inv;
                            const float f1 = l == 0.0f ? 0.0f : __uint_as_float(o[e + 2 * i + 1]) * inv;
                            w[i] = pack2<DT>(f0, f1);
                        }
                        *reinterpret_cast<uint4 *>(out + (c + e) * 2) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                __syncwarp();
            }
        }
    }

    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    if (sh.gave_up) {
        // copies and products may still be in flight: let them end before
        // the memory that they use is given back
        if (threadIdx.x == 0)
            atomicAdd(&f.hdr->stalls, 1u);
        const uint64_t began = global_ns();
        while (global_ns() - began < 20000000u) {
        }
        // no result of this CTA is to be taken for one
        const int64_t all = f.tiles * a.q_heads;
        for (int64_t i = blockIdx.x; i < all; i += gridDim.x) {
            const TileAt at = find_tile(a, a.q_offsets, a.q_tokens, f.tiles - 1 - i / a.q_heads, 256, false, lane);
            const int64_t head = i % a.q_heads;
            for (int32_t r = at.first + warp; at.any && r < at.s.lq && r < at.first + 256; r += S::THREADS / 32) {
                for (int e = lane; e < a.dim; e += 32)
                    static_cast<uint16_t *>(const_cast<void *>(f.out.p))[(at.s.q0 + r) * f.out.ld + head * f.out.hd + e] = 0x7fff;
                if (lane == 0 && f.lse)
                    f.lse[head * a.q_tokens + at.s.q0 + r] = __uint_as_float(0x7fffffffu);
            }
        }
    }
    if (warp == kMma)
        tmem_free<1>(tmem, 512);
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
    if ((tokens > 1 && h->ld == 0) || (heads > 1 && h->hd == 0))
        return ZERO_EINVAL;
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

// The map of an array of heads; both strides are positive or not needed.
int heads_map(HeadsMap *m, const Heads &h, int64_t tokens, int64_t heads, int64_t dim, int32_t dtype)
{
    const EncodeTiled encode = encode_tiled();
    if (!encode) {
        set_cuda_error("cuTensorMapEncodeTiled", 0, "entry point not found");
        return ZERO_ECUDA;
    }
    const int64_t row = (dim + 7) & ~(int64_t)7;
    const int64_t ld = tokens > 1 ? h.ld : heads > 1 ? h.hd * heads : row, hd = heads > 1 ? h.hd : row;
    m->heads_last = ld < hd;
    cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)tokens};
    cuuint64_t strides[2] = {(cuuint64_t)hd * 2, (cuuint64_t)ld * 2};
    cuuint32_t box[3] = {64, 1, 128};
    const cuuint32_t step[3] = {1, 1, 1};
    if (m->heads_last) {
        dims[1] = (cuuint64_t)tokens, dims[2] = (cuuint64_t)heads;
        strides[0] = (cuuint64_t)ld * 2, strides[1] = (cuuint64_t)hd * 2;
        box[1] = 128, box[2] = 1;
    }
    const CUresult r = encode(&m->map, dtype == ZERO_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                              3, const_cast<void *>(h.p), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        set_cuda_error("cuTensorMapEncodeTiled", (int)r, "tensor map refused");
        return ZERO_ECUDA;
    }
    return ZERO_OK;
}

constexpr uint64_t kWaitLimit = 4000000000u;

template <int DT, int DP>
int launch_tiles(const FwdTiles &t, cudaStream_t st)
{
    using S = FwdShape<DP>;
    auto kernel = k_attn_tiles<DT, DP>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    const int64_t units = t.tiles * t.a.q_heads;
    if (e == cudaSuccess) {
        kernel<<<(unsigned)(units < sm_count() ? units : sm_count()), S::THREADS, S::SMEM, st>>>(t);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        set_cuda_error("k_attn_tiles", (int)e, cudaGetErrorString(e));
        return ZERO_ECUDA;
    }
    return ZERO_OK;
}

int forward_tiles(const Fwd &f, const zero_attention_t *a, void *ws, cudaStream_t st)
{
    FwdTiles t{};
    ZERO_TRY(heads_map(&t.q, f.q, a->q_tokens, a->q_heads, a->head_dim, a->dtype));
    ZERO_TRY(heads_map(&t.k, f.k, a->k_tokens, a->k_heads, a->head_dim, a->dtype));
    ZERO_TRY(heads_map(&t.v, f.v, a->k_tokens, a->k_heads, a->head_dim, a->dtype));
    t.a = f.a, t.out = f.out, t.lse = f.lse;
    t.tiles = tile_numbers(a->q_tokens, a->sequences, !a->q_offsets, 256);
    t.scale_log2 = (float)(a->scale * 1.4426950408889634);
    t.hdr = static_cast<WsHeader *>(ws);
    t.limit_ns = kWaitLimit;
    if (a->head_dim <= 64)
        return a->dtype == ZERO_F16 ? launch_tiles<ZERO_F16, 64>(t, st) : launch_tiles<ZERO_BF16, 64>(t, st);
    return a->dtype == ZERO_F16 ? launch_tiles<ZERO_F16, 128>(t, st) : launch_tiles<ZERO_BF16, 128>(t, st);
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
    if (a->k_tokens > 0 && a->q_tokens > 4 * a->sequences)
        return forward_tiles(f, a, ws, st);
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
