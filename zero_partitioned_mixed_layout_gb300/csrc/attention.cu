// Attention with a sliding window and a few first keys that stay visible,
// forward and backward, over packed sequences and caches.
//
// Query i of a sequence stands at key p = i + Lk - Lq and sees key j iff
// 0 <= j <= p and (j > p - window or j < sinks).  Over the keys that it sees
//     s_ij = scale q_i.k_j,  lse_i = log sum_j exp s_ij,  o_i = sum_j exp(s_ij - lse_i) v_j,
// in one pass: with a reference m (about the largest score so far),
// l = sum exp(s - m) and O = sum exp(s - m) v, and both times
// exp(m - m') when the reference moves to m'; o = O / l, lse = m + log l.
// (lse is put together from the largest score itself, rounded as the backward
// pass rounds it, so that of a score past 2^24 its own weight there is 1.)
// Scores, l and O are binary32.  exp(s - m) is rounded to 16 bits once, as
// the second product's operand: by at most half a step (2^-8 in bf16, 2^-11
// in f16) of each weight, as much as the output itself is rounded by; l adds
// up the weights as they were before.  f16 has steps of 2^-24 at its low end,
// and so weights, l and O are all 2^7 times as large there (kShift): up to
// 2^15 instead of 2^8, and rounded by half a step down to 2^-21 of the largest.
// (At 1 and less, 65536 keys of a weight of 2^-25 each beside a first key of
// 1 added up to nothing in O and to 2^-9 in l.)
//
// Three ways: tiles of 128 queries on the tensor cores (k_attn_tiles), a few
// queries per sequence (k_attn_few), and the backward pass (k_attn_stats,
// k_attn_dkv, k_attn_dq, k_attn_join).
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

// A sequence cut to the rows that there are, whatever the arrays hold.
__device__ __forceinline__ Seq sequence_of(const Attn &a, int64_t q_from, int64_t q_to, int64_t k_from, int64_t k_to,
                                           int64_t k_length)
{
    Seq q;
    q.q0 = a.q_offsets ? cut(q_from, 0, a.q_tokens) : 0;
    q.lq = (int32_t)((a.q_offsets ? cut(q_to, q.q0, a.q_tokens) : a.q_tokens) - q.q0);
    if (!a.k_offsets) {
        q.k0 = q.q0, q.lk = q.lq;
        return q;
    }
    q.k0 = cut(k_from, 0, a.k_tokens);
    const int64_t room = cut(k_to, q.k0, a.k_tokens) - q.k0;
    q.lk = (int32_t)(a.k_lengths ? cut(k_length, 0, room) : room);
    return q;
}

__device__ __forceinline__ Seq sequence(const Attn &a, int32_t s)
{
    return sequence_of(a, a.q_offsets ? a.q_offsets[s] : 0, a.q_offsets ? a.q_offsets[s + 1] : 0,
                       a.k_offsets ? a.k_offsets[s] : 0, a.k_offsets ? a.k_offsets[s + 1] : 0,
                       a.k_lengths ? a.k_lengths[s] : 0);
}

struct Fwd {
    Attn a;
    Heads q, k, v, out;
    float *lse;
};

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
    int32_t index;  // of the sequence
    int32_t first;  // row of its sequence
    bool any;
};

// The tile's number that sequence s starts at, of an offset as it is.
__device__ __forceinline__ int64_t first_tile(int64_t offset, int64_t rows, int32_t s, int32_t T)
{
    return (int64_t)((uint32_t)cut(offset, 0, rows) / (uint32_t)T) + s;  // (rows fit 31 bits)
}

// By a whole warp.  Up to 31 sequences' arrays arrive in one round, an entry
// per lane; of more, 32 offsets are looked at in each round of a search.
__device__ __forceinline__ TileAt find_tile(const Attn &a, const int64_t *offsets, int64_t rows, int64_t number, int32_t T,
                                            bool keys, int lane)
{
    TileAt t{};
    int32_t s = 0;
    int64_t first = number * T;
    if (offsets && a.sequences < 32) {
        const int32_t n = a.sequences;
        const bool in = lane <= n;
        const int64_t q = a.q_offsets && in ? a.q_offsets[lane] : 0, k = a.k_offsets && in ? a.k_offsets[lane] : 0;
        const int64_t l = a.k_lengths && lane < n ? a.k_lengths[lane] : 0;
        const int64_t at = first_tile(offsets == a.q_offsets ? q : k, rows, lane, T);
        s = __popc(__ballot_sync(0xffffffffu, lane < n && at <= number)) - 1;
        if (s < 0)
            return t;
        first = (number - __shfl_sync(0xffffffffu, at, s)) * T;
        const int64_t q0 = __shfl_sync(0xffffffffu, q, s), q1 = __shfl_sync(0xffffffffu, q, s + 1);
        const int64_t k0 = __shfl_sync(0xffffffffu, k, s), k1 = __shfl_sync(0xffffffffu, k, s + 1);
        t.s = sequence_of(a, q0, q1, k0, k1, __shfl_sync(0xffffffffu, l, s));
    } else {
        if (offsets) {
            int32_t lo = -1, hi = a.sequences;
            while (hi - lo > 1) {
                const int32_t step = (hi - lo - 1 + 31) / 32, at = lo + (lane + 1) * step;
                const bool before = at < hi && first_tile(offsets[at], rows, at, T) <= number;
                const int32_t n = __popc(__ballot_sync(0xffffffffu, before));
                hi = hi < lo + (n + 1) * step ? hi : lo + (n + 1) * step;
                lo += n * step;
            }
            if (lo < 0)
                return t;
            s = lo;
            first = (number - first_tile(offsets[s], rows, s, T)) * T;
        }
        t.s = sequence(a, s);
    }
    t.index = s;
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

__device__ __forceinline__ F2 exp2_fast(F2 x) { return {exp2_fast(x.x), exp2_fast(x.y)}; }

// The forward pass's weights are 2^kShift exp(s - m).
template <int DT>
constexpr float kShift = DT == ZERO_F16 ? 7.0f : 0.0f;

// log of a row's sum of weights: of the largest score `best`, the reference m
// (up to 2^8 of a weight lower) and l.
template <int DT>
__device__ __forceinline__ float row_lse(float best, float m, float l, float scale)
{
    return __fadd_rn(__fmul_rn(best, scale), logf(DT == ZERO_F16 ? l * 0x1p-7f : l) + (m - best) * scale);
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

// A value that all lanes of a warp hold, in a form that the compiler can tell:
// loops over it are then uniform, and so are the operands of the products
// issued in them.
__device__ __forceinline__ int32_t uniform(int32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

// The tiles of BN keys that 128 queries see, and two such tiles of queries.
struct KeyTiles {
    int32_t low, high;  // of the window
    int32_t sinks;      // first tiles that are seen outside it
    bool any;
};

template <int BN>
__device__ __forceinline__ KeyTiles key_tiles(const Attn &a, int32_t first, int32_t lq, int32_t lk)
{
    KeyTiles t{0, -1, 0, false};
    const int32_t last = first + 127 < lq ? first + 127 : lq - 1;
    const int32_t p0 = first + lk - lq, p1 = last + lk - lq;
    if (first >= lq || p1 < 0)
        return t;
    const int32_t sinks = a.sinks < p1 + 1 ? a.sinks : p1 + 1;
    t.any = true;
    t.low = p0 >= a.window ? (p0 - a.window + 1) / BN : 0;
    t.high = p1 / BN;
    t.sinks = (sinks + BN - 1) / BN;
    return t;
}

__device__ __forceinline__ bool needs(const KeyTiles &t, int32_t kt)
{
    return t.any && kt <= t.high && (kt >= t.low || kt < t.sinks);
}

// The tiles of a pair, from the last to the first.
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

    __device__ __forceinline__ void agree()
    {
        q_row = uniform(q_row), k_row = uniform(k_row), first = uniform(first), lq = uniform(lq), lk = uniform(lk);
        head = uniform(head), end = uniform(end);
    }
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

// D = A B^T over the elements of a head (16 to a step), in boxes of 64
// elements by A_ROWS and B_ROWS rows.
template <int DP, int A_ROWS, int B_ROWS>
__device__ __forceinline__ void inner_products(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, int steps)
{
    tensor_products4<2, 2>(d, a, b, desc, false, steps);
    if (DP == 128 && steps > 4)
        tensor_products4<2, 2>(d, a + (A_ROWS * 128 >> 4), b + (B_ROWS * 128 >> 4), desc, true, steps - 4);
}

// Where a thread's 32 columns of piece c (0, 1) of BN start: a group of four
// warps takes 64 of 128 columns, in two pieces that it shares with the other
// group, so that the products over the first 64 can start when half of the
// work is done; of 64 columns there is one group.  What a thread writes, two
// elements to a column, starts where it read.
template <int BN>
__device__ __forceinline__ int piece_at(int group, int c)
{
    return BN == 128 ? 64 * c + 32 * group : 32 * c;
}

// QT tiles of 128 queries against tiles of BN keys, whose scores take 128
// columns of tensor memory for a tile of queries: one tile's of 128 keys, or
// two's of 64.
template <int DP_, int QT_, int BN_, int PER_SM_>
struct FwdShape {
    static constexpr int DP = DP_, QT = QT_, BN = BN_, PER_SM = PER_SM_;
    static constexpr int HALVES = BN / 64, BUFFERS = 128 / BN;
    static constexpr int BOXES = DP / 64, Q_TILE = BOXES * 16384, K_TILE = BOXES * BN * 128;  // bytes
    static constexpr int STAGES = 2 * BUFFERS;
    static constexpr int ROW_WARPS = 4 * QT, THREADS = (ROW_WARPS + 2) * 32;
    static constexpr int TMEM = QT * (128 + DP) <= 256 ? 256 : 512;
    static constexpr int SMEM = 1024 + QT * Q_TILE + 2 * STAGES * K_TILE + ROW_WARPS * 4096;
    static_assert(SMEM * PER_SM <= 227 * 1024 && TMEM * PER_SM <= 512 && QT * (128 + DP) <= TMEM, "what an SM has");
    static_assert(QT == 1 || BUFFERS == 1, "two barriers of scores");
};

// s_full: of each tile of queries, or of each buffer of one's scores; p_full:
// of its halves, or buffers; sum_done: the later half's products are in the
// sums, or a tile's.
struct FwdShared {
    uint64_t q_full[2], q_empty[2], k_full[4], k_empty[4], v_full[4], v_empty[4], s_full[2], p_full[2][2], sum_done[2], o_full[2];
    uint64_t unit_full[kUnitRing], unit_empty[kUnitRing];
    Unit units[kUnitRing];
    uint32_t tmem, gave_up;
};

// 32 rows of 32 or 64 elements (16 or 32 words) of one warp, a row per lane, through 2 or 4 KB
// of shared memory (16-byte pieces XORed by the row, so that neither way has
// bank conflicts) to rows of memory `ld` elements apart, whole rows at a time.
// Rows from `rows` and elements from `cols` on are not written.
template <int WORDS>
__device__ __forceinline__ void store_rows(uint4 *stage, int lane, const uint32_t (&w)[WORDS], uint16_t *out, int64_t ld, int rows,
                                           int cols)
{
    constexpr int P = WORDS / 4, SHIFT = P == 8 ? 0 : 1;  // pieces of a row
#pragma unroll
    for (int k = 0; k < P; ++k)
        stage[lane * P + (k ^ ((lane >> SHIFT) & (P - 1)))] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
    __syncwarp();
    const int k = lane & (P - 1);
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int r = 32 / P * i + lane / P;
        const uint4 v = stage[r * P + (k ^ ((r >> SHIFT) & (P - 1)))];
        if (r < rows && k * 8 < cols)
            *reinterpret_cast<uint4 *>(out + r * ld + k * 8) = v;
    }
    __syncwarp();
}

// QT tiles of 128 queries of one head at a time, by a persistent CTA: one warp
// loads, one issues the products, and the others hold a row of the scores per
// thread: their largest, the weights (which take the scores' place in tensor
// memory, as the first operand of the product with the values) and their sum.
//
// What bounds it: of 128 x 128 scores the tensor pipe takes 8 clocks per
// element of a head (1024 at 128), the exponentials 512, and the other
// instructions of a row's thread (scores to registers, largest, sum, packing,
// weights back) about as many issue slots again on each of the four
// schedulers, so at 128 elements both pipes have to run without a pause.  With
// one tile per CTA they wait for one another; two tiles take turns.  Measured:
// 16384 tokens of 64 + 8 heads of 128, window 2048: 792 us, 1.34 PFLOP/s, 0.69
// of cuBLAS's burst rate (the same loads and products without the softmax
// between them: 598).  Tiles of 64 keys in two buffers instead, when it took
// 770: 1039.  Heads of 64: 8 x 1024 tokens of 25, window 256: 44.5 us.  128 x 64
// scores are 256 clocks of the tensor pipe, a row's thread takes several times that,
// and the masked edges of a short window are worked out in full.  Tiles of 64
// keys, whose scores are ready in a second buffer when those before are
// through, mask less and wait less than of 128 in one: 50 (both when one
// operation less took 43.5).
template <int DT, class S>
__global__ void __launch_bounds__(S::THREADS, S::PER_SM) k_attn_tiles(const __grid_constant__ FwdTiles f)
{
    constexpr int DP = S::DP, QT = S::QT, BN = S::BN, BUFFERS = S::BUFFERS;
    extern __shared__ unsigned char smem_raw[];
    __shared__ FwdShared sh;
    unsigned char *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023u)) & 1023u);
    unsigned char *const s_q = smem, *const s_k = smem + QT * S::Q_TILE, *const s_v = s_k + S::STAGES * S::K_TILE;
    unsigned char *const s_out = s_v + S::STAGES * S::K_TILE;
    const Attn &a = f.a;
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    constexpr int kTma = S::ROW_WARPS, kMma = S::ROW_WARPS + 1;
    constexpr int kScores = 128, kSums = QT * 128;  // columns of tensor memory: of a tile's scores, where the sums start

    if (threadIdx.x == 0) {
        for (int t = 0; t < QT; ++t) {
            mbar_init_count(&sh.q_full[t], 1);
            mbar_init_count(&sh.q_empty[t], 1);
            mbar_init_count(&sh.p_full[t][0], 4);
            mbar_init_count(&sh.p_full[t][1], 4);
            mbar_init_count(&sh.sum_done[t], 1);
            mbar_init_count(&sh.o_full[t], 1);
        }
        mbar_init_count(&sh.s_full[0], 1);
        mbar_init_count(&sh.s_full[1], 1);
        for (int s = 0; s < S::STAGES; ++s) {
            mbar_init_count(&sh.k_full[s], 1);
            mbar_init_count(&sh.k_empty[s], 1);
            mbar_init_count(&sh.v_full[s], 1);
            mbar_init_count(&sh.v_empty[s], 1);
        }
        for (int s = 0; s < kUnitRing; ++s) {
            mbar_init_count(&sh.unit_full[s], 1);
            mbar_init_count(&sh.unit_empty[s], S::ROW_WARPS + 1);
        }
        sh.gave_up = 0;
        mbar_init_done();
    }
    if (warp == kMma)
        tmem_take(&sh.tmem, S::TMEM);
    if (warp == kTma && lane < 3)
        tma_prefetch_map(lane == 0 ? &f.q.map : lane == 1 ? &f.k.map : &f.v.map);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = (uint32_t)uniform((int32_t)sh.tmem);
    auto wait = [&](uint64_t *bar, uint32_t parity) { return mbar_wait_warp(bar, parity, f.limit_ns, &sh.gave_up); };
    auto second = [&](const Unit &u) { return QT == 2 ? key_tiles<BN>(a, u.first + 128, u.lq, u.lk) : KeyTiles{0, -1, 0, false}; };
    // the next unit, from the loading warp
    uint32_t units = 0;
    auto next = [&](Unit &u) {
        const uint32_t slot = units % kUnitRing;
        if (!wait(&sh.unit_full[slot], (units / kUnitRing) & 1))
            return false;
        u = sh.units[slot];
        u.agree();
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
        auto load = [&](unsigned char *to, const HeadsMap &m, int32_t row, int32_t head, int box, uint64_t *bar) {
            if (elect_one()) {
                mbar_expect(bar, S::BOXES * box);
#pragma unroll
                for (int x = 0; x < S::BOXES; ++x)
                    load_box(smem_addr(to) + x * box, m, 64 * x, row, head, smem_addr(bar));
            }
            __syncwarp();
        };
        const int64_t all = f.tiles * a.q_heads;
        for (int64_t i = blockIdx.x; ok && i < all; i += gridDim.x) {
            // long ones first: a sequence's later queries see more keys
            const int64_t number = f.tiles - 1 - i / a.q_heads;
            const TileAt at = find_tile(a, a.q_offsets, a.q_tokens, number, 128 * QT, false, lane);
            if (!at.any)
                continue;
            const Unit u{(int32_t)at.s.q0 + at.first, (int32_t)at.s.k0, at.first, at.s.lq, at.s.lk, (int32_t)(i % a.q_heads), 0};
            if (!publish(u)) {
                ok = false;
                break;
            }
            const KeyTiles x = key_tiles<BN>(a, u.first, u.lq, u.lk), y = second(u);
            const TileList list = tile_list(x, y);
            const int32_t g = u.head / a.group;
            for (int32_t n = 0; ok && n < list.n; ++n) {
                const int32_t kt = list.at(n);
                if (n == 0)
                    for (int t = 0; ok && t < QT; ++t) {
                        if (!(t ? y.any : x.any))
                            continue;
                        ok = wait(&sh.q_empty[t], (qn[t] & 1) ^ 1);
                        if (ok)
                            load(s_q + t * S::Q_TILE, f.q, u.q_row + 128 * t, u.head, 16384, &sh.q_full[t]);
                        ++qn[t];
                    }
                const uint32_t ks = kn % S::STAGES;
                ok = ok && wait(&sh.k_empty[ks], ((kn / S::STAGES) & 1) ^ 1);
                if (!ok)
                    break;
                load(s_k + ks * S::K_TILE, f.k, u.k_row + kt * BN, g, BN * 128, &sh.k_full[ks]);
                ++kn;
                const uint32_t vs = vn % S::STAGES;
                ok = wait(&sh.v_empty[vs], ((vn / S::STAGES) & 1) ^ 1);
                if (!ok)
                    break;
                load(s_v + vs * S::K_TILE, f.v, u.k_row + kt * BN, g, BN * 128, &sh.v_full[vs]);
                ++vn;
            }
        }
        if (ok)
            publish(Unit{0, 0, 0, 0, 0, 0, 1});
    } else if (warp == kMma) {
        constexpr uint32_t kBf16 = DT == ZERO_BF16;
        const uint32_t desc_s = product_desc(kBf16, false, false, 128, BN);
        const int wide = (a.dim + 15) & ~15, steps = wide / 16;
        const uint32_t desc_o = product_desc(kBf16, false, true, 128, wide);
        const uint64_t q0 = operand_desc(smem_addr(s_q), 16, 1024), k0 = operand_desc(smem_addr(s_k), 16, 1024);
        const uint64_t v0 = operand_desc(smem_addr(s_v), BN * 128, 1024);
        uint32_t kn = 0, vn = 0, qn[2] = {0, 0}, sn = 0, pn[2] = {0, 0};
        bool ok = true;
        Unit u;
        while (ok && next(u)) {
            const KeyTiles kt2[2] = {key_tiles<BN>(a, u.first, u.lq, u.lk), second(u)};
            const TileList list = tile_list(kt2[0], kt2[1]);
            // S_t = Q_t K^T of the n-th tile
            auto scores = [&](int t, uint32_t stage) {
                const uint32_t buffer = BUFFERS == 2 ? sn++ & 1 : 0;
                inner_products<DP, 128, BN>(tmem + t * kScores + buffer * 64, q0 + ((t * S::Q_TILE) >> 4),
                                            k0 + ((stage * S::K_TILE) >> 4), desc_s, steps);
                tensor_commit_elected(&sh.s_full[t + buffer]);
            };
            bool first[2] = {true, true};
            // (the tiles of first keys come last, down to 0; without them the window's end with its lowest)
            const int32_t last[2] = {kt2[0].sinks && kt2[0].low ? 0 : kt2[0].low, kt2[1].sinks && kt2[1].low ? 0 : kt2[1].low};
            // a tile's scores go ahead of the products of the BUFFERS-th tile before
            for (int32_t n = 0; ok && list.n > 0 && n < list.n + BUFFERS; ++n) {
                const bool ended = n >= BUFFERS && n - BUFFERS < list.n;
                const int32_t kt = n < list.n ? list.at(n) : -1, before = ended ? list.at(n - BUFFERS) : -1;
                const uint32_t ks = kn % S::STAGES, vs = vn % S::STAGES;
                bool k_here = false, v_here = false;
#pragma unroll
                for (int t = 0; t < QT; ++t) {
                    if (ended && needs(kt2[t], before)) {
                        if (!v_here)
                            ok = ok && wait(&sh.v_full[vs], (vn / S::STAGES) & 1);
                        v_here = true;
                        // the later keys' weights come first
                        const uint64_t dv = v0 + ((vs * S::K_TILE) >> 4);
#pragma unroll
                        for (int h = S::HALVES - 1; h >= 0; --h) {
                            const uint32_t piece = BUFFERS == 2 ? pn[t] & 1 : h;
                            ok = ok && wait(&sh.p_full[t][piece], BUFFERS == 2 ? (pn[t] >> 1) & 1 : pn[t] & 1);
                            if (!ok)
                                break;
                            tmem_fence_after();
                            tensor_products4_tmem<128, 16>(tmem + kSums + t * DP, tmem + t * kScores + piece * 64, dv + h * 512, desc_o,
                                                           !first[t] || h + 1 < S::HALVES);
                            if (BUFFERS == 2 || h)
                                tensor_commit_elected(&sh.sum_done[t]);
                        }
                        ++pn[t];
                        if (!ok)
                            break;
                        if (before == last[t])
                            tensor_commit_elected(&sh.o_full[t]);
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
                if (ended)
                    tensor_commit_elected(&sh.v_empty[vs]);
                if (kt >= 0)
                    tensor_commit_elected(&sh.k_empty[ks]);
                if (n + 1 == list.n) {
                    if (kt2[0].any)
                        tensor_commit_elected(&sh.q_empty[0]);
                    if (kt2[1].any)
                        tensor_commit_elected(&sh.q_empty[1]);
                }
                vn += ended;
                kn += kt >= 0;
            }
            qn[0] += kt2[0].any;
            qn[1] += kt2[1].any;
        }
    } else {
        const int t = warp >> 2, quarter = warp & 3;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const uint32_t at_s = tmem + lanes + t * kScores, at_o = tmem + lanes + kSums + t * DP;
        uint4 *const stage = reinterpret_cast<uint4 *>(s_out + warp * 4096);
        const float sl = f.scale_log2;
        uint32_t sn = 0, on = 0, vn = 0;
        bool ok = true;
        Unit u;
        while (ok && next(u)) {
            const KeyTiles x = key_tiles<BN>(a, u.first, u.lq, u.lk), y = second(u);
            const KeyTiles mine = t ? y : x;
            const TileList list = tile_list(x, y);
            const int32_t row = u.first + 128 * t + quarter * 32 + lane, p = row + u.lk - u.lq;
            const int32_t p_first = u.first + 128 * t + u.lk - u.lq;
            const int32_t p_last = (u.first + 128 * t + 127 < u.lq ? u.first + 128 * t + 127 : u.lq - 1) + u.lk - u.lq;
            float m = -INFINITY, best = -INFINITY, l = 0.0f;
            for (int32_t n = 0; n < list.n; ++n) {
                const int32_t kt = list.at(n);
                if (!needs(mine, kt))
                    continue;
                const int buffer = BUFFERS == 2 ? sn & 1 : 0;
                ok = ok && wait(&sh.s_full[t + buffer], BUFFERS == 2 ? (sn >> 1) & 1 : sn & 1);
                ++sn;
                if (!ok)
                    break;
                tmem_fence_after();
                const int32_t k_first = kt * BN;
                const bool whole = k_first + BN - 1 <= p_first &&
                                   (k_first > p_last - a.window || k_first + BN - 1 < a.sinks);
                // 64 keys at a time, the later ones first: their largest score,
                // their weights, which go where their scores were, and on to
                // the products while the others are worked on.  (Unrolled, the
                // two halves' code took 805 us where this takes 790.)
#pragma unroll 1
                for (int h = S::HALVES - 1; h >= 0; --h) {
                    const int piece = BUFFERS == 2 ? buffer : h;
                    uint32_t r0[32], r1[32];
                    tmem_load32(at_s + 64 * piece, r0);
                    tmem_load32(at_s + 64 * piece + 32, r1);
                    tmem_wait_loads(r0);
                    tmem_wait_loads(r1);
                    if (!whole) {
                        const uint32_t b0 = seen_bits(p, a.window, a.sinks, k_first + 64 * h);
                        const uint32_t b1 = seen_bits(p, a.window, a.sinks, k_first + 64 * h + 32);
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            r0[e] = b0 & (1u << e) ? r0[e] : 0xff800000u;
                            r1[e] = b1 & (1u << e) ? r1[e] : 0xff800000u;
                        }
                    }
                    float tops[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        tops[e] = fmaxf(__uint_as_float(r0[e]), __uint_as_float(r1[e]));
#pragma unroll
                    for (int e = 8; e < 32; ++e)
                        tops[e & 7] = fmaxf(tops[e & 7], fmaxf(__uint_as_float(r0[e]), __uint_as_float(r1[e])));
                    const float top = fmaxf(fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])),
                                            fmaxf(fmaxf(tops[4], tops[5]), fmaxf(tops[6], tops[7])));
                    // The weights' reference is the largest score so far, or up
                    // to 2^8 below it: the weights stay below 2^(8 + kShift), and
                    // sums are rarely multiplied anew.
                    best = fmaxf(best, top);
                    const bool far = top > m && (m == -INFINITY || (top - m) * sl > 8.0f);
                    if (__any_sync(0xffffffffu, far)) {
                        const float to = far ? top : m;
                        const float keep = m == -INFINITY ? 0.0f : exp2_fast((m - to) * sl);
                        if (__any_sync(0xffffffffu, l != 0.0f)) {
                            // (of halves, what the products before this tile added is
                            // there, and of its later half when they say so; of
                            // buffers, the tile's before when they say so)
                            if (BUFFERS == 2 || h == 0) {
                                ok = wait(&sh.sum_done[t], BUFFERS == 2 ? sn & 1 : (sn - 1) & 1);
                                if (!ok)
                                    break;
                                tmem_fence_after();
                            }
                            for (int c = 0; c < a.dim; c += 16) {
                                uint32_t o[16];
                                tmem_load16(at_o + c, o);
                                tmem_wait_loads16(o);
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
                                tmem_store16(at_o + c, o);
                            }
                        }
                        l *= keep;
                        m = to;
                    }
                    // The difference first: s sl - m sl in one operation would be off
                    // by the rounding of m sl, 2^4 and more from 2^28 on, which
                    // a weight of 16 bits does not hold.  (16384 tokens of 64 + 8
                    // heads of 128: 790 us against 774; a branch to it for
                    // large scores alone: 825 to 860.)
                    const F2 scale2 = twice(sl), less2 = twice(m == -INFINITY ? 0.0f : -m);
                    F2 sums[4] = {};
                    auto weigh = [&](const uint32_t (&r)[32], int c) {
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const F2 s = F2{__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])} + less2;
                            const F2 x = exp2_fast(kShift<DT> == 0.0f ? s * scale2 : fma2(s, scale2, twice(kShift<DT>)));
                            sums[e & 3] = sums[e & 3] + x;
                            w[e] = pack2<DT>(x.x, x.y);
                        }
                        tmem_store16(at_s + 64 * piece + 16 * c, w);
                    };
                    weigh(r0, 0);
                    weigh(r1, 1);
                    if (k_first + BN > u.lk) {
                        // rows behind the last key: zeros, since 0 times what they hold may not be 0
                        const uint32_t now = vn + n, vs = now % S::STAGES;
                        ok = wait(&sh.v_full[vs], (now / S::STAGES) & 1);
                        if (!ok)
                            break;
                        const int32_t from = u.lk - k_first > 64 * h ? u.lk - k_first : 64 * h;
                        for (int i = from * 8 + (threadIdx.x & 127); i < (h + 1) * 512; i += 128)
#pragma unroll
                            for (int b = 0; b < S::BOXES; ++b)
                                *reinterpret_cast<uint4 *>(s_v + vs * S::K_TILE + b * BN * 128 + i * 16) = make_uint4(0, 0, 0, 0);
                        fence_proxy_async();
                    }
                    const F2 sum = (sums[0] + sums[1]) + (sums[2] + sums[3]);
                    l += sum.x + sum.y;
                    tmem_wait_stores();
                    tmem_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive_cluster(smem_addr(&sh.p_full[t][piece]));
                }
                if (!ok)
                    break;
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
                f.lse[(int64_t)u.head * a.q_tokens + out_row] = l == 0.0f ? -INFINITY : row_lse<DT>(best, m, l, a.scale);
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            const int32_t left = u.lq - u.first - 128 * t - quarter * 32;  // rows of this warp
            uint16_t *out = static_cast<uint16_t *>(const_cast<void *>(f.out.p)) +
                            ((int64_t)u.q_row + 128 * t + quarter * 32) * f.out.ld + u.head * f.out.hd;
#pragma unroll 1
            for (int c = 0; c < a.dim; c += 64) {
                uint32_t w[32];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t o[32];
                    if (mine.any && c + 32 * h < a.dim) {
                        tmem_load32(at_o + c + 32 * h, o);
                        tmem_wait_loads(o);
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        w[16 * h + e] = l == 0.0f ? 0u
                                                  : pack2<DT>(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
                }
                store_rows(stage, lane, w, out + c, f.out.ld, left, a.dim - c);
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
            const TileAt at = find_tile(a, a.q_offsets, a.q_tokens, f.tiles - 1 - i / a.q_heads, 128 * QT, false, lane);
            const int64_t head = i % a.q_heads;
            for (int32_t r = at.first + warp; at.any && r < at.s.lq && r < at.first + 128 * QT; r += S::THREADS / 32) {
                for (int e = lane; e < a.dim; e += 32)
                    static_cast<uint16_t *>(const_cast<void *>(f.out.p))[(at.s.q0 + r) * f.out.ld + head * f.out.hd + e] = 0x7fff;
                if (lane == 0 && f.lse)
                    f.lse[head * a.q_tokens + at.s.q0 + r] = __uint_as_float(0x7fffffffu);
            }
        }
    }
    if (warp == kMma)
        tmem_give(tmem, S::TMEM);
}

// ------------------------------------------------------------- a few queries

// Of a few queries per sequence the keys' and values' bytes are all there is,
// so every key head's are read once for all query heads of its group: 8 or 16
// rows (NG groups of 8) of `tokens` queries and the heads of a group meet a
// stretch of the keys in a block, 16 keys at a time per warp.  The products
// are mma.sync's 16 x 8 x 16, whose N of 8 fits these rows (a tcgen05 tile
// would be 128 rows of which 120 are empty), and keys and values go from
// memory to registers in the operands' layout, 16 bytes per lane, without
// shared memory between: S' = K Q^T has keys for rows, O' = V^T P' elements.
// A set of rows is split over its keys among blocks; each leaves sums, a
// reference and the weights' sum, and the last to come joins them in order.
//
// What bounds it: the keys' and values' bytes.  64 requests of up to 8192 keys
// of 8 heads of 128 (0.92 GB): 166 us, 5.5 TB/s; 64 of 4096: 181, 5.9; 64 of
// 4096 keys of 25 heads of 64 (1.68 GB): 281, 6.0.  Alone a request is a few
// trips to memory: 7.5 us over 256 keys of 25 heads of 64, 11 over 4096.  Groups
// of 8 heads' rows one at a time (NG = 1 throughout) read keys twice through
// L2: 64 requests of 64 + 4 heads 165 us against 154.
struct FewArgs {
    Attn a;
    Heads q, k, v, out;
    float *lse;
    int64_t tiles;               // tile numbers of `tokens` queries
    int32_t tokens, parts, splits;  // parts: sets of rows of one query's heads
    float scale_log2;
    uint32_t *tickets;           // one per set of rows, where splits > 1
    float *partial;              // [set of rows][split]: [row][dim] sums, [row] references, [row] the weights' sums
};

constexpr int kFewWarps = 4;
constexpr int kMostTickets = 2048, kMostSplits = 64;

// Read once: not kept in L1.
__device__ __forceinline__ uint4 load_once(const uint4 *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1, bool bf16)
{
    if (bf16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Lane 4 i + j's pair (row i, columns 2 j and 2 j + 1 of 8 x 8) becomes
// (row 2 j and 2 j + 1, column i).
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <int DT, int DP, int NG>
__global__ void __launch_bounds__(kFewWarps * 32) k_attn_few(const __grid_constant__ FewArgs f)
{
    constexpr int R = 8 * NG, KK = DP / 32, JJ = DP / 64;
    constexpr bool kBf16 = DT == ZERO_BF16;
    __shared__ __align__(16) float s_o[kFewWarps][R][DP];
    __shared__ float s_m[kFewWarps][R], s_l[kFewWarps][R];
    __shared__ uint4 s_q[NG][KK][32];  // the queries, as the lanes' operands
    __shared__ uint32_t s_last;
    const Attn &a = f.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int32_t split = blockIdx.x % f.splits;
    const int64_t set = blockIdx.x / f.splits;
    const int32_t part = (int32_t)(set % f.parts), kh = (int32_t)(set / f.parts % a.k_heads);
    const TileAt at = find_tile(a, a.q_offsets, a.q_tokens, set / f.parts / a.k_heads, f.tokens, false, lane);
    if (!at.any)
        return;
    // rows: the group's heads of each query in turn
    const int32_t queries = at.s.lq - at.first < f.tokens ? at.s.lq - at.first : f.tokens;
    const int32_t row0 = part * R, rows = queries * a.group - row0 < R ? queries * a.group - row0 : R;
    const int32_t p0 = at.first + at.s.lk - at.s.lq, p1 = p0 + queries - 1;  // where the queries stand
    // the keys that any of them sees, in a row: first keys, then the window's
    const int32_t low = p0 >= a.window ? p0 - a.window + 1 : 0;
    const int32_t sinks = p1 < 0 ? 0 : a.sinks < low ? a.sinks : low;
    const int32_t n = p1 < 0 ? 0 : sinks + p1 - low + 1;
    const int32_t per = ((n + f.splits - 1) / f.splits + 63) / 64 * 64;
    const int32_t x0 = split * (int64_t)per < n ? split * per : n, x1 = n - x0 < per ? n : x0 + per;
    const int32_t used = n > 0 ? (n + per - 1) / per : 1;  // blocks with keys (the first writes where there are none)

    if (split < used) {
        uint4 k[2][KK], v[4][JJ];
        int32_t p[NG][2];
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            const int32_t r = row0 + 8 * i + g;  // of queries and heads
            const bool live = 8 * i + g < rows;
            const uint16_t *from = static_cast<const uint16_t *>(f.q.p) + (at.s.q0 + at.first + (live ? r / a.group : 0)) * f.q.ld +
                                   (kh * a.group + (live ? r % a.group : 0)) * f.q.hd;
            for (int e = warp; e < KK; e += kFewWarps)
                s_q[i][e][lane] = live && (c + 4 * e) * 8 < a.dim ? __ldg(reinterpret_cast<const uint4 *>(from) + c + 4 * e) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int e = 0; e < 2; ++e)
                p[i][e] = p0 + (row0 + 8 * i + 2 * c + e) / a.group;
        }
        const uint16_t *const kp = static_cast<const uint16_t *>(f.k.p) + kh * f.k.hd;
        const uint16_t *const vp = static_cast<const uint16_t *>(f.v.p) + kh * f.v.hd;
        auto key = [&](int32_t x) { return at.s.k0 + (x < sinks ? x : low + x - sinks); };
        auto load_k = [&](int32_t x) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bool in = x + 8 * h + g < x1;
                const uint4 *from = reinterpret_cast<const uint4 *>(kp + (in ? key(x + 8 * h + g) : 0) * f.k.ld);
#pragma unroll
                for (int e = 0; e < KK; ++e)
                    k[h][e] = in && (c + 4 * e) * 8 < a.dim ? load_once(from + c + 4 * e) : make_uint4(0, 0, 0, 0);
            }
        };
        auto load_v = [&](int32_t x) {
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const int32_t at_x = x + 2 * c + (h & 1) + (h >> 1) * 8;
                const bool in = at_x < x1;
                const uint4 *from = reinterpret_cast<const uint4 *>(vp + (in ? key(at_x) : 0) * f.v.ld);
#pragma unroll
                for (int e = 0; e < JJ; ++e)
                    v[h][e] = in && (g + 8 * e) * 8 < a.dim ? load_once(from + g + 8 * e) : make_uint4(0, 0, 0, 0);
            }
        };
        auto word = [](const uint4 &x, int e) { return e == 0 ? x.x : e == 1 ? x.y : e == 2 ? x.z : x.w; };
        float o[NG][JJ * 4][4] = {}, m[NG][2], best[NG][2], l[NG][2] = {};
#pragma unroll
        for (int i = 0; i < NG; ++i)
            m[i][0] = m[i][1] = best[i][0] = best[i][1] = -INFINITY;
        const bool many = queries > 1;
        int32_t x = x0 + warp * 16;
        if (x < x1) {
            load_k(x);
            load_v(x);
        }
        __syncthreads();
        for (; x < x1; x += 16 * kFewWarps) {
            float t[NG][4] = {};
#pragma unroll
            for (int e = 0; e < KK; ++e)
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    const uint4 q = s_q[i][e][lane];
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        mma16(t[i], word(k[0][e], 2 * h), word(k[1][e], 2 * h), word(k[0][e], 2 * h + 1),
                              word(k[1][e], 2 * h + 1), word(q, 2 * h), word(q, 2 * h + 1), kBf16);
                }
            const int32_t x_next = x + 16 * kFewWarps;
            if (x_next < x1)
                load_k(x_next);
            bool far = false;
            float top[NG][2];
#pragma unroll
            for (int i = 0; i < NG; ++i) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int32_t at_x = x + 8 * h + g, j = at_x < sinks ? at_x : low + at_x - sinks;
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (at_x >= x1 || (many && (j > p[i][e] || (j <= p[i][e] - a.window && j >= a.sinks))))
                            t[i][2 * h + e] = -INFINITY;
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    top[i][e] = fmaxf(t[i][e], t[i][2 + e]);
                    best[i][e] = fmaxf(best[i][e], top[i][e]);
                    far = far || (top[i][e] > m[i][e] && (m[i][e] == -INFINITY || (top[i][e] - m[i][e]) * f.scale_log2 > 8.0f));
                }
            }
            // the reference of a row's weights follows its largest score from up to 2^8 below
            if (__any_sync(0xffffffffu, far)) {
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    float keep[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float to = fmaxf(top[i][e], m[i][e]);
#pragma unroll
                        for (int b = 4; b < 32; b *= 2)
                            to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, b));
                        keep[e] = m[i][e] == -INFINITY ? 0.0f : exp2_fast((m[i][e] - to) * f.scale_log2);
                        m[i][e] = to;
                        l[i][e] *= keep[e];
                    }
#pragma unroll
                    for (int b = 0; b < JJ * 4; ++b)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[i][b][e] *= keep[e & 1];
                }
            }
            uint32_t w[NG][2];
#pragma unroll
            for (int i = 0; i < NG; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float m0 = m[i][0] == -INFINITY ? 0.0f : m[i][0], m1 = m[i][1] == -INFINITY ? 0.0f : m[i][1];
                    const float w0 = exp2_fast(fmaf(t[i][2 * h] - m0, f.scale_log2, kShift<DT>));
                    const float w1 = exp2_fast(fmaf(t[i][2 * h + 1] - m1, f.scale_log2, kShift<DT>));
                    l[i][0] += w0;
                    l[i][1] += w1;
                    w[i][h] = transpose8(pack2<DT>(w0, w1));
                }
#pragma unroll
            for (int e = 0; e < JJ; ++e)
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const uint32_t v0 = word(v[0][e], b), v1 = word(v[1][e], b), v2 = word(v[2][e], b), v3 = word(v[3][e], b);
                    const uint32_t a0 = __byte_perm(v0, v1, 0x5410), a1 = __byte_perm(v0, v1, 0x7632);
                    const uint32_t a2 = __byte_perm(v2, v3, 0x5410), a3 = __byte_perm(v2, v3, 0x7632);
#pragma unroll
                    for (int i = 0; i < NG; ++i)
                        mma16(o[i][e * 4 + b], a0, a1, a2, a3, w[i][0], w[i][1], kBf16);
                }
            if (x_next < x1)
                load_v(x_next);
        }
        // the warps' sums, each with its largest score for a reference in the end
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            float keep[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int b = 4; b < 32; b *= 2) {
                    best[i][e] = fmaxf(best[i][e], __shfl_xor_sync(0xffffffffu, best[i][e], b));
                    l[i][e] += __shfl_xor_sync(0xffffffffu, l[i][e], b);
                }
                keep[e] = m[i][e] == best[i][e] ? 1.0f : exp2_fast((m[i][e] - best[i][e]) * f.scale_log2);
                if (g == 0) {
                    s_m[warp][8 * i + 2 * c + e] = best[i][e];
                    s_l[warp][8 * i + 2 * c + e] = l[i][e] * keep[e];
                }
            }
#pragma unroll
            for (int e = 0; e < JJ; ++e)
#pragma unroll
                for (int b = 0; b < 4; ++b)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        *reinterpret_cast<float2 *>(&s_o[warp][8 * i + 2 * c + h][64 * e + 8 * g + 2 * b]) =
                            make_float2(o[i][e * 4 + b][h] * keep[h], o[i][e * 4 + b][2 + h] * keep[h]);
        }
    }
    __syncthreads();

    // four elements of a row are finished at a time
    auto finish = [&](int32_t r, int32_t e, float4 sum, float m, float l) {
        const int32_t rr = row0 + r;
        const int64_t row = at.s.q0 + at.first + rr / a.group;
        const int32_t head = kh * a.group + rr % a.group;
        uint2 w = make_uint2(0, 0);
        if (l != 0.0f)
            w = make_uint2(pack2<DT>(sum.x / l, sum.y / l), pack2<DT>(sum.z / l, sum.w / l));
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(const_cast<void *>(f.out.p)) + row * f.out.ld + head * f.out.hd + e) = w;
        if (e == 0 && f.lse)
            f.lse[(int64_t)head * a.q_tokens + row] = l == 0.0f ? -INFINITY : row_lse<DT>(m, m, l, a.scale);
    };
    auto add = [](float4 &sum, float4 x, float by) {
        sum.x += x.x * by, sum.y += x.y * by, sum.z += x.z * by, sum.w += x.w * by;
    };
    const int32_t fours = a.dim / 4, part_floats = R * (a.dim + 2);  // of a block: its sums, references and weights' sums
    float *const mine = f.partial + (set * f.splits + split) * part_floats;
    if (split < used)
        for (int32_t i = threadIdx.x; i < rows * fours; i += kFewWarps * 32) {
            const int32_t r = i / fours, e = 4 * (i - r * fours);
            float m = s_m[0][r], l = 0.0f;
            float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int w = 1; w < kFewWarps; ++w)
                m = fmaxf(m, s_m[w][r]);
#pragma unroll
            for (int w = 0; w < kFewWarps; ++w) {
                const float by = s_m[w][r] == -INFINITY ? 0.0f : exp2_fast((s_m[w][r] - m) * f.scale_log2);
                if (s_m[w][r] != -INFINITY || s_l[w][r] != 0.0f) {
                    add(sum, *reinterpret_cast<const float4 *>(&s_o[w][r][e]), by);
                    l += s_l[w][r] * by;
                }
            }
            if (used == 1) {
                finish(r, e, sum, m, l);
            } else {
                *reinterpret_cast<float4 *>(mine + r * a.dim + e) = sum;
                if (e == 0) {
                    mine[R * a.dim + r] = m;
                    mine[R * a.dim + R + r] = l;
                }
            }
        }
    if (used == 1)
        return;
    // the block that comes last joins all of a set's, in order
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0)
        s_last = atomicAdd(&f.tickets[set], 1u) == (uint32_t)f.splits - 1;
    __syncthreads();
    if (!s_last)
        return;
    __threadfence();
    const float *const all = f.partial + set * f.splits * part_floats;
    // what each block's sums are multiplied by, a block to a lane
    float (*const s_by)[kMostSplits] = reinterpret_cast<float (*)[kMostSplits]>(&s_o[0][0][0]);
    static_assert(kMostSplits == 64 && sizeof(s_o) >= R * kMostSplits * 4, "two blocks to a lane, in the sums' place");
    for (int32_t r = warp; r < rows; r += kFewWarps) {
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (lane + 32 * h < used) {
                const float *const from = all + (lane + 32 * h) * part_floats + R * a.dim + r;
                m[h] = __ldcg(from);
                l[h] = __ldcg(from + R);
            }
        float top = fmaxf(m[0], m[1]), sum = 0.0f;
#pragma unroll
        for (int b = 16; b > 0; b >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, b));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float by = m[h] == -INFINITY ? 0.0f : exp2_fast((m[h] - top) * f.scale_log2);
            s_by[r][lane + 32 * h] = by;
            sum += l[h] * by;
        }
#pragma unroll
        for (int b = 16; b > 0; b >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, b);
        if (lane == 0)
            s_m[0][r] = top, s_l[0][r] = sum;
    }
    __syncthreads();
    for (int32_t i = threadIdx.x; i < rows * fours; i += kFewWarps * 32) {
        const int32_t r = i / fours, e = 4 * (i - r * fours);
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const float *const from = all + r * a.dim + e;
#pragma unroll 8
        for (int32_t w = 0; w < used; ++w)
            add(sum, __ldcg(reinterpret_cast<const float4 *>(from + w * part_floats)), s_by[r][w]);
        finish(r, e, sum, s_m[0][r], s_l[0][r]);
    }
    if (threadIdx.x == 0)
        f.tickets[set] = 0;
}

// ------------------------------------------------------------- backward

// What every pair of a query and a key takes from the query's row: lse (+inf
// where no key is seen, which makes every weight 0) and delta = dout . out.
// Laid out by tile of 128 queries, so that a tile's are one aligned copy:
// [head][tile number][lse of 128, delta of 128].
//
// f16 holds neither the weights of many keys (a 16384th and less) nor dS of
// small gradients or of a scaled loss, so there the backward pass rounds
// powers of two times them, which leave the sums at the end.  For P it is
// 2^kShiftP (P is at most 1); for dS the largest that keeps it below 2^15
// whatever the products give:
//     |dS_ij| <= |dout_i| sqrt(d) max |v_j| + |delta_i|    (P is at most 1),
// for the dk of a key by its own value and the largest of its tile's queries,
// for a query's dq by its own row and the values of the tiles of keys that it
// may see.  (What is below 2^-29 of that bound is rounded in steps of 2^-39 of
// it.  Unscaled, dq of normal inputs over 4096 keys and gradients of
// 10^-4 was off by a tenth, and one of 10^5 was inf.)  5340 tokens of 25 heads
// of 64: 117.5 us, 108.3 without: the units' largest rows and values, and
// dS' times its power of two.
struct Sizes {
    float *rows;    // sqrt(d) |dout|: [head][tile number][128]
    float2 *tops;   // of 32 rows, the largest of these and of |delta|: [head][tile number][4]
    float *values;  // largest elements of 32 rows of v, from k_attn_dkv: [key head][tile number of the keys][4]
};

struct StatsArgs {
    Attn a;
    Heads dout, out;
    const float *lse;
    float *stats;
    Sizes sizes;
    int64_t tiles;
};

template <int DT>
constexpr bool kScaled = DT == ZERO_F16;
template <int DT>
constexpr float kShiftP = kScaled<DT> ? 15.0f : 0.0f;

__device__ __forceinline__ float power_of_two(int32_t c) { return __uint_as_float((uint32_t)(c + 127) << 23); }

// c with bound 2^c below 2^15 and not below 2^14 (100 of nothing; as low as
// -100 of what is no number, which reaches what it is in all the same).
__device__ __forceinline__ int32_t dS_exponent(float bound)
{
    const int32_t c = 14 + 127 - (int32_t)(__float_as_uint(bound) >> 23);
    return c < -100 ? -100 : c > 100 ? 100 : c;
}

// Of values that are at least 0, whose bits are in their order.
__device__ __forceinline__ float warp_max(float x)
{
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x)));
}

// Sums over the L lanes of a row, of L rows at once: lane i of them gets that
// of row i, after L - 1 exchanges.
template <int L>
__device__ __forceinline__ float row_sums(float (&x)[L], int at)
{
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const bool upper = at & o;
            const float give = upper ? x[i] : x[i + o], keep = upper ? x[i + o] : x[i];
            x[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    return x[0];
}

// A warp takes 32 queries of a tile and the heads of its block: lse by one
// lane per query, dout and out by 2 to 16 lanes to a row.  Bound by the two
// arrays' bytes: 5340 tokens of 25 heads of 64, 34 MB: 11 us from HBM.
template <int DT, int L>
__global__ void __launch_bounds__(128) k_attn_stats(const __grid_constant__ StatsArgs f)
{
    constexpr int kRows = 32 / L;
    const Attn &a = f.a;
    const int part = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / L, at = lane & (L - 1);
    const bool in = at * 8 < a.dim;
    pdl_launch_next();
    for (int64_t number = blockIdx.x; number < f.tiles; number += gridDim.x) {
        const TileAt t = find_tile(a, a.q_offsets, a.q_tokens, number, 128, false, lane);
        const int32_t first = t.first + 32 * part, left = t.s.lq - first;  // of this warp
        if (!t.any)
            continue;
        const uint16_t *const x0 = static_cast<const uint16_t *>(f.dout.p) + (t.s.q0 + first + sub) * f.dout.ld + at * 8;
        const uint16_t *const y0 = static_cast<const uint16_t *>(f.out.p) + (t.s.q0 + first + sub) * f.out.ld + at * 8;
        for (int32_t h = blockIdx.y; h < a.q_heads; h += gridDim.y) {
            const float lse = lane < left ? f.lse[(int64_t)h * a.q_tokens + t.s.q0 + first + lane] : -INFINITY;
            const uint16_t *const xh = x0 + h * f.dout.hd, *const yh = y0 + h * f.out.hd;
            float sums[L], squares[L];
#pragma unroll
            for (int i = 0; i < L; ++i) {
                sums[i] = squares[i] = 0.0f;
                if (in && kRows * i + sub < left) {
                    const uint4 x = __ldg(reinterpret_cast<const uint4 *>(xh + (int64_t)kRows * i * f.dout.ld));
                    const uint4 y = __ldg(reinterpret_cast<const uint4 *>(yh + (int64_t)kRows * i * f.out.ld));
                    float fx[8], fy[8];
                    Elem<DT>::to_float(&x, fx);
                    Elem<DT>::to_float(&y, fy);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        sums[i] += fx[e] * fy[e];
                        if (kScaled<DT>)
                            squares[i] += fx[e] * fx[e];
                    }
                }
            }
            // lane L s + i has row kRows i + s: query `lane` gets its own
            const int from = (lane & (kRows - 1)) * L + lane / kRows;
            const float delta = __shfl_sync(0xffffffffu, row_sums<L>(sums, at), from);
            float *const to = f.stats + (h * f.tiles + number) * 256 + 32 * part + lane;
            to[0] = lse == -INFINITY ? INFINITY : lse;
            to[128] = delta;
            if (kScaled<DT>) {
                const float size = sqrtf(__shfl_sync(0xffffffffu, row_sums<L>(squares, at), from) * a.dim);
                f.sizes.rows[(h * f.tiles + number) * 128 + 32 * part + lane] = size;
                const float2 tops = make_float2(warp_max(size), warp_max(fabsf(delta)));
                if (lane == 0)
                    f.sizes.tops[(h * f.tiles + number) * 4 + part] = tops;
            }
        }
    }
}

// P of two pairs: exp(s scale - lse), with s scale rounded as the forward
// pass rounds it for lse, so that a key that takes all has a weight of 1
// whatever its score.  (One operation, with scale and lse in units of log 2,
// is off by their roundings: 2^-23 of the score, so by factors from 10^7 on.
// 16384 tokens of 64 + 8 heads of 128 took 2745 us with it and take 2777 with
// three; 5340 of 25 heads of 64 103 and 106.7.)  zero2: see BwdTiles.  Times
// 2^shift.
__device__ __forceinline__ F2 weights(F2 s, F2 scale2, F2 zero2, F2 less_lse, F2 shift2)
{
    return exp2_fast(fma2(fma2(s, scale2, zero2) + less_lse, twice(1.4426950408889634f), shift2));
}

struct BwdTiles {
    HeadsMap q, k, v, dout;
    Attn a;
    Heads dq, dk, dv, v_rows;
    const float *stats;
    Sizes sizes;
    int64_t q_tiles, k_tiles;  // tile numbers of 128 queries, and keys
    // first keys seen by all queries: their tiles' queries in parts of `chunk` tiles
    int32_t chunk, sink_tiles;
    int64_t split_units;
    float *partial;  // [split unit][dv, dk][128][dim]
    float scale;
    float zero;  // 0, but not so that the compiler could tell: added to a product that is to be rounded by itself
    WsHeader *hdr;
    uint64_t limit_ns;
};

// The tiles of T queries that see a key of the tile of 128 from key j on.
struct QueryTiles {
    int32_t low, high;
};

template <int T>
__device__ __forceinline__ QueryTiles query_tiles(const Attn &a, int32_t j, int32_t lq, int32_t lk)
{
    const int32_t shift = lk - lq, last = j + 127 < lk ? j + 127 : lk - 1;
    const int32_t from = j > shift ? j - shift : 0;
    int32_t to = lq - 1;
    if (j >= a.sinks && last - shift + (int64_t)a.window - 1 < to)
        to = last - shift + a.window - 1;
    if (lq == 0 || from > to)
        return {0, -1};
    return {from / T, to / T};
}

// Whether those (of 128) of a tile of first keys are dealt out.
__device__ __forceinline__ bool is_split(const BwdTiles &f, int32_t j, const QueryTiles &t)
{
    return f.chunk > 0 && j < f.a.sinks && t.high - t.low + 1 > 2 * f.chunk;
}

// The n-th unit of a CTA.  Of one sequence units come from the longest down,
// and every other round of them is dealt out from the other end, so that what
// the CTAs get adds up to about the same: 8192 tokens of 16 heads of 64,
// without a window, bf16, 515 us from one end (dq's kernel waits for the last
// CTA of dk's and dv's), 431 so.
__device__ __forceinline__ int64_t nth_unit(int64_t n)
{
    return n * gridDim.x + (n & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

struct KeyUnit {
    int32_t k_row, q_row, first, lq, lk, head;  // first key of its sequence; q_row: the sequence's first query
    int32_t low, high;                          // query tiles
    int64_t stats, keys;                        // tile numbers of query tile 0, of key tile 0
    float row, delta;                           // largest of the queries' (f16)
    int64_t slot;                               // of the partial sums, or -1
    int32_t end;

    __device__ __forceinline__ void agree()
    {
        first = uniform(first), lq = uniform(lq), lk = uniform(lk), head = uniform(head);
        low = uniform(low), high = uniform(high), end = uniform(end);
    }
};

// Tiles of 128 keys (queries) against tiles of BN queries (keys), which a
// group of four warps holds a row of 64 columns per thread of.
template <int DP_, int BN_, int PER_SM_>
struct BwdShape {
    static constexpr int DP = DP_, BN = BN_, PER_SM = PER_SM_;
    static constexpr int BOXES = DP / 64, TILE = BOXES * 16384, MOVING = BOXES * BN * 128;  // bytes
    static constexpr int ROW_WARPS = BN / 16, THREADS = (ROW_WARPS + 2) * 32;
    static constexpr int STAGES = BN == 64 ? 4 : 2;  // of each of the two that move
    static constexpr int SMEM = 1024 + 2 * TILE + STAGES * (2 * MOVING + 2 * BN * 4) + ROW_WARPS * 2048;
    static constexpr int TMEM = 2 * BN + 2 * DP;  // (dq: three of BN and one of DP)
    static_assert(SMEM * PER_SM <= 227 * 1024 && TMEM * PER_SM <= 512 && 3 * BN + DP <= TMEM, "what an SM has");
};

struct KeyShared {
    uint64_t kv_full, kv_empty, q_full[4], q_empty[4], o_full[4], o_empty[4], s_full, dp_full, p_full[2], ds_full[2], acc_full;
    uint64_t unit_full[kUnitRing], unit_empty[kUnitRing];
    KeyUnit units[kUnitRing];
    uint32_t tmem, gave_up;
};

// The work of a unit number, its queries in tiles of T: false if there is none.
template <int T>
__device__ __forceinline__ bool key_unit(const BwdTiles &f, int64_t i, int lane, KeyUnit &u)
{
    const Attn &a = f.a;
    const int64_t *k_offsets = a.k_offsets ? a.k_offsets : a.q_offsets;
    TileAt at;
    u.end = 0;
    if (i < f.split_units) {
        const int64_t chunk = i / a.k_heads / f.sink_tiles;
        at = find_tile(a, a.q_offsets, a.q_tokens, chunk, 128 * f.chunk, false, lane);
        u.head = (int32_t)(i % a.k_heads);
        u.first = (int32_t)(i / a.k_heads % f.sink_tiles) * 128;
        if (!at.any || u.first >= at.s.lk || u.first >= a.sinks)
            return false;
        if (!is_split(f, u.first, query_tiles<128>(a, u.first, at.s.lq, at.s.lk)))
            return false;
        const QueryTiles t = query_tiles<T>(a, u.first, at.s.lq, at.s.lk);
        const int32_t low = at.first / T, high = low + f.chunk * (128 / T) - 1;
        u.low = low > t.low ? low : t.low;
        u.high = high < t.high ? high : t.high;
        if (u.low > u.high)
            return false;
        u.slot = i;
    } else {
        i -= f.split_units;
        at = find_tile(a, k_offsets, a.k_tokens, i / a.k_heads, 128, true, lane);
        if (!at.any)
            return false;
        u.head = (int32_t)(i % a.k_heads);
        u.first = at.first;
        if (is_split(f, u.first, query_tiles<128>(a, u.first, at.s.lq, at.s.lk)))
            return false;
        const QueryTiles t = query_tiles<T>(a, u.first, at.s.lq, at.s.lk);
        u.low = t.low, u.high = t.high;
        u.slot = -1;
    }
    u.k_row = (int32_t)at.s.k0 + u.first;
    u.q_row = (int32_t)at.s.q0;
    u.lq = at.s.lq, u.lk = at.s.lk;
    u.stats = a.q_offsets ? at.s.q0 / 128 + at.index : 0;
    u.keys = k_offsets ? at.s.k0 / 128 + at.index : 0;
    u.row = u.delta = 0.0f;
    return true;
}

// The largest row and delta of a unit's queries, by a whole warp, a share to
// each lane: an entry for every 32 queries and head (they fit 31 bits: there
// is memory for them), 32 at a time.
template <int T>
__device__ __forceinline__ float2 unit_tops(const BwdTiles &f, const KeyUnit &u, int lane)
{
    const int32_t n = (u.high - u.low + 1) * (T / 32), all = n * f.a.group;
    const float2 *const from = f.sizes.tops + ((int64_t)u.head * f.a.group * f.q_tiles + u.stats) * 4 + u.low * (T / 32);
    float2 top = make_float2(0.0f, 0.0f);
#pragma unroll 4
    for (int32_t i = lane; i < all; i += 32) {
        const int32_t h = i / n;
        const float2 x = from[h * f.q_tiles * 4 + i - h * n];
        top.x = fmaxf(top.x, x.x), top.y = fmaxf(top.y, x.y);
    }
    return top;
}

// The largest element of a row of f16 in shared memory: 128 bytes in each of
// BOXES boxes, in whatever order the swizzle left them.
template <int BOXES>
__device__ __forceinline__ float largest_of_row(const unsigned char *tile, int row)
{
    __half2 top = __half2half2(__ushort_as_half(0));
#pragma unroll
    for (int k = 0; k < 8 * BOXES; ++k) {
        const uint4 x = *reinterpret_cast<const uint4 *>(tile + (k >> 3) * 16384 + row * 128 + ((k ^ row) & 7) * 16);
        const __half2 *h = reinterpret_cast<const __half2 *>(&x);
        top = __hmax2(__hmax2(__hmax2(top, __habs2(h[0])), __habs2(h[1])), __hmax2(__habs2(h[2]), __habs2(h[3])));
    }
    return fmaxf(__low2float(top), __high2float(top));
}

// dk and dv of 128 keys of one key head at a time, over the query heads of
// its group and the tiles of queries that see them.  Everything is the
// transpose of the forward pass's, so that the weights and their gradients,
// which the two running products take from tensor memory, have a key per lane:
//     S' = K Q^T, P' = exp(S' - lse), dP' = V dO^T, dS' = P' (dP' - delta),
//     dV += P' dO, dK += dS' Q.
// P' and dS' are rounded to 16 bits once, as the products' operands; P' goes on
// into dS' unrounded.  Rows of statistics come with the queries' tiles, so a
// tile needs no reduction and no running maximum.
//
// What bounds it: four products, 2048 clocks of the tensor pipe for 128 x 128
// pairs at 128 elements, and a chain of products and elementwise work that one
// pair of buffers in tensor memory (two tiles of scores and two sums of
// 128 x 128 are all of its 512 columns) lets overlap only by halves: 16384
// tokens of 64 + 8 heads of 128, window 2048: about 1.27 of the pass's 2.75 ms.
// Heads of 64: tiles of 64 queries, two CTAs per SM.
template <int DT, class S>
__global__ void __launch_bounds__(S::THREADS, S::PER_SM) k_attn_dkv(const __grid_constant__ BwdTiles f)
{
    constexpr int DP = S::DP, BN = S::BN;
    extern __shared__ unsigned char smem_raw[];
    __shared__ KeyShared sh;
    unsigned char *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023u)) & 1023u);
    unsigned char *const s_k = smem, *const s_v = smem + S::TILE, *const s_q = s_v + S::TILE, *const s_o = s_q + S::STAGES * S::MOVING;
    float *const s_stats = reinterpret_cast<float *>(s_o + S::STAGES * S::MOVING);  // [stage][lse, delta][BN]
    unsigned char *const s_out = reinterpret_cast<unsigned char *>(s_stats + S::STAGES * 2 * BN);
    const Attn &a = f.a;
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    constexpr int kTma = S::ROW_WARPS, kMma = S::ROW_WARPS + 1;
    constexpr int kDp = BN, kDv = 2 * BN, kDk = 2 * BN + DP;  // columns of tensor memory

    if (threadIdx.x == 0) {
        mbar_init_count(&sh.kv_full, 1);
        mbar_init_count(&sh.kv_empty, 1);
        for (int s = 0; s < S::STAGES; ++s) {
            mbar_init_count(&sh.q_full[s], 1);
            mbar_init_count(&sh.q_empty[s], 1);
            mbar_init_count(&sh.o_full[s], 1);
            mbar_init_count(&sh.o_empty[s], 1);
        }
        mbar_init_count(&sh.s_full, 1);
        mbar_init_count(&sh.dp_full, 1);
        for (int c = 0; c < BN / 64; ++c) {
            mbar_init_count(&sh.p_full[c], S::ROW_WARPS);
            mbar_init_count(&sh.ds_full[c], S::ROW_WARPS);
        }
        mbar_init_count(&sh.acc_full, 1);
        for (int s = 0; s < kUnitRing; ++s) {
            mbar_init_count(&sh.unit_full[s], 1);
            mbar_init_count(&sh.unit_empty[s], S::ROW_WARPS + 1);
        }
        sh.gave_up = 0;
        mbar_init_done();
    }
    if (warp == kMma)
        tmem_take(&sh.tmem, S::TMEM);
    if (warp == kTma && lane < 4)
        tma_prefetch_map(lane == 0 ? &f.q.map : lane == 1 ? &f.k.map : lane == 2 ? &f.v.map : &f.dout.map);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = (uint32_t)uniform((int32_t)sh.tmem);
    pdl_wait();
    pdl_launch_next();
    auto wait = [&](uint64_t *bar, uint32_t parity) { return mbar_wait_warp(bar, parity, f.limit_ns, &sh.gave_up); };
    uint32_t units = 0;
    auto next = [&](KeyUnit &u) {
        const uint32_t slot = units % kUnitRing;
        if (!wait(&sh.unit_full[slot], (units / kUnitRing) & 1))
            return false;
        u = sh.units[slot];
        u.agree();
        __syncwarp();
        if (lane == 0)
            mbar_arrive_cluster(smem_addr(&sh.unit_empty[slot]));
        ++units;
        return u.end == 0;
    };
    const int64_t all = f.split_units + f.k_tiles * a.k_heads;

    if (warp == kTma) {
        asm volatile("fence.proxy.async.global;" ::: "memory");
        uint32_t kvn = 0, qn = 0;
        bool ok = true;
        auto publish = [&](const KeyUnit &u) {
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
        auto load = [&](unsigned char *to, const HeadsMap &m, int32_t row, int32_t head, int box, uint64_t *bar) {
#pragma unroll
            for (int x = 0; x < S::BOXES; ++x)
                load_box(smem_addr(to) + x * box, m, 64 * x, row, head, smem_addr(bar));
        };
        for (int64_t round = 0; ok && round * gridDim.x < all; ++round) {
            const int64_t i = nth_unit(round);
            if (i >= all)
                continue;
            KeyUnit u;
            if (!key_unit<BN>(f, i, lane, u))
                continue;
            if (u.low > u.high) {
                ok = publish(u);
                continue;
            }
            if (kScaled<DT>) {
                const float2 tops = unit_tops<BN>(f, u, lane);
                u.row = warp_max(tops.x), u.delta = warp_max(tops.y);
            }
            ok = publish(u) && wait(&sh.kv_empty, (kvn & 1) ^ 1);
            if (!ok)
                break;
            if (elect_one()) {
                mbar_expect(&sh.kv_full, 2 * S::TILE);
                load(s_k, f.k, u.k_row, u.head, 16384, &sh.kv_full);
                load(s_v, f.v, u.k_row, u.head, 16384, &sh.kv_full);
            }
            __syncwarp();
            ++kvn;
            for (int32_t h = u.head * a.group; ok && h < (u.head + 1) * a.group; ++h)
                for (int32_t t = u.low; t <= u.high; ++t) {
                    const uint32_t st = qn % S::STAGES, parity = ((qn / S::STAGES) & 1) ^ 1;
                    ok = wait(&sh.q_empty[st], parity);
                    if (!ok)
                        break;
                    if (elect_one()) {
                        mbar_expect(&sh.q_full[st], S::MOVING + 8 * BN);
                        load(s_q + st * S::MOVING, f.q, u.q_row + BN * t, h, BN * 128, &sh.q_full[st]);
                        const float *const from = f.stats + (h * f.q_tiles + u.stats + BN * t / 128) * 256 + BN * t % 128;
                        bulk_copy(smem_addr(s_stats + st * 2 * BN), from, 4 * BN, smem_addr(&sh.q_full[st]));
                        bulk_copy(smem_addr(s_stats + st * 2 * BN + BN), from + 128, 4 * BN, smem_addr(&sh.q_full[st]));
                    }
                    __syncwarp();
                    ok = wait(&sh.o_empty[st], parity);
                    if (!ok)
                        break;
                    if (elect_one()) {
                        mbar_expect(&sh.o_full[st], S::MOVING);
                        load(s_o + st * S::MOVING, f.dout, u.q_row + BN * t, h, BN * 128, &sh.o_full[st]);
                    }
                    __syncwarp();
                    ++qn;
                }
        }
        if (ok) {
            KeyUnit u{};
            u.end = 1;
            publish(u);
        }
    } else if (warp == kMma) {
        constexpr bool kBf16 = DT == ZERO_BF16;
        const uint32_t desc_s = product_desc(kBf16, false, false, 128, BN);
        const int wide = (a.dim + 15) & ~15, steps = wide / 16;
        const uint32_t desc_acc = product_desc(kBf16, false, true, 128, wide);
        const uint64_t dk0 = operand_desc(smem_addr(s_k), 16, 1024), dv0 = operand_desc(smem_addr(s_v), 16, 1024);
        const uint64_t dq0 = operand_desc(smem_addr(s_q), 16, 1024), do0 = operand_desc(smem_addr(s_o), 16, 1024);
        const uint64_t tq0 = operand_desc(smem_addr(s_q), BN * 128, 1024), to0 = operand_desc(smem_addr(s_o), BN * 128, 1024);
        uint32_t kvn = 0, qn = 0, n = 0;
        bool ok = true;
        KeyUnit u;
        while (ok && next(u)) {
            const int32_t count = u.low > u.high ? 0 : (u.high - u.low + 1) * a.group;
            if (count == 0)
                continue;
            ok = wait(&sh.kv_full, kvn & 1) && wait(&sh.q_full[qn % S::STAGES], (qn / S::STAGES) & 1);
            if (!ok)
                break;
            ++kvn;
            tmem_fence_after();
            inner_products<DP, 128, BN>(tmem, dk0, dq0 + (((qn % S::STAGES) * S::MOVING) >> 4), desc_s, steps);
            tensor_commit_elected(&sh.s_full);
            for (int32_t i = 0; i < count; ++i, ++qn, ++n) {
                const uint32_t st = qn % S::STAGES;
                ok = wait(&sh.o_full[st], (qn / S::STAGES) & 1);
                if (!ok)
                    break;
                tmem_fence_after();
                inner_products<DP, 128, BN>(tmem + kDp, dv0, do0 + ((st * S::MOVING) >> 4), desc_s, steps);
                tensor_commit_elected(&sh.dp_full);
#pragma unroll
                for (int c = 0; c < BN / 64; ++c) {
                    ok = ok && wait(&sh.p_full[c], n & 1);
                    if (!ok)
                        break;
                    tmem_fence_after();
                    tensor_products4_tmem<128, 32>(tmem + kDv, tmem + 64 * c, to0 + ((st * S::MOVING) >> 4) + 512 * c, desc_acc,
                                                   i != 0 || c != 0);
                }
                if (!ok)
                    break;
                tensor_commit_elected(&sh.o_empty[st]);
                if (i + 1 < count) {
                    const uint32_t to = (qn + 1) % S::STAGES;
                    ok = wait(&sh.q_full[to], ((qn + 1) / S::STAGES) & 1);
                    if (!ok)
                        break;
                    tmem_fence_after();
                    inner_products<DP, 128, BN>(tmem, dk0, dq0 + ((to * S::MOVING) >> 4), desc_s, steps);
                    tensor_commit_elected(&sh.s_full);
                }
#pragma unroll
                for (int c = 0; c < BN / 64; ++c) {
                    ok = ok && wait(&sh.ds_full[c], n & 1);
                    if (!ok)
                        break;
                    tmem_fence_after();
                    tensor_products4_tmem<128, 32>(tmem + kDk, tmem + kDp + 64 * c, tq0 + ((st * S::MOVING) >> 4) + 512 * c,
                                                   desc_acc, i != 0 || c != 0);
                }
                if (!ok)
                    break;
                tensor_commit_elected(&sh.q_empty[st]);
                if (i + 1 == count) {
                    tensor_commit_elected(&sh.kv_empty);
                    tensor_commit_elected(&sh.acc_full);
                }
            }
        }
    } else {
        const int half = warp >> 2, quarter = warp & 3;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const uint32_t at_s = tmem + lanes, at_p = at_s + kDp;
        uint4 *const stage = reinterpret_cast<uint4 *>(s_out + warp * 2048);
        uint32_t qn = 0, n = 0, accs = 0;
        bool ok = true;
        KeyUnit u;
        while (ok && next(u)) {
            const int32_t count = u.low > u.high ? 0 : (u.high - u.low + 1) * a.group;
            const int32_t j = u.first + quarter * 32 + lane;
            float more = 1.0f;  // from P's power of two to that of this key's dS'
            if (kScaled<DT> && count > 0) {
                ok = wait(&sh.kv_full, accs & 1);
                if (!ok)
                    break;
                const float value = j < u.lk ? largest_of_row<S::BOXES>(s_v, quarter * 32 + lane) : 0.0f;
                more = power_of_two(dS_exponent(u.row * value + u.delta) - (int32_t)kShiftP<DT>);
                const float top = warp_max(value);
                if (lane == 0 && half == 0)
                    f.sizes.values[(u.head * f.k_tiles + u.keys + u.first / 128) * 4 + quarter] = top;
            }
            int32_t t = u.low;
            for (int32_t i = 0; i < count; ++i, ++qn, ++n) {
                const uint32_t st = qn % S::STAGES;
                const int32_t p0 = BN * t + u.lk - u.lq, nq = u.lq - BN * t;
                const bool whole = nq >= BN && u.first + 127 <= p0 &&
                                   (p0 + BN - 1 - u.first < a.window || u.first + 127 < a.sinks);
                ok = wait(&sh.s_full, n & 1) && wait(&sh.q_full[st], (qn / S::STAGES) & 1);
                if (!ok)
                    break;
                tmem_fence_after();
                const float *lse = s_stats + st * 2 * BN, *delta = lse + BN;
                if (nq < BN) {
                    // rows behind the last query: zeros, since 0 times what they hold may not be 0
                    ok = wait(&sh.o_full[st], (qn / S::STAGES) & 1);
                    if (!ok)
                        break;
                    for (int k = nq * 8 + threadIdx.x; k < BN * 8; k += S::ROW_WARPS * 32)
#pragma unroll
                        for (int b = 0; b < S::BOXES; ++b) {
                            *reinterpret_cast<uint4 *>(s_o + st * S::MOVING + b * BN * 128 + k * 16) = make_uint4(0, 0, 0, 0);
                            *reinterpret_cast<uint4 *>(s_q + st * S::MOVING + b * BN * 128 + k * 16) = make_uint4(0, 0, 0, 0);
                        }
                    fence_proxy_async();
                }
                F2 p[2][16];
                uint32_t bits[2] = {~0u, ~0u};
                const F2 scale2 = twice(f.scale), zero2 = twice(f.zero), shift2 = twice(kShiftP<DT>);
                const F2 more2 = twice(more);
                // piece c is done (of 64 columns, both are when the second is)
                auto ready = [&](uint64_t *bar, int c) {
                    if (BN == 64 && c == 0)
                        return;
                    tmem_wait_stores();
                    tmem_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive_cluster(smem_addr(BN == 64 ? bar : bar + c));
                };
                auto weigh = [&](int c) {
                    const int at = piece_at<BN>(half, c);
                    uint32_t r[32], w[16];
                    tmem_load32(at_s + at, r);
                    tmem_wait_loads(r);
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const float4 x = *reinterpret_cast<const float4 *>(lse + at + 2 * e);
                        p[c][e] = weights({__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])}, scale2, zero2, {-x.x, -x.y}, shift2);
                        p[c][e + 1] = weights({__uint_as_float(r[2 * e + 2]), __uint_as_float(r[2 * e + 3])}, scale2, zero2, {-x.z, -x.w}, shift2);
                    }
                    if (!whole) {
                        bits[c] = ~bits_up_to(j - p0 - 1 - at) & bits_up_to(nq - 1 - at);
                        if (j >= a.sinks)
                            bits[c] &= bits_up_to(j - p0 + a.window - 1 - at);
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            p[c][e].x = bits[c] & (1u << 2 * e) ? p[c][e].x : 0.0f;
                            p[c][e].y = bits[c] & (2u << 2 * e) ? p[c][e].y : 0.0f;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        w[e] = pack2<DT>(p[c][e].x, p[c][e].y);
                    tmem_store16(at_s + at, w);
                    ready(sh.p_full, c);
                };
                weigh(0);
                weigh(1);
                ok = wait(&sh.dp_full, n & 1);
                if (!ok)
                    break;
                tmem_fence_after();
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int at = piece_at<BN>(half, c);
                    uint32_t r[32], w[16];
                    tmem_load32(at_p + at, r);
                    tmem_wait_loads(r);
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const float4 x = *reinterpret_cast<const float4 *>(delta + at + 2 * e);
                        p[c][e] = p[c][e] * (F2{__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])} + F2{-x.x, -x.y});
                        p[c][e + 1] = p[c][e + 1] * (F2{__uint_as_float(r[2 * e + 2]), __uint_as_float(r[2 * e + 3])} + F2{-x.z, -x.w});
                        if (kScaled<DT>)
                            p[c][e] = p[c][e] * more2, p[c][e + 1] = p[c][e + 1] * more2;
                    }
                    if (!whole) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            p[c][e].x = bits[c] & (1u << 2 * e) ? p[c][e].x : 0.0f;
                            p[c][e].y = bits[c] & (2u << 2 * e) ? p[c][e].y : 0.0f;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        w[e] = pack2<DT>(p[c][e].x, p[c][e].y);
                    tmem_store16(at_p + at, w);
                    ready(sh.ds_full, c);
                }
                t = t == u.high ? u.low : t + 1;
            }
            if (ok && count > 0) {
                ok = wait(&sh.acc_full, accs & 1);
                ++accs;
                tmem_fence_after();
            }
            if (!ok)
                break;
            // dv by the first four warps and dk by the others, or both by the four that there are
            const int32_t left = u.lk - u.first - quarter * 32;  // rows of this warp
#pragma unroll 1
            for (int which = S::ROW_WARPS == 8 ? half : 0; which < (S::ROW_WARPS == 8 ? half + 1 : 2); ++which) {
                const uint32_t from = tmem + lanes + (which ? kDk : kDv);
                const float by = which ? f.scale : 1.0f;
                const float back = kScaled<DT> ? power_of_two(-(int32_t)kShiftP<DT>) / (which ? more : 1.0f) : 1.0f;
                const Heads to{which ? f.dk.p : f.dv.p, which ? f.dk.ld : f.dv.ld, which ? f.dk.hd : f.dv.hd};
                uint16_t *out = static_cast<uint16_t *>(const_cast<void *>(to.p)) + ((int64_t)u.k_row + quarter * 32) * to.ld +
                                u.head * to.hd;
                float *sums = f.partial + ((u.slot * 2 + which) * 128 + quarter * 32 + lane) * a.dim;
#pragma unroll 1
                for (int c = 0; c < a.dim; c += 32) {
                    uint32_t w[16], o[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o[e] = 0;
                    if (count > 0) {
                        tmem_load32(from + c, o);
                        tmem_wait_loads(o);
                        if (kScaled<DT>)
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * back);
                    }
                    if (u.slot >= 0) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            if (c + e < a.dim)
                                *reinterpret_cast<uint4 *>(sums + c + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                        __syncwarp();
                        continue;
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        w[e] = pack2<DT>(__uint_as_float(o[2 * e]) * by, __uint_as_float(o[2 * e + 1]) * by);
                    store_rows(stage, lane, w, out + c, to.ld, left, a.dim - c);
                }
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
        for (int64_t round = 0; round * gridDim.x < all; ++round) {
            const int64_t i = nth_unit(round);
            if (i >= all)
                continue;
            KeyUnit u;
            if (!key_unit<BN>(f, i, lane, u))
                continue;
            if (kScaled<DT> && u.low <= u.high && warp < 4) {  // (k_attn_dq's results are whole)
                float top = 0.0f;
                for (int32_t r = 32 * warp; r < 32 * warp + 32 && u.first + r < u.lk; ++r)
                    for (int e = lane; e < a.dim; e += 32)
                        top = fmaxf(top, fabsf(load1<DT>(f.v_rows.p, (u.k_row + (int64_t)r) * f.v_rows.ld + u.head * f.v_rows.hd + e)));
                top = warp_max(top);
                if (lane == 0)
                    f.sizes.values[(u.head * f.k_tiles + u.keys + u.first / 128) * 4 + warp] = top;
            }
            for (int32_t r = warp; r < 128; r += S::THREADS / 32)
                for (int e = lane; e < a.dim; e += 32)
                    if (u.slot >= 0) {
                        f.partial[((u.slot * 2) * 128 + r) * a.dim + e] = __uint_as_float(0x7fffffffu);
                        f.partial[((u.slot * 2 + 1) * 128 + r) * a.dim + e] = __uint_as_float(0x7fffffffu);
                    } else if (u.first + r < u.lk) {
                        const int64_t row = (int64_t)u.k_row + r;
                        static_cast<uint16_t *>(const_cast<void *>(f.dk.p))[row * f.dk.ld + u.head * f.dk.hd + e] = 0x7fff;
                        static_cast<uint16_t *>(const_cast<void *>(f.dv.p))[row * f.dv.ld + u.head * f.dv.hd + e] = 0x7fff;
                    }
        }
    }
    if (warp == kMma)
        tmem_give(tmem, S::TMEM);
}

// The sums of the first keys' tiles from their parts, in order: a block takes
// every gridDim.y-th eight keys of a tile's key heads.  A few us: its bytes
// are 1 KB for each key, element and 8 or more tiles of queries.
template <int DT>
__global__ void __launch_bounds__(kThreads) k_attn_join(const __grid_constant__ BwdTiles f)
{
    const Attn &a = f.a;
    for (int64_t i = blockIdx.x; i < (int64_t)a.sequences * f.sink_tiles; i += gridDim.x) {
        const int32_t s = (int32_t)(i / f.sink_tiles), tile = (int32_t)(i % f.sink_tiles), first = tile * 128;
        const Seq sq = sequence(a, s);
        if (first >= sq.lk || first >= a.sinks)
            continue;
        const QueryTiles t = query_tiles<128>(a, first, sq.lq, sq.lk);
        if (!is_split(f, first, t))
            continue;
        const int64_t base = a.q_offsets ? sq.q0 / (128 * f.chunk) + s : 0;
        for (int32_t b = blockIdx.y; b < a.k_heads * 16; b += gridDim.y) {
            const int rows = (b & 15) * 8;
            const int32_t g = b >> 4;
            for (int v = threadIdx.x; v < 2 * 8 * a.dim; v += kThreads) {
                const int which = v / (8 * a.dim), r = rows + (v - which * 8 * a.dim) / a.dim, e = v % a.dim;
                if (first + r >= sq.lk)
                    continue;
                float sum = 0.0f;
#pragma unroll 4
                for (int32_t c = t.low / f.chunk; c <= t.high / f.chunk; ++c) {
                    const int64_t slot = ((base + c) * f.sink_tiles + tile) * a.k_heads + g;
                    sum += f.partial[((slot * 2 + which) * 128 + r) * a.dim + e];
                }
                const Heads to{which ? f.dk.p : f.dv.p, which ? f.dk.ld : f.dv.ld, which ? f.dk.hd : f.dv.hd};
                store1<DT>(const_cast<void *>(to.p), (sq.k0 + first + r) * to.ld + g * to.hd + e, which ? sum * f.scale : sum);
            }
        }
    }
}

struct QueryUnit {
    int32_t q_row, k_row, first, lq, lk, head;
    int64_t stats, keys;  // tile number, and that of key tile 0
    float value;          // the largest of the keys' tiles (f16)
    int32_t end;

    __device__ __forceinline__ void agree()
    {
        first = uniform(first), lq = uniform(lq), lk = uniform(lk), head = uniform(head), end = uniform(end);
    }
};

struct QueryShared {
    uint64_t q_full, q_empty, k_full[4], k_empty[4], v_full[4], v_empty[4], s_full[2], dp_full, ds_full[2], acc_full;
    uint64_t unit_full[kUnitRing], unit_empty[kUnitRing];
    QueryUnit units[kUnitRing];
    uint32_t tmem, gave_up;
};

// dq of 128 queries of one head at a time, over the tiles of keys that they
// see: S = Q K^T, dP = dO V^T, dS = exp(S - lse) (dP - delta), dQ += dS K.
// (S and dP are worked out here again, two products of seven, so that dq is
// summed in one place and in one order, without atomics.)
//
// What bounds it: three products, 1536 clocks of the tensor pipe at 128
// elements, against 64 KB of keys and values: 42 B per clock and SM, 12 TB/s,
// where L2 gives all SMs no more than 7.7: about 1.25 of the 2.75 ms above.
// A window's queries of one key head's group read the same keys at about the
// same time, so DRAM does not bound it.
template <int DT, class S>
__global__ void __launch_bounds__(S::THREADS, S::PER_SM) k_attn_dq(const __grid_constant__ BwdTiles f)
{
    constexpr int DP = S::DP, BN = S::BN;
    extern __shared__ unsigned char smem_raw[];
    __shared__ QueryShared sh;
    unsigned char *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023u)) & 1023u);
    unsigned char *const s_q = smem, *const s_o = smem + S::TILE, *const s_k = s_o + S::TILE, *const s_v = s_k + S::STAGES * S::MOVING;
    unsigned char *const s_out = s_v + S::STAGES * S::MOVING;
    const Attn &a = f.a;
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    constexpr int kTma = S::ROW_WARPS, kMma = S::ROW_WARPS + 1;
    constexpr int kDp = 2 * BN, kDq = 3 * BN;  // columns of tensor memory

    if (threadIdx.x == 0) {
        mbar_init_count(&sh.q_full, 1);
        mbar_init_count(&sh.q_empty, 1);
        for (int s = 0; s < S::STAGES; ++s) {
            mbar_init_count(&sh.k_full[s], 1);
            mbar_init_count(&sh.k_empty[s], 1);
            mbar_init_count(&sh.v_full[s], 1);
            mbar_init_count(&sh.v_empty[s], 1);
            if (s < 2)
                mbar_init_count(&sh.s_full[s], 1);
        }
        mbar_init_count(&sh.dp_full, 1);
        for (int c = 0; c < BN / 64; ++c)
            mbar_init_count(&sh.ds_full[c], S::ROW_WARPS);
        mbar_init_count(&sh.acc_full, 1);
        for (int s = 0; s < kUnitRing; ++s) {
            mbar_init_count(&sh.unit_full[s], 1);
            mbar_init_count(&sh.unit_empty[s], S::ROW_WARPS + 1);
        }
        sh.gave_up = 0;
        mbar_init_done();
    }
    if (warp == kMma)
        tmem_take(&sh.tmem, S::TMEM);
    if (warp == kTma && lane < 4)
        tma_prefetch_map(lane == 0 ? &f.q.map : lane == 1 ? &f.k.map : lane == 2 ? &f.v.map : &f.dout.map);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = (uint32_t)uniform((int32_t)sh.tmem);
    // After k_attn_dkv, which waited for the statistics: what one kernel wrote
    // is visible to one that waits, and to none that the waiting one merely let
    // start.  (5340 tokens of 25 heads of 64: 108.3 us against 106.9 with reads
    // from where k_attn_dkv starts to end; 16384 of 64 + 8 of 128 2756 against 2774.)
    pdl_wait();
    auto wait = [&](uint64_t *bar, uint32_t parity) { return mbar_wait_warp(bar, parity, f.limit_ns, &sh.gave_up); };
    uint32_t units = 0;
    auto next = [&](QueryUnit &u) {
        const uint32_t slot = units % kUnitRing;
        if (!wait(&sh.unit_full[slot], (units / kUnitRing) & 1))
            return false;
        u = sh.units[slot];
        u.agree();
        __syncwarp();
        if (lane == 0)
            mbar_arrive_cluster(smem_addr(&sh.unit_empty[slot]));
        ++units;
        return u.end == 0;
    };
    const int64_t all = f.q_tiles * a.q_heads;
    auto unit_at = [&](int64_t i, QueryUnit &u) {
        const int64_t number = f.q_tiles - 1 - i / a.q_heads;  // long ones first
        const TileAt at = find_tile(a, a.q_offsets, a.q_tokens, number, 128, false, lane);
        u = QueryUnit{(int32_t)at.s.q0 + at.first, (int32_t)at.s.k0, at.first, at.s.lq, at.s.lk, (int32_t)(i % a.q_heads), number,
                      a.k_offsets || a.q_offsets ? at.s.k0 / 128 + at.index : 0, 0.0f, 0};
        return at.any;
    };

    if (warp == kTma) {
        asm volatile("fence.proxy.async.global;" ::: "memory");
        uint32_t un = 0, kn = 0;
        bool ok = true;
        auto publish = [&](const QueryUnit &u) {
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
        auto load = [&](unsigned char *to, const HeadsMap &m, int32_t row, int32_t head, int box, uint64_t *bar) {
#pragma unroll
            for (int x = 0; x < S::BOXES; ++x)
                load_box(smem_addr(to) + x * box, m, 64 * x, row, head, smem_addr(bar));
        };
        for (int64_t round = 0; ok && round * gridDim.x < all; ++round) {
            const int64_t i = nth_unit(round);
            if (i >= all)
                continue;
            QueryUnit u;
            if (!unit_at(i, u))
                continue;
            const KeyTiles kt = key_tiles<BN>(a, u.first, u.lq, u.lk);
            const TileList list = tile_list(kt, KeyTiles{0, -1, 0, false});
            if (list.n == 0) {
                ok = publish(u);
                continue;
            }
            if (kScaled<DT>) {
                // first keys' tiles, then the window's; a share to each lane
                const float4 *const values = reinterpret_cast<const float4 *>(f.sizes.values) + u.head / a.group * f.k_tiles + u.keys;
                const int32_t sinks = (list.sinks * BN + 127) / 128, low = list.low * BN / 128, n = sinks + list.high * BN / 128 - low + 1;
                for (int32_t k = lane; k < n; k += 32) {
                    const float4 v = values[k < sinks ? k : low + k - sinks];
                    u.value = fmaxf(u.value, fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)));
                }
            }
            if (kScaled<DT>)
                u.value = warp_max(u.value);
            ok = publish(u) && wait(&sh.q_empty, (un & 1) ^ 1);
            if (!ok)
                break;
            if (elect_one()) {
                mbar_expect(&sh.q_full, 2 * S::TILE);
                load(s_q, f.q, u.q_row, u.head, 16384, &sh.q_full);
                load(s_o, f.dout, u.q_row, u.head, 16384, &sh.q_full);
            }
            __syncwarp();
            ++un;
            const int32_t g = u.head / a.group;
            for (int32_t n = 0; ok && n < list.n; ++n, ++kn) {
                const uint32_t st = kn % S::STAGES, parity = ((kn / S::STAGES) & 1) ^ 1;
                const int32_t row = u.k_row + BN * list.at(n);
                ok = wait(&sh.k_empty[st], parity);
                if (!ok)
                    break;
                if (elect_one()) {
                    mbar_expect(&sh.k_full[st], S::MOVING);
                    load(s_k + st * S::MOVING, f.k, row, g, BN * 128, &sh.k_full[st]);
                }
                __syncwarp();
                ok = wait(&sh.v_empty[st], parity);
                if (!ok)
                    break;
                if (elect_one()) {
                    mbar_expect(&sh.v_full[st], S::MOVING);
                    load(s_v + st * S::MOVING, f.v, row, g, BN * 128, &sh.v_full[st]);
                }
                __syncwarp();
            }
        }
        if (ok) {
            QueryUnit u{};
            u.end = 1;
            publish(u);
        }
    } else if (warp == kMma) {
        constexpr bool kBf16 = DT == ZERO_BF16;
        const uint32_t desc_s = product_desc(kBf16, false, false, 128, BN);
        const int wide = (a.dim + 15) & ~15, steps = wide / 16;
        const uint32_t desc_acc = product_desc(kBf16, false, true, 128, wide);
        const uint64_t dq0 = operand_desc(smem_addr(s_q), 16, 1024), do0 = operand_desc(smem_addr(s_o), 16, 1024);
        const uint64_t dk0 = operand_desc(smem_addr(s_k), 16, 1024), dv0 = operand_desc(smem_addr(s_v), 16, 1024);
        const uint64_t tk0 = operand_desc(smem_addr(s_k), BN * 128, 1024);
        uint32_t un = 0, kn = 0, dsn = 0;
        bool ok = true;
        QueryUnit u;
        while (ok && next(u)) {
            const KeyTiles kt = key_tiles<BN>(a, u.first, u.lq, u.lk);
            const TileList list = tile_list(kt, KeyTiles{0, -1, 0, false});
            if (list.n == 0)
                continue;
            ok = wait(&sh.q_full, un & 1);
            ++un;
            // scores of tile kn + m of the keys, into the one of two buffers
            auto scores = [&](uint32_t at) {
                const uint32_t st = at % S::STAGES, buf = at & 1;
                ok = ok && wait(&sh.k_full[st], (at / S::STAGES) & 1);
                if (!ok)
                    return;
                tmem_fence_after();
                inner_products<DP, 128, BN>(tmem + buf * BN, dq0, dk0 + ((st * S::MOVING) >> 4), desc_s, steps);
                tensor_commit_elected(&sh.s_full[buf]);
            };
            auto grads = [&](uint32_t at) {
                const uint32_t st = at % S::STAGES;
                ok = ok && wait(&sh.v_full[st], (at / S::STAGES) & 1);
                if (!ok)
                    return;
                tmem_fence_after();
                inner_products<DP, 128, BN>(tmem + kDp, do0, dv0 + ((st * S::MOVING) >> 4), desc_s, steps);
                tensor_commit_elected(&sh.dp_full);
                tensor_commit_elected(&sh.v_empty[st]);
            };
            scores(kn);
            grads(kn);
            for (int32_t n = 0; ok && n < list.n; ++n, ++kn, ++dsn) {
                const uint32_t st = kn % S::STAGES, buf = kn & 1;
                if (n + 1 < list.n)
                    scores(kn + 1);
#pragma unroll
                for (int c = 0; c < BN / 64; ++c) {
                    ok = ok && wait(&sh.ds_full[c], dsn & 1);
                    if (!ok)
                        break;
                    tmem_fence_after();
                    if (c == BN / 64 - 1 && n + 1 < list.n)  // all of dP is read
                        grads(kn + 1);
                    if (!ok)
                        break;
                    tensor_products4_tmem<128, 32>(tmem + kDq, tmem + buf * BN + 64 * c, tk0 + ((st * S::MOVING) >> 4) + 512 * c,
                                                   desc_acc, n != 0 || c != 0);
                }
                if (!ok)
                    break;
                tensor_commit_elected(&sh.k_empty[st]);
                if (n + 1 == list.n) {
                    tensor_commit_elected(&sh.q_empty);
                    tensor_commit_elected(&sh.acc_full);
                }
            }
        }
    } else {
        const int half = warp >> 2, quarter = warp & 3;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        uint4 *const stage = reinterpret_cast<uint4 *>(s_out + warp * 2048);
        uint32_t kn = 0, accs = 0;
        bool ok = true;
        QueryUnit u;
        while (ok && next(u)) {
            const KeyTiles kt = key_tiles<BN>(a, u.first, u.lq, u.lk);
            const TileList list = tile_list(kt, KeyTiles{0, -1, 0, false});
            const int32_t row = u.first + quarter * 32 + lane, p = row + u.lk - u.lq;
            const int32_t p_first = u.first + u.lk - u.lq;
            const int32_t p_last = (u.first + 127 < u.lq ? u.first + 127 : u.lq - 1) + u.lk - u.lq;
            const float *stats = f.stats + (u.head * f.q_tiles + u.stats) * 256 + quarter * 32 + lane;
            const float lse = stats[0], delta = stats[128];
            int32_t exponent = 0;  // of this row's dS
            if (kScaled<DT> && list.n > 0)
                exponent = dS_exponent(f.sizes.rows[(u.head * f.q_tiles + u.stats) * 128 + quarter * 32 + lane] * u.value + fabsf(delta));
            for (int32_t n = 0; n < list.n; ++n, ++kn) {
                const uint32_t st = kn % S::STAGES, buf = kn & 1;
                const int32_t k_first = list.at(n) * BN;
                const bool whole = k_first + BN - 1 <= p_first &&
                                   (k_first > p_last - a.window || k_first + BN - 1 < a.sinks);
                ok = wait(&sh.s_full[buf], (kn >> 1) & 1);
                if (!ok)
                    break;
                tmem_fence_after();
                const uint32_t at_s = tmem + lanes + buf * BN, at_p = tmem + lanes + kDp;
                F2 w2[2][16];
                const F2 scale2 = twice(f.scale), zero2 = twice(f.zero), lse2 = twice(-lse), delta2 = twice(-delta), shift2 = twice((float)exponent);
                // the weights, while dP is worked out
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t r[32];
                    tmem_load32(at_s + piece_at<BN>(half, c), r);
                    tmem_wait_loads(r);
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        w2[c][e] = weights({__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])}, scale2, zero2, lse2, shift2);
                }
                if (k_first + BN > u.lk) {
                    // rows behind the last key: zeros, since 0 times what they hold may not be 0
                    for (int k = (u.lk - k_first) * 8 + threadIdx.x; k < BN * 8; k += S::ROW_WARPS * 32)
#pragma unroll
                        for (int b = 0; b < S::BOXES; ++b)
                            *reinterpret_cast<uint4 *>(s_k + st * S::MOVING + b * BN * 128 + k * 16) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async();
                }
                ok = wait(&sh.dp_full, kn & 1);
                if (!ok)
                    break;
                tmem_fence_after();
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int at = piece_at<BN>(half, c);
                    uint32_t r[32], w[16];
                    tmem_load32(at_p + at, r);
                    tmem_wait_loads(r);
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        w2[c][e] = w2[c][e] * (F2{__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])} + delta2);
                    if (!whole) {
                        const uint32_t bits = seen_bits(p, a.window, a.sinks, k_first + at);
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            w2[c][e].x = bits & (1u << 2 * e) ? w2[c][e].x : 0.0f;
                            w2[c][e].y = bits & (2u << 2 * e) ? w2[c][e].y : 0.0f;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        w[e] = pack2<DT>(w2[c][e].x, w2[c][e].y);
                    tmem_store16(at_s + at, w);
                    if (BN == 128 || c == 1) {
                        tmem_wait_stores();
                        tmem_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive_cluster(smem_addr(&sh.ds_full[BN == 128 ? c : 0]));
                    }
                }
            }
            if (ok && list.n > 0) {
                ok = wait(&sh.acc_full, accs & 1);
                ++accs;
                tmem_fence_after();
            }
            if (!ok)
                break;
            // (of eight warps four take every other 32 columns)
            const int32_t left = u.lq - u.first - quarter * 32;  // rows of this warp
            uint16_t *out = static_cast<uint16_t *>(const_cast<void *>(f.dq.p)) + ((int64_t)u.q_row + quarter * 32) * f.dq.ld +
                            u.head * f.dq.hd;
#pragma unroll 1
            for (int c = half * 32; c < a.dim; c += S::ROW_WARPS * 8) {
                uint32_t w[16], o[32];
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    o[e] = 0;
                if (list.n > 0) {
                    tmem_load32(tmem + lanes + kDq + c, o);
                    tmem_wait_loads(o);
                    if (kScaled<DT>)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * power_of_two(-exponent));
                }
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    w[e] = pack2<DT>(__uint_as_float(o[2 * e]) * f.scale, __uint_as_float(o[2 * e + 1]) * f.scale);
                store_rows(stage, lane, w, out + c, f.dq.ld, left, a.dim - c);
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
        for (int64_t round = 0; round * gridDim.x < all; ++round) {
            const int64_t i = nth_unit(round);
            if (i >= all)
                continue;
            QueryUnit u;
            if (!unit_at(i, u))
                continue;
            for (int32_t r = warp; r < 128 && u.first + r < u.lq; r += S::THREADS / 32)
                for (int e = lane; e < a.dim; e += 32)
                    static_cast<uint16_t *>(const_cast<void *>(f.dq.p))[((int64_t)u.q_row + r) * f.dq.ld + u.head * f.dq.hd + e] = 0x7fff;
        }
    }
    if (warp == kMma)
        tmem_give(tmem, S::TMEM);
}

// ------------------------------------------------------------- host side

constexpr int64_t kMostRows = ((int64_t)1 << 31) - 512;
constexpr int32_t kMostHeads = 1 << 15;

constexpr double kLog2E = 1.4426950408889634;

int check_attention(const zero_attention_t *a)
{
    if (!a)
        return ZERO_EINVAL;
    if (!lp_dtype_ok(a->dtype))
        return ZERO_EDTYPE;
    if (a->q_tokens < 0 || a->k_tokens < 0 || a->sequences < 0 || a->q_heads < 1 || a->k_heads < 1 ||
        a->head_dim < 1 || a->window < 1 || a->sinks < 0 || !(a->scale > 0) || !std::isfinite((float)(a->scale * kLog2E)))
        return ZERO_EINVAL;
    if (a->q_tokens > kMostRows || a->k_tokens > kMostRows || a->sequences > kMostRows || a->q_heads > kMostHeads ||
        a->q_heads % a->k_heads != 0 || a->head_dim % 8 != 0 || a->head_dim > kMostDim)
        return ZERO_ESIZE;
    return ZERO_OK;
}

// The arrays of lengths: checked by a call, not by the workspace's size.
int check_offsets(const zero_attention_t *a, Reach *reach)
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
        if (!reach->has(p))
            return ZERO_EINVAL;
    }
    return ZERO_OK;
}

// An array of heads whose rows are whole 16 bytes.
int check_rows(Heads *h, int64_t tokens, int64_t heads, int64_t dim, int32_t dtype, Reach *reach)
{
    if (tokens == 0)
        return ZERO_OK;
    ZERO_TRY(check_heads(h, tokens, heads, dim, dtype, reach));
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
    // (no window of a call sees further than all of its rows)
    const int64_t rows = 1 + (a->q_tokens > a->k_tokens ? a->q_tokens : a->k_tokens);
    r.window = (int32_t)(a->window < rows ? a->window : rows);
    r.sinks = (int32_t)(a->sinks < most ? a->sinks : most);
    r.scale = (float)a->scale;
    return r;
}

// The map of an array of heads; both strides are positive or not needed.
int heads_map(HeadsMap *m, const Heads &h, int64_t tokens, int64_t heads, int64_t dim, int box_rows, int32_t dtype)
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
    cuuint32_t box[3] = {64, 1, (cuuint32_t)box_rows};
    const cuuint32_t step[3] = {1, 1, 1};
    if (m->heads_last) {
        dims[1] = (cuuint64_t)tokens, dims[2] = (cuuint64_t)heads;
        strides[0] = (cuuint64_t)ld * 2, strides[1] = (cuuint64_t)hd * 2;
        box[1] = (cuuint32_t)box_rows, box[2] = 1;
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

// For tests: kernel test_short (0 the forward tiles, 1 dk and dv, 2 dq) asks
// for boxes of queries eight rows too low, so that no tile of them is ever
// whole and its waits run out after test_limit_ns, in the calls of the
// thread that set it and in no other's.
thread_local int32_t test_short = -1;
thread_local uint64_t test_limit_ns = 0;

int short_by(int kernel, uint64_t *limit_ns)
{
    if (test_short != kernel)
        return 0;
    *limit_ns = test_limit_ns;
    return 8;
}

// Heads of up to 64 leave room for two CTAs of one tile of queries each, which
// start and end apart from one another; wider ones for one CTA of two tiles,
// whose products run while the other's weights are worked out.  At 16 heads of
// 64 (narrow, wide): 8 x 1024 tokens 45, 48 us; 64 x 100 19, 30; 8192 181, 208.
using Narrow = FwdShape<64, 1, 64, 2>;
using Wide = FwdShape<128, 2, 128, 1>;

template <int DT, class S>
int launch_tiles(FwdTiles &t, const Fwd &f, const zero_attention_t *a, cudaStream_t st)
{
    ZERO_TRY(heads_map(&t.q, f.q, a->q_tokens, a->q_heads, a->head_dim, 128 - short_by(0, &t.limit_ns), a->dtype));
    ZERO_TRY(heads_map(&t.k, f.k, a->k_tokens, a->k_heads, a->head_dim, S::BN, a->dtype));
    ZERO_TRY(heads_map(&t.v, f.v, a->k_tokens, a->k_heads, a->head_dim, S::BN, a->dtype));
    t.tiles = tile_numbers(a->q_tokens, a->sequences, !a->q_offsets, 128 * S::QT);
    auto kernel = k_attn_tiles<DT, S>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    const int64_t units = t.tiles * t.a.q_heads, most = (int64_t)sm_count() * S::PER_SM;
    if (e == cudaSuccess) {
        kernel<<<(unsigned)(units < most ? units : most), S::THREADS, S::SMEM, st>>>(t);
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
    t.a = f.a, t.out = f.out, t.lse = f.lse;
    t.scale_log2 = (float)(a->scale * kLog2E);
    t.hdr = static_cast<WsHeader *>(ws);
    t.limit_ns = kWaitLimit;
    if (a->head_dim <= 64)
        return a->dtype == ZERO_F16 ? launch_tiles<ZERO_F16, Narrow>(t, f, a, st) : launch_tiles<ZERO_BF16, Narrow>(t, f, a, st);
    return a->dtype == ZERO_F16 ? launch_tiles<ZERO_F16, Wide>(t, f, a, st) : launch_tiles<ZERO_BF16, Wide>(t, f, a, st);
}

// Up to here, on average over the sequences, queries go a few rows at a time
// over their keys instead of in tiles of 128.  Both ways, 4096 keys, us (few |
// tiles of 128) for 1, 4, 8, 16 queries: one sequence of 32 + 8 heads of 128 11,
// 19, 21, 32 | 47; 64 of them 181, 285, 479, 829 | 595 to 602; one of 25 + 25
// heads of 64 11, 12, 13, 17 | 38, 64 of them 281, 314, 317, 459 | 257 to 273.
// (So where heads share no keys and there are enough sequences to fill every
// SM, tiles would take up to 18 % less; and of a batch of long and short all
// go one way, which is the wrong one for some.)
constexpr int64_t kFewQueries = 8;

struct FewPlan {
    int groups;  // of 8 rows
    int32_t tokens, parts, splits;
    int64_t tiles, sets;
};

FewPlan plan_few(const zero_attention_t *a, int64_t q_tokens, bool one)
{
    FewPlan p{};
    const int64_t group = a->q_heads / a->k_heads, n = a->sequences > 0 ? a->sequences : 1;
    const int64_t queries = (q_tokens + n - 1) / n;
    p.groups = group * (queries > 1 ? queries : 1) > 8 ? 2 : 1;
    const int64_t rows = 8 * p.groups;
    p.tokens = (int32_t)(group < rows ? rows / group : 1);
    p.parts = (int32_t)(group > rows ? (group + rows - 1) / rows : 1);
    p.tiles = tile_numbers(q_tokens, a->sequences, one, p.tokens);
    p.sets = p.tiles * a->k_heads * p.parts;
    // Blocks of at least 64 keys, until there are 2048 of them, and no more to
    // a set than its join is worth: a block's keys take it longer in
    // proportion, the last block's join in proportion to the blocks, and with
    // sqrt(keys / 16) blocks of 4 sqrt(keys) keys the two are about equal.
    const int64_t rows_k = (a->k_tokens + n - 1) / n;
    int64_t keys = a->window < rows_k ? a->window + (a->sinks < rows_k ? a->sinks : rows_k) + p.tokens : rows_k;
    keys = keys < rows_k ? keys : rows_k;
    int64_t splits = p.sets > 0 ? (kMostTickets + p.sets - 1) / p.sets : 1;
    const int64_t most = (keys + 63) / 64 < kMostSplits ? (keys + 63) / 64 : kMostSplits;
    splits = splits < most ? splits : most;
    const int64_t worth = (int64_t)std::sqrt((double)keys / 16);
    splits = splits < worth ? splits : worth;
    p.splits = (int32_t)(splits > 1 ? splits : 1);
    return p;
}

template <int DT, int DP, int NG>
int launch_few(const FewArgs &t, int64_t blocks, cudaStream_t st)
{
    k_attn_few<DT, DP, NG><<<(unsigned)blocks, kFewWarps * 32, 0, st>>>(t);
    return check_launch("k_attn_few");
}

int forward_few(const Fwd &f, const zero_attention_t *a, void *ws, size_t partial, cudaStream_t st)
{
    const FewPlan p = plan_few(a, a->q_tokens, !a->q_offsets);
    FewArgs t{f.a, f.q, f.k, f.v, f.out, f.lse, p.tiles, p.tokens, p.parts, p.splits, (float)(a->scale * kLog2E),
              reinterpret_cast<uint32_t *>(static_cast<char *>(ws) + 256),
              reinterpret_cast<float *>(static_cast<char *>(ws) + partial)};
    const int64_t blocks = p.sets * p.splits;
    if (blocks > 0x7fffffff)
        return ZERO_ESIZE;
#define ZERO_FEW(DT)                                                                                             \
    (a->head_dim <= 64 ? p.groups == 1 ? launch_few<DT, 64, 1>(t, blocks, st) : launch_few<DT, 64, 2>(t, blocks, st) \
                       : p.groups == 1 ? launch_few<DT, 128, 1>(t, blocks, st) : launch_few<DT, 128, 2>(t, blocks, st))
    return a->dtype == ZERO_F16 ? ZERO_FEW(ZERO_F16) : ZERO_FEW(ZERO_BF16);
#undef ZERO_FEW
}

// Whether first keys' tiles are dealt out, in parts of how many query tiles:
// about what a tile of the window's keys has to do.  (Of more than 1024 first
// keys every tile sees so much that there is enough to go round.)  Measured,
// window 1024, 4 first keys, 32 + 8 heads of 128, dealt out or not: 16384
// tokens 891, 1513 us; 2 x 16384 1744, 2309; 4 x 4096 839, 917.
struct SinkPlan {
    int32_t chunk, sink_tiles;
    int64_t units;
};

SinkPlan plan_sinks(const zero_attention_t *a, bool one, bool space)
{
    SinkPlan p{};
    if (a->sinks == 0 || a->sinks > 1024 || a->k_tokens == 0)
        return p;
    const int64_t tiles = a->window < a->q_tokens ? (a->window + 127) / 128 + 1 : a->q_tokens;
    const int64_t chunk = tiles > 8 ? tiles : 8;
    if (a->q_tokens <= 2 * chunk * 128)
        return p;
    // A part's number takes in its sequence's, so of sequences that are short
    // on average most of the room for sums would lie idle: theirs are not
    // dealt out.  (A workspace for more sequences serves fewer.)
    const int64_t most = 4 * (a->q_tokens / (chunk * 128)), n = a->sequences < most ? a->sequences : most;
    if (n < a->sequences && !space)
        return p;
    p.chunk = (int32_t)chunk;
    const int64_t keys = a->sinks < a->k_tokens ? a->sinks : a->k_tokens;
    p.sink_tiles = (int32_t)((keys + 127) / 128);
    p.units = tile_numbers(a->q_tokens, n, one, 128 * p.chunk) * p.sink_tiles * a->k_heads;
    return p;
}

// Workspace: the header, the tickets of a few queries' blocks (which start at
// zero and are left at zero, so nothing else may lie there), and what a call
// keeps: a few queries' partial sums, or the backward pass's rows and sums.
struct AttnSpace {
    size_t partial;         // of a few queries
    size_t stats, rows, tops, values, sums;  // of the backward pass
    size_t total;
};

AttnSpace attn_space(const zero_attention_t *a, bool backward)
{
    AttnSpace s{};
    s.partial = s.stats = 256 + kMostTickets * 4;
    // (a workspace for more queries serves fewer; where there is more than one
    // split there are fewer than 2048 sets, and sets x splits is at most 2048
    // more than sets)
    const int64_t most = kFewQueries * a->sequences, q = a->q_tokens < most ? a->q_tokens : most;
    size_t few = 0;
    for (int groups = 1; groups <= 2; ++groups) {
        const int64_t rows = 8 * groups, group = a->q_heads / a->k_heads;
        const int64_t parts = group > rows ? (group + rows - 1) / rows : 1;
        const int64_t sets = tile_numbers(q, a->sequences, false, (int32_t)(group < rows ? rows / group : 1)) * a->k_heads * parts;
        int64_t keys = a->window < a->k_tokens ? a->window + (a->sinks < a->k_tokens ? a->sinks : a->k_tokens) + rows : a->k_tokens;
        keys = keys < a->k_tokens ? keys : a->k_tokens;
        int64_t blocks = 2 * kMostTickets;
        if (sets < kMostTickets)
            blocks = sets * ((keys + 63) / 64) < sets + kMostTickets ? sets * ((keys + 63) / 64) : sets + kMostTickets;
        const size_t bytes = (size_t)blocks * rows * (a->head_dim + 2) * 4;
        few = few > bytes ? few : bytes;
    }
    s.total = s.partial + align256(few);
    if (backward) {
        const size_t q_tiles = (size_t)a->q_heads * (size_t)tile_numbers(a->q_tokens, a->sequences, false, 128);
        const size_t k_tiles = (size_t)a->k_heads * (size_t)tile_numbers(a->k_tokens, a->sequences, false, 128);
        s.rows = s.stats + q_tiles * 1024;
        s.tops = s.rows + q_tiles * 512;
        s.values = s.tops + align256(q_tiles * 32);
        s.sums = s.values + align256(k_tiles * 16);
        const size_t end = s.sums + align256((size_t)plan_sinks(a, false, true).units * 256 * (size_t)a->head_dim * 4);
        s.total = s.total > end ? s.total : end;
    }
    return s;
}

// As forward: heads of up to 64 leave room for two CTAs, with smaller tiles.
// At 16 heads of 64 bf16 (narrow, wide): 8 x 1024 tokens 119, 137 us; 64 x 100
// 52, 69; 8192 432, 478.
using NarrowBwd = BwdShape<64, 64, 2>;
using WideBwd = BwdShape<128, 128, 1>;

struct BwdArrays {
    Heads dout, q, k, v;
};

template <int DT, class S>
int launch_backward(BwdTiles &t, const BwdArrays &h, const zero_attention_t *a, cudaStream_t st)
{
    const char *what = "k_attn_dkv";
    cudaError_t e = cudaSuccess;
    auto launch = [&](void (*kernel)(BwdTiles), int64_t units) {
        if (e != cudaSuccess || units == 0)
            return;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
        if (e != cudaSuccess)
            return;
        const int64_t most = (int64_t)sm_count() * S::PER_SM;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(units < most ? units : most));
        cfg.blockDim = dim3(S::THREADS);
        cfg.dynamicSmemBytes = S::SMEM;
        cfg.stream = st;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = t.q_tiles > 0;  // (a kernel of this call is before it)
        e = cudaLaunchKernelEx(&cfg, kernel, t);
    };
    // the maps: what a kernel keeps in boxes of 128 rows, what moves past it in boxes of BN
    auto maps = [&](int kernel, int q_rows, int k_rows) {
        t.limit_ns = kWaitLimit;
        if (a->q_tokens > 0) {
            ZERO_TRY(heads_map(&t.q, h.q, a->q_tokens, a->q_heads, a->head_dim, q_rows - short_by(kernel, &t.limit_ns), a->dtype));
            ZERO_TRY(heads_map(&t.dout, h.dout, a->q_tokens, a->q_heads, a->head_dim, q_rows, a->dtype));
        }
        if (a->k_tokens > 0) {
            ZERO_TRY(heads_map(&t.k, h.k, a->k_tokens, a->k_heads, a->head_dim, k_rows, a->dtype));
            ZERO_TRY(heads_map(&t.v, h.v, a->k_tokens, a->k_heads, a->head_dim, k_rows, a->dtype));
        }
        if (a->k_tokens == 0)  // (maps that nothing is loaded by, but that kernels name)
            t.k = t.v = t.q;
        if (a->q_tokens == 0)
            t.q = t.dout = t.k;
        return ZERO_OK;
    };
    ZERO_TRY(maps(1, S::BN, 128));
    const int64_t key_units = t.split_units + t.k_tiles * t.a.k_heads;
    launch(k_attn_dkv<DT, S>, key_units);
    if (e == cudaSuccess) {
        what = "k_attn_dq";
        ZERO_TRY(maps(2, 128, S::BN));
        launch(k_attn_dq<DT, S>, t.q_tiles * t.a.q_heads);
    }
    if (e == cudaSuccess && t.split_units > 0) {
        what = "k_attn_join";
        const int64_t every = (int64_t)t.a.sequences * t.sink_tiles, x = every < 152 * 8 ? every : 152 * 8;
        const int64_t y = 152 * 8 / x, most = (int64_t)t.a.k_heads * 16;
        k_attn_join<DT><<<dim3((unsigned)x, (unsigned)(y < most ? y : most)), kThreads, 0, st>>>(t);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        set_cuda_error(what, (int)e, cudaGetErrorString(e));
        return ZERO_ECUDA;
    }
    return ZERO_OK;
}

}  // namespace
}  // namespace zpml

using namespace zpml;

// For tests, and so not in the header: see test_short.  kernel -1: none (the
// default).
extern "C" void zero_test_window_attention_waits(int32_t kernel, uint64_t limit_ns)
{
    test_short = kernel;
    test_limit_ns = limit_ns;
}

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
    Reach reach;
    ZERO_TRY(check_offsets(a, &reach));
    Fwd f{attn_of(a), {q, q_ld, q_hd}, {k, k_ld, k_hd}, {v, v_ld, v_hd}, {out, out_ld, out_hd}, lse};
    ZERO_TRY(check_rows(&f.q, a->q_tokens, a->q_heads, a->head_dim, a->dtype, &reach));
    ZERO_TRY(check_rows(&f.k, a->k_tokens, a->k_heads, a->head_dim, a->dtype, &reach));
    ZERO_TRY(check_rows(&f.v, a->k_tokens, a->k_heads, a->head_dim, a->dtype, &reach));
    ZERO_TRY(check_rows(&f.out, a->q_tokens, a->q_heads, a->head_dim, a->dtype, &reach));
    if (lse)
        ZERO_TRY(check_array(lse, a->q_tokens, ZERO_F32, &reach));
    ZERO_TRY(check_workspace(ws, ws_bytes, attn_space(a, false).total, &reach));
    if (a->q_tokens == 0 || a->sequences == 0)
        return ZERO_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (a->q_tokens > kFewQueries * a->sequences && a->k_tokens > 0)
        return forward_tiles(f, a, ws, st);
    return forward_few(f, a, ws, attn_space(a, false).partial, st);
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
    Reach reach;
    ZERO_TRY(check_offsets(a, &reach));
    Heads hdout{dout, dout_ld, dout_hd}, hq{q, q_ld, q_hd}, hk{k, k_ld, k_hd}, hv{v, v_ld, v_hd}, hout{out, out_ld, out_hd};
    Heads hdq{dq, dq_ld, dq_hd}, hdk{dk, dk_ld, dk_hd}, hdv{dv, dv_ld, dv_hd};
    for (Heads *h : {&hdout, &hq, &hout, &hdq})
        ZERO_TRY(check_rows(h, a->q_tokens, a->q_heads, a->head_dim, a->dtype, &reach));
    for (Heads *h : {&hk, &hv, &hdk, &hdv})
        ZERO_TRY(check_rows(h, a->k_tokens, a->k_heads, a->head_dim, a->dtype, &reach));
    ZERO_TRY(check_array(lse, a->q_tokens, ZERO_F32, &reach));
    const AttnSpace sp = attn_space(a, true);
    ZERO_TRY(check_workspace(ws, ws_bytes, sp.total, &reach));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (a->sequences == 0 || (a->q_tokens == 0 && a->k_tokens == 0))
        return ZERO_OK;
    BwdTiles t{};
    t.a = attn_of(a);
    t.dq = hdq, t.dk = hdk, t.dv = hdv, t.v_rows = hv;
    const bool one = !a->q_offsets;
    t.q_tiles = a->q_tokens > 0 ? tile_numbers(a->q_tokens, a->sequences, one, 128) : 0;
    t.k_tiles = a->k_tokens > 0 ? tile_numbers(a->k_tokens, a->sequences, one && !a->k_offsets, 128) : 0;
    t.stats = reinterpret_cast<float *>(static_cast<char *>(ws) + sp.stats);
    t.sizes = {reinterpret_cast<float *>(static_cast<char *>(ws) + sp.rows),
               reinterpret_cast<float2 *>(static_cast<char *>(ws) + sp.tops),
               reinterpret_cast<float *>(static_cast<char *>(ws) + sp.values)};
    t.partial = reinterpret_cast<float *>(static_cast<char *>(ws) + sp.sums);
    t.scale = (float)a->scale;
    t.hdr = static_cast<WsHeader *>(ws);
    if (a->q_tokens > 0) {
        const SinkPlan p = plan_sinks(a, one, false);
        t.chunk = p.chunk, t.sink_tiles = p.sink_tiles, t.split_units = p.units;
        const bool f16 = a->dtype == ZERO_F16;
        const StatsArgs s{t.a, hdout, hout, lse, const_cast<float *>(t.stats), t.sizes, t.q_tiles};
        auto kernel = a->head_dim <= 16   ? f16 ? k_attn_stats<ZERO_F16, 2> : k_attn_stats<ZERO_BF16, 2>
                      : a->head_dim <= 64 ? f16 ? k_attn_stats<ZERO_F16, 8> : k_attn_stats<ZERO_BF16, 8>
                                          : f16 ? k_attn_stats<ZERO_F16, 16> : k_attn_stats<ZERO_BF16, 16>;
        // blocks for every SM to hold sixteen, or one for each tile and head
        const int64_t x = t.q_tiles < 152 * 16 ? t.q_tiles : 152 * 16, y = (152 * 16 + x - 1) / x;
        kernel<<<dim3((unsigned)x, (unsigned)(y < a->q_heads ? y : a->q_heads)), 128, 0, st>>>(s);
        ZERO_TRY(check_launch("k_attn_stats"));
    }
    const BwdArrays h{hdout, hq, hk, hv};
    if (a->head_dim <= 64)
        return a->dtype == ZERO_F16 ? launch_backward<ZERO_F16, NarrowBwd>(t, h, a, st) : launch_backward<ZERO_BF16, NarrowBwd>(t, h, a, st);
    return a->dtype == ZERO_F16 ? launch_backward<ZERO_F16, WideBwd>(t, h, a, st) : launch_backward<ZERO_BF16, WideBwd>(t, h, a, st);
}
