// The gated feed-forward block, forward and backward: five products on the
// tensor cores (tcgen05, operands by TMA, sums in tensor memory) with the
// activation and its slope in their epilogues.
#include "sublayer.cuh"
#include "tensor.cuh"

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

// One product C[m, n] = sum over the pairs p and over k of A_p[m, k] B_p[n, k]
// of a launch.  Operands are read by TMA in blocks of 64 k: K-major where k
// runs along a row of the matrix in memory, MN-major where it runs down the
// rows, so no operand is ever transposed in memory.
struct Product {
    CUtensorMap a[2], b[2];  // kGate: b holds the gate's and the up matrix of one pair
    int32_t pairs, kb;       // pairs, blocks of 64 k in each
    int32_t m, n;
    int32_t tiles_n, first;  // tiles along n; the product's first tile in the launch
    void *out;
    int64_t out_ld;
    int32_t out_vec;  // out's rows are whole 16 bytes
};

enum Epilogue {
    kStore,   // C as it is
    kGate,    // two products (b[0] and b[1], not summed): act(C0) * C1, and C0, C1 kept
    kGateBwd  // from dh = C and the kept gate and up: dgate, dup, act(gate) * up
};

template <int NP>
struct ProductArgs {
    Product p[NP];
    int32_t tiles, splits;  // tiles of all products; parts that k is cut into
    int32_t a_rows;         // rows of A that a K-major tile loads (128, or all there are rounded up to 8)
    int32_t act;
    int32_t out_f32;        // kStore: out is binary32
    void *o1, *o2;          // kGate: gate, up (or NULL); kGateBwd: dgate, dup
    const void *gate, *up;  // kGateBwd
    int64_t o_ld, g_ld;     // row strides of o1 and o2, and of gate and up
    int32_t o_vec, g_vec;
    float *partials;        // splits > 1: [tile][split][column][128 rows]
    unsigned int *tickets;  // splits > 1: one per tile, zero between calls
    WsHeader *hdr;
    uint64_t limit_ns;      // of every wait
};

// A kernel's tile: CG CTAs (a pair shares one tile, half of A's rows and
// half of B's each), BN columns, STAGES blocks of k in flight.
template <int CG_, int BN_, int STAGES_, int EPI_WARPS_>
struct Shape {
    static constexpr int CG = CG_, BN = BN_, STAGES = STAGES_, EPI_WARPS = EPI_WARPS_;
    static constexpr int BM = 128 * CG;            // rows of a tile
    static constexpr int B_ROWS = BN / CG;         // rows of B per CTA
    static constexpr int A_BYTES = 128 * 128, B_BYTES = B_ROWS * 128, STAGE = A_BYTES + B_BYTES;
    static constexpr int THREADS = (EPI_WARPS + 2) * 32;
    static constexpr int TMEM = 2 * BN < 32 ? 32 : 2 * BN;  // two accumulators
    static constexpr int SMEM = 1024 + STAGES * STAGE + EPI_WARPS * 2048;
};

struct ProductShared {
    uint64_t full[8], empty[8], tfull[2], tempty[2];
    uint32_t tmem, gave_up, last;
};

// 32 rows of 64 bytes of one warp through 2 KB of shared memory, between a
// row per lane and eight rows of four 16-byte pieces per access (the pieces
// XORed so that neither side meets bank conflicts).
__device__ __forceinline__ uint4 *stage_slot(uint4 *stage, int row, int c) { return stage + row * 4 + (c ^ ((row >> 1) & 3)); }

__device__ __forceinline__ void stage_put_row(uint4 *stage, int lane, const uint32_t (&w)[16])
{
#pragma unroll
    for (int c = 0; c < 4; ++c)
        *stage_slot(stage, lane, c) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
}

// Stage to memory: `rows` rows and `bytes` bytes of each, from p on.
template <int ES>
__device__ __forceinline__ void stage_flush(const uint4 *stage, int lane, char *p, int64_t ld_bytes, int rows,
                                            int64_t bytes, bool vec)
{
    const int c = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = (lane >> 2) + 8 * i;
        const uint4 v = *stage_slot(const_cast<uint4 *>(stage), row, c);
        if (row >= rows)
            continue;
        char *q = p + row * ld_bytes + c * 16;
        if (vec && c * 16 + 16 <= bytes) {
            *reinterpret_cast<uint4 *>(q) = v;
        } else {
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 16 / ES; ++e)
                if (c * 16 + e * ES < bytes) {
                    if (ES == 4)
                        *reinterpret_cast<uint32_t *>(q + e * 4) = w[e];
                    else
                        *reinterpret_cast<uint16_t *>(q + e * 2) = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
                }
        }
    }
}

// Memory to registers, in the flush's pattern (zeros outside).
__device__ __forceinline__ void fetch64(uint4 (&v)[4], int lane, const char *p, int64_t ld_bytes, int rows,
                                        int64_t bytes, bool vec)
{
    const int c = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = (lane >> 2) + 8 * i;
        v[i] = make_uint4(0, 0, 0, 0);
        if (row >= rows)
            continue;
        const char *q = p + row * ld_bytes + c * 16;
        if (vec && c * 16 + 16 <= bytes) {
            v[i] = __ldg(reinterpret_cast<const uint4 *>(q));
        } else {
            uint32_t w[4] = {};
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c * 16 + e * 2 < bytes)
                    w[e >> 1] |= (uint32_t)__ldg(reinterpret_cast<const uint16_t *>(q + e * 2)) << (16 * (e & 1));
            v[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// Those registers through the stage to the row of each lane.
__device__ __forceinline__ void stage_take_row(uint4 *stage, int lane, const uint4 (&v)[4], uint32_t (&w)[16])
{
    const int c = lane & 3;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *stage_slot(stage, (lane >> 2) + 8 * i, c) = v[i];
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint4 x = *stage_slot(stage, lane, k);
        w[4 * k] = x.x, w[4 * k + 1] = x.y, w[4 * k + 2] = x.z, w[4 * k + 3] = x.w;
    }
    __syncwarp();
}

// Two 16-bit elements in a word.
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

template <int DT>
__device__ __forceinline__ float2 unpack2(uint32_t w)
{
    if constexpr (DT == ZERO_F16)
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    else
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w));
}

// One warp's epilogue of 32 columns: C in `r` (kGate: the gate in `r`, up in
// `r1`), rows row0 + lane, columns col .. col + 31 of the output.
template <int DT, int EPI, int NP>
__device__ __forceinline__ void finish32(const ProductArgs<NP> &g, const Product &p, uint4 *stage, int lane,
                                         int64_t row0, int64_t col, const uint32_t (&r)[32], const uint32_t (&r1)[32])
{
    const int64_t left = p.m - row0, cols = p.n - col;
    const int rows = left > 32 ? 32 : (int)left;
    if (left <= 0 || cols <= 0)
        return;
    uint32_t w[16];
    auto flush16 = [&](void *out, int64_t ld, bool vec) {
        __syncwarp();
        stage_put_row(stage, lane, w);
        __syncwarp();
        stage_flush<2>(stage, lane, static_cast<char *>(out) + (row0 * ld + col) * 2, ld * 2, rows, cols * 2, vec);
    };
    auto f = [](uint32_t x) { return __uint_as_float(x); };
    if constexpr (EPI == kStore) {
        if (!g.out_f32) {
#pragma unroll
            for (int k = 0; k < 16; ++k)
                w[k] = pack2<DT>(f(r[2 * k]), f(r[2 * k + 1]));
            flush16(p.out, p.out_ld, p.out_vec);
        } else {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    w[k] = r[16 * half + k];
                __syncwarp();
                stage_put_row(stage, lane, w);
                __syncwarp();
                stage_flush<4>(stage, lane, static_cast<char *>(p.out) + (row0 * p.out_ld + col + 16 * half) * 4,
                               p.out_ld * 4, rows, (cols - 16 * half) * 4, p.out_vec);
            }
        }
    } else if constexpr (EPI == kGate) {
#pragma unroll
        for (int k = 0; k < 16; ++k)
            w[k] = pack2<DT>(activate(g.act, f(r[2 * k])).value * f(r1[2 * k]),
                             activate(g.act, f(r[2 * k + 1])).value * f(r1[2 * k + 1]));
        flush16(p.out, p.out_ld, p.out_vec);
        if (g.o1) {
#pragma unroll
            for (int k = 0; k < 16; ++k)
                w[k] = pack2<DT>(f(r[2 * k]), f(r[2 * k + 1]));
            flush16(g.o1, g.o_ld, g.o_vec);
#pragma unroll
            for (int k = 0; k < 16; ++k)
                w[k] = pack2<DT>(f(r1[2 * k]), f(r1[2 * k + 1]));
            flush16(g.o2, g.o_ld, g.o_vec);
        }
    } else {
        uint4 vg[4], vu[4];
        const int64_t at = (row0 * g.g_ld + col) * 2;
        fetch64(vg, lane, static_cast<const char *>(g.gate) + at, g.g_ld * 2, rows, cols * 2, g.g_vec);
        fetch64(vu, lane, static_cast<const char *>(g.up) + at, g.g_ld * 2, rows, cols * 2, g.g_vec);
        uint32_t wg[16], wu[16];
        stage_take_row(stage, lane, vg, wg);
        stage_take_row(stage, lane, vu, wu);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const float2 gg = unpack2<DT>(wg[k]), uu = unpack2<DT>(wu[k]);
            const float c0 = f(r[2 * k]), c1 = f(r[2 * k + 1]);
            const Act t0 = activate(g.act, gg.x), t1 = activate(g.act, gg.y);
            w[k] = pack2<DT>(t0.value * uu.x, t1.value * uu.y);
            wg[k] = pack2<DT>(c0 * uu.x * t0.slope, c1 * uu.y * t1.slope);
            wu[k] = pack2<DT>(c0 * t0.value, c1 * t1.value);
        }
        flush16(p.out, p.out_ld, p.out_vec);
#pragma unroll
        for (int k = 0; k < 16; ++k)
            w[k] = wg[k];
        flush16(g.o1, g.o_ld, g.o_vec);
#pragma unroll
        for (int k = 0; k < 16; ++k)
            w[k] = wu[k];
        flush16(g.o2, g.o_ld, g.o_vec);
    }
}

// Where a work item lies.
struct Item {
    int32_t product, tile, split, m, n, k0, k1;  // m, n: tile coordinates; k0, k1: blocks over all pairs
};

// Tiles of a product go in groups of kRaster rows of tiles, column by column
// within a group, so that the tiles in flight share operands in L2.
constexpr int kRaster = 8;

template <class S, int NP>
__device__ __forceinline__ Item item_at(const ProductArgs<NP> &g, int32_t index)
{
    Item it;
    it.tile = index / g.splits;
    it.split = index - it.tile * g.splits;
    it.product = 0;
#pragma unroll
    for (int q = 1; q < NP; ++q)
        if (it.tile >= g.p[q].first)
            it.product = q;
    const Product &p = g.p[it.product];
    const int32_t t = it.tile - p.first, tiles_m = (p.m - 1) / S::BM + 1, per = kRaster * p.tiles_n;
    const int32_t group = t / per, within = t - group * per;
    const int32_t rows = tiles_m - group * kRaster < kRaster ? tiles_m - group * kRaster : kRaster;
    it.n = within / rows;
    it.m = group * kRaster + (within - it.n * rows);
    const int64_t kb = (int64_t)p.pairs * p.kb;
    it.k0 = (int32_t)(kb * it.split / g.splits);
    it.k1 = (int32_t)(kb * (it.split + 1) / g.splits);
    return it;
}

// Persistent, one CTA per SM: one warp fills a ring of shared-memory stages
// by TMA, one thread issues the tcgen05 products into one of two accumulators
// in tensor memory, and the other warps empty the accumulator before it.
template <class S, int DT, int EPI, bool AMN, bool BMN, int NP>
__global__ void __launch_bounds__(S::THREADS, 1) k_ffn_product(const __grid_constant__ ProductArgs<NP> g)
{
    constexpr int CG = S::CG, BN = S::BN, STAGES = S::STAGES;
    constexpr int kStepN = EPI == kGate ? BN / 2 : BN;  // output columns per tile
    extern __shared__ unsigned char smem_raw[];
    __shared__ ProductShared sh;
    unsigned char *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023u)) & 1023u);
    unsigned char *stage_area = smem + STAGES * S::STAGE;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_rank() : 0;
    const int32_t workers = gridDim.x / CG, worker = blockIdx.x / CG;
    const int32_t items = g.tiles * g.splits;
    constexpr int kTma = S::EPI_WARPS, kMma = S::EPI_WARPS + 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init_count(&sh.full[s], 1);
            mbar_init_count(&sh.empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init_count(&sh.tfull[s], 1);
            mbar_init_count(&sh.tempty[s], CG * S::EPI_WARPS);
        }
        sh.gave_up = 0;
        mbar_init_done();
    }
    if (warp == kMma)
        tmem_alloc<CG>(&sh.tmem, S::TMEM);
    if (warp == kTma && lane == 0)
        for (int q = 0; q < NP; ++q) {
            tma_prefetch_map(&g.p[q].a[0]);
            tma_prefetch_map(&g.p[q].b[0]);
        }
    tmem_fence_before();
    __syncthreads();
    if (CG == 2)
        cluster_sync();
    tmem_fence_after();
    const uint32_t tmem = sh.tmem;
    pdl_wait();

    if (warp == kTma) {
        if (lane == 0) {
            asm volatile("fence.proxy.async.global;" ::: "memory");
            const uint32_t a_bytes = AMN ? S::A_BYTES : (uint32_t)g.a_rows * 128;
            uint32_t n = 0;  // stages filled
            bool ok = true;
            for (int32_t i = worker; ok && i < items; i += workers) {
                const Item it = item_at<S>(g, i);
                const Product &p = g.p[it.product];
                const int32_t m0 = it.m * S::BM + (int32_t)rank * 128, n0 = it.n * kStepN;
                for (int32_t kb = it.k0; kb < it.k1; ++kb, ++n) {
                    const uint32_t s = n % STAGES;
                    if (!mbar_wait_bounded(&sh.empty[s], ((n / STAGES) & 1) ^ 1, g.limit_ns, &sh.gave_up)) {
                        ok = false;
                        break;
                    }
                    // the leader's barrier counts the bytes of both CTAs
                    uint32_t bar = smem_addr(&sh.full[s]);
                    if (rank == 0)
                        mbar_expect(&sh.full[s], CG * (a_bytes + S::B_BYTES));
                    if (CG == 2)
                        bar = peer_addr(bar, 0);
                    const int pair = kb >= p.kb;
                    const int32_t k = (kb - pair * p.kb) * 64;
                    const uint32_t sa = smem_addr(smem) + s * S::STAGE, sb = sa + S::A_BYTES;
                    if (AMN) {
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            tma_load<CG>(sa + j * 8192, &p.a[pair], m0 + 64 * j, k, bar);
                    } else {
                        tma_load<CG>(sa, &p.a[pair], k, m0, bar);
                    }
                    if (EPI == kGate) {
                        if (CG == 2) {
                            tma_load<CG>(sb, &p.b[rank], k, n0, bar);
                        } else {
                            tma_load<CG>(sb, &p.b[0], k, n0, bar);
                            tma_load<CG>(sb + S::B_BYTES / 2, &p.b[1], k, n0, bar);
                        }
                    } else if (BMN) {
#pragma unroll
                        for (int j = 0; j < S::B_ROWS / 64; ++j)
                            tma_load<CG>(sb + j * 8192, &p.b[pair], n0 + (int32_t)rank * S::B_ROWS + 64 * j, k, bar);
                    } else {
                        tma_load<CG>(sb, &p.b[pair], k, n0 + (int32_t)rank * S::B_ROWS, bar);
                    }
                }
            }
        }
    } else if (warp == kMma) {
        if (lane == 0 && rank == 0) {
            constexpr uint32_t desc = product_desc(DT == ZERO_BF16, AMN, BMN, S::BM, BN);
            uint32_t n = 0, t = 0;
            bool ok = true;
            for (int32_t i = worker; ok && i < items; i += workers, ++t) {
                const Item it = item_at<S>(g, i);
                const uint32_t acc = t & 1;
                if (!mbar_wait_bounded(&sh.tempty[acc], ((t >> 1) & 1) ^ 1, g.limit_ns, &sh.gave_up))
                    break;
                tmem_fence_after();
                const uint32_t d = tmem + acc * BN;
                for (int32_t kb = it.k0; kb < it.k1; ++kb, ++n) {
                    const uint32_t s = n % STAGES;
                    if (!mbar_wait_bounded(&sh.full[s], (n / STAGES) & 1, g.limit_ns, &sh.gave_up)) {
                        ok = false;
                        break;
                    }
                    tmem_fence_after();
                    const uint32_t sa = smem_addr(smem) + s * S::STAGE;
                    const uint64_t da = operand_desc(sa, AMN ? 8192 : 16, 1024);
                    const uint64_t db = operand_desc(sa + S::A_BYTES, BMN ? 8192 : 16, 1024);
#pragma unroll
                    for (int k = 0; k < 4; ++k)  // 16 k: 32 bytes of a row, or 16 rows of 128 bytes
                        tensor_product<CG>(d, da + k * (AMN ? 128 : 2), db + k * (BMN ? 128 : 2), desc,
                                           kb != it.k0 || k != 0);
                    tensor_commit<CG>(&sh.empty[s]);
                }
                if (ok)
                    tensor_commit<CG>(&sh.tfull[acc]);
            }
        }
    } else {
        const int quarter = warp & 3, part = warp >> 2;  // lanes 32 * quarter on; this warp's share of the columns
        constexpr int kParts = S::EPI_WARPS / 4, kCols = kStepN / kParts;  // output columns per warp
        uint4 *stage = reinterpret_cast<uint4 *>(stage_area + warp * 2048);
        uint32_t t = 0;
        bool ok = true;
        for (int32_t i = worker; i < items; i += workers, ++t) {
            const Item it = item_at<S>(g, i);
            const Product &p = g.p[it.product];
            const uint32_t acc = t & 1;
            const int64_t row0 = (int64_t)it.m * S::BM + rank * 128 + quarter * 32;
            const int64_t col0 = (int64_t)it.n * kStepN + part * kCols;
            // a wait that gave up makes this and every later tile NaN
            ok = ok && mbar_wait_bounded(&sh.tfull[acc], (t >> 1) & 1, g.limit_ns, &sh.gave_up);
            ok = __all_sync(0xffffffffu, ok);
            tmem_fence_after();
            const uint32_t from = tmem + acc * BN + ((uint32_t)(quarter * 32) << 16) + part * kCols;
            uint32_t r[32], r1[32];
            auto read = [&](int c) {
                if (!ok) {
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        r[k] = r1[k] = 0x7fffffffu;
                    return;
                }
                tmem_load32(from + c, r);
                if (EPI == kGate)
                    tmem_load32(from + BN / 2 + c, r1);
                tmem_wait_loads();
            };
            auto release = [&] {
                tmem_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_cluster(CG == 2 ? peer_addr(smem_addr(&sh.tempty[acc]), 0) : smem_addr(&sh.tempty[acc]));
            };
            if (g.splits == 1) {
#pragma unroll 1
                for (int c = 0; c < kCols; c += 32) {
                    read(c);
                    if (c + 32 >= kCols)
                        release();
                    finish32<DT, EPI, NP>(g, p, stage, lane, row0, col0 + c, r, r1);
                }
            } else {
                // Each part of k leaves its sums in the workspace; the part
                // that arrives last adds all of them in order.
                const bool mine = row0 + lane < p.m;
                float *base = g.partials + (int64_t)it.tile * g.splits * BN * 128 + quarter * 32 + lane;
                auto slot = [&](int split, int column) { return base + ((int64_t)split * BN + column) * 128; };
#pragma unroll 1
                for (int c = 0; c < kCols; c += 32) {
                    read(c);
                    if (c + 32 >= kCols)
                        release();
                    if (mine) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            __stcg(slot(it.split, part * kCols + c + k), __uint_as_float(r[k]));
                            if (EPI == kGate)
                                __stcg(slot(it.split, BN / 2 + part * kCols + c + k), __uint_as_float(r1[k]));
                        }
                    }
                }
                __threadfence();
                asm volatile("bar.sync 1, %0;" ::"n"(S::EPI_WARPS * 32) : "memory");
                if (threadIdx.x == 0) {
                    sh.last = atomicAdd(&g.tickets[it.tile], 1u) == (unsigned)g.splits - 1;
                    if (sh.last)
                        g.tickets[it.tile] = 0;
                    __threadfence();
                }
                asm volatile("bar.sync 1, %0;" ::"n"(S::EPI_WARPS * 32) : "memory");
                const bool last = sh.last;
                asm volatile("bar.sync 1, %0;" ::"n"(S::EPI_WARPS * 32) : "memory");
                if (!last)
                    continue;
#pragma unroll 1
                for (int c = 0; c < kCols; c += 32) {
                    float s0[32], s1[32];
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        s0[k] = s1[k] = 0.0f;
                    if (mine)
#pragma unroll 1
                        for (int q = 0; q < g.splits; ++q)
#pragma unroll
                            for (int k = 0; k < 32; ++k) {
                                s0[k] += __ldcg(slot(q, part * kCols + c + k));
                                if (EPI == kGate)
                                    s1[k] += __ldcg(slot(q, BN / 2 + part * kCols + c + k));
                            }
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        r[k] = __float_as_uint(s0[k]);
                        r1[k] = __float_as_uint(s1[k]);
                    }
                    finish32<DT, EPI, NP>(g, p, stage, lane, row0, col0 + c, r, r1);
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
            atomicAdd(&g.hdr->stalls, 1u);
        const uint64_t began = global_ns();
        while (global_ns() - began < 20000000u) {
        }
    }
    if (CG == 2)
        cluster_sync();
    if (warp == kMma)
        tmem_free<CG>(tmem, S::TMEM);
}

// ------------------------------------------------------------- a few tokens

// Products for up to four tokens, where the weights' bytes are all there is:
// a warp per row of the weight matrix (kPair: of the gate's and the up matrix
// together), or `parts` warps of a block that each take a stretch of k and
// add up in order through shared memory.  A lane multiplies 16-byte pieces of
// the row with the tokens' pieces (which stay in L1) in binary32; four pieces
// of each row are in flight per lane.
struct TokenArgs {
    const void *x;  // tokens x k, row stride x_ld
    int64_t x_ld;
    const void *w0, *w1;  // n x k, contiguous
    void *out;            // kPair: act(C0) * C1; else C0; tokens x n, row stride out_ld
    int64_t out_ld;
    void *o0, *o1;        // kPair: C0 and C1, kept (or NULL), contiguous
    int32_t tokens, n, k, parts, act;
};

// Eight elements from p[i] on (zeros from k on); kW: 16-byte pieces.
template <bool kW>
__device__ __forceinline__ uint4 load_piece(const uint16_t *p, int32_t i, int32_t k)
{
    if (kW)
        return *reinterpret_cast<const uint4 *>(p + i);
    uint32_t w[4] = {};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (i + e < k)
            w[e >> 1] |= (uint32_t)p[i + e] << (16 * (e & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int DT, int MT, bool kPair, bool kW>
__global__ void __launch_bounds__(kThreads, MT == 4 ? 2 : MT == 2 ? 3 : 4)
    k_ffn_tokens(const __grid_constant__ TokenArgs a)
{
    constexpr int R = kPair ? 2 : 1, U = 4;
    __shared__ float s_part[kWarps][R * MT];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per_block = kWarps / a.parts, unit = warp / a.parts, part = warp - unit * a.parts;
    const int32_t pieces = (a.k + 7) >> 3;  // of a row
    const int32_t p0 = (int32_t)((int64_t)pieces * part / a.parts), p1 = (int32_t)((int64_t)pieces * (part + 1) / a.parts);
    const uint16_t *x = static_cast<const uint16_t *>(a.x);
    bool waited = false;
    pdl_launch_next();
    for (int32_t n0 = blockIdx.x * per_block; n0 < a.n; n0 += gridDim.x * per_block) {
        const int32_t n = n0 + unit;
        float acc[R][MT] = {};
        if (n < a.n) {
            const uint16_t *w[2] = {static_cast<const uint16_t *>(a.w0) + (int64_t)n * a.k,
                                    kPair ? static_cast<const uint16_t *>(a.w1) + (int64_t)n * a.k : nullptr};
            for (int32_t i = p0 + lane; i < p1; i += 32 * U) {
                uint4 wv[U][R];
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int q = 0; q < R; ++q)
                        if (i + 32 * u < p1)
                            wv[u][q] = load_piece<kW>(w[q], (i + 32 * u) * 8, a.k);
                if (!waited) {
                    // the weights are not written by the launch before; x is
                    pdl_wait();
                    waited = true;
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (i + 32 * u >= p1)
                        break;
                    float wf[R][8];
#pragma unroll
                    for (int q = 0; q < R; ++q)
                        Elem<DT>::to_float(&wv[u][q], wf[q]);
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        const int64_t row = (m < a.tokens ? m : a.tokens - 1) * a.x_ld;
                        const uint4 xv = load_piece<kW>(x + row, (i + 32 * u) * 8, a.k);
                        float xf[8];
                        Elem<DT>::to_float(&xv, xf);
#pragma unroll
                        for (int q = 0; q < R; ++q)
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                acc[q][m] += wf[q][e] * xf[e];
                    }
                }
            }
        }
#pragma unroll
        for (int q = 0; q < R; ++q)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    acc[q][m] += __shfl_xor_sync(0xffffffffu, acc[q][m], o);
        if (a.parts > 1) {
            __syncthreads();  // s_part was read for the rows before
            if (lane == 0)
#pragma unroll
                for (int q = 0; q < R; ++q)
#pragma unroll
                    for (int m = 0; m < MT; ++m)
                        s_part[warp][q * MT + m] = acc[q][m];
            __syncthreads();
            if (part == 0)
#pragma unroll
                for (int q = 0; q < R; ++q)
#pragma unroll
                    for (int m = 0; m < MT; ++m)
                        for (int j = 1; j < a.parts; ++j)
                            acc[q][m] += s_part[warp + j][q * MT + m];
        }
        if (part == 0 && n < a.n && lane == 0) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
                if (m < a.tokens) {
                    if (kPair) {
                        store1<DT>(a.out, m * a.out_ld + n, activate(a.act, acc[0][m]).value * acc[R - 1][m]);
                        if (a.o0) {
                            store1<DT>(a.o0, (int64_t)m * a.n + n, acc[0][m]);
                            store1<DT>(a.o1, (int64_t)m * a.n + n, acc[R - 1][m]);
                        }
                    } else {
                        store1<DT>(a.out, m * a.out_ld + n, acc[0][m]);
                    }
                }
        }
    }
    if (!waited)
        pdl_wait();
}

// Rows of 16-bit elements copied to rows of whole 16 bytes (widths that no
// vector divides): up to five matrices in one launch.
struct Copy {
    const uint16_t *src;
    uint16_t *dst;
    int64_t rows, cols, src_ld, dst_ld, first;  // first: the matrix's first 8-element group in the launch
};

struct Copies {
    Copy c[5];
    int32_t n;
    int64_t groups;
};

__global__ void __launch_bounds__(kThreads) k_ffn_copy(const __grid_constant__ Copies a)
{
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < a.groups; i += (int64_t)gridDim.x * kThreads) {
        int q = 0;
#pragma unroll
        for (int j = 1; j < 5; ++j)
            if (j < a.n && i >= a.c[j].first)
                q = j;
        const Copy &c = a.c[q];
        const int64_t per = c.dst_ld >> 3, r = (i - c.first) / per, col = ((i - c.first) - r * per) * 8;
        uint32_t w[4] = {};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (col + e < c.cols)
                w[e >> 1] |= (uint32_t)c.src[r * c.src_ld + col + e] << (16 * (e & 1));
        *reinterpret_cast<uint4 *>(c.dst + r * c.dst_ld + col) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// ------------------------------------------------------------- host side

constexpr int64_t kMostSize = ((int64_t)1 << 31) - 512;
constexpr int kSms = 152;

using Pair256 = Shape<2, 256, 6, 8>;
using One128 = Shape<1, 128, 6, 8>;
using One64 = Shape<1, 64, 8, 4>;

constexpr int kMaxSplitTiles = 512;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t up8(int64_t a) { return (a + 7) & ~(int64_t)7; }

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
    if (ld >= (int64_t)1 << 38)
        return ZERO_ESIZE;  // a tensor map's strides end at 2^40 bytes
    return whole && (!aligned16(p) || (rows > 1 && (ld & 7) != 0)) ? ZERO_EALIGN : ZERO_OK;
}

// How a product is cut: its shape and the parts of k.
enum Cut { kPair256, kOne128, kOne64 };
struct Plan {
    Cut cut;
    int splits;
};

Plan plan_product(int64_t m, int64_t n, int64_t kb, bool gate)
{
    const int64_t step = gate ? 2 : 1;
    if (cdiv(m, 256) * cdiv(n * step, 256) >= kSms / 2)
        return {kPair256, 1};
    if (cdiv(m, 128) * cdiv(n * step, 128) >= kSms)
        return {kOne128, 1};
    const int64_t tiles = cdiv(m, 128) * cdiv(n * step, 64);
    int64_t splits = tiles < kSms ? kSms / tiles : 1;
    if (splits > kb / 4)
        splits = kb / 4;
    return {kOne64, (int)(splits < 1 ? 1 : splits)};
}

// Workspace: the header, the tickets of split products, the products'
// partial sums, then the matrices that a call keeps between its products.
constexpr size_t kWsTickets = 256;
constexpr size_t kWsData = kWsTickets + kMaxSplitTiles * sizeof(unsigned int);

size_t partial_bytes(int64_t m, int64_t n, int64_t k, int pairs, bool gate)
{
    if (m == 0 || n == 0 || k == 0)
        return 0;
    const Plan pl = plan_product(m, n, pairs * cdiv(k, 64), gate);
    return pl.splits == 1 ? 0 : (size_t)(cdiv(m, 128) * cdiv(n * (gate ? 2 : 1), 64)) * pl.splits * 128 * 64 * 4;
}

struct FfnSpace {
    size_t partials, mats, mat_bytes, copies, total;
};

FfnSpace ffn_space(int64_t m, int64_t d, int64_t f, bool backward)
{
    FfnSpace s{};
    size_t part = 0;
    auto most = [&](size_t x) { part = x > part ? x : part; };
    most(partial_bytes(m, f, d, 1, true));
    most(partial_bytes(m, d, f, 1, false));
    if (backward) {
        most(partial_bytes(m, f, d, 1, false));
        most(partial_bytes(m, d, f, 2, false));
    }
    s.partials = kWsData;
    s.mats = s.partials + align256(part);
    s.mat_bytes = align256((size_t)m * (size_t)up8(f) * 2);
    s.copies = s.mats + (backward ? 3 : 1) * s.mat_bytes;
    s.total = s.copies;
    if (((d | f) & 7) != 0)
        s.total += (backward ? 2 : 1) * align256((size_t)m * up8(d) * 2) + 2 * align256((size_t)f * up8(d) * 2) +
                   align256((size_t)d * up8(f) * 2);
    return s;
}

// A matrix as an operand.
struct Mat {
    const void *p;
    int64_t rows, cols, ld;
};

// Operands whose rows are not whole 16 bytes, copied to the workspace; the
// matrices then name the copies.
int copy_operands(Mat **mats, int n, char *to, cudaStream_t st)
{
    Copies a{};
    for (int i = 0; i < n; ++i) {
        Mat &m = *mats[i];
        const int64_t ld = up8(m.cols);
        if (m.rows == 0 || m.cols == 0)
            continue;
        if (aligned16(m.p) && (m.ld & 7) == 0)
            continue;
        Copy &c = a.c[a.n++];
        c = {static_cast<const uint16_t *>(m.p), reinterpret_cast<uint16_t *>(to), m.rows, m.cols, m.ld, ld, a.groups};
        a.groups += m.rows * (ld / 8);
        m.p = to;
        m.ld = ld;
        to += align256((size_t)m.rows * ld * 2);
    }
    if (a.n == 0)
        return ZERO_OK;
    k_ffn_copy<<<grid_for(reinterpret_cast<const void *>(k_ffn_copy), cdiv(a.groups, kThreads), 1 << 30), kThreads, 0,
                 st>>>(a);
    return check_launch("k_ffn_copy");
}

// The tensor maps of one product in the boxes of a shape; A and B are rows of
// k (K-major) or, with amn / bmn, rows of m / n.
template <class S>
int product_maps(Product *p, int i, const Mat &a, bool amn, const Mat &b, bool bmn, int a_rows, bool gate, int32_t dtype)
{
    ZERO_TRY(tensor_map(&p->a[i], a.p, a.rows, a.cols, a.ld, amn ? 64 : a_rows, dtype));
    return tensor_map(&p->b[i], b.p, b.rows, b.cols, b.ld, bmn ? 64 : gate ? (S::CG == 2 ? 128 : S::BN / 2) : S::B_ROWS,
                      dtype);
}

// One launch of up to NP products.
struct Spec {
    Mat a[2], b[2];
    int pairs;
    int64_t m, n, k;
    void *out;
    int64_t out_ld;
};

template <class S, int DT, int EPI, bool AMN, bool BMN, int NP>
int launch_products(const Spec (&specs)[NP], ProductArgs<NP> &g, int splits, int32_t dtype, cudaStream_t st)
{
    constexpr bool gate = EPI == kGate;
    g.splits = splits;
    const int64_t m0 = specs[0].m;
    g.a_rows = !AMN && S::CG == 1 && m0 < 128 ? (int)up8(m0) : 128;
    int64_t tiles = 0, longest = 0;
    for (int q = 0; q < NP; ++q) {
        const Spec &s = specs[q];
        Product &p = g.p[q];
        ZERO_TRY((product_maps<S>(&p, 0, s.a[0], AMN, s.b[0], BMN, g.a_rows, gate, dtype)));
        if (gate)
            ZERO_TRY(tensor_map(&p.b[1], s.b[1].p, s.b[1].rows, s.b[1].cols, s.b[1].ld, S::CG == 2 ? 128 : S::BN / 2,
                                dtype));
        else if (s.pairs == 2)
            ZERO_TRY((product_maps<S>(&p, 1, s.a[1], AMN, s.b[1], BMN, g.a_rows, gate, dtype)));
        p.pairs = s.pairs, p.kb = (int32_t)cdiv(s.k, 64), p.m = (int32_t)s.m, p.n = (int32_t)s.n;
        p.tiles_n = (int32_t)cdiv(s.n, gate ? S::BN / 2 : S::BN);
        p.first = (int32_t)tiles;
        p.out = s.out, p.out_ld = s.out_ld;
        p.out_vec = aligned16(s.out) && (s.out_ld * (EPI == kStore && g.out_f32 ? 4 : 2)) % 16 == 0;
        tiles += cdiv(s.m, S::BM) * p.tiles_n;
        longest = s.pairs * (int64_t)p.kb > longest ? s.pairs * (int64_t)p.kb : longest;
    }
    if (tiles * splits > 0x3fffffff)
        return ZERO_ESIZE;
    g.tiles = (int32_t)tiles;
    g.limit_ns = 2000000000ull + (uint64_t)longest * 4000;
    auto kernel = k_ffn_product<S, DT, EPI, AMN, BMN, NP>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    const int64_t workers = (int64_t)sm_count() / S::CG;
    const int64_t items = tiles * splits;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((items < workers ? items : workers) * S::CG));
    cfg.blockDim = dim3(S::THREADS);
    cfg.dynamicSmemBytes = S::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = S::CG;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = S::CG == 2 ? 1 : 0;
    if (e == cudaSuccess)
        e = cudaLaunchKernelEx(&cfg, kernel, g);
    if (e != cudaSuccess) {
        cudaGetLastError();
        set_cuda_error("k_ffn_product", (int)e, cudaGetErrorString(e));
        return ZERO_ECUDA;
    }
    return ZERO_OK;
}

template <int EPI, bool AMN, bool BMN, int NP>
int products(const Spec (&specs)[NP], ProductArgs<NP> &g, Plan plan, int32_t dtype, cudaStream_t st)
{
    const bool f16 = dtype == ZERO_F16;
#define ZERO_CUT(S)                                                                                       \
    (f16 ? launch_products<S, ZERO_F16, EPI, AMN, BMN, NP>(specs, g, plan.splits, dtype, st)              \
         : launch_products<S, ZERO_BF16, EPI, AMN, BMN, NP>(specs, g, plan.splits, dtype, st))
    if (plan.cut == kPair256)
        return ZERO_CUT(Pair256);
    if (plan.cut == kOne128)
        return ZERO_CUT(One128);
    return ZERO_CUT(One64);
#undef ZERO_CUT
}

// Zeros for a matrix of an empty product.
int zero_matrix(void *p, int64_t ld, int64_t rows, int64_t cols, int es, cudaStream_t st)
{
    if (rows == 0 || cols == 0)
        return ZERO_OK;
    const cudaError_t e = cudaMemset2DAsync(p, (size_t)(rows > 1 ? ld : cols) * es, 0, (size_t)cols * es, (size_t)rows, st);
    if (e != cudaSuccess) {
        cudaGetLastError();
        set_cuda_error("cudaMemset2DAsync", (int)e, cudaGetErrorString(e));
        return ZERO_ECUDA;
    }
    return ZERO_OK;
}

template <int NP>
void workspace_args(ProductArgs<NP> &g, void *ws, const FfnSpace &sp)
{
    g.hdr = static_cast<WsHeader *>(ws);
    g.tickets = reinterpret_cast<unsigned int *>(static_cast<char *>(ws) + kWsTickets);
    g.partials = reinterpret_cast<float *>(static_cast<char *>(ws) + sp.partials);
}

// ------------------------------------------------------------- a few tokens

constexpr int kFewTokens = 4;

// Warps per weight row: k is shared out until a lane has about four pieces of
// 8 elements (1024 elements per warp), as long as there are too few rows to
// give every SM 32 warps.
int token_parts(int64_t n, int64_t k)
{
    int parts = 1;
    while (parts < kWarps && n * parts < (int64_t)kSms * 32 && k >= (int64_t)parts * 2 * 512)
        parts *= 2;
    return parts;
}

template <int DT, bool kPair>
int token_product(TokenArgs &a, bool whole, bool chained, cudaStream_t st)
{
    a.parts = token_parts(a.n, a.k);
    const int64_t units = cdiv(a.n, kWarps / a.parts), most = (int64_t)sm_count() * (a.tokens == 1 ? 4 : a.tokens == 2 ? 3 : 2);
    const int grid = (int)(units < most ? units : most);
    cudaError_t e;
#define ZERO_MT(MT)                                                                                            \
    (whole ? launch_k(k_ffn_tokens<DT, MT, kPair, true>, grid, kThreads, st, chained, a)                        \
           : launch_k(k_ffn_tokens<DT, MT, kPair, false>, grid, kThreads, st, chained, a))
    if (a.tokens == 1)
        e = ZERO_MT(1);
    else if (a.tokens == 2)
        e = ZERO_MT(2);
    else
        e = ZERO_MT(4);
#undef ZERO_MT
    if (e != cudaSuccess) {
        cudaGetLastError();
        set_cuda_error("k_ffn_tokens", (int)e, cudaGetErrorString(e));
        return ZERO_ECUDA;
    }
    return ZERO_OK;
}

// The forward pass of a few tokens.  The second launch is scheduled while the
// first runs and has its first weights in flight when the first ends.
template <int DT>
int tokens_forward(const void *x, int64_t x_ld, const void *wg, const void *wu, const void *wd, void *y, int64_t y_ld,
                   void *gate, void *up, int32_t tokens, int32_t dim, int32_t inner, int32_t act, void *h, bool whole,
                   cudaStream_t st)
{
    TokenArgs a{};
    a.x = x, a.x_ld = x_ld, a.w0 = wg, a.w1 = wu, a.out = h, a.out_ld = up8(inner), a.o0 = gate, a.o1 = up;
    a.tokens = tokens, a.n = inner, a.k = dim, a.act = act;
    ZERO_TRY((token_product<DT, true>(a, whole, false, st)));
    TokenArgs b{};
    b.x = h, b.x_ld = up8(inner), b.w0 = wd, b.out = y, b.out_ld = y_ld;
    b.tokens = tokens, b.n = dim, b.k = inner;
    return token_product<DT, false>(b, whole, true, st);
}

}  // namespace
}  // namespace zpml

using namespace zpml;

extern "C" size_t zero_gated_ffn_workspace_bytes(int64_t tokens, int64_t dim, int64_t inner, int32_t backward)
{
    if (tokens < 0 || dim < 0 || inner < 0 || tokens > kMostSize || dim > kMostSize || inner > kMostSize)
        return 0;
    return ffn_space(tokens, dim, inner, backward != 0).total;
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
    const FfnSpace sp = ffn_space(tokens, dim, inner, false);
    ZERO_TRY(check_workspace(ws, ws_bytes, sp.total));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (tokens == 0)
        return ZERO_OK;
    if (dim == 0 || inner == 0) {
        if (gate) {
            ZERO_TRY(zero_matrix(gate, inner, tokens, inner, 2, st));
            ZERO_TRY(zero_matrix(up, inner, tokens, inner, 2, st));
        }
        return zero_matrix(y, y_ld, tokens, dim, 2, st);
    }
    char *base = static_cast<char *>(ws);
    if (tokens <= kFewTokens)
        return (dtype == ZERO_F16 ? tokens_forward<ZERO_F16> : tokens_forward<ZERO_BF16>)(
            x, x_ld, w_gate, w_up, w_down, y, y_ld, gate, up, (int32_t)tokens, (int32_t)dim, (int32_t)inner, act,
            base + sp.mats, whole, st);
    Mat mx{x, tokens, dim, x_ld}, mg{w_gate, inner, dim, dim}, mu{w_up, inner, dim, dim};
    Mat md{w_down, dim, inner, inner};
    if (!whole) {
        Mat *all[] = {&mx, &mg, &mu, &md};
        ZERO_TRY(copy_operands(all, 4, base + sp.copies, st));
    }
    const Mat h{base + sp.mats, tokens, inner, up8(inner)};
    ProductArgs<1> g{};
    workspace_args(g, ws, sp);
    g.act = act, g.o1 = gate, g.o2 = up, g.o_ld = inner;
    g.o_vec = aligned16(gate) && aligned16(up) && (inner & 7) == 0;
    const Spec s1[1] = {{{mx, mx}, {mg, mu}, 1, tokens, inner, dim, const_cast<void *>(h.p), h.ld}};
    ZERO_TRY((products<kGate, false, false, 1>(s1, g, plan_product(tokens, inner, cdiv(dim, 64), true), dtype, st)));
    ProductArgs<1> d{};
    workspace_args(d, ws, sp);
    const Spec s2[1] = {{{h, h}, {md, md}, 1, tokens, dim, inner, y, y_ld}};
    return products<kStore, false, false, 1>(s2, d, plan_product(tokens, dim, cdiv(inner, 64), false), dtype, st);
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
    const FfnSpace sp = ffn_space(tokens, dim, inner, true);
    ZERO_TRY(check_workspace(ws, ws_bytes, sp.total));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (tokens == 0 || dim == 0 || inner == 0) {
        const int es = gdtype == ZERO_F32 ? 4 : 2;
        ZERO_TRY(zero_matrix(dx, dx_ld, tokens, dim, 2, st));
        ZERO_TRY(zero_matrix(dw_gate, dim, inner, dim, es, st));
        ZERO_TRY(zero_matrix(dw_up, dim, inner, dim, es, st));
        return zero_matrix(dw_down, inner, dim, inner, es, st);
    }
    char *base = static_cast<char *>(ws);
    Mat my{dy, tokens, dim, tokens > 1 ? dy_ld : up8(dim)}, mx{x, tokens, dim, tokens > 1 ? x_ld : up8(dim)};
    Mat mg{w_gate, inner, dim, dim}, mu{w_up, inner, dim, dim}, md{w_down, dim, inner, inner};
    if (!whole) {
        Mat *all[] = {&my, &mx, &mg, &mu, &md};
        ZERO_TRY(copy_operands(all, 5, base + sp.copies, st));
    }
    const int64_t ld = up8(inner);
    const Mat dg{base + sp.mats, tokens, inner, ld}, du{base + sp.mats + sp.mat_bytes, tokens, inner, ld},
        h{base + sp.mats + 2 * sp.mat_bytes, tokens, inner, ld};
    ProductArgs<1> g{};  // dh, and from it dgate, dup and act(gate) * up
    workspace_args(g, ws, sp);
    g.act = act, g.o1 = const_cast<void *>(dg.p), g.o2 = const_cast<void *>(du.p), g.o_ld = ld, g.o_vec = 1;
    g.gate = gate, g.up = up, g.g_ld = inner, g.g_vec = aligned16(gate) && aligned16(up) && (inner & 7) == 0;
    const Spec s1[1] = {{{my, my}, {md, md}, 1, tokens, inner, dim, const_cast<void *>(h.p), ld}};
    ZERO_TRY((products<kGateBwd, false, true, 1>(s1, g, plan_product(tokens, inner, cdiv(dim, 64), false), dtype, st)));
    ProductArgs<1> d{};
    workspace_args(d, ws, sp);
    const Spec s2[1] = {{{dg, du}, {mg, mu}, 2, tokens, dim, inner, dx, dx_ld}};
    ZERO_TRY((products<kStore, false, true, 1>(s2, d, plan_product(tokens, dim, 2 * cdiv(inner, 64), false), dtype, st)));
    ProductArgs<3> w{};
    workspace_args(w, ws, sp);
    w.out_f32 = gdtype == ZERO_F32;
    const Spec s3[3] = {{{dg, dg}, {mx, mx}, 1, inner, dim, tokens, dw_gate, dim},
                        {{du, du}, {mx, mx}, 1, inner, dim, tokens, dw_up, dim},
                        {{my, my}, {h, h}, 1, dim, inner, tokens, dw_down, inner}};
    Plan pl = plan_product(3 * inner, dim, cdiv(tokens, 64), false);
    pl.splits = 1;
    return products<kStore, true, true, 3>(s3, w, pl, dtype, st);
}
