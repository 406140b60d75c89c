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
// The exponential and the reciprocal are CUDA's fast ones (a few units of
// 2^-23, far below the 16-bit rounding that follows): with the exact ones the
// gate's epilogue, not the tensor cores, set the pace.
struct Act {
    float value, slope;
};

__device__ __forceinline__ Act activate(int32_t act, float g)
{
    constexpr float kA = 1.5957691216057308f, kB = 0.044715f;
    const float q = g * g;
    const float k = act == ZERO_ACT_SILU ? g : g * (kA + kA * kB * q);
    const float dk = act == ZERO_ACT_SILU ? 1.0f : kA + 3.0f * kA * kB * q;
    const float s = __fdividef(1.0f, 1.0f + __expf(-k));
    const float v = g * s;
    return {v, s + v * (1.0f - s) * dk};
}

// ------------------------------------------------------------- kernels

// One product C[m, n] = sum over the pairs p and over k of A_p[m, k] B_p[n, k]
// of a launch.  Operands are read by TMA in blocks of 64 k: K-major where k
// runs along a row of the matrix in memory, MN-major where it runs down the
// rows, so no operand is ever transposed in memory.
struct Product {
    CUtensorMap a[2], b[2];  // kGate: b holds the gate's and the up matrix of one pair
    CUtensorMap c;           // the output, where TMA can write it
    int32_t pairs, kb;       // pairs, blocks of 64 k in each
    int32_t m, n;
    int32_t tiles_n, first;  // tiles along n; the product's first tile in the launch
    int32_t c_tma;
    void *out;
    int64_t out_ld;
};

// How the operands of a launch lie: A and B K-major, B MN-major, or both.
enum Major { kKK, kKMn, kMnMn };

enum Epilogue {
    kStore,   // C as it is
    kGate,    // two products (b[0] and b[1], not summed): act(C0) * C1, and C0, C1 kept
    kGateBwd  // from dh = C and the kept gate and up: dgate, dup, act(gate) * up
};

// A matrix beside the output: gate and up, or dgate and dup.
struct Side {
    CUtensorMap map;
    void *p;
    int64_t ld;
    int32_t tma, vec;  // read or written by TMA; rows of whole 16 bytes
};

template <int NP, int EPI>
struct ProductArgs {
    Product p[NP];
    Side side[EPI == kStore ? 1 : EPI == kGate ? 2 : 4];  // kGate: gate, up; kGateBwd: dgate, dup, gate, up
    int32_t products, tiles;
    int32_t splits;   // parts that k is cut into: the CTAs of a cluster
    int32_t a_rows;   // rows of A that a K-major tile loads (128, or all there are rounded up to 8)
    int32_t stages, stage_bytes;  // the ring: a stage is a_rows of A and B's rows
    int32_t act;
    int32_t out_f32;  // kStore: out is binary32
    WsHeader *hdr;
    uint64_t limit_ns;  // of every wait
};

// A kernel's tile: CG CTAs (a pair shares one tile, half of A's rows and
// half of B's each), BN columns, STAGES blocks of k in flight; SETS sets of
// BOXES boxes (32 rows by 64 bytes) per epilogue warp, one set per 32 columns.
template <int CG_, int BN_, int STAGES_, int EPI_WARPS_, int BOXES_, int SETS_>
struct Shape {
    static constexpr int CG = CG_, BN = BN_, STAGES = STAGES_, EPI_WARPS = EPI_WARPS_, BOXES = BOXES_, SETS = SETS_;
    static constexpr int BM = 128 * CG;     // rows of a tile
    static constexpr int B_ROWS = BN / CG;  // rows of B per CTA
    static constexpr int A_BYTES = 128 * 128, B_BYTES = B_ROWS * 128, STAGE = A_BYTES + B_BYTES;
    static constexpr int THREADS = (EPI_WARPS + 2) * 32;
    static constexpr int TMEM = 2 * BN;                // two accumulators
    static constexpr int WARP_OUT = SETS * BOXES * 2048;
    static constexpr int SMEM = 1024 + STAGES * STAGE + EPI_WARPS * WARP_OUT;
    static constexpr int PER_SM = SMEM <= 112 * 1024 ? 2 : 1;
    static_assert(STAGES <= 12 && SMEM <= 232448 - 512, "one CTA's shared memory");
    static_assert(CG == 2 || STAGES * STAGE >= BN * 512, "a split product's sums lie in the stages");
};

constexpr int kMaxStages = 12;
constexpr int kMostParts = 8;  // of k: CTAs of a portable cluster

struct ProductShared {
    uint64_t full[kMaxStages], empty[kMaxStages], tfull[2], tempty[2], in[16];
    uint32_t tmem, gave_up;
};

// 32 rows of 64 bytes of one warp in 2 KB of shared memory, under the 64-byte
// TMA swizzle (16-byte pieces XORed by half the row), which also keeps a row
// per lane and eight rows of four pieces per access free of bank conflicts.
__device__ __forceinline__ uint4 *stage_slot(uint4 *stage, int row, int c) { return stage + row * 4 + (c ^ ((row >> 1) & 3)); }

__device__ __forceinline__ void stage_put_row(uint4 *stage, int lane, const uint32_t (&w)[16])
{
#pragma unroll
    for (int c = 0; c < 4; ++c)
        *stage_slot(stage, lane, c) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
}

__device__ __forceinline__ void stage_get_row(uint4 *stage, int lane, uint32_t (&w)[16])
{
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const uint4 x = *stage_slot(stage, lane, c);
        w[4 * c] = x.x, w[4 * c + 1] = x.y, w[4 * c + 2] = x.z, w[4 * c + 3] = x.w;
    }
}

// Stage to memory element by element (rows that are not whole 16 bytes):
// `rows` rows and `bytes` bytes of each, from p on; a warp writes a row at a
// time.
template <int ES>
__device__ __forceinline__ void stage_flush(uint4 *stage, int lane, char *p, int64_t ld_bytes, int rows, int64_t bytes)
{
    constexpr int kPer = 64 / ES, kAtOnce = 32 / kPer;  // elements of a row: one per lane, or two rows at a time
    const int e = lane % kPer, r0 = lane / kPer;
    if (e * ES >= bytes)
        return;
    p += r0 * ld_bytes + e * ES;
    // sixteen rows read before the first is written: the compiler cannot know
    // that the writes leave the stage alone
#pragma unroll 1
    for (int first = 0; first < rows; first += 16 * kAtOnce) {
        uint32_t v[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const char *s = reinterpret_cast<const char *>(stage_slot(stage, first + k * kAtOnce + r0, e * ES / 16)) + e * ES % 16;
            v[k] = ES == 4 ? *reinterpret_cast<const uint32_t *>(s) : *reinterpret_cast<const uint16_t *>(s);
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            if (first + k * kAtOnce + r0 < rows) {
                if (ES == 4)
                    *reinterpret_cast<uint32_t *>(p) = v[k];
                else
                    *reinterpret_cast<uint16_t *>(p) = (uint16_t)v[k];
            }
            p += kAtOnce * ld_bytes;
        }
    }
}

// Memory to the stage without TMA: 16-byte pieces if vec, else element by
// element; zeros outside.
__device__ __forceinline__ void stage_fetch(uint4 *stage, int lane, const char *p, int64_t ld_bytes, int rows,
                                            int64_t bytes, bool vec)
{
    const int c = lane & 3;
    if (vec) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = (lane >> 2) + 8 * i;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (row < rows && c * 16 < bytes)
                v = __ldg(reinterpret_cast<const uint4 *>(p + row * ld_bytes + c * 16));
            *stage_slot(stage, row, c) = v;
        }
    } else {
        uint16_t v[32];  // all on their way at once
#pragma unroll
        for (int r = 0; r < 32; ++r) {
            v[r] = 0;
            if (r < rows && lane * 2 < bytes)
                v[r] = __ldg(reinterpret_cast<const uint16_t *>(p + r * ld_bytes + lane * 2));
        }
#pragma unroll
        for (int r = 0; r < 32; ++r)
            *(reinterpret_cast<uint16_t *>(stage_slot(stage, r, lane >> 3)) + (lane & 7)) = v[r];
    }
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

// One warp's way out: the boxes of 32 columns make a set; a set's TMA stores
// are one group, and sets are used in turn.
template <class S>
struct Outlet {
    uint4 *stage;
    int lane;
    uint32_t n;  // sets used before

    __device__ __forceinline__ uint4 *box(int k) const { return stage + ((n % S::SETS) * S::BOXES + k) * 128; }

    // The set is free once its last stores have read it.
    __device__ __forceinline__ void begin() const
    {
        if (lane == 0)
            bulk_wait_read<S::SETS - 1>();
        __syncwarp();
    }

    __device__ __forceinline__ void put(int k, const uint32_t (&w)[16]) const { stage_put_row(box(k), lane, w); }

    // Between the last put() and the first store().
    __device__ __forceinline__ void filled() const
    {
        fence_proxy_async();
        __syncwarp();
    }

    template <int ES>
    __device__ __forceinline__ void store(int k, const CUtensorMap *map, bool tma, void *out, int64_t ld, int64_t row0,
                                          int64_t col, int64_t rows, int64_t cols) const
    {
        if (rows <= 0 || cols <= 0)
            return;
        if (!tma)
            stage_flush<ES>(box(k), lane, static_cast<char *>(out) + (row0 * ld + col) * ES, ld * ES,
                            rows > 32 ? 32 : (int)rows, cols * ES);
        else if (lane == 0)
            tma_store(map, smem_addr(box(k)), (int32_t)col, (int32_t)row0);
    }

    // One group per set, empty or not, so that begin() can count.
    __device__ __forceinline__ void end()
    {
        if (lane == 0)
            bulk_commit();
        ++n;
    }
};

// One warp's epilogue of 32 columns.  All of it is binary32; what leaves it
// is rounded to 16 bits once: C, gate and up are outputs of that type, and
// act(gate) * up, dgate and dup are operands of the products that follow,
// which the tensor cores take in 16 bits only.  (Against binary64 the results
// of two products are then off by 0.00029 in float16 and 0.0023 in bfloat16,
// relative in norm, where one rounding at the end leaves 0.00021 and 0.0017.)
// C in `r` (kGate: the gate in `r`, up in
// `r1`; kGateBwd: the kept gate and up in `wg` and `wu`, the set begun),
// rows row0 + lane, columns col .. col + 31 of the output.  `ready` runs when
// the results are in registers.
template <class S, int DT, int EPI, int NP, class Ready>
__device__ __forceinline__ void finish32(const ProductArgs<NP, EPI> &g, const Product &p, Outlet<S> &o, int64_t row0,
                                         int64_t col, const uint32_t (&r)[32], const uint32_t (&r1)[32],
                                         uint32_t (&wg)[16], uint32_t (&wu)[16], Ready ready)
{
    const int64_t rows = p.m - row0, cols = p.n - col;
    uint32_t w[16];
    auto f = [](uint32_t x) { return __uint_as_float(x); };
    if constexpr (EPI == kStore) {
        if (!g.out_f32) {
#pragma unroll
            for (int k = 0; k < 16; ++k)
                w[k] = pack2<DT>(f(r[2 * k]), f(r[2 * k + 1]));
            o.begin();
            o.put(0, w);
            o.filled();
            o.template store<2>(0, &p.c, p.c_tma, p.out, p.out_ld, row0, col, rows, cols);
            o.end();
        } else {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    w[k] = r[16 * half + k];
                o.begin();
                o.put(0, w);
                o.filled();
                o.template store<4>(0, &p.c, p.c_tma, p.out, p.out_ld, row0, col + 16 * half, rows, cols - 16 * half);
                o.end();
            }
        }
    } else {
        if constexpr (EPI == kGate) {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const float g0 = f(r[2 * k]), g1 = f(r[2 * k + 1]), u0 = f(r1[2 * k]), u1 = f(r1[2 * k + 1]);
                w[k] = pack2<DT>(activate(g.act, g0).value * u0, activate(g.act, g1).value * u1);
                wg[k] = pack2<DT>(g0, g1);
                wu[k] = pack2<DT>(u0, u1);
            }
            o.begin();
        } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const float2 gg = unpack2<DT>(wg[k]), uu = unpack2<DT>(wu[k]);
                const float c0 = f(r[2 * k]), c1 = f(r[2 * k + 1]);
                const Act t0 = activate(g.act, gg.x), t1 = activate(g.act, gg.y);
                w[k] = pack2<DT>(t0.value * uu.x, t1.value * uu.y);
                wg[k] = pack2<DT>(c0 * uu.x * t0.slope, c1 * uu.y * t1.slope);
                wu[k] = pack2<DT>(c0 * t0.value, c1 * t1.value);
            }
            ready();
        }
        const bool sides = EPI == kGateBwd || g.side[0].p;
        o.put(2, w);
        if (sides) {
            o.put(0, wg);
            o.put(1, wu);
        }
        o.filled();
        o.template store<2>(2, &p.c, p.c_tma, p.out, p.out_ld, row0, col, rows, cols);
        if (sides) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
                o.template store<2>(k, &g.side[EPI == kStore ? 0 : k].map, g.side[EPI == kStore ? 0 : k].tma,
                                    g.side[EPI == kStore ? 0 : k].p, g.side[EPI == kStore ? 0 : k].ld, row0, col, rows,
                                    cols);
        }
        o.end();
    }
}

// gate's and up's boxes of 32 columns without TMA: into the set and to the
// row of each lane.
template <class S, int NP>
__device__ __forceinline__ void fetch_sides(const ProductArgs<NP, kGateBwd> &g, const Product &p, const Outlet<S> &o,
                                            int64_t row0, int64_t col, uint32_t (&wg)[16], uint32_t (&wu)[16])
{
    const int64_t rows = p.m - row0, cols = p.n - col;
    o.begin();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const Side &sd = g.side[2 + k];
        stage_fetch(o.box(k), o.lane, static_cast<const char *>(sd.p) + (row0 * sd.ld + col) * 2, sd.ld * 2,
                    rows > 32 ? 32 : (int)rows, cols * 2, sd.vec);
    }
    __syncwarp();
    stage_get_row(o.box(0), o.lane, wg);
    stage_get_row(o.box(1), o.lane, wu);
    __syncwarp();
}

// NaN for 32 x 32 results whose sums (or gate and up) did not arrive in time:
// rows row0 + lane, columns from col on.  Plain stores, because a copy that is
// still on its way may yet land in the boxes.
template <int NP, int EPI>
__device__ __forceinline__ void give_up32(const ProductArgs<NP, EPI> &g, const Product &p, int lane, int64_t row0,
                                          int64_t col)
{
    const int64_t row = row0 + lane;
    const int cols = p.n - col < 32 ? (int)(p.n - col) : 32;
    if (row >= p.m)
        return;
    auto fill = [&](void *out, int64_t ld) {
#pragma unroll 1
        for (int c = 0; c < cols; ++c) {
            if (EPI == kStore && g.out_f32)
                static_cast<uint32_t *>(out)[row * ld + col + c] = 0x7fffffffu;
            else
                static_cast<uint16_t *>(out)[row * ld + col + c] = 0x7fffu;
        }
    };
    fill(p.out, p.out_ld);
    if (EPI != kStore && g.side[0].p)
#pragma unroll 1
        for (int k = 0; k < 2; ++k)
            fill(g.side[EPI == kStore ? 0 : k].p, g.side[EPI == kStore ? 0 : k].ld);
}

// Where a tile lies.
struct Tile {
    int32_t product, m, n;  // m, n: tile coordinates
};

// Tiles of a product go in groups of kRaster rows of tiles, column by column
// within a group, so that the tiles in flight share operands in L2.
constexpr int kRaster = 8;

template <int NP, int EPI>
__device__ __forceinline__ int32_t product_at(const ProductArgs<NP, EPI> &g, int32_t index)
{
    int32_t product = 0;
#pragma unroll
    for (int q = 1; q < NP; ++q)
        if (q < g.products && index >= g.p[q].first)
            product = q;
    return product;
}

template <class S, int NP, int EPI>
__device__ __forceinline__ Tile tile_at(const ProductArgs<NP, EPI> &g, int32_t index)
{
    Tile it;
    it.product = product_at(g, index);
    const Product &p = g.p[it.product];
    const int32_t t = index - p.first, tiles_m = (p.m - 1) / S::BM + 1, per = kRaster * p.tiles_n;
    const int32_t group = t / per, within = t - group * per;
    const int32_t rows = tiles_m - group * kRaster < kRaster ? tiles_m - group * kRaster : kRaster;
    it.n = within / rows;
    it.m = group * kRaster + (within - it.n * rows);
    return it;
}

// A product of two matrices, or of two pairs, and what is done with its
// elements.  One warp fills a ring of shared-memory stages by TMA, one thread
// issues the tcgen05 products into one of two accumulators in tensor memory,
// and the other warps empty the accumulator before it.  Large products run at
// the tensor cores' rate under the power limit, less what the last wave and
// tiles past the edge leave idle, and a 256 x 256 pair tile already takes all
// of the 64 bytes per clock that an SM can be fed.  Back to back, with the
// clock that the power limit leaves: 8192 tokens of 1600 x 6400 366 us forward
// (1.37 PFLOP/s), 743 us backward (1.35; the gate's backward epilogue moves
// five matrices), 2048 of 8192 x 32768 4.09 ms backward (1.61); in the first
// milliseconds, before that, 329 us, 703 us and 4.01 ms.
// Small ones are bounded by latency: a launch of one tile per SM takes 5 us
// beside its blocks of k (1000 clocks to start, 1500 to the first operands,
// 2000 for an epilogue, 500 to end).  With splits = 1 the grid is
// persistent and strides over the tiles.  With splits > 1 (one-CTA shapes, a
// grid of tiles * splits) the CTAs of a cluster share a tile's k: each leaves
// its sums in its shared memory, and each then adds up some 32 x 32 blocks
// of the tile over all of them, in order, and finishes them (all threads add,
// 16 bytes at a time, and then a warp finishes a block; a warp that also added
// up its block took 1 us longer).
template <class S, int DT, int EPI, int MAJ, int NP>
__global__ void __launch_bounds__(S::THREADS, S::PER_SM) k_ffn_product(const __grid_constant__ ProductArgs<NP, EPI> g)
{
    constexpr int CG = S::CG, BN = S::BN;
    constexpr int kStepN = EPI == kGate ? BN / 2 : BN;  // output columns per tile
    constexpr bool a_mn = MAJ == kMnMn, b_mn = MAJ != kKK;
    extern __shared__ unsigned char smem_raw[];
    __shared__ ProductShared sh;
    unsigned char *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023u)) & 1023u);
    unsigned char *out_area = smem + S::STAGES * S::STAGE;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool split = CG == 1 && g.splits > 1;
    const uint32_t rank = CG == 2 || split ? cluster_rank() : 0;
    const uint32_t half = CG == 2 ? rank : 0;  // which half of a pair's tile
    const int32_t workers = split ? g.tiles : gridDim.x / CG;
    const int32_t worker = split ? blockIdx.x / g.splits : blockIdx.x / CG;
    constexpr int kTma = S::EPI_WARPS, kMma = S::EPI_WARPS + 1;
    // this CTA's blocks of k in a product
    auto k_first = [&](const Product &p) { return split ? (int32_t)((int64_t)p.pairs * p.kb * rank / g.splits) : 0; };
    auto k_last = [&](const Product &p) {
        return split ? (int32_t)((int64_t)p.pairs * p.kb * (rank + 1) / g.splits) : p.pairs * p.kb;
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < g.stages; ++s) {
            mbar_init_count(&sh.full[s], 1);
            mbar_init_count(&sh.empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init_count(&sh.tfull[s], 1);
            mbar_init_count(&sh.tempty[s], CG * S::EPI_WARPS);
        }
        for (int s = 0; EPI == kGateBwd && s < S::SETS * S::EPI_WARPS; ++s)
            mbar_init_count(&sh.in[s], 1);
        sh.gave_up = 0;
        mbar_init_done();
    }
    if (warp == kMma)
        tmem_alloc<CG>(&sh.tmem, S::TMEM);
    if (warp == kTma && lane < g.products) {
        tma_prefetch_map(&g.p[lane].a[0]);
        tma_prefetch_map(&g.p[lane].b[0]);
    }
    tmem_fence_before();
    __syncthreads();
    if (CG == 2)
        cluster_sync();
    tmem_fence_after();
    const uint32_t tmem = sh.tmem;
    pdl_launch_next();
    pdl_wait();

    if (warp == kTma) {
        asm volatile("fence.proxy.async.global;" ::: "memory");
        const uint32_t a_bytes = a_mn ? S::A_BYTES : (uint32_t)g.a_rows * 128;
        const uint32_t ring = smem_addr(smem);
        uint32_t s = 0, phase = 1;  // the next stage; the phase that ends when it was read
        bool ok = true;
        for (int32_t i = worker; ok && i < g.tiles; i += workers) {
            const Tile it = tile_at<S>(g, i);
            const Product &p = g.p[it.product];
            const int32_t m0 = it.m * S::BM + (int32_t)half * 128, n0 = it.n * kStepN;
            const int32_t k1 = k_last(p);
            for (int32_t kb = k_first(p); kb < k1; ++kb) {
                if (!mbar_wait_warp(&sh.empty[s], phase, g.limit_ns, &sh.gave_up)) {
                    ok = false;
                    break;
                }
                const int pair = kb >= p.kb;
                const int32_t k = (kb - pair * p.kb) * 64;
                const uint32_t sa = ring + s * g.stage_bytes, sb = sa + a_bytes;
                // the leader's barrier counts the bytes of both CTAs
                uint32_t bar = smem_addr(&sh.full[s]);
                if (CG == 2)
                    bar = peer_addr(bar, 0);
                if (elect_one()) {
                    if (half == 0)
                        mbar_expect(&sh.full[s], CG * (a_bytes + S::B_BYTES));
                    if (a_mn) {
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            tma_load<CG>(sa + j * 8192, &p.a[pair], m0 + 64 * j, k, bar);
                    } else {
                        tma_load<CG>(sa, &p.a[pair], k, m0, bar);
                    }
                    if (EPI == kGate) {
                        if (CG == 2) {
                            tma_load<CG>(sb, &p.b[half], k, n0, bar);
                        } else {
                            tma_load<CG>(sb, &p.b[0], k, n0, bar);
                            tma_load<CG>(sb + S::B_BYTES / 2, &p.b[1], k, n0, bar);
                        }
                    } else if (b_mn) {
#pragma unroll
                        for (int j = 0; j < S::B_ROWS / 64; ++j)
                            tma_load<CG>(sb + j * 8192, &p.b[pair], n0 + (int32_t)half * S::B_ROWS + 64 * j, k, bar);
                    } else {
                        tma_load<CG>(sb, &p.b[pair], k, n0 + (int32_t)half * S::B_ROWS, bar);
                    }
                }
                __syncwarp();
                if (++s == (uint32_t)g.stages)
                    s = 0, phase ^= 1;
            }
        }
    } else if (warp == kMma) {
        if (half == 0) {
            constexpr uint32_t desc = product_desc(DT == ZERO_BF16, a_mn, b_mn, S::BM, BN);
            // 16 k further: 32 bytes of a row, or 16 rows of 128 bytes
            constexpr uint32_t step_a = a_mn ? 128 : 2, step_b = b_mn ? 128 : 2;
            const uint32_t a_bytes = a_mn ? S::A_BYTES : (uint32_t)g.a_rows * 128;
            const uint64_t a0 = operand_desc(smem_addr(smem), a_mn ? 8192 : 16, 1024);
            const uint64_t b0 = operand_desc(smem_addr(smem) + a_bytes, b_mn ? 8192 : 16, 1024);
            uint32_t s = 0, phase = 0, t = 0;
            bool ok = true;
            for (int32_t i = worker; ok && i < g.tiles; i += workers, ++t) {
                const Product &p = g.p[product_at(g, i)];
                const uint32_t acc = t & 1;
                if (!mbar_wait_warp(&sh.tempty[acc], ((t >> 1) & 1) ^ 1, g.limit_ns, &sh.gave_up))
                    break;
                tmem_fence_after();
                const uint32_t d = tmem + acc * BN;
                const int32_t k0 = k_first(p), k1 = k_last(p);
                for (int32_t kb = k0; kb < k1; ++kb) {
                    if (!mbar_wait_warp(&sh.full[s], phase, g.limit_ns, &sh.gave_up)) {
                        ok = false;
                        break;
                    }
                    tmem_fence_after();
                    const uint64_t da = a0 + ((s * g.stage_bytes) >> 4), db = b0 + ((s * g.stage_bytes) >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            tensor_product<CG>(d, da + k * step_a, db + k * step_b, desc, kb != k0 || k != 0);
                        tensor_commit<CG>(&sh.empty[s]);
                    }
                    __syncwarp();
                    if (++s == (uint32_t)g.stages)
                        s = 0, phase ^= 1;
                }
                if (ok && elect_one())
                    tensor_commit<CG>(&sh.tfull[acc]);
                __syncwarp();
            }
        }
    } else {
        const int quarter = warp & 3, part = warp >> 2;  // lanes 32 * quarter on; this warp's share of the columns
        constexpr int kParts = S::EPI_WARPS / 4, kCols = kStepN / kParts;  // output columns per warp
        Outlet<S> o{reinterpret_cast<uint4 *>(out_area + warp * S::WARP_OUT), lane, 0};
        // kGateBwd: gate's and up's boxes arrive by TMA in the set that their
        // results leave from, asked for one set ahead
        const bool in_tma = EPI == kGateBwd && !split && g.side[EPI == kGateBwd ? 2 : 0].tma;
        int32_t ask_i = worker, ask_c = 0;
        uint32_t asked = 0;
        auto ask = [&] {
            if (EPI != kGateBwd || !in_tma || ask_i >= g.tiles)
                return;
            const Tile it = tile_at<S>(g, ask_i);
            if (lane == 0) {
                const uint32_t b = asked % S::SETS;
                uint64_t *bar = &sh.in[warp * S::SETS + b];
                const uint32_t dst = smem_addr(o.stage + b * S::BOXES * 128);
                const int32_t row = it.m * S::BM + (int32_t)half * 128 + quarter * 32;
                const int32_t col = it.n * kStepN + part * kCols + ask_c;
                bulk_wait_read<0>();  // the set's last stores have read it
                mbar_expect(bar, 4096);
                tma_load<1>(dst, &g.side[EPI == kGateBwd ? 2 : 0].map, col, row, smem_addr(bar));
                tma_load<1>(dst + 2048, &g.side[EPI == kGateBwd ? 3 : 0].map, col, row, smem_addr(bar));
            }
            ++asked;
            ask_c += 32;
            if (ask_c >= kCols) {
                ask_c = 0;
                ask_i += workers;
            }
        };
        ask();
        uint32_t t = 0;
        bool ok = true;
        for (int32_t i = worker; i < g.tiles; i += workers, ++t) {
            const Tile it = tile_at<S>(g, i);
            const Product &p = g.p[it.product];
            const uint32_t acc = t & 1;
            const int64_t row0 = (int64_t)it.m * S::BM + half * 128 + quarter * 32;
            const int64_t col0 = (int64_t)it.n * kStepN + part * kCols;
            // a wait that gave up makes this and every later tile NaN
            ok = ok && mbar_wait_bounded(&sh.tfull[acc], (t >> 1) & 1, g.limit_ns, &sh.gave_up);
            ok = __all_sync(0xffffffffu, ok);
            tmem_fence_after();
            const uint32_t from = tmem + acc * BN + ((uint32_t)(quarter * 32) << 16) + part * kCols;
            uint32_t r[32], r1[32], wg[16], wu[16];
#pragma unroll 1
            for (int c = 0; c < kCols; c += 32) {
                if constexpr (EPI == kGateBwd) {
                    if (in_tma) {
                        ok = ok && mbar_wait_bounded(&sh.in[warp * S::SETS + o.n % S::SETS], (o.n / S::SETS) & 1,
                                                     g.limit_ns, &sh.gave_up);
                        ok = __all_sync(0xffffffffu, ok);
                        if (ok) {
                            stage_get_row(o.box(0), lane, wg);
                            stage_get_row(o.box(1), lane, wu);
                        }
                        if (S::SETS == 1)
                            __syncwarp();
                    } else if (!split && ok) {
                        fetch_sides<S, NP>(g, p, o, row0, col0 + c, wg, wu);
                    }
                }
                if (ok) {
                    tmem_load32(from + c, r);
                    if (EPI == kGate)
                        tmem_load32(from + BN / 2 + c, r1);
                    tmem_wait_loads(r);
                    if (EPI == kGate)
                        tmem_wait_loads(r1);
                } else if (!split) {
                    give_up32(g, p, lane, row0, col0 + c);
                }
                if (c + 32 >= kCols) {
                    tmem_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive_cluster(CG == 2 ? peer_addr(smem_addr(&sh.tempty[acc]), 0)
                                                    : smem_addr(&sh.tempty[acc]));
                }
                if (!ok)
                    continue;
                if (split) {
                    // this CTA's sums: [column][row] over the stages, which the products have read
                    float *sums = reinterpret_cast<float *>(smem) + (part * kCols + c) * 128 + quarter * 32 + lane;
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        sums[k * 128] = __uint_as_float(r[k]);
                        if (EPI == kGate)
                            sums[(BN / 2 + k) * 128] = __uint_as_float(r1[k]);
                    }
                } else {
                    // (with one set the next is asked for when this one has left it)
                    finish32<S, DT, EPI, NP>(g, p, o, row0, col0 + c, r, r1, wg, wu, [&] {
                        if (S::SETS > 1)
                            ask();
                    });
                    if (S::SETS == 1)
                        ask();
                }
            }
        }
        if (lane == 0)
            bulk_wait_read<0>();
    }

    __syncwarp();
    if (split) {
        cluster_sync();
        const Tile it = tile_at<S>(g, worker);
        const Product &p = g.p[it.product];
        const int64_t m0 = (int64_t)it.m * S::BM, left = p.m - m0;
        // blocks of 32 x 32: quarter q of the rows, 32 columns from c on; every
        // splits-th of them is this CTA's, and all of its threads add it up
        // over the cluster, four rows at a time, in order, in its own memory
        const int quarters = left >= 128 ? 4 : (int)((left + 31) / 32), blocks = quarters * (kStepN / 32);
        constexpr int kPieces = EPI == kGate ? 512 : 256;
        const int pieces = (blocks - (int)rank + g.splits - 1) / g.splits * kPieces;
        // a CTA that gave up has left no sums
        const uint32_t late = threadIdx.x < (unsigned)g.splits ? load_peer1(peer_addr(smem_addr(&sh.gave_up), threadIdx.x)) : 0;
#pragma unroll 2
        for (int v = threadIdx.x; v < pieces; v += S::THREADS) {
            const int u = (int)rank + v / kPieces * g.splits, e = v % kPieces;
            const int column = u / quarters * 32 + (e >> 3 & 31) + (e >> 8) * (BN / 2);
            float4 *sums = reinterpret_cast<float4 *>(smem) + column * 32 + u % quarters * 8 + (e & 7);
            const uint32_t at = smem_addr(sums);
            float4 sum = load_peer4(peer_addr(at, 0));
#pragma unroll
            for (int j = 1; j < kMostParts; ++j)
                if (j < g.splits) {
                    const float4 x = load_peer4(peer_addr(at, j));
                    sum.x += x.x, sum.y += x.y, sum.z += x.z, sum.w += x.w;
                }
            *sums = sum;
        }
        const bool ok = !__syncthreads_or(late);
        if (warp < S::EPI_WARPS) {
            Outlet<S> o{reinterpret_cast<uint4 *>(out_area + warp * S::WARP_OUT), lane, 0};
            for (int u = (int)rank + warp * g.splits; u < blocks; u += S::EPI_WARPS * g.splits) {
                const int q = u % quarters, c = u / quarters * 32;
                const int64_t row0 = m0 + q * 32, col = (int64_t)it.n * kStepN + c;
                if (!ok) {
                    give_up32(g, p, lane, row0, col);
                    continue;
                }
                const uint32_t *sums = reinterpret_cast<const uint32_t *>(smem) + c * 128 + q * 32 + lane;
                uint32_t r[32], r1[32], wg[16], wu[16];
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    r[k] = sums[k * 128];
                    if (EPI == kGate)
                        r1[k] = sums[(BN / 2 + k) * 128];
                }
                if constexpr (EPI == kGateBwd)
                    fetch_sides<S, NP>(g, p, o, row0, col, wg, wu);
                finish32<S, DT, EPI, NP>(g, p, o, row0, col, r, r1, wg, wu, [] {});
            }
            if (lane == 0)
                bulk_wait_read<0>();
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
    if (CG == 2 || split)
        cluster_sync();
    if (warp == kMma)
        tmem_free<CG>(tmem, S::TMEM);
}

// ------------------------------------------------------------- a few tokens

// Products for one or two tokens (up to four where the widths are no multiples
// of 8 and the tensor cores would need copies), where the weights' bytes are
// all there is: a warp per row of the weight matrix (kPair: of the gate's and
// the up matrix together), or `parts` warps of a block that each take a
// stretch of k and add up in order through shared memory.  A lane multiplies
// 16-byte pieces of the row with the tokens' pieces (which stay in L1) in
// binary32; four pieces of each row are in flight per lane.  1600 x 6400, one
// token: 17.6 us for both products, 3.5 TB/s of weights: each is a launch and
// a few trips to memory long, so the time is latency as much as bytes.  Rows
// that start anywhere cost two loads and a shift per piece, registers and
// blocks with them: 1001 x 2731, one token: 9.9 us, four: 15.6 (21.7 by copies
// and tiles; eight tokens this way 25.0, so tiles take over).
struct TokenArgs {
    const void *x;  // tokens x k, row stride x_ld (kPair: of the weights' type; else binary32)
    int64_t x_ld;
    const void *w0, *w1;  // n x k, contiguous
    void *out;            // kPair: act(C0) * C1 in binary32; else C0; tokens x n, row stride out_ld
    int64_t out_ld;
    void *o0, *o1;        // kPair: C0 and C1, kept (or NULL), contiguous
    int32_t tokens, n, k, parts, act;
};

// Eight elements of a row that may start anywhere come out of the two aligned
// 16 bytes that hold them, where those lie in the matrix (lo to hi).  The
// loads stand apart from the shifts, so that several are on their way at once.
struct Window {
    uint4 a, b;
    bool in;
};

__device__ __forceinline__ Window load_window(const uint16_t *src, const uint16_t *lo, const uint16_t *hi)
{
    const uint16_t *base = src - ((uint32_t)(reinterpret_cast<uintptr_t>(src) >> 1) & 7);
    Window x{{}, {}, base >= lo && base + 16 <= hi};
    if (x.in) {
        x.a = __ldg(reinterpret_cast<const uint4 *>(base));
        x.b = __ldg(reinterpret_cast<const uint4 *>(base) + 1);
    }
    return x;
}

// p[i] to p[i + 7], zeros from k on.
__device__ __forceinline__ uint4 shifted_piece(const Window &x, const uint16_t *p, int64_t i, int64_t k)
{
    const uint32_t v[8] = {x.a.x, x.a.y, x.a.z, x.a.w, x.b.x, x.b.y, x.b.z, x.b.w};
    const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(p + i) >> 1) & 7, bits = (off & 1) * 16;
    uint32_t w[4] = {};
#pragma unroll
    for (uint32_t o = 0; o < 4; ++o)  // (most often the same for a whole warp)
        if (off >> 1 == o) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                w[e] = __funnelshift_r(v[o + e], v[o + e + 1 < 8 ? o + e + 1 : 7], bits);
        }
    if (!x.in) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            w[e] = (i + 2 * e < k ? p[i + 2 * e] : 0u) | (i + 2 * e + 1 < k ? (uint32_t)p[i + 2 * e + 1] << 16 : 0u);
    } else if (i + 8 > k) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            w[e] = i + 2 * e + 1 < k ? w[e] : i + 2 * e < k ? w[e] & 0xffffu : 0u;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

constexpr int token_blocks(int tokens, bool whole) { return tokens == 1 ? 4 : whole ? 3 : 2; }

template <int DT, int MT, bool kPair, bool kW>
__global__ void __launch_bounds__(kThreads, token_blocks(MT, kW))
    k_ffn_tokens(const __grid_constant__ TokenArgs a)
{
    constexpr int R = kPair ? 2 : 1, U = kW ? 4 : MT == 1 ? 1 : 2;
    constexpr bool kX = kW || MT > 2;  // x's rows are whole 16 bytes too (zeros past k)
    __shared__ float s_part[kWarps][R * MT];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per_block = kWarps / a.parts, unit = warp / a.parts, part = warp - unit * a.parts;
    const int32_t pieces = (a.k + 7) >> 3;  // of a row
    const int32_t p0 = (int32_t)((int64_t)pieces * part / a.parts), p1 = (int32_t)((int64_t)pieces * (part + 1) / a.parts);
    bool waited = false;
    pdl_launch_next();
    // (unsigned: a matrix may have 2^31 - 512 rows, and a step goes past them)
    const uint32_t rows = a.n;
    for (uint32_t n0 = blockIdx.x * per_block; n0 < rows; n0 += gridDim.x * per_block) {
        const uint32_t n = n0 + unit;
        float acc[R][MT] = {};
        if (n < rows) {
            const uint16_t *const first[2] = {static_cast<const uint16_t *>(a.w0), static_cast<const uint16_t *>(kPair ? a.w1 : a.w0)};
            const uint16_t *const w[2] = {first[0] + (int64_t)n * a.k, first[1] + (int64_t)n * a.k};
            for (int32_t i = p0 + lane; i < p1; i += 32 * U) {
                uint4 wv[kW ? U : 1][R];
                Window win[kW ? 1 : U][R];
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int q = 0; q < R; ++q)
                        if (i + 32 * u < p1)
                            if constexpr (kW)
                                wv[u][q] = __ldg(reinterpret_cast<const uint4 *>(w[q]) + i + 32 * u);
                            else
                                win[u][q] = load_window(w[q] + (i + 32 * u) * 8, first[q], first[q] + (int64_t)a.n * a.k);
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
                    for (int q = 0; q < R; ++q) {
                        if constexpr (!kW)
                            wv[0][q] = shifted_piece(win[u][q], w[q], (i + 32 * u) * 8, a.k);
                        Elem<DT>::to_float(&wv[kW ? u : 0][q], wf[q]);
                    }
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        const int64_t row = (m < a.tokens ? m : a.tokens - 1) * a.x_ld;
                        float xf[8];
                        if (kPair) {
                            const uint16_t *px = static_cast<const uint16_t *>(a.x);
                            const int32_t c = (i + 32 * u) * 8;
                            uint4 xv;
                            if constexpr (kX)
                                xv = reinterpret_cast<const uint4 *>(px + row)[i + 32 * u];
                            else
                                xv = shifted_piece(load_window(px + row + c, px, px + (a.tokens - 1) * a.x_ld + a.k), px + row, c, a.k);
                            Elem<DT>::to_float(&xv, xf);
                        } else {  // rows of whole 32 bytes; past k they meet zeros
                            const float4 *xv = reinterpret_cast<const float4 *>(static_cast<const float *>(a.x) + row) +
                                               (i + 32 * u) * 2;
                            const float4 lo = xv[0], hi = xv[1];
                            xf[0] = lo.x, xf[1] = lo.y, xf[2] = lo.z, xf[3] = lo.w;
                            xf[4] = hi.x, xf[5] = hi.y, xf[6] = hi.z, xf[7] = hi.w;
                            if (!kW)
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    xf[e] = (i + 32 * u) * 8 + e < a.k ? xf[e] : 0.0f;
                        }
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
        if (part == 0 && n < rows && lane == 0) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
                if (m < a.tokens) {
                    if (kPair) {
                        static_cast<float *>(a.out)[m * a.out_ld + n] = activate(a.act, acc[0][m]).value * acc[R - 1][m];
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

// Rows of 16-bit elements copied to rows of whole 16 bytes, which TMA asks
// for (widths that no vector divides): up to five matrices in one launch,
// bounded by memory (75 MB of weights: 32 us, 4.7 TB/s read and written).  It
// is most of a call on few tokens and little of one on thousands.
struct Copy {
    const uint16_t *src;
    uint16_t *dst;
    int64_t rows, cols, src_ld, dst_ld, first;  // first: the matrix's first 8-element group in the launch
    FastDiv per;                                // 8-element groups of a row
};

struct Copies {
    Copy c[5];
    int32_t n;
    int64_t groups;
};

__global__ void __launch_bounds__(kThreads) k_ffn_copy(const __grid_constant__ Copies a)
{
    pdl_launch_next();
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < a.groups; i += (int64_t)gridDim.x * kThreads) {
        int q = 0;
#pragma unroll
        for (int j = 1; j < 5; ++j)
            if (j < a.n && i >= a.c[j].first)
                q = j;
        const Copy &c = a.c[q];
        const int64_t at = i - c.first, per = c.dst_ld >> 3;
        const int64_t r = a.groups < kFastDivMost ? fast_div((uint32_t)at, c.per) : at / per, col = (at - r * per) * 8;
        const uint16_t *row = c.src + r * c.src_ld;
        *reinterpret_cast<uint4 *>(c.dst + r * c.dst_ld + col) =
            shifted_piece(load_window(row + col, c.src, c.src + (c.rows - 1) * c.src_ld + c.cols), row, col, c.cols);
    }
}

// ------------------------------------------------------------- host side

constexpr int64_t kMostSize = ((int64_t)1 << 31) - 512;
constexpr int kSms = 152;

// Pairs of CTAs with 256 x 256 tiles for large products; one-CTA tiles of
// 128 x 128, and of 128 x 64 with two CTAs per SM, for small ones.  The gate's
// epilogues fill three boxes per set, at the cost of stages.
template <int EPI>
using Pair256 = Shape<2, 256, EPI == kStore ? 6 : 4, 8, EPI == kStore ? 1 : 3, 2>;
template <int EPI>
using One128 = Shape<1, 128, 4, 8, EPI == kStore ? 1 : 3, 2>;
template <int EPI>
using One64 = Shape<1, 64, 3, 4, EPI == kStore ? 1 : 3, EPI == kStore ? 2 : 1>;

// Up to here a warp per weight row is faster than tensor-core tiles, which
// hold 128 tokens or a fraction (1600 x 6400, one, two and four tokens: 18, 21
// and 31 us here, 27 us in tiles; widths that need copies for tiles, 3423 x
// 1147, four tokens: 20.7 here, 28.5 in tiles).
constexpr int few_tokens(bool whole) { return whole ? 2 : 4; }

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

// How a launch is cut: its shape and the parts of k.
enum Cut { kPair256, kOne128, kOne64 };
struct Plan {
    Cut cut;
    int splits;
};

// Clusters of one to eight CTAs that the GPU holds at once, one and two CTAs to
// an SM (as cudaOccupancyMaxActiveClusters tells): its SMs come in groups that
// a cluster does not cross.
constexpr int kClusters[2][kMostParts] = {{152, 76, 46, 36, 28, 23, 15, 15}, {304, 152, 97, 74, 58, 46, 38, 36}};

// The cheapest cut by an estimate of a launch's time in ns: a start (with the
// epilogue of the last tile), and per wave of tiles and block of k the larger
// of the issue's time and the tile bytes' through L2.  Its constants were
// fitted to 1344 launches (tokens 5 to 1000, widths 256 to 8192, all cuts);
// the cut it takes is on average 1.7 % slower than the best, at worst 23 %.
// One launch each, measured: 1000 tokens, 4096 x 4096: pairs 26 us, 128 x 128
// tiles 44, 128 x 64 88; 64 tokens, 6400 to 1600: 33, 28 and 26 us whole, 13.0
// and 12.3 us with k in four parts, 10.8 us for 128 x 128 tiles in eight;
// the backward pass of 3125 tokens, 704 x 256: 32.6 us with the three weight
// gradients whole, 28.3 with their k in parts.
Plan plan_product(int64_t m, int64_t n, int64_t k, bool gate, int most_parts)
{
    const int64_t cols = n * (gate ? 2 : 1), kb = cdiv(k, 64);
    const double a_bytes = (double)(m < 128 ? up8(m) : 128) * 128;
    auto larger = [](double a, double b) { return a > b ? a : b; };
    const int64_t pairs = cdiv(m, 256) * cdiv(cols, 256), pair_slots = kSms / 2;
    const double pair_bytes = 65536.0 * (double)(pairs < pair_slots ? pairs : pair_slots);
    Plan best{kPair256, 1};
    double least = 9500 + (double)cdiv(pairs, pair_slots) * kb * larger(285, pair_bytes / 12600);
    for (int c = 0; c < 2; ++c) {
        const int bn = c == 0 ? 128 : 64;
        const int64_t all = cdiv(m, 128) * cdiv(cols, bn);
        if (all > 1 << 24)  // (pairs, by far; and what follows fits 32 bits)
            continue;
        const int tiles = (int)all, blocks = (int)kb, most = blocks < most_parts ? blocks : most_parts;
        for (int parts = 1; parts <= most; ++parts) {
            if (parts == 7)  // clusters of seven started late: 9 tokens, 2731 to 1001: 16 us, five parts 9
                continue;
            const int ctas = tiles * parts, slots = parts * kClusters[c][parts - 1], waves = (ctas - 1) / slots + 1;
            const double bytes = (double)(ctas < slots ? ctas : slots) * (a_bytes + bn * 128);
            const double block = c == 0 ? larger(207, bytes / 14000) : larger(137, bytes / 8400);
            double t = 6400 + (double)waves * ((blocks - 1) / parts + 1) * block;
            if (parts > 1)  // joining the parts; and each wave is a new set of CTAs
                t += 1100 + 130 * parts + 7700.0 * (waves - 1);
            if (t < least)
                least = t, best = {c == 0 ? kOne128 : kOne64, parts};
        }
    }
    return best;
}

struct FfnSpace {
    size_t mats, mat_bytes, copies, total;
};

// Workspace: the header, the matrices that a call keeps between its products,
// and copies of operands whose rows are not whole 16 bytes.
FfnSpace ffn_space(int64_t m, int64_t d, int64_t f, bool backward)
{
    FfnSpace s{};
    s.mats = 256;
    // (a few tokens' act(gate) * up stays in binary32; the matrix of more tokens
    // has that much room too, so that a workspace for many serves fewer)
    const int64_t few = few_tokens(((d | f) & 7) == 0), wide = m < few ? m : few;
    const int64_t elems = !backward && m < 2 * wide ? 2 * wide : m;
    s.mat_bytes = align256((size_t)elems * (size_t)up8(f) * 2);
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

// Operands whose rows are not whole 16 bytes (`zeros`: nor followed by zeros
// up to the next 16), copied to the workspace; the matrices then name the
// copies.
int copy_operands(Mat **mats, int n, char *to, bool *copied, bool zeros, cudaStream_t st)
{
    *copied = false;
    Copies a{};
    for (int i = 0; i < n; ++i) {
        Mat &m = *mats[i];
        const int64_t ld = up8(m.cols);
        if (m.rows == 0 || m.cols == 0)
            continue;
        if (aligned16(m.p) && (m.ld & 7) == 0 && !(zeros && (m.cols & 7) != 0))
            continue;
        Copy &c = a.c[a.n++];
        c = {static_cast<const uint16_t *>(m.p), reinterpret_cast<uint16_t *>(to), m.rows, m.cols, m.ld, ld, a.groups,
             fast_divisor((uint32_t)(ld / 8))};
        a.groups += m.rows * (ld / 8);
        m.p = to;
        m.ld = ld;
        to += align256((size_t)m.rows * ld * 2);
    }
    if (a.n == 0)
        return ZERO_OK;
    *copied = true;
    k_ffn_copy<<<grid_for(reinterpret_cast<const void *>(k_ffn_copy), cdiv(a.groups, kThreads), 1 << 30), kThreads, 0,
                 st>>>(a);
    return check_launch("k_ffn_copy");
}

// For tests: products whose epilogue is test_short ask for boxes of A eight
// rows too low, so that no block of k is ever whole and their waits run out
// after test_limit_ns, in the calls of the thread that set it and in no
// other's.
thread_local int32_t test_short = -1;
thread_local uint64_t test_limit_ns = 0;

// One product of a launch.
struct Spec {
    Mat a[2], b[2];
    int pairs;
    int64_t m, n, k;
    void *out;
    int64_t out_ld;
    int64_t out_cols;  // n, or a matrix of the workspace's padded width (the columns past n get zeros)
};

// Whether TMA may write a matrix: it writes whole 16 bytes, so rows must be.
bool tma_ready(const void *p, int64_t rows, int64_t cols, int64_t ld, int es)
{
    return aligned16(p) && (cols * es) % 16 == 0 && (rows == 1 || (ld * es) % 16 == 0) && ld < (int64_t)1 << 38;
}

// An output (or side matrix) in boxes of 32 rows by 64 bytes.
int box_map(CUtensorMap *map, int32_t *tma, const void *p, int64_t rows, int64_t cols, int64_t ld, int32_t dtype)
{
    const int es = elem_bytes(dtype);
    *tma = tma_ready(p, rows, cols, ld, es);
    return *tma ? tensor_map(map, p, rows, cols, rows == 1 ? cols : ld, 64 / es, 32, dtype) : ZERO_OK;
}

int side_matrix(Side *s, const void *p, int64_t rows, int64_t cols, int64_t ld, int32_t dtype)
{
    s->p = const_cast<void *>(p);
    s->ld = ld;
    s->vec = aligned16(p) && (cols & 7) == 0 && (ld & 7) == 0;
    return p ? box_map(&s->map, &s->tma, p, rows, cols, ld, dtype) : ZERO_OK;
}

template <class S, int DT, int EPI, int MAJ, int NP>
int launch_products(const Spec *specs, int n, ProductArgs<NP, EPI> &g, int splits, bool chained, int32_t dtype,
                    cudaStream_t st)
{
    constexpr bool gate = EPI == kGate, a_mn = MAJ == kMnMn, b_mn = MAJ != kKK;
    g.splits = splits;
    g.products = n;
    const int64_t m0 = specs[0].m;
    g.a_rows = S::CG == 1 && n == 1 && m0 < 128 ? (int)up8(m0) : 128;
    // With few rows of A the ring's memory holds more, smaller stages (the
    // products still read 128 rows; what lies past a_rows lands in rows of the
    // accumulator that no one reads).
    g.stage_bytes = g.a_rows * 128 + S::B_BYTES;
    g.stages = S::STAGES * S::STAGE / g.stage_bytes;
    g.stages = g.stages < kMaxStages ? g.stages : kMaxStages;
    const bool fails = test_short == EPI;
    const int a_box = (a_mn ? 64 : g.a_rows) - (fails ? 8 : 0);
    int64_t tiles = 0, longest = 0;
    for (int q = 0; q < n; ++q) {
        const Spec &s = specs[q];
        Product &p = g.p[q];
        for (int i = 0; i < (gate ? 1 : s.pairs); ++i)
            ZERO_TRY(tensor_map(&p.a[i], s.a[i].p, s.a[i].rows, s.a[i].cols, s.a[i].ld, 64, a_box, dtype));
        for (int i = 0; i < (gate ? 2 : s.pairs); ++i)
            ZERO_TRY(tensor_map(&p.b[i], s.b[i].p, s.b[i].rows, s.b[i].cols, s.b[i].ld, 64,
                                b_mn ? 64 : gate && S::CG == 1 ? S::BN / 2 : S::B_ROWS, dtype));
        p.pairs = s.pairs, p.kb = (int32_t)cdiv(s.k, 64), p.m = (int32_t)s.m, p.n = (int32_t)s.n;
        p.tiles_n = (int32_t)cdiv(s.n, gate ? S::BN / 2 : S::BN);
        p.first = (int32_t)tiles;
        p.out = s.out, p.out_ld = s.out_ld;
        ZERO_TRY(box_map(&p.c, &p.c_tma, s.out, s.m, s.out_cols, s.out_ld, EPI == kStore && g.out_f32 ? ZERO_F32 : dtype));
        tiles += cdiv(s.m, S::BM) * p.tiles_n;
        longest = s.pairs * (int64_t)p.kb > longest ? s.pairs * (int64_t)p.kb : longest;
    }
    if (tiles * splits > 0x3fffffff)
        return ZERO_ESIZE;
    g.tiles = (int32_t)tiles;
    g.limit_ns = fails ? test_limit_ns : 2000000000ull + (uint64_t)longest * 4000;
    auto kernel = k_ffn_product<S, DT, EPI, MAJ, NP>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    const int64_t workers = (int64_t)sm_count() / S::CG * S::PER_SM;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(splits > 1 ? tiles * splits : (tiles < workers ? tiles : workers) * S::CG));
    cfg.blockDim = dim3(S::THREADS);
    cfg.dynamicSmemBytes = S::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    cfg.attrs = attr;
    if (S::CG == 2 || splits > 1) {
        cudaLaunchAttribute &c = attr[cfg.numAttrs++];
        c.id = cudaLaunchAttributeClusterDimension;
        c.val.clusterDim.x = S::CG == 2 ? 2 : splits;
        c.val.clusterDim.y = c.val.clusterDim.z = 1;
    }
    if (chained) {
        cudaLaunchAttribute &c = attr[cfg.numAttrs++];
        c.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        c.val.programmaticStreamSerializationAllowed = 1;
    }
    if (e == cudaSuccess)
        e = cudaLaunchKernelEx(&cfg, kernel, g);
    if (e != cudaSuccess) {
        cudaGetLastError();
        set_cuda_error("k_ffn_product", (int)e, cudaGetErrorString(e));
        return ZERO_ECUDA;
    }
    return ZERO_OK;
}

// chained: the launch before is this call's own, and this one may be
// scheduled while it ends.
template <int EPI, int MAJ, int NP>
int products(const Spec *specs, int n, ProductArgs<NP, EPI> &g, Plan plan, bool chained, int32_t dtype, cudaStream_t st)
{
    const bool f16 = dtype == ZERO_F16;
#define ZERO_CUT(S)                                                                                              \
    (f16 ? launch_products<S<EPI>, ZERO_F16, EPI, MAJ, NP>(specs, n, g, plan.splits, chained, dtype, st)              \
         : launch_products<S<EPI>, ZERO_BF16, EPI, MAJ, NP>(specs, n, g, plan.splits, chained, dtype, st))
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

// ------------------------------------------------------------- a few tokens

// Warps per weight row: one per 2048 of k (8192 x 32768, one token: 240 us; a
// warp for whole rows 293), and more, down to 512 of k each, while there are
// too few rows to give every SM 32 warps.
int token_parts(int64_t n, int64_t k)
{
    int parts = 1;
    while (parts < kWarps && (k > (int64_t)parts * 2048 ||
                              (n * parts < (int64_t)kSms * 32 && k >= (int64_t)parts * 2 * 512)))
        parts *= 2;
    return parts;
}

template <int DT, bool kPair>
int token_product(TokenArgs &a, bool whole, bool chained, cudaStream_t st)
{
    a.parts = token_parts(a.n, a.k);
    const int64_t units = cdiv(a.n, kWarps / a.parts), most = (int64_t)sm_count() * token_blocks(a.tokens, whole);
    const int grid = (int)(units < most ? units : most);
    cudaError_t e;
#define ZERO_MT(MT)                                                                                            \
    (whole ? launch_k(k_ffn_tokens<DT, MT, kPair, true>, grid, kThreads, st, chained, a)                        \
           : launch_k(k_ffn_tokens<DT, MT, kPair, false>, grid, kThreads, st, chained, a))
    if (a.tokens == 1)
        e = ZERO_MT(1);
    else if (a.tokens == 2)
        e = ZERO_MT(2);
    else  // (widths that no 16 bytes divide)
        e = launch_k(k_ffn_tokens<DT, 4, kPair, false>, grid, kThreads, st, chained, a);
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
                   bool copied, cudaStream_t st)
{
    TokenArgs a{};
    a.x = x, a.x_ld = x_ld, a.w0 = wg, a.w1 = wu, a.out = h, a.out_ld = up8(inner), a.o0 = gate, a.o1 = up;
    a.tokens = tokens, a.n = inner, a.k = dim, a.act = act;
    ZERO_TRY((token_product<DT, true>(a, whole, copied, st)));
    TokenArgs b{};
    b.x = h, b.x_ld = up8(inner), b.w0 = wd, b.out = y, b.out_ld = y_ld;
    b.tokens = tokens, b.n = dim, b.k = inner;
    return token_product<DT, false>(b, whole, true, st);
}

}  // namespace
}  // namespace zpml

using namespace zpml;

// For tests, and so not in the header: see test_short.  epilogue: 0 the
// products that store, 1 the gate's, 2 the gate's backward; -1 none (the
// default).
extern "C" void zero_test_gated_ffn_waits(int32_t epilogue, uint64_t limit_ns)
{
    test_short = epilogue;
    test_limit_ns = limit_ns;
}

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
    if (tokens <= few_tokens(whole)) {
        Mat mx{x, tokens, dim, x_ld}, *only[] = {&mx};
        bool copied = false;
        if (tokens > 2 && !whole)
            ZERO_TRY(copy_operands(only, 1, base + sp.copies, &copied, true, st));
        return (dtype == ZERO_F16 ? tokens_forward<ZERO_F16> : tokens_forward<ZERO_BF16>)(
            mx.p, mx.ld, w_gate, w_up, w_down, y, y_ld, gate, up, (int32_t)tokens, (int32_t)dim, (int32_t)inner, act,
            base + sp.mats, whole, copied, st);
    }
    Mat mx{x, tokens, dim, x_ld}, mg{w_gate, inner, dim, dim}, mu{w_up, inner, dim, dim};
    Mat md{w_down, dim, inner, inner};
    bool copied = false;
    if (!whole) {
        Mat *all[] = {&mx, &mg, &mu, &md};
        ZERO_TRY(copy_operands(all, 4, base + sp.copies, &copied, false, st));
    }
    const Mat h{base + sp.mats, tokens, inner, up8(inner)};
    ProductArgs<1, kGate> g{};
    g.hdr = static_cast<WsHeader *>(ws);
    g.act = act;
    ZERO_TRY(side_matrix(&g.side[0], gate, tokens, inner, inner, dtype));
    ZERO_TRY(side_matrix(&g.side[1], up, tokens, inner, inner, dtype));
    const Spec s1{{mx, mx}, {mg, mu}, 1, tokens, inner, dim, const_cast<void *>(h.p), h.ld, h.ld};
    ZERO_TRY((products<kGate, kKK, 1>(&s1, 1, g, plan_product(tokens, inner, dim, true, kMostParts), copied, dtype, st)));
    ProductArgs<1, kStore> d{};
    d.hdr = g.hdr;
    const Spec s2{{h, h}, {md, md}, 1, tokens, dim, inner, y, y_ld, dim};
    return products<kStore, kKK, 1>(&s2, 1, d, plan_product(tokens, dim, inner, false, kMostParts), true, dtype, st);
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
    bool copied = false;
    if (!whole) {
        Mat *all[] = {&my, &mx, &mg, &mu, &md};
        ZERO_TRY(copy_operands(all, 5, base + sp.copies, &copied, false, st));
    }
    const int64_t ld = up8(inner);
    const Mat dg{base + sp.mats, tokens, inner, ld}, du{base + sp.mats + sp.mat_bytes, tokens, inner, ld},
        h{base + sp.mats + 2 * sp.mat_bytes, tokens, inner, ld};
    ProductArgs<1, kGateBwd> g{};  // dh, and from it dgate, dup and act(gate) * up
    g.hdr = static_cast<WsHeader *>(ws);
    g.act = act;
    ZERO_TRY(side_matrix(&g.side[0], dg.p, tokens, ld, ld, dtype));
    ZERO_TRY(side_matrix(&g.side[1], du.p, tokens, ld, ld, dtype));
    ZERO_TRY(side_matrix(&g.side[2], gate, tokens, inner, inner, dtype));
    ZERO_TRY(side_matrix(&g.side[3], up, tokens, inner, inner, dtype));
    g.side[2].tma = g.side[3].tma = g.side[2].tma && g.side[3].tma;
    const Spec s1{{my, my}, {md, md}, 1, tokens, inner, dim, const_cast<void *>(h.p), ld, ld};
    ZERO_TRY((products<kGateBwd, kKMn, 1>(&s1, 1, g, plan_product(tokens, inner, dim, false, kMostParts), copied, dtype, st)));
    // dx, then the weight gradients
    const Spec s2{{dg, du}, {mg, mu}, 2, tokens, dim, inner, dx, dx_ld, dim};
    ProductArgs<1, kStore> d{};
    d.hdr = g.hdr;
    ZERO_TRY((products<kStore, kKMn, 1>(&s2, 1, d, plan_product(tokens, dim, 2 * inner, false, kMostParts), true, dtype, st)));
    const Spec s3[3] = {{{dg, dg}, {mx, mx}, 1, inner, dim, tokens, dw_gate, dim, dim},
                        {{du, du}, {mx, mx}, 1, inner, dim, tokens, dw_up, dim, dim},
                        {{my, my}, {h, h}, 1, dim, inner, tokens, dw_down, inner, inner}};
    ProductArgs<3, kStore> w{};
    w.hdr = g.hdr;
    w.out_f32 = gdtype == ZERO_F32;
    return products<kStore, kMnMn, 3>(s3, 3, w, plan_product(3 * inner, dim, tokens, false, kMostParts), true, dtype, st);
}
