// bf16 products grouped by expert, groups of any number of rows.
//
// x [M, K] holds the rows of group g at offsets[g] ..; W_g [K, N]:
//   forward            y[rows of g] = x[rows of g] W_g, or act(x Wg) * (x Wu)
//   input gradient     dx[rows of g] = dy[rows of g] W_g^T
//   weight gradient    dW_g = x[rows of g]^T dy[rows of g]
// The offsets stay on the device; the grid depends on sizes the host knows.
//
// The first two (k_rows) run on the tensor cores transposed, D^T = W_g^T x^T:
// 256 columns of W_g are the M of a CTA pair's product and the group's rows its N,
// which may be any multiple of 32.  With rows as M, every group would be padded
// to 256 rows, a sixth more products for experts of 768 rows each, and a few
// rows per expert (decoding) would cost as much as 256.  A group's rows are
// split evenly into tiles of at most 256.  Rows are read in place: a tile
// that is too long for the group reads the next one's rows, whose results are not
// stored (a product's rows do not mix).  D^T is turned round on its way to
// memory by the matrix stores to shared memory.
// The weight gradient (k_wgrad) contracts over the group's rows.  The TMA brings
// whole 16-row steps; the up to 15 rows that remain come in a 16-row step of their own,
// which two warps fill with plain loads a tile ahead, zeros behind the last row (in both
// operands: zero times a next group's infinity would not be zero).  Zeros
// written over the TMA's own last step instead held up every tile by 0.8 us.
//
// Tiles of 256 columns x up to 256 rows (k_wgrad: 256 x 256), 64 deep per stage, six
// stages of 32 KB per CTA, two accumulators in TMEM.  Bound by the tensor cores under
// the power cap when groups have hundreds of rows (64 groups of 718 to 818 rows, 2,048 x
// 7,168: forward 0.97 ms, 1.49 PFLOP/s back to back; weight gradient 1.00 ms, in
// bursts too short for the cap 0.84 ms, 1.71; a weight gradient of many groups is also bound by
// writing dW), by the reading of W when they have few (32 rows over 256 experts,
// 7,168 x 2 * 2,048: 240 us, 7.1 TB/s of the touched weights), by set-up, first
// loads and last stores when everything is small (both gradients of 300 rows, 16 groups of
// 515 x 259: 11 us).  Short of a step the rows of one group cost what 32 do.
//
// Warps: 0 TMA, 1 MMA (of the leader CTA), 2 and 3 (k_wgrad) a group's last rows,
// 4-11 epilogue.  All waits are bounded.
#include <algorithm>

#include "pair_bf16.cuh"

namespace moe {

// gemm.cu
bool make_bf16_map3(CUtensorMap* m, const void* base, int64_t G, int64_t rows, int64_t cols, int64_t ld, int64_t gs,
                    int box_rows);
bool make_store_map3(CUtensorMap* m, void* base, int64_t G, int64_t rows, int64_t cols, int64_t ld, int64_t gs,
                     bool f32);

namespace grouped {

using namespace dense;

constexpr int ACC_COLS = 256;                   // TMEM columns of an accumulator
constexpr int NACC = 2;
constexpr int HALF_BYTES = 128 * TK * 2;        // one CTA's 128 rows of an operand per stage
// six of 32 KB; eight of 18 KB where rows are few (32 experts' gated projections, 7,168 x
// 2 * 2,048, a row each: 259 us, with six or ten 263 and 267)
constexpr int MAX_STAGES = 8;
constexpr int SMEM_WORK = 14 * HALF_BYTES;      // stages, then the epilogue's boxes
constexpr int OFF_BAR = SMEM_WORK;              // full[S], empty[S], tfull[A], tempty[A], xfull[4], xempty[4], drain
constexpr int NBAR = 2 * MAX_STAGES + 2 * NACC + 9;
constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;
constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory budget");
constexpr int MAX_GROUPS = 65536;
// k_wgrad: a box of 32 rows of 64 bytes per epilogue warp, and before them two
// buffers of a group's last rows, 16 rows of 256 columns each
constexpr int W_BOX = 2048, LAST_BYTES = 8192;
constexpr int OFF_LAST = SMEM_WORK - EPI_WARPS * W_BOX - 2 * LAST_BYTES;

struct Params {
    const int32_t* offsets;      // [G + 1]
    const int32_t* rows;         // [G] or NULL: up to the next offset
    int G;
    int64_t M;
    int N, K;                    // k_rows: columns of D (GLU: f), depth; k_wgrad: D_g is [K, N]
    int nk;                      // k_rows: steps of the depth
    int n_max;                   // k_rows: most rows of a tile, a multiple of 32
    int col_tiles;               // k_rows: tiles along N; k_wgrad: tiles along N
    int m_tiles, bn;             // k_wgrad: tiles along K, columns of a tile
    int64_t max_tiles;
    int stages, stage_bytes;
    int up;                      // GLU: column of W where the up half begins
    const __nv_bfloat16 *x, *dy; // k_wgrad: the operands, for the last rows
    int64_t ldx, lddy;
    void* y;
    int64_t ldy, gsy;
    __nv_bfloat16* a;            // GLU: [gate | up] or NULL
    int64_t lda;
    int32_t* err;
    uint64_t timeout_ns;
};

// First row and number of rows of group g; none where the offsets are wrong.
struct Span {
    int start, rows;
};
__device__ __forceinline__ Span span_of(const Params& p, int g) {
    Span s{0, 0};
    if (g >= p.G) return s;
    const int a = p.offsets[g], b = p.offsets[g + 1];
    const int n = p.rows ? p.rows[g] : b - a;
    if (a < 0 || b < a || b > p.M || n < 0 || n > b - a) {
        set_err(p.err, MOE_ERR_BAD_OFFSETS);
        return s;
    }
    s.start = a, s.rows = n;
    return s;
}

// Where tile t of k_rows lies.  A warp keeps 32 groups, a lane each, and moves on
// to the next 32 as its tiles do (t only grows).
struct Tile {
    int g, ct;          // group, tile of W's columns
    int row0, rows;     // of x
};
struct Cursor {
    int base = -32;                 // of the 32 groups
    int64_t first = 0, end = 0;     // this lane's group's first tile; the tiles up to the last lane's
    int start, rows, parts, tiles;  // of this lane's group; tiles down its rows, and in all
    __device__ __forceinline__ bool find(const Params& p, int64_t t, int lane, Tile& out) {
        while (t >= end) {
            base += 32;
            if (base >= p.G) return false;
            const Span s = span_of(p, base + lane);
            start = s.start, rows = s.rows;
            parts = (rows + p.n_max - 1) / p.n_max;
            tiles = parts * p.col_tiles;
            int64_t sum = tiles;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
                if (lane >= o) sum += v;
            }
            first = end + sum - tiles;
            if (first + tiles > p.max_tiles) tiles = 0;      // groups that overlap
            end = min(end + __shfl_sync(0xFFFFFFFFu, sum, 31), p.max_tiles);
        }
        const uint32_t here = __ballot_sync(0xFFFFFFFFu, t >= first && t < first + tiles);
        if (here == 0) return false;
        const int src = __ffs(here) - 1;
        const int i = (int)(t - __shfl_sync(0xFFFFFFFFu, first, src));
        const int n_rows = __shfl_sync(0xFFFFFFFFu, rows, src), n = __shfl_sync(0xFFFFFFFFu, parts, src);
        // bands of 8 row tiles, consecutive tiles down a band: those under way share
        // W's columns and x's rows in L2
        const int band = 8 * p.col_tiles, b = i / band, rem = i - b * band, width = min(8, n - 8 * b);
        out.g = base + src;
        out.ct = rem / width;
        // the group's rows, 32 by 32, evenly over its tiles (all but the last full, the
        // pairs whose turn is always the last one would have less to do)
        const int r = 8 * b + rem - out.ct * width, units = (n_rows + 31) / 32, each = units / n, more = units - each * n;
        const int first_row = 32 * (r * each + min(r, more));
        out.row0 = __shfl_sync(0xFFFFFFFFu, start, src) + first_row;
        out.rows = min(32 * (each + (r < more)), n_rows - first_row);
        return true;
    }
};

// A CTA's place: in its pair, in the grid, in shared memory.
struct Place {
    uint8_t* smem;
    uint32_t bar0, rank;
    int warp, lane, first, step;      // the pair's tiles: first, first + step, ..
    volatile int* abort_flag;
    __device__ __forceinline__ uint32_t bar(int i) const { return bar0 + 8u * i; }
    __device__ __forceinline__ uint32_t full(int s) const { return bar(s); }
    __device__ __forceinline__ uint32_t empty(int s) const { return bar(MAX_STAGES + s); }
    __device__ __forceinline__ uint32_t tfull(int a) const { return bar(2 * MAX_STAGES + a); }
    __device__ __forceinline__ uint32_t tempty(int a) const { return bar(2 * MAX_STAGES + NACC + a); }
    // k_rows: from a gate warp to its up warp and back; k_wgrad: a group's last rows
    __device__ __forceinline__ uint32_t xfull(int i) const { return bar(2 * MAX_STAGES + 2 * NACC + i); }
    __device__ __forceinline__ uint32_t xempty(int i) const { return bar(2 * MAX_STAGES + 2 * NACC + 4 + i); }
    __device__ __forceinline__ uint32_t drain() const { return bar(2 * MAX_STAGES + 2 * NACC + 8); }
};

// Barriers, TMEM; returns its base to every warp.
__device__ __forceinline__ uint32_t set_up(Place& pl, int stages, int x_arrivals) {
    extern __shared__ uint8_t smem_raw[];
    pl.smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    pl.warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0), pl.lane = threadIdx.x & 31;
    pl.rank = cluster_ctarank();
    pl.first = blockIdx.x / 2, pl.step = gridDim.x / 2;
    pl.bar0 = smem_u32(pl.smem + OFF_BAR);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(pl.smem + OFF_MISC);
    pl.abort_flag = reinterpret_cast<volatile int*>(pl.smem + OFF_MISC + 4);
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(pl.full(s), 1);
            mbar_init(pl.empty(s), 1);
        }
        for (int a = 0; a < NACC; ++a) {
            mbar_init(pl.tfull(a), 1);
            mbar_init(pl.tempty(a), 2 * EPI_WARPS);
        }
        for (int i = 0; i < 4; ++i) mbar_init(pl.xfull(i), x_arrivals), mbar_init(pl.xempty(i), 1);
        mbar_init(pl.drain(), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        *pl.abort_flag = 0;
    }
    __syncthreads();
    cluster_sync();      // the peer's barriers are initialised
    if (pl.warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(TMEM_COLS));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        tc_fence_before();
    }
    if (pl.warp == 1 || pl.warp >= 4) {      // the producer need not wait for TMEM
        asm volatile("bar.sync 1, %0;" ::"n"(32 + 32 * EPI_WARPS) : "memory");
        tc_fence_after();
    }
    return pl.warp == 1 || pl.warp >= 4 ? *tmem_slot : 0u;
}
__device__ __forceinline__ void tear_down(const Place& pl, uint32_t tmem_base) {
    tc_fence_before();
    __syncthreads();
    cluster_sync();      // both CTAs are done with TMEM and with each other's barriers
    tc_fence_after();
    if (pl.warp == 1) {
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(TMEM_COLS));
    }
}
__device__ __forceinline__ Params patient(const Params& p) {      // for what is in flight after an abort
    Params q = p;
    q.timeout_ns = 200000000ull;
    return q;
}
// wait (bounded) for the products issued
__device__ __forceinline__ void products_end(const Place& pl, const Params& p, const Ring& ring) {
    if (ring.count > 0) {
        if (elect_one()) tc_commit_local2(pl.drain());
        volatile int no_abort = 0;
        mbar_wait(pl.drain(), 0, patient(p), &no_abort);
    }
    __syncwarp();
}

// ---------------------------------------- forward and input gradient ----

// 16 TMEM lanes x 32 columns: thread T holds of every 8 columns 2 (T % 4) and
// the next one, of lanes T / 4 (first two registers) and T / 4 + 8.
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// The way out of an epilogue warp: a chunk of D^T, 32 columns of D (lanes) x 32
// rows (TMEM columns), in bf16 and turned round, as a box of 32 rows of 64 bytes
// (64-byte swizzle).  A TMA store writes it; where the group ends inside the
// box, or a width that is no multiple of 8 does, the rows are copied out.
template <int BOXES>
struct Out {
    uint32_t buf;
    int lane;
    uint32_t at;      // which of the two boxes
    // v: what tmem_ld_16x32 gave for lanes 0..15 and 16..31
    __device__ __forceinline__ void put(const CUtensorMap* map, __nv_bfloat16* d, int64_t ld, int col, int cols,
                                        int64_t row, int rows, const float* v) {
        const uint32_t b = buf + at;
        if (BOXES == 2) at ^= 2048u;
        if (lane == 0) {      // this box has been read
            if (BOXES == 2) bulk_wait_group_read1();
            else bulk_wait_group_read0();
        }
        __syncwarp();
        // one store for 8 rows: its four 8 x 8 matrices are 8 columns each
        const uint32_t r = (uint32_t)lane & 7u, c = (uint32_t)lane >> 3;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const uint32_t line = 8u * n + r;
            asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                             b + 64u * line + ((c ^ (line >> 1 & 3u)) << 4)),
                         "r"(pack_bf16x2(v[4 * n], v[4 * n + 1])), "r"(pack_bf16x2(v[4 * n + 2], v[4 * n + 3])),
                         "r"(pack_bf16x2(v[16 + 4 * n], v[16 + 4 * n + 1])),
                         "r"(pack_bf16x2(v[16 + 4 * n + 2], v[16 + 4 * n + 3]))
                         : "memory");
        }
        const bool whole = rows >= 32 && (cols >= 32 || (cols & 7) == 0);
        if (whole) fence_proxy_async_shared();
        __syncwarp();
        if (whole) {
            if (lane == 0) tma_store_2d(map, b, col, (int)row);
        } else if (lane < rows) {
            __nv_bfloat16* dst = d + (row + lane) * ld + col;
#pragma unroll
            for (uint32_t q = 0; q < 4; ++q) {
                const int n = cols - 8 * (int)q;
                if (n <= 0) break;
                uint32_t w[4];
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                             : "r"(b + 64u * lane + ((q ^ ((uint32_t)lane >> 1 & 3u)) << 4))
                             : "memory");
                if (n >= 8) {
                    *reinterpret_cast<uint4*>(dst + 8 * q) = make_uint4(w[0], w[1], w[2], w[3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 7; ++i)
                        if (i < n) dst[8 * q + i] = __ushort_as_bfloat16((unsigned short)(w[i >> 1] >> (16 * (i & 1))));
                }
            }
        }
        if (lane == 0) bulk_commit_group();      // (an empty one, so that every box counts)
        __syncwarp();
    }
};

// The tiles of D = x op(W), from the pair's next one, t, on; t is behind the last
// one afterwards.  W_MN: the forward product (D's columns are contiguous in W).
// GLU: the tile's 128 columns per CTA are 64 of gate and the same 64 of up.
template <bool W_MN, bool GLU>
__device__ __forceinline__ void load_rows(const Place& pl, const Params& p, const CUtensorMap* tmW,
                                          const CUtensorMap* tmX16, const CUtensorMap* tmX32, const CUtensorMap* tmX64,
                                          const CUtensorMap* tmX128, Cursor& cur, int64_t& t, Ring& ring) {
    constexpr int TILE_COLS = GLU ? 128 : 256;        // of D, per pair
    Tile ti;
    const bool elected = elect_one();
    const uint32_t lead_full = mapa(pl.full(0), 0);
    for (; !ring.aborted && cur.find(p, t, pl.lane, ti); t += pl.step) {
        const int half = (ti.rows + 31) / 32 * 16;     // rows of this CTA
        const CUtensorMap* tmX = half <= 16 ? tmX16 : (half <= 32 ? tmX32 : (half <= 64 ? tmX64 : tmX128));
        const uint32_t x_rows = half <= 16 ? 16 : (half <= 32 ? 32 : (half <= 64 ? 64 : 128));
        const uint32_t bytes = 2u * (HALF_BYTES + x_rows * TK * 2);
        const int col = ti.ct * TILE_COLS + (GLU ? 64 : 128) * (int)pl.rank, row = ti.row0 + half * (int)pl.rank;
        for (int ks = 0; ks < p.nk; ++ks) {
            if (!mbar_wait_cluster(pl.empty(ring.at), ring.phase ^ 1u, p, pl.abort_flag)) {
                ring.aborted = true;
                break;
            }
            // both CTAs' bytes complete on the leader's full barrier
            const uint32_t fb = lead_full + 8u * ring.at;
            if (elected) {
                if (pl.rank == 0) mbar_expect_tx(pl.full(ring.at), bytes);
                const uint32_t sw = smem_u32(pl.smem + ring.at * p.stage_bytes);
                if constexpr (W_MN) {
                    tma2_load_3d(sw, tmW, col, ks * TK, ti.g, fb);
                    tma2_load_3d(sw + HALF_BYTES / 2, tmW, GLU ? col + p.up : col + 64, ks * TK, ti.g, fb);
                } else {
                    tma2_load_3d(sw, tmW, ks * TK, col, ti.g, fb);
                }
                tma2_load_2d(sw + HALF_BYTES, tmX, ks * TK, row, fb);
            }
            ring.next(p.stages);
        }
        ring.aborted = __any_sync(0xFFFFFFFFu, ring.aborted);      // the warp goes on as one
    }
}
template <bool W_MN>
__device__ __forceinline__ void multiply_rows(const Place& pl, const Params& p, uint32_t tmem_base, Cursor& cur,
                                              int64_t& t, Ring& ring, Ring& acc) {
    Tile ti;
    const bool elected = elect_one();
    const uint64_t adesc0 = operand_desc<W_MN>(smem_u32(pl.smem));
    const uint64_t bdesc0 = operand_desc<false>(smem_u32(pl.smem) + HALF_BYTES);
    const uint32_t stage_step = (uint32_t)p.stage_bytes >> 4;
    for (; !ring.aborted && cur.find(p, t, pl.lane, ti); t += pl.step) {
        const uint32_t idesc = make_idesc_pair<W_MN, false>((ti.rows + 31) / 32 * 32);
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_cluster(pl.tempty(acc.at), acc.phase ^ 1u, p, pl.abort_flag))) {
            ring.aborted = true;
            break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(acc.at * ACC_COLS);
        for (int ks = 0; ks < p.nk; ++ks) {
            if (!mbar_wait(pl.full(ring.at), ring.phase, p, pl.abort_flag)) {
                ring.aborted = true;
                break;
            }
            tc_fence_after();
            if (elected) {
                const uint64_t adesc = adesc0 + ring.at * stage_step, bdesc = bdesc0 + ring.at * stage_step;
#pragma unroll
                for (int kk = 0; kk < TK / 16; ++kk)
                    tc_mma2_bf16(d_tmem, adesc + k16_step<W_MN>() * kk, bdesc + k16_step<false>() * kk, idesc,
                                 (ks != 0 || kk != 0) ? 1u : 0u);
                tc_commit_pair(pl.empty(ring.at), 0);
            }
            ring.next(p.stages);
        }
        ring.aborted = __any_sync(0xFFFFFFFFu, ring.aborted);
        if (ring.aborted) break;
        if (elected) tc_commit_pair(pl.tfull(acc.at), 0);
        acc.next(NACC);
    }
}
// BOXES: 2 KB boxes of a warp on their way out
template <bool GLU, int ACT, int BOXES>
__device__ __forceinline__ bool store_rows(const Place& pl, const Params& p, const CUtensorMap* tmY,
                                           const CUtensorMap* tmA, const CUtensorMap* tmA2, uint32_t tmem_base,
                                           Cursor& cur, int64_t& t, Ring& acc) {
    Tile ti;
    const int lane = pl.lane, ew = pl.warp - 4, quarter = ew & 3, half = ew >> 2;
    const uint32_t lane_base = tmem_base + ((uint32_t)(quarter * 32) << 16);
    const uint32_t stage = smem_u32(pl.smem + SMEM_WORK - (EPI_WARPS - ew) * 2048 * BOXES);
    Out<BOXES> out{stage, lane, 0u};
    // GLU: lanes 0..63 hold gate columns, 64..127 the up columns of the same h;
    // the gate warp hands act(gate) in fp32 to the up warp two quarters on
    const bool gate = GLU && quarter < 2;
    const int pair = (quarter & 1) + 2 * half;
    const uint32_t to_up = smem_u32(pl.smem + SMEM_WORK - EPI_WARPS * 2048 * BOXES - (4 - pair) * 4096) + 16u * lane;
    uint32_t handed = 0;
    bool ok = true;
    for (; ok && cur.find(p, t, lane, ti); t += pl.step) {
        ok = __all_sync(0xFFFFFFFFu, mbar_wait_cluster(pl.tfull(acc.at), acc.phase, p, pl.abort_flag));
        if (!ok) break;
        tc_fence_after();
        const int chunks = (ti.rows + 31) / 32;
        const int c0 = half == 0 ? 0 : (chunks + 1) / 2, c1 = half == 0 ? (chunks + 1) / 2 : chunks;
        const uint32_t tacc = lane_base + (uint32_t)(acc.at * ACC_COLS);
        const int col = GLU ? ti.ct * 128 + 64 * (int)pl.rank + 32 * (quarter & 1)
                            : ti.ct * 256 + 128 * (int)pl.rank + 32 * quarter;
        const int cols = p.N - col;
        for (int c = c0; c < c1 && ok; ++c) {
            uint32_t r[32];
            tmem_ld_16x32(tacc + 32 * c, r);
            tmem_ld_16x32(tacc + (16u << 16) + 32 * c, r + 16);
            tmem_wait_ld();
            if (c + 1 == c1) {      // the accumulator is read: the next tile may have it
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(mapa(pl.tempty(acc.at), 0));
            }
            float v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
            const int64_t row = ti.row0 + 32 * c;
            const int rows = ti.rows - 32 * c;
            if constexpr (!GLU) {
                if (cols > 0) out.put(tmY, static_cast<__nv_bfloat16*>(p.y), p.ldy, col, cols, row, rows, v);
            } else {
                if (cols <= 0) continue;      // both warps
                if (p.a != nullptr)
                    out.put(gate ? tmA : tmA2, p.a + (gate ? 0 : p.N), p.lda, col, cols, row, rows, v);
                if (gate) {
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(pl.xempty(pair), handed & 1u ^ 1u, p, pl.abort_flag));
                    if (!ok) break;
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = act_of(v[i], ACT);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        st_shared_v4(to_up + 512u * i, __float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                                     __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3]));
                    __syncwarp();
                    if (lane == 0) mbar_arrive(pl.xfull(pair));
                } else {
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(pl.xfull(pair), handed & 1u, p, pl.abort_flag));
                    if (!ok) break;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float g[4];
                        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                                     : "=f"(g[0]), "=f"(g[1]), "=f"(g[2]), "=f"(g[3])
                                     : "r"(to_up + 512u * i)
                                     : "memory");
#pragma unroll
                        for (int j = 0; j < 4; ++j) v[4 * i + j] *= g[j];
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(pl.xempty(pair));
                    out.put(tmY, static_cast<__nv_bfloat16*>(p.y), p.ldy, col, cols, row, rows, v);
                }
                ++handed;
            }
        }
        if (c0 >= c1) {      // nothing of this tile is this warp's
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(mapa(pl.tempty(acc.at), 0));
        }
        acc.next(NACC);
    }
    return ok;
}
// After an abort: wait (bounded) for the copies in flight.  The leader's full
// barriers count both CTAs' bytes, and the follower leaves only after the
// closing cluster barrier, i.e. after this.
__device__ __forceinline__ void loads_end(const Place& pl, const Params& p, const Ring& ring) {
    __syncwarp();
    if (!ring.aborted || pl.rank != 0) return;
    const Params q = patient(p);
    volatile int no_abort = 0;
    for (int i = ring.count - min(ring.count, p.stages); i < ring.count; ++i)
        mbar_wait_cluster(pl.full(i % p.stages), (uint32_t)(i / p.stages) & 1u, q, &no_abort);
}
__device__ __forceinline__ void stores_end(int lane) {
    if (lane == 0) bulk_wait_group0();      // the stores are complete
    __syncwarp();
}

template <bool W_MN, bool GLU, int ACT>
__global__ void __launch_bounds__(THREADS, 1)
    k_rows(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX16,
           const __grid_constant__ CUtensorMap tmX32, const __grid_constant__ CUtensorMap tmX64,
           const __grid_constant__ CUtensorMap tmX128, const __grid_constant__ CUtensorMap tmY,
           const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA2, const Params p) {
    if (threadIdx.x == 64) {
        prefetch_map(&tmW);
        prefetch_map(&tmX128);
        prefetch_map(&tmY);
    }
    Place pl;
    const uint32_t tmem_base = set_up(pl, p.stages, 1);
    wait_for_previous_kernels();
    Cursor cur;
    Ring ring, acc;
    int64_t t = pl.first;
    if (pl.warp == 0) {
        load_rows<W_MN, GLU>(pl, p, &tmW, &tmX16, &tmX32, &tmX64, &tmX128, cur, t, ring);
        loads_end(pl, p, ring);
    } else if (pl.warp == 1 && pl.rank == 0) {
        multiply_rows<W_MN>(pl, p, tmem_base, cur, t, ring, acc);
        products_end(pl, p, ring);
    } else if (pl.warp >= 4) {
        store_rows<GLU, ACT, GLU ? 1 : 2>(pl, p, &tmY, &tmA, &tmA2, tmem_base, cur, t, acc);
        stores_end(pl.lane);
    }
    tear_down(pl, tmem_base);
}

// ----------------------------------------------------- weight gradient ----

// Tiles of 256 x p.bn of every group's D_g = x^T dy, the groups one after the
// other; an empty group's are zeros.
struct WTile {
    int g, mt, nt, start, rows;
};
__device__ __forceinline__ WTile w_tile(const Params& p, int64_t t) {
    const int per = p.m_tiles * p.col_tiles;
    WTile w;
    w.g = (int)(t / per);
    const int i = (int)(t - (int64_t)w.g * per);
    const int band = 8 * p.col_tiles, b = i / band, rem = i - b * band, width = min(8, p.m_tiles - 8 * b);
    w.nt = rem / width;
    w.mt = 8 * b + rem - w.nt * width;
    const Span s = span_of(p, w.g);
    w.start = s.start, w.rows = s.rows;
    return w;
}

// 32 rows (a lane each) x 32 columns of D_g out of registers: a TMA store of a
// staged box, or, of a width whose last columns are no whole 16 bytes, from here.
template <bool F32>
struct WOut {
    uint32_t buf;
    int lane;
    bool zeros;      // the box holds zeros, from an empty group's tile before
    __device__ __forceinline__ void store(const CUtensorMap* map, int g, int row0, int col) {
        asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(map),
                     "r"(buf), "r"(col), "r"(row0), "r"(g)
                     : "memory");
        bulk_commit_group();
    }
    // an empty group's chunk: the box is filled once and stored as often as it is wanted
    __device__ __forceinline__ void put_zeros(const Params& p, const CUtensorMap* map, int g, int row0, int col) {
        const int cols = p.N - col;
        if (cols < 32 && (cols & 7) != 0) {
            const float v[32] = {};
            put(p, map, g, row0, col, v);
            return;
        }
        if (!zeros) {
            if (lane == 0) bulk_wait_group_read0();
            __syncwarp();
#pragma unroll
            for (int c = 0; c < 4; ++c) st_shared_v4(buf + 64u * lane + 16u * c, 0u, 0u, 0u, 0u);
            fence_proxy_async_shared();
            __syncwarp();
            zeros = true;
        }
        if (lane == 0) {
            store(map, g, row0, col);
            if (F32 && cols > 16) store(map, g, row0, col + 16);
        }
    }
    __device__ __forceinline__ void put(const Params& p, const CUtensorMap* map, int g, int row0, int col,
                                        const float* v) {
        const int cols = p.N - col;
        if (cols < 32 && (cols & 7) != 0) {
            const int row = row0 + lane;
            if (row >= p.K) return;
            const int64_t o = g * p.gsy + (int64_t)row * p.ldy + col;
#pragma unroll
            for (int i = 0; i < 31; ++i) {
                if (i < cols) {
                    if (F32) static_cast<float*>(p.y)[o + i] = v[i];
                    else static_cast<__nv_bfloat16*>(p.y)[o + i] = __float2bfloat16_rn(v[i]);
                }
            }
            return;
        }
        zeros = false;
#pragma unroll
        for (int h = 0; h < (F32 ? 2 : 1); ++h) {
            if (F32 && 16 * h >= cols) break;
            if (lane == 0) bulk_wait_group_read0();
            __syncwarp();
            const uint32_t row = buf + 64u * lane, sw = (uint32_t)(lane >> 1) & 3u;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float* u = F32 ? v + 16 * h + 4 * c : v + 8 * c;
                const uint32_t at = row + (((uint32_t)c ^ sw) << 4);
                if constexpr (F32)
                    st_shared_v4(at, __float_as_uint(u[0]), __float_as_uint(u[1]), __float_as_uint(u[2]),
                                 __float_as_uint(u[3]));
                else
                    st_shared_v4(at, pack_bf16x2(u[0], u[1]), pack_bf16x2(u[2], u[3]), pack_bf16x2(u[4], u[5]),
                                 pack_bf16x2(u[6], u[7]));
            }
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) store(map, g, row0, col + 16 * h);
        }
    }
};

// The weight gradients' tiles from the pair's next one, t, on.
__device__ __forceinline__ void load_wgrad(const Place& pl, const Params& p, const CUtensorMap* tmX,
                                           const CUtensorMap* tmDY, int64_t t, Ring& ring) {
    const bool elected = elect_one();
    const int bh = p.bn / 2, boxes = (bh + 63) / 64;      // of dy's columns, per CTA
    const uint32_t bytes = HALF_BYTES + boxes * (HALF_BYTES / 2);
    const uint32_t lead_full = mapa(pl.full(0), 0);
    for (; t < p.max_tiles && !ring.aborted; t += pl.step) {
        const WTile w = w_tile(p, t);
        const int nk = (w.rows / 16 + 3) / 4;      // steps of 64 rows, the last of fewer 16-row ones
        const int am = w.mt * TM + 128 * (int)pl.rank, bn = w.nt * p.bn + bh * (int)pl.rank;
        for (int ks = 0; ks < nk; ++ks) {
            if (!mbar_wait_cluster(pl.empty(ring.at), ring.phase ^ 1u, p, pl.abort_flag)) {
                ring.aborted = true;
                break;
            }
            const uint32_t fb = lead_full + 8u * ring.at;
            if (elected) {
                if (pl.rank == 0) mbar_expect_tx(pl.full(ring.at), 2u * bytes);
                const uint32_t sa = smem_u32(pl.smem + ring.at * p.stage_bytes), sb = sa + HALF_BYTES;
                const int row = w.start + ks * TK;
                tma2_load_2d(sa, tmX, am, row, fb);
                tma2_load_2d(sa + HALF_BYTES / 2, tmX, am + 64, row, fb);
                tma2_load_2d(sb, tmDY, bn, row, fb);
                if (boxes > 1) tma2_load_2d(sb + HALF_BYTES / 2, tmDY, bn + 64, row, fb);
            }
            ring.next(p.stages);
        }
    }
}
__device__ __forceinline__ void fill_last_rows(const Place& pl, const Params& p, int64_t t) {
    // ------------------- a group's last rows, fewer than 16, two buffers ----
    // laid out as the TMA does: boxes of 64 columns, rows of 128 bytes, their
    // 16-byte units swizzled by the row
    const int lane = pl.lane, bh = p.bn / 2, boxes = (bh + 63) / 64;
    const uint32_t lead = mapa(pl.xfull(0), 0);
    Ring last;
    for (; t < p.max_tiles; t += pl.step) {
        const WTile w = w_tile(p, t);
        const int n = w.rows & 15;
        if (n == 0) continue;
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_cluster(pl.xempty(last.at), last.phase ^ 1u, p, pl.abort_flag))) break;
        const uint32_t buf = smem_u32(pl.smem + OFF_LAST + last.at * LAST_BYTES);
        const int64_t row0 = (int64_t)w.start + w.rows - n;
        const int am = w.mt * TM + 128 * (int)pl.rank, bn = w.nt * p.bn + bh * (int)pl.rank;
        const int lane2 = (int)threadIdx.x - 64, unit = lane2 & 7;
        // two boxes of x, then dy's: 8 units of 16 rows each
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            if (b >= 2 + boxes) break;
            const bool is_x = b < 2;
            const int col = (is_x ? am + 64 * b : bn + 64 * (b - 2)) + 8 * unit;
            const int cols = min((is_x ? p.K : p.N) - col, 8);
            uint4 v[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = (lane2 >> 3) + 8 * i;
                v[i] = make_uint4(0u, 0u, 0u, 0u);
                if (r < n && cols > 0)
                    v[i] = load_vec8(is_x ? p.x + (row0 + r) * p.ldx + col : p.dy + (row0 + r) * p.lddy + col, cols);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = (lane2 >> 3) + 8 * i;
                st_shared_v4(buf + 2048u * b + 128u * r + (((uint32_t)unit ^ (r & 7u)) << 4), v[i].x, v[i].y, v[i].z,
                             v[i].w);
            }
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(lead + 8u * last.at);
        last.next(2);
    }
}
__device__ __forceinline__ void multiply_wgrad(const Place& pl, const Params& p, uint32_t tmem_base, int64_t t, Ring& ring,
                                               Ring& acc) {
    const bool elected = elect_one();
    Ring last;
    const uint32_t idesc = make_idesc_pair<true, true>(p.bn);
    const uint64_t adesc0 = operand_desc<true>(smem_u32(pl.smem));
    const uint64_t bdesc0 = operand_desc<true>(smem_u32(pl.smem) + HALF_BYTES);
    const uint32_t stage_step = (uint32_t)p.stage_bytes >> 4;
    for (; t < p.max_tiles && !ring.aborted; t += pl.step) {
        const WTile w = w_tile(p, t);
        if (w.rows == 0) continue;
        const int steps = w.rows / 16, nk = (steps + 3) / 4;
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_cluster(pl.tempty(acc.at), acc.phase ^ 1u, p, pl.abort_flag))) {
            ring.aborted = true;
            break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(acc.at * ACC_COLS);
        // (the loop has to be short: a step's four products take 512 cycles)
        for (int ks = 0; ks < nk; ++ks) {
            if (!mbar_wait(pl.full(ring.at), ring.phase, p, pl.abort_flag)) {
                ring.aborted = true;
                break;
            }
            tc_fence_after();
            if (elected) {
                const uint64_t adesc = adesc0 + ring.at * stage_step, bdesc = bdesc0 + ring.at * stage_step;
#pragma unroll
                for (int kk = 0; kk < TK / 16; ++kk)
                    if (4 * ks + kk < steps)
                        tc_mma2_bf16(d_tmem, adesc + k16_step<true>() * kk, bdesc + k16_step<true>() * kk, idesc,
                                     (ks != 0 || kk != 0) ? 1u : 0u);
                tc_commit_pair(pl.empty(ring.at), 0);
            }
            ring.next(p.stages);
        }
        if ((w.rows & 15) != 0 && !ring.aborted) {      // both CTAs have filled the last step
            if (mbar_wait_cluster(pl.xfull(last.at), last.phase, p, pl.abort_flag)) {
                tc_fence_after();
                if (elected) {
                    const uint32_t buf = smem_u32(pl.smem + OFF_LAST + last.at * LAST_BYTES);
                    tc_mma2_bf16(d_tmem, desc_mn_sw128(buf, 2048), desc_mn_sw128(buf + 4096, 2048), idesc,
                                 steps > 0 ? 1u : 0u);
                    tc_commit_pair(pl.xempty(last.at), 0);
                }
                last.next(2);
            } else {
                ring.aborted = true;
            }
        }
        ring.aborted = __any_sync(0xFFFFFFFFu, ring.aborted);      // the warp goes on as one
        if (ring.aborted) break;
        if (elected) tc_commit_pair(pl.tfull(acc.at), 0);
        acc.next(NACC);
    }
}
template <bool F32>
__device__ __forceinline__ void store_wgrad(const Place& pl, const Params& p, const CUtensorMap* tmD, uint32_t tmem_base,
                                            int64_t t, Ring& acc) {
    const int lane = pl.lane, ew = pl.warp - 4, quarter = ew & 3, half = ew >> 2;
    const uint32_t lane_base = tmem_base + ((uint32_t)(quarter * 32) << 16);
    WOut<F32> out{smem_u32(pl.smem + SMEM_WORK - (EPI_WARPS - ew) * W_BOX), lane, false};
    const int chunks = p.bn / 32, c0 = half == 0 ? 0 : (chunks + 1) / 2, c1 = half == 0 ? (chunks + 1) / 2 : chunks;
    for (; t < p.max_tiles; t += pl.step) {
        const WTile w = w_tile(p, t);
        const int row0 = w.mt * TM + 128 * (int)pl.rank + quarter * 32;
        const uint32_t tacc = lane_base + (uint32_t)(acc.at * ACC_COLS);
        const int col0 = w.nt * p.bn;
        if (w.rows == 0) {
            for (int c = c0; c < c1; ++c)
                if (col0 + 32 * c < p.N && row0 < p.K) out.put_zeros(p, tmD, w.g, row0, col0 + 32 * c);
            continue;
        }
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_cluster(pl.tfull(acc.at), acc.phase, p, pl.abort_flag))) break;
        tc_fence_after();
        for (int c = c0; c < c1; ++c) {
            float v[32];
            tmem_ld32(tacc + 32 * c, v);
            if (c + 1 == c1) {      // the accumulator is read: the next tile may have it
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(mapa(pl.tempty(acc.at), 0));
            }
            const int col = col0 + 32 * c;
            if (col < p.N && row0 < p.K) out.put(p, tmD, w.g, row0, col, v);      // the whole warp
        }
        acc.next(NACC);
    }
}

template <bool F32>
__global__ void __launch_bounds__(THREADS, 1)
    k_wgrad(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmDY,
            const __grid_constant__ CUtensorMap tmD, const Params p) {
    if (threadIdx.x == 64) {
        prefetch_map(&tmX);
        prefetch_map(&tmDY);
        prefetch_map(&tmD);
    }
    Place pl;
    const uint32_t tmem_base = set_up(pl, p.stages, 4);      // warps 2 and 3 of both CTAs
    wait_for_previous_kernels();
    Ring ring, acc;
    if (pl.warp == 0) {
        load_wgrad(pl, p, &tmX, &tmDY, pl.first, ring);
        loads_end(pl, p, ring);
    } else if (pl.warp == 1 && pl.rank == 0) {
        multiply_wgrad(pl, p, tmem_base, pl.first, ring, acc);
        products_end(pl, p, ring);
    } else if (pl.warp == 2 || pl.warp == 3) {
        fill_last_rows(pl, p, pl.first);
    } else if (pl.warp >= 4) {
        store_wgrad<F32>(pl, p, &tmD, tmem_base, pl.first, acc);
        stores_end(pl.lane);
    }
    tear_down(pl, tmem_base);
}

// Both gradients of a layer, dx = dz W^T (p) and then dW = x^T dz (q), as the tiles
// of one launch: one set-up, and the short tiles of dW fill the last wave of
// the long ones of dx.  A pair's tile t of the launch is dW's tile t - end, where
// end is the number of dx's, known when the groups have been gone through.
__device__ __forceinline__ int64_t wgrad_first(const Place& pl, const Cursor& cur, int64_t t) {
    int64_t u = t - cur.end;
    while (u < 0) u += pl.step;      // (offsets out of order)
    return u;
}
template <bool F32>
__global__ void __launch_bounds__(THREADS, 1)
    k_both(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmZ16,
           const __grid_constant__ CUtensorMap tmZ32, const __grid_constant__ CUtensorMap tmZ64,
           const __grid_constant__ CUtensorMap tmZ128, const __grid_constant__ CUtensorMap tmDX,
           const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmDY,
           const __grid_constant__ CUtensorMap tmD, const Params p, const Params q) {
    if (threadIdx.x == 64) {
        prefetch_map(&tmW);
        prefetch_map(&tmZ128);
        prefetch_map(&tmX);
        prefetch_map(&tmDY);
    }
    Place pl;
    const uint32_t tmem_base = set_up(pl, p.stages, 4);
    wait_for_previous_kernels();
    Cursor cur;
    Ring ring, acc;
    int64_t t = pl.first;
    if (pl.warp == 0) {
        load_rows<false, false>(pl, p, &tmW, &tmZ16, &tmZ32, &tmZ64, &tmZ128, cur, t, ring);
        if (!ring.aborted) load_wgrad(pl, q, &tmX, &tmDY, wgrad_first(pl, cur, t), ring);
        loads_end(pl, p, ring);
    } else if (pl.warp == 1 && pl.rank == 0) {
        multiply_rows<false>(pl, p, tmem_base, cur, t, ring, acc);
        if (!ring.aborted) multiply_wgrad(pl, q, tmem_base, wgrad_first(pl, cur, t), ring, acc);
        products_end(pl, p, ring);
    } else if (pl.warp == 2 || pl.warp == 3) {
        Tile ti;
        while (cur.find(p, t, pl.lane, ti)) t += pl.step;
        fill_last_rows(pl, q, wgrad_first(pl, cur, t));
    } else if (pl.warp >= 4) {
        if (store_rows<false, 0, 1>(pl, p, &tmDX, nullptr, nullptr, tmem_base, cur, t, acc))
            store_wgrad<F32>(pl, q, &tmD, tmem_base, wgrad_first(pl, cur, t), acc);
        stores_end(pl.lane);
    }
    tear_down(pl, tmem_base);
}

// -------------------------------------------- elementwise gated backward ----

// da = [dh * up * act'(gate) | dh * act(gate)] of the rows that belong to a
// group (da may be a itself).  `tpr` threads take a row; bound by its 10 bytes
// per element of h.
__global__ void __launch_bounds__(256) k_glu_rows(const __nv_bfloat16* __restrict__ dh, int64_t lddh,
                                                  const __nv_bfloat16* a, int64_t lda, int act, __nv_bfloat16* da,
                                                  int64_t ldda, int tpr, const Params p) {
    wait_for_previous_kernels();
    const int f = p.N, per = 256 / tpr;
    const int64_t step = (int64_t)gridDim.x * per;
    for (int64_t row = (int64_t)blockIdx.x * per + threadIdx.x / tpr; row < p.M; row += step) {
        int lo = 0, hi = p.G;      // offsets[lo] <= row < offsets[hi], were they in order
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.offsets[mid] <= row) lo = mid;
            else hi = mid;
        }
        const Span s = span_of(p, lo);
        if (row < s.start || row >= (int64_t)s.start + s.rows) continue;
        for (int c = threadIdx.x % tpr * 8; c < f; c += tpr * 8) {
            float d[8], g[8], u[8];
            unpack8(*reinterpret_cast<const uint4*>(dh + row * lddh + c), d);
            unpack8(*reinterpret_cast<const uint4*>(a + row * lda + c), g);
            unpack8(*reinterpret_cast<const uint4*>(a + row * lda + f + c), u);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float gj = g[j];
                g[j] = d[j] * u[j] * act_slope(gj, act);
                u[j] = d[j] * act_of(gj, act);
            }
            *reinterpret_cast<uint4*>(da + row * ldda + c) = pack8(g);
            *reinterpret_cast<uint4*>(da + row * ldda + f + c) = pack8(u);
        }
    }
}

// ----------------------------------------------------------------- host ----

static PerDevice<int> g_max_clusters;      // CTA pairs that run at a time
static int max_clusters() { return g_max_clusters.here(); }

static cudaLaunchConfig_t launch_cfg(int64_t pairs, cudaStream_t stream, cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * pairs), 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cfg;
}

static cudaError_t set_attributes() {
    const void* ks[] = {(const void*)k_rows<true, false, 0>,
                        (const void*)k_rows<false, false, 0>,
                        (const void*)k_rows<true, true, MOE_ACT_NONE>,
                        (const void*)k_rows<true, true, MOE_ACT_RELU>,
                        (const void*)k_rows<true, true, MOE_ACT_GELU>,
                        (const void*)k_rows<true, true, MOE_ACT_SILU>,
                        (const void*)k_wgrad<false>,
                        (const void*)k_wgrad<true>,
                        (const void*)k_both<false>,
                        (const void*)k_both<true>};
    for (const void* k : ks) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = launch_cfg(1024, nullptr, attr);
    return cudaOccupancyMaxActiveClusters(&g_max_clusters.here(), k_wgrad<false>, &cfg);
}

struct Mat {
    const void* p;
    int64_t rows, cols, ld, gs;      // gs: from one group's matrix to the next
};
constexpr int64_t kMaxTiles = 0x3FFFFFFF;

// The fields of p that sizes decide, for D = x op(W) of x [M, depth]; the maps of x.
template <bool GLU>
static moe_status_t plan_rows(Params& p) {
    const int cols = GLU ? 128 : 256;
    p.col_tiles = (p.N + cols - 1) / cols;
    p.n_max = (int)std::min<int64_t>(256, (p.M + 31) / 32 * 32);
    // Where even M rows in one group give fewer tiles than half of the pairs, tiles of
    // fewer rows: a step of 64 rows takes half the time of one of 256 (428 rows, 1,589 x 432: 8.8 us, with
    // 256 rows 13.0; gated 411 rows, 3,713 x 2 * 72: 18.1 and 27.6).
    const int most = max_clusters();
    while (p.n_max > 64 && (p.M + p.n_max - 1) / p.n_max * p.col_tiles * 2 <= most)
        p.n_max = (p.n_max / 2 + 31) / 32 * 32;
    int box = 16;      // rows of x per CTA that a stage has room for
    while (2 * box < p.n_max) box *= 2;
    p.stage_bytes = HALF_BYTES + box * TK * 2;
    p.nk = (p.K + TK - 1) / TK;
    p.max_tiles = (p.M / p.n_max + std::min<int64_t>(p.G, p.M)) * p.col_tiles;
    p.timeout_ns = 2000000000ull;
    return p.max_tiles <= kMaxTiles ? MOE_OK : MOE_ERR_UNSUPPORTED;
}
static bool rows_maps(CUtensorMap* tmX, CUtensorMap* tmY, const Mat& x, const Params& p) {
    bool ok = true;
    for (int i = 0; i < 4; ++i) ok = ok && make_bf16_map(&tmX[i], x.p, x.rows, x.cols, x.ld, 16 << i);
    // boxes that end inside 16 bytes are not stored through the map
    return ok && make_store_map(tmY, p.y, p.M, std::max(p.N & ~7, 8), p.ldy, false);
}

// D = x op(W) of every group; D's columns are W's (W_MN) or its rows.
template <bool W_MN, bool GLU, int ACT>
static moe_status_t product_rows(const Mat& x, const Mat& w, Params p, cudaStream_t s) {
    MOE_REQUIRE(max_clusters() > 0, MOE_ERR_NOT_INITIALIZED);
    const moe_status_t st = plan_rows<GLU>(p);
    if (st != MOE_OK) return st;
    // eight warps' boxes (GLU: half as many, and four gate warps' way to up)
    p.stages = std::min(MAX_STAGES, (SMEM_WORK - EPI_WARPS * 4096) / p.stage_bytes);
    CUtensorMap tmW, tmX[4], tmY, tmA, tmA2;
    bool ok = make_bf16_map3(&tmW, w.p, p.G, w.rows, w.cols, w.ld, w.gs, W_MN ? TK : 128) && rows_maps(tmX, &tmY, x, p);
    tmA = tmA2 = tmY;
    if (p.a != nullptr)
        ok = ok && make_store_map(&tmA, p.a, p.M, p.N, p.lda, false) &&
             make_store_map(&tmA2, p.a + p.N, p.M, p.N, p.lda, false);
    MOE_REQUIRE(ok, MOE_ERR_CUDA);
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = launch_cfg(std::min<int64_t>(p.max_tiles, max_clusters()), s, attr);
    if (cudaLaunchKernelEx(&cfg, k_rows<W_MN, GLU, ACT>, tmW, tmX[0], tmX[1], tmX[2], tmX[3], tmY, tmA, tmA2, p) !=
        cudaSuccess)
        return MOE_ERR_CUDA;
    MOE_CHECK_LAUNCH();
    return MOE_OK;
}

// Columns of a weight gradient's tiles: the narrower ones' steps take 0.91, 0.80
// and 0.56 of 256 columns', and fill 256-wide waves or odd widths better; no tile is
// shorter than its epilogue.
static int wgrad_width(int64_t tiles256, int N, double nk, int slots) {
    const struct {
        int bn;
        double step;
    } widths[] = {{256, 1.0}, {224, 0.91}, {192, 0.80}, {128, 0.56}};
    int best = 256;
    double least = 1e300;
    for (const auto& w : widths) {
        const int64_t tiles = tiles256 * ((N + w.bn - 1) / w.bn);
        const double cost = (double)((tiles + slots - 1) / slots) * (std::max(nk * w.step, 5. * w.bn / 256.) + 1.);
        if (cost < least) least = cost, best = w.bn;
    }
    return best;
}
static moe_status_t plan_wgrad(Params& p) {
    p.m_tiles = (p.K + TM - 1) / TM;
    p.bn = wgrad_width((int64_t)p.G * p.m_tiles, p.N, (double)p.M / p.G / TK, max_clusters());
    p.col_tiles = (p.N + p.bn - 1) / p.bn;
    p.max_tiles = (int64_t)p.G * p.m_tiles * p.col_tiles;
    p.stage_bytes = HALF_BYTES + (p.bn / 2 + 63) / 64 * (HALF_BYTES / 2);
    p.timeout_ns = 2000000000ull;
    return p.max_tiles <= kMaxTiles ? MOE_OK : MOE_ERR_UNSUPPORTED;
}
static bool wgrad_maps(CUtensorMap* tmX, CUtensorMap* tmDY, CUtensorMap* tmD, const Mat& x, const Mat& dy, Params& p,
                       bool f32) {
    p.x = static_cast<const __nv_bfloat16*>(x.p), p.ldx = x.ld;
    p.dy = static_cast<const __nv_bfloat16*>(dy.p), p.lddy = dy.ld;
    return make_bf16_map(tmX, x.p, x.rows, x.cols, x.ld, TK) && make_bf16_map(tmDY, dy.p, dy.rows, dy.cols, dy.ld, TK) &&
           make_store_map3(tmD, p.y, p.G, p.K, std::max(p.N & ~7, 8), p.ldy, p.gsy, f32);
}

// D_g [K, N] = x^T dy of every group
static moe_status_t product_wgrad(const Mat& x, const Mat& dy, Params p, bool f32, cudaStream_t s) {
    MOE_REQUIRE(max_clusters() > 0, MOE_ERR_NOT_INITIALIZED);
    const size_t size = f32 ? 4 : 2;
    if (p.M == 0) {
        const bool joined = p.gsy == p.K * p.ldy;      // one matrix of G K rows
        for (int g = 0; g < (joined ? 1 : p.G); ++g)
            if (cudaMemset2DAsync(static_cast<char*>(p.y) + g * p.gsy * size, p.ldy * size, 0, p.N * size,
                                  (size_t)p.K * (joined ? p.G : 1), s) != cudaSuccess)
                return MOE_ERR_CUDA;
        return MOE_OK;
    }
    const moe_status_t st = plan_wgrad(p);
    if (st != MOE_OK) return st;
    p.stages = std::min(MAX_STAGES, OFF_LAST / p.stage_bytes);
    CUtensorMap tmX, tmDY, tmD;
    MOE_REQUIRE(wgrad_maps(&tmX, &tmDY, &tmD, x, dy, p, f32), MOE_ERR_CUDA);
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = launch_cfg(std::min<int64_t>(p.max_tiles, max_clusters()), s, attr);
    const cudaError_t e = f32 ? cudaLaunchKernelEx(&cfg, k_wgrad<true>, tmX, tmDY, tmD, p)
                              : cudaLaunchKernelEx(&cfg, k_wgrad<false>, tmX, tmDY, tmD, p);
    if (e != cudaSuccess) return MOE_ERR_CUDA;
    MOE_CHECK_LAUNCH();
    return MOE_OK;
}

// dx = dz W^T (p) and dW = x^T dz (q) in one launch
static moe_status_t product_both(const Mat& dz, const Mat& x, const Mat& w, Params p, Params q, bool f32,
                                 cudaStream_t s) {
    MOE_REQUIRE(max_clusters() > 0, MOE_ERR_NOT_INITIALIZED);
    moe_status_t st = plan_rows<false>(p);
    if (st == MOE_OK) st = plan_wgrad(q);
    if (st != MOE_OK) return st;
    p.stage_bytes = q.stage_bytes = std::max(p.stage_bytes, q.stage_bytes);
    p.stages = q.stages = std::min(MAX_STAGES, OFF_LAST / p.stage_bytes);
    CUtensorMap tmW, tmZ[4], tmDX, tmX, tmDY, tmD;
    MOE_REQUIRE(make_bf16_map3(&tmW, w.p, p.G, w.rows, w.cols, w.ld, w.gs, 128) && rows_maps(tmZ, &tmDX, dz, p) &&
                    wgrad_maps(&tmX, &tmDY, &tmD, x, dz, q, f32),
                MOE_ERR_CUDA);
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = launch_cfg(std::min<int64_t>(p.max_tiles + q.max_tiles, max_clusters()), s, attr);
    const cudaError_t e =
        f32 ? cudaLaunchKernelEx(&cfg, k_both<true>, tmW, tmZ[0], tmZ[1], tmZ[2], tmZ[3], tmDX, tmX, tmDY, tmD, p, q)
            : cudaLaunchKernelEx(&cfg, k_both<false>, tmW, tmZ[0], tmZ[1], tmZ[2], tmZ[3], tmDX, tmX, tmDY, tmD, p, q);
    if (e != cudaSuccess) return MOE_ERR_CUDA;
    MOE_CHECK_LAUNCH();
    return MOE_OK;
}

static bool size_ok(int64_t v) { return v >= 1 && v <= 0x7FFFFF00LL; }
static bool row_ok(const void* p, int64_t ld) { return moe_aligned16(p) && ld % 8 == 0; }
// strides that mean nothing (of one row, of one group), as the maps want them
static int64_t stride_of(int64_t rows, int64_t cols, int64_t ld) {
    return rows == 1 && ld >= cols ? (cols + 7) / 8 * 8 : ld;
}
static int64_t group_stride_of(int G, int64_t rows, int64_t ld, int64_t gs) { return G == 1 ? rows * ld : gs; }
static bool groups_apart(int G, int64_t rows, int64_t cols, int64_t ld, int64_t gs) {
    return G == 1 || gs >= (rows - 1) * ld + cols;
}
static bool act_ok(int a) { return a >= MOE_ACT_NONE && a <= MOE_ACT_SILU; }
static bool groups_ok(const int32_t* offsets, const int32_t* rows) {
    return reinterpret_cast<uintptr_t>(offsets) % 4 == 0 && reinterpret_cast<uintptr_t>(rows) % 4 == 0;
}

// dx = dz W^T and dW = x^T dz, each if asked for; W_g [K, N]
static moe_status_t gradients(const Mat& dz, const Mat& x, const Mat& w, const Params& groups, int N, int K, void* dx,
                              int64_t lddx, void* dw, bool f32, int64_t lddw, int64_t gsdw, cudaStream_t s) {
    Params p = groups, q = groups;
    p.N = K, p.K = N, p.y = dx, p.ldy = lddx;
    q.N = N, q.K = K, q.y = dw, q.ldy = lddw, q.gsy = gsdw;
    // One launch saves a set-up and a last wave (16 groups' 300 rows, 515 x 259: 11.2 us,
    // 15.8 in two); long work runs faster in two (64 groups of 768 rows, 2,048 x
    // 7,168: 1.85 ms, 1.90 in one; 8,192 x 4,096 x 7,168 551 us, 567): up to about 1,000 steps of
    // 256 x 256 x 64 a pair.
    const double steps = 2. * groups.M * K * N / (256. * 256. * 64.);
    if (dx && dw && groups.M > 0 && steps < 1000. * max_clusters()) return product_both(dz, x, w, p, q, f32, s);
    if (dx && groups.M > 0) {
        const moe_status_t st = product_rows<false, false, 0>(dz, w, p, s);
        if (st != MOE_OK) return st;
    }
    return dw ? product_wgrad(x, dz, q, f32, s) : MOE_OK;
}

}  // namespace grouped

cudaError_t grouped_set_attributes() { return grouped::set_attributes(); }

}  // namespace moe

using namespace moe;
using grouped::group_stride_of;
using grouped::groups_apart;
using grouped::row_ok;
using grouped::size_ok;
using grouped::stride_of;

extern "C" moe_status_t grouped_linear_fwd(const void* x, int64_t ldx, const void* w, int64_t ldw, int64_t gsw,
                                           const int32_t* offsets, const int32_t* rows, int G, int64_t M, int N,
                                           int64_t K, void* y, int64_t ldy, int32_t* err, void* stream) {
    MOE_REQUIRE(M >= 0 && N >= 1 && K >= 1 && G >= 1, MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(ldx >= K && ldw >= N && ldy >= N && groups_apart(G, K, N, ldw, gsw), MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(M <= 0x7FFFFF00LL && size_ok(N) && size_ok(K) && G <= grouped::MAX_GROUPS, MOE_ERR_UNSUPPORTED);
    if (M == 0) return MOE_OK;
    MOE_REQUIRE(x && w && y && offsets, MOE_ERR_INVALID_ARG);
    ldx = stride_of(M, K, ldx), ldy = stride_of(M, N, ldy), ldw = stride_of(K, N, ldw);
    gsw = group_stride_of(G, K, ldw, gsw);
    MOE_REQUIRE(row_ok(x, ldx) && row_ok(w, ldw) && row_ok(y, ldy) && gsw % 8 == 0 && grouped::groups_ok(offsets, rows),
                MOE_ERR_ALIGNMENT);
    MOE_REQUIRE(device_initialized(), MOE_ERR_NOT_INITIALIZED);
    grouped::Params p{};
    p.offsets = offsets, p.rows = rows, p.G = G, p.M = M, p.N = N, p.K = (int)K;
    p.y = y, p.ldy = ldy, p.err = err;
    return grouped::product_rows<true, false, 0>({x, M, K, ldx, 0}, {w, K, N, ldw, gsw}, p, (cudaStream_t)stream);
}

extern "C" moe_status_t grouped_linear_bwd(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* w,
                                           int64_t ldw, int64_t gsw, const int32_t* offsets, const int32_t* rows, int G,
                                           int64_t M, int N, int64_t K, void* dx, int64_t lddx, void* dw, int dw_type,
                                           int64_t lddw, int64_t gsdw, int32_t* err, void* stream) {
    MOE_REQUIRE(M >= 0 && N >= 1 && K >= 1 && G >= 1 && (dx || dw), MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(dw_type == MOE_TYPE_BF16 || dw_type == MOE_TYPE_F32, MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(lddy >= N && (!dx || (ldw >= N && lddx >= K && groups_apart(G, K, N, ldw, gsw))) &&
                    (!dw || (ldx >= K && lddw >= N && groups_apart(G, K, N, lddw, gsdw))),
                MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(M <= 0x7FFFFF00LL && size_ok(N) && size_ok(K) && G <= grouped::MAX_GROUPS, MOE_ERR_UNSUPPORTED);
    MOE_REQUIRE(M == 0 || (dy && offsets && (!dx || w) && (!dw || x)), MOE_ERR_INVALID_ARG);
    lddy = stride_of(M, N, lddy), ldx = stride_of(M, K, ldx), lddx = stride_of(M, K, lddx);
    ldw = stride_of(K, N, ldw), lddw = stride_of(K, N, lddw);
    gsw = group_stride_of(G, K, ldw, gsw), gsdw = group_stride_of(G, K, lddw, gsdw);
    MOE_REQUIRE(row_ok(dy, lddy) && (!dx || (row_ok(w, ldw) && gsw % 8 == 0 && row_ok(dx, lddx))) &&
                    (!dw || (row_ok(x, ldx) && row_ok(dw, lddw) && gsdw % 8 == 0)) && grouped::groups_ok(offsets, rows),
                MOE_ERR_ALIGNMENT);
    MOE_REQUIRE(device_initialized(), MOE_ERR_NOT_INITIALIZED);
    grouped::Params p{};
    p.offsets = offsets, p.rows = rows, p.G = G, p.M = M, p.err = err;
    return grouped::gradients({dy, M, N, lddy, 0}, {x, M, K, ldx, 0}, {w, K, N, ldw, gsw}, p, N, (int)K, dx, lddx, dw,
                              dw_type == MOE_TYPE_F32, lddw, gsdw, (cudaStream_t)stream);
}

extern "C" moe_status_t grouped_ffn_fwd(const void* x, int64_t ldx, const void* w1, int64_t ldw, int64_t gsw, int act,
                                        const int32_t* offsets, const int32_t* rows, int G, int64_t M, int f, int64_t d,
                                        void* h, int64_t ldh, void* a, int64_t lda, int32_t* err, void* stream) {
    const int64_t f2 = 2 * (int64_t)f;
    MOE_REQUIRE(M >= 0 && f >= 1 && d >= 1 && G >= 1 && grouped::act_ok(act), MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(ldx >= d && ldw >= f2 && ldh >= f && (!a || lda >= f2) && groups_apart(G, d, f2, ldw, gsw),
                MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(f % 8 == 0 && M <= 0x7FFFFF00LL && f <= 0x3FFFFF00 && size_ok(d) && G <= grouped::MAX_GROUPS,
                MOE_ERR_UNSUPPORTED);
    if (M == 0) return MOE_OK;
    MOE_REQUIRE(x && w1 && h && offsets, MOE_ERR_INVALID_ARG);
    ldx = stride_of(M, d, ldx), ldw = stride_of(d, f2, ldw), ldh = stride_of(M, f, ldh), lda = stride_of(M, f2, lda);
    gsw = group_stride_of(G, d, ldw, gsw);
    MOE_REQUIRE(row_ok(x, ldx) && row_ok(w1, ldw) && row_ok(h, ldh) && (!a || row_ok(a, lda)) && gsw % 8 == 0 &&
                    grouped::groups_ok(offsets, rows),
                MOE_ERR_ALIGNMENT);
    MOE_REQUIRE(device_initialized(), MOE_ERR_NOT_INITIALIZED);
    grouped::Params p{};
    p.offsets = offsets, p.rows = rows, p.G = G, p.M = M, p.N = f, p.K = (int)d, p.up = f;
    p.y = h, p.ldy = ldh, p.a = static_cast<__nv_bfloat16*>(a), p.lda = lda, p.err = err;
    const grouped::Mat mx{x, M, d, ldx, 0}, mw{w1, d, f2, ldw, gsw};
    cudaStream_t s = (cudaStream_t)stream;
    switch (act) {
        case MOE_ACT_RELU: return grouped::product_rows<true, true, MOE_ACT_RELU>(mx, mw, p, s);
        case MOE_ACT_GELU: return grouped::product_rows<true, true, MOE_ACT_GELU>(mx, mw, p, s);
        case MOE_ACT_SILU: return grouped::product_rows<true, true, MOE_ACT_SILU>(mx, mw, p, s);
        default: return grouped::product_rows<true, true, MOE_ACT_NONE>(mx, mw, p, s);
    }
}

extern "C" moe_status_t grouped_ffn_bwd(const void* dh, int64_t lddh, const void* a, int64_t lda, const void* x,
                                        int64_t ldx, const void* w1, int64_t ldw, int64_t gsw, int act,
                                        const int32_t* offsets, const int32_t* rows, int G, int64_t M, int f, int64_t d,
                                        void* da, int64_t ldda, void* dx, int64_t lddx, void* dw1, int dw_type,
                                        int64_t lddw, int64_t gsdw, int32_t* err, void* stream) {
    const int64_t f2 = 2 * (int64_t)f;
    MOE_REQUIRE(M >= 0 && f >= 1 && d >= 1 && G >= 1 && grouped::act_ok(act), MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(dw_type == MOE_TYPE_BF16 || dw_type == MOE_TYPE_F32, MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(lddh >= f && lda >= f2 && ldda >= f2 &&
                    (!dx || (ldw >= f2 && lddx >= d && groups_apart(G, d, f2, ldw, gsw))) &&
                    (!dw1 || (ldx >= d && lddw >= f2 && groups_apart(G, d, f2, lddw, gsdw))),
                MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(f % 8 == 0 && M <= 0x7FFFFF00LL && f <= 0x3FFFFF00 && size_ok(d) && G <= grouped::MAX_GROUPS,
                MOE_ERR_UNSUPPORTED);
    MOE_REQUIRE(M == 0 || (dh && a && da && offsets && (!dx || w1) && (!dw1 || x)), MOE_ERR_INVALID_ARG);
    lddh = stride_of(M, f, lddh), lda = stride_of(M, f2, lda), ldda = stride_of(M, f2, ldda);
    ldx = stride_of(M, d, ldx), lddx = stride_of(M, d, lddx), ldw = stride_of(d, f2, ldw), lddw = stride_of(d, f2, lddw);
    gsw = group_stride_of(G, d, ldw, gsw), gsdw = group_stride_of(G, d, lddw, gsdw);
    MOE_REQUIRE(M == 0 || da != a || ldda == lda, MOE_ERR_INVALID_ARG);      // in place: row by row
    MOE_REQUIRE(row_ok(dh, lddh) && row_ok(a, lda) && row_ok(da, ldda) &&
                    (!dx || (row_ok(w1, ldw) && gsw % 8 == 0 && row_ok(dx, lddx))) &&
                    (!dw1 || (row_ok(x, ldx) && row_ok(dw1, lddw) && gsdw % 8 == 0)) && grouped::groups_ok(offsets, rows),
                MOE_ERR_ALIGNMENT);
    MOE_REQUIRE(device_initialized(), MOE_ERR_NOT_INITIALIZED);
    grouped::Params p{};
    p.offsets = offsets, p.rows = rows, p.G = G, p.M = M, p.err = err;
    cudaStream_t s = (cudaStream_t)stream;
    if (M > 0) {
        int tpr = 8;
        while (tpr < 256 && tpr * 8 < f) tpr *= 2;
        const int64_t blocks = std::min<int64_t>((M * tpr + 255) / 256, (int64_t)device_sm_count() * 8);
        grouped::Params q = p;
        q.N = f;
        if (launch_early(dim3((unsigned)blocks), 256, 0, s, grouped::k_glu_rows, static_cast<const __nv_bfloat16*>(dh),
                         lddh, static_cast<const __nv_bfloat16*>(a), lda, act, static_cast<__nv_bfloat16*>(da), ldda, tpr,
                         q) != cudaSuccess)
            return MOE_ERR_CUDA;
    }
    return grouped::gradients({da, M, f2, ldda, 0}, {x, M, d, ldx, 0}, {w1, d, f2, ldw, gsw}, p, (int)f2, (int)d, dx, lddx,
                              dw1, dw_type == MOE_TYPE_F32, lddw, gsdw, s);
}
