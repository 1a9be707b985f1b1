// Dense bf16 matrix products with fused epilogues: the gated feed-forward
// projections, the linear layer, and their backward passes.
//
// One kernel serves the three products of a layer y = x W (x [M, K], W [K, N],
// both row-major as they lie in memory):
//   forward            D[M, N] = x W        A = x  (K-major),  B = W  (N-major)
//   input gradient     D[M, K] = dy W^T     A = dy (K-major),  B = W  (K-major)
//   weight gradient    D[K, N] = x^T dy     A = x  (M-major),  B = dy (N-major)
// ("X-major": X is the contiguous axis.)  The tensor core takes either order
// of both operands, so nothing is transposed or copied beforehand.
//
// Tile: 256 x bn of D per CTA pair (tcgen05.mma.cta_group::2, M = 256,
// N = bn <= 256), 64 deep per pipeline stage; CTA r of the pair holds 128 of
// the A rows and bn / 2 of the B rows, 32 KB per stage with bn = 256.  Two
// accumulators of 256 TMEM columns, so that the epilogue of one tile runs
// under the next tile's products.  Per k-step the pair reads 64 KB for
// 256 x 256 x 64 products: half the operand traffic per SM of a 128 x 256
// tile on one SM.
// D leaves through shared memory: each epilogue warp stages 32 rows x 32
// columns and one TMA store writes them, clipped at D's edges, which
// leaves whole lines to the memory system and the warp free.
//
// When the tiles are too few for the SMs, `splits` pairs of a cluster share a
// tile, each with its part of K.  They swap their fp32 partial tiles through
// distributed shared memory, each pair adding up (in the order of the parts)
// and writing its share of the columns: no workspace, no atomics, the same
// bits on every run.
//
// Bound by the tensor cores under the power cap when the product is large
// (4,096 x 4,096 x 4,096 73 us, 1.87 PFLOP/s; gated 2,003 x 4,096 x 2 * 14,336 284 to
// 293 us, 1.61 to 1.66, from card to card, 240 in bursts too short for the cap),
// by set-up, first loads and last stores when it is small (512 x 512 x 512 4.3 us).
// Rows that start at no multiple of 128 bytes cost the TMA two lines for one:
// 4,096 x 4,096 x 4,096 then 105 to 120 us.
//
// Warps: 0 TMA, 1 MMA (of the leader CTA), 4-11 epilogue.  All waits are
// bounded, as in the grouped GEMM kernels.

#include <algorithm>

#include "pair_bf16.cuh"

namespace moe {

namespace dense {

using namespace gg;

constexpr int ACC_COLS = 256;                   // TMEM columns of an accumulator
constexpr int HALF_BYTES = 128 * TK * 2;        // one CTA's rows of an operand per stage
constexpr int MAX_STAGES = 8;
constexpr int NACC = 2;
constexpr int SMEM_TILES = 12 * HALF_BYTES;     // 6 stages with bn = 256, 8 with bn = 128
constexpr int OFF_EPI = SMEM_TILES;             // staging, 4 KB per epilogue warp
constexpr int EPI_STAGE = 4096;
constexpr int OFF_BAR = OFF_EPI + EPI_WARPS * EPI_STAGE;      // full[S], empty[S], tfull[A], tempty[A], drain
constexpr int NBAR = 2 * MAX_STAGES + 2 * NACC + 1;
constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;
constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory budget");
// a partial chunk of 128 rows x 32 columns on its way to another pair: rows
// of 36 words, so that the row-per-lane accesses meet no bank twice
constexpr int PART_ROW = 144;
constexpr int PART_BYTES = 128 * PART_ROW;

// Shared memory of a tile in parts, over the pipeline stages: from the start on
// the chunks that the other parts send, below the end the boxes on their way
// out, where a warp finds room for all of its units (a unit is what finish()
// takes: a chunk of 32 columns, GLU a gate and an up chunk).  A warp fills its
// boxes while others still read chunks, so the two must not overlap.
constexpr int swap_units(bool glu, int bn) { return glu ? bn / 64 : bn / 32; }
constexpr int swap_own(bool glu, int bn, int splits) { return (swap_units(glu, bn) + splits - 1) / splits; }
constexpr int swap_bytes(bool glu, int bn, int splits) {
    return (splits - 1) * swap_own(glu, bn, splits) * (glu ? 2 : 1) * PART_BYTES;
}
// of one warp, which takes every second unit: GLU three boxes of 2 KB a unit
// (gate, up, h), else two (z, y) or one of 4 KB (fp32)
constexpr int swap_boxes(bool glu, int bn, int splits) {
    return (swap_own(glu, bn, splits) + 1) / 2 * (glu ? 6144 : 4096);
}
constexpr int kWidths[] = {256, 224, 192, 128, 64};      // of a tile
constexpr int kMaxSplits = 4;
constexpr bool swap_fits() {
    for (int bn : kWidths)
        for (int splits = 2; splits <= kMaxSplits; ++splits)
            for (int glu = 0; glu < 2; ++glu)
                if (swap_bytes(glu, bn, splits) + EPI_WARPS * swap_boxes(glu, bn, splits) > SMEM_TILES) return false;
    return true;
}
static_assert(swap_fits(), "boxes over chunks that other warps read");

// What the epilogue makes of the product v:
//   EPI_PLAIN   y = v (bf16)
//   EPI_F32     y = v (fp32)
//   EPI_LINEAR  z = v + bias; y = act(z) + residual (bf16; z stored when asked for)
//   EPI_GLU     columns [0, bn / 2) of the tile are gate, [bn / 2, bn) up:
//               h = act(gate) * up; a = [gate | up] stored when asked for
// (the activation is a template argument of the pair kernel: an epilogue of
// 32 columns in registers, unrolled for each of four activations, would be
// fetched from memory at every launch's first tile)
enum { EPI_PLAIN = 0, EPI_F32 = 1, EPI_LINEAR = 2, EPI_GLU = 3 };

struct Params {
    int64_t M;              // rows and columns of D (GLU: N = f)
    int N;
    int64_t K;
    int m_tiles, n_tiles, nk, band;
    int bn;                 // columns of the pair's tile
    int stages, stage_bytes;
    int splits;             // pairs that share a tile (cluster of 2 * splits)
    int up;                 // GLU: column of W where the up half begins
    int act;
    void* y;                // bf16, EPI_F32: fp32
    int64_t ldy;
    __nv_bfloat16* z;       // EPI_LINEAR: z, EPI_GLU: a; may be NULL
    int64_t ldz;
    const __nv_bfloat16* bias;
    const __nv_bfloat16* res;
    int64_t ldres;
    int32_t* err;
    uint64_t timeout_ns;
};

// 32 columns of one row from memory; `n` of them exist.  Rows start at
// multiples of 16 bytes and columns at multiples of 32.  (Plain loads: the
// residual may be y itself, which this kernel writes.)
__device__ __forceinline__ void load32(const __nv_bfloat16* p, int n, float* f) {
    if (n >= 32) {
#pragma unroll
        for (int g = 0; g < 4; ++g) unpack8(reinterpret_cast<const uint4*>(p)[g], f + 8 * g);
    } else {
#pragma unroll
        for (int g = 0; g < 4; ++g)
            unpack8(n > 8 * g ? load_vec8(p + 8 * g, min(n - 8 * g, 8)) : make_uint4(0u, 0u, 0u, 0u), f + 8 * g);
    }
}
// The last n % 8 of the n < 32 columns of a row from `p` on.
template <typename T>
__device__ __forceinline__ void store_tail(T* p, int n, const float* v) {
#pragma unroll
    for (int i = 0; i < 31; ++i) {
        if (i < n && i >= (n & ~7)) {
            if constexpr (sizeof(T) == 4) p[i] = v[i];
            else p[i] = __float2bfloat16_rn(v[i]);
        }
    }
}

// A warp's way out: 32 rows (one per lane) x 32 columns staged in shared
// memory and written by a TMA store (bf16: boxes of 2 KB, 64-byte swizzle;
// fp32: 4 KB, 128-byte swizzle; either way the row-per-lane stores to shared
// memory meet no bank twice).  While tiles follow, a warp has 4 KB, two
// bf16 boxes or one fp32 box, and waits until a box has been read before it
// fills it again; its last tile goes through the pipeline stages, free
// by then, 16 KB a warp, where every chunk finds a box of its own and one
// fence and one round of stores at the end do for all.
struct Out {
    uint32_t buf, last;
    int lane;
    uint32_t at;          // bytes of the buffer used so far
    bool wide;            // the last tile
    __device__ __forceinline__ void last_tile() { wide = true, at = 0; }
    __device__ __forceinline__ void send(const CUtensorMap* map, uint32_t b, int col, int64_t row0) {
        if (wide) return;      // flush()
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
            tma_store_2d(map, b, col, (int)row0);
            bulk_commit_group();
        }
    }
    __device__ __forceinline__ void bf16(const CUtensorMap* map, int col, int64_t row0, const float* v) {
        const uint32_t b = wide ? last + at : buf + (at & 2048u);
        at += 2048u;
        if (!wide) {
            if (lane == 0) bulk_wait_group_read1();      // the box before the last one has been read
            __syncwarp();
        }
        const uint32_t row = b + 64u * lane, sw = (uint32_t)(lane >> 1) & 3u;
#pragma unroll
        for (int c = 0; c < 4; ++c)
            st_shared_v4(row + (((uint32_t)c ^ sw) << 4), pack_bf16x2(v[8 * c], v[8 * c + 1]),
                         pack_bf16x2(v[8 * c + 2], v[8 * c + 3]), pack_bf16x2(v[8 * c + 4], v[8 * c + 5]),
                         pack_bf16x2(v[8 * c + 6], v[8 * c + 7]));
        send(map, b, col, row0);
    }
    __device__ __forceinline__ void f32(const CUtensorMap* map, int col, int64_t row0, const float* v) {
        const uint32_t b = wide ? last + at : buf;
        at += 4096u;
        if (!wide) {
            if (lane == 0) bulk_wait_group_read0();
            __syncwarp();
        }
        const uint32_t row = b + 128u * lane, sw = (uint32_t)lane & 7u;
#pragma unroll
        for (int c = 0; c < 8; ++c)
            st_shared_v4(row + (((uint32_t)c ^ sw) << 4), __float_as_uint(v[4 * c]), __float_as_uint(v[4 * c + 1]),
                         __float_as_uint(v[4 * c + 2]), __float_as_uint(v[4 * c + 3]));
        send(map, b, col, row0);
    }
};
static_assert(8 * EPI_WARPS * 2048 <= SMEM_TILES, "the last tile's boxes (z and y of four chunks)");

// Tiles in bands of p.band row tiles, consecutive ones down a band, so that
// the tiles under way at a time share operand tiles in L2.
struct Tile {
    int mt, nt;
};
__device__ __forceinline__ Tile get_tile(const Params& p, int t) {
    const int band_tiles = p.band * p.n_tiles, b = t / band_tiles, rem = t - b * band_tiles;
    const int m0 = b * p.band, bw = min(p.band, p.m_tiles - m0);
    Tile r;
    r.nt = rem / bw;
    r.mt = m0 + rem - r.nt * bw;
    return r;
}
__device__ __forceinline__ void st_cluster_v4(uint32_t addr, const float* v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                 "f"(v[3])
                 : "memory");
}

// 32 columns of a warp's 32 rows from the product (v; GLU: gate v and up u)
// to memory.  `col`: the first one in D, `n` of them exist (n > 0).
template <int EPI, int ACT>
__device__ __forceinline__ void finish(const Params& p, const CUtensorMap* tmY, const CUtensorMap* tmZ,
                                       const CUtensorMap* tmZ2, Out& out, int64_t row0, int64_t row, int col, int n,
                                       float* v, float* u) {
    // a TMA store is clipped at D's edge to whole 16 bytes: of a width that is
    // no multiple of 8 the boxes end at the last one, and the columns after it
    // are stored from here (GLU: f is a multiple)
    const bool tail = EPI != EPI_GLU && n < 32 && (n & 7) != 0, box = !tail || n > 8;
    if constexpr (EPI == EPI_GLU) {
        if (p.z != nullptr) {
            out.bf16(tmZ, col, row0, v);
            out.bf16(tmZ2, col, row0, u);
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) u[i] *= act_of(v[i], ACT);
        out.bf16(tmY, col, row0, u);
    } else if constexpr (EPI == EPI_F32) {
        if (box) out.f32(tmY, col, row0, v);
        if (tail && row < p.M) store_tail(static_cast<float*>(p.y) + row * p.ldy + col, n, v);
    } else {
        if constexpr (EPI == EPI_LINEAR) {
            if (p.bias != nullptr) {
                const float b = out.lane < n ? __bfloat162float(p.bias[col + out.lane]) : 0.f;
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] += __shfl_sync(0xFFFFFFFFu, b, i);
            }
            if (p.z != nullptr) {
                if (box) out.bf16(tmZ, col, row0, v);
                if (tail && row < p.M) store_tail(p.z + row * p.ldz + col, n, v);
            }
            if constexpr (ACT != MOE_ACT_NONE) {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = act_of(v[i], ACT);
            }
            if (p.res != nullptr && row < p.M) {
                float r[32];
                load32(p.res + row * p.ldres + col, n, r);
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] += r[i];
            }
        }
        if (box) out.bf16(tmY, col, row0, v);
        if (tail && row < p.M) store_tail(static_cast<__nv_bfloat16*>(p.y) + row * p.ldy + col, n, v);
    }
}

// The last tile's boxes go out, in the order in which finish() filled them:
// chunks [c0, c1) at `stride` of the tile whose first column in D is col0.
template <int EPI>
__device__ __forceinline__ void flush(const Params& p, const CUtensorMap* tmY, const CUtensorMap* tmZ,
                                      const CUtensorMap* tmZ2, Out& out, int64_t row0, int col0, int c0, int c1,
                                      int stride) {
    fence_proxy_async_shared();
    __syncwarp();
    if (out.lane != 0 || row0 >= p.M) return;
    uint32_t b = out.last;
    for (int c = c0; c < c1; c += stride) {
        const int col = col0 + 32 * c, n = p.N - col;
        if (n <= 0 || (EPI != EPI_GLU && n < 8)) continue;
        if (EPI == EPI_LINEAR || EPI == EPI_GLU) {
            if (p.z != nullptr) {
                tma_store_2d(tmZ, b, col, (int)row0);
                b += 2048u;
                if (EPI == EPI_GLU) {
                    tma_store_2d(tmZ2, b, col, (int)row0);
                    b += 2048u;
                }
            }
        }
        tma_store_2d(tmY, b, col, (int)row0);
        b += EPI == EPI_F32 ? 4096u : 2048u;
    }
    bulk_commit_group();
}

// A CTA's place: in its pair, in the grid, in shared memory.
struct Place {
    uint8_t* smem;
    uint32_t bar0, rank, lead;      // rank in the pair; the pair's leader in the cluster
    int warp, lane, first, step;    // the pair's tiles: first, first + step, ..
    volatile int* abort_flag;
    __device__ __forceinline__ uint32_t full_bar(int s) const { return bar0 + 8u * s; }
    __device__ __forceinline__ uint32_t empty_bar(int s) const { return bar0 + 8u * (MAX_STAGES + s); }
    __device__ __forceinline__ uint32_t tfull_bar(int a) const { return bar0 + 8u * (2 * MAX_STAGES + a); }
    __device__ __forceinline__ uint32_t tempty_bar(int a) const { return bar0 + 8u * (2 * MAX_STAGES + NACC + a); }
    __device__ __forceinline__ uint32_t drain_bar() const { return bar0 + 8u * (2 * MAX_STAGES + 2 * NACC); }
};
// Barriers, TMEM; returns what the warps that use TMEM have to know of it.
__device__ __forceinline__ uint32_t set_up(Place& pl, int splits, int stages) {
    extern __shared__ uint8_t smem_raw[];
    pl.smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    pl.warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0), pl.lane = threadIdx.x & 31;
    const uint32_t crank = cluster_ctarank();
    pl.rank = crank & 1u, pl.lead = crank & ~1u;
    pl.first = blockIdx.x / (2 * splits), pl.step = gridDim.x / (2 * splits);
    pl.bar0 = smem_u32(pl.smem + OFF_BAR);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(pl.smem + OFF_MISC);
    pl.abort_flag = reinterpret_cast<volatile int*>(pl.smem + OFF_MISC + 4);
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(pl.full_bar(s), 1);
            mbar_init(pl.empty_bar(s), 1);
        }
        for (int a = 0; a < NACC; ++a) {
            mbar_init(pl.tfull_bar(a), 1);
            mbar_init(pl.tempty_bar(a), 2 * EPI_WARPS);
        }
        mbar_init(pl.drain_bar(), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        *pl.abort_flag = 0;
    }
    __syncthreads();
    cluster_sync();      // the peer's barriers are initialised
    // TMEM is for the MMA and epilogue warps to wait for; the producer loads
    if (pl.warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(TMEM_COLS));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        tc_fence_before();
    }
    if (pl.warp == 1 || pl.warp >= 4) {
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

// The TMA warp: k-steps [k0, k1) of the product's tiles, which are tiles
// [t0, t1) of the launch; t: the pair's next one.
template <bool A_MN, bool B_MN, int EPI>
__device__ __forceinline__ void load_tiles(const Place& pl, const Params& p, const CUtensorMap* tmA,
                                           const CUtensorMap* tmB, int k0, int k1, int& t, int t0, int t1, Ring& r) {
    const bool elected = elect_one();
    const uint32_t lead_full = mapa(pl.full_bar(0), pl.lead);
    // B: bn / 2 rows, or bn / 2 columns in boxes of 64
    const int bh = p.bn / 2, b_boxes = (bh + 63) / 64;
    const uint32_t bytes = HALF_BYTES + (B_MN ? 64 * b_boxes : bh) * TK * 2;
    for (; t < t1 && !r.aborted; t += pl.step) {
        const Tile ti = get_tile(p, t - t0);
        const int am = ti.mt * TM + 128 * (int)pl.rank;
        const int bn = EPI == EPI_GLU ? ti.nt * bh + p.up * (int)pl.rank : ti.nt * p.bn + bh * (int)pl.rank;
        for (int ks = k0; ks < k1; ++ks) {
            if (!mbar_wait_cluster(pl.empty_bar(r.at), r.phase ^ 1u, p, pl.abort_flag)) {
                r.aborted = true;
                break;
            }
            const int k = ks * TK;
            // both CTAs' bytes complete on the leader's full barrier
            const uint32_t fb = lead_full + 8u * r.at;
            if (elected) {
                if (pl.rank == 0) mbar_expect_tx(pl.full_bar(r.at), 2u * bytes);
                const uint32_t sa = smem_u32(pl.smem + r.at * p.stage_bytes), sb = sa + HALF_BYTES;
                if constexpr (A_MN) {
                    tma2_load_2d(sa, tmA, am, k, fb);
                    tma2_load_2d(sa + HALF_BYTES / 2, tmA, am + 64, k, fb);
                } else {
                    tma2_load_2d(sa, tmA, k, am, fb);
                }
                if constexpr (B_MN) {
                    tma2_load_2d(sb, tmB, bn, k, fb);
                    if (b_boxes > 1) tma2_load_2d(sb + HALF_BYTES / 2, tmB, bn + 64, k, fb);
                } else {
                    tma2_load_2d(sb, tmB, k, bn, fb);
                }
            }
            r.next(p.stages);
        }
    }
}
// After an abort: wait (bounded) for the copies in flight.  The leader's full
// barriers count both CTAs' bytes, and the follower leaves only after the
// closing cluster barrier, i.e. after this.
__device__ __forceinline__ void loads_end(const Place& pl, const Params& p, const Ring& r) {
    __syncwarp();
    if (!r.aborted || pl.rank != 0) return;
    Params q = p;
    q.timeout_ns = 200000000ull;
    volatile int no_abort = 0;
    for (int i = r.count - min(r.count, p.stages); i < r.count; ++i)
        mbar_wait_cluster(pl.full_bar(i % p.stages), (uint32_t)(i / p.stages) & 1u, q, &no_abort);
}

// The MMA warp of the pair's leader.  The whole warp goes through the loop,
// one elected lane issues: with warp-uniform control the descriptors stay in
// uniform registers, and the loop has to be short -- a k-step's four products
// take 512 cycles.  (`ring`: stages; `acc`: accumulators)
template <bool A_MN, bool B_MN>
__device__ __forceinline__ void multiply_tiles(const Place& pl, const Params& p, uint32_t tmem_base, int k0, int k1,
                                               int& t, int t1, Ring& ring, Ring& acc) {
    const bool elected = elect_one();
    const uint32_t idesc = make_idesc_pair<A_MN, B_MN>(p.bn);
    const uint64_t adesc0 = operand_desc<A_MN>(smem_u32(pl.smem));
    const uint64_t bdesc0 = operand_desc<B_MN>(smem_u32(pl.smem) + HALF_BYTES);
    const uint32_t stage_step = (uint32_t)p.stage_bytes >> 4;
    for (; t < t1 && !ring.aborted; t += pl.step) {
        if (!mbar_wait_cluster(pl.tempty_bar(acc.at), acc.phase ^ 1u, p, pl.abort_flag)) {
            ring.aborted = true;
            break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(acc.at * ACC_COLS);
        for (int ks = k0; ks < k1; ++ks) {
            if (!mbar_wait(pl.full_bar(ring.at), ring.phase, p, pl.abort_flag)) {
                ring.aborted = true;
                break;
            }
            tc_fence_after();
            if (elected) {
                const uint64_t adesc = adesc0 + ring.at * stage_step, bdesc = bdesc0 + ring.at * stage_step;
#pragma unroll
                for (int kk = 0; kk < TK / 16; ++kk)
                    tc_mma2_bf16(d_tmem, adesc + k16_step<A_MN>() * kk, bdesc + k16_step<B_MN>() * kk, idesc,
                                 (ks != k0 || kk != 0) ? 1u : 0u);
                tc_commit_pair(pl.empty_bar(ring.at), pl.lead);
            }
            ring.next(p.stages);
        }
        if (ring.aborted) break;
        if (elected) tc_commit_pair(pl.tfull_bar(acc.at), pl.lead);
        acc.next(NACC);
    }
}
// wait (bounded) for the products issued
__device__ __forceinline__ void products_end(const Place& pl, const Params& p, const Ring& ring) {
    if (ring.count > 0) {
        if (elect_one()) tc_commit_local2(pl.drain_bar());
        Params q = p;
        q.timeout_ns = 200000000ull;
        volatile int no_abort = 0;
        mbar_wait(pl.drain_bar(), 0, q, &no_abort);
    }
    __syncwarp();
}

// An epilogue warp (its 32 rows of the accumulator, its half of the columns);
// the launch has `total` tiles.
template <int EPI, int ACT>
__device__ __forceinline__ void store_tiles(const Place& pl, const Params& p, const CUtensorMap* tmY,
                                            const CUtensorMap* tmZ, const CUtensorMap* tmZ2, Out& out,
                                            uint32_t lane_base, int& t, int t0, int t1, int total, Ring& acc) {
    const int quarter = (pl.warp - 4) & 3, half = (pl.warp - 4) >> 2, lane = pl.lane;
    // this warp's chunks of 32 columns: the first or the second half of them
    const int chunks = EPI == EPI_GLU ? p.bn / 64 : p.bn / 32;
    const int c0 = half == 0 ? 0 : (chunks + 1) / 2, c1 = half == 0 ? (chunks + 1) / 2 : chunks;
    for (; t < t1 && !acc.aborted; t += pl.step) {
        const Tile ti = get_tile(p, t - t0);
        const int64_t row0 = (int64_t)ti.mt * TM + 128 * pl.rank + quarter * 32;
        if (!mbar_wait_cluster(pl.tfull_bar(acc.at), acc.phase, p, pl.abort_flag)) {
            acc.aborted = true;
            break;
        }
        tc_fence_after();
        if (t + pl.step >= total) out.last_tile();
        const uint32_t tacc = lane_base + (uint32_t)(acc.at * ACC_COLS);
        const int col0 = ti.nt * (EPI == EPI_GLU ? p.bn / 2 : p.bn);
        uint32_t v[32], u[EPI == EPI_GLU ? 32 : 1];
        tmem_ld32_issue(tacc + 32 * c0, v);
        if constexpr (EPI == EPI_GLU) tmem_ld32_issue(tacc + p.bn / 2 + 32 * c0, u);
        for (int c = c0; c < c1; ++c) {
            float fv[32], fu[EPI == EPI_GLU ? 32 : 1];
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) fv[i] = __uint_as_float(v[i]);
            if constexpr (EPI == EPI_GLU) {
#pragma unroll
                for (int i = 0; i < 32; ++i) fu[i] = __uint_as_float(u[i]);
            }
            if (c + 1 < c1) {      // the next chunk is on its way while this one is worked on
                tmem_ld32_issue(tacc + 32 * (c + 1), v);
                if constexpr (EPI == EPI_GLU) tmem_ld32_issue(tacc + p.bn / 2 + 32 * (c + 1), u);
            } else if (!out.wide) {      // the accumulator is read: the next tile may have it
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(mapa(pl.tempty_bar(acc.at), pl.lead));
            }
            const int col = col0 + 32 * c, n = p.N - col;
            if (n > 0 && row0 < p.M)      // the whole warp
                finish<EPI, ACT>(p, tmY, tmZ, tmZ2, out, row0, row0 + lane, col, n, fv, fu);
        }
        if (out.wide) flush<EPI>(p, tmY, tmZ, tmZ2, out, row0, col0, c0, c1, 1);
        acc.next(NACC);
    }
}
__device__ __forceinline__ void stores_end(int lane) {
    if (lane == 0) bulk_wait_group0();      // the stores are complete
    __syncwarp();
}

// tmY, tmZ, tmZ2: y (h), z (a's gate half) and a's up half as TMA stores see
// them, boxes of 32 columns x 32 rows.
template <bool A_MN, bool B_MN, int EPI, int ACT>
__global__ void __launch_bounds__(THREADS, 1)
    k_dense_pair(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmZ,
                 const __grid_constant__ CUtensorMap tmZ2, const Params p) {
    if (threadIdx.x == 64) {
        prefetch_map(&tmA);
        prefetch_map(&tmB);
        prefetch_map(&tmY);
    }
    Place pl;
    const uint32_t tmem_base = set_up(pl, p.splits, p.stages);
    const int part = (int)(pl.lead >> 1);      // of K
    const int k0 = p.nk / p.splits * part + min(part, p.nk % p.splits);
    const int k1 = k0 + p.nk / p.splits + (part < p.nk % p.splits);
    wait_for_previous_kernels();

    const int total = p.m_tiles * p.n_tiles;
    const int warp = pl.warp, lane = pl.lane, ew = warp - 4, quarter = ew & 3, half = ew >> 2;
    const uint32_t lane_base = tmem_base + ((uint32_t)(quarter * 32) << 16);
    Out out{smem_u32(pl.smem + OFF_EPI + ew * EPI_STAGE), smem_u32(pl.smem + ew * 16384), lane, 0u, false};
    int t = pl.first;
    Ring ring, acc;
    if (warp == 0) {
        load_tiles<A_MN, B_MN, EPI>(pl, p, &tmA, &tmB, k0, k1, t, 0, total, ring);
        loads_end(pl, p, ring);
    } else if (warp == 1 && pl.rank == 0) {
        multiply_tiles<A_MN, B_MN>(pl, p, tmem_base, k0, k1, t, total, ring, acc);
        products_end(pl, p, ring);
    } else if (warp >= 4 && p.splits == 1) {
        store_tiles<EPI, ACT>(pl, p, &tmY, &tmZ, &tmZ2, out, lane_base, t, 0, total, total, acc);
        stores_end(lane);
    }
    if (p.splits > 1) {
        // ------------------------- one tile per cluster: swap and add up ----
        // Part j owns units [j * own, (j + 1) * own), those that exist.
        constexpr bool GLU = EPI == EPI_GLU;
        constexpr int CPU = GLU ? 2 : 1;      // chunks per unit
        const int units = swap_units(GLU, p.bn), own = swap_own(GLU, p.bn, p.splits);
        const int u0 = part * own, u1 = min(u0 + own, units);
        const uint32_t buf = smem_u32(pl.smem);
        const int r = quarter * 32 + lane;
        bool ok = true;
        __syncwarp();
        if (warp >= 4) {
            ok = mbar_wait_cluster(pl.tfull_bar(0), 0, p, pl.abort_flag);
            tc_fence_after();
        }
        cluster_sync();      // every part's products are done: its stages are free to write to
        if (warp >= 4 && ok) {
            for (int un = half; un < units; un += 2) {
                const int to = un / own;
                if (to == part) continue;
                const int slot = part < to ? part : part - 1;      // of the receiver's other parts
#pragma unroll
                for (int c = 0; c < CPU; ++c) {
                    float v[32];
                    tmem_ld32(lane_base + (uint32_t)(32 * un + (c == 0 ? 0 : p.bn / 2)), v);
                    const int chunk = (slot * own + un - to * own) * CPU + c;
                    const uint32_t at = buf + (uint32_t)(chunk * PART_BYTES + r * PART_ROW);
                    const uint32_t dst = mapa(at, (uint32_t)(2 * to) + pl.rank);
#pragma unroll
                    for (int i = 0; i < 8; ++i) st_cluster_v4(dst + 16u * i, v + 4 * i);
                }
            }
        }
        cluster_sync();      // every part has what it adds up
        if (warp >= 4 && ok) {
            const Tile ti = get_tile(p, pl.first);
            const int64_t row0 = (int64_t)ti.mt * TM + 128 * pl.rank + quarter * 32;
            const int col0 = ti.nt * (EPI == EPI_GLU ? p.bn / 2 : p.bn);
            out.last = smem_u32(pl.smem + SMEM_TILES - (ew + 1) * swap_boxes(GLU, p.bn, p.splits));
            out.last_tile();
            for (int un = u0 + half; un < u1; un += 2) {
                float s[2][32];
#pragma unroll
                for (int c = 0; c < CPU; ++c) {
                    float v[32];
                    tmem_ld32(lane_base + (uint32_t)(32 * un + (c == 0 ? 0 : p.bn / 2)), v);
#pragma unroll
                    for (int i = 0; i < 32; ++i) s[c][i] = 0.f;
                    for (int j = 0; j < p.splits; ++j) {
                        if (j == part) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) s[c][i] += v[i];
                            continue;
                        }
                        const int slot = j < part ? j : j - 1;
                        const float4* q = reinterpret_cast<const float4*>(
                            pl.smem + ((slot * own + un - u0) * CPU + c) * PART_BYTES + r * PART_ROW);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 x = q[i];
                            s[c][4 * i] += x.x, s[c][4 * i + 1] += x.y, s[c][4 * i + 2] += x.z, s[c][4 * i + 3] += x.w;
                        }
                    }
                }
                const int col = col0 + 32 * un, n = p.N - col;
                if (n > 0 && row0 < p.M)
                    finish<EPI, ACT>(p, &tmY, &tmZ, &tmZ2, out, row0, row0 + lane, col, n, s[0], s[1]);
            }
            flush<EPI>(p, &tmY, &tmZ, &tmZ2, out, row0, col0, u0 + half, u1, 2);
            if (lane == 0) bulk_wait_group0();
            __syncwarp();
        }
    }

    tear_down(pl, tmem_base);
}

// The two products of a backward pass, dx = dz W^T (p) and dW = x^T dz (q), as
// the tiles of one launch.  One set-up and one last wave instead of two (us,
// in two launches): 512 x 512 x 512 4.4 (8.3), 1,024 x 1,024 x 1,024 6.9 (11.8), 1,839 x
// 314 x 3,013 10.9 (19.2), 2,048 x 2,048 x 2,048 23.3 (28.8), 4,096 x 4,096 x 4,096 140 (149).
template <int EPI_W>
__global__ void __launch_bounds__(THREADS, 1)
    k_dense_both(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmA2,
                 const __grid_constant__ CUtensorMap tmB2, const __grid_constant__ CUtensorMap tmY2, const Params p,
                 const Params q) {
    if (threadIdx.x == 64) {
        prefetch_map(&tmA);
        prefetch_map(&tmB);
        prefetch_map(&tmA2);
        prefetch_map(&tmB2);
    }
    Place pl;
    const uint32_t tmem_base = set_up(pl, 1, p.stages);
    wait_for_previous_kernels();

    const int mid = p.m_tiles * p.n_tiles, total = mid + q.m_tiles * q.n_tiles;
    const int ew = pl.warp - 4;
    const uint32_t lane_base = tmem_base + ((uint32_t)((ew & 3) * 32) << 16);
    int t = pl.first;
    Ring ring, acc;
    if (pl.warp == 0) {
        load_tiles<false, false, EPI_PLAIN>(pl, p, &tmA, &tmB, 0, p.nk, t, 0, mid, ring);
        load_tiles<true, true, EPI_W>(pl, q, &tmA2, &tmB2, 0, q.nk, t, mid, total, ring);
        loads_end(pl, p, ring);
    } else if (pl.warp == 1 && pl.rank == 0) {
        multiply_tiles<false, false>(pl, p, tmem_base, 0, p.nk, t, mid, ring, acc);
        multiply_tiles<true, true>(pl, q, tmem_base, 0, q.nk, t, total, ring, acc);
        products_end(pl, p, ring);
    } else if (pl.warp >= 4) {
        Out out{smem_u32(pl.smem + OFF_EPI + ew * EPI_STAGE), smem_u32(pl.smem + ew * 16384), pl.lane, 0u, false};
        store_tiles<EPI_PLAIN, 0>(pl, p, &tmY, &tmY, &tmY, out, lane_base, t, 0, mid, total, acc);
        store_tiles<EPI_W, 0>(pl, q, &tmY2, &tmY2, &tmY2, out, lane_base, t, mid, total, total, acc);
        stores_end(pl.lane);
    }
    tear_down(pl, tmem_base);
}

// ------------------------------------------------------- few rows ----
//
// With few rows of x the product is the reading of W, and 256 x 256 tiles
// would leave most SMs without one.  Here the roles are swapped: W is the A
// operand (128 of its columns, or rows for the input gradient, are the M of
// the MMA) and up to 128 rows of x are its N, so a tile costs what the rows
// cost.  The contraction is split over the S CTAs of a cluster; each leaves
// its fp32 partial tile in its shared memory, and after a cluster barrier
// each CTA adds every S-th row over all of them, in rank order, and runs the
// epilogue on it (no workspace, no atomics, the same bits on every run).
// About 96 KB of shared memory per CTA, so that two share an SM and one's
// reduction runs under the other's loads.  Bound by the reading of W: 1 x 14,336
// x 4,096 21 us, 5.6 TB/s; 4 rows gated, 4,096 x 2 * 14,336, 37 us, 6.3 TB/s.
namespace few {

constexpr int ROWS = 128;                       // most rows of x per tile
constexpr int W_BYTES = 128 * TK * 2;
constexpr int SMEM_TILES = 98304;               // pipeline stages, then the partial tile
constexpr int MAX_STAGES = 5;
constexpr int OFF_BAR = SMEM_TILES;             // full[S], empty[S], done
constexpr int OFF_MISC = OFF_BAR + 8 * (2 * MAX_STAGES + 1);
constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;
constexpr int THREADS = 256;                    // warps 0 and 1 load and multiply, all of them join the parts

struct Split {
    int rows;          // rows of x per tile, padded to 16
    int stages;
    int splits;        // CTAs of a cluster
    uint32_t tmem_cols;
};

__device__ __forceinline__ void ld_cluster_v4(uint32_t addr, float* v) {
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                 : "r"(addr));
}
// 32 lanes x 16 columns
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* v) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// 4 columns of a row; `n` of them exist, columns start at multiples of 4
__device__ __forceinline__ void load4(const __nv_bfloat16* p, int n, float* f) {
    if (n >= 4) {
        const uint2 q = *reinterpret_cast<const uint2*>(p);
        f[0] = __uint_as_float(q.x << 16), f[1] = __uint_as_float(q.x & 0xFFFF0000u);
        f[2] = __uint_as_float(q.y << 16), f[3] = __uint_as_float(q.y & 0xFFFF0000u);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = i < n ? __bfloat162float(p[i]) : 0.f;
    }
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, int n, const float* f) {
    if (n >= 4) {
        *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) p[i] = __float2bfloat16_rn(f[i]);
    }
}

// 4 columns a lane of a row of the tile, from the product to memory (GLU:
// lanes 0..15 hold gate columns, lanes 16..31 the up columns of the same h).
template <int EPI>
__device__ __forceinline__ void finish_row(const Params& p, int64_t row, int nt, int lane, float* v) {
    if constexpr (EPI == EPI_GLU) {
        float u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = __shfl_down_sync(0xFFFFFFFFu, v[i], 16);
        const int col = nt * 64 + lane * 4, n = p.N - col;
        if (lane < 16 && n > 0) {
            if (p.z != nullptr) {
                store4(p.z + row * p.ldz + col, n, v);
                store4(p.z + row * p.ldz + p.N + col, n, u);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] *= act_of(v[i], p.act);
            store4(static_cast<__nv_bfloat16*>(p.y) + row * p.ldy + col, n, u);
        }
    } else {
        const int col = nt * 128 + lane * 4, n = p.N - col;
        if (n <= 0) return;
        if (p.bias != nullptr) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] += i < n ? __bfloat162float(p.bias[col + i]) : 0.f;
        }
        if (p.z != nullptr) store4(p.z + row * p.ldz + col, n, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = act_of(v[i], p.act);
        if (p.res != nullptr) {
            float q[4];
            load4(p.res + row * p.ldres + col, n, q);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] += q[i];
        }
        store4(static_cast<__nv_bfloat16*>(p.y) + row * p.ldy + col, n, v);
    }
}

// Rows rank, rank + splits, ... of the tile from the parts' partial tiles
// ([rows][128] fp32 at `part` of each CTA): a warp takes a row, 4 columns a
// lane.  ROWS rows and PARTS parts of each are on their way at a time; one
// after the other, 128 rows were joined at the latency of distributed shared memory.
template <int EPI, int ROWS, int PARTS>
__device__ __forceinline__ void join(const Params& p, const Split& s, uint32_t part, uint32_t rank, int64_t m0, int m,
                                     int nt) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int stride = s.splits * (THREADS / 32);
    for (int r0 = (int)rank + s.splits * warp; r0 < m; r0 += stride * ROWS) {
        float v[ROWS][4];
#pragma unroll
        for (int j = 0; j < ROWS; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[j][i] = 0.f;
        for (int c0 = 0; c0 < s.splits; c0 += PARTS) {      // splits is a multiple of PARTS
            float q[ROWS][PARTS][4];
#pragma unroll
            for (int j = 0; j < ROWS; ++j) {
                const int r = r0 + j * stride;
                if (r >= m) continue;
#pragma unroll
                for (int c = 0; c < PARTS; ++c)
                    ld_cluster_v4(mapa(part + (uint32_t)(r * 128 + lane * 4) * 4u, (uint32_t)(c0 + c)), q[j][c]);
            }
#pragma unroll
            for (int j = 0; j < ROWS; ++j)
#pragma unroll
                for (int c = 0; c < PARTS; ++c)
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[j][i] += q[j][c][i];      // (rows past the end: not used)
        }
#pragma unroll
        for (int j = 0; j < ROWS; ++j)
            if (r0 + j * stride < m) finish_row<EPI>(p, m0 + r0 + j * stride, nt, lane, v[j]);      // the whole warp
    }
}

// tmW: W, boxes of 64 columns x 64 k (W_MN) or 64 k x 128 rows; tmX: x, boxes
// of 64 k x s.rows rows.
template <bool W_MN, int EPI>
__global__ void __launch_bounds__(THREADS, 2)
    k_dense_few(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const Params p,
                const Split s) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const uint32_t rank = s.splits > 1 ? cluster_ctarank() : 0;
    const int tile = blockIdx.x / s.splits, mt = tile / p.n_tiles, nt = tile - mt * p.n_tiles;
    const int64_t m0 = (int64_t)mt * s.rows;
    const int m = (int)min((int64_t)s.rows, p.M - m0);
    const int k0 = p.nk / s.splits * (int)rank + min((int)rank, p.nk % s.splits);
    const int k1 = k0 + p.nk / s.splits + ((int)rank < p.nk % s.splits);
    const int stage_bytes = W_BYTES + s.rows * TK * 2;

    const uint32_t bar0 = smem_u32(smem + OFF_BAR);
    auto full_bar = [&](int i) { return bar0 + 8u * i; };
    auto empty_bar = [&](int i) { return bar0 + 8u * (MAX_STAGES + i); };
    const uint32_t done_bar = bar0 + 8u * (2 * MAX_STAGES);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_MISC + 4);
    if (threadIdx.x == 0) {
        for (int i = 0; i < s.stages; ++i) {
            mbar_init(full_bar(i), 1);
            mbar_init(empty_bar(i), 1);
        }
        mbar_init(done_bar, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        *abort_flag = 0;
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(s.tmem_cols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    wait_for_previous_kernels();

    if (warp == 0 && lane == 0) {
        // ------------------------------------------------ TMA producer ----
        int stage = 0, issued = 0;
        uint32_t phase = 0;
        bool aborted = false;
        for (int k = k0; k < k1; ++k) {
            if (!mbar_wait(empty_bar(stage), phase ^ 1u, p, abort_flag)) {
                aborted = true;
                break;
            }
            const uint32_t fb = full_bar(stage);
            const uint32_t sw = smem_u32(smem + stage * stage_bytes), sx = sw + W_BYTES;
            mbar_expect_tx(fb, stage_bytes);
            if constexpr (W_MN) {
                const int c = EPI == EPI_GLU ? nt * 64 : nt * 128;
                tma_load_2d(sw, &tmW, c, k * TK, fb);
                tma_load_2d(sw + W_BYTES / 2, &tmW, EPI == EPI_GLU ? c + p.up : c + 64, k * TK, fb);
            } else {
                tma_load_2d(sw, &tmW, k * TK, nt * 128, fb);
            }
            tma_load_2d(sx, &tmX, k * TK, (int)m0, fb);
            ++issued;
            if (++stage == s.stages) {
                stage = 0;
                phase ^= 1u;
            }
        }
        if (aborted) {      // wait (bounded) for the copies in flight
            Params q = p;
            q.timeout_ns = 200000000ull;
            volatile int no_abort = 0;
            for (int i = issued - min(issued, s.stages); i < issued; ++i)
                mbar_wait(full_bar(i % s.stages), (uint32_t)(i / s.stages) & 1u, q, &no_abort);
        }
    } else if (warp == 1) {
        // ------------------------- MMA issuer (one lane of the warp) ----
        const bool elected = elect_one();
        // bf16 A and B, fp32 D, M = 128, N = s.rows, A along M (W_MN) or K
        const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (W_MN ? 1u << 15 : 0u) |
                               ((uint32_t)(s.rows >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
        int stage = 0;
        uint32_t phase = 0;
        const uint32_t sw0 = smem_u32(smem), stage_step = (uint32_t)stage_bytes >> 4;
        const uint64_t wdesc0 = operand_desc<W_MN>(sw0), xdesc0 = desc_sw128(sw0 + W_BYTES);
        for (int k = k0; k < k1; ++k) {
            if (!mbar_wait(full_bar(stage), phase, p, abort_flag)) break;
            tc_fence_after();
            if (elected) {
                const uint64_t wdesc = wdesc0 + stage * stage_step, xdesc = xdesc0 + stage * stage_step;
#pragma unroll
                for (int kk = 0; kk < TK / 16; ++kk)
                    tc_mma_bf16(tmem, wdesc + k16_step<W_MN>() * kk, xdesc + k16_step<false>() * kk, idesc,
                                (k != k0 || kk != 0) ? 1u : 0u);
                tc_commit(empty_bar(stage));
            }
            if (++stage == s.stages) {
                stage = 0;
                phase ^= 1u;
            }
        }
        if (elected) tc_commit(done_bar);
    }
    __syncwarp();
    // every product of this CTA is done (and every stage read), or the CTA gives up
    const bool ready = mbar_wait(done_bar, 0, p, abort_flag);
    __syncthreads();      // the aborting producer's copies have landed
    tc_fence_after();
    float* part = reinterpret_cast<float*>(smem);          // [rows of x][128]
    if (ready) {
        // a warp reads its lane quarter, the upper four warps every second 16 rows
        const int quarter = warp & 3;
        for (int c = 16 * (warp >> 2); c < m; c += 32) {
            float v[16];
            tmem_ld16(tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)c, v);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (c + i < m) part[(c + i) * 128 + quarter * 32 + lane] = v[i];
        }
    }
    tc_fence_before();
    if (s.splits > 1) cluster_sync();
    else __syncthreads();
    if (s.splits == 1) join<EPI, 8, 1>(p, s, smem_u32(part), rank, m0, m, nt);
    else if (s.splits == 2) join<EPI, 4, 2>(p, s, smem_u32(part), rank, m0, m, nt);
    else join<EPI, 2, 4>(p, s, smem_u32(part), rank, m0, m, nt);
    if (s.splits > 1) cluster_sync();      // nobody leaves while its partial tile is read
    else __syncthreads();
    if (warp == 1) {
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(s.tmem_cols));
    }
}

}  // namespace few

// ------------------------------------------------- elementwise backward ----

// da = [dh * up * act'(gate) | dh * act(gate)] from a = [gate | up].  Bound by
// its 10 bytes per element of h (8,192 x 14,336: 178 us, 6.6 TB/s); each product is rounded to bf16 once, as the
// operand of the two GEMMs that follow.
// (da may be a itself: neither is __restrict__, which would let a be read
// through the cache for memory that no one writes.)
__global__ void __launch_bounds__(256) k_glu_bwd(const __nv_bfloat16* __restrict__ dh, int64_t lddh,
                                                 const __nv_bfloat16* a, int64_t lda, int64_t M, int f, int act,
                                                 __nv_bfloat16* da, int64_t ldda) {
    wait_for_previous_kernels();
    const int nvec = f / 8;
    const int64_t n = M * nvec, stride = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += stride) {
        const int64_t row = i / nvec;
        const int c = (int)(i - row * nvec) * 8;
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

// dz = dy * act'(z) (bf16, when ACT is not MOE_ACT_NONE) and the column sums of
// the unrounded dz over this CTA's rows: one row of partial sums per
// blockIdx.y, or, in up to kJoin parts, a cluster's CTAs add theirs up through
// distributed shared memory, in the order of the parts, and part is dbias
// itself.  A thread owns 8 columns; the CTA's 8 warps take every eighth
// row, kActRowsInFlight of them loaded before the first is worked on (with
// one at a time the loads covered 60 % of the memory's latency), and are added in
// order at the end.  Bound by its 6 bytes an element (8,192 x 7,168: 60 us, 5.9 TB/s).
constexpr int kActRowsInFlight = 4;
constexpr int kJoin = 8;

__device__ __forceinline__ float ld_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

template <int ACT>
__global__ void __launch_bounds__(256) k_act_bwd(const __nv_bfloat16* __restrict__ dy, int64_t lddy,
                                                 const __nv_bfloat16* __restrict__ z, int64_t ldz, int64_t M, int N,
                                                 __nv_bfloat16* __restrict__ dz, int64_t lddz,
                                                 float* __restrict__ part) {
    __shared__ float s_sum[8][257], s_part[256];
    wait_for_previous_kernels();
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const int c = blockIdx.x * 256 + lane * 8;
    const int n = N - c < 0 ? 0 : (N - c > 8 ? 8 : N - c);
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const int64_t step = (int64_t)gridDim.y * 8;
    if (n > 0) {
        for (int64_t row0 = (int64_t)blockIdx.y * 8 + grp; row0 < M; row0 += step * kActRowsInFlight) {
            uint4 a[kActRowsInFlight], b[kActRowsInFlight];
#pragma unroll
            for (int i = 0; i < kActRowsInFlight; ++i) {
                const int64_t row = row0 + i * step;
                if (row >= M) continue;
                a[i] = load_vec8(dy + row * lddy + c, n);
                if (ACT != MOE_ACT_NONE) b[i] = load_vec8(z + row * ldz + c, n);
            }
#pragma unroll
            for (int i = 0; i < kActRowsInFlight; ++i) {
                const int64_t row = row0 + i * step;
                if (row >= M) continue;
                float d[8];
                unpack8(a[i], d);
                if (ACT != MOE_ACT_NONE) {
                    float v[8];
                    unpack8(b[i], v);
#pragma unroll
                    for (int j = 0; j < 8; ++j) d[j] *= act_slope(v[j], ACT);
                    if (n == 8) {
                        *reinterpret_cast<uint4*>(dz + row * lddz + c) = pack8(d);
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (j < n) dz[row * lddz + c + j] = __float2bfloat16_rn(d[j]);
                    }
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[j] += d[j];
            }
        }
    }
    if (part == nullptr) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) s_sum[grp][lane * 8 + j] = sum[j];
    __syncthreads();
    float t = 0.f;
#pragma unroll
    for (int g = 0; g < 8; ++g) t += s_sum[g][threadIdx.x];
    const int col = blockIdx.x * 256 + threadIdx.x;
    if (gridDim.y == 1 || gridDim.y > kJoin) {
        if (col < N) part[(int64_t)blockIdx.y * N + col] = t;
        return;
    }
    s_part[threadIdx.x] = t;
    cluster_sync();
    const int own = 256 / gridDim.y, at = blockIdx.y * own + threadIdx.x;      // this CTA's columns
    if (threadIdx.x < own && blockIdx.x * 256 + at < N) {
        const uint32_t src = smem_u32(&s_part[at]);
        float v[kJoin], total = 0.f;
#pragma unroll
        for (int j = 0; j < kJoin; ++j)
            v[j] = j < gridDim.y ? ld_cluster(mapa(src, (uint32_t)j)) : 0.f;
#pragma unroll
        for (int j = 0; j < kJoin; ++j) total += v[j];
        part[blockIdx.x * 256 + at] = total;
    }
    cluster_sync();      // nobody leaves while its sums are read
}

// ----------------------------------------------------------------- host ----

struct MaxClusters {
    int n[kMaxSplits];      // clusters of 2, 4, 6, 8 CTAs that run at a time
};
static PerDevice<MaxClusters> g_max_clusters;
static int* max_clusters() { return g_max_clusters.here().n; }

// attr: room for two (the cluster, and the early start described at
// wait_for_previous_kernels)
static cudaLaunchConfig_t launch_cfg(int clusters, int splits, cudaStream_t stream, cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * splits * clusters, 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2 * splits;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cfg;
}

// the products that are built: plain forward, input gradient and weight
// gradient (bf16, fp32); forward with an epilogue, gated forward
#define MOE_DENSE_INSTANCES(X)                                                                                       \
    X(false, true, EPI_PLAIN, 0) X(false, false, EPI_PLAIN, 0) X(true, true, EPI_PLAIN, 0) X(true, true, EPI_F32, 0) \
    X(false, true, EPI_LINEAR, 0) X(false, true, EPI_LINEAR, 1) X(false, true, EPI_LINEAR, 2)                        \
    X(false, true, EPI_LINEAR, 3) X(false, true, EPI_GLU, 0) X(false, true, EPI_GLU, 1) X(false, true, EPI_GLU, 2)   \
    X(false, true, EPI_GLU, 3)

static cudaError_t set_attributes() {
#define X(A, B, E, ACT)                                                                                                \
    {                                                                                                               \
        const cudaError_t e = cudaFuncSetAttribute(k_dense_pair<A, B, E, ACT>,                                      \
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);        \
        if (e != cudaSuccess) return e;                                                                             \
    }
    MOE_DENSE_INSTANCES(X)
#undef X
    for (const void* k : {(const void*)k_dense_both<EPI_PLAIN>, (const void*)k_dense_both<EPI_F32>}) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
        if (e != cudaSuccess) return e;
    }
    const void* ks[] = {(const void*)few::k_dense_few<true, EPI_LINEAR>, (const void*)few::k_dense_few<true, EPI_GLU>,
                        (const void*)few::k_dense_few<false, EPI_LINEAR>};
    for (const void* k : ks) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, few::SMEM_BYTES);
        if (e != cudaSuccess) return e;
    }
    for (int i = 0; i < kMaxSplits; ++i) {
        cudaLaunchAttribute attr[2];
        cudaLaunchConfig_t cfg = launch_cfg(1024, i + 1, nullptr, attr);
        const cudaError_t e =
            cudaOccupancyMaxActiveClusters(&max_clusters()[i], k_dense_pair<false, true, EPI_PLAIN, 0>, &cfg);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// One matrix operand as it lies in memory: [rows, cols], rows of ld elements.
struct Mat {
    const void* p;
    int64_t rows, cols, ld;
};

// The pair's tile width and the parts of K, by what a launch costs in k-steps
// of the widest tile (0.27 us): waves of tiles, each nk / splits k-steps of
// step_cost(bn), no shorter than the epilogue that runs under it, the last tile's
// epilogue, and the swap when K is split.  Steps, measured alone / on a full
// machine under its power cap, relative to 256 columns: 224 0.87 / 0.94, 192
// 0.75 / 0.84, 128 0.54 / 0.57, bound by the products; 64 0.56 alone, bound by the
// loads in flight, and 1.2 on a full machine.
// Narrower tiles win where the wide ones are fewer than the SM pairs or leave the
// last wave half empty (256 x 4,096 x 4,096: 13.8 us with 128 columns, 22.0 with 256, 17.9
// with 256 in two parts; 256 x 1,024 x 1,024: 5.4 with 64 columns, 5.8 with 128), parts of
// K where even those are few (256 x 14,336 x 2,048: 23.4 us with 128 columns in two
// parts, 38.3 with 256; 512 x 2,000 x 608: 8.7 with 64 columns, 7.7 in two parts).
struct Choice {
    int bn, splits;
    double cost;
};
static double step_cost(int bn) { return bn == 256 ? 1.0 : (bn == 224 ? 0.91 : (bn == 192 ? 0.80 : 0.56)); }
// 1.5 to 2 us for 64 columns in two parts, 2.7 for 128, 4.3 for 256; 6 for 256 in three, 3.5 for 64 in four
static double swap_cost(int bn, int splits) { return (4. + 12. * bn / 256.) * (1. + 0.4 * (splits - 2)); }
constexpr double kEpilogue = 5. / 256.;      // a column
static double tile_cost(int nk, int bn) { return std::max(nk * step_cost(bn), kEpilogue * bn) + 1.; }
// clusters: those of 2, 4, 6, 8 CTAs that run at a time
static Choice choose(int64_t m_tiles, int N, int nk, bool glu, const int* clusters) {
    Choice best{256, 1, 1e300};
    for (int bn : kWidths) {
        // gate and up in whole chunks of 32, one at least for each half of the epilogue's warps
        if (glu && (bn == 224 || bn == 64)) continue;
        const int cols = glu ? bn / 2 : bn;
        const int64_t tiles = m_tiles * ((N + cols - 1) / cols);
        if (bn == 64 && tiles > clusters[1]) continue;
        for (int splits = 1; splits <= kMaxSplits; ++splits) {
            const int slots = clusters[splits - 1];
            if (splits > 1 && (tiles > slots || nk < 4 * splits)) continue;
            const int64_t waves = (tiles + slots - 1) / slots;
            const double cost = (double)waves * tile_cost((nk + splits - 1) / splits, bn) + kEpilogue * bn +
                                (splits > 1 ? swap_cost(bn, splits) : 0.);
            if (cost < best.cost) best = {bn, splits, cost};
        }
    }
    return best;
}
// Both products of a backward pass in one launch (k_dense_both): the
// longest share of its tiles, nk steps each (p) or nk2 (q).  Two launches
// instead where they split K and come out shorter by more than the second
// set-up (8 steps: with 3 instead, 2,048 x 1,024 x 4,096 27.6 us instead of 24.0), and
// where the work is long and a set-up does not count (8,192 x 4,096 x 7,168 with
// SiLU: 566 us, in one launch 577; 4,096 x 1,024 x 14,336 still 148, in one 131).
constexpr double kBothSaves = 8., kBothMax = 1000.;
static Choice choose_both(int64_t m_tiles, int N, int nk, int64_t m_tiles2, int N2, int nk2, const int* clusters) {
    const int64_t slots = clusters[0];
    Choice best{256, 1, 1e300};
    for (int bn : kWidths) {
        const int64_t mid = m_tiles * ((N + bn - 1) / bn), total = mid + m_tiles2 * ((N2 + bn - 1) / bn);
        if (bn == 64 && total > clusters[1]) continue;
        double cost = 0.;
        for (int64_t i : {(int64_t)0, mid % slots, total % slots}) {      // the shares change there
            const int64_t n = (std::max<int64_t>(mid - i, 0) + slots - 1) / slots;
            const int64_t all = (std::max<int64_t>(total - i, 0) + slots - 1) / slots;
            cost = std::max(cost, n * tile_cost(nk, bn) + (all - n) * tile_cost(nk2, bn));
        }
        cost += kEpilogue * bn;
        if (cost < best.cost) best = {bn, 1, cost};
    }
    const double two = choose(m_tiles, N, nk, false, clusters).cost + choose(m_tiles2, N2, nk2, false, clusters).cost;
    if (best.cost > kBothMax || best.cost > two + kBothSaves) best.bn = 0;      // two launches
    return best;
}

// The fields of p that the tile width decides; the maps of a product's operands and of y.
static void set_width(Params& p, int bn, int stage_bytes, bool glu) {
    p.bn = bn;
    p.stage_bytes = stage_bytes;
    p.stages = std::min(MAX_STAGES, SMEM_TILES / stage_bytes);
    const int cols = glu ? bn / 2 : bn;      // of D per tile
    p.n_tiles = (p.N + cols - 1) / cols;
    p.band = 8;
    p.timeout_ns = 2000000000ull;
}
static int stage_size(bool b_mn, int bn) { return HALF_BYTES + (b_mn ? (bn / 2 + 63) / 64 * 64 : bn / 2) * TK * 2; }
static int boxed(int N) { return std::max(N & ~7, 8); }      // finish(): N < 8 sends no box
template <bool A_MN, bool B_MN, int EPI>
static bool make_maps(CUtensorMap* tmA, CUtensorMap* tmB, CUtensorMap* tmY, const Mat& a, const Mat& b,
                      const Params& p) {
    return make_bf16_map(tmA, a.p, a.rows, a.cols, a.ld, A_MN ? TK : 128) &&
           make_bf16_map(tmB, b.p, b.rows, b.cols, b.ld, B_MN ? TK : p.bn / 2) &&
           make_store_map(tmY, p.y, p.M, boxed(p.N), p.ldy, EPI == EPI_F32);
}

template <bool A_MN, bool B_MN, int EPI, int ACT>
static moe_status_t product(const Mat& a, const Mat& b, Params p, cudaStream_t s) {
    const int* most = max_clusters();
    MOE_REQUIRE(most[0] > 0, MOE_ERR_NOT_INITIALIZED);
    p.m_tiles = (int)((p.M + TM - 1) / TM);
    p.nk = (int)((p.K + TK - 1) / TK);
    const Choice c = choose(p.m_tiles, p.N, p.nk, EPI == EPI_GLU, most);
    p.splits = c.splits;
    set_width(p, c.bn, stage_size(B_MN, c.bn), EPI == EPI_GLU);
    CUtensorMap tmA, tmB, tmY, tmZ, tmZ2;
    MOE_REQUIRE((make_maps<A_MN, B_MN, EPI>(&tmA, &tmB, &tmY, a, b, p)), MOE_ERR_CUDA);
    tmZ = tmZ2 = tmY;
    if (p.z != nullptr)
        MOE_REQUIRE(make_store_map(&tmZ, p.z, p.M, boxed(p.N), p.ldz, false) &&
                        (EPI != EPI_GLU || make_store_map(&tmZ2, p.z + p.N, p.M, p.N, p.ldz, false)),
                    MOE_ERR_CUDA);
    const int64_t tiles = (int64_t)p.m_tiles * p.n_tiles;
    MOE_REQUIRE(tiles <= 0x3FFFFFFF, MOE_ERR_UNSUPPORTED);
    const int clusters = (int)(p.splits > 1 ? tiles : std::min<int64_t>(tiles, most[0]));
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = launch_cfg(clusters, p.splits, s, attr);
    if (cudaLaunchKernelEx(&cfg, k_dense_pair<A_MN, B_MN, EPI, ACT>, tmA, tmB, tmY, tmZ, tmZ2, p) != cudaSuccess)
        return MOE_ERR_CUDA;
    MOE_CHECK_LAUNCH();
    return MOE_OK;
}

// dx = dz W^T (p) and dW = x^T dz (q) in one launch
template <int EPI_W>
static moe_status_t product_both(const Mat& x, const Mat& w, const Mat& dz, Params p, Params q, int bn,
                                 cudaStream_t s) {
    const int bytes = std::max(stage_size(false, bn), stage_size(true, bn));
    set_width(p, bn, bytes, false);
    set_width(q, bn, bytes, false);
    p.splits = q.splits = 1;
    CUtensorMap tmA, tmB, tmY, tmA2, tmB2, tmY2;
    MOE_REQUIRE((make_maps<false, false, EPI_PLAIN>(&tmA, &tmB, &tmY, dz, w, p)) &&
                    (make_maps<true, true, EPI_W>(&tmA2, &tmB2, &tmY2, x, dz, q)),
                MOE_ERR_CUDA);
    const int64_t tiles = (int64_t)p.m_tiles * p.n_tiles + (int64_t)q.m_tiles * q.n_tiles;
    MOE_REQUIRE(tiles <= 0x3FFFFFFF, MOE_ERR_UNSUPPORTED);
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = launch_cfg((int)std::min<int64_t>(tiles, max_clusters()[0]), 1, s, attr);
    if (cudaLaunchKernelEx(&cfg, k_dense_both<EPI_W>, tmA, tmB, tmY, tmA2, tmB2, tmY2, p, q) != cudaSuccess)
        return MOE_ERR_CUDA;
    MOE_CHECK_LAUNCH();
    return MOE_OK;
}

// Twice the parts save nk / (2 splits) k-steps and lengthen the swap by rows x splits
// (128 x 2,048 x 2,048: 7.6 us in four parts, 9.9 in eight; 128 x 7,168 x 512: 11.8, 9.8),
// the more the fuller the machine is (128 x 4,096 x 4,096: 13.3 in four, 15.2 in eight).
static int few_splits(int64_t tiles, int rows, int nk, int sms) {
    int splits = 1;
    while (splits < 8 && tiles * splits * 2 <= 2 * sms && nk >= 8 * splits &&
           (tiles * splits * 2 <= sms ? 40 : 16) * nk > rows * splits * splits)
        splits *= 2;
    return splits;
}

// Few rows: see k_dense_few.  The product D[M, N] = x op(W), W's columns
// (W_MN) or rows in tiles of 128 (GLU: 64 gate and 64 up columns).
template <bool W_MN, int EPI>
static moe_status_t product_few(const Mat& x, const Mat& w, Params p, cudaStream_t st) {
    few::Split s{};
    const int rows = (int)std::min<int64_t>(p.M, few::ROWS);
    s.rows = (rows + 15) / 16 * 16;
    s.stages = std::min(few::MAX_STAGES, few::SMEM_TILES / (few::W_BYTES + s.rows * TK * 2));
    s.tmem_cols = s.rows <= 32 ? 32 : (s.rows <= 64 ? 64 : 128);
    p.n_tiles = EPI == EPI_GLU ? (p.N + 63) / 64 : (p.N + 127) / 128;
    p.m_tiles = (int)((p.M + s.rows - 1) / s.rows);
    p.nk = (int)((p.K + TK - 1) / TK);
    p.timeout_ns = 2000000000ull;
    const int64_t tiles = (int64_t)p.m_tiles * p.n_tiles;
    const int sms = device_sm_count();
    s.splits = few_splits(tiles, s.rows, p.nk, sms);
    MOE_REQUIRE(tiles * s.splits <= 0x7FFFFFFFLL, MOE_ERR_UNSUPPORTED);
    CUtensorMap tmW, tmX;
    MOE_REQUIRE(make_bf16_map(&tmW, w.p, w.rows, w.cols, w.ld, W_MN ? TK : 128) &&
                    make_bf16_map(&tmX, x.p, x.rows, x.cols, x.ld, s.rows),
                MOE_ERR_CUDA);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * s.splits), 1, 1);
    cfg.blockDim = dim3(few::THREADS, 1, 1);
    cfg.dynamicSmemBytes = few::SMEM_BYTES;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = s.splits;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, few::k_dense_few<W_MN, EPI>, tmW, tmX, p, s) != cudaSuccess) return MOE_ERR_CUDA;
    MOE_CHECK_LAUNCH();
    return MOE_OK;
}

// Few rows go to k_dense_few, whose tile costs what the rows cost and which
// splits K over more CTAs than the pair kernel.  Measured in graphs of 16
// (us, k_dense_few / pairs): up to 64 rows nearly always (64 x 4,096 x 4,096 10.3 / 13.4);
// up to 128 where K has steps to split (128 x 2,048 x 2,048 7.6 / 8.0, 128 x 4,096 x 1,024
// 8.6 / 9.8, but 128 x 1,024 x 1,024 6.7 / 5.4); none above (256 x 4,096 x 1,024 10.8 / 9.9).
static bool few_rows(int64_t M, int64_t K) { return M <= 64 || (M <= few::ROWS && K > 16 * TK); }

static bool act_ok(int a) { return a >= MOE_ACT_NONE && a <= MOE_ACT_SILU; }
// sizes the tensor maps and the tile counts hold
static bool size_ok(int64_t v) { return v >= 1 && v <= 0x7FFFFF00LL; }
static bool row_ok(const void* p, int64_t ld) { return moe_aligned16(p) && ld % 8 == 0; }
// The stride of a matrix of one row means nothing; the tensor maps want some
// multiple of 16 bytes.
static int64_t stride_of(int64_t rows, int64_t cols, int64_t ld) { return rows == 1 && ld >= cols ? (cols + 7) / 8 * 8 : ld; }

// Parts of k_act_bwd's rows: for up to 256 rows of dy 1, 2, 4 or 8 CTAs of a
// cluster, which write dbias itself (128 x 1,024 dy, bias gradient only: 2.3 us, 3.2
// in one CTA per 256 columns; with SiLU in a whole backward 8.8 against 12.3); else one
// for every 32 rows, 256 at most, whose sums a second launch adds up (504 x 2,004:
// 4.3 us, 4.7 in a cluster, with SiLU in a whole backward 19.8 against 21.9).
static int act_parts(int64_t M) {
    if (M > 256) return (int)std::min<int64_t>((M + 31) / 32, 256);
    int parts = 1;
    while (parts < kJoin && M > 16 * parts) parts *= 2;
    return parts;
}

}  // namespace dense

cudaError_t dense_set_attributes() { return dense::set_attributes(); }
void launch_column_sum(const float* part, int P, int N, float* out, cudaStream_t s);      // norm.cu

}  // namespace moe

using namespace moe;
using namespace moe::dense;

extern "C" moe_status_t linear_fwd(const void* x, int64_t ldx, const void* w, int64_t ldw, const void* bias, int act,
                                   const void* res, int64_t ldres, int64_t M, int N, int64_t K, void* y, int64_t ldy,
                                   void* z, int64_t ldz, int32_t* err, void* stream) {
    MOE_REQUIRE(M >= 0 && N >= 1 && K >= 1 && act_ok(act), MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(ldx >= K && ldw >= N && ldy >= N && (!res || ldres >= N) && (!z || ldz >= N), MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(M <= 0x7FFFFF00LL && size_ok(N) && size_ok(K), MOE_ERR_UNSUPPORTED);
    if (M == 0) return MOE_OK;
    ldx = stride_of(M, K, ldx), ldw = stride_of(K, N, ldw), ldy = stride_of(M, N, ldy);
    ldres = stride_of(M, N, ldres), ldz = stride_of(M, N, ldz);
    MOE_REQUIRE(x && w && y, MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(row_ok(x, ldx) && row_ok(w, ldw) && row_ok(y, ldy) && (!res || row_ok(res, ldres)) &&
                    (!z || row_ok(z, ldz)) && reinterpret_cast<uintptr_t>(bias) % 2 == 0,
                MOE_ERR_ALIGNMENT);
    MOE_REQUIRE(device_initialized(), MOE_ERR_NOT_INITIALIZED);
    dense::Params p{};
    p.M = M, p.N = N, p.K = K, p.act = act;
    p.y = y, p.ldy = ldy, p.z = static_cast<__nv_bfloat16*>(z), p.ldz = ldz;
    p.bias = static_cast<const __nv_bfloat16*>(bias);
    p.res = static_cast<const __nv_bfloat16*>(res), p.ldres = ldres;
    p.err = err;
    const Mat mx{x, M, K, ldx}, mw{w, K, N, ldw};
    cudaStream_t s = (cudaStream_t)stream;
    if (few_rows(M, K)) return product_few<true, EPI_LINEAR>(mx, mw, p, s);
    if (!bias && !res && !z && act == MOE_ACT_NONE) return product<false, true, EPI_PLAIN, 0>(mx, mw, p, s);
    switch (act) {
        case MOE_ACT_RELU: return product<false, true, EPI_LINEAR, MOE_ACT_RELU>(mx, mw, p, s);
        case MOE_ACT_GELU: return product<false, true, EPI_LINEAR, MOE_ACT_GELU>(mx, mw, p, s);
        case MOE_ACT_SILU: return product<false, true, EPI_LINEAR, MOE_ACT_SILU>(mx, mw, p, s);
        default: return product<false, true, EPI_LINEAR, MOE_ACT_NONE>(mx, mw, p, s);
    }
}

// dx[M, K] = dz W^T and dw[K, N] = x^T dz, each if asked for
static moe_status_t gradients(const void* dz, int64_t lddz, const void* x, int64_t ldx, const void* w, int64_t ldw,
                              int64_t M, int N, int64_t K, void* dx, int64_t lddx, void* dw, int dw_type,
                              int64_t lddw, int32_t* err, cudaStream_t s) {
    const bool f32 = dw_type == MOE_TYPE_F32;
    if (M == 0)
        return dw && cudaMemset2DAsync(dw, lddw * (f32 ? 4 : 2), 0, (size_t)N * (f32 ? 4 : 2), K, s) != cudaSuccess
                   ? MOE_ERR_CUDA : MOE_OK;
    const Mat mz{dz, M, N, lddz}, mx{x, M, K, ldx}, mw{w, K, N, ldw};
    dense::Params p{}, q{};
    p.M = M, p.N = (int)K, p.K = N, p.act = MOE_ACT_NONE, p.y = dx, p.ldy = lddx, p.err = err;
    q.M = K, q.N = N, q.K = M, q.act = MOE_ACT_NONE, q.y = dw, q.ldy = lddw, q.err = err;
    const bool few = few_rows(M, N);
    if (dx && dw && !few) {
        const int* most = max_clusters();
        MOE_REQUIRE(most[0] > 0, MOE_ERR_NOT_INITIALIZED);
        p.m_tiles = (int)((M + TM - 1) / TM), p.nk = (N + TK - 1) / TK;
        q.m_tiles = (int)((K + TM - 1) / TM), q.nk = (int)((M + TK - 1) / TK);
        const Choice c = choose_both(p.m_tiles, p.N, p.nk, q.m_tiles, q.N, q.nk, most);
        if (c.bn > 0)
            return f32 ? product_both<EPI_F32>(mx, mw, mz, p, q, c.bn, s)
                       : product_both<EPI_PLAIN>(mx, mw, mz, p, q, c.bn, s);
    }
    if (dx) {
        const moe_status_t st = few ? product_few<false, EPI_LINEAR>(mz, mw, p, s)
                                    : product<false, false, EPI_PLAIN, 0>(mz, mw, p, s);
        if (st != MOE_OK) return st;
    }
    if (!dw) return MOE_OK;
    return f32 ? product<true, true, EPI_F32, 0>(mx, mz, q, s) : product<true, true, EPI_PLAIN, 0>(mx, mz, q, s);
}

static size_t dz_bytes(int64_t M, int N) { return ((size_t)M * ((N + 7) / 8 * 8) * 2 + 255) / 256 * 256; }

extern "C" size_t linear_bwd_workspace_size(int64_t M, int N) {
    if (M < 0 || M > 0x7FFFFF00LL || !size_ok(N)) return (size_t)-1;
    const int rows = act_parts(M) > kJoin ? act_parts(M) : 1;      // of partial sums
    return dz_bytes(M, N) + (size_t)rows * N * sizeof(float);
}

extern "C" moe_status_t linear_bwd(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* w, int64_t ldw,
                                   const void* z, int64_t ldz, int act, int64_t M, int N, int64_t K, void* dx,
                                   int64_t lddx, void* dw, int dw_type, int64_t lddw, float* dbias, void* ws,
                                   size_t ws_bytes, int32_t* err, void* stream) {
    MOE_REQUIRE(M >= 0 && N >= 1 && K >= 1 && act_ok(act), MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(dw_type == MOE_TYPE_BF16 || dw_type == MOE_TYPE_F32, MOE_ERR_INVALID_ARG);
    const bool with_z = act != MOE_ACT_NONE;
    MOE_REQUIRE(lddy >= N && (!with_z || ldz >= N) && (!dx || (ldw >= N && lddx >= K)) &&
                    (!dw || (ldx >= K && lddw >= N)),
                MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(M <= 0x7FFFFF00LL && size_ok(N) && size_ok(K), MOE_ERR_UNSUPPORTED);
    MOE_REQUIRE(dx || dw || dbias, MOE_ERR_INVALID_ARG);
    lddy = stride_of(M, N, lddy), ldz = stride_of(M, N, ldz), ldx = stride_of(M, K, ldx);
    lddx = stride_of(M, K, lddx), ldw = stride_of(K, N, ldw), lddw = stride_of(K, N, lddw);
    MOE_REQUIRE(M == 0 || (dy && (!with_z || z) && (!dx || w) && (!dw || x)), MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(row_ok(dy, lddy) && (!with_z || row_ok(z, ldz)) && (!dx || (row_ok(w, ldw) && row_ok(dx, lddx))) &&
                    (!dw || (row_ok(x, ldx) && row_ok(dw, lddw))) && reinterpret_cast<uintptr_t>(dbias) % 4 == 0 &&
                    moe_aligned16(ws),
                MOE_ERR_ALIGNMENT);
    const bool need_ws = M > 0 && (dbias || (with_z && (dx || dw)));
    MOE_REQUIRE(!need_ws || (ws && ws_bytes >= linear_bwd_workspace_size(M, N)), MOE_ERR_WORKSPACE);
    MOE_REQUIRE(device_initialized(), MOE_ERR_NOT_INITIALIZED);
    cudaStream_t s = (cudaStream_t)stream;
    const void* g = dy;
    int64_t ldg = lddy;
    const int parts = act_parts(M);
    const bool joined = M > 0 && parts <= kJoin;
    float* part = nullptr;
    if (need_ws && dbias) part = joined ? dbias : reinterpret_cast<float*>(static_cast<char*>(ws) + dz_bytes(M, N));
    if (need_ws) {
        __nv_bfloat16* dz = static_cast<__nv_bfloat16*>(ws);
        const int64_t lddz = (N + 7) / 8 * 8;
        void (*const kernels[])(const __nv_bfloat16*, int64_t, const __nv_bfloat16*, int64_t, int64_t, int,
                                __nv_bfloat16*, int64_t, float*) = {
            k_act_bwd<MOE_ACT_NONE>, k_act_bwd<MOE_ACT_RELU>, k_act_bwd<MOE_ACT_GELU>, k_act_bwd<MOE_ACT_SILU>};
        if (launch_early_clusters(joined ? parts : 1, dim3((N + 255) / 256, parts), 256, 0, s, kernels[act],
                                  static_cast<const __nv_bfloat16*>(dy), lddy, static_cast<const __nv_bfloat16*>(z),
                                  ldz, M, N, dz, lddz, part) != cudaSuccess)
            return MOE_ERR_CUDA;
        if (with_z) g = dz, ldg = lddz;
    }
    if (dbias && !joined) {
        launch_column_sum(part, M > 0 ? parts : 0, N, dbias, s);
        MOE_CHECK_LAUNCH();
    }
    return gradients(g, ldg, x, ldx, w, ldw, M, N, K, dx, lddx, dw, dw_type, lddw, err, s);
}

extern "C" moe_status_t gated_ffn_fwd(const void* x, int64_t ldx, const void* w1, int64_t ldw, int act, int64_t M,
                                      int f, int64_t d, void* h, int64_t ldh, void* a, int64_t lda, int32_t* err,
                                      void* stream) {
    MOE_REQUIRE(M >= 0 && f >= 1 && d >= 1 && act_ok(act), MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(ldx >= d && ldw >= 2 * (int64_t)f && ldh >= f && (!a || lda >= 2 * (int64_t)f), MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(f % 8 == 0 && M <= 0x7FFFFF00LL && f <= 0x3FFFFF00 && size_ok(d), MOE_ERR_UNSUPPORTED);
    if (M == 0) return MOE_OK;
    ldx = stride_of(M, d, ldx), ldw = stride_of(d, 2 * (int64_t)f, ldw), ldh = stride_of(M, f, ldh);
    lda = stride_of(M, 2 * (int64_t)f, lda);
    MOE_REQUIRE(x && w1 && h, MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(row_ok(x, ldx) && row_ok(w1, ldw) && row_ok(h, ldh) && (!a || row_ok(a, lda)), MOE_ERR_ALIGNMENT);
    MOE_REQUIRE(device_initialized(), MOE_ERR_NOT_INITIALIZED);
    dense::Params p{};
    p.M = M, p.N = f, p.K = d, p.act = act, p.up = f;
    p.y = h, p.ldy = ldh, p.z = static_cast<__nv_bfloat16*>(a), p.ldz = lda;
    p.err = err;
    if (few_rows(M, d))
        return product_few<true, EPI_GLU>({x, M, d, ldx}, {w1, d, 2 * (int64_t)f, ldw}, p, (cudaStream_t)stream);
    const Mat mx{x, M, d, ldx}, mw{w1, d, 2 * (int64_t)f, ldw};
    cudaStream_t s = (cudaStream_t)stream;
    switch (act) {
        case MOE_ACT_RELU: return product<false, true, EPI_GLU, MOE_ACT_RELU>(mx, mw, p, s);
        case MOE_ACT_GELU: return product<false, true, EPI_GLU, MOE_ACT_GELU>(mx, mw, p, s);
        case MOE_ACT_SILU: return product<false, true, EPI_GLU, MOE_ACT_SILU>(mx, mw, p, s);
        default: return product<false, true, EPI_GLU, MOE_ACT_NONE>(mx, mw, p, s);
    }
}

extern "C" moe_status_t gated_ffn_bwd(const void* dh, int64_t lddh, const void* a, int64_t lda, const void* x,
                                      int64_t ldx, const void* w1, int64_t ldw, int act, int64_t M, int f, int64_t d,
                                      void* da, int64_t ldda, void* dx, int64_t lddx, void* dw1, int dw_type,
                                      int64_t lddw, int32_t* err, void* stream) {
    MOE_REQUIRE(M >= 0 && f >= 1 && d >= 1 && act_ok(act), MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(dw_type == MOE_TYPE_BF16 || dw_type == MOE_TYPE_F32, MOE_ERR_INVALID_ARG);
    const int64_t f2 = 2 * (int64_t)f;
    MOE_REQUIRE(lddh >= f && lda >= f2 && ldda >= f2 && (!dx || (ldw >= f2 && lddx >= d)) &&
                    (!dw1 || (ldx >= d && lddw >= f2)),
                MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(f % 8 == 0 && M <= 0x7FFFFF00LL && f <= 0x3FFFFF00 && size_ok(d), MOE_ERR_UNSUPPORTED);
    lddh = stride_of(M, f, lddh), lda = stride_of(M, f2, lda), ldda = stride_of(M, f2, ldda);
    ldx = stride_of(M, d, ldx), lddx = stride_of(M, d, lddx), ldw = stride_of(d, f2, ldw);
    lddw = stride_of(d, f2, lddw);
    MOE_REQUIRE(M == 0 || (dh && a && da && (!dx || w1) && (!dw1 || x)), MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(M == 0 || da != a || ldda == lda, MOE_ERR_INVALID_ARG);      // in place: row by row
    MOE_REQUIRE(row_ok(dh, lddh) && row_ok(a, lda) && row_ok(da, ldda) &&
                    (!dx || (row_ok(w1, ldw) && row_ok(dx, lddx))) &&
                    (!dw1 || (row_ok(x, ldx) && row_ok(dw1, lddw))),
                MOE_ERR_ALIGNMENT);
    MOE_REQUIRE(device_initialized(), MOE_ERR_NOT_INITIALIZED);
    const int sms = device_sm_count();
    MOE_REQUIRE(sms > 0, MOE_ERR_NOT_INITIALIZED);
    cudaStream_t s = (cudaStream_t)stream;
    if (M > 0) {
        const int64_t n = M * (f / 8);
        if (launch_early(dim3((unsigned)std::min<int64_t>((n + 255) / 256, (int64_t)sms * 8)), 256, 0, s, k_glu_bwd,
                         static_cast<const __nv_bfloat16*>(dh), lddh, static_cast<const __nv_bfloat16*>(a), lda, M, f,
                         act, static_cast<__nv_bfloat16*>(da), ldda) != cudaSuccess)
            return MOE_ERR_CUDA;
    }
    return gradients(da, ldda, x, ldx, w1, ldw, M, 2 * f, d, dx, lddx, dw1, dw_type, lddw, err, s);
}

extern "C" moe_status_t moe_selftest_dense_plan(int product, int64_t M, int64_t N, int64_t K, const int* clusters,
                                                moe_dense_plan_t* plan) {
    MOE_REQUIRE(plan && product >= MOE_DENSE_FWD && product <= MOE_DENSE_BACKWARD, MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(M >= 1 && N >= 1 && K >= 1, MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(M <= 0x7FFFFF00LL && size_ok(N) && size_ok(K), MOE_ERR_UNSUPPORTED);
    *plan = {};
    const int* slots = clusters ? clusters : max_clusters();
    const int sms = clusters ? 2 * clusters[0] : device_sm_count();
    const bool glu = product == MOE_DENSE_GATED;
    const int nk = (int)((K + TK - 1) / TK);
    if (product == MOE_DENSE_BACKWARD ? few_rows(M, N) : product != MOE_DENSE_WGRAD && few_rows(M, K)) {
        plan->few_rows = 1;
        if (product == MOE_DENSE_BACKWARD) return MOE_OK;
        MOE_REQUIRE(sms > 0, clusters ? MOE_ERR_INVALID_ARG : MOE_ERR_NOT_INITIALIZED);
        plan->few_parts = few_splits(glu ? (N + 63) / 64 : (N + 127) / 128, (int)(M + 15) / 16 * 16, nk, sms);
        return MOE_OK;
    }
    MOE_REQUIRE(slots[0] > 0, clusters ? MOE_ERR_INVALID_ARG : MOE_ERR_NOT_INITIALIZED);
    if (product == MOE_DENSE_BACKWARD) {
        plan->tile_cols = choose_both((M + TM - 1) / TM, (int)K, (int)((N + TK - 1) / TK), (K + TM - 1) / TM, (int)N,
                                      (int)((M + TK - 1) / TK), slots).bn;
        return MOE_OK;
    }
    const Choice c = choose((M + TM - 1) / TM, (int)N, nk, glu, slots);
    plan->tile_cols = c.bn;
    plan->parts = c.splits;
    if (c.splits > 1) {
        plan->swap_bytes = swap_bytes(glu, c.bn, c.splits);
        plan->box_bytes = swap_boxes(glu, c.bn, c.splits);
        plan->box_at = SMEM_TILES - EPI_WARPS * plan->box_bytes;
    }
    return MOE_OK;
}
