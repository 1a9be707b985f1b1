// Root-mean-square norm with the residual's addition, its MXFP8 output, and
// its backward pass.
//
//   r    = x + res                     (the residual stream)
//   rstd = 1 / sqrt(mean_j r_j^2 + eps)
//   y_j  = r_j rstd w_j
//
// One pass: a row's values stay in registers between the sum of squares and
// the output, so x and res are read once and r, y and the codes written once;
// the kernel is bound by that traffic.  Everything between the loads and the
// stores is fp32: the norm uses the unrounded sum r (not the copy of r that is
// stored in the residual's type), and the MXFP8 codes are taken from the
// unrounded y, so each output is rounded once.
#include <algorithm>

#include "gemm_common.cuh"

namespace moe {
namespace norm {

constexpr int kMaxN = 32768;
constexpr int kVec = 8;             // elements per thread and vector
constexpr int kMaxPartials = 608;   // rows of dw partial sums (4 per SM)

// ---- loads and stores of 8 consecutive elements as fp32 ----
// `n` of them exist (8 in the interior of a row); `vec` says that the
// address is a multiple of 16 bytes.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, int n, bool vec, float* f) {
    if (vec && n >= kVec) {
        unpack8(*reinterpret_cast<const uint4*>(p), f);
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) f[i] = i < n ? __bfloat162float(p[i]) : 0.f;
    }
}
__device__ __forceinline__ void load8(const float* p, int n, bool vec, float* f) {
    if (vec && n >= kVec) {
        const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) f[i] = i < n ? p[i] : 0.f;
    }
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, int n, bool vec, const float* f) {
    if (vec && n >= kVec) {
        *reinterpret_cast<uint4*>(p) = pack8(f);
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (i < n) p[i] = __float2bfloat16_rn(f[i]);
    }
}
__device__ __forceinline__ void store8(float* p, int n, bool vec, const float* f) {
    if (vec && n >= kVec) {
        reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (i < n) p[i] = f[i];
    }
}
// an operand whose type is known at run time only (uniform branch)
__device__ __forceinline__ void load8(const void* p, int type, int64_t at, int n, bool vec, float* f) {
    if (type == MOE_TYPE_F32)
        load8(static_cast<const float*>(p) + at, n, vec, f);
    else
        load8(static_cast<const __nv_bfloat16*>(p) + at, n, vec, f);
}
__device__ __forceinline__ void store8(void* p, int type, int64_t at, int n, bool vec, const float* f) {
    if (type == MOE_TYPE_F32)
        store8(static_cast<float*>(p) + at, n, vec, f);
    else
        store8(static_cast<__nv_bfloat16*>(p) + at, n, vec, f);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Sum over the threads that share a row: one warp, or (`block`) the CTA.
// The CTA form alternates between two halves of `s_part` (two rows in
// flight need one barrier between them), every warp adding the partial sums
// in the same order.
__device__ __forceinline__ float row_sum(float v, bool block, float* s_part, int half) {
    v = warp_sum(v);
    if (!block) return v;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    float* s = s_part + 32 * half;
    if (lane == 0) s[warp] = v;
    __syncthreads();
    return warp_sum(lane < nw ? s[lane] : 0.f);
}

// Smallest e (as the byte e + 127) with amax <= 448 * 2^e, for an fp32 amax:
// amax = M * 2^q with M in [1, 2) fits e = q - 8 when M <= 1.75, e = q - 7
// otherwise.  Zero and fp32-subnormal amax give byte 0, infinity 247 (a NaN is
// no part of a block's amax, and has a NaN code).
__device__ __forceinline__ uint32_t e8m0_byte_f32(float amax) {
    const uint32_t bits = __float_as_uint(amax);
    const int be = (int)((bits >> 23) & 0xFF);
    if (be == 0) return 0u;
    const int b = be - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return (uint32_t)(b < 0 ? 0 : b);
}

struct FwdParams {
    const void* x;
    const void* res;       // may be NULL
    const void* w;
    void* r;               // may be NULL
    void* y;               // may be NULL
    float* rstd;           // may be NULL
    uint8_t* codes;        // may be NULL
    uint8_t* scales;
    int64_t ldx, ldres, ldr, ldy;
    int64_t M, rows;       // rows >= M: padding rows of the codes (zeros)
    int N, w_type, y_type, sf_canonical;
    float eps;
    bool block_row, vec_x, vec_res, vec_w, vec_r, vec_y;
};

// Padding row of the codes: zero codes and scale bytes.
template <int VPT>
__device__ __forceinline__ void pad_row(const FwdParams& p, int64_t row, int t, int tpr) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int c = (t + v * tpr) * kVec;
        if (c >= p.N) continue;
        *reinterpret_cast<uint2*>(p.codes + row * p.N + c) = make_uint2(0, 0);
        if ((c & 31) == 0) p.scales[sf_atom_offset(row, c >> 5, p.rows)] = 0;
    }
}

// Everything that is written of 8 columns from c on (`in`: they exist, n of
// them): r, y, and codes with their scale.  All lanes of a warp call it.
template <typename RT>
__device__ __forceinline__ void fwd_outputs(const FwdParams& p, int64_t row, int c, bool in, int n, float rstd,
                                            const float* f, const float* w) {
    float y[kVec];
    if (in) {
        if (p.r != nullptr) store8(static_cast<RT*>(p.r) + row * p.ldr + c, n, p.vec_r, f);
#pragma unroll
        for (int i = 0; i < kVec; ++i) y[i] = f[i] * rstd * w[i];
        if (p.y != nullptr) store8(p.y, p.y_type, row * p.ldy + c, n, p.vec_y, y);
    }
    if (p.codes != nullptr) {       // N % 32 == 0: the four lanes of a block are in or out together
        float m = 0.f;
        if (in) {
#pragma unroll
            for (int i = 0; i < kVec; ++i) m = fmaxf(m, fabsf(y[i]));
        }
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        if (in) {
            const uint32_t b = e8m0_byte_f32(m);
            const float inv = e8m0_inv_scale(b);
            uint32_t q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) q[i] = cvt_e4m3x2(y[2 * i] * inv, y[2 * i + 1] * inv);
            *reinterpret_cast<uint2*>(p.codes + row * p.N + c) = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
            if ((c & 31) == 0)
                p.scales[p.sf_canonical ? row * (p.N >> 5) + (c >> 5) : sf_atom_offset(row, c >> 5, p.rows)] = (uint8_t)b;
        }
    }
}

// A row's thread t owns the vectors t, t + T, ... (T threads per row): the
// lanes of a warp read consecutive 16 bytes, and an MXFP8 block of 32 columns
// is four neighbouring lanes.
// MAXT: the most threads a CTA of the instance has; with fewer
// threads each may hold more registers.
template <typename XT, typename RT, int VPT, int MAXT>
__global__ void __launch_bounds__(MAXT) k_rms_fwd(const FwdParams p) {
    __shared__ float s_part[32];
    wait_for_previous_kernels();
    const int tpr = p.block_row ? (int)blockDim.x : 32;
    const int t = p.block_row ? (int)threadIdx.x : (int)(threadIdx.x & 31);
    const int64_t row = p.block_row ? (int64_t)blockIdx.x
                                    : (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (row >= p.rows) return;          // whole warps only (block_row: never)
    if (row >= p.M) {
        pad_row<VPT>(p, row, t, tpr);
        return;
    }
    const XT* x = static_cast<const XT*>(p.x) + row * p.ldx;
    const RT* res = static_cast<const RT*>(p.res) + row * p.ldres;
    float f[VPT][kVec];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int c = (t + v * tpr) * kVec;
        if (c < p.N) {
            load8(x + c, p.N - c, p.vec_x, f[v]);
        } else {
#pragma unroll
            for (int i = 0; i < kVec; ++i) f[v][i] = 0.f;
        }
    }
    if (p.res != nullptr) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int c = (t + v * tpr) * kVec;
            if (c < p.N) {
                float a[kVec];
                load8(res + c, p.N - c, p.vec_res, a);
#pragma unroll
                for (int i = 0; i < kVec; ++i) f[v][i] += a[i];
            }
        }
    }
    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int i = 0; i < kVec; ++i) ss = fmaf(f[v][i], f[v][i], ss);
    ss = row_sum(ss, p.block_row, s_part, 0);
    const float rstd = 1.f / sqrtf(ss / (float)p.N + p.eps);
    if (t == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int c = (t + v * tpr) * kVec;
        float w[kVec];
        if (c < p.N) load8(p.w, p.w_type, c, p.N - c, p.vec_w, w);
        fwd_outputs<RT>(p, row, c, c < p.N, p.N - c, rstd, f[v], w);
    }
}

// ---- long runs of aligned rows: a ring of rows in shared memory ----
//
// The kernels above load a row, wait for it, and compute while nothing of
// that CTA is on its way; their registers allow too few CTAs to cover that
// (62 % of the copy bandwidth at 24,576 x 7,168).  Here a CTA takes every G-th
// row, and bulk copies bring the next rows into a ring of stages while it
// works on one.  A thread reads its part of a stage into registers before the
// row's barrier, so the stage is refilled right after it.  24,576 x 7,168 with
// bf16 and MXFP8 outputs: 272 us, 5.85 TB/s, 86 % of the copy bandwidth (366 us
// without the ring); the backward pass of 8,191 x 4,096, fp32 residual
// stream: 75 us, 6.3 TB/s, 92 % (189 us).

constexpr int kMaxStages = 2;
constexpr int kRingBytes = 200 * 1024;      // of all CTAs of an SM

// Wait for a stage's bytes, bounded (about 2^16 polls of up to 50 us).
__device__ __forceinline__ bool ring_wait(uint32_t bar, uint32_t parity) {
    for (int i = 0; i < (1 << 16); ++i)
        if (gg::mbar_try_wait(bar, parity)) return true;
    return false;
}

template <typename XT, typename RT, int VPT>
__global__ void __launch_bounds__(512) k_rms_fwd_ring(const FwdParams p, int stages, int stage_bytes) {
    extern __shared__ __align__(128) uint8_t s_rows[];
    __shared__ __align__(8) uint64_t s_bar[kMaxStages];
    __shared__ float s_part[64];
    const int t = (int)threadIdx.x, T = (int)blockDim.x;
    const uint32_t xb = (uint32_t)p.N * sizeof(XT), rb = p.res != nullptr ? (uint32_t)p.N * sizeof(RT) : 0u;
    const int64_t G = gridDim.x;
    auto issue = [&](int st, int64_t row) {
        const uint32_t bar = gg::smem_u32(&s_bar[st]), dst = gg::smem_u32(s_rows + st * stage_bytes);
        gg::mbar_expect_tx(bar, xb + rb);
        gg::bulk_load(dst, static_cast<const XT*>(p.x) + row * p.ldx, xb, bar);
        if (rb != 0u) gg::bulk_load(dst + xb, static_cast<const RT*>(p.res) + row * p.ldres, rb, bar);
    };
    if (t == 0) {
        for (int i = 0; i < stages; ++i) gg::mbar_init(gg::smem_u32(&s_bar[i]), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    wait_for_previous_kernels();
    if (t == 0) {
        for (int i = 0; i < stages; ++i)
            if (blockIdx.x + i * G < p.M) issue(i, blockIdx.x + i * G);
    }
    float w[VPT][kVec];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int c = (t + v * T) * kVec;
        if (c < p.N) load8(p.w, p.w_type, c, kVec, p.vec_w, w[v]);
    }
    __syncthreads();
    int st = 0, half = 0;
    uint32_t phase = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += G) {
        if (row >= p.M) {
            pad_row<VPT>(p, row, t, T);
            continue;
        }
        const bool ok = ring_wait(gg::smem_u32(&s_bar[st]), phase);
        const XT* x = reinterpret_cast<const XT*>(s_rows + st * stage_bytes);
        const RT* res = reinterpret_cast<const RT*>(s_rows + st * stage_bytes + xb);
        float f[VPT][kVec];
        float ss = ok ? 0.f : __uint_as_float(0x7FC00000u);      // bytes that never came: the row is NaN
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int c = (t + v * T) * kVec;
            if (c < p.N) {
                load8(x + c, kVec, true, f[v]);
                if (rb != 0u) {
                    float a[kVec];
                    load8(res + c, kVec, true, a);
#pragma unroll
                    for (int i = 0; i < kVec; ++i) f[v][i] += a[i];
                }
#pragma unroll
                for (int i = 0; i < kVec; ++i) ss = fmaf(f[v][i], f[v][i], ss);
            }
        }
        ss = row_sum(ss, true, s_part, half);
        half ^= 1;
        if (t == 0 && row + stages * G < p.M) issue(st, row + stages * G);
        if (++st == stages) {
            st = 0;
            phase ^= 1u;
        }
        const float rstd = 1.f / sqrtf(ss / (float)p.N + p.eps);
        if (t == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int c = (t + v * T) * kVec;
            fwd_outputs<RT>(p, row, c, c < p.N, kVec, rstd, f[v], w[v]);
        }
    }
}

struct BwdParams {
    const void* dy;
    const void* r;
    const void* w;
    const float* rstd;
    const void* dres;      // may be NULL
    void* dx;
    float* part;           // [partials, N], or NULL when dw is not asked for
    int64_t lddy, ldr, lddres, lddx, M;
    int N, w_type;
    bool block_row, vec_dy, vec_r, vec_w, vec_dres, vec_dx;
};

// With xhat = r rstd and t = dy w:
//   dx = rstd (t - xhat mean_j(t xhat)) + dres,   dw = sum_rows dy xhat.
// A group of threads (a warp, or the CTA) takes every G-th row and keeps its
// dw sums in registers; they go out once, as one of G rows of partial sums,
// which k_dw_sum adds in a fixed order (no atomics, so dw is the same on
// every run).
template <typename YT, typename RT, int VPT, int MAXT>
__global__ void __launch_bounds__(MAXT) k_rms_bwd(const BwdParams p) {
    __shared__ float s_part[64];
    wait_for_previous_kernels();
    const int tpr = p.block_row ? (int)blockDim.x : 32;
    const int t = p.block_row ? (int)threadIdx.x : (int)(threadIdx.x & 31);
    const int64_t group = p.block_row ? (int64_t)blockIdx.x
                                      : (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int64_t groups = p.block_row ? (int64_t)gridDim.x : (int64_t)gridDim.x * (blockDim.x >> 5);
    float dw[VPT][kVec];
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int i = 0; i < kVec; ++i) dw[v][i] = 0.f;
    int half = 0;
    for (int64_t row = group; row < p.M; row += groups) {
        const float rstd = p.rstd[row];
        const YT* dyp = static_cast<const YT*>(p.dy) + row * p.lddy;
        const RT* rp = static_cast<const RT*>(p.r) + row * p.ldr;
        float tv[VPT][kVec], xh[VPT][kVec];
        float dot = 0.f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int c = (t + v * tpr) * kVec;
            if (c < p.N) {
                load8(dyp + c, p.N - c, p.vec_dy, tv[v]);
                load8(rp + c, p.N - c, p.vec_r, xh[v]);
            } else {
#pragma unroll
                for (int i = 0; i < kVec; ++i) tv[v][i] = xh[v][i] = 0.f;
            }
        }
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int c = (t + v * tpr) * kVec;
            float w[kVec];
#pragma unroll
            for (int i = 0; i < kVec; ++i) w[i] = 0.f;
            if (c < p.N) load8(p.w, p.w_type, c, p.N - c, p.vec_w, w);
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                xh[v][i] *= rstd;
                dw[v][i] = fmaf(tv[v][i], xh[v][i], dw[v][i]);
                tv[v][i] *= w[i];
                dot = fmaf(tv[v][i], xh[v][i], dot);
            }
        }
        const float mean = row_sum(dot, p.block_row, s_part, half) / (float)p.N;
        half ^= 1;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int c = (t + v * tpr) * kVec;
            if (c >= p.N) continue;
            float d[kVec], a[kVec];
#pragma unroll
            for (int i = 0; i < kVec; ++i) d[i] = rstd * (tv[v][i] - xh[v][i] * mean);
            if (p.dres != nullptr) {
                load8(static_cast<const RT*>(p.dres) + row * p.lddres + c, p.N - c, p.vec_dres, a);
#pragma unroll
                for (int i = 0; i < kVec; ++i) d[i] += a[i];
            }
            store8(static_cast<RT*>(p.dx) + row * p.lddx + c, p.N - c, p.vec_dx, d);
        }
    }
    if (p.part != nullptr) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int c = (t + v * tpr) * kVec;
            if (c < p.N) store8(p.part + group * p.N + c, p.N - c, (p.N & 3) == 0, dw[v]);
        }
    }
}

// The backward pass on a ring of rows (dy, r, dres); see k_rms_fwd_ring.
template <typename YT, typename RT, int VPT>
__global__ void __launch_bounds__(512) k_rms_bwd_ring(const BwdParams p, int stages, int stage_bytes) {
    extern __shared__ __align__(128) uint8_t s_rows[];
    __shared__ __align__(8) uint64_t s_bar[kMaxStages];
    __shared__ float s_part[64];
    const int t = (int)threadIdx.x, T = (int)blockDim.x;
    const uint32_t yb = (uint32_t)p.N * sizeof(YT), rb = (uint32_t)p.N * sizeof(RT);
    const bool with_dres = p.dres != nullptr;
    const int64_t G = gridDim.x;
    auto issue = [&](int st, int64_t row) {
        const uint32_t bar = gg::smem_u32(&s_bar[st]), dst = gg::smem_u32(s_rows + st * stage_bytes);
        gg::mbar_expect_tx(bar, yb + rb + (with_dres ? rb : 0u));
        gg::bulk_load(dst, static_cast<const YT*>(p.dy) + row * p.lddy, yb, bar);
        gg::bulk_load(dst + yb, static_cast<const RT*>(p.r) + row * p.ldr, rb, bar);
        if (with_dres) gg::bulk_load(dst + yb + rb, static_cast<const RT*>(p.dres) + row * p.lddres, rb, bar);
    };
    if (t == 0) {
        for (int i = 0; i < stages; ++i) gg::mbar_init(gg::smem_u32(&s_bar[i]), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    wait_for_previous_kernels();
    if (t == 0) {
        for (int i = 0; i < stages; ++i)
            if (blockIdx.x + i * G < p.M) issue(i, blockIdx.x + i * G);
    }
    float w[VPT][kVec], dw[VPT][kVec];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int c = (t + v * T) * kVec;
        if (c < p.N) load8(p.w, p.w_type, c, kVec, p.vec_w, w[v]);
#pragma unroll
        for (int i = 0; i < kVec; ++i) dw[v][i] = 0.f;
    }
    __syncthreads();
    int st = 0, half = 0;
    uint32_t phase = 0;
    for (int64_t row = blockIdx.x; row < p.M; row += G) {
        const float rstd = p.rstd[row];
        const bool ok = ring_wait(gg::smem_u32(&s_bar[st]), phase);
        const uint8_t* s = s_rows + st * stage_bytes;
        float tv[VPT][kVec], xh[VPT][kVec], a[VPT][kVec];
        float dot = ok ? 0.f : __uint_as_float(0x7FC00000u);      // bytes that never came: the row is NaN
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int c = (t + v * T) * kVec;
            if (c < p.N) {
                load8(reinterpret_cast<const YT*>(s) + c, kVec, true, tv[v]);
                load8(reinterpret_cast<const RT*>(s + yb) + c, kVec, true, xh[v]);
                if (with_dres) load8(reinterpret_cast<const RT*>(s + yb + rb) + c, kVec, true, a[v]);
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    xh[v][i] *= rstd;
                    dw[v][i] = fmaf(tv[v][i], xh[v][i], dw[v][i]);
                    tv[v][i] *= w[v][i];
                    dot = fmaf(tv[v][i], xh[v][i], dot);
                }
            }
        }
        const float mean = row_sum(dot, true, s_part, half) / (float)p.N;
        half ^= 1;
        if (t == 0 && row + stages * G < p.M) issue(st, row + stages * G);
        if (++st == stages) {
            st = 0;
            phase ^= 1u;
        }
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int c = (t + v * T) * kVec;
            if (c >= p.N) continue;
            float d[kVec];
#pragma unroll
            for (int i = 0; i < kVec; ++i) d[i] = rstd * (tv[v][i] - xh[v][i] * mean) + (with_dres ? a[v][i] : 0.f);
            store8(static_cast<RT*>(p.dx) + row * p.lddx + c, kVec, p.vec_dx, d);
        }
    }
    if (p.part != nullptr) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int c = (t + v * T) * kVec;
            if (c < p.N) store8(p.part + (int64_t)blockIdx.x * p.N + c, kVec, true, dw[v]);
        }
    }
}

// Column sums of partial sums [P, N]: a CTA owns 32 columns, its warps every
// 32nd row, and one warp adds the 32 results in order.  P = 0 writes zeros.
__global__ void __launch_bounds__(1024) k_dw_sum(const float* __restrict__ part, int P, int N, float* __restrict__ dw) {
    __shared__ float s[32][33];
    wait_for_previous_kernels();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float a = 0.f;
    if (c < N) {
#pragma unroll 8
        for (int r = warp; r < P; r += 32) a += part[(int64_t)r * N + c];
    }
    s[warp][lane] = a;
    __syncthreads();
    // warp w adds column w of the 32 x 32 sums
    const float v = warp_sum(s[lane][warp]);
    if (lane == 0 && blockIdx.x * 32 + warp < N) dw[blockIdx.x * 32 + warp] = v;
}

// Threads of a row: rows of up to 1024 columns take a warp each, four rows
// to a CTA; longer ones a CTA with 4 vectors per thread.
struct Shape {
    bool block_row;
    int vpt, threads, rows_per_cta;
};
static Shape shape_of(int N) {
    const int nvec = (N + kVec - 1) / kVec;
    if (nvec <= 128) return {false, nvec <= 32 ? 1 : (nvec <= 64 ? 2 : 4), 128, 4};
    return {true, 4, (nvec + 127) / 128 * 32, 1};
}

// The ring kernels' launch: CTAs of an SM, stages, threads.
struct Ring {
    bool use;
    int vpt, threads, ctas, stages, stage_bytes;
};
// `row_bytes`: what a stage holds.  Rows of 1,025 to 16,384 columns, at least
// two stages, and enough rows that every CTA has some to run ahead on.
static Ring ring_of(int64_t M, int N, size_t row_bytes, bool aligned, int sms) {
    Ring r{};
    const int nvec = N / kVec;
    if (!aligned || N % kVec != 0 || N <= 1024 || N > 16384) return r;
    r.vpt = N <= 8192 ? 2 : 4;
    r.threads = (nvec + 32 * r.vpt - 1) / (32 * r.vpt) * 32;
    r.stage_bytes = (int)((row_bytes + 127) / 128 * 128);
    // more CTAs than are resident at a time (their registers allow 1,024
    // threads an SM): the rest start as those before end, which evens them out
    r.ctas = std::max(1, std::min(16, 4096 / r.threads));
    while (r.ctas > 1 && kRingBytes / r.ctas < 2 * r.stage_bytes) --r.ctas;
    r.stages = std::min(kMaxStages, kRingBytes / r.ctas / r.stage_bytes);
    r.use = r.stages >= 2 && M >= 2 * (int64_t)sms;
    return r;
}

static int esize(int type) { return type == MOE_TYPE_F32 ? 4 : 2; }
static bool type_ok(int t) { return t == MOE_TYPE_BF16 || t == MOE_TYPE_F32; }
// 16-byte loads of 8 elements: the base and every row's start are aligned
static bool vec_ok(const void* p, int64_t ld, int type) {
    return moe_aligned16(p) && (ld * esize(type)) % 16 == 0;
}
static bool elem_aligned(const void* p, int type) { return reinterpret_cast<uintptr_t>(p) % esize(type) == 0; }

static int partials(int64_t M, int N) {
    const Shape s = shape_of(N);
    const int64_t cap = s.block_row ? kMaxPartials : 4 * kMaxPartials;
    int64_t g = std::min<int64_t>(M, cap);
    if (!s.block_row) g = (g + s.rows_per_cta - 1) / s.rows_per_cta * s.rows_per_cta;
    return (int)g;
}

template <typename XT, typename RT>
static void launch_fwd(const FwdParams& p, const Shape& s, const Ring& q, int sms, cudaStream_t st) {
    if (q.use) {
        const unsigned g = (unsigned)std::min<int64_t>(p.rows, (int64_t)sms * q.ctas);
        const size_t bytes = (size_t)q.stages * q.stage_bytes;
        if (q.vpt == 2)
            (void)launch_early(dim3(g), q.threads, bytes, st, k_rms_fwd_ring<XT, RT, 2>, p, q.stages, q.stage_bytes);
        else
            (void)launch_early(dim3(g), q.threads, bytes, st, k_rms_fwd_ring<XT, RT, 4>, p, q.stages, q.stage_bytes);
        return;
    }
    const unsigned grid = (unsigned)((p.rows + s.rows_per_cta - 1) / s.rows_per_cta);
    if (s.vpt == 1)
        (void)launch_early(dim3(grid), s.threads, 0, st, k_rms_fwd<XT, RT, 1, 128>, p);
    else if (s.vpt == 2)
        (void)launch_early(dim3(grid), s.threads, 0, st, k_rms_fwd<XT, RT, 2, 128>, p);
    else if (s.threads <= 256)
        (void)launch_early(dim3(grid), s.threads, 0, st, k_rms_fwd<XT, RT, 4, 256>, p);
    else if (s.threads <= 512)
        (void)launch_early(dim3(grid), s.threads, 0, st, k_rms_fwd<XT, RT, 4, 512>, p);
    else
        (void)launch_early(dim3(grid), s.threads, 0, st, k_rms_fwd<XT, RT, 4, 1024>, p);
}
template <typename YT, typename RT>
static void launch_bwd(const BwdParams& p, const Shape& s, const Ring& q, int groups, cudaStream_t st) {
    if (q.use) {
        const size_t bytes = (size_t)q.stages * q.stage_bytes;
        if (q.vpt == 2)
            (void)launch_early(dim3(groups), q.threads, bytes, st, k_rms_bwd_ring<YT, RT, 2>, p, q.stages, q.stage_bytes);
        else
            (void)launch_early(dim3(groups), q.threads, bytes, st, k_rms_bwd_ring<YT, RT, 4>, p, q.stages, q.stage_bytes);
        return;
    }
    const unsigned grid = (unsigned)(groups / s.rows_per_cta);
    if (s.vpt == 1)
        (void)launch_early(dim3(grid), s.threads, 0, st, k_rms_bwd<YT, RT, 1, 128>, p);
    else if (s.vpt == 2)
        (void)launch_early(dim3(grid), s.threads, 0, st, k_rms_bwd<YT, RT, 2, 128>, p);
    else if (s.threads <= 256)
        (void)launch_early(dim3(grid), s.threads, 0, st, k_rms_bwd<YT, RT, 4, 256>, p);
    else if (s.threads <= 512)
        (void)launch_early(dim3(grid), s.threads, 0, st, k_rms_bwd<YT, RT, 4, 512>, p);
    else
        (void)launch_early(dim3(grid), s.threads, 0, st, k_rms_bwd<YT, RT, 4, 1024>, p);
}

template <typename XT, typename RT>
static cudaError_t set_ring() {
    const void* ks[] = {(const void*)k_rms_fwd_ring<XT, RT, 2>, (const void*)k_rms_fwd_ring<XT, RT, 4>,
                        (const void*)k_rms_bwd_ring<XT, RT, 2>, (const void*)k_rms_bwd_ring<XT, RT, 4>};
    for (const void* k : ks) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace norm

cudaError_t norm_set_attributes() {
    using namespace norm;
    const cudaError_t es[] = {set_ring<__nv_bfloat16, __nv_bfloat16>(), set_ring<__nv_bfloat16, float>(),
                              set_ring<float, __nv_bfloat16>(), set_ring<float, float>()};
    for (cudaError_t e : es)
        if (e != cudaSuccess) return e;
    return cudaSuccess;
}

// out[c] = sum over the P rows of part [P, N], in a fixed order; zeros for P = 0
void launch_column_sum(const float* part, int P, int N, float* out, cudaStream_t s) {
    (void)launch_early(dim3((N + 31) / 32), 1024, 0, s, norm::k_dw_sum, part, P, N, out);
}

}  // namespace moe

extern "C" moe_status_t rmsnorm_residual_fwd(const void* x, int x_type, int64_t ldx, const void* res, int res_type,
                                             int64_t ldres, const void* w, int w_type, float eps, int64_t M, int N,
                                             void* r, int64_t ldr, void* y, int y_type, int64_t ldy, float* rstd,
                                             uint8_t* codes, uint8_t* scales, int sf_layout, void* stream) {
    using namespace moe;
    using namespace moe::norm;
    MOE_REQUIRE(M >= 0 && N >= 1 && type_ok(x_type) && type_ok(res_type) && type_ok(w_type) && type_ok(y_type),
                MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(eps >= 0.f && ldx >= N && (!res || ldres >= N) && (!r || ldr >= N) && (!y || ldy >= N),
                MOE_ERR_INVALID_ARG);
    MOE_REQUIRE((codes == nullptr) == (scales == nullptr), MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(sf_layout == MOE_SF_ATOMS || sf_layout == MOE_SF_CANONICAL, MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(N <= kMaxN && M <= 0x7FFFFF00LL, MOE_ERR_UNSUPPORTED);
    if (codes) MOE_REQUIRE(N % (sf_layout == MOE_SF_ATOMS ? 128 : 32) == 0, MOE_ERR_UNSUPPORTED);
    if (M == 0) return MOE_OK;
    MOE_REQUIRE(x && w && (y || codes || r || rstd), MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(elem_aligned(x, x_type) && elem_aligned(res, res_type) && elem_aligned(w, w_type) &&
                    elem_aligned(r, res_type) && elem_aligned(y, y_type) &&
                    reinterpret_cast<uintptr_t>(rstd) % 4 == 0 && moe_aligned16(codes),
                MOE_ERR_ALIGNMENT);
    MOE_REQUIRE(device_initialized(), MOE_ERR_NOT_INITIALIZED);
    const Shape s = shape_of(N);
    FwdParams p{};
    p.x = x, p.res = res, p.w = w, p.r = r, p.y = y, p.rstd = rstd, p.codes = codes, p.scales = scales;
    p.ldx = ldx, p.ldres = ldres, p.ldr = ldr, p.ldy = ldy;
    p.M = M, p.N = N;
    p.sf_canonical = sf_layout == MOE_SF_CANONICAL;
    p.rows = codes && !p.sf_canonical ? (M + 127) / 128 * 128 : M;
    p.w_type = w_type, p.y_type = y_type, p.eps = eps;
    p.block_row = s.block_row;
    p.vec_x = vec_ok(x, ldx, x_type), p.vec_res = vec_ok(res, ldres, res_type), p.vec_w = moe_aligned16(w);
    p.vec_r = vec_ok(r, ldr, res_type), p.vec_y = vec_ok(y, ldy, y_type);
    const int sms = device_sm_count();
    const Ring q = ring_of(M, N, (size_t)N * (esize(x_type) + (res ? esize(res_type) : 0)),
                           p.vec_x && (!res || p.vec_res), sms);
    cudaStream_t st = (cudaStream_t)stream;
    if (x_type == MOE_TYPE_BF16 && res_type == MOE_TYPE_BF16)
        launch_fwd<__nv_bfloat16, __nv_bfloat16>(p, s, q, sms, st);
    else if (x_type == MOE_TYPE_BF16)
        launch_fwd<__nv_bfloat16, float>(p, s, q, sms, st);
    else if (res_type == MOE_TYPE_BF16)
        launch_fwd<float, __nv_bfloat16>(p, s, q, sms, st);
    else
        launch_fwd<float, float>(p, s, q, sms, st);
    MOE_CHECK_LAUNCH();
    return MOE_OK;
}

extern "C" size_t rmsnorm_bwd_workspace_size(int64_t M, int N) {
    if (M < 0 || M > 0x7FFFFF00LL || N < 1 || N > moe::norm::kMaxN) return (size_t)-1;
    return (size_t)moe::norm::partials(M, N) * N * sizeof(float);
}

extern "C" moe_status_t rmsnorm_residual_bwd(const void* dy, int dy_type, int64_t lddy, const void* r, int r_type,
                                             int64_t ldr, const void* w, int w_type, const float* rstd,
                                             const void* dres, int64_t lddres, int64_t M, int N, void* dx,
                                             int64_t lddx, float* dw, void* ws, size_t ws_bytes, void* stream) {
    using namespace moe;
    using namespace moe::norm;
    MOE_REQUIRE(M >= 0 && N >= 1 && type_ok(dy_type) && type_ok(r_type) && type_ok(w_type), MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(lddy >= N && ldr >= N && lddx >= N && (!dres || lddres >= N), MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(N <= kMaxN && M <= 0x7FFFFF00LL, MOE_ERR_UNSUPPORTED);
    MOE_REQUIRE(M == 0 || (dy && r && w && rstd && dx), MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(elem_aligned(dy, dy_type) && elem_aligned(r, r_type) && elem_aligned(w, w_type) &&
                    elem_aligned(dres, r_type) && elem_aligned(dx, r_type) &&
                    reinterpret_cast<uintptr_t>(rstd) % 4 == 0 && reinterpret_cast<uintptr_t>(dw) % 4 == 0 &&
                    moe_aligned16(ws),
                MOE_ERR_ALIGNMENT);
    const Shape s = shape_of(N);
    int groups = partials(M, N);
    MOE_REQUIRE(!dw || M == 0 || (ws && ws_bytes >= rmsnorm_bwd_workspace_size(M, N)), MOE_ERR_WORKSPACE);
    MOE_REQUIRE(device_initialized(), MOE_ERR_NOT_INITIALIZED);
    cudaStream_t st = (cudaStream_t)stream;
    if (M > 0) {
        BwdParams p{};
        p.dy = dy, p.r = r, p.w = w, p.rstd = rstd, p.dres = dres, p.dx = dx;
        p.part = dw ? static_cast<float*>(ws) : nullptr;
        p.lddy = lddy, p.ldr = ldr, p.lddres = lddres, p.lddx = lddx, p.M = M, p.N = N, p.w_type = w_type;
        p.block_row = s.block_row;
        p.vec_dy = vec_ok(dy, lddy, dy_type), p.vec_r = vec_ok(r, ldr, r_type), p.vec_w = moe_aligned16(w);
        p.vec_dres = vec_ok(dres, lddres, r_type), p.vec_dx = vec_ok(dx, lddx, r_type);
        const int sms = device_sm_count();
        const Ring q = ring_of(M, N, (size_t)N * (esize(dy_type) + (dres ? 2 : 1) * esize(r_type)),
                               p.vec_dy && p.vec_r && (!dres || p.vec_dres), sms);
        if (q.use) groups = (int)std::min<int64_t>(groups, (int64_t)sms * q.ctas);
        if (dy_type == MOE_TYPE_BF16 && r_type == MOE_TYPE_BF16)
            launch_bwd<__nv_bfloat16, __nv_bfloat16>(p, s, q, groups, st);
        else if (dy_type == MOE_TYPE_BF16)
            launch_bwd<__nv_bfloat16, float>(p, s, q, groups, st);
        else if (r_type == MOE_TYPE_BF16)
            launch_bwd<float, __nv_bfloat16>(p, s, q, groups, st);
        else
            launch_bwd<float, float>(p, s, q, groups, st);
        MOE_CHECK_LAUNCH();
    }
    if (dw) {
        launch_column_sum(static_cast<const float*>(ws), M > 0 ? groups : 0, N, dw, st);
        MOE_CHECK_LAUNCH();
    }
    return MOE_OK;
}
