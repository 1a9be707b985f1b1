// One AdamW step over many tensors in one launch, states in 32 or 8 bits.
//
//   g <- grad_scale g
//   m <- b1 m + (1 - b1) g,   v <- b2 v + (1 - b2) g^2
//   p <- p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps)
//
// All arithmetic is fp32 on the values as read; p, its 16-bit copy, m and v
// are each rounded once, when they are stored.  The update uses m and v
// before they are rounded to 8 bits.
//
// States in 8 bits: per block of 256 elements of a tensor an fp32 scale s
// and 256 E4M3 codes; m is held as code * s, v by its square root,
// v = (code * s)^2, which halves the range of exponents the codes have to
// span.  s is the block's largest magnitude over 448.  v moves by a
// thousandth of itself in a step (b2 = 0.999) while neighbouring codes are a
// sixteenth to an eighth apart: rounding to nearest would leave it where it
// is for ever.  So codes are rounded down or up with the probability that
// keeps their mean (dithered by 16 mixed bits of the element's counter, the
// step and the seed: the same inputs give the same codes).  A v that is not
// zero is never rounded to zero, which would let m / (sqrt(v) + eps) explode.
//
// m, v and the 8-bit rounding are a stated sequence of single fp32 operations
// (products and sums rounded one by one), so that states, which feed the next
// step, are the same bits wherever they are computed.
//
// The pass has to read p, g, m, v and write p, m, v once.
#include <math.h>

#include <algorithm>

#include "gemm_common.cuh"

namespace moe {
namespace adamw {

constexpr int kBlock = 256;                 // elements per 8-bit scale: one warp, 8 per lane
constexpr int kThreads = 256;
constexpr int kSub = kThreads * 8;          // elements that a CTA works on at a time
// Elements of a tile, the unit that CTAs take.  8-bit states of bf16 tensors
// take two parts in one stage, with one barrier for both (344 against 358 us
// for 130 M elements); with fp32 tensors, whose stages are larger, that costs
// a CTA per SM (60 M elements, fp32 p and g: 169 against 155 us).
constexpr int tile_of(int bits, int p_and_g_bytes) { return bits == 8 && p_and_g_bytes == 4 ? 2 * kSub : kSub; }
constexpr int kMaxTensors = 1 << 20;

// One tensor in the device table (moe_adamw_tensor_t plus what the kernel
// needs to know about its addresses).
struct Entry {
    void* p;
    const void* g;
    void* m;
    void* v;
    float* ms;
    float* vs;
    __nv_bfloat16* copy;
    int64_t n;
    int64_t rng;
    float wd;
    int vec;        // every address allows 8-element vectors (1), and bulk copies (2)
};
static_assert(sizeof(Entry) == 80, "table layout");

struct Params {
    const Entry* e;
    const int64_t* tile0;     // [tensors + 1]: first tile of each tensor
    int tensors;
    int64_t tiles;
    float lr, b1, b2, c1, c2, eps;      // c = 1 - b
    float inv_bc1, inv_bc2;             // 1 / (1 - b^t), host step
    float ln_b1, ln_b2;                 // device step
    uint32_t key;                       // mixed seed and step, host step
    uint32_t seed;
    const float* lr_dev;
    int32_t* step_dev;
    uint32_t* ticket;
    const float* grad_scale;
};

// 32 mixed bits of 32: two rounds of xor-shift and an odd multiplier, and
// the upper half folded onto the lower one.
__host__ __device__ __forceinline__ uint32_t mix_unfolded(uint32_t x) {
    x = (x ^ (x >> 16)) * 0x9E3779B1u;
    return (x ^ (x >> 15)) * 0x85EBCA77u;
}
__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
    x = mix_unfolded(x);
    return x ^ (x >> 16);
}

__device__ __forceinline__ void load8(const float* p, float* f) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* f) {
    unpack8(*reinterpret_cast<const uint4*>(p), f);
}
__device__ __forceinline__ void store8(float* p, const float* f) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* f) { *reinterpret_cast<uint4*>(p) = pack8(f); }
__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float* p, float v) { *p = v; }
__device__ __forceinline__ void from_f(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <typename T>
__device__ __forceinline__ void load(const T* p, int n, bool vec, float* f) {
    if (vec && n >= 8) {
        load8(p, f);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = i < n ? to_f(p[i]) : 0.f;
    }
}
template <typename T>
__device__ __forceinline__ void store(T* p, int n, bool vec, const float* f) {
    if (vec && n >= 8) {
        store8(p, f);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) from_f(p + i, f[i]);
    }
}

// Two fp32 at a time (the packed forms take one issue slot for two results;
// each is rounded as the single form rounds it).
struct F2 {
    uint64_t v;
    __device__ __forceinline__ F2() {}
    __device__ __forceinline__ F2(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
    __device__ __forceinline__ explicit F2(float a) : F2(a, a) {}
    __device__ __forceinline__ void get(float& a, float& b) const {
        asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
    }
};
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
// The sum stays two single additions: a packed product whose only use is a
// packed sum is contracted into a fused multiply-add, which rounds once where
// the states' arithmetic rounds twice.
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    float x0, x1, y0, y1;
    a.get(x0, x1);
    b.get(y0, y1);
    return F2(__fadd_rn(x0, y0), __fadd_rn(x1, y1));
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Square roots of two values from 2^-100 on, correctly rounded: y = x rsqrt(x)
// from the approximate instruction, then one step along the exact residual,
// y + (x - y^2) rsqrt(x) / 2 in fused multiply-adds (Markstein's correction).
// No branch for the cases that sqrtf sets apart, and half the issue slots.
// Infinity and NaN give themselves; zero does where ZERO says that it may come.
constexpr float kSqrtLeast = 7.888609052e-31f;      // 2^-100: below, x - y^2 has bits that fp32 does not hold
template <bool ZERO>
__device__ __forceinline__ F2 sqrt2(F2 x) {
    float x0, x1, r0, r1;
    x.get(x0, x1);
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(ZERO ? fmaxf(x0, 1.17549435e-38f) : x0));
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(ZERO ? fmaxf(x1, 1.17549435e-38f) : x1));
    const F2 r(r0, r1), y = mul2(x, r);
    float z0, z1;
    fma2(fma2(mul2(y, F2(-1.f)), y, x), mul2(r, F2(0.5f)), y).get(z0, z1);
    return F2(x0 <= 3.402823466e38f ? z0 : x0, x1 <= 3.402823466e38f ? z1 : x1);
}
// The same of any value >= 0: below 2^-100, zero and subnormals among them,
// as 2^-50 sqrt(2^100 x), both factors exact.
__device__ __forceinline__ F2 sqrt2_any(F2 x) {
    float x0, x1;
    x.get(x0, x1);
    const bool s0 = x0 < kSqrtLeast, s1 = x1 < kSqrtLeast;
    const F2 up(s0 ? 1.267650600e30f : 1.f, s1 ? 1.267650600e30f : 1.f);
    const F2 down(s0 ? 8.881784197e-16f : 1.f, s1 ? 8.881784197e-16f : 1.f);
    return mul2(sqrt2<true>(mul2(x, up)), down);
}

// E4M3 codes to fp32 times 2^-120, in integer arithmetic (the conversion
// instructions run at a quarter of its rate): the code's exponent and
// mantissa moved into those of an fp32, exact, subnormal codes included.
// (Code 0x7F is written only where the block's scale is not finite.)
template <bool SIGNED>
__device__ __forceinline__ float e4m3_bits(uint32_t w, int i) {      // byte i of w
    if (SIGNED) return __uint_as_float((uint32_t)((int32_t)(w << (24 - 8 * i)) >> 4) & 0x87F00000u);
    return __uint_as_float((i == 3 ? w >> 4 : w << (20 - 8 * i)) & 0x07F00000u);
}
template <bool SIGNED>
__device__ __forceinline__ void load_codes(const uint8_t* p, int n, bool vec, float* f) {
    uint32_t w[2] = {0u, 0u};
    if (vec && n >= 8) {
        const uint2 q = *reinterpret_cast<const uint2*>(p);
        w[0] = q.x, w[1] = q.y;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) w[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = e4m3_bits<SIGNED>(w[i >> 2], i & 3);
}
__device__ __forceinline__ void store_codes(uint8_t* p, int n, bool vec, const uint32_t* w) {
    if (vec && n >= 8) {
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
    }
}

// |x| (up to 448) rounded to E4M3 as 16 dither bits say,
//   floor(|x| / step + dither / 2^16) * step,  step = 2^(exponent - 3), 2^-9 below 2^-6.
// `x` comes times 2^-120: its fp32 pattern then has the code in bits 20..26,
// subnormal where the code is, and the dither is added right below bit 20
// (`d` holds it in bits 8..23, four places up).  The code is returned
// in bits 24..30, with noise below and bit 31 clear.
__device__ __forceinline__ uint32_t e4m3_code(float x, uint32_t d) { return (__float_as_uint(x) << 4) + d; }
// the top bytes of four words
__device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
}

// Largest of a block's values (>= 0, or NaN), over its warp.
__device__ __forceinline__ float block_top(const float* f) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(fabsf(f[i])));
    return __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, m));
}
// A block's scale and its inverse; a block whose largest magnitude is under
// 1e-35 (whose inverse scale fp32 does not hold) is zero.
__device__ __forceinline__ void block_scale(float top, float& scale, float& inv) {
    const bool some = !(top <= 1e-35f);      // NaN too
    scale = some ? __fmul_rn(top, 1.f / 448.f) : 0.f;
    inv = some ? __fmul_rn(__frcp_rn(top), 448.f) : 0.f;
}

// A tile's bytes in shared memory (8 bits only): p, g, m, v, and the scales of each state.
template <typename PT, typename GT, int BITS>
struct Stage {
    static constexpr int kTile = tile_of(BITS, (int)(sizeof(PT) + sizeof(GT)));
    static constexpr int P = kTile * (int)sizeof(PT), G = kTile * (int)sizeof(GT), S = kTile;
    static constexpr int SC = kTile / kBlock * 4;
    static constexpr int OFF_G = P, OFF_M = P + G, OFF_V = OFF_M + S, OFF_MS = OFF_V + S, OFF_VS = OFF_MS + SC;
    static constexpr int BYTES = OFF_VS + SC;
    // CTAs of an SM and stages of a CTA: about 192 KB on their way per SM
    static constexpr int CTAS = BITS == 32 ? 3 : 4;
    static constexpr int FIT = 204800 / CTAS / BYTES;
    static constexpr int STAGES = BITS == 32 ? 1 : (FIT >= 4 ? 4 : (FIT >= 3 ? 3 : 2));
    static constexpr int RING = BITS == 32 ? 0 : STAGES * BYTES;
};

// A place in the table: a tile's tensor, and the tensor's tiles.
struct Cursor {
    int k;
    int64_t first, next;
    __device__ __forceinline__ bool seek(const Params& p, int64_t t) {      // whether the tensor changed
        if (t < next) return false;                                         // (tiles are visited in order)
        int hi = p.tensors - 1;      // the last tensor that starts at or before t
        while (k < hi) {
            const int mid = (k + hi + 1) >> 1;
            if (p.tile0[mid] <= t) k = mid;
            else hi = mid - 1;
        }
        first = p.tile0[k];
        next = p.tile0[k + 1];
        return true;
    }
};
// Whole tiles of aligned tensors come through the ring of stages.
template <typename S>
__device__ __forceinline__ bool in_ring(const Entry& e, int64_t tile) {
    return S::RING > 0 && e.vec == 2 && (tile + 1) * S::kTile <= e.n;
}

// A CTA takes every G-th tile, so that many small tensors in a row are spread
// over all CTAs.
//
// 32 bits: 28 bytes and about 30 instructions an element; loads straight into
// registers, three CTAs an SM (176 M elements, fp32 p, bf16 g and copy: 751 us,
// 6.57 TB/s, 97 % of the copy bandwidth; through a ring in shared memory 805 us).
// 8 bits: 10 bytes and 73 instructions an element (a third of them the rounding
// of the codes).  Loads into registers covered less than half of the memory's
// latency at the occupancy those leave, so bulk copies bring the next whole
// tiles into a ring in shared memory while the CTA works on one (130 M
// elements, bf16 p and g: 340 us, 3.8 TB/s; 410 us without the ring, when that
// was measured).  Nothing is at its limit: 70 % of the issue slots and 45 % of the
// memory's rate are used, a sixth of the warps' time goes at the CTA's barrier
// and as much waiting for the math pipes; with every slot used it would be 240 us.
template <typename PT, typename GT, int BITS>
__global__ void __launch_bounds__(kThreads, (Stage<PT, GT, BITS>::CTAS)) k_adamw(const Params p) {
    using S = Stage<PT, GT, BITS>;
    extern __shared__ __align__(128) uint8_t s_ring[];
    __shared__ __align__(8) uint64_t s_bar[S::STAGES];
    __shared__ float s_h[4];
    __shared__ uint32_t s_key;
    const int64_t t0 = blockIdx.x, t1 = p.tiles, G = gridDim.x;
    Cursor pc{0, 0, 0};         // thread 0: the next tile to fetch
    int64_t pt = t0;
    int pstage = 0;
    // Fetches up to `most` more whole tiles of the CTA's share.
    auto fetch = [&](int most) {
        while (most > 0 && pt < t1) {
            pc.seek(p, pt);
            const Entry& e = p.e[pc.k];
            const int64_t tile = pt - pc.first;
            pt += G;
            if (!in_ring<S>(e, tile)) continue;
            const uint32_t bar = gg::smem_u32(&s_bar[pstage]), dst = gg::smem_u32(s_ring + pstage * S::BYTES);
            gg::mbar_expect_tx(bar, S::BYTES);
            gg::bulk_load(dst, static_cast<const uint8_t*>(e.p) + tile * S::P, S::P, bar);
            gg::bulk_load(dst + S::OFF_G, static_cast<const uint8_t*>(e.g) + tile * S::G, S::G, bar);
            gg::bulk_load(dst + S::OFF_M, static_cast<const uint8_t*>(e.m) + tile * S::S, S::S, bar);
            gg::bulk_load(dst + S::OFF_V, static_cast<const uint8_t*>(e.v) + tile * S::S, S::S, bar);
            gg::bulk_load(dst + S::OFF_MS, e.ms + tile * (S::kTile / kBlock), S::SC, bar);
            gg::bulk_load(dst + S::OFF_VS, e.vs + tile * (S::kTile / kBlock), S::SC, bar);
            if (++pstage == S::STAGES) pstage = 0;
            --most;
        }
    };
    wait_for_previous_kernels();
    if (threadIdx.x == 0) {
        float i1 = p.inv_bc1, i2 = p.inv_bc2;
        uint32_t key = p.key;
        if (p.step_dev != nullptr) {
            const int t = *(volatile int32_t*)p.step_dev + 1;
            i1 = 1.f / -expm1f((float)t * p.ln_b1);
            i2 = 1.f / -expm1f((float)t * p.ln_b2);
            key = mix(p.seed ^ mix((uint32_t)t));
        }
        s_h[0] = i1, s_h[1] = sqrtf(i2);
        s_h[2] = p.lr_dev ? *p.lr_dev : p.lr;
        const float gs = p.grad_scale ? *p.grad_scale : 1.f;
        s_h[3] = gs;
        s_key = key;
        if constexpr (S::RING > 0) {
            for (int i = 0; i < S::STAGES; ++i) gg::mbar_init(gg::smem_u32(&s_bar[i]), 1);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
            if (fabsf(gs) <= 3.402823466e38f) fetch(S::STAGES);
        }
    }
    __syncthreads();
    const float lr = s_h[2], gs = s_h[3], root2 = s_h[1], lr1 = lr * s_h[0];
    const uint32_t key = s_key;
    const bool skip = !(fabsf(gs) <= 3.402823466e38f);      // NaN or infinite: the step is not taken
    Cursor cur{0, 0, 0};
    Entry e{};
    int stage = 0;
    uint32_t phase = 0;
    for (int64_t t = t0; t < t1 && !skip; t += G) {
        if (cur.seek(p, t)) e = p.e[cur.k];
        const int64_t tile = t - cur.first;
        const bool ring = in_ring<S>(e, tile);
        bool ok = true;
        if (ring) {
            ok = false;
            for (int i = 0; i < (1 << 16) && !ok; ++i) ok = gg::mbar_try_wait(gg::smem_u32(&s_bar[stage]), phase);
        }
#pragma unroll 1
        for (int sub = 0; sub < S::kTile; sub += kSub) {
            const int64_t at = tile * S::kTile + sub + 8 * (int)threadIdx.x;
            const int64_t left = e.n - at;
            const int n = left >= 8 ? 8 : (left > 0 ? (int)left : 0);
            const bool vec = e.vec != 0;
            float g[8], w[8], m[8], v[8], u[8];
            float sm = 0.f, sv = 0.f;
            if (ring) {
                const uint8_t* s = s_ring + stage * S::BYTES;
                const int o = sub + 8 * (int)threadIdx.x;
                load(reinterpret_cast<const PT*>(s) + o, 8, true, w);
                load(reinterpret_cast<const GT*>(s + S::OFF_G) + o, 8, true, g);
                load_codes<true>(s + S::OFF_M + o, 8, true, m);
                load_codes<false>(s + S::OFF_V + o, 8, true, v);
                sm = reinterpret_cast<const float*>(s + S::OFF_MS)[o / kBlock];
                sv = reinterpret_cast<const float*>(s + S::OFF_VS)[o / kBlock];
                if (sub == S::kTile - kSub) {
                    __syncthreads();      // the stage is read
                    if (threadIdx.x == 0) fetch(1);
                    if (++stage == S::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            } else {
                load(static_cast<const GT*>(e.g) + at, n, vec, g);
                load(static_cast<PT*>(e.p) + at, n, vec, w);
                if (BITS == 32) {
                    load(static_cast<float*>(e.m) + at, n, vec, m);
                    load(static_cast<float*>(e.v) + at, n, vec, v);
                } else {
                    load_codes<true>(static_cast<uint8_t*>(e.m) + at, n, vec, m);
                    load_codes<false>(static_cast<uint8_t*>(e.v) + at, n, vec, v);
                    // the warp's block: its first element exists or the whole warp is past the end
                    const int64_t b = (at - 8 * (int)(threadIdx.x & 31)) / kBlock;
                    if (b * kBlock < e.n) {
                        sm = e.ms[b];
                        sv = e.vs[b];
                    }
                }
            }
            if (BITS == 8) {
                // code * 2^-120 * (2^120 * scale), rounded once; scales of 128 and
                // more, whose product fp32 does not hold, in two steps
                const float up = __uint_as_float((120u + 127u) << 23);
                const bool one = sm < 128.f && sv < 128.f;
                const F2 sm2(one ? sm * up : up), sv2(one ? sv * up : up);
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    mul2(F2(m[i], m[i + 1]), sm2).get(m[i], m[i + 1]);
                    mul2(F2(v[i], v[i + 1]), sv2).get(v[i], v[i + 1]);
                }
                if (!one) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) m[i] *= sm, v[i] *= sv;
                }
#pragma unroll
                for (int i = 0; i < 8; i += 2) mul2(F2(v[i], v[i + 1]), F2(v[i], v[i + 1])).get(v[i], v[i + 1]);
            }
            const F2 decay(1.f - lr * e.wd);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const F2 g2 = mul2(F2(g[i], g[i + 1]), F2(gs));
                const F2 m2 = add2(mul2(F2(p.b1), F2(m[i], m[i + 1])), mul2(F2(p.c1), g2));
                const F2 v2 = add2(mul2(F2(p.b2), F2(v[i], v[i + 1])), mul2(mul2(F2(p.c2), g2), g2));
                m2.get(m[i], m[i + 1]);
                v2.get(v[i], v[i + 1]);
                if (BITS == 32) sqrt2_any(v2).get(u[i], u[i + 1]);
            }
            if (BITS == 8) {
                // instructions count here: four an element fewer while none of the eight
                // is small (with 32 bits, bound by memory, they are free, and the smallest
                // steps take 4.8 us without the branch, 5.1 with it)
                float least = v[0];
#pragma unroll
                for (int i = 1; i < 8; ++i) least = fminf(least, v[i]);
                if (least >= kSqrtLeast) {
#pragma unroll
                    for (int i = 0; i < 8; i += 2) sqrt2<false>(F2(v[i], v[i + 1])).get(u[i], u[i + 1]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; i += 2) sqrt2_any(F2(v[i], v[i + 1])).get(u[i], u[i + 1]);
                }
            }
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                float d0, d1;
                fma2(F2(u[i], u[i + 1]), F2(root2), F2(p.eps)).get(d0, d1);
                const F2 q = mul2(mul2(F2(m[i], m[i + 1]), F2(-lr1)), F2(rcp_approx(d0), rcp_approx(d1)));
                fma2(F2(w[i], w[i + 1]), decay, q).get(w[i], w[i + 1]);
            }
            if (!ok) {      // bytes that never came: the parameters say so
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = __uint_as_float(0x7FC00000u);
            }
            store(static_cast<PT*>(e.p) + at, n, vec, w);
            if (e.copy != nullptr) store(e.copy + at, n, vec, w);
            if (BITS == 32) {
                store(static_cast<float*>(e.m) + at, n, vec, m);
                store(static_cast<float*>(e.v) + at, n, vec, v);
            } else {
                const int64_t b = (at - 8 * (int)(threadIdx.x & 31)) / kBlock;
                if (n < 8) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        m[i] = i < n ? m[i] : 0.f;
                        u[i] = i < n ? u[i] : 0.f;
                    }
                }
                float im, su, iu;
                block_scale(block_top(m), sm, im);
                block_scale(block_top(u), su, iu);
                const uint64_t c = (uint64_t)(e.rng + at);     // blocks start at multiples of 256 of the counter
                const uint32_t lo = (uint32_t)c + mix((uint32_t)(c >> 32) ^ key);
                const F2 down(__uint_as_float((127u - 120u) << 23));
                uint32_t cm[8], cu[8];
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    mul2(mul2(F2(m[i], m[i + 1]), F2(im)), down).get(m[i], m[i + 1]);
                    float x[2];
                    mul2(mul2(F2(u[i], u[i + 1]), F2(iu)), down).get(x[0], x[1]);
#pragma unroll
                    for (int j = i; j < i + 2; ++j) {
                        const uint32_t bits = mix_unfolded(lo + (uint32_t)j);
                        // the low 16 bits of bits ^ bits >> 16, and the high ones, in bits 8..23
                        cm[j] = e4m3_code(m[j], __byte_perm(bits ^ (bits >> 16), 0u, 0x4104));
                        // not zero: never rounded to zero
                        cu[j] = max(e4m3_code(x[j - i], __byte_perm(bits, 0u, 0x4324)),
                                    min(__float_as_uint(u[j]), 1u) << 24);
                    }
                }
                uint32_t wm[2], wu[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t sign[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) sign[i] = __float_as_uint(m[4 * j + i]);
                    wm[j] = top_bytes(cm[4 * j], cm[4 * j + 1], cm[4 * j + 2], cm[4 * j + 3]) |
                            (top_bytes(sign[0], sign[1], sign[2], sign[3]) & 0x80808080u);
                    wu[j] = top_bytes(cu[4 * j], cu[4 * j + 1], cu[4 * j + 2], cu[4 * j + 3]);
                }
                store_codes(static_cast<uint8_t*>(e.m) + at, n, vec, wm);
                store_codes(static_cast<uint8_t*>(e.v) + at, n, vec, wu);
                if ((threadIdx.x & 31) == 0 && n > 0) {
                    e.ms[b] = sm;
                    e.vs[b] = su;
                }
            }
        }
    }
    if (p.step_dev != nullptr) {
        // the last CTA to come here counts the step: every CTA has read it by then
        if (threadIdx.x == 0) {
            __threadfence();
            if (atomicAdd(p.ticket, 1u) == gridDim.x - 1) {
                *p.ticket = 0u;
                if (!skip) *p.step_dev += 1;
            }
        }
    }
}

static int esize(int type) { return type == MOE_TYPE_F32 ? 4 : 2; }
static bool type_ok(int t) { return t == MOE_TYPE_BF16 || t == MOE_TYPE_F32; }
static bool al(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

static size_t tile_table_at(int tensors) { return 16 + (size_t)tensors * sizeof(Entry); }

template <typename PT, typename GT, int BITS>
static void launch(const Params& p, int sms, cudaStream_t s) {
    using S = Stage<PT, GT, BITS>;
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(p.tiles, (int64_t)sms * (BITS == 32 ? 8 : S::CTAS)));
    (void)launch_early(dim3(grid), kThreads, S::RING, s, k_adamw<PT, GT, BITS>, p);
}
template <typename PT, typename GT>
static void launch(int bits, const Params& p, int sms, cudaStream_t s) {
    if (bits == 32) launch<PT, GT, 32>(p, sms, s);
    else launch<PT, GT, 8>(p, sms, s);
}
template <typename PT, typename GT, int BITS>
static cudaError_t set_one() {
    using S = Stage<PT, GT, BITS>;
    static_assert(BITS == 32 || S::STAGES >= 2, "ring");
    return cudaFuncSetAttribute(k_adamw<PT, GT, BITS>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::RING);
}

}  // namespace adamw

cudaError_t adamw_set_attributes() {
    using namespace adamw;
    using B = __nv_bfloat16;
    const cudaError_t es[] = {set_one<float, float, 32>(), set_one<float, B, 32>(), set_one<B, float, 32>(),
                              set_one<B, B, 32>(),         set_one<float, float, 8>(), set_one<float, B, 8>(),
                              set_one<B, float, 8>(),      set_one<B, B, 8>()};
    for (cudaError_t e : es)
        if (e != cudaSuccess) return e;
    return cudaSuccess;
}

}  // namespace moe

extern "C" size_t adamw_plan_bytes(int tensors) {
    if (tensors < 1 || tensors > moe::adamw::kMaxTensors) return (size_t)-1;
    return moe::adamw::tile_table_at(tensors) + (size_t)(tensors + 1) * sizeof(int64_t);
}

extern "C" moe_status_t adamw_plan_encode(const moe_adamw_tensor_t* t, int tensors, int p_type, int g_type,
                                          int state_bits, void* plan, int64_t* tiles) {
    using namespace moe::adamw;
    MOE_REQUIRE(t && plan && tiles && tensors >= 1 && tensors <= kMaxTensors, MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(type_ok(p_type) && type_ok(g_type) && (state_bits == 32 || state_bits == 8), MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(al(plan, 8), MOE_ERR_ALIGNMENT);
    unsigned char* base = static_cast<unsigned char*>(plan);
    int64_t* head = reinterpret_cast<int64_t*>(base);
    head[0] = head[1] = 0;
    Entry* e = reinterpret_cast<Entry*>(base + 16);
    int64_t* tile0 = reinterpret_cast<int64_t*>(base + tile_table_at(tensors));
    int64_t at = 0;
    const size_t sb = state_bits == 32 ? 4 : 1;
    const int tile = tile_of(state_bits, esize(p_type) + esize(g_type));
    for (int i = 0; i < tensors; ++i) {
        const moe_adamw_tensor_t& a = t[i];
        MOE_REQUIRE(a.n >= 0 && a.n <= (1LL << 40), MOE_ERR_INVALID_ARG);
        if (a.n > 0) {
            MOE_REQUIRE(a.p && a.g && a.m && a.v, MOE_ERR_INVALID_ARG);
            MOE_REQUIRE(state_bits == 32 || (a.m_scale && a.v_scale && a.rng_base >= 0 && a.rng_base % kBlock == 0),
                        MOE_ERR_INVALID_ARG);
            MOE_REQUIRE(al(a.p, esize(p_type)) && al(a.g, esize(g_type)) && al(a.m, sb) && al(a.v, sb) &&
                            al(a.m_scale, 4) && al(a.v_scale, 4) && al(a.copy, 2),
                        MOE_ERR_ALIGNMENT);
        }
        Entry& o = e[i];
        o.p = a.p, o.g = a.g, o.m = a.m, o.v = a.v;
        o.ms = a.m_scale, o.vs = a.v_scale, o.copy = static_cast<__nv_bfloat16*>(a.copy);
        o.n = a.n, o.rng = a.rng_base, o.wd = a.weight_decay;
        o.vec = al(a.p, 16) && al(a.g, 16) && al(a.m, state_bits == 32 ? 16 : 8) &&
                al(a.v, state_bits == 32 ? 16 : 8) && al(a.copy, 16);
        if (o.vec && al(a.m, 16) && al(a.v, 16) && al(a.m_scale, 16) && al(a.v_scale, 16)) o.vec = 2;
        tile0[i] = at;
        at += (a.n + tile - 1) / tile;
    }
    tile0[tensors] = at;
    *tiles = at;
    return MOE_OK;
}

extern "C" moe_status_t adamw_step(void* plan, int tensors, int64_t tiles, int p_type, int g_type, int state_bits,
                                   const moe_adamw_opts_t* o, void* stream) {
    using namespace moe;
    using namespace moe::adamw;
    MOE_REQUIRE(plan && o && tensors >= 1 && tensors <= kMaxTensors && tiles >= 0, MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(type_ok(p_type) && type_ok(g_type) && (state_bits == 32 || state_bits == 8), MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(o->beta1 >= 0. && o->beta1 < 1. && o->beta2 >= 0. && o->beta2 < 1. && o->eps >= 0. &&
                    (o->step_dev || o->step >= 1),
                MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(al(plan, 16) && al(o->step_dev, 4) && al(o->lr_dev, 4) && al(o->grad_scale, 4), MOE_ERR_ALIGNMENT);
    MOE_REQUIRE(device_initialized(), MOE_ERR_NOT_INITIALIZED);
    const int sms = device_sm_count();
    MOE_REQUIRE(sms > 0, MOE_ERR_NOT_INITIALIZED);
    unsigned char* base = static_cast<unsigned char*>(plan);
    Params p{};
    p.ticket = reinterpret_cast<uint32_t*>(base);
    p.e = reinterpret_cast<const Entry*>(base + 16);
    p.tile0 = reinterpret_cast<const int64_t*>(base + tile_table_at(tensors));
    p.tensors = tensors;
    p.tiles = tiles;
    p.lr = (float)o->lr, p.b1 = (float)o->beta1, p.b2 = (float)o->beta2, p.eps = (float)o->eps;
    p.c1 = (float)(1. - o->beta1), p.c2 = (float)(1. - o->beta2);
    p.seed = o->seed;
    p.lr_dev = o->lr_dev, p.step_dev = o->step_dev, p.grad_scale = o->grad_scale;
    if (o->step_dev) {
        p.ln_b1 = (float)log(o->beta1), p.ln_b2 = (float)log(o->beta2);      // -inf at 0: 1 - 0^t = 1
    } else {
        p.inv_bc1 = (float)(1. / (1. - pow(o->beta1, (double)o->step)));
        p.inv_bc2 = (float)(1. / (1. - pow(o->beta2, (double)o->step)));
        p.key = mix(o->seed ^ mix((uint32_t)o->step));
    }
    if (tiles == 0 && !o->step_dev) return MOE_OK;
    cudaStream_t s = (cudaStream_t)stream;
    if (p_type == MOE_TYPE_F32 && g_type == MOE_TYPE_F32)
        launch<float, float>(state_bits, p, sms, s);
    else if (p_type == MOE_TYPE_F32)
        launch<float, __nv_bfloat16>(state_bits, p, sms, s);
    else if (g_type == MOE_TYPE_F32)
        launch<__nv_bfloat16, float>(state_bits, p, sms, s);
    else
        launch<__nv_bfloat16, __nv_bfloat16>(state_bits, p, sms, s);
    MOE_CHECK_LAUNCH();
    return MOE_OK;
}
