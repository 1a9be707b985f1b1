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
// The pass is bound by its traffic: p, g, m, v read and p, m, v written once.
#include <math.h>

#include <algorithm>

#include "common.cuh"

namespace moe {
namespace adamw {

constexpr int kBlock = 256;                 // elements per 8-bit scale: one warp, 8 per lane
constexpr int kThreads = 256;
constexpr int kTile = kThreads * 8;         // elements per CTA and iteration
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
    int vec;        // every address allows 8-element vectors
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

// 32 mixed bits of 32: two rounds of xor-shift and an odd multiplier.
__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
    x = (x ^ (x >> 16)) * 0x9E3779B1u;
    x = (x ^ (x >> 15)) * 0x85EBCA77u;
    return x ^ (x >> 16);
}

__device__ __forceinline__ void load8(const float* p, float* f) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* f) { unpack8(*reinterpret_cast<const uint4*>(p), f); }
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

// E4M3 codes <-> fp32.  Two codes to two fp16 and on; exact.
__device__ __forceinline__ void e4m3x2_to_f32(uint32_t two, float& lo, float& hi) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h));
}
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
    for (int i = 0; i < 4; ++i) e4m3x2_to_f32((w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu, f[2 * i], f[2 * i + 1]);
}
__device__ __forceinline__ void store_codes(uint8_t* p, int n, bool vec, const float* f) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        w[i] = cvt_e4m3x2(f[4 * i], f[4 * i + 1]) | (cvt_e4m3x2(f[4 * i + 2], f[4 * i + 3]) << 16);
    if (vec && n >= 8) {
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
    }
}

// 0 <= x (up to about 448) to a multiple of its E4M3 step, down or up as the
// 16 dither bits say.  Steps: 2^(exponent - 3), 2^-9 below 2^-6.
__device__ __forceinline__ float dithered(float x, uint32_t bits16) {
    const int e = max((int)(__float_as_uint(x) >> 23) - 127 - 3, -9);
    const float step = __uint_as_float((uint32_t)(e + 127) << 23), inv = __uint_as_float((uint32_t)(127 - e) << 23);
    const float k = floorf(fmaf(x, inv, (float)bits16 * (1.f / 65536.f)));
    return fminf(k * step, 448.f);
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
    scale = some ? __fdiv_rn(top, 448.f) : 0.f;
    inv = some ? __fdiv_rn(448.f, top) : 0.f;
}

template <typename PT, typename GT, int BITS>
__global__ void __launch_bounds__(kThreads) k_adamw(const Params p) {
    __shared__ float s_h[4];
    __shared__ uint32_t s_key;
    __shared__ int s_last;
    if (threadIdx.x == 0) {
        float i1 = p.inv_bc1, i2 = p.inv_bc2;
        uint32_t key = p.key;
        if (p.step_dev != nullptr) {
            const int t = *(volatile int32_t*)p.step_dev + 1;
            i1 = 1.f / -expm1f((float)t * p.ln_b1);
            i2 = 1.f / -expm1f((float)t * p.ln_b2);
            key = mix(p.seed ^ mix((uint32_t)t));
        }
        s_h[0] = i1, s_h[1] = i2;
        s_h[2] = p.lr_dev ? *p.lr_dev : p.lr;
        s_h[3] = p.grad_scale ? *p.grad_scale : 1.f;
        s_key = key;
    }
    __syncthreads();
    const float lr = s_h[2], gs = s_h[3], inv_bc2 = s_h[1], lr1 = lr * s_h[0];
    const uint32_t key = s_key;
    const bool skip = !(fabsf(gs) <= 3.402823466e38f);      // NaN or infinite: the step is not taken
    // the CTA's share of the tiles, in order
    const int64_t t0 = p.tiles * blockIdx.x / gridDim.x, t1 = p.tiles * (blockIdx.x + 1) / gridDim.x;
    int k = 0;
    {
        int hi = p.tensors - 1;      // the last tensor that starts at or before t0
        while (k < hi) {
            const int mid = (k + hi + 1) >> 1;
            if (p.tile0[mid] <= t0) k = mid;
            else hi = mid - 1;
        }
    }
    int64_t first = p.tile0[k], next = p.tile0[k + 1];
    Entry e = p.e[k];
    for (int64_t t = t0; t < t1 && !skip; ++t) {
        while (t >= next) {
            first = next;
            next = p.tile0[++k + 1];
            e = p.e[k];
        }
        const int64_t at = (t - first) * kTile + 8 * (int)threadIdx.x;
        const int64_t left = e.n - at;
        const int n = left >= 8 ? 8 : (left > 0 ? (int)left : 0);
        if (BITS == 32 && n == 0) continue;      // 8 bits: the warp works together
        const bool vec = e.vec != 0;
        float g[8], w[8], m[8], v[8];
        load(static_cast<const GT*>(e.g) + at, n, vec, g);
        load(static_cast<PT*>(e.p) + at, n, vec, w);
        if (BITS == 32) {
            load(static_cast<float*>(e.m) + at, n, vec, m);
            load(static_cast<float*>(e.v) + at, n, vec, v);
        } else {
            load_codes(static_cast<uint8_t*>(e.m) + at, n, vec, m);
            load_codes(static_cast<uint8_t*>(e.v) + at, n, vec, v);
            // the warp's block: its first element exists or the whole warp is past the end
            const int64_t b = (at - 8 * (int)(threadIdx.x & 31)) / kBlock;
            const bool some = b * kBlock < e.n;
            const float sm = some ? e.ms[b] : 0.f, sv = some ? e.vs[b] : 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                m[i] *= sm;
                v[i] *= sv;
                v[i] *= v[i];
            }
        }
        const float decay = 1.f - lr * e.wd;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float gi = g[i] * gs;
            m[i] = p.b1 * m[i] + p.c1 * gi;
            v[i] = p.b2 * v[i] + p.c2 * gi * gi;
            w[i] = w[i] * decay - __fdividef(lr1 * m[i], sqrtf(v[i] * inv_bc2) + p.eps);
        }
        store(static_cast<PT*>(e.p) + at, n, vec, w);
        if (e.copy != nullptr) store(e.copy + at, n, vec, w);
        if (BITS == 32) {
            store(static_cast<float*>(e.m) + at, n, vec, m);
            store(static_cast<float*>(e.v) + at, n, vec, v);
        } else {
            const int64_t b = (at - 8 * (int)(threadIdx.x & 31)) / kBlock;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                m[i] = i < n ? m[i] : 0.f;
                v[i] = i < n ? sqrtf(v[i]) : 0.f;
            }
            float sm, im, sv, iv;
            block_scale(block_top(m), sm, im);
            block_scale(block_top(v), sv, iv);
            const uint64_t c = (uint64_t)(e.rng + at);     // blocks start at multiples of 256 of the counter
            const uint32_t hi = mix((uint32_t)(c >> 32) ^ key);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t bits = mix((uint32_t)c + (uint32_t)i + hi);
                m[i] = copysignf(dithered(fabsf(m[i]) * im, bits & 0xFFFFu), m[i]);
                const float q = dithered(v[i] * iv, bits >> 16);
                v[i] = v[i] > 0.f && q == 0.f ? 0.001953125f : q;
            }
            store_codes(static_cast<uint8_t*>(e.m) + at, n, vec, m);
            store_codes(static_cast<uint8_t*>(e.v) + at, n, vec, v);
            if ((threadIdx.x & 31) == 0 && n > 0) {
                e.ms[b] = sm;
                e.vs[b] = sv;
            }
        }
    }
    if (p.step_dev != nullptr) {
        // the last CTA to come here counts the step: every CTA has read it by then
        if (threadIdx.x == 0) {
            __threadfence();
            s_last = atomicAdd(p.ticket, 1u) == gridDim.x - 1;
            if (s_last) {
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

template <typename PT, typename GT>
static void launch(int bits, int grid, const Params& p, cudaStream_t s) {
    if (bits == 32)
        k_adamw<PT, GT, 32><<<grid, kThreads, 0, s>>>(p);
    else
        k_adamw<PT, GT, 8><<<grid, kThreads, 0, s>>>(p);
}

}  // namespace adamw
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
        tile0[i] = at;
        at += (a.n + kTile - 1) / kTile;
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
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(tiles, (int64_t)sms * 8));
    cudaStream_t s = (cudaStream_t)stream;
    if (p_type == MOE_TYPE_F32 && g_type == MOE_TYPE_F32)
        launch<float, float>(state_bits, grid, p, s);
    else if (p_type == MOE_TYPE_F32)
        launch<float, __nv_bfloat16>(state_bits, grid, p, s);
    else if (g_type == MOE_TYPE_F32)
        launch<__nv_bfloat16, float>(state_bits, grid, p, s);
    else
        launch<__nv_bfloat16, __nv_bfloat16>(state_bits, grid, p, s);
    MOE_CHECK_LAUNCH();
    return MOE_OK;
}
