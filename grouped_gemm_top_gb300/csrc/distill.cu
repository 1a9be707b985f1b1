// Distillation from a teacher's top logits: the loss of every token, the
// gradient of the student's logits, or both from one read of the logits.
//
// With x a row of V logits, e_i = exp((x_i - max x) / tau), s = sum e_i, and
// the teacher's probabilities p_j of the tokens i_j it kept,
//   loss = tau^2 (sum_j p_j (log p_j - log q_{i_j}) + rest term),   q = e / s
//   dx_i = dloss tau (mass e_i / s - sum_{j: i_j = i} p_j)
// p is the softmax of the kept logits / tau (mass 1), or, when the teacher's
// log-sum-exp over its whole vocabulary is known, exp(t / tau - lse); then
// rest = 1 - sum p is held against the student's other tokens together, whose
// sum is s_rest: loss gains rest (log rest - log(s_rest / s)) and the other
// tokens' dx lose dloss tau rest e_i / s_rest.  s_rest is summed over those
// tokens themselves (a bit per token says which were kept): as s - sum of the
// kept it would be lost where the student is sure of them.  Its terms are relative to
// the others' own maximum: relative to max x they would all be zero 87 tau below it.
//
// Loss and gradient together read the logits once: a row's parts lie in the
// shared memory of a cluster's CTAs, whose maxima and sums are exchanged
// through distributed shared memory; 4 bytes an element of bf16 logits instead
// of 6 in two calls.  The loss alone and the gradient alone keep nothing, and
// stream whole rows, one CTA each, through a ring; there a cluster shares a row
// only when rows are few.
// Warps 0 .. W - 1 go over the logits.  A thread loads the 16-byte units that it
// works on itself (asynchronous copies to shared memory, in groups; rows may
// start at any element, what is read of the neighbouring rows is not used) and
// sends for the next ones as it is done with some, so that nobody waits for
// another's loads.  (Bulk copies by one thread were no faster.)  Warp W works on
// the teacher's tokens a row ahead.  All waits are bounded.
// Bound by the memory for large vocabularies (a plain copy 6.8 TB/s): 8,192 x 129,280 bf16
// loss 322 us (6.6 TB/s), loss and gradient 733 us (5.8; 62 % of the issue slots, the rest of
// the gap is the chain of a row's sums through the cluster, three CTAs an SM in turn),
// gradient of 2,048 rows 172 us (6.2), loss of 4,099 x 50,257 fp32 137 us (6.0); by that chain
// for small ones; 5.5 us for 4 x 32,000.
#include <algorithm>

#include "gemm_common.cuh"

namespace moe {
namespace distill {

using namespace gg;

constexpr int MAX_K = 1024;              // tokens of the teacher
constexpr int MAX_C = 8;                 // CTAs of a cluster
constexpr int CHUNKS = 4;                // groups of copies on their way: of the part, or the ring's
constexpr int MAX_PART = 11264;          // 16-byte units of a part
constexpr float kLog2e = 1.4426950408889634f;
enum { FWD = 1, BWD = 2, BOTH = 3 };

struct Params {
    const void* x;
    int64_t ldx;
    void* dx;
    int64_t lddx;
    const int32_t* idx;
    int64_t ldi;
    const void* t;
    int64_t ldt;
    int t_f32;
    const float* lse;         // teacher's, or NULL
    const float* dloss;
    float* loss;
    float* stats;             // [M, 3]: see put_stats; BWD: read
    int64_t M;
    int V, k;
    float tau, inv_tau, c;    // c = log2(e) / tau
    int part, chunk, held;    // 16-byte units of a CTA's part, of a chunk, in shared memory
    int32_t* err;
    uint64_t timeout_ns;
};

// what a warp knows of a row's teacher, per buffer
struct Teacher {
    float mass, rest, p_sum;        // mass = sum p + rest
    float fit, x_ref, t_lse;        // sum p ((t - max t) - (x - x_ref) / tau); log-sum-exp of t - max t
    float again;                    // tokens of this CTA's part that occur several times: what the loss gains, P log P - sum p log p
    float top_max, top_sum;         // of the kept tokens in this CTA's part
    float dloss, stats[3];          // of the row (BWD: what the forward pass kept)
    int some;                       // 0: no teacher, loss and gradient are zero
};

// Shared memory: the part or the ring of its chunks, then (two buffers each) a
// byte per 16-byte unit of the part, and of each of the teacher's tokens its column
// (bit 31: counted with an earlier one; -1: none), its probability and the
// student's logit.
struct Smem {
    uint8_t* rows;
    int held, part, k;      // units in shared memory, of the part
    __device__ __forceinline__ uint8_t* bits(int b) const;
    __device__ __forceinline__ int* col(int b) const;
    __device__ __forceinline__ float* p(int b) const { return reinterpret_cast<float*>(col(b)) + k; }
    __device__ __forceinline__ float* x(int b) const { return p(b) + k; }
    __device__ __forceinline__ uint8_t* fixed() const { return reinterpret_cast<uint8_t*>(col(2)); }
};
struct Fixed {
    unsigned long long bar[6];
    float4 mail[2][MAX_C];          // of the cluster's parts, see Sums: m, s, again, or (TAIL) kept m, s, the others' m, s
    float again[2][MAX_C];          // TAIL: the first CTA's, of the others' parts
    float2 warp_part[2][8];
    Teacher teacher[2];
    int abort_flag;
};

__host__ __device__ inline int bits_bytes(int part) { return (part + 15) / 16 * 16; }
__host__ __device__ inline size_t smem_bytes(int held, int part, int k) {
    return (size_t)held * 16 + 2 * (bits_bytes(part) + 12 * (size_t)((k + 3) / 4 * 4)) + sizeof(Fixed);
}
__device__ __forceinline__ uint8_t* Smem::bits(int b) const { return rows + 16 * held + b * bits_bytes(part); }
__device__ __forceinline__ int* Smem::col(int b) const { return reinterpret_cast<int*>(bits(2)) + 3 * b * k; }
static_assert(MAX_PART * 18 + 24 * MAX_K + sizeof(Fixed) <= 232448 && MAX_PART % 16 == 0, "shared memory budget");

__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
    return n;
}
// this thread's copies have landed, all but the last n groups
__device__ __forceinline__ void wait_group(int n) {
    if (n == 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
    else if (n == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else if (n == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else asm volatile("cp.async.wait_group 3;" ::: "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// exp of (x - m) / tau; the difference first, so that rows of the type's
// lowest value do not overflow
__device__ __forceinline__ float e_of(float x, float m, float c) { return ex2((x - m) * c); }
__device__ __forceinline__ float finite_max(float m) { return m == -INFINITY ? 0.f : m; }

// Two fp32 at a time (the FMA pipe's packed form).
typedef unsigned long long f2;
__device__ __forceinline__ f2 pack(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack(f2 v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// e_of of two, for -m and c twice
__device__ __forceinline__ f2 e_of2(f2 x, f2 neg_m, f2 c) {
    float a, b;
    unpack(mul2(add2(x, neg_m), c), a, b);
    return pack(ex2(a), ex2(b));
}

// 16 bytes of logits, E of them: as they lie in memory, as pairs of fp32, their maximum.
template <typename T>
struct Unit;
template <>
struct Unit<__nv_bfloat16> {
    static constexpr int E = 8;
    static __device__ __forceinline__ void pairs(const uint4& v, f2* f) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    }
    static __device__ __forceinline__ __nv_bfloat162 two(uint32_t w) { return *reinterpret_cast<__nv_bfloat162*>(&w); }
    template <int N>
    static __device__ __forceinline__ float max_of(const uint4* v) {
        __nv_bfloat162 m = __hmax2(__hmax2(two(v[0].x), two(v[0].y)), __hmax2(two(v[0].z), two(v[0].w)));
#pragma unroll
        for (int n = 1; n < N; ++n)
            m = __hmax2(m, __hmax2(__hmax2(two(v[n].x), two(v[n].y)), __hmax2(two(v[n].z), two(v[n].w))));
        return fmaxf(__low2float(m), __high2float(m));
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* f) {
        *reinterpret_cast<uint4*>(p) = pack8(f);
    }
    static __device__ __forceinline__ float one(const void* p, int64_t i) {
        return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    }
    static __device__ __forceinline__ __nv_bfloat16 to(float f) { return __float2bfloat16_rn(f); }
};
template <>
struct Unit<float> {
    static constexpr int E = 4;
    static __device__ __forceinline__ void pairs(const uint4& v, f2* f) {
        f[0] = pack(__uint_as_float(v.x), __uint_as_float(v.y)), f[1] = pack(__uint_as_float(v.z), __uint_as_float(v.w));
    }
    template <int N>
    static __device__ __forceinline__ float max_of(const uint4* v) {
        float m = -INFINITY;
#pragma unroll
        for (int n = 0; n < N; ++n)
            m = fmaxf(fmaxf(fmaxf(m, __uint_as_float(v[n].x)), fmaxf(__uint_as_float(v[n].y), __uint_as_float(v[n].z))),
                      __uint_as_float(v[n].w));
        return m;
    }
    static __device__ __forceinline__ void store(float* p, const float* f) {
        *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    }
    static __device__ __forceinline__ float one(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }
    static __device__ __forceinline__ float to(float f) { return f; }
};
// the elements that `out` (a bit each) names become -inf
template <int E>
__device__ __forceinline__ void leave_out(uint4& v, uint32_t out) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (E == 4) {
            if (out >> i & 1) w[i] = 0xFF800000u;
        } else {
            if (out >> (2 * i) & 1) w[i] = (w[i] & 0xFFFF0000u) | 0xFF80u;
            if (out >> (2 * i + 1) & 1) w[i] = (w[i] & 0xFFFFu) | 0xFF800000u;
        }
    }
    v = make_uint4(w[0], w[1], w[2], w[3]);
}

// A thread's running maximum and sum of exponentials (two accumulators of
// two), N units at a time.
struct Sum {
    float m = -INFINITY;
    f2 s[2] = {0ull, 0ull};
    template <typename T, int N>
    __device__ __forceinline__ void add(const uint4* v, float c) {
        constexpr int E = Unit<T>::E;
        const float um = Unit<T>::template max_of<N>(v);
        if (um > m) {
            const float r = e_of(m, um, c);
            s[0] = mul2(s[0], pack(r, r)), s[1] = mul2(s[1], pack(r, r));
            m = um;
        }
        const float ref = -finite_max(m);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            f2 f[E / 2];
            Unit<T>::pairs(v[n], f);
#pragma unroll
            for (int i = 0; i < E / 2; ++i) s[i & 1] = add2(s[i & 1], e_of2(f[i], pack(ref, ref), pack(c, c)));
        }
    }
    __device__ __forceinline__ float total() const {
        float a, b;
        unpack(add2(s[0], s[1]), a, b);
        return a + b;
    }
};

// Where a row's part lies: its units [g0, g0 + n) counted from the row's first
// 16-byte boundary; element e of unit g is column g E + e - head.
struct Part {
    int head, g0, n;
    int lo, hi;        // the row's elements among the part's
    int u0, u1;        // units that are the row's entirely
};
// the elements of unit u that are not the row's, a bit each
template <int E>
__device__ __forceinline__ uint32_t outside(const Part& pt, int u) {
    const int a = pt.lo - u * E, b = pt.hi - u * E;
    uint32_t out = 0;
    if (a > 0) out |= (1u << a) - 1u;             // a < E: the row begins in its first unit
    if (b < E) out |= ~((1u << b) - 1u);          // b > 0: it ends in its last one
    return out & ((1u << E) - 1u);
}
template <typename T>
__device__ __forceinline__ Part part_of(const Params& p, int64_t row, uint32_t rank) {
    constexpr int E = Unit<T>::E;
    Part r;
    const uintptr_t at = reinterpret_cast<uintptr_t>(static_cast<const T*>(p.x) + row * p.ldx);
    r.head = (int)(at & 15) / (int)sizeof(T);
    const int units = (r.head + p.V + E - 1) / E;
    r.g0 = (int)rank * p.part;
    r.n = max(0, min(p.part, units - r.g0));
    r.lo = r.head - r.g0 * E;
    r.hi = r.head + p.V - r.g0 * E;
    r.u0 = r.lo > 0 ? 1 : 0;
    r.u1 = r.n * E > r.hi ? r.n - 1 : r.n;
    return r;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}
// two at a time take no longer than one
__device__ __forceinline__ void warp_max2(float& a, float& b) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float x = __shfl_xor_sync(0xFFFFFFFFu, a, o), y = __shfl_xor_sync(0xFFFFFFFFu, b, o);
        a = fmaxf(a, x), b = fmaxf(b, y);
    }
}
__device__ __forceinline__ void warp_sum2(float& a, float& b) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float x = __shfl_xor_sync(0xFFFFFFFFu, a, o), y = __shfl_xor_sync(0xFFFFFFFFu, b, o);
        a += x, b += y;
    }
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// What the teacher's warp loads before a row's turn comes: 128 of its tokens,
// four a lane, and the row's own numbers.
struct Ahead {
    int i[4];
    uint32_t t[4];
    float lse, dloss, stats[3];
};
template <int MODE, bool TAIL>
__device__ __forceinline__ void load_tokens(const Params& p, int64_t row, int j0, int lane, Ahead& a) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int j = j0 + 32 * q + lane;
        a.i[q] = -1, a.t[q] = 0u;
        if (row < p.M && j < p.k) {
            const int64_t at = row * p.ldt + j;
            a.i[q] = p.idx[row * p.ldi + j];
            a.t[q] = p.t_f32 ? static_cast<const uint32_t*>(p.t)[at] : static_cast<const uint16_t*>(p.t)[at];
        }
    }
    if (row < p.M && j0 == 0) {
        if (TAIL) a.lse = p.lse[row];
        if (MODE != FWD) a.dloss = p.dloss[row];
        if (MODE == BWD)
            for (int i = 0; i < 3; ++i) a.stats[i] = p.stats[3 * row + i];
    }
}
// of the tokens in this CTA's part; the first CTA, which works out the loss, of all
template <typename T, int MODE>
__device__ __forceinline__ void load_logits(const Params& p, int64_t row, uint32_t rank, const Ahead& a, float* x) {
    const Part pt = part_of<T>(p, row, rank);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int i = a.i[q], g = (i + pt.head) / Unit<T>::E - pt.g0;
        x[q] = 0.f;
        if (i >= 0 && i < p.V && row < p.M && ((g >= 0 && g < pt.n) || (rank == 0 && MODE != BWD)))
            x[q] = Unit<T>::one(p.x, row * p.ldx + i);
    }
}

// Whether the teacher's tokens set bits: where only repeated ones are looked for, up to 32
// compare themselves with one another (16,384 x 4,096, loss alone: 43.6 us, 44.6 by bits).
template <int MODE, bool TAIL>
__device__ __forceinline__ bool by_bits(const Params& p) {
    return TAIL || MODE != FWD || p.k > 32;
}
__device__ __forceinline__ float p_log_p(float p) { return p == 0.f ? 0.f : p * logf(p); }

// The teacher's row (one warp): probabilities, what the loss needs of them,
// and, of the tokens in this CTA's part, their bits, sums and logits.
template <typename T, int MODE, bool TAIL>
__device__ __forceinline__ void teacher_row(const Params& p, const Smem& sm, Teacher& out, int b, int64_t row,
                                            int64_t next, uint32_t rank, int lane, Ahead& ah) {
    constexpr int E = Unit<T>::E;
    const Part pt = part_of<T>(p, row, rank);
    int* col = sm.col(b);
    float *pr = sm.p(b), *xs = sm.x(b);
    uint32_t* words = reinterpret_cast<uint32_t*>(sm.bits(b));
    const float inv_tau = p.inv_tau;
    const bool bits = by_bits<MODE, TAIL>(p);
    bool any = false, dup = false;
    float t_max = -INFINITY, x_max = -INFINITY;
    for (int j0 = 0; j0 < p.k; j0 += 128) {
        float x[4];
        if (j0 > 0) load_tokens<MODE, TAIL>(p, row, j0, lane, ah);
        load_logits<T, MODE>(p, row, rank, ah, x);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int j = j0 + 32 * q + lane, i = ah.i[q];
            if (j >= p.k) continue;
            const bool ok = i >= 0 && i < p.V;
            if (i >= p.V) set_err(p.err, MOE_ERR_BAD_INDEX);
            const float t = ok ? __uint_as_float(p.t_f32 ? ah.t[q] : ah.t[q] << 16) * inv_tau : -INFINITY;
            if (ok) {
                any = true;
                const int u = i + pt.head, g = u / E - pt.g0;
                if (bits && g >= 0 && g < pt.n) {
                    const uint32_t bit = 1u << (8 * (g & 3) + u % E);
                    dup |= (atomicOr(words + (g >> 2), bit) & bit) != 0;
                }
                if (t > -INFINITY) x_max = fmaxf(x_max, x[q]);
            }
            col[j] = ok ? i : -1;
            pr[j] = t;
            xs[j] = x[q];
            t_max = fmaxf(t_max, t);
        }
    }
    if (!bits) {
        const int i = ah.i[0];
        dup = __popc(__match_any_sync(0xFFFFFFFFu, i >= 0 && i < p.V ? i : -1 - lane)) > 1;
    }
    if (lane == 0 && MODE != FWD) {
        out.dloss = ah.dloss;
        for (int i = 0; i < 3; ++i) out.stats[i] = ah.stats[i];
    }
    const float row_lse = ah.lse;
    load_tokens<MODE, TAIL>(p, next, 0, lane, ah);
    any = __any_sync(0xFFFFFFFFu, any);
    dup = __any_sync(0xFFFFFFFFu, dup);
    warp_max2(t_max, x_max);
    const float t_ref = finite_max(t_max), x_ref = finite_max(x_max);
    __syncwarp();
    float sum = 0.f;
    if (!TAIL) {
        for (int j = lane; j < p.k; j += 32)
            if (col[j] >= 0) sum += expf(pr[j] - t_ref);
        sum = warp_sum(sum);
    }
    const float t_lse = TAIL ? row_lse - t_ref : logf(sum), inv = 1.f / sum;
    // a NaN among the teacher's logits is a teacher: it shows in the loss
    const bool some = any && (TAIL || sum != 0.f);
    float mass = 0.f, fit = 0.f;
    for (int j = lane; j < p.k; j += 32) {
        float q = 0.f;
        if (some && col[j] >= 0) {
            const float t = pr[j] - t_ref;
            q = TAIL ? expf(t - t_lse) : expf(t) * inv;
            if (q != 0.f) fit += q * (t - (xs[j] - x_ref) * inv_tau);
        }
        pr[j] = q;
        mass += q;
    }
    warp_sum2(mass, fit);
    __syncwarp();
    float again = 0.f;
    if (dup) {      // the first of several holds the sum of their probabilities
        for (int j = lane; j < p.k; j += 32) {
            const int cj = col[j];
            if (cj == -1) continue;
            bool first = true;
            int others = 0;
            float q = pr[j], apart = MODE != BWD ? p_log_p(q) : 0.f;
            for (int i = 0; i < p.k; ++i) {
                if (i == j || col[i] == -1 || (col[i] & 0x7FFFFFFF) != cj) continue;
                if (i < j) {
                    first = false;
                } else {
                    q += pr[i], ++others;
                    if (MODE != BWD) apart += p_log_p(pr[i]);
                }
            }
            if (first) {
                pr[j] = q;
                const int g = (cj + pt.head) / E - pt.g0;
                if (MODE != BWD && others > 0 && g >= 0 && g < pt.n) again += p_log_p(q) - apart;
            } else {
                col[j] = cj | (int)0x80000000;
            }
        }
        if (MODE != BWD) again = warp_sum(again);
        __syncwarp();
    }
    float top_max = -INFINITY, top_sum = 0.f;
    if (TAIL && MODE != BWD) {
        for (int pass = 0; pass < 2; ++pass) {
            for (int j = lane; j < p.k; j += 32) {
                const int g = (col[j] + pt.head) / E - pt.g0;
                if (col[j] < 0 || g < 0 || g >= pt.n) continue;
                if (pass == 0) top_max = fmaxf(top_max, xs[j]);
                else top_sum += e_of(xs[j], finite_max(top_max), p.c);
            }
            if (pass == 0) top_max = warp_max(top_max);
            else top_sum = warp_sum(top_sum);
        }
    }
    if (lane == 0) {
        out.rest = TAIL && some ? fmaxf(1.f - mass, 0.f) : 0.f;
        out.p_sum = mass;
        out.mass = mass + out.rest;
        out.fit = fit, out.x_ref = x_ref, out.t_lse = t_lse, out.again = again;
        out.top_max = top_max, out.top_sum = top_sum;
        out.some = some;
    }
    __syncwarp();
}
// the bits of the row that this buffer held
template <typename T>
__device__ __forceinline__ void clear_bits(const Params& p, const Smem& sm, int b, const Part& pt, int lane) {
    constexpr int E = Unit<T>::E;
    for (int j = lane; j < p.k; j += 32) {
        const int cj = sm.col(b)[j];
        if (cj == -1) continue;
        const int g = ((cj & 0x7FFFFFFF) + pt.head) / E - pt.g0;
        if (g >= 0 && g < pt.n) reinterpret_cast<uint32_t*>(sm.bits(b))[g >> 2] = 0u;
    }
    __syncwarp();
}

// Sums over a row of exp((x - maximum) / tau): over all tokens, and over those that were
// not kept with a maximum of their own (TAIL).
struct Sums {
    float m, s, m_rest, s_rest;
};
// the sums from those of the kept tokens and of the others
__device__ __forceinline__ Sums joined(float m_top, float s_top, float m_rest, float s_rest, float c) {
    const float m = fmaxf(m_top, m_rest), ref = finite_max(m);
    return {m, s_top * e_of(m_top, ref, c) + s_rest * e_of(m_rest, ref, c), m_rest, s_rest};
}

// What the loss and the gradient go by.  Others whose largest logit lies more than 700 tau
// below max x count as none: a maximum of the type's lowest value is a mask.  From
// 50 tau on the student is `sure`: the others' gradient is then that of rest alone (what
// mass adds to it, q_rest / rest of it, is less than a rounding: V e^-50, and rest is at
// least 2^-24), taken relative to their own maximum, so that rest / s_rest does not
// overflow.
constexpr float kNone = -700.f * kLog2e, kSure = -50.f * kLog2e;
struct View {
    float m, s;               // maximum and sum, for the kept tokens (not sure: for all)
    float m_rest, s_rest;     // for the others; s_rest = 0: none; not sure: relative to m
    bool sure;
};
template <bool TAIL>
__device__ __forceinline__ View view_of(const Params& p, const Sums& r) {
    if (!TAIL) return {r.m, r.s, r.m, r.s, false};
    const float below = (r.m_rest - finite_max(r.m)) * p.c;
    if (below < kSure && below >= kNone) return {r.m, r.s, r.m_rest, r.s_rest, true};
    return {r.m, r.s, r.m, r.s_rest * ex2(below), false};
}
// The view in three numbers: m, s, s_rest, or, of a student who is sure, the kept
// tokens' log-sum-exp (tau of it, in the logits' scale), minus s_rest, m_rest.
__device__ __forceinline__ void put_stats(const Params& p, float* out, const View& v) {
    out[0] = v.sure ? v.m + p.tau * logf(v.s) : v.m;
    out[1] = v.sure ? -v.s_rest : v.s;
    out[2] = v.sure ? v.m_rest : v.s_rest;
}
template <bool TAIL>
__device__ __forceinline__ View view_of_stats(const float* st) {
    if (TAIL && st[1] < 0.f) return {st[0], 1.f, st[2], -st[1], true};
    return {st[0], st[1], st[0], st[2], false};
}

// The row's loss, and what the backward pass needs.
template <bool TAIL>
__device__ __forceinline__ void write_loss(const Params& p, int64_t row, const Teacher& te, const View& v,
                                           float again) {
    if (p.stats) put_stats(p, p.stats + 3 * row, v);
    if (p.loss) {
        const float log_s = logf(v.s);
        float loss = te.fit + again + te.p_sum * ((finite_max(v.m) - te.x_ref) * p.inv_tau + log_s - te.t_lse);
        if (TAIL && te.rest > 0.f && v.s_rest > 0.f) {
            const float log_rest = (v.sure ? (v.m_rest - v.m) * p.inv_tau : 0.f) + logf(v.s_rest) - log_s;      // log q_rest
            loss += te.rest * (logf(te.rest) - log_rest);
        }
        p.loss[row] = te.some ? loss * p.tau * p.tau : 0.f;
    }
}

// The row's gradient: e times a factor, one for the kept tokens and one for the
// others, and the kept ones' probabilities.
template <typename T, bool TAIL>
struct Slope {
    static constexpr int E = Unit<T>::E;
    float g, f_top, ref, c;
    f2 neg2, f2_all, c2;
    bool zero, vec;
    T* dx;      // element 0 of the part
    __device__ __forceinline__ Slope(const Params& p, const Part& pt, const Teacher& te, int64_t row, const View& v) {
        g = te.dloss * p.tau;
        zero = !te.some || g == 0.f;
        const bool with_rest = TAIL && te.rest > 0.f && v.s_rest > 0.f;
        const float mass = with_rest ? te.mass : te.p_sum;
        f_top = g * (mass / v.s);
        const bool alone = with_rest && v.sure;      // the others have rest alone
        const float f_all = with_rest ? g * ((alone ? 0.f : mass / v.s) - te.rest / v.s_rest) : f_top;
        ref = finite_max(v.m), c = p.c;
        const float ref_all = alone ? v.m_rest : ref;
        neg2 = pack(-ref_all, -ref_all), f2_all = pack(f_all, f_all), c2 = pack(c, c);
        dx = static_cast<T*>(p.dx) + row * p.lddx - pt.head + (int64_t)pt.g0 * E;
        vec = (reinterpret_cast<uintptr_t>(dx) & 15) == 0;
    }
    __device__ __forceinline__ void unit(const uint8_t* x, float* d) const {
        f2 f[E / 2];
        Unit<T>::pairs(*reinterpret_cast<const uint4*>(x), f);
#pragma unroll
        for (int i = 0; i < E / 2; ++i) unpack(mul2(e_of2(f[i], neg2, c2), f2_all), d[2 * i], d[2 * i + 1]);
    }
    // units u, u + step, .. of `rows` (unit 0 of the part at rows) before u1
    __device__ __forceinline__ void units(const Part& pt, const uint8_t* rows, int u, int u1, int step) const {
        if (vec && !zero) {
#pragma unroll 2
            for (; u < min(u1, pt.u1); u += step) {
                if (u < pt.u0) break;
                float d[E];
                unit(rows + 16 * u, d);
                Unit<T>::store(dx + u * E, d);
            }
        }
        // the row's ends, and rows that do not lie as the logits do
        for (; u < u1; u += step) {
            float d[E] = {};
            if (!zero) unit(rows + 16 * u, d);
            if (vec && u >= pt.u0 && u < pt.u1) {
                Unit<T>::store(dx + u * E, d);
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (u * E + e >= pt.lo && u * E + e < pt.hi) dx[u * E + e] = Unit<T>::to(d[e]);
            }
        }
    }
    // the kept tokens first, first + step, .., over what units() stored there
    __device__ __forceinline__ void kept(const Params& p, const Part& pt, const Smem& sm, int b, int first, int step) const {
        if (zero) return;
        for (int j = first; j < p.k; j += step) {
            const int cj = sm.col(b)[j];
            const int u = cj + pt.lo;      // element of the part
            if (cj >= 0 && u >= 0 && u < pt.n * E)
                dx[u] = Unit<T>::to(e_of(sm.x(b)[j], ref, c) * f_top - g * sm.p(b)[j]);
        }
    }
};

// T: logits; W warps go over them.
template <typename T, int MODE, bool TAIL, int W>
__global__ void __launch_bounds__(32 * W + 32, W == 8 ? 3 : 10) k_distill(const Params p) {
    constexpr int E = Unit<T>::E;
    extern __shared__ __align__(16) uint8_t smem[];
    const Smem sm{smem, p.held, p.part, (p.k + 3) / 4 * 4};
    Fixed& fx = *reinterpret_cast<Fixed*>(sm.fixed());
    const uint32_t bar0 = smem_u32(&fx.bar[0]);
    auto tfull = [&](int i) { return bar0 + 8u * i; };
    auto tempty = [&](int i) { return bar0 + 8u * (2 + i); };
    auto xbar = [&](int i) { return bar0 + 8u * (4 + i); };
    volatile int* abort_flag = &fx.abort_flag;
    const uint32_t C = cluster_size(), rank = C > 1 ? cluster_ctarank() : 0u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) mbar_init(tfull(i), 1), mbar_init(tempty(i), MODE == FWD ? 1 : W), mbar_init(xbar(i), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fx.abort_flag = 0;
    }
    __syncthreads();
    if (C > 1) cluster_sync();      // the peers' barriers are initialised
    wait_for_previous_kernels();
    const int64_t row0 = blockIdx.x / C, step = gridDim.x / C;

    // the row's maximum and sums from the parts'
    auto gather_mail = [&](int b) {
        float m = -INFINITY, m_rest = -INFINITY, s = 0.f, s_rest = 0.f;
        for (int i = 0; i < (int)C; ++i) {
            m = fmaxf(m, fx.mail[b][i].x);
            if (TAIL) m_rest = fmaxf(m_rest, fx.mail[b][i].z);
        }
        const float ref = finite_max(m), ref_rest = finite_max(m_rest);
        for (int i = 0; i < (int)C; ++i) {
            const float4 v = fx.mail[b][i];
            s += v.y * e_of(v.x, ref, p.c);
            if (TAIL) s_rest += v.w * e_of(v.z, ref_rest, p.c);
        }
        return TAIL ? joined(m, s, m_rest, s_rest, p.c) : Sums{m, s, m, s};
    };
    auto gather_again = [&](int b) {
        float sum = fx.teacher[b].again;      // the first CTA's own
        for (int i = 1; i < (int)C; ++i) sum += TAIL ? fx.again[b][i] : fx.mail[b][i].z;
        return sum;
    };
    // (what peers sent is read behind a wait that acquires at cluster scope)
    auto wait_mail = [&](int b, uint32_t phase) { return mbar_wait_cluster(xbar(b), phase, p, abort_flag); };
    if (warp == W) {
        // ---------------------------------------------- teacher, a row ahead ----
        const bool bits = by_bits<MODE, TAIL>(p);
        if (bits) {
            for (int i = lane; i < bits_bytes(p.part) / 2; i += 32) reinterpret_cast<uint32_t*>(sm.bits(0))[i] = 0u;
            __syncwarp();
        }
        int it = 0;
        Ahead ah = {};
        load_tokens<MODE, TAIL>(p, row0, 0, lane, ah);
        for (int64_t row = row0; row < p.M; row += step, ++it) {
            const int b = it & 1;
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(tempty(b), (uint32_t)(it >> 1 & 1) ^ 1u, p, abort_flag))) break;
            if (it >= 2 && bits) clear_bits<T>(p, sm, b, part_of<T>(p, row - 2 * step, rank), lane);
            teacher_row<T, MODE, TAIL>(p, sm, fx.teacher[b], b, row, row + step, rank, lane, ah);
            if (lane == 0) mbar_arrive(tfull(b));
        }
    } else {
        // (a warp whose wait gave up goes on through the barriers, so that the
        // others do not wait for it, and touches nothing)
        int it = 0;
        bool ok = true;
        // this thread's units [c0, c0 + chunk) of a row's part go to `slot`, one group of copies
        auto send_for = [&](int64_t row, int c0, int slot) {
            if (row < p.M) {
                const Part pt = part_of<T>(p, row, rank);
                const uint8_t* src = reinterpret_cast<const uint8_t*>(static_cast<const T*>(p.x) + row * p.ldx) -
                                     pt.head * (int)sizeof(T) + (int64_t)(pt.g0 + c0) * 16;
                const int n = min(p.chunk, pt.n - c0);
                const uint32_t dst = smem_u32(sm.rows + 16 * slot);
#pragma unroll 4
                for (int u = (int)threadIdx.x; u < n; u += 32 * W)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + 16 * u), "l"(src + 16 * (int64_t)u)
                                 : "memory");
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        // STREAM: the ring's next chunk to send for, and its slot
        constexpr bool STREAM = MODE != BOTH;
        int64_t next_row = row0;
        int next_c0 = 0, next_slot = 0, slot = 0;
        auto send_next = [&] {
            send_for(next_row, next_c0, next_slot);
            next_slot = next_slot == (CHUNKS - 1) * p.chunk ? 0 : next_slot + p.chunk;
            next_c0 += p.chunk;
            if (next_c0 >= p.part) next_c0 = 0, next_row += step;
        };
        auto advance = [&] { slot = slot == (CHUNKS - 1) * p.chunk ? 0 : slot + p.chunk; };
        for (int ch = 0; ch < CHUNKS; ++ch) {
            if (STREAM) send_next();
            else send_for(row0, ch * p.chunk, ch * p.chunk);
        }
        for (int64_t row = row0; row < p.M; row += step, ++it) {
            const int b = it & 1;
            const uint32_t buf_phase = (uint32_t)(it >> 1 & 1);
            const Part pt = part_of<T>(p, row, rank);
            const Teacher& te = fx.teacher[b];
            // which of a unit's tokens were kept has to be known before the sums
            if (TAIL || MODE == BWD) ok = ok && mbar_wait(tfull(b), buf_phase, p, abort_flag);
            View view{0.f, 1.f, 0.f, 1.f, false};
            if constexpr (MODE != BWD) {
                // -------------------------------- maximum and sum ----
                const uint8_t* bits = sm.bits(b);
                Sum sum;
                for (int c0 = 0, ch = 0; STREAM ? c0 < p.part : ch < CHUNKS; c0 += p.chunk, ++ch) {
                    wait_group(STREAM ? CHUNKS - 1 : CHUNKS - 1 - ch);
                    const uint8_t* rows = STREAM ? sm.rows + 16 * (slot - c0) : sm.rows;
                    const int u1 = ok ? min(c0 + p.chunk, pt.n) : 0;
                    int u = c0 + (int)threadIdx.x;
                    constexpr int N = 4;
                    for (; u + (N - 1) * 32 * W < min(u1, pt.u1); u += N * 32 * W) {
                        uint4 v[N];
                        uint32_t kept[N], any = u < pt.u0;
#pragma unroll
                        for (int n = 0; n < N; ++n) {
                            v[n] = *reinterpret_cast<const uint4*>(rows + 16 * (u + n * 32 * W));
                            if (TAIL) any |= kept[n] = bits[u + n * 32 * W];
                        }
                        if (any) {
#pragma unroll
                            for (int n = 0; n < N; ++n) {
                                uint32_t out = n == 0 && u < pt.u0 ? outside<E>(pt, u) : 0u;
                                if (TAIL) out |= kept[n];
                                leave_out<E>(v[n], out);
                            }
                        }
                        sum.add<T, N>(v, p.c);
                    }
                    for (; u < u1; u += 32 * W) {
                        uint4 v = *reinterpret_cast<const uint4*>(rows + 16 * u);
                        uint32_t out = TAIL ? bits[u] : 0u;
                        if (u < pt.u0 || u >= pt.u1) out |= outside<E>(pt, u);
                        if (out) leave_out<E>(v, out);
                        sum.add<T, 1>(&v, p.c);
                    }
                    if (STREAM) {
                        send_next();
                        advance();
                    }
                }
                const float wm = warp_max(sum.m);
                const float ws = warp_sum(sum.total() * e_of(sum.m, finite_max(wm), p.c));
                if (lane == 0) fx.warp_part[it & 1][warp] = make_float2(wm, ws);
                // (also keeps the warps within a row of one another: warp_part has two rows)
                asm volatile("bar.sync 1, %0;" ::"n"(32 * W) : "memory");
                if (warp == 0) {      // this CTA's sums, to every CTA that goes on with them
                    if (!TAIL) ok = ok && mbar_wait(tfull(b), buf_phase, p, abort_flag);
                    const float2* part = fx.warp_part[it & 1];
                    float cm = -INFINITY, cs = 0.f;
#pragma unroll
                    for (int w = 0; w < W; ++w) cm = fmaxf(cm, part[w].x);
                    const float ref = finite_max(cm);
#pragma unroll
                    for (int w = 0; w < W; ++w) cs += part[w].y * e_of(part[w].x, ref, p.c);
                    const float4 v = TAIL ? make_float4(te.top_max, te.top_sum, cm, cs) : make_float4(cm, cs, te.again, 0.f);
                    // the bytes themselves count on the barriers: a release at cluster scope
                    // would wait for every store of this warp, 1 to 2 us a row
                    if (lane == 0 && ok) {
                        mbar_expect_tx(xbar(b), 16u * C + (TAIL && rank == 0 ? 4u * (C - 1u) : 0u));
                        if (TAIL && rank > 0) asm volatile(
                            "st.async.shared::cluster.mbarrier::complete_tx::bytes.f32 [%0], %1, [%2];" ::"r"(
                                mapa(smem_u32(&fx.again[b][rank]), 0u)),
                            "f"(te.again), "r"(mapa(xbar(b), 0u))
                            : "memory");
                    }
                    if (lane < (int)C && ok)
                        asm volatile(
                            "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                                mapa(smem_u32(&fx.mail[b][rank]), (uint32_t)lane)),
                            "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(mapa(xbar(b), (uint32_t)lane))
                            : "memory");
                }
                if (MODE == FWD) {      // the other warps go on to the next row
                    if (warp == 0) {
                        ok = __all_sync(0xFFFFFFFFu, ok && wait_mail(b, buf_phase));
                        if (rank == 0 && lane == 0 && ok)
                            write_loss<TAIL>(p, row, te, view_of<TAIL>(p, gather_mail(b)), gather_again(b));
                        __syncwarp();
                        if (lane == 0) mbar_arrive(tempty(b));
                    }
                } else {
                    if (!TAIL) ok = ok && mbar_wait(tfull(b), buf_phase, p, abort_flag);
                    ok = ok && wait_mail(b, buf_phase);
                    view = view_of<TAIL>(p, gather_mail(b));
                    if (rank == 0 && threadIdx.x == 0 && ok) write_loss<TAIL>(p, row, te, view, gather_again(b));
                }
            } else {
                view = view_of_stats<TAIL>(te.stats);
            }
            if constexpr (MODE != FWD) {
                // ------------------------------------------ gradient ----
                const Slope<T, TAIL> slope(p, pt, te, row, view);
#pragma unroll 1
                for (int c0 = 0, ch = 0; STREAM ? c0 < p.part : ch < CHUNKS; c0 += p.chunk, ++ch) {
                    if (STREAM) wait_group(CHUNKS - 1);
                    const uint8_t* rows = STREAM ? sm.rows + 16 * (slot - c0) : sm.rows;
                    const int u1 = ok ? min(c0 + p.chunk, pt.n) : 0;
                    slope.units(pt, rows, c0 + (int)threadIdx.x, u1, 32 * W);
                    if (STREAM) {
                        send_next();
                        advance();
                    } else {
                        send_for(row + step, c0, c0);
                    }
                }
                asm volatile("bar.sync 1, %0;" ::"n"(32 * W) : "memory");      // what the other warps stored is there
                if (ok) slope.kept(p, pt, sm, b, threadIdx.x, 32 * W);
            }
            if (MODE != FWD) {
                __syncwarp();
                if (lane == 0) mbar_arrive(tempty(b));
            }
        }
    }
    wait_group(0);
    __syncthreads();
    if (C > 1) cluster_sync();      // nobody leaves while its mail is written
}

// Small vocabularies: one warp does all of a row, the next row's logits on
// their way meanwhile, and up to 28 rows are under way on an SM.  The chain of a
// row's sums, which bounds them, has no barrier in it (16,384 x 1,000 bf16, loss and
// gradient: 27 us, 54 by three warps with 10 rows an SM; 2,500 columns 56 and 75).
constexpr int kWarpPerSm = 28;
template <typename T, int MODE, bool TAIL>
__global__ void __launch_bounds__(32, kWarpPerSm) k_distill_warp(const Params p) {
    constexpr int E = Unit<T>::E;
    extern __shared__ __align__(16) uint8_t smem[];
    const Smem sm{smem, p.held, p.part, (p.k + 3) / 4 * 4};
    Teacher& te = *reinterpret_cast<Teacher*>(sm.fixed());
    const int lane = threadIdx.x;
    const int64_t step = gridDim.x;
    auto send_for = [&](int64_t row, int buf) {      // this lane's units of a row
        if (row < p.M) {
            const Part pt = part_of<T>(p, row, 0u);
            const uint8_t* src = reinterpret_cast<const uint8_t*>(static_cast<const T*>(p.x) + row * p.ldx) -
                                 pt.head * (int)sizeof(T);
            const uint32_t dst = smem_u32(smem + 16 * buf * p.part);
#pragma unroll 4
            for (int u = lane; u < pt.n; u += 32)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + 16 * u), "l"(src + 16 * (int64_t)u)
                             : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int i = lane; i < bits_bytes(p.part) / 4; i += 32) reinterpret_cast<uint32_t*>(sm.bits(0))[i] = 0u;
    __syncwarp();
    wait_for_previous_kernels();
    Ahead ah = {};
    int buf = 0;
    send_for(blockIdx.x, 0);
    load_tokens<MODE, TAIL>(p, blockIdx.x, 0, lane, ah);
    for (int64_t row = blockIdx.x; row < p.M; row += step, buf ^= 1) {
        send_for(row + step, buf ^ 1);
        const Part pt = part_of<T>(p, row, 0u);
        teacher_row<T, MODE, TAIL>(p, sm, te, 0, row, row + step, 0u, lane, ah);
        wait_group(1);
        const uint8_t* rows = smem + 16 * buf * p.part;
        View view;
        if constexpr (MODE != BWD) {
            Sum sum;
#pragma unroll 2
            for (int u = lane; u < pt.n; u += 32) {
                uint4 v = *reinterpret_cast<const uint4*>(rows + 16 * u);
                uint32_t out = TAIL ? sm.bits(0)[u] : 0u;
                if (u < pt.u0 || u >= pt.u1) out |= outside<E>(pt, u);
                if (out) leave_out<E>(v, out);
                sum.add<T, 1>(&v, p.c);
            }
            const float m = warp_max(sum.m), s = warp_sum(sum.total() * e_of(sum.m, finite_max(m), p.c));
            view = view_of<TAIL>(p, TAIL ? joined(te.top_max, te.top_sum, m, s, p.c) : Sums{m, s, m, s});
            if (lane == 0) write_loss<TAIL>(p, row, te, view, te.again);
        } else {
            view = view_of_stats<TAIL>(te.stats);
        }
        if constexpr (MODE != FWD) {
            const Slope<T, TAIL> slope(p, pt, te, row, view);
            slope.units(pt, rows, lane, pt.n, 32);
            __syncwarp();      // what the other lanes stored is there
            slope.kept(p, pt, sm, 0, lane, 32);
        }
        __syncwarp();
        if (by_bits<MODE, TAIL>(p)) clear_bits<T>(p, sm, 0, pt, lane);
    }
    wait_group(0);
}

// ----------------------------------------------------------------- host ----

#define MOE_DISTILL_INSTANCES(X)                                                                            \
    X(__nv_bfloat16, FWD, false) X(__nv_bfloat16, FWD, true) X(__nv_bfloat16, BWD, false)                   \
    X(__nv_bfloat16, BWD, true) X(__nv_bfloat16, BOTH, false) X(__nv_bfloat16, BOTH, true)                  \
    X(float, FWD, false) X(float, FWD, true) X(float, BWD, false) X(float, BWD, true) X(float, BOTH, false) \
    X(float, BOTH, true)

constexpr int kPerSm = 3, kNarrowPerSm = 10;      // CTAs of an SM, by registers
constexpr int kSmemSm = 233472;                   // shared memory of an SM, 1 KB of it the system's per CTA
struct Clusters {                                 // that run at a time: wide CTAs or not; of 1, 2, 4, 8; CTAs an SM
    int n[2][4][kPerSm];
};
static PerDevice<Clusters> g_clusters;
static size_t smem_of(int per_sm) { return kSmemSm / per_sm / 128 * 128 - 1024; }

static cudaLaunchConfig_t launch_cfg(int64_t clusters, int C, bool wide, size_t smem, cudaStream_t stream,
                                     cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(clusters * C));
    cfg.blockDim = dim3(wide ? 288 : 96);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cfg;
}

static cudaError_t set_attributes() {
    const int most = 232448;
#define X(T, M, R)                                                                                             \
    for (const void* k :                                                                                       \
         {(const void*)k_distill<T, M, R, 2>, (const void*)k_distill<T, M, R, 8>, (const void*)k_distill_warp<T, M, R>}) { \
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, most);       \
        if (e != cudaSuccess) return e;                                                                        \
    }
    MOE_DISTILL_INSTANCES(X)
#undef X
    Clusters& at = g_clusters.here();
    for (int wide = 0; wide < 2; ++wide)
        for (int c = 0; c < 4; ++c)
            for (int n = 1; n <= (wide ? kPerSm : 1); ++n) {
                cudaLaunchAttribute attr[2];
                const cudaLaunchConfig_t cfg = launch_cfg(1024, 1 << c, wide, wide ? smem_of(n) : smem_of(kNarrowPerSm), nullptr, attr);
                const cudaError_t e = cudaOccupancyMaxActiveClusters(
                    &at.n[wide][c][n - 1],
                    wide ? k_distill<__nv_bfloat16, BOTH, true, 8> : k_distill<__nv_bfloat16, BOTH, true, 2>, &cfg);
                if (e != cudaSuccess) return e;
            }
    return cudaSuccess;
}
typedef void (*Kernel)(const Params);
static Kernel kernel_of(bool f32, int mode, bool tail, bool wide) {
#define X(T, M, R)                                                                  \
    if (f32 == (sizeof(T) == 4) && mode == M && tail == R)                           \
        return wide ? (Kernel)k_distill<T, M, R, 8> : (Kernel)k_distill<T, M, R, 2>;
    MOE_DISTILL_INSTANCES(X)
#undef X
    return nullptr;
}
static Kernel warp_kernel_of(bool f32, int mode, bool tail) {
#define X(T, M, R) \
    if (f32 == (sizeof(T) == 4) && mode == M && tail == R) return (Kernel)k_distill_warp<T, M, R>;
    MOE_DISTILL_INSTANCES(X)
#undef X
    return nullptr;
}

// Rows of up to 320 16-byte units, more of them than a few for every SM: a warp each.
constexpr int kWarpUnits = 320;
static moe_status_t launch_warps(Params p, bool f32, int mode, int sms, cudaStream_t stream) {
    const int E = f32 ? 4 : 8;
    p.part = (E - 1 + p.V + E - 1) / E;
    p.held = 2 * p.part;
    const size_t smem = smem_bytes(p.held, p.part, p.k);
    const int64_t per_sm = std::min<int64_t>(kWarpPerSm, kSmemSm / (smem + 1024));
    const dim3 grid((unsigned)std::min<int64_t>(p.M, sms * per_sm));
    if (launch_early(grid, 32, smem, stream, warp_kernel_of(f32, mode, p.lse != nullptr), p) != cudaSuccess)
        return MOE_ERR_CUDA;
    MOE_CHECK_LAUNCH();
    return MOE_OK;
}
static bool warps_do(int64_t M, int V, bool f32, int sms) {
    const int E = f32 ? 4 : 8;
    return (E - 1 + V + E - 1) / E <= kWarpUnits && M > 4 * (int64_t)sms;
}

// How a call is spread: CTAs of a cluster (they share a row), 288 threads each
// or, for small parts, 96, of which three times as many rows are under way on
// an SM (16,384 x 4,096 bf16, loss and gradient: 75 us, 149 with 288; 8,000 columns 101
// and 179, 16,000 240 and 229), and clusters, no more than run at a time, so that rows are
// dealt out evenly.  Of the sizes of clusters the one with the shortest
// time by this count, in ns: a 16-byte unit takes an SM 0.36 to read at the
// memory's rate and as much to write, shared by its CTAs (one alone gets no more
// than half of it), and a row 700 besides for the chain of its sums (800 more where they
// go through the cluster), 600 for the gradient alone.  The count ranks the
// sizes; where a row's chain is not covered it is below what is measured (loss and
// gradient of 16,384 rows: 8,000 columns 87 and 101 us, 16,000 181 and 229).
struct Spread {
    int C, part, chunk, held, per_sm;
    bool wide;
    size_t smem;
    int64_t clusters;
};
static Spread spread(int64_t M, int V, int elem, int k, int mode, int sms) {
    const int E = 16 / elem, units = (E - 1 + V + E - 1) / E;
    const Clusters& at = g_clusters.here();
    Spread best{};
    double least = 1e300;
    for (int c = 0; c < 4; ++c) {
        Spread s{};
        s.C = 1 << c;
        s.part = (units + s.C - 1) / s.C;
        s.wide = s.part > 1200 || (s.part > 256 && M * s.C <= (int64_t)sms * kPerSm);
        const int turn = s.wide ? 256 : 64;      // units that a CTA's threads take at a time
        s.chunk = mode == BOTH ? (s.part + CHUNKS * turn - 1) / (CHUNKS * turn) * turn
                               : std::min(4, (s.part + turn - 1) / turn) * turn;
        s.held = mode == BOTH ? s.part : CHUNKS * s.chunk;
        s.smem = smem_bytes(s.held, s.part, k);
        if (s.smem > 232448 || (c > 0 && s.part < 32)) continue;
        s.per_sm = s.wide ? kPerSm : kNarrowPerSm;
        while (s.per_sm > 1 && s.smem > smem_of(s.per_sm)) --s.per_sm;
        const int64_t slots =
            s.wide ? at.n[1][c][s.per_sm - 1] : (int64_t)at.n[0][c][0] * s.per_sm / kNarrowPerSm;
        s.clusters = std::min<int64_t>(M, std::max<int64_t>(1, slots));
        const double ctas = std::max(2., std::min<double>(s.per_sm, (double)s.clusters * s.C / sms));
        const double cost = (double)((M + s.clusters - 1) / s.clusters) *
                            (s.part * 0.36 * (mode == FWD ? 1 : 2) * ctas + (mode == BWD ? 600 : (c ? 1500 : 700)));
        if (cost < least) least = cost, best = s;
    }
    return best;
}

static moe_status_t launch(Params p, bool f32, int mode, cudaStream_t stream) {
    const int sms = device_sm_count();
    MOE_REQUIRE(sms > 0, MOE_ERR_NOT_INITIALIZED);
    if (warps_do(p.M, p.V, f32, sms)) return launch_warps(p, f32, mode, sms, stream);
    const Spread d = spread(p.M, p.V, f32 ? 4 : 2, p.k, mode, sms);
    MOE_REQUIRE(d.C > 0, MOE_ERR_UNSUPPORTED);
    p.part = d.part, p.chunk = d.chunk, p.held = d.held;
    p.timeout_ns = 2000000000ull;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = launch_cfg(d.clusters, d.C, d.wide, d.smem, stream, attr);
    if (cudaLaunchKernelEx(&cfg, kernel_of(f32, mode, p.lse != nullptr, d.wide), p) != cudaSuccess) return MOE_ERR_CUDA;
    MOE_CHECK_LAUNCH();
    return MOE_OK;
}

}  // namespace distill

cudaError_t distill_set_attributes() { return distill::set_attributes(); }

}  // namespace moe

using namespace moe;

// What the three calls check alike; M = 0 is the caller's.
static moe_status_t fill(distill::Params& p, const void* x, int x_type, int64_t ldx, const int32_t* idx, int64_t ldi,
                         const void* t, int t_type, int64_t ldt, const float* lse, float tau, int64_t M, int V, int k,
                         int32_t* err) {
    MOE_REQUIRE((x_type == MOE_TYPE_BF16 || x_type == MOE_TYPE_F32) && (t_type == MOE_TYPE_BF16 || t_type == MOE_TYPE_F32),
                MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(M >= 0 && V >= 1 && k >= 1 && tau > 0.f && tau <= 1e6f && tau >= 1e-6f, MOE_ERR_INVALID_ARG);
    MOE_REQUIRE((M <= 1 || (ldx >= V && ldi >= k && ldt >= k)), MOE_ERR_INVALID_ARG);
    const int E = x_type == MOE_TYPE_F32 ? 4 : 8;
    MOE_REQUIRE(M <= 0x7FFFFF00LL && k <= distill::MAX_K &&
                    (int64_t)V + 2 * E - 2 <= (int64_t)E * distill::MAX_C * distill::MAX_PART,
                MOE_ERR_UNSUPPORTED);
    MOE_REQUIRE(M == 0 || (x && idx && t), MOE_ERR_INVALID_ARG);
    auto at = [](const void* q, int n) { return reinterpret_cast<uintptr_t>(q) % n == 0; };
    MOE_REQUIRE(at(x, x_type == MOE_TYPE_F32 ? 4 : 2) && at(idx, 4) && at(t, t_type == MOE_TYPE_F32 ? 4 : 2) && at(lse, 4),
                MOE_ERR_ALIGNMENT);
    p.x = x, p.ldx = ldx, p.idx = idx, p.ldi = ldi, p.t = t, p.ldt = ldt, p.t_f32 = t_type == MOE_TYPE_F32;
    p.lse = lse, p.M = M, p.V = V, p.k = k, p.err = err;
    p.tau = tau, p.inv_tau = 1.f / tau, p.c = distill::kLog2e / tau;
    return MOE_OK;
}
static moe_status_t fill_gradient(distill::Params& p, const float* dloss, int x_type, void* dx, int64_t lddx) {
    MOE_REQUIRE(p.M <= 1 || lddx >= p.V, MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(p.M == 0 || (dloss && dx), MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(dx != p.x || lddx == p.ldx || p.M <= 1, MOE_ERR_INVALID_ARG);      // in place: row by row
    MOE_REQUIRE(reinterpret_cast<uintptr_t>(dloss) % 4 == 0 &&
                    reinterpret_cast<uintptr_t>(dx) % (x_type == MOE_TYPE_F32 ? 4 : 2) == 0,
                MOE_ERR_ALIGNMENT);
    p.dloss = dloss, p.dx = dx, p.lddx = lddx;
    return MOE_OK;
}
static bool aligned4(const void* q) { return reinterpret_cast<uintptr_t>(q) % 4 == 0; }

extern "C" moe_status_t distill_loss_fwd(const void* x, int x_type, int64_t ldx, const int32_t* idx, int64_t ldi,
                                         const void* t, int t_type, int64_t ldt, const float* teacher_lse, float tau,
                                         int64_t M, int V, int k, float* loss, float* stats, int32_t* err,
                                         void* stream) {
    distill::Params p{};
    const moe_status_t st = fill(p, x, x_type, ldx, idx, ldi, t, t_type, ldt, teacher_lse, tau, M, V, k, err);
    if (st != MOE_OK) return st;
    MOE_REQUIRE(loss || stats, MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(aligned4(loss) && aligned4(stats), MOE_ERR_ALIGNMENT);
    if (M == 0) return MOE_OK;
    MOE_REQUIRE(device_initialized(), MOE_ERR_NOT_INITIALIZED);
    p.loss = loss, p.stats = stats;
    return distill::launch(p, x_type == MOE_TYPE_F32, distill::FWD, (cudaStream_t)stream);
}

extern "C" moe_status_t distill_loss_bwd(const float* dloss, const void* x, int x_type, int64_t ldx, const int32_t* idx,
                                         int64_t ldi, const void* t, int t_type, int64_t ldt, const float* stats,
                                         const float* teacher_lse, float tau, int64_t M, int V, int k, void* dx,
                                         int64_t lddx, int32_t* err, void* stream) {
    distill::Params p{};
    moe_status_t st = fill(p, x, x_type, ldx, idx, ldi, t, t_type, ldt, teacher_lse, tau, M, V, k, err);
    if (st == MOE_OK) st = fill_gradient(p, dloss, x_type, dx, lddx);
    if (st != MOE_OK) return st;
    MOE_REQUIRE(M == 0 || stats, MOE_ERR_INVALID_ARG);
    MOE_REQUIRE(aligned4(stats), MOE_ERR_ALIGNMENT);
    if (M == 0) return MOE_OK;
    MOE_REQUIRE(device_initialized(), MOE_ERR_NOT_INITIALIZED);
    p.stats = const_cast<float*>(stats);
    return distill::launch(p, x_type == MOE_TYPE_F32, distill::BWD, (cudaStream_t)stream);
}

extern "C" moe_status_t distill_loss(const float* dloss, const void* x, int x_type, int64_t ldx, const int32_t* idx,
                                     int64_t ldi, const void* t, int t_type, int64_t ldt, const float* teacher_lse,
                                     float tau, int64_t M, int V, int k, float* loss, void* dx, int64_t lddx,
                                     int32_t* err, void* stream) {
    distill::Params p{};
    moe_status_t st = fill(p, x, x_type, ldx, idx, ldi, t, t_type, ldt, teacher_lse, tau, M, V, k, err);
    if (st == MOE_OK) st = fill_gradient(p, dloss, x_type, dx, lddx);
    if (st != MOE_OK) return st;
    MOE_REQUIRE(aligned4(loss), MOE_ERR_ALIGNMENT);
    if (M == 0) return MOE_OK;
    MOE_REQUIRE(device_initialized(), MOE_ERR_NOT_INITIALIZED);
    p.loss = loss;
    return distill::launch(p, x_type == MOE_TYPE_F32, distill::BOTH, (cudaStream_t)stream);
}
