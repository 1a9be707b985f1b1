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
// kept it would be lost where the student is sure of them.
//
// A row is split over the CTAs of a cluster, and each keeps its part in
// shared memory, so that loss and gradient together read the logits once: 4
// bytes an element of bf16 logits instead of 6 in two calls.  The parts'
// maxima and sums are exchanged through distributed shared memory.  Several
// CTAs share an SM: one's loads run under another's arithmetic and stores.
// Warps: 0 .. W - 1 go over the logits, W loads them (bulk copies of whole
// 16-byte units, so rows may start at any element; what is read of the
// neighbouring rows is not used), W + 1 works on the teacher's tokens a row
// ahead.  All waits are bounded.
#include <algorithm>

#include "gemm_common.cuh"

namespace moe {
namespace distill {

using namespace gg;

constexpr int MAX_K = 1024;              // tokens of the teacher
constexpr int MAX_C = 8;                 // CTAs of a cluster
constexpr int CHUNKS = 4;                // of a part, each with its own barriers
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
    float* stats;             // [M, 3]: max x, s, s_rest; BWD: read
    int64_t M;
    int V, k;
    float tau, inv_tau, c;    // c = log2(e) / tau
    int part, chunk;          // 16-byte units of a CTA's part, of a chunk
    int32_t* err;
    uint64_t timeout_ns;
};

// what a warp knows of a row's teacher, per buffer
struct Teacher {
    float mass, rest, p_sum;        // mass = sum p + rest
    float fit, x_ref, t_lse;        // sum p ((t - max t) - (x - x_ref) / tau); log-sum-exp of t - max t
    float top_max, top_sum;         // of the kept tokens in this CTA's part
    int some;                       // 0: no teacher, loss and gradient are zero
};

// Shared memory: the part, then (two buffers each) a byte per 16-byte unit,
// and of each of the teacher's tokens its column (bit 31: counted with an
// earlier one; -1: none), its probability and the student's logit.
struct Smem {
    uint8_t* rows;
    int part, k;
    __device__ __forceinline__ uint8_t* bits(int b) const;
    __device__ __forceinline__ int* col(int b) const;
    __device__ __forceinline__ float* p(int b) const { return reinterpret_cast<float*>(col(b)) + k; }
    __device__ __forceinline__ float* x(int b) const { return p(b) + k; }
    __device__ __forceinline__ uint8_t* fixed() const { return reinterpret_cast<uint8_t*>(col(2)); }
};
struct Fixed {
    unsigned long long bar[2 * CHUNKS + 6];
    float4 mail[2][MAX_C];          // max, s, s_rest of the cluster's parts
    float2 warp_part[8];
    Teacher teacher[2];
    int abort_flag;
};

__host__ __device__ inline int bits_bytes(int part) { return (part + 15) / 16 * 16; }
__host__ __device__ inline size_t smem_bytes(int part, int k) {
    return (size_t)part * 16 + 2 * bits_bytes(part) + 24 * (size_t)((k + 3) / 4 * 4) + sizeof(Fixed);
}
__device__ __forceinline__ uint8_t* Smem::bits(int b) const { return rows + 16 * part + b * bits_bytes(part); }
__device__ __forceinline__ int* Smem::col(int b) const { return reinterpret_cast<int*>(bits(2)) + 3 * b * k; }
static_assert(MAX_PART * 18 + 24 * MAX_K + sizeof(Fixed) <= 232448 && MAX_PART % 16 == 0, "shared memory budget");

__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
    return n;
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

template <typename T>
struct Unit;      // 16 bytes of logits
template <>
struct Unit<__nv_bfloat16> {
    static constexpr int E = 8;
    static __device__ __forceinline__ void load(const uint8_t* p, float* f) {
        unpack8(*reinterpret_cast<const uint4*>(p), f);
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
    static __device__ __forceinline__ void load(const uint8_t* p, float* f) {
        const float4 v = *reinterpret_cast<const float4*>(p);
        f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
    }
    static __device__ __forceinline__ void store(float* p, const float* f) {
        *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    }
    static __device__ __forceinline__ float one(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }
    static __device__ __forceinline__ float to(float f) { return f; }
};

// Where a row's part lies: its units [g0, g0 + n) counted from the row's first
// 16-byte boundary; element e of unit g is column g E + e - head.
struct Part {
    int head, g0, n;
};
template <typename T>
__device__ __forceinline__ Part part_of(const Params& p, int64_t row, uint32_t rank) {
    constexpr int E = Unit<T>::E;
    Part r;
    const uintptr_t at = reinterpret_cast<uintptr_t>(static_cast<const T*>(p.x) + row * p.ldx);
    r.head = (int)(at & 15) / (int)sizeof(T);
    const int units = (r.head + p.V + E - 1) / E;
    r.g0 = (int)rank * p.part;
    r.n = max(0, min(p.part, units - r.g0));
    return r;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// The teacher's row (one warp): probabilities, what the loss needs of them,
// and, of the tokens in this CTA's part, their bits, sums and logits.
template <typename T, int MODE, bool TAIL>
__device__ __forceinline__ void teacher_row(const Params& p, const Smem& sm, Teacher& out, int b, int64_t row,
                                            uint32_t rank, int lane, bool fresh) {
    constexpr int E = Unit<T>::E;
    const Part pt = part_of<T>(p, row, rank);
    int* col = sm.col(b);
    float *pr = sm.p(b), *xs = sm.x(b);
    uint32_t* words = reinterpret_cast<uint32_t*>(sm.bits(b));
    if (fresh) {
        for (int i = lane; i < bits_bytes(p.part) / 4; i += 32) words[i] = 0u;
        __syncwarp();
    }
    const float inv_tau = p.inv_tau;
    bool any = false, dup = false;
    float t_max = -INFINITY, x_max = -INFINITY;
    for (int j = lane; j < p.k; j += 32) {
        const int i = p.idx[row * p.ldi + j];
        const bool ok = i >= 0 && i < p.V;
        if (i >= p.V) set_err(p.err, MOE_ERR_BAD_INDEX);
        float t = -INFINITY, x = 0.f;
        if (ok) {
            const int64_t at = row * p.ldt + j;
            t = p.t_f32 ? static_cast<const float*>(p.t)[at]
                        : __bfloat162float(static_cast<const __nv_bfloat16*>(p.t)[at]);
            t *= inv_tau;
            const int u = i + pt.head, g = u / E - pt.g0;
            const bool mine = g >= 0 && g < pt.n;
            if (mine || (rank == 0 && MODE != BWD)) x = Unit<T>::one(p.x, row * p.ldx + i);
            if (mine && (TAIL || MODE != FWD)) {
                const uint32_t bit = 1u << (8 * (g & 3) + u % E);
                dup |= (atomicOr(words + (g >> 2), bit) & bit) != 0;
            }
            any = true;
        }
        col[j] = ok ? i : -1;
        pr[j] = t;
        xs[j] = x;
        t_max = fmaxf(t_max, t);
        if (ok && t > -INFINITY) x_max = fmaxf(x_max, x);
    }
    any = __any_sync(0xFFFFFFFFu, any);
    dup = __any_sync(0xFFFFFFFFu, dup);
    const float top = warp_max(t_max), t_ref = finite_max(top);
    const float x_ref = finite_max(warp_max(x_max));
    __syncwarp();
    float sum = 0.f;
    if (!TAIL) {
        for (int j = lane; j < p.k; j += 32)
            if (col[j] >= 0) sum += expf(pr[j] - t_ref);
        sum = warp_sum(sum);
    }
    const float t_lse = TAIL ? p.lse[row] - t_ref : logf(sum), inv = 1.f / sum;
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
    mass = warp_sum(mass);
    fit = warp_sum(fit);
    __syncwarp();
    if (dup) {      // the first of several holds the sum of their probabilities
        for (int j = lane; j < p.k; j += 32) {
            const int cj = col[j];
            if (cj == -1) continue;
            bool first = true;
            float q = pr[j];
            for (int i = 0; i < p.k; ++i) {
                if (i == j || col[i] == -1 || (col[i] & 0x7FFFFFFF) != cj) continue;
                if (i < j) first = false;
                else q += pr[i];
            }
            if (first) pr[j] = q;
            else col[j] = cj | (int)0x80000000;
        }
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
        out.fit = fit, out.x_ref = x_ref, out.t_lse = t_lse;
        out.top_max = top_max, out.top_sum = top_sum;
        out.some = some;
    }
    __syncwarp();
}
// the bits of the row before last in this buffer
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

// T: logits; W warps go over them.
template <typename T, int MODE, bool TAIL, int W>
__global__ void __launch_bounds__(32 * W + 64, W == 8 ? 4 : 12) k_distill(const Params p) {
    constexpr int E = Unit<T>::E;
    extern __shared__ __align__(16) uint8_t smem[];
    const Smem sm{smem, p.part, (p.k + 3) / 4 * 4};
    Fixed& fx = *reinterpret_cast<Fixed*>(sm.fixed());
    const uint32_t bar0 = smem_u32(&fx.bar[0]);
    auto full = [&](int i) { return bar0 + 8u * i; };
    auto empty = [&](int i) { return bar0 + 8u * (CHUNKS + i); };
    auto tfull = [&](int i) { return bar0 + 8u * (2 * CHUNKS + i); };
    auto tempty = [&](int i) { return bar0 + 8u * (2 * CHUNKS + 2 + i); };
    auto xbar = [&](int i) { return bar0 + 8u * (2 * CHUNKS + 4 + i); };
    volatile int* abort_flag = &fx.abort_flag;
    const uint32_t C = cluster_size(), rank = C > 1 ? cluster_ctarank() : 0u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < CHUNKS; ++i) mbar_init(full(i), 1), mbar_init(empty(i), W);
        for (int i = 0; i < 2; ++i) mbar_init(tfull(i), 1), mbar_init(tempty(i), W), mbar_init(xbar(i), C);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fx.abort_flag = 0;
    }
    __syncthreads();
    if (C > 1) cluster_sync();      // the peers' barriers are initialised
    wait_for_previous_kernels();
    const int64_t row0 = blockIdx.x / C, step = gridDim.x / C;

    if (warp == W) {
        // ------------------------------------------------------ loads ----
        if (lane == 0) {
            int it = 0, issued = 0;
            bool ok = true;
            for (int64_t row = row0; row < p.M && ok; row += step, ++it) {
                const Part pt = part_of<T>(p, row, rank);
                const uint8_t* src = reinterpret_cast<const uint8_t*>(static_cast<const T*>(p.x) + row * p.ldx) -
                                     pt.head * sizeof(T) + (size_t)pt.g0 * 16;
                for (int ch = 0; ch < CHUNKS; ++ch) {
                    if (!mbar_wait(empty(ch), (uint32_t)(it & 1) ^ 1u, p, abort_flag)) {
                        ok = false;
                        break;
                    }
                    const int u0 = ch * p.chunk, n = min(p.chunk, pt.n - u0);
                    if (n > 0) {
                        mbar_expect_tx(full(ch), 16u * n);
                        bulk_load(smem_u32(sm.rows + 16 * u0), src + 16 * (size_t)u0, 16u * n, full(ch));
                    } else {
                        mbar_arrive(full(ch));
                    }
                    ++issued;
                }
            }
            // nobody leaves with copies in flight
            Params q = p;
            q.timeout_ns = 200000000ull;
            volatile int no_abort = 0;
            for (int i = issued - min(issued, CHUNKS); i < issued; ++i)
                mbar_wait(full(i % CHUNKS), (uint32_t)(i / CHUNKS) & 1u, q, &no_abort);
        }
        __syncwarp();
    } else if (warp == W + 1) {
        // ---------------------------------------------- teacher, a row ahead ----
        int it = 0;
        for (int64_t row = row0; row < p.M; row += step, ++it) {
            const int b = it & 1;
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(tempty(b), (uint32_t)((it >> 1) & 1) ^ 1u, p, abort_flag))) break;
            if (it >= 2 && (TAIL || MODE != FWD)) clear_bits<T>(p, sm, b, part_of<T>(p, row - 2 * step, rank), lane);
            teacher_row<T, MODE, TAIL>(p, sm, fx.teacher[b], b, row, rank, lane, it < 2);
            if (lane == 0) mbar_arrive(tfull(b));
        }
    } else {
        // (a warp whose wait gave up goes on through the barriers, so that the
        // others do not wait for it, and touches nothing)
        int it = 0;
        bool ok = true;
        for (int64_t row = row0; row < p.M; row += step, ++it) {
            const int b = it & 1;
            const uint32_t row_phase = (uint32_t)(it & 1), buf_phase = (uint32_t)((it >> 1) & 1);
            const Part pt = part_of<T>(p, row, rank);
            ok = ok && mbar_wait(tfull(b), buf_phase, p, abort_flag);
            const Teacher& te = fx.teacher[b];
            const uint8_t* bits = sm.bits(b);
            const int lo0 = pt.head - pt.g0 * E, hi0 = pt.head + p.V - pt.g0 * E;      // of the part's elements, those of the row
            float m = 0.f, s = 1.f, s_rest = 1.f;
            if constexpr (MODE != BWD) {
                // -------------------------------- maximum and sum ----
                float tm = -INFINITY, ts = 0.f;
                for (int ch = 0; ch < CHUNKS; ++ch) {
                    ok = ok && mbar_wait(full(ch), row_phase, p, abort_flag);
                    const int u1 = min((ch + 1) * p.chunk, pt.n);
                    for (int u = ch * p.chunk + (int)threadIdx.x; u < u1 && ok; u += 32 * W) {
                        float f[E];
                        Unit<T>::load(sm.rows + 16 * u, f);
                        if (u * E < lo0 || u * E + E > hi0) {
#pragma unroll
                            for (int e = 0; e < E; ++e)
                                if (u * E + e < lo0 || u * E + e >= hi0) f[e] = -INFINITY;
                        }
                        if constexpr (TAIL) {
                            const uint32_t kept = bits[u];
                            if (kept) {
#pragma unroll
                                for (int e = 0; e < E; ++e)
                                    if (kept >> e & 1) f[e] = -INFINITY;
                            }
                        }
                        float um = f[0];
#pragma unroll
                        for (int e = 1; e < E; ++e) um = fmaxf(um, f[e]);
                        if (um > tm) {
                            ts *= e_of(tm, um, p.c);
                            tm = um;
                        }
                        const float ref = finite_max(tm);
#pragma unroll
                        for (int e = 0; e < E; ++e) ts += e_of(f[e], ref, p.c);
                    }
                    if (MODE == FWD) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(empty(ch));
                    }
                }
                const float wm = warp_max(tm);
                ts = warp_sum(ts * e_of(tm, finite_max(wm), p.c));
                if (lane == 0) fx.warp_part[warp] = make_float2(wm, ts);
                asm volatile("bar.sync 1, %0;" ::"n"(32 * W) : "memory");
                if (warp == 0 && ok) {
                    float cm = te.top_max, rest = 0.f;
#pragma unroll
                    for (int w = 0; w < W; ++w) cm = fmaxf(cm, fx.warp_part[w].x);
                    const float ref = finite_max(cm);
#pragma unroll
                    for (int w = 0; w < W; ++w) rest += fx.warp_part[w].y * e_of(fx.warp_part[w].x, ref, p.c);
                    const float all = TAIL ? rest + te.top_sum * e_of(te.top_max, ref, p.c) : rest;
                    if (lane < (int)C) {
                        const uint32_t to = mapa(smem_u32(&fx.mail[b][rank]), (uint32_t)lane);
                        asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to), "f"(cm), "f"(all),
                                     "f"(rest), "f"(0.f)
                                     : "memory");
                        mbar_arrive_remote(mapa(xbar(b), (uint32_t)lane));
                    }
                }
                ok = ok && mbar_wait_cluster(xbar(b), buf_phase, p, abort_flag);
                m = -INFINITY, s = 0.f, s_rest = 0.f;
                for (int i = 0; i < (int)C; ++i) m = fmaxf(m, fx.mail[b][i].x);
                const float ref = finite_max(m);
                for (int i = 0; i < (int)C; ++i) {
                    const float4 v = fx.mail[b][i];
                    const float f = e_of(v.x, ref, p.c);
                    s += v.y * f;
                    s_rest += v.z * f;
                }
                if (rank == 0 && threadIdx.x == 0 && ok) {
                    if (p.stats) p.stats[3 * row] = m, p.stats[3 * row + 1] = s, p.stats[3 * row + 2] = s_rest;
                    if (p.loss) {
                        float loss = te.fit + te.p_sum * ((ref - te.x_ref) * p.inv_tau + logf(s) - te.t_lse);
                        if (TAIL && te.rest > 0.f && s_rest > 0.f) loss += te.rest * (logf(te.rest) - logf(s_rest / s));
                        p.loss[row] = te.some ? loss * p.tau * p.tau : 0.f;
                    }
                }
            } else {
                m = p.stats[3 * row], s = p.stats[3 * row + 1], s_rest = p.stats[3 * row + 2];
            }
            if constexpr (MODE != FWD) {
                // ------------------------------------------ gradient ----
                const float g = p.dloss[row] * p.tau;
                const bool zero = !te.some || g == 0.f;
                const bool with_rest = TAIL && te.rest > 0.f && s_rest > 0.f;
                const float mass = with_rest ? te.mass : te.p_sum;
                const float f_top = g * (mass / s);
                const float f_all = with_rest ? g * (mass / s - te.rest / s_rest) : f_top;
                const float ref = finite_max(m);
                T* dx = static_cast<T*>(p.dx) + row * p.lddx - pt.head + (int64_t)pt.g0 * E;
                const bool vec = (reinterpret_cast<uintptr_t>(dx) & 15) == 0;
                for (int ch = 0; ch < CHUNKS; ++ch) {
                    if (MODE == BWD) ok = ok && mbar_wait(full(ch), row_phase, p, abort_flag);
                    const int u1 = min((ch + 1) * p.chunk, pt.n);
                    for (int u = ch * p.chunk + (int)threadIdx.x; u < u1 && ok; u += 32 * W) {
                        float f[E];
                        Unit<T>::load(sm.rows + 16 * u, f);
#pragma unroll
                        for (int e = 0; e < E; ++e) f[e] = zero ? 0.f : e_of(f[e], ref, p.c) * f_all;
                        if (vec && u * E >= lo0 && u * E + E <= hi0) {
                            Unit<T>::store(dx + (int64_t)u * E, f);
                        } else {
#pragma unroll
                            for (int e = 0; e < E; ++e)
                                if (u * E + e >= lo0 && u * E + e < hi0) dx[(int64_t)u * E + e] = Unit<T>::to(f[e]);
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(empty(ch));
                }
                // the kept tokens, over what was just stored there
                asm volatile("bar.sync 1, %0;" ::"n"(32 * W) : "memory");
                if (!zero && ok) {
                    for (int j = threadIdx.x; j < p.k; j += 32 * W) {
                        const int cj = sm.col(b)[j];
                        const int u = cj + lo0;      // element of the part
                        if (cj >= 0 && u >= 0 && u < pt.n * E)
                            dx[u] = Unit<T>::to(e_of(sm.x(b)[j], ref, p.c) * f_top - g * sm.p(b)[j]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty(b));
        }
    }
    __syncthreads();
    if (C > 1) cluster_sync();      // nobody leaves while its mail is written
}

// ----------------------------------------------------------------- host ----

#define MOE_DISTILL_INSTANCES(X)                                                                            \
    X(__nv_bfloat16, FWD, false) X(__nv_bfloat16, FWD, true) X(__nv_bfloat16, BWD, false)                   \
    X(__nv_bfloat16, BWD, true) X(__nv_bfloat16, BOTH, false) X(__nv_bfloat16, BOTH, true)                  \
    X(float, FWD, false) X(float, FWD, true) X(float, BWD, false) X(float, BWD, true) X(float, BOTH, false) \
    X(float, BOTH, true)

static cudaError_t set_attributes() {
    const int most = (int)smem_bytes(MAX_PART, MAX_K);
#define X(T, M, R)                                                                                             \
    for (const void* k : {(const void*)k_distill<T, M, R, 2>, (const void*)k_distill<T, M, R, 8>}) {            \
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, most);       \
        if (e != cudaSuccess) return e;                                                                        \
    }
    MOE_DISTILL_INSTANCES(X)
#undef X
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

// CTAs that share a row, and its part in 16-byte units: parts of at most 36
// KB, so that four CTAs and more share an SM; smaller ones while rows are too
// few to give every SM a part.
static int cluster_of(int64_t M, int V, int elem, int sms, int* part) {
    const int E = 16 / elem, units = (E - 1 + V + E - 1) / E;
    int c = 1;
    auto size = [&] { return (units + c - 1) / c; };
    while (c < MAX_C && (size() > 2304 || (M * c * 2 <= sms && size() > 128))) c *= 2;
    *part = size();
    return c;
}

static moe_status_t launch(Params p, bool f32, int mode, cudaStream_t stream) {
    const int sms = device_sm_count();
    MOE_REQUIRE(sms > 0, MOE_ERR_NOT_INITIALIZED);
    const int C = cluster_of(p.M, p.V, f32 ? 4 : 2, sms, &p.part);
    p.chunk = (p.part + CHUNKS - 1) / CHUNKS;
    p.timeout_ns = 2000000000ull;
    const bool wide = p.part > 256;
    const size_t smem = smem_bytes(p.part, p.k);
    const int per_sm = std::max(1, std::min(wide ? 4 : 12, (int)(233472 / (smem + 1024))));
    const int64_t clusters = std::min<int64_t>(p.M, std::max(1, sms * per_sm / C));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(clusters * C));
    cfg.blockDim = dim3(wide ? 320 : 128);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kernel_of(f32, mode, p.lse != nullptr, wide), p) != cudaSuccess) return MOE_ERR_CUDA;
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
