// bf16 products on CTA pairs (tcgen05.mma.cta_group::2): what the dense and the
// grouped kernels share -- descriptors, the instruction, activations, the state
// of a ring.
#pragma once

#include "gemm_common.cuh"

namespace moe {

// gemm.cu
bool make_bf16_map(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t ld, int box_rows);
bool make_store_map(CUtensorMap* m, void* base, int64_t rows, int64_t cols, int64_t ld, bool f32);

namespace dense {

using namespace gg;

constexpr int TM = 256, TK = 64;                // rows of the pair's tile, the k-step

// Instruction descriptor: bf16 A and B, fp32 D, M = 256 over the pair,
// N = bn; bits 15 and 16 say that A and B lie M- and N-major.
template <bool A_MN, bool B_MN>
__device__ __forceinline__ uint32_t make_idesc_pair(int bn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (A_MN ? 1u << 15 : 0u) | (B_MN ? 1u << 16 : 0u) |
           ((uint32_t)(bn >> 3) << 17) | ((uint32_t)(TM >> 4) << 24);
}

// Shared-memory descriptor of an operand that lies M- or N-major, 128-byte
// swizzle: rows of 64 elements (128 bytes) of the M/N axis, one row per k;
// 8 k-rows are 1024 bytes apart (stride offset), the next 64 elements of the
// M/N axis `block` bytes further (leading offset).
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr, uint32_t block) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(block >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}
template <bool MN>
__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr) {
    if constexpr (MN) return desc_mn_sw128(saddr, 64 * TK * 2);
    else return desc_sw128(saddr);
}
// 16 deeper along k: 32 bytes inside the rows, or 16 rows of 128 bytes
template <bool MN>
__device__ __forceinline__ constexpr uint64_t k16_step() {
    return MN ? (16 * 128) >> 4 : 32 >> 4;
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

__device__ __forceinline__ void tc_mma2_bf16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ float act_of(float z, int act) {
    if (act == MOE_ACT_SILU) return z * fast_sigmoid(z);
    if (act == MOE_ACT_GELU) return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
    if (act == MOE_ACT_RELU) return z < 0.f ? 0.f : z;
    return z;
}
// d act(z) / dz
__device__ __forceinline__ float act_slope(float z, int act) {
    if (act == MOE_ACT_SILU) {
        const float s = fast_sigmoid(z);
        return s * (1.f + z * (1.f - s));
    }
    if (act == MOE_ACT_GELU)
        return 0.5f * (1.f + erff(z * 0.70710678118654752f)) + z * __expf(-0.5f * z * z) * 0.39894228040143268f;
    if (act == MOE_ACT_RELU) return z > 0.f ? 1.f : 0.f;
    return 1.f;
}

__device__ __forceinline__ uint4 load_vec8(const __nv_bfloat16* p, int n) {      // n < 8: zeros after them
    if (n == 8) return *reinterpret_cast<const uint4*>(p);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < n) w[j >> 1] |= (uint32_t)__bfloat16_as_ushort(p[j]) << (16 * (j & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}
// arrive on the barrier at the same shared offset in both CTAs of the pair
// that starts at cluster rank `lead`
__device__ __forceinline__ void tc_commit_pair(uint32_t bar, uint32_t lead) {
    const uint16_t mask = (uint16_t)(0x3u << lead);
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::
                     "r"(bar),
                 "h"(mask)
                 : "memory");
}

// Where a role is in the ring of stages, or in that of accumulators.
struct Ring {
    int at = 0, count = 0;
    uint32_t phase = 0;
    bool aborted = false;
    __device__ __forceinline__ void next(int n) {
        ++count;
        if (++at == n) {
            at = 0;
            phase ^= 1u;
        }
    }
};

}  // namespace dense
}  // namespace moe
