// Helpers of the 8-bit operators (e4m3 product, key/value cache, routed MLP).
#pragma once

#include "common.h"

namespace q4 {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));

constexpr int WIDE_RSRC3 = 0x00020000;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, WIDE_RSRC3);
}

// Loads from memory straight into LDS: 16 (or 4) bytes a lane from rsrc at voff
// + soff to LDS address lds + 16 (4) * lane; `lds`, rsrc and soff are the same in
// all lanes. In assembly because the compiler, where it tracks these loads,
// waits for all of them before any LDS read that it cannot tell apart, which
// would leave none in flight. There is no result register: what they write is
// LDS, whose address the statement takes (so it is not seen as unwritten), and
// no LDS read may pass join_with_loads_left(), which waits for them.
__device__ __forceinline__ v4i resource(const void* p, uint32_t bytes) {
    const uint64_t at = (uint64_t)(uintptr_t)p;
    return v4i{(int)(uint32_t)at, (int)(uint32_t)(at >> 32) & 0xFFFF, (int)bytes, WIDE_RSRC3};
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}
__device__ __forceinline__ void load_to_lds16(v4i rsrc, uint32_t lds, uint32_t voff, uint32_t soff) {
    __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(lds), "v"(voff),
                     "s"(rsrc), "s"(soff)
                     : "memory", "m0");
}
__device__ __forceinline__ void load_to_lds4(v4i rsrc, uint32_t lds, uint32_t voff, uint32_t soff) {
    __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds" ::"s"(lds), "v"(voff),
                     "s"(rsrc), "s"(soff)
                     : "memory", "m0");
}

// Waits until at most LEFT of this wavefront's global loads are on their way and
// all its LDS accesses are done, then joins the workgroup. Unlike
// __syncthreads() it leaves the newest loads in flight.
template <int LEFT>
__device__ __forceinline__ void join_with_loads_left() {
    static_assert(LEFT < 64, "the counter has six bits");
    __asm__ volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LEFT) : "memory");
}

// f32 -> bf16 bits, round half to even (the hardware conversion of gfx950).
__device__ __forceinline__ uint32_t bf16_bits(float f) {
    return __builtin_bit_cast(uint16_t, (__bf16)f);
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) { return bf16_bits(lo) | (bf16_bits(hi) << 16); }

// Element i of an array of float32 or bfloat16.
template <bool BF16>
__device__ __forceinline__ float load_as_float(const void* p, long long i) {
    if (BF16) return bf16_to_float(static_cast<const uint16_t*>(p)[i]);
    return static_cast<const float*>(p)[i];
}

// Eight consecutive elements that start on 16 bytes.
template <bool BF16>
__device__ __forceinline__ void load8_aligned(const void* p, long long at, float* v) {
    if (BF16) {
        const uint4 x = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_to_float(w[i] & 0xFFFFu);
            v[2 * i + 1] = bf16_to_float(w[i] >> 16);
        }
    } else {
        const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
        const float4 x = q[0], y = q[1];
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
        v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
    }
}

// Maximum over the 16 lanes of a DPP row (quad permutes, row mirrors).
__device__ __forceinline__ float row_max16(float v) {
    v = fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0xB1, 0xF, 0xF, false)));
    v = fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x4E, 0xF, 0xF, false)));
    v = fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x141, 0xF, 0xF, false)));
    v = fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x140, 0xF, 0xF, false)));
    return v;
}

// The same for unsigned integers: of magnitude() bits, which order as the values do with NaN above infinity.
__device__ __forceinline__ uint32_t row_max16(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));
    return v;
}
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// ---- e4m3 -------------------------------------------------------------------

constexpr float F8_TOP = 448.0f;

// The quotient v / s that is rounded to a code: float32, correctly rounded,
// cut at +-448 (a scale that is subnormal can be coarse enough to exceed it);
// 0 where the scale is 0. A NaN passes.
__device__ __forceinline__ float f8_quotient(float v, float s) {
    float r = v / s;
    if (fabsf(r) > F8_TOP) r = copysignf(F8_TOP, r);
    return s == 0.0f ? (v == v ? 0.0f : v) : r;
}

// Inverse of a block's scale for the fast path of f8_codes4, 0 where that must
// not be used (scales near the ends of float32, zero, infinity, NaN).
__device__ __forceinline__ float f8_inverse(float s) {
    return s >= 0x1p-100f && s <= 0x1p100f ? __builtin_amdgcn_rcpf(s) : 0.0f;
}

// Four codes of four quotients (hardware conversion, round half to even).
__device__ __forceinline__ uint32_t f8_pack4(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// Codes of four values under scale s: e4m3 of the correctly rounded float32
// quotients. v * rcp(s) is within 2^-22 of itself from the quotient (v_rcp_f32 is
// good to one ulp); if both ends of an interval of 2^-21 round to the same codes,
// those are the codes, and the division (ten instructions a value) is left to
// the few that lie near a tie.
__device__ __forceinline__ uint32_t f8_codes4(const float* v, float s, float inv) {
    const float a = v[0] * inv, b = v[1] * inv, c = v[2] * inv, d = v[3] * inv;
    constexpr float LO = 1.0f - 0x1p-21f, HI = 1.0f + 0x1p-21f;
    const uint32_t lo = f8_pack4(a * LO, b * LO, c * LO, d * LO), hi = f8_pack4(a * HI, b * HI, c * HI, d * HI);
    if (lo == hi && inv != 0.0f) return lo;
    return f8_pack4(f8_quotient(v[0], s), f8_quotient(v[1], s), f8_quotient(v[2], s), f8_quotient(v[3], s));
}

}  // namespace q4
