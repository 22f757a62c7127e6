// What the kernels that write the KV cache share: 8-value loads, the fp16
// scale of a vector and the codes of eight of its values (the rules of
// spin_kv_quant / spin_kv_quant8 in include/libspin.h).
#pragma once

#include "spin_device.h"

namespace spin {

template <typename TIn>
__device__ __forceinline__ void load8(const TIn* p, float* v);

template <>
__device__ __forceinline__ void load8<__half>(const __half* p, float* v) {
    const uint4 raw = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __half2float(__ushort_as_half(static_cast<unsigned short>(w[i] & 0xFFFFu)));
        v[2 * i + 1] = __half2float(__ushort_as_half(static_cast<unsigned short>(w[i] >> 16)));
    }
}

template <>
__device__ __forceinline__ void load8<float>(const float* p, float* v) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// Quantize eight held values z (true value = sign * z * norm) of one vector
// whose fp16 scale is s16: returns one dword of codes.  Fast path when s16 is
// a normal fp16 (then |y / s16| < 7.5 so no clamp is needed and the
// magic-number estimate plus exact near-tie fallback applies; 1/s16 from
// v_rcp_f32 keeps the estimate well inside the fallback window); otherwise the
// exact quotient and clamp.
__device__ __forceinline__ uint32_t kv_codes(const float* z, float sign, float norm, float sf) {
    if (sf >= 0x1p-14f && sf <= 65504.0f) {
        const float cr = sign * (norm * __builtin_amdgcn_rcpf(sf));
        uint32_t f[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = __float_as_uint(__builtin_fmaf(z[k], cr, kQuantMagic));
        const uint32_t m01 = min(f[0] & 0xFFFFu, f[1] & 0xFFFFu), m23 = min(f[2] & 0xFFFFu, f[3] & 0xFFFFu);
        const uint32_t m45 = min(f[4] & 0xFFFFu, f[5] & 0xFFFFu), m67 = min(f[6] & 0xFFFFu, f[7] & 0xFFFFu);
        if (min(min(m01, m23), min(m45, m67)) >= 3u) {
            const uint32_t ev = __builtin_amdgcn_perm(__builtin_amdgcn_perm(f[6], f[4], 0x0c0c0602u),
                                                      __builtin_amdgcn_perm(f[2], f[0], 0x0c0c0602u), 0x05040100u);
            const uint32_t od = __builtin_amdgcn_perm(__builtin_amdgcn_perm(f[7], f[5], 0x0c0c0602u),
                                                      __builtin_amdgcn_perm(f[3], f[1], 0x0c0c0602u), 0x05040100u);
            return (ev & 0x0F0F0F0Fu) | ((od << 4) & 0xF0F0F0F0u);
        }
    }
    int c8[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) c8[k] = quant_exact((z[k] * sign) * norm, sf);
    return pack8(c8);
}

// The 8-bit variant of kv_codes: two dwords of byte codes.
__device__ __forceinline__ uint2 kv_codes8(const float* z, float sign, float norm, float sf) {
    if (sf >= 0x1p-14f && sf <= 65504.0f) {
        const float cr = sign * (norm * __builtin_amdgcn_rcpf(sf));
        uint32_t f[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = __float_as_uint(__builtin_fmaf(z[k], cr, kQuant8Magic));
        if (!any_near_tie8(f)) return make_uint2(pack4_magic8(f), pack4_magic8(f + 4));
    }
    int c8[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) c8[k] = quant_exact8((z[k] * sign) * norm, sf);
    return make_uint2(pack4b(c8), pack4b(c8 + 4));
}

// The fp16 scale of a vector whose largest magnitude is mx: fp16_rne(fl32(mx /
// 7)), or 127 at 8 bits.
template <int BITS>
__device__ __forceinline__ __half kv_scale(float mx) {
    // Any absmax above 65504 * 7 rounds to an fp16 infinity; clamping
    // at 2^100 keeps that result for an infinite absmax, whose
    // remainder step in div_by_qmax would otherwise give NaN.
    mx = __builtin_fminf(mx, 0x1p100f);
    return __float2half_rn(BITS == 4 ? div_by_qmax(mx, kSeven, kRcpSeven) : div_by_qmax(mx, kQmax8, kRcpQmax8));
}

}  // namespace spin
