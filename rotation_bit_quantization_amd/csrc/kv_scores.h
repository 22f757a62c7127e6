// What the kernels that score cached keys share: codes as matrix operands, sums
// over the lanes of a token, and what turns a product into a score (its cap and
// the numbers that it is held to).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace spin {
namespace {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
// Caps up to this one go by capped_plus, whose error is that of a number of the cap's size, above by capped_wide, which is
// ten operations longer (8 tokens on 32768, INT8, cap 50: 108 and 111 us; 1723 in chunks, cap 30 and a bias: 160 and 191).
constexpr float kNearCap = 64.0f;

union Frag {
    uint32_t w[4];
    h8 v;
};

// Two fp16 integers 1024 + u (u in the low bits of each half) minus `off`: exact.
__device__ __forceinline__ uint32_t minus(uint32_t x, float off) {
    const h2 o = {static_cast<_Float16>(-off), static_cast<_Float16>(-off)};
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(h2, x) + o);
}

// Eight codes of one token as an operand.  The order of the eight within the
// operand (order8) is the one that needs fewest instructions; queries are
// loaded in the same order.
template <int BITS>
__device__ __forceinline__ int order8(int i) {
    // 4 bits: 0 4 1 5 2 6 3 7;  8 bits: 0 2 1 3 4 6 5 7
    if (BITS == 4) return (i >> 1) + 4 * (i & 1);
    return (i & 4) + ((i & 2) >> 1) + 2 * (i & 1);
}
template <int BITS>
__device__ __forceinline__ h8 key_operand(const uint32_t* w) {
    Frag f;
    if (BITS == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f.w[i] = minus(((w[0] >> (4 * i)) & 0x000F000Fu) ^ 0x64086408u, 1032.0f);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) f.w[i] = minus(((w[i >> 1] >> (8 * (i & 1))) & 0x00FF00FFu) ^ 0x64806480u, 1152.0f);
    }
    return f.v;
}

// The same without the subtraction: u = code + 8 (128) as the fp16 number u 2^-24, subnormal, which the matrix cores
// take as it is.  The sum over a query is then 2^-24 (sum q code + 8 sum q): the second term goes into the accumulator
// that the sum starts from.  The matrix cores align subnormal operands as if their leading bit were there: at queries of 2 a
// sum of 128 products is off by 3e-4 (rms, 4-bit codes) in place of 1e-6, a score by about 1e-5, far below what weights
// rounded to fp16 tell apart.
template <int BITS>
__device__ __forceinline__ h8 key_operand_small(const uint32_t* w) {
    Frag f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f.w[i] = BITS == 4 ? ((w[0] >> (4 * i)) & 0x000F000Fu) ^ 0x00080008u
                           : ((w[i >> 1] >> (8 * (i & 1))) & 0x00FF00FFu) ^ 0x00800080u;
    return f.v;
}

__device__ __forceinline__ float max_over_groups(float v) {   // lanes l, l ^ 16, l ^ 32, l ^ 48
    u2 s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __builtin_fmaxf(__uint_as_float(s.x), __uint_as_float(s.y));
    s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __builtin_fmaxf(__uint_as_float(s.x), __uint_as_float(s.y));
}
__device__ __forceinline__ float sum_over_groups(float v) {
    u2 s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(s.x) + __uint_as_float(s.y);
    s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(s.x) + __uint_as_float(s.y);
}

// A capped score in the exponent: cap log2(e) tanh(z / cap) = top - 2 top / (2^y + 1), y = 2 log2(e) z / cap, right at
// both infinities.  `lm` is what is added to it, `top` = cap log2(e) already among it.  The two terms are of the size of
// the cap whatever the score is, so that their roundings are: ten of 2^-24 cap (2^-21.7 cap measured).  At caps up to
// kNearCap that is below a twelfth of the rounding of the weight to fp16.
__device__ __forceinline__ float capped_plus(float y, float top, float lm) {
    return __builtin_fmaf(__builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(y) + 1.0f), -2.0f * top, lm);
}

// The same for any cap, off by at most 2^-18 of the score: z tanh(u) / u by its series (the next term is 2^-26 at 1/4)
// where |u| = |z| / cap is small, the form above where the score is a quarter of the cap or more.  z in units of
// 1 / log2(e), `rtop` = 1 / top.
__device__ __forceinline__ float capped_wide(float z, float top, float rtop) {
    const float u = z * rtop, u2 = u * u;
    float p = __builtin_fmaf(u2, 62.0f / 2835.0f, -17.0f / 315.0f);
    p = __builtin_fmaf(p, u2, 2.0f / 15.0f);
    p = __builtin_fmaf(p, u2, -1.0f / 3.0f);
    p = __builtin_fmaf(p, u2, 1.0f);
    const float far = __builtin_fmaf(__builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(u * (2.0f * kLog2e)) + 1.0f), -2.0f * top, top);
    return __builtin_fabsf(u) < 0.25f ? z * p : far;
}

// What a kernel does to the scores: nothing; a distance bias, a cap up to kNearCap, or both; a cap above, with or without
// a bias; a cap up to kNearCap and surely no bias.
enum Scores { kPlain, kFancy, kWideCap, kCapped };
constexpr bool biased(int scores) { return scores == kFancy || scores == kWideCap; }

// A factor of scores within the numbers that keep them finite.  Products are multiples of 2^-48, or zero: scores that this
// brings down still lie past every cap up to kNearCap, or so far apart that their roundings, 2^-24 of them, are past what
// weights tell apart.  In a scalar register: as a vector one it makes kv_attn_tile spill four more (chunks 159 -> 162 us).
__device__ __forceinline__ float held(float factor) {
    factor = __builtin_fminf(__builtin_fmaxf(factor, -0x1p100f), 0x1p100f);
    return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(factor)));
}

// How a score is capped: the factor of a product and its key's scale, the cap in units of 1 / log2(e) (0: none) and its
// reciprocal.
struct Cap {
    float factor, top, rtop;
};
template <int SCORES, typename Args>
__device__ __forceinline__ Cap cap_of(const Args& a) {
    if (SCORES == kWideCap) {
        const float top = __builtin_fminf(a.softcap * kLog2e, 0x1p126f);       // its double has to be finite
        return {a.scale * kLog2e, top, 1.0f / top};
    }
    const bool capped = SCORES == kCapped || (SCORES == kFancy && a.softcap > 0.0f);
    return {capped ? 2.0f * kLog2e * (a.scale / a.softcap) : a.scale * kLog2e, capped ? a.softcap * kLog2e : 0.0f, 0.0f};
}

// Tokens of sequence b that its table has room for.
template <typename Args>
__device__ __forceinline__ int context(const Args& a, int b) {
    return min(max(a.kv_len[b], 0), a.max_pages << a.page_log2);
}

// A border of the batch, held to its T rows.
__device__ __forceinline__ int within(int row, int T) { return min(max(row, 0), T); }

}  // namespace
}  // namespace spin
