// spin_kv_append kernel: the rows that qkv_proj wrote, turned into rotated
// queries and into codes in a paged KV cache, in one pass.
//
// For a query or key vector x of 128 values
//   x <- x / sqrt(mean(x^2) + eps) * w        where a norm weight is given
//   (a, b) <- (a cos - b sin, b cos + a sin)  on the first rot_dim values, pairs
//                                             (i, i + rot_dim / 2) or (2 i, 2 i + 1)
//   y = x . H_128 / sqrt(128)                 R3, page "SpinQuant, Reproduced", Q5
// queries are written as fp16, keys as codes of fl32(y) by the rules of
// spin_kv_quant, values as codes of themselves.
//
// Bound: HBM.  A vector is read once (256 or 512 bytes) and written once.
//
// Keys are held in 64 bits from the load to fl32(y).  A code is decided by
// which side of a border fl32(y) / s lies on, and with 24-bit sums about one
// code in 10^6 falls on the other side, by the order of the sums; with 53 bits
// the codes are those of the exact value.  The fp64 vector rate equals the
// fp32 one here, so this costs the doubled registers and cross-lane moves of
// a sixth of the vectors (at 32 query and 8 key heads).  Queries are rounded to
// fp16 at the end and are held in float32; the sum of their squares is not, so
// that no fp32 input overflows it.
//
// Layout: one vector per 16 lanes, 8 consecutive values each, as in kv_quant;
// a workgroup's 16 vectors are all keys, all values or all queries.
#include "kv_batch.h"
#include "kv_common.h"
#include "spin_internal.h"

namespace spin {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kAppendVectors = kAppendThreads / 16;

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __uint_as_float(__builtin_amdgcn_mov_dpp(static_cast<int>(__float_as_uint(v)), CTRL, 0xF, 0xF, true));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
    const unsigned long long u = __double_as_longlong(v);
    const unsigned lo = __builtin_amdgcn_mov_dpp(static_cast<int>(u), CTRL, 0xF, 0xF, true);
    const unsigned hi = __builtin_amdgcn_mov_dpp(static_cast<int>(u >> 32), CTRL, 0xF, 0xF, true);
    return __longlong_as_double((static_cast<unsigned long long>(hi) << 32) | lo);
}

// The value of lane l ^ MASK of the 16 lanes, MASK = 1, 2, 4 or 8: quad
// permutations, a half-row mirror (^ 7) followed by a quad mirror (^ 3), a
// rotation by 8.
template <int MASK, typename F>
__device__ __forceinline__ F lane_xor(F v) {
    if (MASK == 1) return dpp<0xB1>(v);
    if (MASK == 2) return dpp<0x4E>(v);
    if (MASK == 4) return dpp<0x1B>(dpp<0x141>(v));
    return dpp<0x128>(v);
}

template <typename F>
__device__ __forceinline__ F fused(F a, F b, F c);
template <>
__device__ __forceinline__ float fused(float a, float b, float c) { return __builtin_fmaf(a, b, c); }
template <>
__device__ __forceinline__ double fused(double a, double b, double c) { return __builtin_fma(a, b, c); }

template <int MASK, typename F>
__device__ __forceinline__ void lane_level(F* v, int l) {
    const F sign = (l & MASK) ? F(-1) : F(1);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = fused(v[j], sign, lane_xor<MASK>(v[j]));
}

// v <- v . H_128 (not normalised), lane l holding values 8 l .. 8 l + 7.
template <typename F>
__device__ __forceinline__ void wht128(F* v, int l) {
#pragma unroll
    for (int h = 1; h < 8; h <<= 1) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j & h) continue;
            const F a = v[j], b = v[j + h];
            v[j] = a + b;
            v[j + h] = a - b;
        }
    }
    lane_level<1>(v, l);
    lane_level<2>(v, l);
    lane_level<4>(v, l);
    lane_level<8>(v, l);
}

// Norm, position rotation and Hadamard of the vector at x, in the precision F.
template <typename F, typename TIn>
__device__ __forceinline__ void turned(const TIn* __restrict__ x, const float* __restrict__ weight, double eps,
                                       const float* __restrict__ rope_row, int rot_dim, bool interleaved, int l, F* v) {
    float raw[8];
    load8<TIn>(x + 8 * l, raw);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = raw[j];
    F r = F(1);
    if (weight) {
        double sum = 0.0;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = __builtin_fma(static_cast<double>(raw[j]), static_cast<double>(raw[j]), sum);
        sum += lane_xor<1>(sum);
        sum += lane_xor<2>(sum);
        sum += lane_xor<4>(sum);
        sum += lane_xor<8>(sum);
        r = static_cast<F>(1.0 / sqrt(sum * (1.0 / 128.0) + eps));
        float w[8];
        load8<float>(weight + 8 * l, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = v[j] * r * F(w[j]);
    }
    if (8 * l < rot_dim) {
        const int n = rot_dim >> 1;
        if (interleaved) {
            const float4 c4 = *reinterpret_cast<const float4*>(rope_row + 4 * l);
            const float4 s4 = *reinterpret_cast<const float4*>(rope_row + n + 4 * l);
            const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const F a = v[2 * i], b = v[2 * i + 1];
                v[2 * i] = fused(a, F(c[i]), -(b * F(s[i])));
                v[2 * i + 1] = fused(b, F(c[i]), a * F(s[i]));
            }
        } else {
            // n is a multiple of 8: the eight values lie in one half, their partners in the other
            const bool low = 8 * l < n;
            const int at = low ? 8 * l : 8 * l - n, other = low ? 8 * l + n : 8 * l - n;
            float c[8], s[8], p[8], w[8];
            load8<float>(rope_row + at, c);
            load8<float>(rope_row + n + at, s);
            load8<TIn>(x + other, p);
            if (weight) load8<float>(weight + other, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                F b = p[j];
                if (weight) b = b * r * F(w[j]);
                v[j] = fused(v[j], F(c[j]), low ? -(b * F(s[j])) : b * F(s[j]));
            }
        }
    }
    wht128<F>(v, l);
}

// Where token t's vector goes: its position, and the page and slot that hold it.
struct Place {
    bool in_batch;      // the row belongs to a sequence
    long long pos;      // position within the sequence's own pages, -1 if there is none
    int page;           // -1 if there is none
    int slot;
};

__device__ __forceinline__ Place find_place(const KvAppendArgs& a, int t, int l) {
    Place p = {false, -1, -1, 0};
    const int b = find_sequence16(a.q_start, a.B, t, l);
    if (b < 0) return p;
    p.in_batch = true;
    const long long pos = static_cast<long long>(a.kv_len[b]) - a.q_start[b + 1] + t;
    if (pos < 0 || pos >= static_cast<long long>(a.max_pages) << a.page_log2) return p;
    if (a.rope && pos + a.pos0 >= a.rope_len) return p;
    p.pos = pos;
    const int page = a.page_table[static_cast<long long>(b) * a.max_pages + (pos >> a.page_log2)];
    p.page = page >= 0 && page < a.n_pages ? page : -1;
    p.slot = static_cast<int>(pos & ((1 << a.page_log2) - 1));
    return p;
}

// Codes and scale of eight values of a vector, written where the cache holds them.
template <int BITS, bool IS_V>
__device__ __forceinline__ void put_codes(const KvAppendArgs& a, const float* y, const Place& p, int h, int l) {
    float mx = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) mx = __builtin_fmaxf(mx, __builtin_fabsf(y[j]));
    const __half s16 = kv_scale<BITS>(row16_max(mx));
    const float sf = __half2float(s16);
    const long long head = static_cast<long long>(p.page) * a.Hkv + h;   // (page, head)
    const long long token = (head << a.page_log2) + p.slot;
    uint8_t* codes = IS_V ? a.V_codes + (((token >> 2) * 16 + l) * 4 + (p.slot & 3)) * BITS
                          : a.K_codes + (token * 16 + l) * BITS;
    if (BITS == 4)
        *reinterpret_cast<uint32_t*>(codes) = kv_codes(y, 1.0f, 1.0f, sf);
    else
        *reinterpret_cast<uint2*>(codes) = kv_codes8(y, 1.0f, 1.0f, sf);
    if (l == 0) (IS_V ? a.V_scale : a.K_scale)[token] = __half_as_ushort(s16);
}

template <int BITS, typename TIn>
__global__ __launch_bounds__(kAppendThreads) void kv_append_kernel(KvAppendArgs a) {
    const int l = threadIdx.x & 15;
    long long block = blockIdx.x;
    const int kind = block < a.kv_blocks ? 0 : block < 2 * a.kv_blocks ? 1 : 2;   // keys, values, queries
    block -= kind * a.kv_blocks;
    const int H = kind == 2 ? a.Hq : a.Hkv;
    const long long g = block * kAppendVectors + (threadIdx.x >> 4);
    if (g >= static_cast<long long>(a.T) * H) return;   // the 16 lanes of a vector leave together
    const int t = static_cast<int>(g / H), h = static_cast<int>(g - static_cast<long long>(t) * H);
    const Place p = find_place(a, t, l);
    if (kind == 2) {
        if (!p.in_batch) return;
        float v[8] = {};
        if (p.pos >= 0)
            turned<float, TIn>(static_cast<const TIn*>(a.Q) + t * a.q_stride + h * 128, a.q_norm, a.eps,
                               a.rope + (p.pos + a.pos0) * a.rot_dim, a.rot_dim, a.interleaved, l, v);
        union { _Float16 f[8]; uint4 u; } out;
#pragma unroll
        for (int j = 0; j < 8; ++j) out.f[j] = static_cast<_Float16>(v[j] * a.norm);
        *reinterpret_cast<uint4*>(a.Q_out + g * 128 + 8 * l) = out.u;
        return;
    }
    if (p.pos < 0 || p.page < 0) return;
    float y[8];
    if (kind == 0) {
        double v[8];
        turned<double, TIn>(static_cast<const TIn*>(a.K) + t * a.k_stride + h * 128, a.k_norm, a.eps,
                            a.rope + (p.pos + a.pos0) * a.rot_dim, a.rot_dim, a.interleaved, l, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = static_cast<float>(v[j] * 0.08838834764831844055);   // 1 / sqrt(128)
        put_codes<BITS, false>(a, y, p, h, l);
    } else {
        load8<TIn>(static_cast<const TIn*>(a.V) + t * a.v_stride + h * 128 + 8 * l, y);
        put_codes<BITS, true>(a, y, p, h, l);
    }
}

template <int BITS>
hipError_t launch_bits(const KvAppendArgs& a, bool x_f16, long long blocks, hipStream_t s) {
    if (x_f16)
        hipLaunchKernelGGL((kv_append_kernel<BITS, __half>), dim3(static_cast<unsigned>(blocks)), dim3(kAppendThreads), 0, s, a);
    else
        hipLaunchKernelGGL((kv_append_kernel<BITS, float>), dim3(static_cast<unsigned>(blocks)), dim3(kAppendThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace

long long kv_append_blocks(int T, int Hq, int Hkv) {
    const long long kv = (static_cast<long long>(T) * Hkv + kAppendVectors - 1) / kAppendVectors;
    return 2 * kv + (static_cast<long long>(T) * Hq + kAppendVectors - 1) / kAppendVectors;
}

hipError_t launch_kv_append(KvAppendArgs a, bool x_f16, int bits, hipStream_t s) {
    a.kv_blocks = (static_cast<long long>(a.T) * a.Hkv + kAppendVectors - 1) / kAppendVectors;
    a.norm = static_cast<float>(1.0 / __builtin_sqrt(128.0));
    const long long blocks = kv_append_blocks(a.T, a.Hq, a.Hkv);
    if (blocks == 0) return hipSuccess;
    return bits == 8 ? launch_bits<8>(a, x_f16, blocks, s) : launch_bits<4>(a, x_f16, blocks, s);
}

}  // namespace spin
