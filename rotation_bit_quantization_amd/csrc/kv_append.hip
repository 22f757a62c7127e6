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
// Bound: HBM at many tokens.  A vector is read once (256 or 512 bytes) and
// written once.  Measured with 32 + 8 heads of float32, norms and the whole head
// rotated: 8192 tokens 61 us (280 MB, 4.6 TB/s, what a copy of them takes); 1037
// tokens of 32 + 32 heads of fp16 18 us (43 MB, 2.4 TB/s: a third of the vectors
// are keys in 64 bits, and a launch's 4 us are a good part); 16 tokens 4.8 us.
//
// Keys are held in 64 bits from the load to fl32(y).  A code is decided by
// which side of a border fl32(y) / s lies on, and with 24-bit sums about one
// code in 10^6 falls on the other side, by the order of the sums; with 53 bits
// the codes are those of the exact value.  The fp64 vector rate equals the
// fp32 one here, so this costs the doubled registers and cross-lane moves of
// a sixth of the vectors (at 32 query and 8 key heads), which load and derive
// everything of 64 bits anew for every head to stay at 82 registers.  Queries are rounded to
// fp16 at the end and are held in float32; the sum of their squares is not, so
// that no fp32 input overflows it.
//
// Layout: one vector at a time per 16 lanes, 8 consecutive values each, as in
// kv_quant; a lane group takes up to kMostHeads heads of one token, one after
// the other, so that its place in the batch, its page and its cosines are
// looked up once.  A workgroup's 16 groups hold keys, values or queries only.
#include "kv_batch.h"
#include "kv_common.h"
#include "spin_internal.h"

namespace spin {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kAppendVectors = kAppendThreads / 16;
constexpr int kMostHeads = 4;

// The 16 lanes of a vector exchange values along l ^ 1, l ^ 2, l ^ 7 and l ^ 8,
// each one DPP operand (l ^ 4 would take two): the lanes are numbered by a, with
// l = a_0 1 ^ a_1 2 ^ a_2 7 ^ a_3 8, which butterflies on a_0 .. a_3 transform
// as well as any other numbering.  Lane l then holds the result's octet
// out_octet(l), the k whose signs (-1)^<k, m> are those of (-1)^<a(l), a(m)>.
enum { kXor1 = 0xB1, kXor2 = 0x4E, kXor7 = 0x141, kXor8 = 0x128 };   // quad permutations, half-row mirror, row rotation

__device__ __forceinline__ int out_octet(int l) {
    const int b0 = l & 1, b1 = l >> 1 & 1, b2 = l >> 2 & 1;
    return (b0 ^ b2) | (b1 ^ b2) << 1 | (b0 ^ b1 ^ b2) << 2 | (l & 8);
}

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

__device__ __forceinline__ float fused(float a, float b, float c) { return __builtin_fmaf(a, b, c); }
__device__ __forceinline__ double fused(double a, double b, double c) { return __builtin_fma(a, b, c); }

// The four butterflies across lanes.  A level makes v + x of one lane of a pair
// and x - v of the other, x its partner's; the second is held negated, v - x,
// which makes each value one multiply-add with the partner as an operand.
// Later levels pair lanes of equal sign, so the signs leave together: the
// product of the four is the result's.
__device__ __forceinline__ double lane_levels(double* v, int l) {
    const int b2 = l >> 2 & 1;
    const double s1 = (l & 1) ^ b2 ? -1 : 1, s2 = (l >> 1 & 1) ^ b2 ? -1 : 1, s7 = b2 ? -1 : 1, s8 = l & 8 ? -1 : 1;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = fused(dpp<kXor1>(v[j]), s1, v[j]);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = fused(dpp<kXor2>(v[j]), s2, v[j]);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = fused(dpp<kXor7>(v[j]), s7, v[j]);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = fused(dpp<kXor8>(v[j]), s8, v[j]);
    return s1 * s2 * s7 * s8;
}
#define SPIN_LEVEL(at, sign)                                                                                      \
    "v_fmac_f32_dpp %0, %0, " sign " " at " row_mask:0xf bank_mask:0xf bound_ctrl:0\n\t"                          \
    "v_fmac_f32_dpp %1, %1, " sign " " at " row_mask:0xf bank_mask:0xf bound_ctrl:0\n\t"                          \
    "v_fmac_f32_dpp %2, %2, " sign " " at " row_mask:0xf bank_mask:0xf bound_ctrl:0\n\t"                          \
    "v_fmac_f32_dpp %3, %3, " sign " " at " row_mask:0xf bank_mask:0xf bound_ctrl:0\n\t"                          \
    "v_fmac_f32_dpp %4, %4, " sign " " at " row_mask:0xf bank_mask:0xf bound_ctrl:0\n\t"                          \
    "v_fmac_f32_dpp %5, %5, " sign " " at " row_mask:0xf bank_mask:0xf bound_ctrl:0\n\t"                          \
    "v_fmac_f32_dpp %6, %6, " sign " " at " row_mask:0xf bank_mask:0xf bound_ctrl:0\n\t"                          \
    "v_fmac_f32_dpp %7, %7, " sign " " at " row_mask:0xf bank_mask:0xf bound_ctrl:0\n\t"
// In float32 as the one instruction a value that it is; the compiler takes two.  A DPP operand is read two wait states
// after its write at the earliest: the s_nop sees to that for the first level, seven other values for the later ones.
__device__ __forceinline__ float lane_levels(float* v, int l) {
    const int b2 = l >> 2 & 1;
    const float s1 = (l & 1) ^ b2 ? -1 : 1, s2 = (l >> 1 & 1) ^ b2 ? -1 : 1, s7 = b2 ? -1 : 1, s8 = l & 8 ? -1 : 1;
    asm("s_nop 1\n\t" SPIN_LEVEL("quad_perm:[1,0,3,2]", "%8") SPIN_LEVEL("quad_perm:[2,3,0,1]", "%9")
            SPIN_LEVEL("row_half_mirror", "%10") SPIN_LEVEL("row_ror:8", "%11")
        : "+v"(v[0]), "+v"(v[1]), "+v"(v[2]), "+v"(v[3]), "+v"(v[4]), "+v"(v[5]), "+v"(v[6]), "+v"(v[7])
        : "v"(s1), "v"(s2), "v"(s7), "v"(s8));
    return s1 * s2 * s7 * s8;
}
#undef SPIN_LEVEL

// v <- v . H_128 (not normalised), lane l holding values 8 l .. 8 l + 7 and then
// those of octet out_octet(l), times the sign that is returned.
template <typename F>
__device__ __forceinline__ F wht128(F* v, int l) {
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
    return lane_levels(v, l);
}

// The position rotation of a token: value j becomes v[j] c[j] + partner s[j].
struct Turn {
    float c[8], s[8];
    int other;          // pairs in two halves: where the partners begin
};

__device__ __forceinline__ Turn load_turn(const float* __restrict__ rope_row, int rot_dim, bool interleaved, int l) {
    Turn r = {};
    if (8 * l >= rot_dim) return r;
    const int n = rot_dim >> 1;
    if (interleaved) {
        const float4 c = *reinterpret_cast<const float4*>(rope_row + 4 * l);
        const float4 s = *reinterpret_cast<const float4*>(rope_row + n + 4 * l);
        const float c4[4] = {c.x, c.y, c.z, c.w}, s4[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r.c[2 * i] = r.c[2 * i + 1] = c4[i];
            r.s[2 * i] = -s4[i];
            r.s[2 * i + 1] = s4[i];
        }
    } else {
        // n is a multiple of 8: the eight values lie in one half, their partners in the other
        const bool low = 8 * l < n;
        const int at = low ? 8 * l : 8 * l - n;
        load8<float>(rope_row + at, r.c);
        load8<float>(rope_row + n + at, r.s);
#pragma unroll
        for (int j = 0; j < 8; ++j) r.s[j] = low ? -r.s[j] : r.s[j];
        r.other = low ? 8 * l + n : 8 * l - n;
    }
    return r;
}

// 1 / sqrt(x), in the precision F.  The hardware's estimate has about 2^-24; one
// step of y (3 - x y^2) / 2 leaves far less than a float32 rounding.
__device__ __forceinline__ void rsqrt_of(double x, double* r) { *r = 1.0 / sqrt(x); }
__device__ __forceinline__ void rsqrt_of(double x, float* r) {
    const double y = __builtin_amdgcn_rsq(x);
    *r = static_cast<float>(y * __builtin_fma(-0.5 * x * y, y, 1.5));
}

// Norm, position rotation and Hadamard of the vector at x, in the precision F.  Returns the result's sign.
template <typename F, typename TIn>
__device__ __forceinline__ F turned(const TIn* __restrict__ x, const float* __restrict__ weight, double eps,
                                    const Turn& turn, int rot_dim, bool interleaved, int l, F* v) {
    float raw[8];
    load8<TIn>(x + 8 * l, raw);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = raw[j];
    F r = F(1);
    if (weight) {
        double sum = 0.0;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = __builtin_fma(static_cast<double>(raw[j]), static_cast<double>(raw[j]), sum);
        sum += dpp<kXor1>(sum);
        sum += dpp<kXor2>(sum);
        sum += dpp<kXor7>(sum);
        sum += dpp<kXor8>(sum);
        rsqrt_of(sum * (1.0 / 128.0) + eps, &r);
        float w[8];
        load8<float>(weight + 8 * l, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = v[j] * r * F(w[j]);
    }
    if (8 * l < rot_dim) {
        if (interleaved) {
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const F a = v[j], b = v[j + 1];
                v[j] = fused(a, F(turn.c[j]), b * F(turn.s[j]));
                v[j + 1] = fused(b, F(turn.c[j + 1]), a * F(turn.s[j + 1]));
            }
        } else if (rot_dim == 128) {   // the partners are those of lane l ^ 8
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = fused(dpp<kXor8>(v[j]), F(turn.s[j]), v[j] * F(turn.c[j]));
        } else {
            float p[8], w[8];
            load8<TIn>(x + turn.other, p);
            if (weight) load8<float>(weight + turn.other, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                F b = p[j];
                if (weight) b = b * r * F(w[j]);
                v[j] = fused(b, F(turn.s[j]), v[j] * F(turn.c[j]));
            }
        }
    }
    return wht128<F>(v, l);
}

// Where token t's vector goes: its position, and the page and slot that hold it.
struct Place {
    bool in_batch;      // the row belongs to a sequence
    long long pos;      // position within the sequence's own pages, -1 if there is none
    long long turn;     // position that it is turned by, its row of the rotary table
    int page;           // -1 if there is none
    int slot;
};

__device__ __forceinline__ Place find_place(const KvAppendArgs& a, int t, int l) {
    Place p = {false, -1, 0, -1, 0};
    const int b = find_sequence16(a.q_start, a.B, t, l);
    if (b < 0) return p;
    p.in_batch = true;
    const long long pos = static_cast<long long>(placed(a.kv_len[b])) - a.q_start[b + 1] + t;
    if (pos < 0 || pos >= static_cast<long long>(a.max_pages) << a.page_log2) return p;
    p.turn = a.positions ? a.positions[t] : pos + a.pos0;
    if (a.rope && (p.turn < 0 || p.turn >= a.rope_len)) return p;
    p.pos = pos;
    const int page = a.page_table[static_cast<long long>(b) * a.max_pages + (pos >> a.page_log2)];
    p.page = page >= 0 && page < a.n_pages ? page : -1;
    p.slot = static_cast<int>(pos & ((1 << a.page_log2) - 1));
    return p;
}

// Codes and scale of a vector's values 8 o .. 8 o + 7 of head h, written where the cache holds them.
template <int BITS, bool IS_V>
__device__ __forceinline__ void put_codes(const KvAppendArgs& a, const float* y, const Place& p, int h, int o) {
    float mx = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) mx = __builtin_fmaxf(mx, __builtin_fabsf(y[j]));
    const __half s16 = kv_scale<BITS>(row16_max(mx));
    const float sf = __half2float(s16);
    const long long head = static_cast<long long>(p.page) * a.Hkv + h;   // (page, head)
    const long long token = (head << a.page_log2) + p.slot;
    uint8_t* codes = IS_V ? a.V_codes + (((token >> 2) * 16 + o) * 4 + (p.slot & 3)) * BITS
                          : a.K_codes + (token * 16 + o) * BITS;
    if (BITS == 4)
        *reinterpret_cast<uint32_t*>(codes) = kv_codes(y, 1.0f, 1.0f, sf);
    else
        *reinterpret_cast<uint2*>(codes) = kv_codes8(y, 1.0f, 1.0f, sf);
    if (o == 0) (IS_V ? a.V_scale : a.K_scale)[token] = __half_as_ushort(s16);
}

template <int BITS, typename TIn>
__global__ __launch_bounds__(kAppendThreads, 4) void kv_append_kernel(KvAppendArgs a) {
    const int l = threadIdx.x & 15;
    unsigned block = blockIdx.x;
    const int kind = block < a.kv_blocks ? 0 : block < 2 * a.kv_blocks ? 1 : 2;   // keys, values, queries
    block -= kind * a.kv_blocks;
    const int H = kind == 2 ? a.Hq : a.Hkv;
    const unsigned per_token = (H + a.heads - 1) / a.heads;
    const unsigned g = block * kAppendVectors + (threadIdx.x >> 4);
    const unsigned t = g / per_token;
    if (t >= static_cast<unsigned>(a.T)) return;   // the 16 lanes of a vector leave together
    const int h0 = (g - t * per_token) * a.heads, heads = min(a.heads, H - h0);
    const Place p = find_place(a, t, l);
    const bool written = p.pos >= 0 && p.page >= 0;
    const TIn* x = kind == 0 ? static_cast<const TIn*>(a.K) + t * a.k_stride
                 : kind == 1 ? static_cast<const TIn*>(a.V) + t * a.v_stride : static_cast<const TIn*>(a.Q) + t * a.q_stride;
    x += h0 * 128LL;
    if (kind == 2 ? !p.in_batch : !written) return;
    if (kind == 2 && p.pos < 0) {
        for (int i = 0; i < heads; ++i)
            *reinterpret_cast<uint4*>(a.Q_out + (static_cast<long long>(t) * a.Hq + h0 + i) * 128 + 8 * l) = uint4{};
        return;
    }
    const float* rope_row = a.rope + p.turn * a.rot_dim;
    if (kind == 0) {
        // Everything of 64 bits is loaded and derived anew for every head: kept, it would take 80 registers.
        for (int i = 0; i < heads; ++i, x += 128) {
            int lane = l;
            asm("" : "+v"(lane));
            double v[8];
            const double norm = 0.08838834764831844055 /* 1 / sqrt(128) */ *
                                turned<double, TIn>(x, a.k_norm, a.eps, load_turn(rope_row, a.rot_dim, a.interleaved, lane),
                                                    a.rot_dim, a.interleaved, lane, v);
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = static_cast<float>(v[j] * norm);
            put_codes<BITS, false>(a, y, p, h0 + i, out_octet(lane));
        }
    } else if (kind == 1) {
        for (int i = 0; i < heads; ++i, x += 128) {
            float y[8];
            load8<TIn>(x + 8 * l, y);
            put_codes<BITS, true>(a, y, p, h0 + i, l);
        }
    } else {
        const Turn turn = load_turn(rope_row, a.rot_dim, a.interleaved, l);
        uint16_t* out = a.Q_out + (static_cast<long long>(t) * a.Hq + h0) * 128 + 8 * out_octet(l);
        for (int i = 0; i < heads; ++i, x += 128, out += 128) {
            float v[8];
            const float norm = a.norm * turned<float, TIn>(x, a.q_norm, a.eps, turn, a.rot_dim, a.interleaved, l, v);
            union { _Float16 f[8]; uint4 u; } y;
#pragma unroll
            for (int j = 0; j < 8; ++j) y.f[j] = static_cast<_Float16>(v[j] * norm);
            *reinterpret_cast<uint4*>(out) = y.u;
        }
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

// Heads of a token that a lane group takes.  Measured in us at 1, 2 and 4 with 32 + 8 heads of float32: 128 tokens 4.6, 5.5,
// 7.5; 384 5.8, 6.3, 8.0; 512 7.3, 6.6, 8.4; 1024 11.3, 10.0, 10.5; 2048 20.7, 16.4, 14.9; 8192 95, 72, 61.
int heads_of(int T, int Hq, int Hkv) {
    const long long vectors = static_cast<long long>(T) * (Hq + 2LL * Hkv);
    return vectors >= 65536 ? kMostHeads : vectors >= 20480 ? 2 : 1;
}

long long blocks_of(int T, int H, int heads) {
    return (static_cast<long long>(T) * ((H + heads - 1) / heads) + kAppendVectors - 1) / kAppendVectors;
}

}  // namespace

long long kv_append_blocks(int T, int Hq, int Hkv) { return 2 * blocks_of(T, Hkv, 1) + blocks_of(T, Hq, 1); }

hipError_t launch_kv_append(KvAppendArgs a, bool x_f16, int bits, hipStream_t s) {
    a.heads = heads_of(a.T, a.Hq, a.Hkv);
    a.kv_blocks = static_cast<unsigned>(blocks_of(a.T, a.Hkv, a.heads));
    a.norm = static_cast<float>(1.0 / __builtin_sqrt(128.0));
    const long long blocks = 2LL * a.kv_blocks + blocks_of(a.T, a.Hq, a.heads);
    if (blocks == 0) return hipSuccess;
    return bits == 8 ? launch_bits<8>(a, x_f16, blocks, s) : launch_bits<4>(a, x_f16, blocks, s);
}

}  // namespace spin
