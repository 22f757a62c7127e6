// spin_kv_weights kernel: the attention weight that every cached token of a
// sequence draws from the sequence's query rows.
//
// With the logarithm lse_r of each row's sum of exponentials (attention leaves
// it), token j's weight is
//   W_j = decay prior_j + sum_r e^(z_rj - lse_r)     over the rows and the heads of the group that see it,
// z as in attention.  Keys are read once, values not at all, and a token's sum
// stays in one lane: no atomics, and the same bits every time.
//
// The product is S = Q K^T with a token per lane: the matrix cores' result then
// holds four rows of one token in a lane's registers, so that a token's key factor
// is one register and the sum over rows is additions within the lane.
//
// Codes go into the product as the integers they are.  As attention takes them,
// code + 8 as a subnormal number and the offset in the accumulator, they save a
// subtraction, but the matrix cores align subnormal operands as if their leading
// bit were there: at queries of 2 and 4-bit codes a sum of 128 products is off by
// 3e-4 (rms; 1e-6 with the integers), which attention rounds off with its fp16
// weights and an fp32 weight would keep.
#include "kv_batch.h"
#include "kv_scores.h"
#include "spin_device.h"
#include "spin_internal.h"

namespace spin {
namespace {

constexpr int kWeightThreads = 256;
constexpr int kWeightTokens = 64;                                        // of a wave
constexpr int kWeightChunk = kWeightThreads / 64 * kWeightTokens;        // of a workgroup

template <int BITS, int SCORES>
__global__ __launch_bounds__(kWeightThreads, 2) void kv_weights_kernel(KvWeightsArgs a, int chunks) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    const int G = a.Hq / a.Hkv;
    // workgroup L runs on XCD L % 8: the heads of an item follow each other on one, which share lines of scales
    const int h = (blockIdx.x >> 3) % a.Hkv;
    const int item = (blockIdx.x >> 3) / a.Hkv * 8 + (blockIdx.x & 7);
    const int b = item / chunks;
    if (b >= a.B) return;
    const int j0 = (item - b * chunks) * kWeightChunk + wave * kWeightTokens;
    const int tokens = context(a, b);
    if (j0 >= tokens) return;
    const int q0 = within(a.q_start[b], a.T), q1 = within(a.q_start[b + 1], a.T);
    const int news = max(q1 - q0, 0);
    const int start = a.pos0 + placed(a.kv_len[b]) - news;               // position of the first row
    const int both = a.bidir_len ? max(a.bidir_len[b], 0) : 0;

    // where the tokens lie, 16 of them in one page: the number of the first, ~0 if nowhere
    unsigned long long place[4];
    uint32_t kraw[4][BITS];
    float kf[4];
    const Cap cap = cap_of<SCORES>(a);
    const float key_factor = held(cap.factor);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int j = j0 + 16 * i;
        const int page = j < tokens ? a.page_table[static_cast<long long>(b) * a.max_pages + (j >> a.page_log2)] : -1;
        const bool good = page >= 0 && page < a.n_pages;
        const unsigned long long token = ((static_cast<unsigned long long>(good ? page : 0) * a.Hkv + h) << a.page_log2) + (good ? j & ((1 << a.page_log2) - 1) : 0);
        place[i] = good ? token : ~0ull;
        const u4* kp = reinterpret_cast<const u4*>(a.K_codes + token * (16 * BITS));
#pragma unroll
        for (int x = 0; x < BITS / 4; ++x) {
            const u4 y = kp[(n * 4 + g) * (BITS / 4) + x];
            kraw[i][4 * x] = y.x; kraw[i][4 * x + 1] = y.y; kraw[i][4 * x + 2] = y.z; kraw[i][4 * x + 3] = y.w;
        }
        // a row that sees a scale that is not finite has no weights
        const float ks = __half2float(__ushort_as_half(a.K_scale[token + n]));
        kf[i] = good && __builtin_fabsf(ks) <= 65504.0f ? ks * key_factor : 0.0f;
    }

    // the rows that may see any of the tokens, of the sequence's new ones
    const int last = min(j0 + kWeightTokens, tokens) - 1;
    long long lo = 0, hi = news;
    if (a.causal && a.pos0 + j0 >= both) lo = max(lo, static_cast<long long>(a.pos0) + j0 - start);
    if (a.window > 0) {
        lo = max(lo, static_cast<long long>(a.pos0) + j0 - a.window + 1 - start);
        hi = min(hi, static_cast<long long>(a.pos0) + last + a.window - start);
    }
    float acc[4] = {};
    const int row_end = hi > lo ? static_cast<int>(hi) * G : 0;
    for (int r0 = __builtin_amdgcn_readfirstlane(hi > lo ? static_cast<int>(lo) * G : 0); r0 < row_end; r0 += 16) {
        // lane (n, g): values 32 g .. 32 g + 31 of row n, in the order of the keys' codes
        const int r = r0 + n;
        const bool valid = r < row_end;
        const int i_row = valid ? static_cast<int>(static_cast<unsigned>(r) / static_cast<unsigned>(G)) : 0;
        const int head = h * G + (valid ? r - i_row * G : 0);
        const long long at = static_cast<long long>(q0 + i_row) * a.Hq + head;
        float lse2 = valid ? a.lse[at] * kLog2e : __builtin_inff();
        const bool counts = __builtin_fabsf(lse2) < __builtin_inff();
        lse2 = counts ? lse2 : __builtin_inff();         // every exponential is 0
        h8 q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            Frag raw, f;
            const u4 x = counts ? *reinterpret_cast<const u4*>(a.Q + at * 128 + 32 * g + 8 * j) : u4{0, 0, 0, 0};
            raw.w[0] = x.x; raw.w[1] = x.y; raw.w[2] = x.z; raw.w[3] = x.w;
#pragma unroll
            for (int i = 0; i < 8; ++i) f.v[i] = raw.v[order8<BITS>(i)];
            q[j] = f.v;
        }
        const float slope = SCORES != kPlain && a.slopes ? a.slopes[head] * kLog2e : 0.0f;
        const int pos = start + i_row;
        float less[4], slopes[4];
        int where[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            less[e] = __shfl(lse2, 4 * g + e, 64);
            slopes[e] = SCORES != kPlain ? __shfl(slope, 4 * g + e, 64) : 0.0f;
            where[e] = __shfl(pos, 4 * g + e, 64);
        }
        // does every row see every token
        const int pmin = start + r0 / G, pmax = start + min(r0 + 15, row_end - 1) / G;
        bool whole = true;
        if (a.causal) whole = a.pos0 + last <= pmin || a.pos0 + last < both;
        if (a.window > 0) whole = whole && static_cast<long long>(pmax) - a.pos0 - j0 < a.window && static_cast<long long>(a.pos0) + last - pmin < a.window;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f4 s = {};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                s = __builtin_amdgcn_mfma_f32_16x16x32_f16(q[j], key_operand<BITS>(kraw[i] + j * (BITS / 4)), s, 0, 0, 0);
            const int p = a.pos0 + j0 + 16 * i + n;      // the token's position
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float lm = -less[e];
                if (SCORES != kPlain) lm = __builtin_fmaf(-slopes[e], __builtin_fabsf(static_cast<float>(where[e] - p)), lm);
                x[e] = SCORES == kWideCap ? capped_wide(s[e] * kf[i], cap.top, cap.rtop) + lm
                       : SCORES == kFancy && a.softcap > 0.0f ? capped_plus(s[e] * kf[i], cap.top, lm + cap.top) : __builtin_fmaf(s[e], kf[i], lm);
            }
            if (!whole) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    bool seen = !a.causal || p <= where[e] || p < both;
                    if (a.window > 0) seen = seen && static_cast<uint32_t>(where[e] - p) + static_cast<uint32_t>(a.window) - 1u < 2u * static_cast<uint32_t>(a.window) - 1u;
                    x[e] = seen ? x[e] : -__builtin_inff();
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i] += __builtin_amdgcn_exp2f(x[e]);
        }
    }
    // lane l has token l
    float w = 0.0f;
    unsigned long long token = ~0ull;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float sum = sum_over_groups(acc[i]);
        w = g == i ? sum : w;
        token = g == i ? place[i] : token;
    }
    if (token == ~0ull || j0 + lane >= tokens) return;
    token += n;
    const float ks = __half2float(__ushort_as_half(a.K_scale[token]));
    w = __builtin_fabsf(ks) <= 65504.0f ? w : 0.0f;
    a.W[token] = a.prior ? __builtin_fmaf(a.decay, a.prior[token], w) : w;
}

template <int BITS>
hipError_t launch_bits(const KvWeightsArgs& a, hipStream_t s) {
    const int chunks = ((a.max_pages << a.page_log2) + kWeightChunk - 1) / kWeightChunk;
    const long long items = static_cast<long long>(a.B) * chunks;
    const dim3 grid(static_cast<unsigned>((items + 7) / 8 * 8 * a.Hkv));
    if (a.softcap > kNearCap)
        hipLaunchKernelGGL((kv_weights_kernel<BITS, kWideCap>), grid, dim3(kWeightThreads), 0, s, a, chunks);
    else if (a.softcap > 0.0f || a.slopes)
        hipLaunchKernelGGL((kv_weights_kernel<BITS, kFancy>), grid, dim3(kWeightThreads), 0, s, a, chunks);
    else
        hipLaunchKernelGGL((kv_weights_kernel<BITS, kPlain>), grid, dim3(kWeightThreads), 0, s, a, chunks);
    return hipGetLastError();
}

}  // namespace

bool kv_weights_fits(int T, int Hq, int Hkv, int B, int max_kv) {
    const long long items = static_cast<long long>(B) * ((static_cast<long long>(max_kv) + kWeightChunk - 1) / kWeightChunk);
    return Hkv <= 65535 && items <= (1LL << 24) && (items + 7) * Hkv <= (1LL << 24) - 1 && static_cast<long long>(T) * Hq <= (1LL << 26);
}

hipError_t launch_kv_weights(const KvWeightsArgs& a, int bits, hipStream_t s) {
    return bits == 8 ? launch_bits<8>(a, s) : launch_bits<4>(a, s);
}

}  // namespace spin
