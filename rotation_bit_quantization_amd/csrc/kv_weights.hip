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
// weights and an fp32 weight would keep.  Attention's logarithms keep it, averaged
// over the tokens: 9e-6 (rms) at 4 bits, and a weight with them is off by as much.
// It is common to all tokens of a row, so that it moves their sums, not their order
// within a row, where the integers' 3e-7 remains.
#include "kv_batch.h"
#include "kv_scores.h"
#include "spin_device.h"
#include "spin_internal.h"

namespace spin {
namespace {

constexpr int kWeightThreads = 256;
constexpr int kWeightWaves = kWeightThreads / 64;
constexpr int kGroup = 64;                 // tokens that a wave takes at a time, one a lane in the end
// Rows of a key head, on the mean over the sequences, from which they are staged 32 at a time (16 sequences on 4000 tokens,
// 20 rows each: 20.6 us 16 at a time, 19.5 staged; 256 on 500: 60 and 38).
constexpr int kManyRows = 17;
// Workgroups of 256 tokens from which a wave holds 64 of them, without a cap or bias (a prompt of 8192 320 us, with 32 a wave
// 369; of 2000, 64 workgroups, 40 and 36); with them the registers for 64 leave two waves a SIMD (3 prompts of 1670,
// capped and biased, 140 us against 124).
constexpr int kTilesWanted = 256;
// Workgroups that shares of the rows bring a call to, tiles of 32 rows that a share has at least, and the most shares: a
// prompt of 2000 takes 204 us in one share, 37 in up to 16, one of 500 59 and 15.
constexpr int kSharesWanted = 4096, kLeastTiles = 4, kMostShares = 16;
constexpr int kCounted = 256;              // sequences up to which their chunks are counted
// Groups that a wave takes, where there are enough for it (64 sequences on up to 8192 tokens, 16 rows at a time, 61 us with
// one, 47 with four, 53 with twelve), and what enough is.
constexpr int kMostTurns = 4, kGroupsEnough = 8192;

// Tokens of sequence b, the first ones, that have a prior.
__device__ __forceinline__ int priors(const KvWeightsArgs& a, int b) {
    return !a.prior ? 0 : a.prior_len ? a.prior_len[b] : 0x7FFFFFFF;
}

// What a row adds to tokens, as the kernels hold it: its position, the logarithm in units of log2 (infinite where it adds
// nothing: every exponential is 0) and its bias.
struct Row {
    long long at;          // of [T][Hq]
    float lse2, slope;
    int pos;
};
template <int SCORES>
__device__ __forceinline__ Row row_of(const KvWeightsArgs& a, int r, bool valid, int q0, int start, int h, int G) {
    const int i = valid ? static_cast<int>(static_cast<unsigned>(r) / static_cast<unsigned>(G)) : 0;
    const int head = h * G + (valid ? r - i * G : 0);
    Row row;
    row.at = static_cast<long long>(q0 + i) * a.Hq + head;
    const float lse2 = valid ? a.lse[row.at] * kLog2e : __builtin_inff();
    row.lse2 = __builtin_fabsf(lse2) < __builtin_inff() ? lse2 : __builtin_inff();
    row.slope = SCORES != kPlain && a.slopes ? a.slopes[head] * kLog2e : 0.0f;
    row.pos = start + i;
    return row;
}

// What a kernel does to the scores here: nothing, a bias, or (kWideCap) a cap, with or without a bias.
//
// A capped score is z tanh(u) / u with u = z / cap.  Up to |u| = sqrt(1/2) the ratio is a polynomial of degree 5 in u^2,
// fitted to the least relative error, 2^-24.7, six multiply-adds and no transcendental; above the exponential's form, whose
// error is of the cap's size, ten of 2^-24, and then of the score's too.  Attention's form for caps up to 64 is off by that
// at any score, which fp32 weights show (cap 30 and 50: errors of weights 1.1e-6 in place of 4e-7).
constexpr float kNear = 0.70710678f;       // of |u|
__device__ __forceinline__ float capped_near(float z, float rtop, float lm) {
    const float u = z * rtop, t = u * u;
    float p = __builtin_fmaf(t, -0.005034888628870249f, 0.01996474526822567f);
    p = __builtin_fmaf(p, t, -0.05350292846560478f);
    p = __builtin_fmaf(p, t, 0.13328056037425995f);
    p = __builtin_fmaf(p, t, -0.3333311080932617f);
    p = __builtin_fmaf(p, t, 1.0f);
    return __builtin_fmaf(z, p, lm);
}
__device__ __forceinline__ float capped_any(float z, const Cap& cap, float lm) {
    const float u = z * cap.rtop;
    const float far = __builtin_fmaf(__builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(u * (2.0f * kLog2e)) + 1.0f), -2.0f * cap.top, cap.top + lm);
    return __builtin_fabsf(u) <= kNear ? capped_near(z, cap.rtop, lm) : far;
}

// N scores, held in s as products and left there as exponents of weights: `factor` of the products, `lm` added to a score.
template <int SCORES, int N, typename S, typename Less>
__device__ __forceinline__ void exponents(const Cap& cap, S& s, float factor, Less lm) {
    if (SCORES != kWideCap) {
#pragma unroll
        for (int e = 0; e < N; ++e) s[e] = __builtin_fmaf(s[e], factor, lm(e));
        return;
    }
    float top = 0.0f;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        s[e] *= factor;
        top = __builtin_fmaxf(top, __builtin_fabsf(s[e]));
    }
    if (__ballot(!(top * cap.rtop <= kNear)) == 0) {
#pragma unroll
        for (int e = 0; e < N; ++e) s[e] = capped_near(s[e], cap.rtop, lm(e));
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) s[e] = capped_any(s[e], cap, lm(e));
    }
}

__device__ __forceinline__ bool sees(const KvWeightsArgs& a, int pos, int p, int both) {
    const bool near = !a.causal || p <= pos || p < both;
    return near && (a.window <= 0 || static_cast<uint32_t>(pos - p) + static_cast<uint32_t>(a.window) - 1u < 2u * static_cast<uint32_t>(a.window) - 1u);
}

// The rows, of a sequence's `news` new ones, that may see any of the tokens at positions p0 .. p1.
struct Range {
    int lo, hi;
};
__device__ __forceinline__ Range rows_on(const KvWeightsArgs& a, int p0, int p1, int start, int news, int both) {
    long long lo = 0, hi = news;
    if (a.causal && p0 >= both) lo = max(lo, static_cast<long long>(p0) - start);
    if (a.window > 0) {
        lo = max(lo, static_cast<long long>(p0) - a.window + 1 - start);
        hi = min(hi, static_cast<long long>(p1) + a.window - start);
    }
    return hi > lo ? Range{static_cast<int>(lo), static_cast<int>(hi)} : Range{0, 0};
}

// Does every row at positions pmin .. pmax see every token at p0 .. p1.
__device__ __forceinline__ bool all_seen(const KvWeightsArgs& a, int pmin, int pmax, int p0, int p1, int both) {
    bool whole = true;
    if (a.causal) whole = p1 <= pmin || p1 < both;
    if (a.window > 0) whole = whole && static_cast<long long>(pmax) - p0 < a.window && static_cast<long long>(p1) - pmin < a.window;
    return whole;
}

// Where 16 tokens from place j on lie, as the number of the first, ~0 if nowhere.
__device__ __forceinline__ unsigned long long place_of(const KvWeightsArgs& a, int b, int h, int j, int tokens) {
    const int page = j < tokens ? a.page_table[static_cast<long long>(b) * a.max_pages + (j >> a.page_log2)] : -1;
    if (page < 0 || page >= a.n_pages) return ~0ull;
    return ((static_cast<unsigned long long>(page) * a.Hkv + h) << a.page_log2) + (j & ((1 << a.page_log2) - 1));
}

__device__ __forceinline__ float scale_of(uint32_t raw) { return __half2float(__ushort_as_half(static_cast<unsigned short>(raw))); }

// Few rows: 4 N at a time (N is 1, 2 or 4), groups of 64 tokens in turn, the next one's keys in flight.  A lane's results
// are N rows of a token: rows stand in the matrix cores' operand so that its four places hold rows g, g + 4, ..
//
// Bound: reading the keys, 16 BITS + 2 bytes a token and head, from the second round of workgroups on; before that loads
// that wait for each other (length, page, keys).  Measured: 64 single tokens of 32 + 8 heads on 2000 to 8192, INT4, 43 us
// from the last-level cache and 51 from memory (189 MB, 3.7 TB/s), capped 47 and 53, INT8 83; in a table for 32768 47, for
// 131072 75; 16 on 2000 to 8192 17 us, one on 30000 6, one on 1000 4.5.  With 16 rows at a time whatever there is, capped
// 65.  Five waves a SIMD spill (62 us).
//
// A sequence of more rows than the batch's mean (the host knows no other number) takes them all past each of its groups,
// 4 N at a time: a prompt of 4000 among 255 single tokens, 8 + 8 heads, 1618 us (the single tokens alone 25), one of 200
// among 63, 32 + 8 heads, 244 (39).  Its sums are then carried with what their additions have lost, as a tile's are, in
// LDS, since registers are spent (added plainly 1532 and 230 us, and off by 6e-6 of themselves).
template <int BITS, int SCORES, int N>
__global__ __launch_bounds__(kWeightThreads, BITS == 4 && SCORES != kWideCap ? 4 : 3) void kv_weights_rows16(KvWeightsArgs a, int chunks, int turns) {
    // a lane's sums over more than 4 N rows, and what their additions have lost; no other lane's
    __shared__ f4 sums[kWeightThreads], lost[kWeightThreads];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    const int G = a.Hq / a.Hkv;
    // workgroup L runs on XCD L % 8: the heads of an item follow each other on one, which share lines of scales
    const int h = (blockIdx.x >> 3) % a.Hkv;
    int item = (blockIdx.x >> 3) / a.Hkv * 8 + (blockIdx.x & 7), b = -1;
    if (a.B <= kCounted) {
        // numbered without the chunks that sequences are too short for (64 of 2000 to 8192
        // tokens: 57 to 63 us with gaps, by their number, 47 to 50 without)
        const int chunk = turns * kWeightWaves * kGroup;
        for (int b0 = 0; b0 < a.B && b < 0; b0 += 64) {
            const int own = b0 + lane < a.B ? (context(a, b0 + lane) + chunk - 1) / chunk : 0, upto = sums_up_to(own);
            const unsigned long long hit = __ballot(upto > item);
            if (hit == 0) {
                item -= __builtin_amdgcn_readlane(upto, 63);
            } else {
                const int l = __builtin_ctzll(hit);
                b = b0 + l;
                item -= __builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(own, l);
            }
        }
        if (b < 0) return;
    } else {
        b = item / chunks;
        item -= b * chunks;
        if (b >= a.B) return;
    }
    const int tokens = context(a, b);
    const int first = (item * turns * kWeightWaves + wave) * kGroup;      // then every kWeightWaves-th group
    if (first >= tokens) return;
    const int q0 = within(a.q_start[b], a.T), q1 = within(a.q_start[b + 1], a.T);
    const int news = max(q1 - q0, 0);
    const int start = a.pos0 + placed(a.kv_len[b]) - news;               // position of the first row
    const int both = a.bidir_len ? max(a.bidir_len[b], 0) : 0;
    const Cap cap = cap_of<SCORES>(a);
    const float key_factor = held(cap.factor);

    const int weighed = priors(a, b);
    const int unit = first + (lane >> 2) * kWeightWaves * kGroup + (lane & 3) * 16;
    const unsigned long long places = (lane >> 2) < turns ? place_of(a, b, h, unit, tokens) : ~0ull;
    auto place = [&](int t, int i) __attribute__((always_inline)) {
        const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(places), 4 * t + i);
        const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(places >> 32), 4 * t + i);
        return (static_cast<unsigned long long>(hi) << 32) | lo;
    };
    struct Raw {
        uint32_t k[4][BITS], scale;        // lane (n, g): 32 codes of token n of each 16; the scale and prior of token 16 g + n
        float prior;
        unsigned long long token;          // the lane's, ~0 if it is nowhere
    };
    auto fetch = [&](int t) __attribute__((always_inline)) {
        Raw raw;
        raw.token = ~0ull;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned long long p = place(t, i), token = p == ~0ull ? static_cast<unsigned long long>(h) << a.page_log2 : p;
            const u4* kp = reinterpret_cast<const u4*>(a.K_codes + token * (16 * BITS));
#pragma unroll
            for (int x = 0; x < BITS / 4; ++x) {
                const u4 y = kp[(n * 4 + g) * (BITS / 4) + x];
                raw.k[i][4 * x] = y.x; raw.k[i][4 * x + 1] = y.y; raw.k[i][4 * x + 2] = y.z; raw.k[i][4 * x + 3] = y.w;
            }
            raw.token = g == i && p != ~0ull ? p + n : raw.token;
        }
        if (first + t * kWeightWaves * kGroup + lane >= tokens) raw.token = ~0ull;
        const bool there = raw.token != ~0ull;
        raw.scale = there ? a.K_scale[raw.token] : 0u;
        raw.prior = there && first + t * kWeightWaves * kGroup + lane < weighed ? a.prior[raw.token] : 0.0f;
        return raw;
    };

    h8 q[4];
    float less[N], slopes[N];
    int where[N];
    auto load_rows = [&](int r0, int row_end) __attribute__((always_inline)) {
        // lane (n, g): values 32 g .. 32 g + 31 of row n / 4 + 4 (n % 4), in the order of the keys' codes
        const int r = r0 + (n >> 2) + 4 * (n & 3);
        const Row row = row_of<SCORES>(a, r, r < row_end && (n & 3) < N, q0, start, h, G);
        const bool counts = row.lse2 < __builtin_inff();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            Frag raw, f;
            const u4 x = counts ? *reinterpret_cast<const u4*>(a.Q + row.at * 128 + 32 * g + 8 * j) : u4{0, 0, 0, 0};
            raw.w[0] = x.x; raw.w[1] = x.y; raw.w[2] = x.z; raw.w[3] = x.w;
#pragma unroll
            for (int i = 0; i < 8; ++i) f.v[i] = raw.v[order8<BITS>(i)];
            q[j] = f.v;
        }
#pragma unroll
        for (int e = 0; e < N; ++e) {
            less[e] = __shfl(row.lse2, 4 * g + e, 64);
            slopes[e] = SCORES != kPlain ? __shfl(row.slope, 4 * g + e, 64) : 0.0f;
            where[e] = __shfl(row.pos, 4 * g + e, 64);
        }
    };

    const int groups = min(turns, (tokens - first + kWeightWaves * kGroup - 1) / (kWeightWaves * kGroup));
    Raw raw = fetch(0);
    const int rows = news * G;
    const bool many = rows > 4 * N;
    if (!many) load_rows(0, rows);
    for (int t = 0; t < groups; ++t) {
        const int j0 = first + t * kWeightWaves * kGroup, last = min(j0 + kGroup, tokens) - 1;
        // a row that sees a scale that is not finite has no weights
        const float ks = scale_of(raw.scale);
        const bool fine = __builtin_fabsf(ks) <= 65504.0f;
        const float kf_own = fine ? ks * key_factor : 0.0f;
        float kf[4], acc[4] = {};          // of 4 N rows
#pragma unroll
        for (int i = 0; i < 4; ++i) kf[i] = __shfl(kf_own, 16 * i + n, 64);
        const unsigned long long token = raw.token;
        const float prior = raw.prior;
        Raw next = raw;
        if (t + 1 < groups) next = fetch(t + 1);
        const Range on = rows_on(a, a.pos0 + j0, a.pos0 + last, start, news, both);
        const int row_end = on.hi * G;
        if (many) sums[threadIdx.x] = f4{}, lost[threadIdx.x] = f4{};
        for (int r0 = many ? on.lo * G : 0; r0 < row_end; r0 += 4 * N) {
            if (many) load_rows(r0, row_end);
            const bool whole = all_seen(a, start + r0 / G, start + (min(r0 + 4 * N, rows) - 1) / G, a.pos0 + j0, a.pos0 + last, both);
            // unpacked anew for these rows: kept, the operands of 64 tokens take 64 registers
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int x = 0; x < BITS; ++x) asm("" : "+v"(raw.k[i][x]));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f4 s = {};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    s = __builtin_amdgcn_mfma_f32_16x16x32_f16(q[j], key_operand<BITS>(raw.k[i] + j * (BITS / 4)), s, 0, 0, 0);
                const int p = a.pos0 + j0 + 16 * i + n;      // the token's position
                exponents<SCORES, N>(cap, s, kf[i], [&](int e) __attribute__((always_inline)) {
                    return SCORES == kPlain ? -less[e] : __builtin_fmaf(-slopes[e], __builtin_fabsf(static_cast<float>(where[e] - p)), -less[e]);
                });
                if (!whole) {
                    asm volatile("" ::: "memory");           // keeps this a branch
#pragma unroll
                    for (int e = 0; e < N; ++e) s[e] = sees(a, where[e], p, both) ? s[e] : -__builtin_inff();
                }
                acc[i] = __builtin_amdgcn_exp2f(s[0]);
#pragma unroll
                for (int e = 1; e < N; ++e) acc[i] += __builtin_amdgcn_exp2f(s[e]);
            }
            if (many) {
                const f4 old = sums[threadIdx.x], y = f4{acc[0], acc[1], acc[2], acc[3]} - lost[threadIdx.x], sum = old + y;
                lost[threadIdx.x] = (sum - old) - y;
                sums[threadIdx.x] = sum;
            }
        }
        if (many) {
            const f4 sum = sums[threadIdx.x];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = sum[i];
        }
        // lane l has token l
        float w = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float sum = sum_over_groups(acc[i]);
            w = g == i ? sum : w;
        }
        w = fine ? w : 0.0f;
        if (token != ~0ull) a.W[token] = a.prior ? __builtin_fmaf(a.decay, prior, w) : w;
        raw = next;
    }
}

typedef float f16v __attribute__((ext_vector_type(16)));

constexpr int kTileRows = 32;

// Many rows: the workgroup stages 32 rows at a time in LDS, and each wave holds the keys of 32 M tokens as operands and
// takes all rows past them.
//
// Bound: the vector work of the weights beside the matrix work, 24 cycles (a multiply-add, an exponential, an addition) of
// 64 scores against 16, with a cap and a bias 66, and what staging 32 rows takes.  A token's sum is carried with what its
// additions have lost, 32 rows at a time, so that it is as exact for a long prompt as for a row.  Measured with 32 + 8 heads
// and INT4: a prompt of 8192 tokens 320 - 334 us (0.82 - 0.86 PFLOP/s), of 2000 37 (in a table for 8192 40, for 131072, where
// its rows are one share, 290), 32 tokens each of two on 16384 22; three uneven prompts of 5011 together, 32 + 32 heads, INT8,
// capped and biased, 106 - 123.
template <int BITS, int SCORES, int M>
__global__ __launch_bounds__(kWeightThreads, 2) void kv_weights_tile(KvWeightsArgs a, int splits) {
    struct Stage {
        u4 q[kTileRows * 17];              // 16 chunks of 8 values a row, and one more, so that rows lie in different banks
        // of each row: what is added to its scores, its bias, its position behind the first row's
        f4 less[kTileRows / 4], slope[kTileRows / 4], pos[kTileRows / 4];
    };
    __shared__ Stage sh[2];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 31, hf = lane >> 5;
    const int G = a.Hq / a.Hkv;
    // key heads alternate fastest: with 8 of them a head, and the queries that its workgroups share, stays on one XCD; the
    // first tokens of all sequences come first, which most rows see
    const int h = blockIdx.x % a.Hkv, rest = blockIdx.x / a.Hkv;
    const int split = rest % splits, item = rest / splits, b = item % a.B, first = item / a.B * (kWeightWaves * 32 * M);
    const int tokens = context(a, b);
    if (first >= tokens) return;
    const int q0 = within(a.q_start[b], a.T), q1 = within(a.q_start[b + 1], a.T);
    const int news = max(q1 - q0, 0);
    const int start = a.pos0 + placed(a.kv_len[b]) - news;               // position of the first row
    const int both = a.bidir_len ? max(a.bidir_len[b], 0) : 0;
    const Cap cap = cap_of<SCORES>(a);
    const float key_factor = held(cap.factor);

    // keys: lane (n, hf) holds values 64 hf .. 64 hf + 63 of token n of each 32, eight to an operand
    h8 key[M][8];
    float kf[M], sum[M], rest_of[M];       // what the sum has lost to rounding
    unsigned long long token[M];
    bool fine[M];
    const int j0 = first + wave * 32 * M;
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const int j = j0 + 32 * m + n;
        const unsigned long long p = place_of(a, b, h, j & ~15, tokens);
        token[m] = p == ~0ull || j >= tokens ? ~0ull : p + (j & 15);
        const unsigned long long from = token[m] == ~0ull ? static_cast<unsigned long long>(h) << a.page_log2 : token[m];
        const u4* codes = reinterpret_cast<const u4*>(a.K_codes + (from * 2 + hf) * (8 * BITS));
        uint32_t w[2 * BITS];
#pragma unroll
        for (int x = 0; x < BITS / 2; ++x) {
            const u4 y = codes[x];
            w[4 * x] = y.x; w[4 * x + 1] = y.y; w[4 * x + 2] = y.z; w[4 * x + 3] = y.w;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) key[m][k] = key_operand<BITS>(w + k * (BITS / 4));
        // a row that sees a scale that is not finite has no weights
        const float ks = token[m] == ~0ull ? 0.0f : scale_of(a.K_scale[from]);
        fine[m] = __builtin_fabsf(ks) <= 65504.0f;
        kf[m] = fine[m] ? ks * key_factor : 0.0f;
        sum[m] = rest_of[m] = 0.0f;
    }

    const int end = min(first + kWeightWaves * 32 * M, tokens) - 1;      // the workgroup's last token, and the wave's
    const int last = min(j0 + 32 * M, tokens) - 1;
    const Range on = rows_on(a, a.pos0 + first, a.pos0 + end, start, news, both);
    const Range mine = j0 < tokens ? rows_on(a, a.pos0 + j0, a.pos0 + last, start, news, both) : Range{0, 0};
    // the workgroup's share of them, of 32 at a time
    const int tiles = ((on.hi - on.lo) * G + kTileRows - 1) / kTileRows, share = (tiles + splits - 1) / splits;
    const int first_row = on.lo * G + split * share * kTileRows;
    const int row_end = min(on.hi * G, first_row + share * kTileRows);
    // Numbers of rows as token and head of the group, which follow the steps of 32 without a division.
    const int step_i = kTileRows / G, step_g = kTileRows - step_i * G;
    struct At {
        int i, g;
    };
    auto at_row = [&](int r) __attribute__((always_inline)) { return At{r / G, r - r / G * G}; };
    auto advance = [&](At& x) __attribute__((always_inline)) {
        x.g += step_g;
        x.i += step_i + (x.g >= G ? 1 : 0);
        x.g -= x.g >= G ? G : 0;
    };
    // a thread stages chunks x and x + 8 of row threadIdx / 8
    const int s_row = threadIdx.x >> 3, s_chunk = threadIdx.x & 7;
    struct Raw {
        u4 q[2];
        float lse2, slope;
        int pos;
    };
    At staged = at_row(first_row + s_row), lowest = at_row(first_row), highest = at_row(first_row + kTileRows - 1);
    auto fetch = [&](int r0) __attribute__((always_inline)) {
        Raw raw;
        const bool valid = r0 + s_row < row_end;
        const int head = h * G + staged.g;
        const long long at = valid ? static_cast<long long>(q0 + staged.i) * a.Hq + head : 0;
        const float lse2 = valid ? a.lse[at] * kLog2e : __builtin_inff();
        const bool counts = __builtin_fabsf(lse2) < __builtin_inff();
        raw.lse2 = counts ? lse2 : __builtin_inff();
        raw.slope = SCORES != kPlain && a.slopes && valid ? a.slopes[head] * kLog2e : 0.0f;
        raw.pos = staged.i;
#pragma unroll
        for (int x = 0; x < 2; ++x)
            raw.q[x] = counts ? *reinterpret_cast<const u4*>(a.Q + at * 128 + 8 * (s_chunk + 8 * x)) : u4{0, 0, 0, 0};
        advance(staged);
        return raw;
    };
    auto stage = [&](const Raw& raw, int i0, int buf) __attribute__((always_inline)) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {      // in the order of the keys' codes
            Frag in, out;
            in.w[0] = raw.q[x].x; in.w[1] = raw.q[x].y; in.w[2] = raw.q[x].z; in.w[3] = raw.q[x].w;
#pragma unroll
            for (int i = 0; i < 8; ++i) out.v[i] = in.v[order8<BITS>(i)];
            sh[buf].q[s_row * 17 + s_chunk + 8 * x] = u4{out.w[0], out.w[1], out.w[2], out.w[3]};
        }
        if (s_chunk == 0) {
            reinterpret_cast<float*>(sh[buf].less)[s_row] = -raw.lse2;
            if (SCORES != kPlain) reinterpret_cast<float*>(sh[buf].slope)[s_row] = raw.slope;
            reinterpret_cast<float*>(sh[buf].pos)[s_row] = static_cast<float>(raw.pos - i0);
        }
    };
    int buf = 0;
    if (first_row < row_end) stage(fetch(first_row), lowest.i, 0);
    __syncthreads();
    for (int r0 = first_row; r0 < row_end; r0 += kTileRows, buf ^= 1) {
        const bool more = r0 + kTileRows < row_end;
        Raw raw;
        if (more) raw = fetch(r0 + kTileRows);
        const int pmin = start + lowest.i, pmax = start + min(highest.i, on.hi - 1);
        const bool some = pmax - start >= mine.lo && pmin - start < mine.hi;
        advance(lowest);
        advance(highest);
        if (some) {
            const bool whole = all_seen(a, pmin, pmax, a.pos0 + j0, a.pos0 + last, both);
            f16v s[M];
#pragma unroll
            for (int m = 0; m < M; ++m) s[m] = f16v{};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const h8 q = __builtin_bit_cast(h8, sh[buf].q[n * 17 + 8 * hf + k]);
#pragma unroll
                for (int m = 0; m < M; ++m) s[m] = __builtin_amdgcn_mfma_f32_32x32x16_f16(q, key[m][k], s[m], 0, 0, 0);
            }
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const int p = a.pos0 + j0 + 32 * m + n;
                const float at = static_cast<float>(p - pmin);
                float w[4] = {};
                exponents<SCORES, 16>(cap, s[m], kf[m], [&](int e) __attribute__((always_inline)) {
                    const int i = 2 * (e >> 2) + hf;       // rows 8 (e / 4) + 4 hf .. + 3
                    const float less = sh[buf].less[i][e & 3];
                    return SCORES == kPlain ? less
                                            : __builtin_fmaf(-sh[buf].slope[i][e & 3], __builtin_fabsf(sh[buf].pos[i][e & 3] - at), less);
                });
                if (!whole) {
                    asm volatile("" ::: "memory");     // keeps this a branch
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            s[m][4 * i + e] = sees(a, pmin + static_cast<int>(sh[buf].pos[2 * i + hf][e]), p, both) ? s[m][4 * i + e] : -__builtin_inff();
                    }
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) w[e & 3] += __builtin_amdgcn_exp2f(s[m][e]);
                const float y = ((w[0] + w[1]) + (w[2] + w[3])) - rest_of[m], t = sum[m] + y;
                rest_of[m] = (t - sum[m]) - y;
                sum[m] = t;
            }
        }
        if (more) stage(raw, lowest.i, buf ^ 1);
        __syncthreads();
    }
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const u2 halves = __builtin_amdgcn_permlane32_swap(__float_as_uint(sum[m]), __float_as_uint(sum[m]), false, false);
        const float w = fine[m] ? __uint_as_float(halves.x) + __uint_as_float(halves.y) : 0.0f;
        if (hf != (m & 1)) continue;
        const int j = j0 + 32 * m + n;
        if (splits > 1) {
            if (j < tokens) a.partial[((static_cast<long long>(split) * a.B + b) * a.Hkv + h) * (static_cast<long long>(a.max_pages) << a.page_log2) + j] = w;
        } else if (token[m] != ~0ull) {
            a.W[token[m]] = j < priors(a, b) ? __builtin_fmaf(a.decay, a.prior[token[m]], w) : w;
        }
    }
}

// Adds the shares of the rows, a token a lane.
__global__ __launch_bounds__(kWeightThreads) void kv_weights_join(KvWeightsArgs a, int splits, int chunks) {
    const int chunk = blockIdx.x % chunks, head = blockIdx.x / chunks, b = head / a.Hkv, h = head - b * a.Hkv;
    const int tokens = context(a, b), j = chunk * kWeightThreads + static_cast<int>(threadIdx.x);
    if (j >= tokens) return;
    const unsigned long long p = place_of(a, b, h, j & ~15, tokens);
    if (p == ~0ull) return;
    const long long room = static_cast<long long>(a.max_pages) << a.page_log2;
    const float* part = a.partial + head * room + j;
    float w = 0.0f;
    for (int s = 0; s < splits; ++s) w += part[s * (static_cast<long long>(a.B) * a.Hkv * room)];
    const unsigned long long token = p + (j & 15);
    a.W[token] = j < priors(a, b) ? __builtin_fmaf(a.decay, a.prior[token], w) : w;
}

// How a call of these sizes is dealt out.
struct Plan {
    bool tile;
    int m, splits;                 // tiles: 32-token operands of a wave, shares of the rows
    int n;                         // few rows: four times as many at a time
    int turns;                     // few rows: groups that a wave takes, several where there are workgroups enough
};

Plan plan(int T, int Hq, int Hkv, int B, int room, bool plain) {
    Plan p = {};
    const long long heads = static_cast<long long>(B) * Hkv, rows = static_cast<long long>(T) * (Hq / Hkv) / B;
    p.tile = rows >= kManyRows;
    if (p.tile) {
        p.m = plain && heads * ((room + 255) / 256) >= kTilesWanted ? 2 : 1;
        const long long groups = heads * ((room + 128 * p.m - 1) / (128 * p.m));
        long long splits = kSharesWanted / groups;
        if (splits > rows / (kTileRows * kLeastTiles)) splits = rows / (kTileRows * kLeastTiles);
        p.splits = static_cast<int>(splits < 1 ? 1 : splits > kMostShares ? kMostShares : splits);
    } else {
        const long long turns = heads * ((room + kGroup - 1) / kGroup) / kGroupsEnough;
        p.n = rows <= 4 ? 1 : rows <= 8 ? 2 : 4;
        p.turns = static_cast<int>(turns < 1 ? 1 : turns > kMostTurns ? kMostTurns : turns);
    }
    return p;
}

template <int BITS, int SCORES>
hipError_t launch_scores(const KvWeightsArgs& a, const Plan& p, hipStream_t s) {
    const int room = a.max_pages << a.page_log2;
    if (p.tile) {
        const dim3 grid(static_cast<unsigned>(a.B) * a.Hkv * p.splits * ((room + 128 * p.m - 1) / (128 * p.m)));
        if constexpr (SCORES == kPlain) {
            if (p.m == 2) {
                hipLaunchKernelGGL((kv_weights_tile<BITS, SCORES, 2>), grid, dim3(kWeightThreads), 0, s, a, p.splits);
                return hipGetLastError();
            }
        }
        hipLaunchKernelGGL((kv_weights_tile<BITS, SCORES, 1>), grid, dim3(kWeightThreads), 0, s, a, p.splits);
        return hipGetLastError();
    }
    const int chunk = kWeightWaves * kGroup * p.turns, chunks = (room + chunk - 1) / chunk;
    const long long items = static_cast<long long>(a.B) * chunks;
    const dim3 grid(static_cast<unsigned>((items + 7) / 8 * 8 * a.Hkv));
    if (p.n == 1)
        hipLaunchKernelGGL((kv_weights_rows16<BITS, SCORES, 1>), grid, dim3(kWeightThreads), 0, s, a, chunks, p.turns);
    else if (p.n == 2)
        hipLaunchKernelGGL((kv_weights_rows16<BITS, SCORES, 2>), grid, dim3(kWeightThreads), 0, s, a, chunks, p.turns);
    else
        hipLaunchKernelGGL((kv_weights_rows16<BITS, SCORES, 4>), grid, dim3(kWeightThreads), 0, s, a, chunks, p.turns);
    return hipGetLastError();
}

template <int BITS>
hipError_t launch_bits(const KvWeightsArgs& a, const Plan& p, hipStream_t s) {
    if (a.softcap > 0.0f) return launch_scores<BITS, kWideCap>(a, p, s);
    return a.slopes ? launch_scores<BITS, kFancy>(a, p, s) : launch_scores<BITS, kPlain>(a, p, s);
}

}  // namespace

size_t kv_weights_workspace(int T, int Hq, int Hkv, int B, int max_kv) {
    // with a cap or bias there are as many workgroups or more, and as many shares or fewer
    const Plan p = plan(T, Hq, Hkv, B, max_kv, true);
    return p.splits > 1 ? static_cast<size_t>(p.splits) * B * Hkv * max_kv * sizeof(float) : 0;
}

bool kv_weights_fits(int T, int Hq, int Hkv, int B, int max_kv) {
    // workgroups of 128 tokens, each sequence's first one whole, below 2^24; shares are taken far below that
    const double items = static_cast<double>(B) * ((static_cast<double>(max_kv) + 127) / 128);
    return Hkv <= 65535 && (items + 8) * Hkv <= (1 << 24) - 1 && static_cast<long long>(T) * Hq <= (1LL << 26);
}

hipError_t launch_kv_weights(const KvWeightsArgs& a, int bits, hipStream_t s) {
    const int room = a.max_pages << a.page_log2;
    const Plan p = plan(a.T, a.Hq, a.Hkv, a.B, room, a.softcap == 0.0f && !a.slopes);
    const hipError_t e = bits == 8 ? launch_bits<8>(a, p, s) : launch_bits<4>(a, p, s);
    if (e != hipSuccess || p.splits <= 1) return e;
    const int chunks = (room + kWeightThreads - 1) / kWeightThreads;
    hipLaunchKernelGGL(kv_weights_join, dim3(static_cast<unsigned>(a.B) * a.Hkv * chunks), dim3(kWeightThreads), 0, s, a, p.splits, chunks);
    return hipGetLastError();
}

}  // namespace spin
