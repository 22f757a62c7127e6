// spin_kv_attn / spin_kv_attn_shared / spin_kv_attn_ex kernels: attention over the paged INT4 or
// INT8 KV cache (the abstract's 4-bit KV cache; page "SpinQuant, Reproduced",
// Q5: queries and keys both carry R3, so their products are unchanged).
//
// For query row q (one token, one head) over the visible tokens j of its
// sequence, with integer codes a_j, b_j and fp16 scales ks_j, vs_j
//   z_j = scale ks_j (q . a_j),  z <- cap tanh(z / cap),  z <- z - slope |pos - j|
//   o   = sum_j e^(z_j) vs_j b_j / sum_j e^(z_j),   0 where nothing is visible.
// Codes go into the fp16 matrix cores as the integers they are: exact.  The
// value scale goes into the exponent,
//   t_j = z_j log2(e) + log2(vs_j),  w_j = 2^(t_j - M),  o = sum w_j b_j / sum w_j / vs_j,
// M no more than the largest t_j and at most kSlack below it, so that the largest of the weights, which are rounded to
// fp16 for the second product, lies between 1 and 2^kSlack = 256 whatever the scales are.  The rounding is half a step,
// 2^-11 relative, of each weight; a weight below 2^-14 is off by up to 2^-25, at most 2^-25 of the largest.  Scores,
// maxima and sums are float32; exponentials, logarithms and reciprocals are the hardware's, off by a unit in the last
// place, 2^-23, which the rounding of the weights passes by far.
//
// Weights are rounded because the matrix instructions take 16 bits, and to fp16 because it holds three bits more than bf16; the
// rounding goes to either side, and the sum that divides is of the weights as they were, as the logarithm below needs it.
// Outputs are off by 2.4 to 2.6e-4 (rms, relative), of which the output's own fp16 leaves 2.1e-4: three of ten values are a
// step beside the nearest.
//
// With a tree a row sees the context and, of its sequence's new tokens, those that its bits name.  Only steps that hold new
// tokens look at them (tree_mask).  Measured with 32 + 8 heads: a tree of 16 tokens on 1000, INT4, 12 us; 16 of 60 on 4096
// 98 - 112 us (as many rows in order 97 - 107), INT8 and capped 119 - 134 (127 - 134), with a distance bias 153 (120), INT8
// with both 183 (144): there the masks spill 20 to 26 registers; 64 of 8 on 2000 54 (55); 16 of 60 on 500 behind a prefix
// of 4096 131 (127), 64 of 8 78 (77).
//
// A row's log sum e^z is M and the sum of w_j / vs_j, which attention divides by, together.  It keeps what the products are
// off by (key_operand_small), averaged over the tokens: 9e-6 rms at 4 bits, 1e-6 at 8.
//
// Both products are computed transposed: S^T = A Q^T leaves a lane with one
// query and four tokens of a tile of 16, which is what the second product O^T =
// B^T W^T takes as its right operand: the weights of two tiles of tokens go
// from accumulators to operands without leaving the lane, and the rescaling of
// a row is one multiplication per register.
#include "kv_batch.h"
#include "kv_scores.h"
#include "spin_device.h"
#include "spin_internal.h"

namespace spin {
namespace {

constexpr int kAttnThreads = 256;
constexpr int kAttnWaves = kAttnThreads / 64;
constexpr int kRows = 16;                 // query rows of a tile
constexpr int kStep = 32;                 // tokens a wave takes at a time
// Shares of a sequence's tokens, tiles of 16 rows: waves that fill the card, and per wave of a workgroup the fewest tokens
// worth a share and those of a share where there are workgroups enough without.  Up to kShort tokens there is one share and
// no join (one token on 1000 tokens 11.9 us a call against 16.7 with shares of 128 and a join, 16 on 1500 15.4 and 17.7; 1 on
// 3000 21.9 and 16.3); up to kShortest and in many workgroups four waves do (256 on 300: 28 us, with eight 39).
constexpr int kRowsWaves = 4096, kLeastShare = 32, kLongShare = 1024;
constexpr int kShort = 2048, kShortest = 512;
constexpr int kTilesWanted = 256, kTilesLeast = 256;      // tiles of 128 and 256: one a CU
constexpr int kMostSplits = 256;
constexpr int kCounted = 256;             // sequences up to which tiles of 16 rows are found by counting
constexpr float kSlack = 8.0f;            // M may lag a row's maximum by this many powers of two
static_assert(kSlack <= 12.0f, "weights of 2^kSlack lie well below the largest fp16, 65504");
// Rows on the same tokens, and rows times tokens of all heads, from which tiles of 128 rows are taken, and of 256 (twice
// that for a sequence's own tokens: masks leave half of them).  Measured in us on tiles of 16, 128, 256 rows with 32 + 8
// heads: 16 sequences on 4096 tokens with 64 rows a key head each 56, 58, 77; 128 89, 67, 84; 256 153, 94, 106; 512 278,
// 183, 151; 2048 1005, 661, 559.  One sequence on 4096: 256 rows 27, 29, 32; 512 36, 34, 40; 8192 219, 147, 143.  A prefix of
// 2048: 1024 rows 48, 54, 62; of 8192: 512 55, 55, 60, 2048 172, 137, 132; of 32768: 128 53, 54, 62, 256 89, 72, 74, 2048 604,
// 369, 335.
constexpr int kManyRows = 64;
constexpr double kTileWork = 1 << 25, kWideWork = 1 << 27;
constexpr int kPartial = 130;             // floats of a row's partial result: 128 sums, M, sum

// Code j of an octet, of eight tokens: w[BITS / 4 * token + ...], as an operand; 16 times the code for odd j at 4 bits,
// where it is not shifted down.
template <int BITS>
__device__ __forceinline__ h8 value_operand(const uint32_t* w, int j) {
    Frag f;
    constexpr int kW = BITS / 4;   // dwords of an octet
    const int byte = BITS == 4 ? j >> 1 : j & 3, dw = BITS == 4 ? 0 : j >> 2;
    const uint32_t sel = 0x0c000c04u + byte * 0x00010001u;   // byte of the first token below, of the second above
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t x = __builtin_amdgcn_perm(w[kW * (2 * i) + dw], w[kW * (2 * i + 1) + dw], sel);
        if (BITS == 4)
            f.w[i] = j & 1 ? minus((x & 0x00F000F0u) ^ 0x64806480u, 1152.0f) : minus((x & 0x000F000Fu) ^ 0x64086408u, 1032.0f);
        else
            f.w[i] = minus(x ^ 0x64806480u, 1152.0f);
    }
    return f.v;
}

template <int N>
__device__ __forceinline__ float row_lane(float v) {   // lane N of the 16 lanes of a row, for all of them
    return __uint_as_float(__builtin_amdgcn_update_dpp(0, static_cast<int>(__float_as_uint(v)), 0x150 + N, 0xF, 0xF, true));
}

// Of 32 tokens, the `first` of them counted among a sequence's new ones (below 0: the context), those that a row of the
// tree names, the context among them.
__device__ __forceinline__ uint32_t tree_bits(const uint32_t* __restrict__ row, int words, int first) {
    const int w = first >> 5;
    const uint32_t lo = w < 0 ? ~0u : w < words ? row[w] : 0u;
    const uint32_t hi = w + 1 < 0 ? ~0u : w + 1 < words ? row[w + 1] : 0u;
    return static_cast<uint32_t>(((static_cast<unsigned long long>(hi) << 32) | lo) >> (first & 31));
}

// Is any of 32 tokens new, the `first` of them counted among the new ones.
__device__ __forceinline__ bool any_new(int first) { return first > -32; }

// A new token's position, held to what differences of two fit 32 bits with.
__device__ __forceinline__ int position(const KvAttnArgs& a, int t) { return min(max(a.positions[t], 0), 1 << 30); }

// Masks a row's exponents of N of 32 tokens, the `first` of which is counted among the new ones, by the tree and the
// window, and adds the bias where some of them are new: their distances go by their positions, the others' by `rel`, the
// row's position less the lane's first place.  Exponent e is that of token lane0 + e % 4 + 128 / N (e / 4) of the 32.  One
// position at a time: all of them at once take registers that the main path lacks.
template <int SCORES, int N, typename X>
__device__ __forceinline__ void tree_mask(const KvAttnArgs& a, X& x, int t, bool valid, int first, int lane0, int news, int new0, int pos, int rel,
                                          float slope) {
    const uint32_t named = valid ? tree_bits(a.tree + static_cast<long long>(t) * a.tree_words, a.tree_words, first) >> lane0 : 0u;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const int c = 128 / N * (e >> 2) + (e & 3);
        x[e] = named >> c & 1 ? x[e] : -__builtin_inff();
    }
    if (a.window <= 0 && !(biased(SCORES) && a.slopes)) return;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        asm volatile("" ::: "memory");
        const int c = 128 / N * (e >> 2) + (e & 3), i = first + lane0 + c;
        const int far = i >= 0 && i < news ? pos - position(a, new0 + i) : rel - c;
        if (biased(SCORES) && any_new(first)) x[e] = __builtin_fmaf(-slope, __builtin_fabsf(static_cast<float>(far)), x[e]);
        if (a.window > 0)
            x[e] = static_cast<uint32_t>(far) + static_cast<uint32_t>(a.window) - 1u < 2u * static_cast<uint32_t>(a.window) - 1u ? x[e] : -__builtin_inff();
    }
}

// The logarithm of a row's sum of exponentials.
__device__ __forceinline__ float log_sum(float M, float l) {
    return l == 0.0f ? -__builtin_inff() : (M + __builtin_amdgcn_logf(l)) * 0.6931471805599453f;
}

// Which tokens a workgroup has.
struct Span {
    const int32_t* table;
    int n_table;        // entries of the table that may be read
    int tokens;         // tokens the table's pages hold
    int base;           // position of the first of them
};

// Tiles are numbered through the sequences without gaps, by counting them, 64 sequences at a time.  floor(q_start[b] G /
// ROWS) + b would number them, with gaps, in one step, but workgroups go to the XCDs and to the shader engines of each in
// a fixed turn, and gaps at every second number leave half of those without work: 16 sequences of 128 rows on 4096
// tokens took 113 us so, 70 without gaps (of 64 rows, 176 and 96); 32 single tokens with 16 heads a key head on 8192, 105
// and 62.  From some hundred sequences on counting takes longer than a tile of 16 rows has (256 single
// tokens of 16 heads on 500 tokens: 36 us counted, 39 with gaps; 512: 83 and 78; 4096 of 4 heads on 64: 609 and 224); there
// numbers with gaps visit the XCDs in a turn that shifts.

// Tiles of sequence b0 + lane.
template <int ROWS>
__device__ __forceinline__ int count_tiles(const KvAttnArgs& a, int G, int b0, int lane) {
    const int i = b0 + lane;
    const int rows = i < a.B ? (within(a.q_start[i + 1], a.T) - within(a.q_start[i], a.T)) * G : 0;
    return rows > 0 ? (rows + ROWS - 1) / ROWS : 0;
}

// Where `tile` is among the lanes' tiles, b is set and the tile's number in its sequence returned, otherwise its number
// behind them.
__device__ __forceinline__ int find_tile(int tiles, int b0, int tile, int& b) {
    const int upto = sums_up_to(tiles);
    const unsigned long long hit = __ballot(upto > tile);
    if (hit == 0) return tile - __builtin_amdgcn_readlane(upto, 63);
    const int l = __builtin_ctzll(hit);
    b = b0 + l;
    return tile - (__builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(tiles, l));
}

// Up to 64 sequences, a lane each: their tiles' counts and their numbers in the order of their lengths, the longest first,
// in steps of a sixteenth of the longest.  Workgroups take sequences in this order, which costs equal lengths 0.5 us and
// brings 64 of 0.25 .. 1 times 8192 tokens from 85 to 73 us, 48 of u^4 times 16384 (u even in 0 .. 1) from 92 to 59.
__device__ __forceinline__ void longest_first(const KvAttnArgs& a, int lane, int& tiles, int& id) {
    const bool there = lane < a.B;
    const float length = there ? static_cast<float>(context(a, lane)) : 0.0f;
    float top = max_over_groups(length);
#pragma unroll
    for (int m = 1; m < 16; m <<= 1) top = __builtin_fmaxf(top, __shfl_xor(top, m, 64));
    const int step = there ? 15 - min(static_cast<int>(length * 15.999f * __builtin_amdgcn_rcpf(__builtin_fmaxf(top, 1.0f))), 15) : 16;
    int rank = lane, before = 0;       // lanes without a sequence stay behind the others
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const unsigned long long same = __ballot(step == k);
        const int at = before + __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(same >> 32), __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(same), 0));
        rank = step == k ? at : rank;
        before += __popcll(same);
    }
    tiles = __builtin_amdgcn_ds_permute(rank << 2, tiles);
    id = __builtin_amdgcn_ds_permute(rank << 2, id);
}

// One tile of 16 query rows of one key head, over a share of the tokens: the
// WAVES (4 or 8) waves take steps of 32 tokens in turn and are joined in LDS.
// With one share the rows are finished here, with what a prefix has left in the
// workspace in an earlier launch, otherwise they go to the workspace, [share][T *
// Hq] rows.
//
// Bound at few rows: reading the cache, 2 (16 BITS + 2) bytes a token and head.
// Codes go from memory to the lane that multiplies them, without LDS: 16 rows
// leave nothing to share between waves.  Measured: 8 tokens of 32 + 8 heads on
// 32768 each, INT8, capped, 102 us + 5 us for the join (550 MB, 5.4 TB/s); 64
// on 0.25 .. 1 times 8192, INT4, 73 us (340 MB, 4.7 TB/s; the vector pipes are
// busy half of it with turning INT4 codes to fp16, and the last sequences run
// alone), on 8192 each 5.4 TB/s; 1 on 1000 10 us, of which four loads that wait
// for each other (sequence, length, page, codes) and four steps.
template <int BITS, int SCORES, int WAVES, bool TREE>
__global__ __launch_bounds__(64 * WAVES, TREE && BITS == 4 && SCORES == kPlain ? 4 : 3) void kv_attn_rows16(KvAttnArgs a, int prefix_tiles, int prefix_splits, int prefix_chunk,
                                                                  int own_tiles, int own_splits, int own_chunk) {
    __shared__ float o_sh[WAVES][kRows][129];
    __shared__ float m_sh[WAVES][kRows], l_sh[WAVES][kRows];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    const int G = a.Hq / a.Hkv;
    // Workgroup L runs on XCD L % 8: the heads of an item follow each other on one, so that the lines that hold several
    // heads' scales come into one L2.
    const int h = (blockIdx.x >> 3) % a.Hkv;
    const int eight = (blockIdx.x >> 3) / a.Hkv;
    const int index = eight * 8 + ((blockIdx.x + eight + (eight >> 3)) & 7);   // gaps in the numbers visit every XCD
    const int prefix_items = prefix_tiles * prefix_splits;
    if (index >= prefix_items + own_tiles * own_splits) return;
    const bool shared = index < prefix_items;
    const int item = shared ? index : index - prefix_items;
    const int splits = shared ? prefix_splits : own_splits;
    const int tile = item / splits, split = item - tile * splits;
    const int first_slot = shared ? 0 : prefix_splits;   // of the workspace

    // the rows: (token, head of the group) pairs, of one sequence or (prefix) of all
    Span span;
    int t, head;             // this lane's row
    bool valid;
    int b;
    int fresh = 0x7FFFFFFF, new0 = 0, news = 0;      // TREE: place of the sequence's first new token, its row, how many
    if (shared) {
        const int r = tile * kRows + n;
        t = r / G;
        head = h * G + r - t * G;
        b = t < a.T ? find_sequence(a.q_start, a.B, t) : -1;
        valid = b >= 0;
        span = {a.prefix_table, (a.prefix_len + (1 << a.page_log2) - 1) >> a.page_log2, a.prefix_len, 0};
    } else {
        int own = tile;
        if (a.B == 1) {
            b = 0;
        } else if (a.B <= 64) {
            int tiles = count_tiles<kRows>(a, G, 0, lane), id = lane;
            if (a.B > 8 && a.max_pages << a.page_log2 > kShort) {
                // Two workgroups of eight waves a CU: the longest first, and where they all run at once those that come
                // second to a CU the shortest first.
                longest_first(a, lane, tiles, id);
                const int all = __builtin_amdgcn_readlane(sums_up_to(tiles), 63), half = 256 / a.Hkv;
                if (all <= 2 * half && own >= half && own < all) own = half + all - 1 - own;
            }
            b = -1;
            own = find_tile(tiles, 0, own, b);
            if (b < 0) return;
            b = __builtin_amdgcn_readlane(id, b);
        } else if (a.B <= kCounted) {
            b = -1;
            for (int b0 = 0; b0 < a.B && b < 0; b0 += 64) own = find_tile(count_tiles<kRows>(a, G, b0, lane), b0, own, b);
            if (b < 0) return;             // the grid has room for a ragged tile of every sequence
        } else {
            b = find_last64(a.B, lane, [&](int i) { return static_cast<long long>(a.q_start[i]) * G / kRows + i <= tile; });
            own -= static_cast<int>(static_cast<long long>(within(a.q_start[b], a.T)) * G / kRows + b);
        }
        const int q0 = within(a.q_start[b], a.T), q1 = within(a.q_start[b + 1], a.T);
        const int r = own * kRows + n;
        valid = r >= 0 && r < (q1 - q0) * G;
        const int i = valid ? static_cast<int>(static_cast<unsigned>(r) / static_cast<unsigned>(G)) : 0;
        t = q0 + i;
        head = h * G + (valid ? r - i * G : 0);
        span = {a.page_table + static_cast<long long>(b) * a.max_pages, a.max_pages, context(a, b), a.prefix_len};
        if (TREE) {
            new0 = __builtin_amdgcn_readfirstlane(q0);
            news = __builtin_amdgcn_readfirstlane(q1 - q0);
            fresh = __builtin_amdgcn_readfirstlane(placed(a.kv_len[b])) - news;
        }
    }
    if (__ballot(valid) == 0) return;      // the same 16 rows in every wave: the workgroup leaves together

    int pos = 0, both = 0;                 // the row's position, and the tokens that it sees whatever their order
    if (TREE) {
        if (valid && a.positions) pos = position(a, t);
    } else if (valid) {
        pos = a.prefix_len + placed(a.kv_len[b]) - a.q_start[b + 1] + t;
        if (a.bidir_len) both = max(a.bidir_len[b], 0);    // no token stands below 0: differences of it fit 32 bits
    }
    // the tokens that any of the rows sees
    int lo = 0, hi = span.tokens;
    int pmin = valid ? pos : 0x7FFFFFFF, pmax = valid ? max(pos + 1, both) : -0x7FFFFFFF, wmax = valid ? pos : -0x7FFFFFFF;
    int bmin = valid ? both : 0x7FFFFFFF;
#pragma unroll
    for (int x = 1; x < 16; x <<= 1) {
        pmin = min(pmin, __shfl_xor(pmin, x, 64));
        pmax = max(pmax, __shfl_xor(pmax, x, 64));
        wmax = max(wmax, __shfl_xor(wmax, x, 64));
        bmin = min(bmin, __shfl_xor(bmin, x, 64));
    }
    if (a.causal) hi = min(hi, pmax - span.base);
    if (a.window > 0) {
        lo = static_cast<int>(max(static_cast<long long>(pmin) - a.window + 1 - span.base, 0LL));
        if (TREE)
            lo = min(lo, max(fresh, 0));       // new tokens stand where `positions` says
        else
            hi = static_cast<int>(min(static_cast<long long>(hi), static_cast<long long>(wmax) + a.window - span.base));
    }
    int step0 = lo / kStep;
    const int steps_all = hi > lo ? (hi + kStep - 1) / kStep - step0 : 0;
    const int share = max((steps_all + splits - 1) / splits, (shared ? prefix_chunk : own_chunk) / kStep);
    const int steps = __builtin_amdgcn_readfirstlane(max(0, min(share, steps_all - split * share)));
    step0 = __builtin_amdgcn_readfirstlane(step0 + split * share);
    // every row sees every token of the steps whole0 .. whole1 - 1
    int whole0 = 0, whole1 = span.tokens;
    if (a.causal) whole1 = min(whole1, max(pmin + 1, bmin) - span.base);
    if (TREE) whole1 = min(whole1, fresh);
    if (a.window > 0) {
        whole0 = static_cast<int>(max(static_cast<long long>(wmax) - a.window + 1 - span.base, 0LL));
        whole1 = static_cast<int>(min(static_cast<long long>(whole1), static_cast<long long>(pmin) + a.window - span.base));
    }
    whole0 = __builtin_amdgcn_readfirstlane((whole0 + kStep - 1) / kStep);
    whole1 = __builtin_amdgcn_readfirstlane(whole1 >= 0 ? whole1 / kStep : -1);

    // queries, in the order of the keys' codes: lane (n, g) holds values 32 g .. 32 g + 31 of row n
    h8 q[4];
    {
        const uint16_t* src = a.Q + (static_cast<long long>(t) * a.Hq + head) * 128 + 32 * g;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            Frag raw, f;
            const u4 x = valid ? *reinterpret_cast<const u4*>(src + 8 * j) : u4{0, 0, 0, 0};
            raw.w[0] = x.x; raw.w[1] = x.y; raw.w[2] = x.z; raw.w[3] = x.w;
#pragma unroll
            for (int i = 0; i < 8; ++i) f.v[i] = raw.v[order8<BITS>(i)];
            q[j] = f.v;
        }
    }
    // what the sum over a query starts from (key_operand_small)
    f4 start;
    {
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += static_cast<float>(q[j][e]);
        }
        const float c = sum_over_groups(sum) * (BITS == 4 ? -0x1p-21f : -0x1p-17f);
        start = f4{c, c, c, c};
    }
    const float slope = biased(SCORES) && a.slopes && valid ? a.slopes[head] * kLog2e : 0.0f;
    const bool near_cap = SCORES == kCapped || (SCORES == kFancy && a.softcap > 0.0f);
    const Cap cap = cap_of<SCORES>(a);
    const float key_factor = held(cap.factor * 0x1p24f);

    // Of the wave's next 32 steps, a lane each and half of a step: where the 16 tokens lie, as the number of the first, ~0
    // if nowhere.
    uint32_t place_lo = 0, place_hi = 0;
    auto load_places = [&](int i) __attribute__((always_inline)) {      // the wave's steps i .. i + 31
        const long long j = static_cast<long long>(step0 + wave + WAVES * (i + (lane >> 1))) * kStep + 16 * (lane & 1);
        const int page = j < span.tokens ? span.table[min(static_cast<int>(j >> a.page_log2), span.n_table - 1)] : -1;
        const long long token = ((static_cast<long long>(page) * a.Hkv + h) << a.page_log2) + (j & ((1 << a.page_log2) - 1));
        const bool good = page >= 0 && page < a.n_pages;
        place_lo = good ? static_cast<uint32_t>(token) : ~0u;
        place_hi = good ? static_cast<uint32_t>(token >> 32) : ~0u;
    };
    // A step's codes and scales.  Lane (n, g) takes 32 codes of token n of each 16 and an octet of tokens 4 g .. 4 g + 3,
    // and the scales of one token: of lanes 0 .. 7 of a row of 16 lanes token 4 g + l of the first 16 (l < 4) or 4 g + l - 4
    // of the second, lanes 8 .. 15 again.  The next step's keys are loaded as soon as these are used, the values as soon
    // as these are: each load has the other half of a step to arrive in, with one set of registers, so that at 4 bits four
    // waves fit a SIMD.
    uint32_t kraw[2][BITS], vraw[2 * BITS], ks_raw = 0, vs_raw = 0;
    bool there = false;
    const int s_half = (n >> 2) & 1, s_token = 4 * g + (n & 3);
    auto place = [&](int i, int half, bool& good) __attribute__((always_inline)) {
        const uint32_t lo_ = __builtin_amdgcn_readlane(place_lo, 2 * (i & 31) + half);
        const uint32_t hi_ = __builtin_amdgcn_readlane(place_hi, 2 * (i & 31) + half);
        good = hi_ != ~0u;
        return good ? (static_cast<unsigned long long>(hi_) << 32) | lo_ : static_cast<unsigned long long>(h) << a.page_log2;
    };
    auto fetch_keys = [&](int i) __attribute__((always_inline)) {
        bool good[2];
        const unsigned long long token[2] = {place(i, 0, good[0]), place(i, 1, good[1])};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const u4* kp = reinterpret_cast<const u4*>(a.K_codes + token[half] * (16 * BITS));
#pragma unroll
            for (int x = 0; x < BITS / 4; ++x) {
                const u4 y = kp[(n * 4 + g) * (BITS / 4) + x];
                kraw[half][4 * x] = y.x; kraw[half][4 * x + 1] = y.y; kraw[half][4 * x + 2] = y.z; kraw[half][4 * x + 3] = y.w;
            }
        }
        const unsigned long long at = (s_half ? token[1] : token[0]) + s_token;
        ks_raw = a.K_scale[at];
        vs_raw = a.V_scale[at];
        there = (s_half ? good[1] : good[0]) && (step0 + wave + WAVES * i) * kStep + 16 * s_half + s_token < span.tokens;
    };
    auto fetch_values = [&](int i) __attribute__((always_inline)) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            bool good;
            const u4* vp = reinterpret_cast<const u4*>(a.V_codes + place(i, half, good) * (16 * BITS));
#pragma unroll
            for (int x = 0; x < BITS / 4; ++x) {
                const u4 z = vp[(g * 16 + n) * (BITS / 4) + x];
                vraw[half * BITS + 4 * x] = z.x; vraw[half * BITS + 4 * x + 1] = z.y;
                vraw[half * BITS + 4 * x + 2] = z.z; vraw[half * BITS + 4 * x + 3] = z.w;
            }
        }
    };

    // M: what a row's exponents are relative to.  It follows the row's maximum by more than kSlack powers of two, up, and
    // is set to it with the row's first token (`low` is infinite until then).
    float M = 0.0f, low = __builtin_inff(), l_sum = 0.0f;
    f4 o[8] = {};

    const int turns = steps > wave ? (steps - wave + WAVES - 1) / WAVES : 0;
    if (turns > 0) {
        load_places(0);
        fetch_keys(0);
        fetch_values(0);
    }
    for (int i = 0; i < turns; ++i) {
        const float ks = __half2float(__ushort_as_half(static_cast<unsigned short>(ks_raw)));
        const float vs = __half2float(__ushort_as_half(static_cast<unsigned short>(vs_raw)));
        const bool here = there;
        // a scale of 0 has codes of 0: its weight stays in the sum of weights through any other scale
        const float vsf = vs == 0.0f ? 0x1p-24f : vs;
        const float kf = here ? __builtin_fmaf(ks, key_factor, ks * 0.0f) : 0.0f;      // NaN where ks is not finite
        const float lv = here ? __builtin_amdgcn_logf(vsf) : -__builtin_inff();
        const float rv = here && vsf <= 65504.0f ? __builtin_amdgcn_rcpf(vsf) : 0.0f;
        const int st = step0 + wave + WAVES * i;
        const int j0 = st * kStep + span.base;

        float x[8];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            f4 s = start;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                s = __builtin_amdgcn_mfma_f32_16x16x32_f16(key_operand_small<BITS>(kraw[half] + j * (BITS / 4)), q[j], s, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < 4; ++r) x[4 * half + r] = s[r];
        }
        // behind the last step it is loaded once more, for nothing
        const int next = i + 1 < turns ? i + 1 : i;
        if ((next & 31) == 0 && next > 0) load_places(next);
        fetch_keys(next);
        const float from = SCORES == kFancy || SCORES == kCapped ? M - cap.top : M;
        const float rel = static_cast<float>(pos - j0 - 4 * g);
        const float slope_here = TREE && any_new(st * kStep - fresh) ? 0.0f : slope;       // tree_mask adds it then
        auto exponent = [&](int e, float k, float lm, bool capped) __attribute__((always_inline)) {
            if (biased(SCORES)) lm = __builtin_fmaf(-slope_here, __builtin_fabsf(rel - static_cast<float>(16 * (e >> 2) + (e & 3))), lm);
            x[e] = SCORES == kWideCap ? capped_wide(x[e] * k, cap.top, cap.rtop) + lm
                                      : capped ? capped_plus(x[e] * k, cap.top, lm) : __builtin_fmaf(x[e], k, lm);
        };
#define SPIN_ONE(N, CAP) exponent(N, row_lane<N>(kf), row_lane<N>(lv) - from, CAP);
#define SPIN_ALL(CAP)                                                                     \
    SPIN_ONE(0, CAP) SPIN_ONE(1, CAP) SPIN_ONE(2, CAP) SPIN_ONE(3, CAP) SPIN_ONE(4, CAP) \
    SPIN_ONE(5, CAP) SPIN_ONE(6, CAP) SPIN_ONE(7, CAP)
        if (near_cap) {
            SPIN_ALL(true)
        } else {
            SPIN_ALL(false)
        }
#undef SPIN_ALL
#undef SPIN_ONE
        if (st < whole0 || st >= whole1) {
            asm volatile("" ::: "memory");     // keeps this a branch
            const int rel = pos - j0 - 4 * g;
            const int end = a.causal ? max(rel, both - j0 - 4 * g - 1) : 32;
            const uint32_t off = a.window > 0 ? static_cast<uint32_t>(rel) + static_cast<uint32_t>(a.window) - 1u : 32u;
            const uint32_t wide = a.window > 0 ? 2u * static_cast<uint32_t>(a.window) - 1u : 64u;
            if (TREE) {
                tree_mask<SCORES, 8>(a, x, t, valid, st * kStep - fresh, 4 * g, news, new0, pos, rel, slope);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int c = 16 * (e >> 2) + (e & 3);
                    const bool seen = (end >= c) & (off - static_cast<uint32_t>(c) < wide);
                    x[e] = seen ? x[e] : -__builtin_inff();
                }
            }
        }
        float top = x[0];
#pragma unroll
        for (int e = 1; e < 8; ++e) top = __builtin_fmaxf(top, x[e]);
        top = max_over_groups(top);
        if (__ballot(top > kSlack || top < low) != 0) {
            const bool none = top == -__builtin_inff(), first = low > 0.0f;
            const float up = none ? 0.0f : first ? top : __builtin_fmaxf(top, 0.0f);
            const float keep = first ? 0.0f : __builtin_amdgcn_exp2f(-up);     // nothing is kept of nothing, whatever up is
            low = none ? low : -__builtin_inff();
            M += up;
            l_sum *= keep;
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] *= keep;
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] -= up;
        }
        const float r8[8] = {row_lane<0>(rv), row_lane<1>(rv), row_lane<2>(rv), row_lane<3>(rv),
                             row_lane<4>(rv), row_lane<5>(rv), row_lane<6>(rv), row_lane<7>(rv)};
        h8 w_op;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const f2 w = {__builtin_amdgcn_exp2f(x[2 * e]), __builtin_amdgcn_exp2f(x[2 * e + 1])};
            l_sum = __builtin_fmaf(w.x, r8[2 * e], __builtin_fmaf(w.y, r8[2 * e + 1], l_sum));
            const h2 p = __builtin_convertvector(w, h2);
            w_op[2 * e] = p.x;
            w_op[2 * e + 1] = p.y;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            o[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(value_operand<BITS>(vraw, j), w_op, o[j], 0, 0, 0);
        fetch_values(next);
    }
    if (BITS == 4) {
#pragma unroll
        for (int j = 1; j < 8; j += 2) o[j] *= 0.0625f;      // 16 times the code
    }
    if (low > 0.0f) M = -__builtin_inff();     // no token seen

    // join the waves
    asm volatile("" ::"s"(a.lse));             // read now: behind the sums everything would wait for it
    l_sum = sum_over_groups(l_sum);
    if (g == 0) m_sh[wave][n] = M;
    __syncthreads();
    float M_all = m_sh[0][n];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) M_all = __builtin_fmaxf(M_all, m_sh[w][n]);
    const float f = M == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(M - M_all);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
        for (int r = 0; r < 4; ++r) o_sh[wave][n][8 * (4 * g + r) + j] = o[j][r] * f;
    }
    if (g == 0) l_sh[wave][n] = l_sum * f;
    __syncthreads();
    // 16 threads a row, 8 values each
    if (WAVES > 4 && threadIdx.x >= 256) return;
    const int row = threadIdx.x >> 4, c = threadIdx.x & 15;
    const int t_row = __shfl(t, row, 64), head_row = __shfl(head, row, 64);   // lane `row` of every wave has row `row`
    const bool valid_row = __shfl(static_cast<int>(valid), row, 64) != 0;
    if (!valid_row) return;
    float l_all = 0.0f, out[8] = {};
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        l_all += l_sh[w][row];
#pragma unroll
        for (int i = 0; i < 8; ++i) out[i] += o_sh[w][row][8 * c + i];
    }
    const long long at = static_cast<long long>(t_row) * a.Hq + head_row;
    float M_row = m_sh[0][row];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) M_row = __builtin_fmaxf(M_row, m_sh[w][row]);
    const bool last = prefix_tiles == 0 && own_splits == 1;        // what the prefix gave is there: an earlier launch's
    if (!last) {
        float* p = a.partial + ((first_slot + split) * static_cast<long long>(a.T) * a.Hq + at) * kPartial;
        if (l_all != 0.0f) {
#pragma unroll
            for (int i = 0; i < 4; ++i) reinterpret_cast<f2*>(p + 8 * c)[i] = f2{out[2 * i], out[2 * i + 1]};
        }
        if (c == 0) {
            p[128] = M_row;
            p[129] = l_all;
        }
        return;
    }
    // joins them, as kv_attn_join does, four shares at a time
    float M_run = l_all == 0.0f ? -__builtin_inff() : M_row;
    for (int s0 = 0; s0 < prefix_splits; s0 += 4) {
        f2 ml[4], y[4][4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const float* p = a.partial + (min(s0 + s, prefix_splits - 1) * static_cast<long long>(a.T) * a.Hq + at) * kPartial;
            ml[s] = *reinterpret_cast<const f2*>(p + 128);
#pragma unroll
            for (int i = 0; i < 4; ++i) y[s][i] = reinterpret_cast<const f2*>(p + 8 * c)[i];
        }
        float M_new = M_run;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            ml[s].y = s0 + s < prefix_splits ? ml[s].y : 0.0f;
            M_new = ml[s].y == 0.0f ? M_new : __builtin_fmaxf(M_new, ml[s].x);
        }
        const float keep = M_run == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(M_run - M_new);
        l_all = l_all == 0.0f ? 0.0f : l_all * keep;
#pragma unroll
        for (int i = 0; i < 8; ++i) out[i] = l_all == 0.0f ? 0.0f : out[i] * keep;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            if (ml[s].y == 0.0f) continue;         // no token seen: its sums are not written
            const float f = __builtin_amdgcn_exp2f(ml[s].x - M_new);
            l_all = __builtin_fmaf(ml[s].y, f, l_all);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                out[2 * i] = __builtin_fmaf(y[s][i].x, f, out[2 * i]);
                out[2 * i + 1] = __builtin_fmaf(y[s][i].y, f, out[2 * i + 1]);
            }
        }
        M_run = M_new;
    }
    const float rl = l_all == 0.0f ? 0.0f : 1.0f / l_all;
    if (a.lse && c == 0) a.lse[at] = log_sum(M_run, l_all);
    Frag res;
#pragma unroll
    for (int i = 0; i < 8; ++i) res.v[i] = static_cast<_Float16>(out[i] * rl);
    *reinterpret_cast<u4*>(a.O + at * 128 + 8 * c) = u4{res.w[0], res.w[1], res.w[2], res.w[3]};
}

// ---------------------------------------------------------------------------------------------- many rows

typedef float f16v __attribute__((ext_vector_type(16)));

constexpr int kTileThreads = 512;
constexpr int kTileWaves = kTileThreads / 64;
constexpr int kTileTokens = 64;            // tokens staged at a time

// Two tokens' code j of an octet (w: BITS / 4 dwords a token) as fp16.
template <int BITS>
__device__ __forceinline__ uint32_t value_pair(const uint32_t* w, int j) {
    const int byte = BITS == 4 ? j >> 1 : j & 3, dw = BITS == 4 ? 0 : j >> 2;
    const uint32_t x = __builtin_amdgcn_perm(w[dw], w[BITS / 4 + dw], 0x0c000c04u + byte * 0x00010001u);
    return BITS == 4 ? minus(((j & 1 ? x >> 4 : x) & 0x000F000Fu) ^ 0x64086408u, 1032.0f) : minus(x ^ 0x64806480u, 1152.0f);
}

__device__ __forceinline__ float swap_halves_max(float v) {
    const u2 s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __builtin_fmaxf(__uint_as_float(s.x), __uint_as_float(s.y));
}
__device__ __forceinline__ float swap_halves_sum(float v) {
    const u2 s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(s.x) + __uint_as_float(s.y);
}

// A barrier that orders the waves, and keeps the compiler's order, without waiting for loads in flight.
__device__ __forceinline__ void part_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// The same for tiles of ROWS = 256 rows, 32 a wave, or of 128, 32 for two waves
// that take half of the tokens each.  The waves share 64 tokens at a time,
// which the workgroup turns into fp16 codes in LDS once, keys as [token][d] and
// values as [d][token].
//
// Bound: the vector work of the softmax and of staging beside the matrix work.
// Two waves share a SIMD; a step of 64 tokens and 256 rows holds 2 x 1024
// cycles of MFMA, and 2 x (2 x 850) of exponents and weights, which overlap across
// the waves but for the loads and the staging, 400 - 550 cycles.  Measured: a prompt of 8192 tokens, 32 + 8 heads,
// INT4, 615 - 634 us a call, 690 - 735 traced (0.55 TFLOP, 0.75 - 0.89 PFLOP/s); uneven chunks of 1723
// tokens, 32 + 32 heads, INT8, capped and with a distance bias, on up to 2900,
// 149 - 160 us a call, 172 traced (32 exponentials and reciprocals a lane and 32 tokens more).
template <int BITS, int ROWS, int SCORES, bool TREE>
__global__ __launch_bounds__(kTileThreads, 2) void kv_attn_tile(KvAttnArgs a, int prefix_tiles, int prefix_splits, int prefix_chunk,
                                                                int own_tiles, int own_splits, int own_chunk) {
    constexpr bool kPair = ROWS == 128;            // two waves a row
    constexpr int kBuffers = kPair ? 3 : 2;
    // Rows of one chunk more than they hold, so that eight rows' same chunk lies in different banks and every address
    // is a base and a constant.  Value d is row 16 (d % 8) + d / 8.
    struct Step {
        u4 k[kTileTokens * 17];                    // 16 chunks of 8 values a token, the even ones first
        u4 v[128 * 9];                             // 8 chunks of 8 tokens a value
        f4 f[3][kTileTokens / 4];                  // per token: key factor, log2 of the value scale, its reciprocal
    };
    __shared__ Step sh[kBuffers];
    __shared__ int range_sh[kTileWaves][3];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 31, hf = lane >> 5;
    const int row_wave = kPair ? wave & 3 : wave;
    const int G = a.Hq / a.Hkv;
    // key heads alternate fastest: with 8 of them a head stays on one XCD
    const int h = blockIdx.x % a.Hkv;
    const int prefix_items = prefix_tiles * prefix_splits;
    const int index = blockIdx.x / a.Hkv;
    const bool shared = index < prefix_items;
    const int splits = shared ? prefix_splits : own_splits;
    const int item = shared ? index : index - prefix_items;
    int tile = item / splits;
    const int split = item - tile * splits;
    const int first_slot = shared ? 0 : prefix_splits;
    const int total_splits = prefix_splits + own_splits;

    Span span;
    int t, head, pos = 0, both = 0;
    bool valid;
    int fresh = 0x7FFFFFFF, new0 = 0, news = 0;      // TREE: place of the sequence's first new token, its row, how many
    if (shared) {
        span = {a.prefix_table, (a.prefix_len + (1 << a.page_log2) - 1) >> a.page_log2, a.prefix_len, 0};
        const unsigned r = static_cast<unsigned>(tile) * ROWS + row_wave * 32 + n;
        t = static_cast<int>(r / G);
        head = h * G + static_cast<int>(r - static_cast<unsigned>(t) * G);
        // every row's own sequence: a search in LDS, where the borders fit it
        constexpr int kFit = sizeof(sh) / sizeof(int32_t);
        int32_t* const borders = reinterpret_cast<int32_t*>(sh);
        const bool fits = a.B < kFit;
        if (fits) {
            for (int i = threadIdx.x; i <= a.B; i += kTileThreads) borders[i] = a.q_start[i];
            __syncthreads();
        }
        const int b = t < a.T ? find_sequence(fits ? borders : a.q_start, a.B, t) : -1;
        if (fits) __syncthreads();
        valid = b >= 0;
        if (TREE) {
            if (valid && a.positions) pos = position(a, t);
        } else if (valid) {
            pos = a.prefix_len + placed(a.kv_len[b]) - a.q_start[b + 1] + t;
            if (a.bidir_len) both = max(a.bidir_len[b], 0);    // no token stands below 0: differences of it fit 32 bits
        }
    } else {
        // The longest sequences come first (12 chunks of 7566 tokens on up to 5000: 383 -> 341 us), and of each its last tiles;
        // the grid has room for a ragged tile of every sequence.
        int b = -1;
        if (a.B <= 64) {
            int tiles = count_tiles<ROWS>(a, G, 0, lane), id = lane;
            if (a.B > 1) longest_first(a, lane, tiles, id);
            tile = find_tile(tiles, 0, tile, b);
            if (b < 0) return;
            tile = __builtin_amdgcn_readlane(tiles, b) - 1 - tile;
            b = __builtin_amdgcn_readlane(id, b);
        } else {
            int all = 0;
            for (int b0 = 0; b0 < a.B; b0 += 64) all += count_tiles<ROWS>(a, G, b0, lane);
            all = __builtin_amdgcn_readlane(sums_up_to(all), 63);
            if (tile >= all) return;
            tile = all - 1 - tile;
            for (int b0 = 0; b0 < a.B && b < 0; b0 += 64) tile = find_tile(count_tiles<ROWS>(a, G, b0, lane), b0, tile, b);
            if (b < 0) return;                     // borders that do not ascend
        }
        const int first = tile * ROWS;
        const int q0 = within(a.q_start[b], a.T), q1 = within(a.q_start[b + 1], a.T);
        span = {a.page_table + static_cast<long long>(b) * a.max_pages, a.max_pages, context(a, b), a.prefix_len};
        const int r = first + row_wave * 32 + n;
        valid = r >= 0 && r < (q1 - q0) * G;
        const int i = valid ? static_cast<int>(static_cast<unsigned>(r) / static_cast<unsigned>(G)) : 0;
        t = q0 + i;
        head = h * G + (valid ? r - i * G : 0);
        if (TREE) {
            new0 = __builtin_amdgcn_readfirstlane(q0);
            news = __builtin_amdgcn_readfirstlane(q1 - q0);
            fresh = __builtin_amdgcn_readfirstlane(placed(a.kv_len[b])) - news;
            if (valid && a.positions) pos = position(a, t);
        } else if (valid) {
            pos = a.prefix_len + placed(a.kv_len[b]) - a.q_start[b + 1] + t;
            if (a.bidir_len) both = max(a.bidir_len[b], 0);    // no token stands below 0: differences of it fit 32 bits
        }
    }
    // positions of the wave's rows, then of the workgroup's: which tokens any of them sees
    int pmin = valid ? pos : 0x7FFFFFFF, pmax = valid ? pos : -0x7FFFFFFF;
    int bmin = valid ? both : 0x7FFFFFFF, bmax = valid ? both : -0x7FFFFFFF;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        pmin = min(pmin, __shfl_xor(pmin, m, 64));
        pmax = max(pmax, __shfl_xor(pmax, m, 64));
        bmax = max(bmax, __shfl_xor(bmax, m, 64));
        bmin = min(bmin, __shfl_xor(bmin, m, 64));
    }
    pmin = __builtin_amdgcn_readfirstlane(pmin);
    pmax = __builtin_amdgcn_readfirstlane(pmax);
    bmax = __builtin_amdgcn_readfirstlane(bmax);
    bmin = __builtin_amdgcn_readfirstlane(bmin);
    const bool wave_any = __ballot(valid) != 0;
    if (lane == 0) {
        range_sh[wave][0] = pmin;
        range_sh[wave][1] = pmax;
        range_sh[wave][2] = max(pmax == -0x7FFFFFFF ? pmax : pmax + 1, bmax);
    }
    __syncthreads();
    int lo = 0, hi = span.tokens;
    {
        int gmin = range_sh[0][0], gmax = range_sh[0][1], gend = range_sh[0][2];
#pragma unroll
        for (int w = 1; w < kTileWaves; ++w) {
            gmin = min(gmin, range_sh[w][0]);
            gmax = max(gmax, range_sh[w][1]);
            gend = max(gend, range_sh[w][2]);
        }
        if (gmin == 0x7FFFFFFF) return;    // no row of a sequence: the workgroup leaves together
        if (a.causal) hi = min(hi, gend - span.base);
        if (a.window > 0) {
            lo = static_cast<int>(max(static_cast<long long>(gmin) - a.window + 1 - span.base, 0LL));
            if (TREE)
                lo = min(lo, max(fresh, 0));       // new tokens stand where `positions` says
            else
                hi = static_cast<int>(min(static_cast<long long>(hi), static_cast<long long>(gmax) + a.window - span.base));
        }
    }
    lo = __builtin_amdgcn_readfirstlane(lo);
    hi = __builtin_amdgcn_readfirstlane(hi);
    int step0 = lo / kTileTokens;
    const int steps_all = hi > lo ? (hi + kTileTokens - 1) / kTileTokens - step0 : 0;
    const int share = max((steps_all + splits - 1) / splits, (shared ? prefix_chunk : own_chunk) / kTileTokens);
    const int steps = __builtin_amdgcn_readfirstlane(max(0, min(share, steps_all - split * share)));
    step0 = __builtin_amdgcn_readfirstlane(step0 + split * share);

    const int group = 16 * (wave >> 1);            // of a step's tokens, those that the wave stages
    // Of steps st .. st + 63, a lane each: where the wave's 16 tokens lie, as the number of the first, ~0 if nowhere.
    uint32_t place_lo = 0, place_hi = 0;
    auto load_places = [&](int st) __attribute__((always_inline)) {
        const long long j = static_cast<long long>(step0 + st + lane) * kTileTokens + group;
        const int page = j < span.tokens ? span.table[min(static_cast<int>(j >> a.page_log2), span.n_table - 1)] : -1;
        const long long token = ((static_cast<long long>(page) * a.Hkv + h) << a.page_log2) + (j & ((1 << a.page_log2) - 1));
        const bool good = page >= 0 && page < a.n_pages;
        place_lo = good ? static_cast<uint32_t>(token) : ~0u;
        place_hi = good ? static_cast<uint32_t>(token >> 32) : ~0u;
    };
    load_places(0);

    // queries: lane (n, hf) holds values 16 k + 8 hf .. + 7 of its row, k = 0 .. 7, in the order of the keys' codes
    h8 q[8];
    {
        const uint16_t* src = a.Q + (static_cast<long long>(t) * a.Hq + head) * 128 + 8 * hf;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            Frag raw, f;
            const u4 y = valid ? *reinterpret_cast<const u4*>(src + 16 * k) : u4{0, 0, 0, 0};
            raw.w[0] = y.x; raw.w[1] = y.y; raw.w[2] = y.z; raw.w[3] = y.w;
#pragma unroll
            for (int i = 0; i < 8; ++i) f.v[i] = raw.v[order8<BITS>(i)];
            q[k] = f.v;
        }
    }
    const int at_row = valid ? t * a.Hq + head : -1;       // T * Hq is below 2^26
    const float slope = biased(SCORES) && a.slopes && valid ? a.slopes[head] * kLog2e : 0.0f;
    const bool near_cap = SCORES == kCapped || (SCORES == kFancy && a.softcap > 0.0f);
    const Cap cap = cap_of<SCORES>(a);
    const float key_factor = held(cap.factor);

    // What a wave stages of a step: eight tokens' keys, eight tokens' values and eight tokens' scales of both, all of the
    // same 16 tokens, which lie in one page.  The keys are tokens 8 w .. 8 w + 7 of the step, the values those of two
    // quads that share a chunk.  Codes are loaded a step ahead, the numbers of 64 steps' pages at once, a lane each.
    // Lanes are dealt out so that 16 of them load consecutive bytes, and those that write at one time write to different
    // banks.
    const int k_token = 8 * wave + (lane >> 3), k_part = lane & 7;
    const int v_octet = ((lane >> 1) & 7) + 8 * (lane >> 5), v_pair = lane & 1, v_half = (lane >> 4) & 1;
    const int k_at = ((k_token & 15) * 8 + k_part) * 2 * BITS;                                 // bytes within the 16 tokens
    const int v_at = ((((wave & 1) + 2 * v_half) * 16 + v_octet) * 2 + v_pair) * 2 * BITS;
    const bool s_values = (lane & 8) != 0;                  // of 16 lanes 0 .. 7 stage key, 8 .. 15 value scales, four times over
    const uint16_t* const scales = s_values ? a.V_scale : a.K_scale;
    const int s_token = 8 * wave + (lane & 7);
    struct Raw {
        uint32_t k[BITS / 2], v[BITS / 2], scale;
        bool there;
    };
    auto fetch = [&](int st) __attribute__((always_inline)) {
        Raw raw;
        const uint32_t lo = __builtin_amdgcn_readlane(place_lo, st & 63), hi = __builtin_amdgcn_readlane(place_hi, st & 63);
        const bool good = hi != ~0u;
        const unsigned long long token = good ? (static_cast<unsigned long long>(hi) << 32) | lo : static_cast<unsigned long long>(h) << a.page_log2;
        const uint8_t* kp = a.K_codes + token * (16 * BITS);
        const uint8_t* vp = a.V_codes + token * (16 * BITS);
        if (BITS == 4) {
            const u2 x = *reinterpret_cast<const u2*>(kp + k_at), y = *reinterpret_cast<const u2*>(vp + v_at);
            raw.k[0] = x.x; raw.k[1] = x.y;
            raw.v[0] = y.x; raw.v[1] = y.y;
        } else {
            const u4 x = *reinterpret_cast<const u4*>(kp + k_at), y = *reinterpret_cast<const u4*>(vp + v_at);
            raw.k[0] = x.x; raw.k[1] = x.y; raw.k[BITS / 2 - 2] = x.z; raw.k[BITS / 2 - 1] = x.w;
            raw.v[0] = y.x; raw.v[1] = y.y; raw.v[BITS / 2 - 2] = y.z; raw.v[BITS / 2 - 1] = y.w;
        }
        raw.scale = scales[token + (s_token & 15)];
        raw.there = good && (step0 + st) * kTileTokens + s_token < span.tokens;
        return raw;
    };
    auto stage_keys = [&](const Raw& raw, int buf, int part) __attribute__((always_inline)) {          // part 0, 1: eight codes each
        sh[buf].k[k_token * 17 + k_part + 8 * part] = __builtin_bit_cast(u4, key_operand<BITS>(raw.k + part * (BITS / 4)));
    };
    auto stage_values = [&](const Raw& raw, int buf, int part) __attribute__((always_inline)) {        // part 0 .. 3: two values of two tokens
        uint32_t* p = reinterpret_cast<uint32_t*>(&sh[buf].v[v_octet * 9 + wave]) + 2 * v_half + v_pair;
#pragma unroll
        for (int j = 2 * part; j < 2 * part + 2; ++j) p[j * 576] = value_pair<BITS>(raw.v, j);
    };
    auto stage_scales = [&](const Raw& raw, int buf) __attribute__((always_inline)) {
        const float s = __half2float(__ushort_as_half(static_cast<unsigned short>(raw.scale)));
        // a scale of 0 has codes of 0: its weight stays in the sum of weights through any other scale
        const float vs = s == 0.0f ? 0x1p-24f : s;
        const float key = raw.there ? __builtin_fmaf(s, key_factor, s * 0.0f) : 0.0f;      // NaN where s is not finite
        const float log_v = raw.there ? __builtin_amdgcn_logf(vs) : -__builtin_inff();
        const float rcp_v = raw.there && vs <= 65504.0f ? __builtin_amdgcn_rcpf(vs) : 0.0f;
        float* f = reinterpret_cast<float*>(sh[buf].f) + s_token;
        f[s_values ? kTileTokens : 0] = s_values ? log_v : key;
        f[s_values ? 2 * kTileTokens : 0] = s_values ? rcp_v : key;
    };

    // M: what a row's exponents are relative to.  It follows the row's maximum by more than kSlack powers of two, up, and
    // is set to it with the row's first token (`low` is infinite until then).
    float M = 0.0f, low = __builtin_inff(), l_sum = 0.0f;
    f16v o[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) o[m] = f16v{};

    f16v s;            // products of 32 tokens with their codes, then their exponents
    h8 w[2];           // their weights
    u4 vc[8];          // the tokens' values
    Raw raw;           // what the next step to be staged was loaded as
    f4 kf[4], rv[4];   // factors of the tokens: key, reciprocal value scale,
    float lv;          // log2 of the value scale, lane c of 16 for the lane's token c

    // does any row of the wave see any token of a step; does every row see all of them
    auto seen_some = [&](int j0) __attribute__((always_inline)) {
        bool some = wave_any;
        const int last = j0 + kTileTokens - 1;
        if (a.causal) some = some && j0 < max(pmax + 1, bmax);
        if (a.window > 0 && (!TREE || last - span.base < fresh))
            some = some && static_cast<long long>(last) > static_cast<long long>(pmin) - a.window &&
                   static_cast<long long>(j0) < static_cast<long long>(pmax) + a.window;
        return some;
    };
    auto seen_whole = [&](int j0) __attribute__((always_inline)) {
        bool whole = true;
        const int last = j0 + kTileTokens - 1;
        if (a.causal) whole = last <= pmin || last < bmin;
        if (TREE) whole = last - span.base < fresh;
        if (a.window > 0) whole = whole && static_cast<long long>(pmax) - j0 < a.window && static_cast<long long>(last) - pmin < a.window;
        return whole;
    };
    auto key_chunk = [&](int buf, int sub, int k) __attribute__((always_inline)) {
        const int token = 32 * sub + n;
        return sh[buf].k[token * 17 + k + 8 * hf];
    };
    auto value_chunk = [&](int buf, int sub, int i) __attribute__((always_inline)) {      // i = 4 kk + m
        return sh[buf].v[(32 * (i & 3) + n) * 9 + 4 * sub + 2 * (i >> 2) + hf];
    };
    auto load_factors = [&](int buf, int sub) __attribute__((always_inline)) {
        lv = reinterpret_cast<const float*>(sh[buf].f[1])[32 * sub + 8 * ((lane & 15) >> 2) + 4 * hf + (lane & 3)];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            kf[i] = sh[buf].f[0][8 * sub + 2 * i + hf];
            rv[i] = sh[buf].f[2][8 * sub + 2 * i + hf];
        }
    };
    // products to exponents of the tokens at positions j0 .. j0 + 31, relative to M
    auto exponents = [&](int j0) __attribute__((always_inline)) {
        const float from = SCORES == kFancy || SCORES == kCapped ? M - cap.top : M;
        const float rel = static_cast<float>(pos - j0 - 4 * hf);
        const float slope_here = TREE && any_new(j0 - span.base - fresh) ? 0.0f : slope;   // tree_mask adds it then
        auto one = [&](int e, float lm, bool capped) __attribute__((always_inline)) {
            const float k = kf[e >> 2][e & 3];
            if (biased(SCORES)) lm = __builtin_fmaf(-slope_here, __builtin_fabsf(rel - static_cast<float>(8 * (e >> 2) + (e & 3))), lm);
            s[e] = SCORES == kWideCap ? capped_wide(s[e] * k, cap.top, cap.rtop) + lm
                                      : capped ? capped_plus(s[e] * k, cap.top, lm) : __builtin_fmaf(s[e], k, lm);
        };
#define SPIN_ONE(N, CAP) one(N, row_lane<N>(lv) - from, CAP);
#define SPIN_ALL(CAP)                                                                     \
    SPIN_ONE(0, CAP) SPIN_ONE(1, CAP) SPIN_ONE(2, CAP) SPIN_ONE(3, CAP) SPIN_ONE(4, CAP) \
    SPIN_ONE(5, CAP) SPIN_ONE(6, CAP) SPIN_ONE(7, CAP) SPIN_ONE(8, CAP) SPIN_ONE(9, CAP) \
    SPIN_ONE(10, CAP) SPIN_ONE(11, CAP) SPIN_ONE(12, CAP) SPIN_ONE(13, CAP) SPIN_ONE(14, CAP) SPIN_ONE(15, CAP)
        if (near_cap) {
            SPIN_ALL(true)
        } else {
            SPIN_ALL(false)
        }
#undef SPIN_ALL
#undef SPIN_ONE
    };
    auto mask = [&](int j0) __attribute__((always_inline)) {
        // token c of the lane's half (c = 8 i + r): the row's last token in order, and its window, counted from there
        const int rel = pos - j0 - 4 * hf;
        const int end = a.causal ? max(rel, both - j0 - 4 * hf - 1) : 32;
        const uint32_t off = a.window > 0 ? static_cast<uint32_t>(rel) + static_cast<uint32_t>(a.window) - 1u : 32u;
        const uint32_t wide = a.window > 0 ? 2u * static_cast<uint32_t>(a.window) - 1u : 64u;
        if (TREE) {
            const int row = static_cast<int>(static_cast<unsigned>(max(at_row, 0)) / static_cast<unsigned>(a.Hq));
            tree_mask<SCORES, 16>(a, s, row, at_row >= 0, j0 - span.base - fresh, 4 * hf, news, new0, pos, rel, slope);
            return;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int c = 8 * (e >> 2) + (e & 3);
            const bool seen = (end >= c) & (off - static_cast<uint32_t>(c) < wide);
            s[e] = seen ? s[e] : -__builtin_inff();
        }
    };
    // masks the exponents, and moves M where it has to
    auto settle = [&](int j0, bool whole) __attribute__((always_inline)) {
        if (!whole) {
            asm volatile("" ::: "memory");     // keeps this a branch: the selects are not worth it elsewhere
            mask(j0);
        }
        float top = s[0];
#pragma unroll
        for (int e = 1; e < 16; ++e) top = __builtin_fmaxf(top, s[e]);
        top = swap_halves_max(top);
        if (__ballot(top > kSlack || top < low) != 0) {
            const bool none = top == -__builtin_inff(), first = low > 0.0f;
            const float up = none ? 0.0f : first ? top : __builtin_fmaxf(top, 0.0f);
            const float keep = first ? 0.0f : __builtin_amdgcn_exp2f(-up);     // nothing is kept of nothing, whatever up is
            low = none ? low : -__builtin_inff();
            M += up;
            l_sum *= keep;
#pragma unroll
            for (int m = 0; m < 4; ++m) o[m] *= keep;
#pragma unroll
            for (int e = 0; e < 16; ++e) s[e] -= up;
        }
    };
    // Vector work on 32 tokens at positions j0 ..: their exponents, M, their weights
    auto vector_part = [&](int j0, bool whole) __attribute__((always_inline)) {
        exponents(j0);
        settle(j0, whole);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float e[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                e[r] = __builtin_amdgcn_exp2f(s[4 * i + r]);
                l_sum = __builtin_fmaf(e[r], rv[i][r], l_sum);
            }
            const h2 p0 = __builtin_convertvector((f2{e[0], e[1]}), h2), p1 = __builtin_convertvector((f2{e[2], e[3]}), h2);
            h8& d = w[i >> 1];
            d[4 * (i & 1)] = p0.x;
            d[4 * (i & 1) + 1] = p0.y;
            d[4 * (i & 1) + 2] = p1.x;
            d[4 * (i & 1) + 3] = p1.y;
        }
    };
    auto load_values = [&](int buf, int sub) __attribute__((always_inline)) {
#pragma unroll
        for (int c = 0; c < 8; ++c) vc[c] = value_chunk(buf, sub, c);
    };
    // Matrix work: 32 tokens' weighted values, and the products of the next 32 (buf, sub), in turn, since the latter depend
    // on each other; if STAGE, between them, where the wave would wait, what it stages of a later step into buffer `to`
    auto matrix_part = [&](int buf, int sub, bool STAGE, int to) __attribute__((always_inline)) {
        u4 kc[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) kc[k] = key_chunk(buf, sub, k);
        s = f16v{};
        auto weighted = [&](int c) __attribute__((always_inline)) {
            o[c & 3] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8, vc[c]), w[c >> 2], o[c & 3], 0, 0, 0);
        };
        auto product = [&](int k) __attribute__((always_inline)) {
            s = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8, kc[k]), q[k], s, 0, 0, 0);
        };
        __builtin_amdgcn_s_setprio(1);      // before the other wave's vector work: prompt of 8192 tokens 785 -> 737 us
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            weighted(c);
            if (STAGE) stage_values(raw, to, c);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            product(c);
            if (STAGE && c < 2) stage_keys(raw, to, c);
            if (STAGE && c == 2) stage_scales(raw, to);
            __builtin_amdgcn_sched_barrier(0);
            weighted(4 + c);
            __builtin_amdgcn_sched_barrier(0);
        }
        load_factors(buf, sub);
#pragma unroll
        for (int k = 4; k < 8; ++k) product(k);
        __builtin_amdgcn_s_setprio(0);
    };

    auto stage_all = [&](const Raw& of, int buf) __attribute__((always_inline)) {
        stage_keys(of, buf, 0);
        stage_keys(of, buf, 1);
#pragma unroll
        for (int c = 0; c < 4; ++c) stage_values(of, buf, c);
        stage_scales(of, buf);
    };
    auto fetch_later = [&](int st) __attribute__((always_inline)) {       // nothing, past the last step
        if ((st & 63) == 0) load_places(st);
        raw = fetch(st);
    };
    // Two waves share a SIMD, one of each half of the workgroup.  The upper half runs a part behind the lower one, so
    // that of the two waves one has matrix and one has vector work, always:
    //   lower   V0  M0  V1  M1  V0 ..        V: exponents and weights, M: the two products, of 32 tokens (0, 1)
    //   upper       V0  M0  V1  M1 ..
    // 256 rows: the next step's tokens go into the other buffer in each half's M0.  The upper half's V1 reads that buffer
    // last, two parts before the lower half writes, and the lower half's M1 reads it first, a part after the upper half
    // has written.  128 rows: the lower half has a step's first 32 tokens, the upper the others,
    //   lower   V  M  V  M ..
    //   upper      V  M  V ..
    // and the tokens of the step after the next go into a third buffer in M, which the upper half's V read last, two
    // parts before, and the lower half's M reads first, a part after.
    // What a part reads of LDS is waited for in the part behind it at the latest, two before it is written again: only
    // a barrier behind writes, which publishes them, has to wait for the LDS.
    const bool upper = wave >= kTileWaves / 2;
    const int own_sub = kPair && upper ? 1 : 0;
    const int base = step0 * kTileTokens + span.base;
    if (steps > 0) {
        const Raw first = fetch(0), second = fetch(1);
        stage_all(first, 0);
        if (kPair) {
            raw = fetch(2);
            stage_all(second, 1);
        } else {
            raw = second;
        }
    }
    __syncthreads();
    if (steps > 0) {
        load_factors(0, own_sub);
        s = f16v{};
#pragma unroll
        for (int k = 0; k < 8; ++k)
            s = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8, key_chunk(0, own_sub, k)), q[k], s, 0, 0, 0);
    }
    if (upper) part_barrier();
    int buf = 0;
    for (int st = 0; st < steps; ++st) {
        const int j0 = base + st * kTileTokens;     // position of the first token
        const bool some = seen_some(j0), whole = seen_whole(j0);
        const int next = buf + 1 == kBuffers ? 0 : buf + 1;
        load_values(buf, own_sub);
        if (some) {
            vector_part(j0 + 32 * own_sub, whole);
        } else {
            w[0] = w[1] = h8{};
        }
        part_barrier();
        // behind the last step what is staged is of no use, and does no harm
        if (kPair) {
            const int after = next + 1 == kBuffers ? 0 : next + 1;
            matrix_part(next, own_sub, true, after);
            fetch_later(st + 3);
        } else {
            matrix_part(buf, 1, true, next);
            __syncthreads();
            load_values(buf, 1);
            if (some) vector_part(j0 + 32, whole);
            part_barrier();
            matrix_part(next, 0, false, 0);
            fetch_later(st + 2);           // here, not behind M0, which staging makes the longer part: 735 against 752 us
        }
        if (kPair)
            __syncthreads();
        else
            part_barrier();
        buf = next;
    }
    if (!upper) part_barrier();

    if (kPair) {
        // the upper half's sums, to the lower half's lane of the same row
        u4* slot = reinterpret_cast<u4*>(sh) + row_wave * 17 * 64 + lane;
        __syncthreads();
        if (upper) {
#pragma unroll
            for (int c = 0; c < 16; ++c)
                slot[64 * c] = __builtin_bit_cast(u4, (f4{o[c >> 2][4 * (c & 3)], o[c >> 2][4 * (c & 3) + 1], o[c >> 2][4 * (c & 3) + 2], o[c >> 2][4 * (c & 3) + 3]}));
            slot[64 * 16] = __builtin_bit_cast(u4, (f4{M, l_sum, low, 0.0f}));
        }
        __syncthreads();
        if (upper) return;
        const f4 other = __builtin_bit_cast(f4, slot[64 * 16]);
        const bool mine_none = low > 0.0f, other_none = other.z > 0.0f;
        const float M_all = mine_none ? other.x : other_none ? M : __builtin_fmaxf(M, other.x);
        const float f_mine = mine_none ? 0.0f : __builtin_amdgcn_exp2f(M - M_all);
        const float f_other = other_none ? 0.0f : __builtin_amdgcn_exp2f(other.x - M_all);
        l_sum = l_sum * f_mine + other.y * f_other;
        M = M_all;
#pragma unroll
        for (int c = 0; c < 16; ++c) {
            const f4 y = __builtin_bit_cast(f4, slot[64 * c]);
#pragma unroll
            for (int r = 0; r < 4; ++r) o[c >> 2][4 * (c & 3) + r] = o[c >> 2][4 * (c & 3) + r] * f_mine + y[r] * f_other;
        }
    }

    const float l = swap_halves_sum(l_sum);
    if (at_row < 0) return;
    const long long at = at_row;
    // the lane's values 8 c .. 8 c + 7, c = 8 (i & 1) + 4 hf + r, are rows 16 v + c: register 4 i + r of o[v / 2], i = 2 (v & 1) + (c > 7)
    float* partial = a.partial + ((first_slot + split) * static_cast<long long>(a.T) * a.Hq + at) * kPartial;
    const float rl = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int c = 8 * i + 4 * hf + r;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = o[e >> 1][4 * (2 * (e & 1) + i) + r];
            if (total_splits == 1) {
                Frag f;
#pragma unroll
                for (int e = 0; e < 8; ++e) f.v[e] = static_cast<_Float16>(v[e] * rl);
                *reinterpret_cast<u4*>(a.O + at * 128 + 8 * c) = u4{f.w[0], f.w[1], f.w[2], f.w[3]};
            } else if (l != 0.0f) {
                f2* dst = reinterpret_cast<f2*>(partial + 8 * c);
#pragma unroll
                for (int e = 0; e < 4; ++e) dst[e] = f2{v[2 * e], v[2 * e + 1]};
            }
        }
    }
    if (a.lse && total_splits == 1 && hf == 0) a.lse[at] = log_sum(M, l);
    if (total_splits > 1 && hf == 0) *reinterpret_cast<f2*>(partial + 128) = f2{l == 0.0f ? -__builtin_inff() : M, l};
}

// Joins the shares of a row: one wave a row, two values a lane, eight shares'
// sums in flight.  Shares without a visible token have not written their sums,
// and are not read.  Bound by the launch and by loads in turn: 4 - 6 us at up to
// 8192 rows.
__global__ __launch_bounds__(kAttnThreads) void kv_attn_join(KvAttnArgs a, int splits) {
    const long long rows = static_cast<long long>(a.T) * a.Hq;
    const long long at = static_cast<long long>(blockIdx.x) * kAttnWaves + (threadIdx.x >> 6);
    if (at >= rows) return;
    const int lane = threadIdx.x & 63;
    const int t = static_cast<int>(at / a.Hq);
    const int b = find_last64(a.B, lane, [&](int i) { return a.q_start[i] <= t; });
    if (t < a.q_start[b] || t >= a.q_start[b + 1]) return;
    const float* row = a.partial + at * kPartial;
    asm volatile("" ::"s"(a.lse));             // read now: behind the sums everything would wait for it
    float M = -__builtin_inff(), l = 0.0f;
    f2 o = {};
    for (int s0 = 0; s0 < splits; s0 += 64) {
        // 64 shares' maxima and sums at once, a lane each
        f2 ml = {-__builtin_inff(), 0.0f};
        if (s0 + lane < splits) ml = *reinterpret_cast<const f2*>(row + (s0 + lane) * rows * kPartial + 128);
        float top = max_over_groups(ml.x);
#pragma unroll
        for (int x = 1; x < 16; x <<= 1) top = __builtin_fmaxf(top, __shfl_xor(top, x, 64));
        const float M_new = __builtin_fmaxf(M, top);
        if (M_new == -__builtin_inff() && __ballot(ml.y != 0.0f) == 0) continue;
        const float keep = M == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(M - M_new);
        l *= keep;
        o *= keep;
        M = M_new;
        const float f = ml.y == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(ml.x - M);
        unsigned long long left = __ballot(ml.y != 0.0f);
        while (left != 0) {
            f2 y[8];
            float fs[8], ls[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool any = left != 0;
                const int s = any ? __builtin_ctzll(left) : 0;
                left &= left - 1;
                fs[i] = any ? __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(f), s)) : 0.0f;
                ls[i] = any ? __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(ml.y), s)) : 0.0f;
                y[i] = any ? reinterpret_cast<const f2*>(row + (s0 + s) * rows * kPartial)[lane] : f2{};
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                l = __builtin_fmaf(ls[i], fs[i], l);
                o.x = __builtin_fmaf(y[i].x, fs[i], o.x);
                o.y = __builtin_fmaf(y[i].y, fs[i], o.y);
            }
        }
    }
    if (a.lse && lane == 0) a.lse[at] = log_sum(M, l);
    const float rl = l == 0.0f ? 0.0f : 1.0f / l;
    const h2 res = {static_cast<_Float16>(o.x * rl), static_cast<_Float16>(o.y * rl)};
    reinterpret_cast<h2*>(a.O)[at * 64 + lane] = res;
}

// How the rows on one stretch of tokens, a shared prefix or the sequences' own, are dealt out: rows of a tile, tiles,
// shares of the tokens and the fewest tokens of one.
struct Part {
    int rows;                      // 16: kv_attn_rows16; 128, 256: kv_attn_tile; 0: no tokens
    long long tiles;
    int splits, chunk;
    int waves;                     // of a workgroup with 16 rows
};

struct Plan {
    Part prefix, own;
    int splits;
    size_t workspace;
};

// `groups`: stretches of tokens (sequences, or one prefix); `ragged`: every group's rows begin a tile; `tokens`: the most
// of a group.
Part deal(int tile, int waves, long long rows, long long groups, bool ragged, int Hkv, int tokens) {
    Part p = {};
    if (tokens <= 0) return p;
    p.rows = tile;
    p.waves = waves;
    p.tiles = ragged ? rows / p.rows + groups : (rows + p.rows - 1) / p.rows;
    const long long busy = (rows / p.rows > groups ? rows / p.rows : groups) * Hkv;     // workgroups with rows
    long long splits;
    if (tile != kRows) {
        // one workgroup a CU: no more than there are
        splits = kTilesWanted / busy;
        p.chunk = kTilesLeast;
    } else if (busy * waves >= kRowsWaves / 2) {
        // shares of one size for all sequences, so that a long one does not hold up the rest
        p.chunk = kLongShare * waves;
        splits = (tokens + p.chunk - 1) / p.chunk;
    } else {
        splits = (kRowsWaves + busy * waves - 1) / (busy * waves);
        p.chunk = kLeastShare * waves;
    }
    if (splits * p.chunk > tokens) splits = (tokens + p.chunk - 1) / p.chunk;
    if (splits > kMostSplits) splits = kMostSplits;
    p.splits = static_cast<int>(splits < 1 ? 1 : splits);
    return p;
}

Plan plan(int T, int Hq, int Hkv, int B, int max_kv, int prefix_len) {
    const long long rows = static_cast<long long>(T) * (Hq / Hkv);
    Plan p = {};
    // rows times tokens, of all key heads: what there is to do
    const double prefix_work = static_cast<double>(rows) * prefix_len * Hkv, own_work = static_cast<double>(rows) * max_kv * Hkv;
    const int prefix_tile = rows < kManyRows || prefix_work < kTileWork ? kRows : prefix_work < kWideWork ? 128 : 256;
    int own_tile = rows / B < kManyRows || own_work < kTileWork ? kRows : own_work < 2 * kWideWork ? 128 : 256;
    if (own_tile != kRows && prefix_len > 0 && prefix_tile != kRows) own_tile = prefix_tile;     // one launch
    const long long busy = (rows / kRows > B ? rows / kRows : B) * Hkv;
    // a prefix's rows are many, and their tiles' waves work on shares: four suffice (64 tokens behind 8192: 38 us, eight 43)
    const int waves = prefix_len > 0 || (max_kv <= kShortest && busy * 8 >= kRowsWaves / 2) ? 4 : 8;
    p.prefix = deal(prefix_tile, waves, rows, 1, false, Hkv, prefix_len);
    p.own = deal(own_tile, waves, rows, B, true, Hkv, max_kv);
    if (own_tile == kRows && prefix_len == 0 && max_kv <= kShort) p.own.splits = 1;     // the kernel's share is all
    p.splits = p.prefix.splits + p.own.splits;
    p.workspace = p.splits > 1 ? static_cast<size_t>(p.splits) * T * Hq * kPartial * sizeof(float) : 0;
    return p;
}

template <int BITS, int ROWS, int SCORES, bool TREE>
hipError_t launch_part(const KvAttnArgs& a, const Part& prefix, const Part& own, hipStream_t s) {
    const unsigned items = static_cast<unsigned>(prefix.tiles * prefix.splits + own.tiles * own.splits);
    const int pt = static_cast<int>(prefix.tiles), ot = static_cast<int>(own.tiles);
    if constexpr (ROWS == kRows) {
        const dim3 grid((items + 7) / 8 * 8 * a.Hkv);
        if (own.waves == 8)
            hipLaunchKernelGGL((kv_attn_rows16<BITS, SCORES, 8, TREE>), grid, dim3(512), 0, s, a, pt, prefix.splits, prefix.chunk, ot, own.splits,
                               own.chunk);
        else
            hipLaunchKernelGGL((kv_attn_rows16<BITS, SCORES, 4, TREE>), grid, dim3(256), 0, s, a, pt, prefix.splits, prefix.chunk, ot, own.splits,
                               own.chunk);
    } else {
        hipLaunchKernelGGL((kv_attn_tile<BITS, ROWS, SCORES, TREE>), dim3(items * a.Hkv), dim3(kTileThreads), 0, s, a, pt,
                           prefix.splits, prefix.chunk, ot, own.splits, own.chunk);
    }
    return hipGetLastError();
}

template <int BITS, int ROWS, bool TREE>
hipError_t launch_rows(const KvAttnArgs& a, Part prefix, Part own, hipStream_t s) {
    // a part with another tile has a launch of its own; its share of the workspace stays where it is
    if (prefix.rows != ROWS) prefix.tiles = 0;
    if (own.rows != ROWS) own.tiles = 0;
    if (prefix.tiles == 0 && own.tiles == 0) return hipSuccess;
    if (a.softcap > kNearCap) return launch_part<BITS, ROWS, kWideCap, TREE>(a, prefix, own, s);
    // the tree's masks take registers that a cap with a bias has none of (16 trees of 60 on 4096, INT8, capped: 134 us, with the bias in the kernel 185)
    if constexpr (TREE) {
        if (a.softcap > 0.0f && !a.slopes) return launch_part<BITS, ROWS, kCapped, TREE>(a, prefix, own, s);
    }
    return a.softcap > 0.0f || a.slopes ? launch_part<BITS, ROWS, kFancy, TREE>(a, prefix, own, s)
                                        : launch_part<BITS, ROWS, kPlain, TREE>(a, prefix, own, s);
}

template <int BITS, bool TREE>
hipError_t launch_bits(const KvAttnArgs& a, const Plan& p, hipStream_t s) {
    hipError_t e = launch_rows<BITS, 256, TREE>(a, p.prefix, p.own, s);
    if (e == hipSuccess) e = launch_rows<BITS, 128, TREE>(a, p.prefix, p.own, s);
    if (e == hipSuccess) e = launch_rows<BITS, kRows, TREE>(a, p.prefix, p.own, s);
    return e;
}

}  // namespace

size_t kv_attn_workspace(int T, int Hq, int Hkv, int B, int max_kv, int prefix_len) {
    return plan(T, Hq, Hkv, B, max_kv, prefix_len).workspace;
}

bool kv_attn_fits(int T, int Hq, int Hkv, int B, int max_kv, int prefix_len) {
    const Plan p = plan(T, Hq, Hkv, B, max_kv, prefix_len);
    // workgroups of 512 a launch dimension holds, halved: the rows of a key head stay below 2^30
    constexpr long long kMost = (1LL << 22) - 1;
    return (p.prefix.tiles * p.prefix.splits + p.own.tiles * p.own.splits + 8) * Hkv <= kMost && Hkv <= 65535 &&
           static_cast<long long>(T) * Hq <= (1LL << 26);
}

hipError_t launch_kv_attn(const KvAttnArgs& a, int bits, hipStream_t s) {
    const Plan p = plan(a.T, a.Hq, a.Hkv, a.B, a.max_pages << a.page_log2, a.prefix_len);
    const hipError_t e = a.tree ? (bits == 8 ? launch_bits<8, true>(a, p, s) : launch_bits<4, true>(a, p, s))
                                : (bits == 8 ? launch_bits<8, false>(a, p, s) : launch_bits<4, false>(a, p, s));
    // where a prefix has an earlier launch and the sequences' own tokens one share of 16 rows, that joins what both give
    if (e != hipSuccess || p.splits == 1 || (p.own.rows == kRows && p.own.splits == 1 && p.prefix.rows > kRows)) return e;
    const long long rows = static_cast<long long>(a.T) * a.Hq;
    hipLaunchKernelGGL(kv_attn_join, dim3(static_cast<unsigned>((rows + kAttnWaves - 1) / kAttnWaves)), dim3(kAttnThreads), 0,
                       s, a, p.splits);
    return hipGetLastError();
}

}  // namespace spin
