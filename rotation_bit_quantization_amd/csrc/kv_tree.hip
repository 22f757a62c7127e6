// spin_kv_tree kernel: ancestors and positions of drafted tokens.
//
// Token i of a sequence's new ones has a parent p(i) < i among them, or none (it
// follows the context).  Its row of the tree names i, p(i), p(p(i)), ...; its
// position is the context's end plus its depth, the row's bits less one.
//
// Bound: the launch, and a chain of loads as long as the tree is deep, from L1: a
// sequence's parents are a few cache lines.  Measured: 64 trees of 60 tokens 3.6
// us, 5 of 1337 together 4.8; chains of 60 8, of 512 44 (0.09 us a level), one of 4096, whose lanes hold eight words each,
// 766 (0.19).  16 lanes walk the same chain and hold the row's words, so that a row is written once.
#include "kv_batch.h"
#include "spin_internal.h"

namespace spin {
namespace {

constexpr int kTreeThreads = 256;
constexpr int kTreeRows = kTreeThreads / 16;

// WORDS: words of a row that a lane holds.
template <int WORDS>
__global__ __launch_bounds__(kTreeThreads) void kv_tree_kernel(KvTreeArgs a) {
    const int l = threadIdx.x & 15;
    const int t = blockIdx.x * kTreeRows + (threadIdx.x >> 4);
    if (t >= a.T) return;                  // the 16 lanes of a row leave together
    const int b = find_sequence16(a.q_start, a.B, t, l);
    if (b < 0) return;
    const int row0 = max(a.q_start[b], 0);
    const int news = static_cast<int>(static_cast<uint32_t>(a.q_start[b + 1]) - static_cast<uint32_t>(a.q_start[b]));
    uint32_t bits[WORDS] = {};
    int depth = -1;
    // parents lie before their children, so that the walk ends, and within the sequence's rows
    for (int i = t - row0 < 32 * a.words ? t - row0 : -1; i >= 0;) {
#pragma unroll
        for (int w = 0; w < WORDS; ++w) bits[w] |= i >> 5 == l + 16 * w ? 1u << (i & 31) : 0u;
        ++depth;
        const int p = a.parent[row0 + i];
        i = p < i ? p : -1;
    }
    uint32_t* row = a.tree + static_cast<long long>(t) * a.words;
#pragma unroll
    for (int w = 0; w < WORDS; ++w)
        if (l + 16 * w < a.words) row[l + 16 * w] = bits[w];
    if (l == 0)
        a.positions[t] = static_cast<int>(static_cast<uint32_t>(a.pos0) + static_cast<uint32_t>(placed(a.kv_len[b])) -
                                          static_cast<uint32_t>(news) + static_cast<uint32_t>(max(depth, 0)));
}

}  // namespace

hipError_t launch_kv_tree(const KvTreeArgs& a, hipStream_t s) {
    const dim3 grid((static_cast<unsigned>(a.T) + kTreeRows - 1) / kTreeRows);
    if (a.words <= 16)
        hipLaunchKernelGGL((kv_tree_kernel<1>), grid, dim3(kTreeThreads), 0, s, a);
    else
        hipLaunchKernelGGL((kv_tree_kernel<SPIN_KV_TREE_MAX_WORDS / 16>), grid, dim3(kTreeThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace spin
