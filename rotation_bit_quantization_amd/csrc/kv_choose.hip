// spin_kv_choose kernel: of a sequence's tokens, per key head, those of greatest
// weight, in the order of their places.
//
// A selection, not a sort: the weight of the last token that stays is found
// digit by digit from the top (four counts of 8 bits of a number that is ordered
// as the weights are), then one pass in order of places writes the tokens above it
// and the first of those equal to it.  Ties go to the lowest place, so that the
// result is one for any order of work.
#include "kv_batch.h"
#include "spin_internal.h"

namespace spin {
namespace {

constexpr int kChooseThreads = 1024;
constexpr int kChooseWaves = kChooseThreads / 64;

// An unsigned number that rises with the weight; NaN, and a token that lies nowhere, below all.
__device__ __forceinline__ uint32_t rank_of(float w) {
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.0f);        // -0 is 0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ uint32_t rank_at(const KvChooseArgs& a, int b, int h, int j) {
    const int page = a.page_table[static_cast<long long>(b) * a.max_pages + (j >> a.page_log2)];
    if (page < 0 || page >= a.n_pages) return 0u;
    return rank_of(a.W[((static_cast<long long>(page) * a.Hkv + h) << a.page_log2) + (j & ((1 << a.page_log2) - 1))]);
}

// The sum of v over the workgroup's threads before this one, and (all) over all of them.
__device__ __forceinline__ int before_of(int v, int* sh, int& all) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int upto = v;
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) {
        const int y = __shfl_up(upto, x, 64);
        upto += lane >= x ? y : 0;
    }
    if (lane == 63) sh[wave] = upto;
    __syncthreads();
    int front = 0;
    all = 0;
    for (int w = 0; w < kChooseWaves; ++w) {
        front += w < wave ? sh[w] : 0;
        all += sh[w];
    }
    __syncthreads();
    return front + upto - v;
}

__global__ __launch_bounds__(kChooseThreads) void kv_choose_kernel(KvChooseArgs a) {
    __shared__ int count[256];
    __shared__ int sums[kChooseWaves];
    __shared__ int digit_sh, above_sh;
    const int h = blockIdx.x % a.Hkv, b = blockIdx.x / a.Hkv;
    const int n = min(max(a.kv_len[b], 0), a.max_pages << a.page_log2);
    int32_t* kept = a.kept + (static_cast<long long>(b) * a.Hkv + h) * a.keep;
    if (h == 0 && threadIdx.x == 0) a.lens[b] = min(n, a.keep);
    if (n <= a.keep) {
        for (int i = threadIdx.x; i < a.keep; i += kChooseThreads) kept[i] = i < n ? i : -1;
        return;
    }
    // n > keep >= first + recent: the candidates are places first .. n - recent - 1, more than are wanted of them
    const int end = n - a.recent, want = a.keep - a.first - a.recent;
    for (int i = threadIdx.x; i < a.first; i += kChooseThreads) kept[i] = i;
    for (int i = threadIdx.x; i < a.recent; i += kChooseThreads) kept[a.keep - a.recent + i] = end + i;
    if (want == 0) return;
    uint32_t top = 0;                      // the digits that are known, of the rank of the last that stays
    int above = 0;                         // candidates whose known digits are greater
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (threadIdx.x < 256) count[threadIdx.x] = 0;
        __syncthreads();
        for (int j = a.first + static_cast<int>(threadIdx.x); j < end; j += kChooseThreads) {
            const uint32_t u = rank_at(a, b, h, j);
            if (shift == 24 || (u >> (shift + 8)) == (top >> (shift + 8))) atomicAdd(&count[u >> shift & 255], 1);
        }
        __syncthreads();
        // the digit at which as many as are wanted are reached, from the greatest digit down
        int all;
        const int mine = threadIdx.x < 256 ? count[255 - threadIdx.x] : 0;
        const int greater = above + before_of(mine, sums, all);
        if (greater < want && want <= greater + mine) {
            digit_sh = 255 - threadIdx.x;
            above_sh = greater;
        }
        __syncthreads();
        top |= static_cast<uint32_t>(digit_sh) << shift;
        above = above_sh;
    }
    // in order of places: all above, and the first of the equal ones
    int equal = want - above, at = a.first;
    for (int j0 = a.first; j0 < end; j0 += kChooseThreads) {
        const int j = j0 + static_cast<int>(threadIdx.x);
        const uint32_t u = j < end ? rank_at(a, b, h, j) : 0u;
        int same, stay;
        const bool tie = j < end && u == top;
        const int ties = before_of(tie, sums, same);
        const bool yes = j < end && (u > top || (tie && ties < equal));
        const int slot = at + before_of(yes, sums, stay);
        if (yes) kept[slot] = j;
        at += stay;
        equal -= min(equal, same);
    }
}

}  // namespace

bool kv_choose_fits(int Hkv, int B) { return static_cast<long long>(Hkv) * B <= (1LL << 22) - 1; }

hipError_t launch_kv_choose(const KvChooseArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(kv_choose_kernel, dim3(static_cast<unsigned>(a.B) * a.Hkv), dim3(kChooseThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace spin
