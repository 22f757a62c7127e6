// spin_kv_choose kernels: of a sequence's tokens, per key head, those of greatest
// weight, in the order of their places.
//
// A selection, not a sort: the weight of the last token that stays is found
// digit by digit from the top (counts of 11, 11 and 10 bits of a number that is
// ordered as the weights are), then the tokens above it and the first of those
// equal to it are written in order of places.  Ties go to the lowest place, so
// that the result is one for any order of work.
#include "kv_batch.h"
#include "spin_internal.h"

namespace spin {
namespace {

constexpr int kChooseThreads = 1024;
constexpr int kChooseWaves = kChooseThreads / 64;
constexpr int kDigits = 3, kBins = 2048;
__device__ __forceinline__ int digit_shift(int d) { return d == 0 ? 21 : d == 1 ? 10 : 0; }
__device__ __forceinline__ uint32_t digit_of(uint32_t u, int d) { return d == 2 ? u & 1023u : u >> digit_shift(d) & 2047u; }
// whether the digits above digit d, 1 or 2, are those of top
__device__ __forceinline__ bool same_above(uint32_t u, uint32_t top, int d) { return (u ^ top) < (d == 1 ? 1u << 21 : 1u << 10); }

// An unsigned number that rises with the weight: a token that always stays above all, NaN and a token that lies nowhere
// below all weights, and a place behind the last token, which never stays, below everything.
constexpr uint32_t kAlways = ~0u, kNone = 1u, kBehind = 0u;
__device__ __forceinline__ uint32_t rank_of(float w) {
    const uint32_t u = __float_as_uint(w + 0.0f);        // -0 is 0
    return w != w ? kNone : u ^ (static_cast<uint32_t>(static_cast<int>(u) >> 31) | 0x80000000u);
}

// The sum of v over the workgroup's threads before this one.
__device__ __forceinline__ int before_of(int v, int* sh) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int upto = sums_up_to(v);
    if (lane == 63) sh[wave] = upto;
    __syncthreads();
    const int waves = sums_up_to(lane < kChooseWaves ? sh[lane] : 0);
    const int front = wave > 0 ? __shfl(waves, wave - 1, 64) : 0;
    __syncthreads();
    return front + upto - v;
}

// From the counts of a digit, its value for the token that is the want-th from the top, and how many have a greater one.
__device__ __forceinline__ void find_digit(const int* count, int want, int* sums, int* found, int& digit, int& greater) {
    const int t = 2 * (kChooseThreads - 1 - static_cast<int>(threadIdx.x));        // from the greatest down, two each
    const int2 mine = {count[t + 1], count[t]};
    const int before = before_of(mine.x + mine.y, sums);
    if (before < want && want <= before + mine.x) {
        found[0] = t + 1;
        found[1] = before;
    } else if (before + mine.x < want && want <= before + mine.x + mine.y) {
        found[0] = t;
        found[1] = before + mine.x;
    }
    __syncthreads();
    digit = found[0];
    greater = found[1];
}

// What a workgroup knows of its head.
struct Head {
    int b, h, n;                   // tokens
    int32_t* kept;
};
__device__ __forceinline__ Head head_of(const KvChooseArgs& a, int head) {
    Head x;
    x.b = head / a.Hkv;
    x.h = head - x.b * a.Hkv;
    x.n = min(max(a.kv_len[x.b], 0), a.max_pages << a.page_log2);
    x.kept = a.kept + static_cast<long long>(head) * a.keep;
    return x;
}

// All of a head's tokens stay: entries i0 .. i1 - 1 of the list.
__device__ __forceinline__ void keep_all(const Head& x, int i0, int i1) {
    for (int i = i0 + static_cast<int>(threadIdx.x); i < i1; i += kChooseThreads) x.kept[i] = i < x.n ? i : -1;
}

// The ranks of tokens p0 + 4096 r + 4 thread .. + 3, each four in one page.
template <int R>
__device__ __forceinline__ void load_ranks(const KvChooseArgs& a, const Head& x, int p0, uint4* u) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int j0 = p0 + 4 * r * kChooseThreads, j = j0 + 4 * static_cast<int>(threadIdx.x);
        const int page = j < x.n ? a.page_table[static_cast<long long>(x.b) * a.max_pages + (j >> a.page_log2)] : -1;
        u[r] = uint4{kNone, kNone, kNone, kNone};
        if (page >= 0 && page < a.n_pages) {
            const float4 w = *reinterpret_cast<const float4*>(a.W + (((static_cast<long long>(page) * a.Hkv + x.h) << a.page_log2) + (j & ((1 << a.page_log2) - 1))));
            u[r] = uint4{rank_of(w.x), rank_of(w.y), rank_of(w.z), rank_of(w.w)};
        }
        if (j0 < a.first || j0 + 4 * kChooseThreads > x.n - a.recent) {
            auto held = [&](uint32_t v, int i) { return i >= x.n ? kBehind : i < a.first || i >= x.n - a.recent ? kAlways : v; };
            u[r] = uint4{held(u[r].x, j), held(u[r].y, j + 1), held(u[r].z, j + 2), held(u[r].w, j + 3)};
        }
    }
}

// Counts digit d of the tokens whose higher digits are top's; not places behind the last token, which would all wait for
// one address.
template <int R>
__device__ __forceinline__ void count_digit(const uint4* u, int d, uint32_t top, int* count) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const uint32_t v[4] = {u[r].x, u[r].y, u[r].z, u[r].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (d == 0 ? v[e] != kBehind : same_above(v[e], top, d)) atomicAdd(&count[digit_of(v[e], d)], 1);
    }
}

// How many of four tokens are above top, and above 16 bits how many are equal to it.
__device__ __forceinline__ int over_and_ties(const uint4& u, uint32_t top) {
    return ((u.x > top) + (u.y > top) + (u.z > top) + (u.w > top)) + (((u.x == top) + (u.y == top) + (u.z == top) + (u.w == top)) << 16);
}

// Writes those that stay, in order of places; `overs` and `ties` are how many there are before token p0.  4096 R tokens
// are 32768 at most, so that their counts fit 16 bits.
template <int R>
__device__ __forceinline__ void write_kept(const KvChooseArgs& a, const Head& x, const uint4* u, int p0, uint32_t top, int equal, int overs, int ties, int* sums) {
    static_assert(R <= 8, "two counts a number, and two of the waves' counts a lane");
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int before[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int v = over_and_ties(u[r], top);
        const int upto = sums_up_to(v);
        before[r] = upto - v;
        if (lane == 63) sums[r * kChooseWaves + wave] = upto;
    }
    __syncthreads();
    if (wave == 0) {
        const int at = 2 * lane;
        const int one = at < R * kChooseWaves ? sums[at] : 0, two = at < R * kChooseWaves ? sums[at + 1] : 0;
        const int upto = sums_up_to(one + two) - one - two;
        if (at < R * kChooseWaves) {
            sums[at] = upto;
            sums[at + 1] = upto + one;
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const uint32_t v[4] = {u[r].x, u[r].y, u[r].z, u[r].w};
        const int j = p0 + 4 * (r * kChooseThreads + static_cast<int>(threadIdx.x));
        const uint32_t front = static_cast<uint32_t>(before[r]) + static_cast<uint32_t>(sums[r * kChooseWaves + wave]);
        const int same = ties + static_cast<int>(front >> 16);
        int at = overs + static_cast<int>(front & 0xFFFFu) + min(same, equal), left = equal - same;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool tie = v[e] == top;
            if (v[e] > top || (tie && left > 0)) {
                if (at < a.keep) x.kept[at] = j + e;         // not behind the list, if the weights change meanwhile
                ++at;
            }
            left -= tie;
        }
    }
}

// One workgroup for all tokens of a head, which it holds in registers.  Bound by what depends on what: length, page, weight,
// then for each digit the counts, their sum over the workgroup, and the next.  Measured: 8 heads of 64 sequences of 2000 to
// 8192 tokens, of which 2048 stay, 12.6 us on two batches in turn (14 MB), 11 on one again and again; there 18 us in a
// table for 16384 and 26 for 32768, whose kernels hold as many ranks.  Of one sequence of 2500, 16000 and 32000 6.9, 11.9
// and 18.7 us.
template <int R>
__global__ __launch_bounds__(kChooseThreads) void kv_choose_kernel(KvChooseArgs a) {
    __shared__ int count[kBins];
    __shared__ int sums[R * kChooseWaves];
    __shared__ int found[2];
    const Head x = head_of(a, blockIdx.x);
    if (a.lens && x.h == 0 && threadIdx.x == 0) a.lens[x.b] = min(x.n, a.keep);
    if (x.n <= a.keep) {
        keep_all(x, 0, a.keep);
        return;
    }
    uint4 u[R];
    load_ranks<R>(a, x, 0, u);
    uint32_t top = 0;                      // the digits that are known, of the rank of the last that stays
    int above = 0;                         // tokens that are greater by them
    for (int d = 0; d < kDigits; ++d) {
        reinterpret_cast<int2*>(count)[threadIdx.x] = int2{0, 0};
        __syncthreads();
        count_digit<R>(u, d, top, count);
        __syncthreads();
        int digit, greater;
        find_digit(count, a.keep - above, sums, found, digit, greater);
        top |= static_cast<uint32_t>(digit) << digit_shift(d);
        above += greater;
    }
    write_kept<R>(a, x, u, 0, top, a.keep - above, 0, 0, sums);
}

// Longer tables: a workgroup for 8192 tokens of a head, and a launch for each step: the counts cleared, then each digit's
// counts added up over the workgroups (whole numbers, in any order), then how many of each workgroup's stay, then their
// places.  Each step finds the digits that are known from their counts again.  Measured: one document of 131072 tokens, 8
// heads, 28 us (one workgroup a head, which read the weights four times over: 137); 16 of 130000 128 us (with 32768 tokens
// a workgroup 147).  The table's room decides, the host knows no lengths: 64 sequences of 2000 to 8192 tokens in tables for
// 33000 take 70 us, for 131072 398.
constexpr int kPartRounds = 2, kPart = 4 * kPartRounds * kChooseThreads;

__global__ __launch_bounds__(kChooseThreads) void kv_choose_clear(KvChooseArgs a) {
    reinterpret_cast<int2*>(a.counts)[static_cast<long long>(blockIdx.x) * kChooseThreads + threadIdx.x] = int2{0, 0};
}

// step 0, 1, 2: count that digit; 3: how many stay; 4: write them
template <int STEP>
__global__ __launch_bounds__(kChooseThreads) void kv_choose_part(KvChooseArgs a, int parts) {
    constexpr int R = kPartRounds;
    __shared__ int count[kBins];
    __shared__ int sums[R * kChooseWaves];
    __shared__ int found[2];
    const int head = blockIdx.x / parts, part = blockIdx.x - head * parts, p0 = part * kPart;
    const Head x = head_of(a, head);
    if (STEP == 4 && a.lens && x.h == 0 && part == 0 && threadIdx.x == 0) a.lens[x.b] = min(x.n, a.keep);
    if (x.n <= a.keep) {
        if (STEP == 4) keep_all(x, p0, part == parts - 1 ? a.keep : min(a.keep, p0 + kPart));
        return;
    }
    if (p0 >= x.n) return;
    uint4 u[R];
    load_ranks<R>(a, x, p0, u);
    int* const counts = a.counts + static_cast<long long>(head) * (kDigits * kBins);
    uint32_t top = 0;
    int above = 0;
    for (int d = 0; d < (STEP < kDigits ? STEP : kDigits); ++d) {
        int digit, greater;
        find_digit(counts + d * kBins, a.keep - above, sums, found, digit, greater);
        top |= static_cast<uint32_t>(digit) << digit_shift(d);
        above += greater;
    }
    if (STEP < 3) {
        reinterpret_cast<int2*>(count)[threadIdx.x] = int2{0, 0};
        __syncthreads();
        count_digit<R>(u, STEP, top, count);
        __syncthreads();
        for (int i = threadIdx.x; i < kBins; i += kChooseThreads)
            if (count[i] != 0) atomicAdd(counts + STEP * kBins + i, count[i]);
        return;
    }
    int2* const stay = reinterpret_cast<int2*>(a.counts + static_cast<long long>(a.B) * a.Hkv * (kDigits * kBins)) + static_cast<long long>(head) * parts;
    if (STEP == 3) {
        int packed = 0;
#pragma unroll
        for (int r = 0; r < R; ++r) packed += over_and_ties(u[r], top);
        packed += before_of(packed, sums);
        if (threadIdx.x == kChooseThreads - 1) stay[part] = int2{packed & 0xFFFF, static_cast<int>(static_cast<uint32_t>(packed) >> 16)};
        return;
    }
    // what stays of the tokens before; every wave adds it up
    int overs = 0, ties = 0;
    for (int i = threadIdx.x & 63; i < part; i += 64) {
        overs += stay[i].x;
        ties += stay[i].y;
    }
    overs = __builtin_amdgcn_readlane(sums_up_to(overs), 63);
    ties = __builtin_amdgcn_readlane(sums_up_to(ties), 63);
    write_kept<R>(a, x, u, p0, top, a.keep - above, overs, ties, sums);
}

// How many stay, where that takes the place of the lengths: behind the kernels, all of whose heads read them.
__global__ __launch_bounds__(kChooseThreads) void kv_choose_lens(int32_t* lens, int B, int room, int keep) {
    const int b = blockIdx.x * kChooseThreads + static_cast<int>(threadIdx.x);
    if (b < B) lens[b] = min(min(max(lens[b], 0), room), keep);
}

bool in_parts(int room) { return room > 32 * kChooseThreads; }

int parts_of(int room) { return (room + kPart - 1) / kPart; }

}  // namespace

size_t kv_choose_workspace(int Hkv, int B, int room) {
    const long long heads = static_cast<long long>(B) * Hkv;
    return in_parts(room) ? heads * (kDigits * kBins * sizeof(int) + parts_of(room) * sizeof(int2)) : 0;
}

bool kv_choose_fits(int Hkv, int B, int room) {
    // workgroups of 1024 a launch dimension holds; those that clear are three a head
    const long long heads = static_cast<long long>(Hkv) * B, most = (1 << 22) - 1;
    return heads <= most && (!in_parts(room) || (heads * 3 <= most && heads * parts_of(room) <= most));
}

namespace {

hipError_t launch_choice(const KvChooseArgs& a, hipStream_t s) {
    const unsigned heads = static_cast<unsigned>(a.B) * a.Hkv;
    const int room = a.max_pages << a.page_log2;
    const dim3 threads(kChooseThreads);
    if (!in_parts(room)) {
        if (room <= 8 * kChooseThreads)
            hipLaunchKernelGGL((kv_choose_kernel<2>), dim3(heads), threads, 0, s, a);
        else if (room <= 16 * kChooseThreads)
            hipLaunchKernelGGL((kv_choose_kernel<4>), dim3(heads), threads, 0, s, a);
        else
            hipLaunchKernelGGL((kv_choose_kernel<8>), dim3(heads), threads, 0, s, a);
        return hipGetLastError();
    }
    const int parts = parts_of(room);
    const dim3 grid(heads * parts);
    hipLaunchKernelGGL(kv_choose_clear, dim3(heads * (kDigits * kBins / 2 / kChooseThreads)), threads, 0, s, a);
    hipLaunchKernelGGL((kv_choose_part<0>), grid, threads, 0, s, a, parts);
    hipLaunchKernelGGL((kv_choose_part<1>), grid, threads, 0, s, a, parts);
    hipLaunchKernelGGL((kv_choose_part<2>), grid, threads, 0, s, a, parts);
    hipLaunchKernelGGL((kv_choose_part<3>), grid, threads, 0, s, a, parts);
    hipLaunchKernelGGL((kv_choose_part<4>), grid, threads, 0, s, a, parts);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_choose(const KvChooseArgs& a, hipStream_t s) {
    if (a.lens != a.kv_len) return launch_choice(a, s);
    KvChooseArgs places = a;
    places.lens = nullptr;
    const hipError_t e = launch_choice(places, s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kv_choose_lens, dim3((static_cast<unsigned>(a.B) + kChooseThreads - 1) / kChooseThreads), dim3(kChooseThreads), 0, s, a.lens, a.B,
                       a.max_pages << a.page_log2, a.keep);
    return hipGetLastError();
}

}  // namespace spin
