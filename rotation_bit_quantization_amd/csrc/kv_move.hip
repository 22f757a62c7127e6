// spin_kv_move kernel: tokens of the paged cache to other slots of it.
//
// A workgroup takes 64 tokens of one head of one sequence: it loads all that
// they hold (codes, scales, a weight) and then stores it.  In place the chunks of
// a head follow each other in one workgroup: token i of the list comes from place
// list[i] >= i, the list ascends, so that what a chunk stores lies before
// everything that a later chunk loads.  Into other pages the chunks are
// independent.
#include "kv_batch.h"
#include "spin_internal.h"

namespace spin {
namespace {

constexpr int kMoveThreads = 256;
constexpr int kMoveTokens = 64;

template <int BITS>
__global__ __launch_bounds__(kMoveThreads) void kv_move_kernel(KvMoveArgs a, int chunks, int turns) {
    struct alignas(BITS) Piece { uint32_t w[BITS / 4]; };
    __shared__ long long from_sh[kMoveTokens], to_sh[kMoveTokens];
    const int h = blockIdx.x % a.Hkv;
    const int item = blockIdx.x / a.Hkv;
    const int b = item / chunks, chunk = item - b * chunks;
    const int32_t* list = a.kept + (static_cast<long long>(b) * a.kept_heads + (a.kept_heads > 1 ? h : 0)) * a.n;
    const long long at = a.at ? a.at[b] : 0;
    auto token = [&](const int32_t* table, int pages, long long place) -> long long {
        if (place < 0 || place >= static_cast<long long>(pages) << a.page_log2) return -1;
        const int page = table[static_cast<long long>(b) * pages + (place >> a.page_log2)];
        if (page < 0 || page >= a.n_pages) return -1;
        return ((static_cast<long long>(page) * a.Hkv + h) << a.page_log2) + (place & ((1 << a.page_log2) - 1));
    };
    for (int turn = 0; turn < turns; ++turn) {
        const int i0 = (chunk + turn) * kMoveTokens;
        if (threadIdx.x < kMoveTokens) {
            const int i = i0 + static_cast<int>(threadIdx.x);
            const int src = i < a.n ? list[i] : -1;
            long long from = src >= 0 ? token(a.page_table, a.max_pages, at + src) : -1;
            const long long to = from >= 0 ? token(a.to_table ? a.to_table : a.page_table, a.to_table ? a.to_pages : a.max_pages, at + i) : -1;
            if (to < 0 || to == from) from = -1;
            from_sh[threadIdx.x] = from;
            to_sh[threadIdx.x] = to;
        }
        __syncthreads();
        uint4 k[BITS / 4];
        Piece v[4];
        uint32_t s = 0;
        const int s_token = threadIdx.x & 63, s_kind = threadIdx.x >> 6;        // a wave each: key scales, value scales, weights
#pragma unroll
        for (int x = 0; x < BITS / 4; ++x) {
            const int p = x * kMoveThreads + threadIdx.x;                       // BITS pieces of 16 bytes a token
            const long long from = from_sh[p / BITS];
            if (from >= 0) k[x] = reinterpret_cast<const uint4*>(a.K_codes)[from * BITS + p % BITS];
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int p = x * kMoveThreads + threadIdx.x;                       // 16 octets of four tokens
            const long long from = from_sh[p >> 6 << 2 | (p & 3)];
            if (from >= 0) v[x] = reinterpret_cast<const Piece*>(a.V_codes)[((from >> 2) * 16 + (p >> 2 & 15)) * 4 + (from & 3)];
        }
        {
            const long long from = from_sh[s_token];
            if (from >= 0) {
                if (s_kind == 0) s = a.K_scale[from];
                if (s_kind == 1) s = a.V_scale[from];
                if (s_kind == 2 && a.W) s = __float_as_uint(a.W[from]);
            }
        }
        // all loads have arrived before the first store
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
#pragma unroll
        for (int x = 0; x < BITS / 4; ++x) {
            const int p = x * kMoveThreads + threadIdx.x;
            if (from_sh[p / BITS] >= 0) reinterpret_cast<uint4*>(a.K_codes)[to_sh[p / BITS] * BITS + p % BITS] = k[x];
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int p = x * kMoveThreads + threadIdx.x, i = p >> 6 << 2 | (p & 3);
            const long long to = to_sh[i];
            if (from_sh[i] >= 0) reinterpret_cast<Piece*>(a.V_codes)[((to >> 2) * 16 + (p >> 2 & 15)) * 4 + (to & 3)] = v[x];
        }
        if (from_sh[s_token] >= 0) {
            const long long to = to_sh[s_token];
            if (s_kind == 0) a.K_scale[to] = static_cast<uint16_t>(s);
            if (s_kind == 1) a.V_scale[to] = static_cast<uint16_t>(s);
            if (s_kind == 2 && a.W) a.W[to] = __uint_as_float(s);
        }
        __syncthreads();
    }
}

int chunks_of(int n) { return (n + kMoveTokens - 1) / kMoveTokens; }

}  // namespace

bool kv_move_fits(int Hkv, int B, int n) { return static_cast<double>(Hkv) * B * ((static_cast<double>(n) + kMoveTokens - 1) / kMoveTokens) <= (1 << 24) - 1; }

hipError_t launch_kv_move(const KvMoveArgs& a, int bits, hipStream_t s) {
    const int chunks = a.to_table ? chunks_of(a.n) : 1, turns = a.to_table ? 1 : chunks_of(a.n);
    const dim3 grid(static_cast<unsigned>(a.B) * a.Hkv * chunks);
    if (bits == 8)
        hipLaunchKernelGGL((kv_move_kernel<8>), grid, dim3(kMoveThreads), 0, s, a, chunks, turns);
    else
        hipLaunchKernelGGL((kv_move_kernel<4>), grid, dim3(kMoveThreads), 0, s, a, chunks, turns);
    return hipGetLastError();
}

}  // namespace spin
