// spin_kv_move kernel: tokens of the paged cache to other slots of it.
//
// A workgroup takes 16 tokens a wave of one head of one sequence: it loads what
// they hold (codes, scales, a weight) and stores it when all of it has arrived.
//
// In place a workgroup takes all chunks of its head, one after the other: token i
// of the list comes from place list[i] >= i and the list ascends, so that what a
// chunk stores lies before everything that later chunks load.  The next chunk's
// tokens are therefore loaded before this one's are stored, and looked up before
// this one's have arrived.  Keys and values go apart where there are few heads.
// Into other pages all chunks are independent.
//
// Bound: into other pages memory, and in place the loads that wait for each other
// (the list, the tables, the codes).  Measured: 2048 tokens of each of 16
// sequences and 8 heads, INT4, with weights, into other pages 20 us (72 MB, 3.6
// TB/s: sources are spread, four bytes of a value's octet at a time), in place 24 us
// (of 64 sequences 77; 4096 of one of 131072 tokens, 16 turns of 16 workgroups, 33,
// into other pages 5.6); the accepted paths of 64 trees 4.6 us.
#include "kv_batch.h"
#include "spin_internal.h"

namespace spin {
namespace {

constexpr int kFewWaves = 4, kManyWaves = 16;
constexpr int kWaveTokens = 16;
constexpr int kHeadsEnough = 256;          // in place: workgroups from which keys and values go together

template <int BITS, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void kv_move_kernel(KvMoveArgs a, int chunks, int turns, int parts) {
    constexpr int kThreads = 64 * WAVES, kTokens = kWaveTokens * WAVES;
    typedef uint32_t U4 __attribute__((ext_vector_type(4)));
    typedef uint32_t Piece __attribute__((ext_vector_type(BITS / 4)));       // a token's octet of values
    // of three chunks: one is stored while the next is loaded and the one behind it looked up
    __shared__ long long from_sh[3][kTokens], to_sh[3][kTokens];
    const int part = blockIdx.x % parts, head = blockIdx.x / parts, h = head % a.Hkv;
    const bool keys = part == 0, values = part == parts - 1;
    const int item = head / a.Hkv, b = item / chunks, chunk = item - b * chunks;
    const int32_t* list = a.kept + (static_cast<long long>(b) * a.kept_heads + (a.kept_heads > 1 ? h : 0)) * a.n;
    const long long at = a.at ? a.at[b] : 0;
    auto token = [&](const int32_t* table, int pages, long long place) -> long long {
        if (place < 0 || place >= static_cast<long long>(pages) << a.page_log2) return -1;
        const int page = table[static_cast<long long>(b) * pages + (place >> a.page_log2)];
        if (page < 0 || page >= a.n_pages) return -1;
        return ((static_cast<long long>(page) * a.Hkv + h) << a.page_log2) + (place & ((1 << a.page_log2) - 1));
    };
    auto look_up = [&](int turn) __attribute__((always_inline)) {
        if (threadIdx.x >= kTokens) return;
        const long long i = static_cast<long long>(chunk + turn) * kTokens + threadIdx.x;
        const int src = i < a.n ? list[i] : -1;
        long long from = src >= 0 ? token(a.page_table, a.max_pages, at + src) : -1;
        const long long to = src >= 0 ? token(a.to_table ? a.to_table : a.page_table, a.to_pages, at + i) : -1;
        if (to < 0 || to == from) from = -1;
        from_sh[turn % 3][threadIdx.x] = from;
        to_sh[turn % 3][threadIdx.x] = to;
    };
    // a thread's share of a chunk: BITS / 4 of a token's BITS pieces of 16 bytes of keys, four tokens' octets of values,
    // and of a wave in four a scale or weight
    struct Held {
        U4 k[BITS / 4];
        Piece v[4];
        uint32_t s;
    };
    const int s_token = threadIdx.x % kTokens, s_kind = threadIdx.x / kTokens;          // key scales, value scales, weights
    auto load = [&](int turn) __attribute__((always_inline)) {
        Held x;
        const long long* const sources = from_sh[turn % 3];
        if (keys) {
#pragma unroll
            for (int y = 0; y < BITS / 4; ++y) {
                const int p = y * kThreads + threadIdx.x;
                const long long from = sources[p / BITS];
                if (from >= 0) x.k[y] = reinterpret_cast<const U4*>(a.K_codes)[from * BITS + p % BITS];
            }
        }
        if (values) {
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int p = y * kThreads + threadIdx.x;                               // 16 octets of four tokens
                const long long from = sources[p >> 6 << 2 | (p & 3)];
                if (from >= 0) x.v[y] = reinterpret_cast<const Piece*>(a.V_codes)[((from >> 2) * 16 + (p >> 2 & 15)) * 4 + (from & 3)];
            }
        }
        const long long from = sources[s_token];
        if (from >= 0) {
            if (s_kind == 0 && keys) x.s = a.K_scale[from];
            if (s_kind == 1 && values) x.s = a.V_scale[from];
            if (s_kind == 2 && values && a.W) x.s = __float_as_uint(a.W[from]);
        }
        return x;
    };
    auto store = [&](int turn, const Held& x) __attribute__((always_inline)) {
        const long long *const sources = from_sh[turn % 3], *const places = to_sh[turn % 3];
        if (keys) {
#pragma unroll
            for (int y = 0; y < BITS / 4; ++y) {
                const int p = y * kThreads + threadIdx.x;
                if (sources[p / BITS] >= 0) reinterpret_cast<U4*>(a.K_codes)[places[p / BITS] * BITS + p % BITS] = x.k[y];
            }
        }
        if (values) {
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int p = y * kThreads + threadIdx.x, i = p >> 6 << 2 | (p & 3);
                const long long to = places[i];
                if (sources[i] >= 0) reinterpret_cast<Piece*>(a.V_codes)[((to >> 2) * 16 + (p >> 2 & 15)) * 4 + (to & 3)] = x.v[y];
            }
        }
        if (sources[s_token] >= 0) {
            const long long to = places[s_token];
            if (s_kind == 0 && keys) a.K_scale[to] = static_cast<uint16_t>(x.s);
            if (s_kind == 1 && values) a.V_scale[to] = static_cast<uint16_t>(x.s);
            if (s_kind == 2 && values && a.W) a.W[to] = __uint_as_float(x.s);
        }
    };
    look_up(0);
    __syncthreads();
    Held x = load(0);
    for (int turn = 0; turn < turns; ++turn) {
        if (turn + 1 < turns) look_up(turn + 1);
        // every wave's loads have arrived before any wave stores
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (turn + 1 == turns) {
            store(turn, x);
            break;
        }
        const Held next = load(turn + 1);
        store(turn, x);
        x = next;
    }
}

template <int BITS, int WAVES>
hipError_t launch_waves(const KvMoveArgs& a, hipStream_t s) {
    constexpr int kTokens = kWaveTokens * WAVES;
    const int all = static_cast<int>((static_cast<long long>(a.n) + kTokens - 1) / kTokens);
    const int chunks = a.to_table ? all : 1, turns = a.to_table ? 1 : all;
    const int parts = !a.to_table && static_cast<long long>(a.B) * a.Hkv < kHeadsEnough ? 2 : 1;
    hipLaunchKernelGGL((kv_move_kernel<BITS, WAVES>), dim3(static_cast<unsigned>(a.B) * a.Hkv * chunks * parts), dim3(64 * WAVES), 0, s, a,
                       chunks, turns, parts);
    return hipGetLastError();
}

template <int BITS>
hipError_t launch_bits(const KvMoveArgs& a, hipStream_t s) {
    return !a.to_table && a.n > kWaveTokens * kFewWaves ? launch_waves<BITS, kManyWaves>(a, s) : launch_waves<BITS, kFewWaves>(a, s);
}

}  // namespace

bool kv_move_fits(int Hkv, int B, int n) {
    // workgroups of 256 a launch dimension holds; in place there are fewer, of 1024
    return static_cast<double>(Hkv) * B * ((static_cast<double>(n) + kWaveTokens * kFewWaves - 1) / (kWaveTokens * kFewWaves)) <= (1 << 24) - 1 &&
           static_cast<double>(Hkv) * B <= (1 << 22) - 1;
}

hipError_t launch_kv_move(const KvMoveArgs& a, int bits, hipStream_t s) {
    return bits == 8 ? launch_bits<8>(a, s) : launch_bits<4>(a, s);
}

}  // namespace spin
