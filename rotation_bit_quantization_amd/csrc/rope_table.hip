// spin_rope_table kernel: the cosines and sines of the position rotation that
// spin_kv_append applies (the rotation between qkv_proj and the R3 Hadamard,
// page "SpinQuant, Reproduced", Q5, puts positions into queries and keys).
//
// Row p holds cos(a_p) * s and sin(a_p) * s, a_p = fl64((pos0 + p) * inv_freq[i]).
// A position of 2^20 turns the fastest pair by 2^20 radians, where a float32
// angle is 2^-4 wide: the angle, its reduction and the functions are held in
// 64 bits and rounded once.
//
// The functions cost about 125 instructions a pair, four times what their two
// stores take.  So a thread takes them at the middle m of kRun positions and at
// inv_freq, and turns from there a step at a time:
//   cos(a_m + j f) = cos(a_m + (j - 1) f) cos f - sin(a_m + (j - 1) f) sin f
// and likewise the sine.  The angle wanted is the rounded a_{m + j}, not a_m + j f:
// the difference e = (a_{m + j} - a_m) - j f, at most two roundings, 2^-52 of
// the angle, turns the pair by the first order, (c - s e, s + c e).  Below 2^25
// radians e^2 / 2 is below 2^-55; angles above take the functions every time.
// Eight steps add less than 27 * 2^-53 (a step 2.4 * 2^-53 in each of the pair).
//
// Bound: writing the table.  Measured: 40960 positions of 64 pairs 7.4 us (21 MB,
// 2.8 TB/s; a launch's 3 us among them), 262144 of 32 12.9 us (67 MB, 5.2 TB/s);
// with the functions for every pair 12 and 29 us.  Runs of 8 and 32: 7.5 and 14.4,
// 7.2 and 14.6.
#include "spin_internal.h"

namespace spin {
namespace {

constexpr int kRopeThreads = 256;

constexpr int kRun = 16;

// One thread per (run of positions, frequency): the two stores of a wave are
// runs of n consecutive floats.
__global__ __launch_bounds__(kRopeThreads) void rope_table_kernel(const double* __restrict__ inv_freq, int n, int pos0,
                                                                  int P, long long work, double attn_scale,
                                                                  float* __restrict__ table) {
#pragma clang fp contract(off)   // the angles are rounded products
    const long long at = static_cast<long long>(blockIdx.x) * kRopeThreads + threadIdx.x;
    if (at >= work) return;
    const unsigned run = static_cast<unsigned>(at) / n, i = static_cast<unsigned>(at) - run * n;
    const int first = static_cast<int>(run * kRun);
    const double f = inv_freq[i], start = static_cast<double>(pos0) + first;
    float* row = table + static_cast<long long>(first) * 2 * n + i;
    auto put = [&](int k, double c, double s) __attribute__((always_inline)) {
        if (k >= P - first) return;
        row[2LL * n * k] = static_cast<float>(c * attn_scale);
        row[2LL * n * k + n] = static_cast<float>(s * attn_scale);
    };
    if (!(__builtin_fabs((start + kRun) * f) <= 0x1p25)) {
        for (int k = 0; k < kRun && k < P - first; ++k) {
            double s, c;
            sincos((start + k) * f, &s, &c);
            put(k, c, s);
        }
        return;
    }
    constexpr int m = kRun / 2;
    const double middle = (start + m) * f;
    double s_m, c_m, s_f, c_f;
    sincos(middle, &s_m, &c_m);
    sincos(f, &s_f, &c_f);
    double c = c_m, s = s_m;
#pragma unroll
    for (int j = 0; j < m; ++j) {
        const double e = __builtin_fma(-static_cast<double>(j), f, (start + (m + j)) * f - middle);
        put(m + j, __builtin_fma(-s, e, c), __builtin_fma(c, e, s));
        const double turned = __builtin_fma(c, c_f, -(s * s_f));
        s = __builtin_fma(s, c_f, c * s_f);
        c = turned;
    }
    c = c_m;
    s = s_m;
#pragma unroll
    for (int j = 1; j <= m; ++j) {
        const double turned = __builtin_fma(c, c_f, s * s_f);
        s = __builtin_fma(s, c_f, -(c * s_f));
        c = turned;
        const double e = __builtin_fma(static_cast<double>(j), f, (start + (m - j)) * f - middle);
        put(m - j, __builtin_fma(-s, e, c), __builtin_fma(c, e, s));
    }
}

}  // namespace

hipError_t launch_rope_table(const double* inv_freq, int n, int pos0, int P, double attn_scale, float* table,
                             hipStream_t s) {
    const long long work = (static_cast<long long>(P) + kRun - 1) / kRun * n;
    hipLaunchKernelGGL(rope_table_kernel, dim3(static_cast<unsigned>((work + kRopeThreads - 1) / kRopeThreads)),
                       dim3(kRopeThreads), 0, s, inv_freq, n, pos0, P, work, attn_scale, table);
    return hipGetLastError();
}

}  // namespace spin
