// spin_rope_table kernel: the cosines and sines of the position rotation that
// spin_kv_append applies (the rotation between qkv_proj and the R3 Hadamard,
// page "SpinQuant, Reproduced", Q5, puts positions into queries and keys).
//
// Row p holds cos(a_i) * s and sin(a_i) * s, a_i = (pos0 + p) * inv_freq[i].
// A position of 2^20 turns the fastest pair by 2^20 radians, where a float32
// angle is 2^-4 wide: the angle, its reduction and the functions are held in
// 64 bits and rounded once.
#include "spin_internal.h"

namespace spin {
namespace {

constexpr int kRopeThreads = 256;

// One thread per (position, frequency): the two stores of a wave are runs of n
// consecutive floats.
__global__ __launch_bounds__(kRopeThreads) void rope_table_kernel(const double* __restrict__ inv_freq, int n, int pos0,
                                                                  long long pairs, double attn_scale,
                                                                  float* __restrict__ table) {
    const long long at = static_cast<long long>(blockIdx.x) * kRopeThreads + threadIdx.x;
    if (at >= pairs) return;
    const unsigned p = static_cast<unsigned>(at / n), i = static_cast<unsigned>(at - static_cast<long long>(p) * n);
    double s, c;
    sincos((static_cast<double>(pos0) + p) * inv_freq[i], &s, &c);
    float* row = table + static_cast<long long>(p) * 2 * n;
    row[i] = static_cast<float>(c * attn_scale);
    row[n + i] = static_cast<float>(s * attn_scale);
}

}  // namespace

hipError_t launch_rope_table(const double* inv_freq, int n, int pos0, int P, double attn_scale, float* table,
                             hipStream_t s) {
    const long long pairs = static_cast<long long>(P) * n;
    hipLaunchKernelGGL(rope_table_kernel, dim3(static_cast<unsigned>((pairs + kRopeThreads - 1) / kRopeThreads)),
                       dim3(kRopeThreads), 0, s, inv_freq, n, pos0, pairs, attn_scale, table);
    return hipGetLastError();
}

}  // namespace spin
