// Host-side launchers behind the libspin C ABI.  abi.cpp validates every
// argument before calling these; the launchers only pick a kernel and launch.
#pragma once

#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "libspin.h"

namespace spin {

// Hadamard order n = 2^log2p * (has12 ? 12 : 1).
struct HadOrder {
    int n;
    int log2p;
    bool has12;
};

// bits = 4: packed nibbles [M][K/2]; bits = 8: one signed byte per code [M][K].
hipError_t launch_fwht_quant(const void* X, bool x_f16, int M, int K, HadOrder h, int bits,
                             uint8_t* Xq, float* x_scale, float* X_rot, hipStream_t s);

// kernel: 0 the automatic choice, 1 the int8 kernels, 2 the FP6 kernel
// (abi.cpp has checked that the FP6 kernel takes K).
hipError_t launch_w4a4_gemm(const uint8_t* Xq, const float* x_scale, const uint8_t* Wq,
                            const float* w_scale, int M, int N, int K, float* Y,
                            int32_t* acc_out, int kernel, hipStream_t s);

hipError_t launch_kv_quant(const void* X, bool x_f16, int T, int H, bool rotate, int bits,
                           uint8_t* codes, uint16_t* scale, float* X_rot, hipStream_t s);

// Q (optional, rotate only), K (rotate + quantize) and V (quantize) in one launch.
hipError_t launch_kv_qkv(const void* Q, const void* K, const void* V, bool x_f16, int T, int Hq, int Hkv,
                         int bits, float* Q_rot, uint8_t* K_codes, uint16_t* K_scale, float* K_rot,
                         uint8_t* V_codes, uint16_t* V_scale, hipStream_t s);

// cos | sin rows of positions pos0 .. pos0 + P - 1 for n frequencies.
hipError_t launch_rope_table(const double* inv_freq, int n, int pos0, int P, double attn_scale, float* table,
                             hipStream_t s);

// Norm + position rotation + R3 of queries and keys, codes of keys and values
// into the paged cache (include/libspin.h has the layout).
struct KvAppendArgs {
    const void* Q;                 // NULL: no queries (Hq is 0)
    const void* K;
    const void* V;
    int T, Hq, Hkv;
    long long q_stride, k_stride, v_stride;   // values between tokens
    const float* q_norm;           // [128] or NULL
    const float* k_norm;
    double eps;
    const float* rope;             // [rope_len][rot_dim] cos | sin, NULL with rot_dim 0
    int rope_len, rot_dim;
    bool interleaved;
    int pos0, B;
    const int32_t* positions;      // [T]: in place of pos0 + place, or NULL
    const int32_t* q_start;
    const int32_t* kv_len;
    const int32_t* page_table;
    int max_pages, n_pages, page_log2;
    uint8_t* K_codes;
    uint16_t* K_scale;
    uint8_t* V_codes;
    uint16_t* V_scale;
    uint16_t* Q_out;
    unsigned kv_blocks;            // set by the launcher
    int heads;
    float norm;
};
hipError_t launch_kv_append(KvAppendArgs a, bool x_f16, int bits, hipStream_t s);
long long kv_append_blocks(int T, int Hq, int Hkv);

// Attention over the paged cache.
struct KvAttnArgs {
    const uint16_t* Q;
    int T, Hq, Hkv;
    const uint8_t* K_codes;
    const uint16_t* K_scale;
    const uint8_t* V_codes;
    const uint16_t* V_scale;
    int n_pages, page_log2, B;
    const int32_t* q_start;
    const int32_t* kv_len;
    const int32_t* page_table;
    int max_pages;
    const int32_t* prefix_table;   // [ceil(prefix_len / page)], read if prefix_len > 0
    int prefix_len;
    float scale, softcap;
    const float* slopes;
    int window;
    bool causal;
    const int32_t* bidir_len;
    const uint32_t* tree;          // [T][tree_words], NULL: new tokens see each other by `causal`, which is false with a tree
    int tree_words;
    const int32_t* positions;      // [T], read with a tree; NULL: no window, no slopes
    uint16_t* O;
    float* lse;                    // [T][Hq] or NULL
    float* partial;                // the workspace
};
// Bytes of workspace the launch needs (0: none), and whether it fits one launch.
size_t kv_attn_workspace(int T, int Hq, int Hkv, int B, int max_kv, int prefix_len);
bool kv_attn_fits(int T, int Hq, int Hkv, int B, int max_kv, int prefix_len);
hipError_t launch_kv_attn(const KvAttnArgs& a, int bits, hipStream_t s);

// Ancestors and positions of drafted tokens.
struct KvTreeArgs {
    const int32_t* parent;
    int T, B;
    const int32_t* q_start;
    const int32_t* kv_len;
    int pos0, words;
    uint32_t* tree;
    int32_t* positions;
};
hipError_t launch_kv_tree(const KvTreeArgs& a, hipStream_t s);

// Attention weight of cached tokens.
struct KvWeightsArgs {
    const uint16_t* Q;
    const float* lse;
    int T, Hq, Hkv;
    const uint8_t* K_codes;
    const uint16_t* K_scale;
    int n_pages, page_log2, B;
    const int32_t* q_start;
    const int32_t* kv_len;
    const int32_t* page_table;
    int max_pages, pos0;
    float scale, softcap;
    const float* slopes;
    int window;
    bool causal;
    const int32_t* bidir_len;
    const float* prior;            // NULL: none
    const int32_t* prior_len;      // [B]: tokens that have one, NULL: all
    float decay;
    float* W;
    float* partial;                // the workspace
};
size_t kv_weights_workspace(int T, int Hq, int Hkv, int B, int max_kv);
bool kv_weights_fits(int T, int Hq, int Hkv, int B, int max_kv);
hipError_t launch_kv_weights(const KvWeightsArgs& a, int bits, hipStream_t s);

// The tokens of greatest weight.
struct KvChooseArgs {
    const float* W;
    int Hkv, n_pages, page_log2, B;
    const int32_t* kv_len;
    const int32_t* page_table;
    int max_pages, keep, first, recent;
    int32_t* kept;
    int32_t* lens;                 // or kv_len itself
    int* counts;                   // the workspace
};
size_t kv_choose_workspace(int Hkv, int B, int room);
bool kv_choose_fits(int Hkv, int B, int room);
hipError_t launch_kv_choose(const KvChooseArgs& a, hipStream_t s);

// Tokens to other slots of the cache.
struct KvMoveArgs {
    uint8_t* K_codes;
    uint16_t* K_scale;
    uint8_t* V_codes;
    uint16_t* V_scale;
    float* W;                      // or NULL
    int Hkv, n_pages, page_log2, B;
    const int32_t* page_table;
    int max_pages;
    const int32_t* kept;
    int kept_heads, n;             // 1 or Hkv
    const int32_t* at;             // or NULL: 0
    const int32_t* to_table;       // NULL: page_table, in place
    int to_pages;                  // of to_table; in place, those of page_table that tokens may go to
};
bool kv_move_fits(int Hkv, int B, int n);
hipError_t launch_kv_move(const KvMoveArgs& a, int bits, hipStream_t s);

// The FP6 matrix-core path of launch_w4a4_gemm (exact for K <= kGemmFp6MaxK).
constexpr int kGemmFp6MaxK = 65536;
bool w4a4_gemm_fp6_applies(int M, int N, int K);
int w4a4_gemm_fp6_split_slices(int M, int N, int K, bool forced);
hipError_t launch_w4a4_gemm_fp6_split(const uint8_t* Xq, const float* x_scale, const uint8_t* Wq,
                                      const float* w_scale, int M, int N, int K, int slices, float* Y,
                                      int32_t* acc_out, hipStream_t s);
hipError_t launch_codes_f6(const uint8_t* Wq, int N, int K, uint8_t* Wf6, int32_t* w_sum, hipStream_t s);
hipError_t launch_w4a4_gemm_f6f6(const uint8_t* Xf6, const int32_t* x_sum, const float* x_scale,
                                 const uint8_t* Wf6, const int32_t* w_sum, const float* w_scale, int M, int N, int K,
                                 float* Y, int32_t* acc_out, hipStream_t s);
hipError_t launch_w4a4_gemm_fp6(const uint8_t* Xq, const float* x_scale, const uint8_t* Wq,
                                const float* w_scale, int M, int N, int K, float* Y,
                                int32_t* acc_out, hipStream_t s);

// Int8 activation codes [M][K] against packed INT4 weights [N][K/2]; K % 128 == 0.
hipError_t launch_w4a8_gemm(const int8_t* Xq8, const float* x_scale, const uint8_t* Wq,
                            const float* w_scale, int M, int N, int K, float* Y,
                            int32_t* acc_out, hipStream_t s);

// fwht_quant (fp16, K = had_n = 12288, INT4) then the FP6 GEMM, one cooperative launch.
hipError_t launch_fwht_quant_gemm(const __half* X, int M, int K, const uint8_t* Wq, const float* w_scale, int N,
                                  uint8_t* Xq, float* x_scale, float* Y, int32_t* acc_out, uint32_t* workspace,
                                  hipStream_t s);

// Device address of the current device's library-owned flags for the fused
// kernel (SPIN_FWHT_QUANT_GEMM_WORKSPACE_WORDS words, zero between calls),
// looked up once per device.
hipError_t fwht_quant_gemm_scratch(uint32_t** out);

// fp16 rows of 12288, H_12 (x) H_1024, INT4 codes in the FP6 operand layout + row code sums.
hipError_t launch_fwht_quant_f6(const __half* X, int M, uint8_t* Xf6, int32_t* x_sum, float* x_scale,
                                hipStream_t s);
// had_n = 1: fp16 / fp32 rows of K (K % 128 == 0, K <= SPIN_FWHT_F6_QUANT_MAX_K), per-token INT4 codes in
// the FP6 operand layout + row code sums.
hipError_t launch_quant_rows_f6(const void* X, bool x_f16, int M, int K, uint8_t* Xf6, int32_t* x_sum,
                                float* x_scale, hipStream_t s);
// The FP6 GEMM on activation codes in that layout.
hipError_t launch_w4a4_gemm_f6(const uint8_t* Xf6, const int32_t* x_sum, const float* x_scale, const uint8_t* Wq,
                               const float* w_scale, int M, int N, int K, float* Y, int32_t* acc_out,
                               hipStream_t s);

// Compute units of the current device, queried once per device and cached
// (0 if the runtime cannot tell); safe to call from several threads.
int device_cu_count();

hipError_t launch_fold_rotation(const float* W, int K, int N, const float* R, int r_block,
                                HadOrder h, float* W_rot, uint8_t* Wq, float* w_scale,
                                hipStream_t s);

}  // namespace spin
