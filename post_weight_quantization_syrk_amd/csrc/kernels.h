// Internal launchers behind the C ABI (include/gptq.h).  Each returns the
// hipError_t of its launches; argument validation happens in gptq_abi.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stddef.h>

namespace gptq {

// ---- Hessian: H(lower) += 2 X^T X --------------------------------------
struct SyrkPlan {
  int tile;        // output tile edge (256 for bf16, 64 for fp32)
  int ntile;       // tiles per dimension
  int ntri;        // lower-triangle tiles
  int splits;      // token splits (split-K)
  int64_t kper;    // tokens per split
  size_t partial_bytes; // split-K partial tiles [splits][ntri][tile * tile] fp32
  size_t ws_bytes;      // = partial_bytes
};
SyrkPlan syrk_plan(int64_t d, int64_t n, int x_dtype);
// The allocation-free entry point: its split-K partials live in a fixed
// per-device array of NOALLOC_SCRATCH_BYTES; the split count is capped to fit
// (splits = 0: even one split does not fit).
constexpr size_t NOALLOC_SCRATCH_BYTES = (size_t)64 << 20;
constexpr int MAX_DEVICES = 64;
SyrkPlan syrk_plan_capped(int64_t d, int64_t n, int x_dtype, size_t max_bytes);
hipError_t syrk_scratch(void** ptr);  // this device's copy of the array
hipError_t syrk_launch(float* H, int64_t d, const void* X, int x_dtype, int64_t n, int64_t ldx,
                       void* ws, const SyrkPlan& plan, hipStream_t stream);

// ---- prepare: dead channels, damping, factorization, U ------------------
size_t prepare_workspace(int64_t d);
hipError_t prepare_launch(float* H, int64_t d, double damp, float* U, uint8_t* dead,
                          int32_t* dev_status, void* ws, hipStream_t stream);
// The same for H[perm][:, perm] (perm null: natural order); dead stays in
// natural order, U is the permuted problem's factor.
hipError_t prepare_perm_launch(float* H, int64_t d, double damp, const int32_t* perm, float* U,
                               uint8_t* dead, int32_t* dev_status, void* ws, hipStream_t stream);

// Several weight matrices that share U (one Hessian), stacked by rows in
// order; outputs stacked the same way.
hipError_t quantize_multi_launch(const void* const* Ws, const int64_t* d_outs, int count,
                                 int w_dtype, int64_t d_in, const float* U, const uint8_t* dead,
                                 int bits, int group_size, int sym, uint8_t* codes,
                                 float* scales, float* zeros, float* loss_rows, void* ws,
                                 hipStream_t stream);

// ---- activation order: perm = columns by ascending sum_t |x_t,c| ----------
size_t act_order_workspace(int64_t d, int64_t n_tokens);
hipError_t act_order_launch(const void* X, int x_dtype, int64_t n_tokens, int64_t ldx, int64_t d,
                            int32_t* perm, double* act_sum, void* ws, hipStream_t stream);

// ---- quantize ------------------------------------------------------------
size_t quantize_workspace(int64_t d_out, int64_t d_in, int block);
hipError_t quantize_launch(const void* W, int w_dtype, int64_t d_out, int64_t d_in,
                           const float* U, const uint8_t* dead, int bits, int group_size,
                           int sym, uint8_t* codes, float* scales, float* zeros,
                           float* loss_rows, void* ws, hipStream_t stream);
// Columns processed in the order perm (null: natural order), static or
// dynamic groups; codes come back in natural order, g_idx (may be null) maps
// each column to its group.
size_t quantize_perm_workspace(int64_t d_out, int64_t d_in, int block);
hipError_t quantize_perm_launch(const void* W, int w_dtype, int64_t d_out, int64_t d_in,
                                const float* U, const uint8_t* dead, const int32_t* perm,
                                int static_groups, int bits, int group_size, int sym,
                                uint8_t* codes, float* scales, float* zeros, int32_t* g_idx,
                                float* loss_rows, void* ws, hipStream_t stream);

// ---- pack ----------------------------------------------------------------
hipError_t pack_launch(const uint8_t* codes, const float* scales, const float* zeros,
                       int64_t d_out, int64_t d_in, int bits, int n_groups, int sym,
                       uint32_t* qweight, uint16_t* scales_f16, uint16_t* zeros_f16,
                       hipStream_t stream);

// ---- dequantized product with 4-bit packed weights ------------------------
hipError_t w4a16_launch(const void* X, int64_t m, int64_t ldx, const uint32_t* qweight,
                        const uint16_t* scales_f16, const uint16_t* zeros_f16, int64_t d_out,
                        int64_t d_in, int group_size, float* Y, hipStream_t stream);

// ---- the same product for a few tokens (m <= 64) ---------------------------
size_t w4a16_vec_workspace(int64_t m, int64_t d_out, int64_t d_in, int group_size);
hipError_t w4a16_vec_launch(const void* X, int64_t m, int64_t ldx, const uint32_t* qweight,
                            const uint16_t* scales_f16, const uint16_t* zeros_f16, int64_t d_out,
                            int64_t d_in, int group_size, float* Y, void* ws, hipStream_t stream);

// ---- residual addition, RMS norm, bf16 or 8-bit output ---------------------
hipError_t add_rmsnorm_launch(const void* X, int x_dtype, int64_t ldx, const void* R, int r_dtype,
                              int64_t ldr, void* R_out, int64_t ldro, const void* weight,
                              int w_dtype, double eps, int64_t m, int64_t d, void* out,
                              int out_dtype, int64_t ldo, float* out_scales, hipStream_t stream);

// ---- product of 4-bit packed weights with 8-bit activations ----------------
size_t w4a8_workspace(int64_t m, int64_t d_out, int64_t d_in, int group_size);
hipError_t w4a8_launch(const int8_t* X, const float* x_scales, int64_t m, int64_t ldx,
                       const uint32_t* qweight, const uint16_t* scales_f16,
                       const uint16_t* zeros_f16, int64_t d_out, int64_t d_in, int group_size,
                       float* Y, void* ws, hipStream_t stream);

// ---- W4A16 product with bias, activation, gate and residual ----------------
enum Activation { ACT_NONE = 0, ACT_RELU = 1, ACT_SILU = 2, ACT_GELU = 3, ACT_GELU_TANH = 4 };

struct Epilogue {
  const void* bias;  // [d_out], null: none
  const void* res;   // [m][ldr], null: none
  void* y;           // [m][ldy]
  int64_t ldr, ldy;
  int F;             // columns of Y
  int act;
  bool bias_f32, res_f32, y_f32;
  bool vec4;         // four neighbouring values of Y at a multiple of 4 are one aligned store
};

size_t linear_workspace(int64_t m, int64_t d_out, int64_t d_in, int group_size, bool gated);
hipError_t linear_launch(const void* X, int64_t m, int64_t ldx, const uint32_t* qweight,
                         const uint16_t* scales_f16, const uint16_t* zeros_f16, int64_t d_out,
                         int64_t d_in, int group_size, bool gated, const Epilogue& e, void* ws,
                         hipStream_t stream);
// for few tokens
size_t linear_vec_workspace(int64_t m, int64_t d_out, int64_t d_in, int group_size, bool gated);
hipError_t linear_vec_launch(const void* X, int64_t m, int64_t ldx, const uint32_t* qweight,
                             const uint16_t* scales_f16, const uint16_t* zeros_f16, int64_t d_out,
                             int64_t d_in, int group_size, bool gated, const Epilogue& e, void* ws,
                             hipStream_t stream);

// ---- norms of queries and keys, rotation, rows of a cache ------------------
// Strides in elements: ld* between tokens (rows), hs* between heads.
struct RopeArgs {
  const void *q, *k, *v;  // v null: none
  int64_t ldq, hsq, ldk, hsk, ldv, hsv;
  int64_t m;
  int hq, hk, hd, rot;
  const int32_t* positions;
  const double* inv_freq;
  const void *q_weight, *k_weight;  // null: no norm
  bool w_f32, interleaved;
  double eps;
  const int64_t* slots;  // null: row t
  int64_t kv_rows;       // rows of k_out and v_out
  uint16_t *q_out, *k_out, *v_out;
  int64_t ldqo, hsqo, ldko, hsko, ldvo, hsvo;
};
hipError_t qk_norm_rope_launch(const RopeArgs& a, bool f32, hipStream_t stream);

// ---- attention over packed queries and runs of keys ------------------------
struct AttnArgs {
  const uint16_t *q, *k, *v;
  int64_t ldq, hsq, ldk, hsk, ldv, hsv;  // elements, as above
  int64_t tq, kv_rows;
  int batch, hq, hk, hd;
  const int32_t* cu_q;
  const int64_t* kv_start;  // null, with kv_len: the keys are packed as the queries
  const int32_t* kv_len;
  int causal;
  float scale;
  uint16_t* out;
  int64_t ldo, hso;
};
size_t attention_workspace(int64_t tq, int64_t batch, int hq, int hk, int hd, int64_t max_kv_len);
hipError_t attention_launch(const AttnArgs& a, int64_t max_kv_len, void* ws, hipStream_t stream);

// Polls a bounded wait between workgroups may take before it gives up
// (environment GPTQ_SYNC_SPIN_LIMIT, default 2^20), read once per process.
int64_t sync_spin_limit();

// ---- two-sided rounding (anti-diagonal schedule) ----------------------------
size_t gptq2d_workspace(int64_t n);
hipError_t gptq2d_launch(const double* Y, const double* RL, const double* RR, int64_t n,
                         double* Z, void* ws, hipStream_t stream);

}  // namespace gptq
