// Launchers of the MXFP4 format (4 in launch_quant, launch_encode_weights and
// launch_decode_weights), the grouped products, the router's balance loss, the
// residual norm and the sorted rows.
// Apart from launch.h, whose text the recorded traffic of the older kernels is
// tied to.
#pragma once

#include "launch.h"
#include "moe_common.h"

namespace moe {

// Shared exponent of an MXFP4 block (E2M1 elements, emax 2) from its maximum.  An infinite maximum
// gives exponent 126, so 2^-E is a normal fp32 number.
__host__ __device__ inline int mxfp4_exponent(float amax) {
  const int e = (int)((f_bits(amax) >> 23) & 0xFFu) - 127 - 2;
  return e < -127 ? -127 : e;
}

// MXFP4 (mxfp4.hip): n elements (a multiple of 32) encoded and decoded, and
// rows [g | u] of the fp32 gate/up product through the capped SwiGLU to MXFP4
// rows of F columns.  rows_dev: device row count that further limits `rows`.
// launch_quant takes none with this format: the layer's h, whose row count is
// on the device, is encoded by launch_swiglu_mxfp4.
int launch_mxfp4_encode(int dtype, const void* x, long n, uint8_t* codes, uint8_t* scales, hipStream_t stream);
int launch_mxfp4_decode(const uint8_t* codes, const uint8_t* scales, long n, float* out, hipStream_t stream);
int launch_swiglu_mxfp4(const float* gu, int rows, const int* rows_dev, int F, int form, float cap, uint8_t* codes,
                        uint8_t* scales, hipStream_t stream);

// Grouped MXFP4 product (group_product.hip).
struct ProductArgs {
  const uint8_t* a;         // [a_rows][K/2] codes, [a_rows][K/32] scales
  const uint8_t* a_sc;
  int a_rows;
  const int32_t* row_ids;   // nullable: row r reads A row row_ids[r] / id_div
  int id_div;
  int M;                    // rows of out
  int expect;               // rows that the groups are expected to hold, at most M: what the kernel is chosen by
  const uint8_t* w;         // [G][N][K/2], [G][N][K/32]
  const uint8_t* w_sc;
  int G, N, K;
  const int32_t* offsets;   // [G+1]
  void* out;                // [M][N]
  int out_f32;
};
int launch_group_product(const ProductArgs& p, hipStream_t stream);

// Router balance loss (balance.hip).  z: dtype 0 bf16, 1 fp32.
struct BalanceArgs {
  const void* z;            // [T][E] logits
  int dtype, T, E, k;
  const int32_t* ids;       // [T][k]
  const int32_t* bounds;    // [S+1] first token of each sequence; null: one sequence of T
  int S;
  const uint8_t* mask;      // [T] nullable: 0 = not a token
  int32_t* counts;          // [S][E]
  int32_t* live;            // [S]
  // forward
  float* probs;             // [S][E]
  float* loss;              // [S]
  void* ws;
  // backward
  const float* d_loss;      // [S]
  const float* d_w;         // [T][k] nullable
  int norm_topk;
  float routed_scale;
  void* dz;                 // [T][E], z's type
};
size_t balance_ws_bytes(int T, int E, int S);
int launch_balance_forward(const BalanceArgs& a, hipStream_t stream);
int launch_balance_backward(const BalanceArgs& a, hipStream_t stream);

// Residual norm (norm.hip).  dtype of x, y, dy, dx; res_dtype of the stream
// (0 bf16, 1 fp32; a bf16 stream only under bf16 x).
struct NormArgs {
  const void* x;            // [T][cols]
  const void* res;          // [T][cols] nullable
  int dtype, res_dtype, T, cols;
  double inv_cols;          // 1 / cols, set by the launcher
  const float* weight;      // [cols]
  float eps;
  void* res_out;            // [T][cols] nullable
  void* y;                  // [T][cols] nullable
  float* rstd;              // [T] nullable
  int fmt;                  // 0, or the format of the codes
  uint8_t* codes;
  uint8_t* scales;
  float* row_gs;            // NVFP4
  int gs_row;               // NVFP4: 1 the row's own scale, 0 gs_val
  float gs_val;
};
struct NormGradArgs {
  const void* dy;           // [T][cols]
  const void* res;          // the stream that was normed
  const void* d_res_out;    // nullable
  int dtype, res_dtype, T, cols;
  const float* weight;
  const float* rstd;
  void* d_res;
  void* dx;                 // nullable
  float* partial;           // [workgroups][pitch], set by the launcher
  int pitch;
};
size_t norm_ws_bytes(int T, int cols);
int launch_norm_forward(NormArgs a, hipStream_t stream);
int launch_norm_backward(NormGradArgs a, float* d_weight, void* ws, hipStream_t stream);

// Tokens sorted by expert and back (rows.hip).
struct RowsArgs {
  int T, k, cols, M;
  const int32_t* pos;       // [T][k]
  const float* w;           // [T][k] nullable: all 1
  int token_dtype, row_dtype;
  const void* token;        // [T][cols]
  const void* rows_in;      // [M][cols]
  void* token_out;
  void* rows_out;
  float* d_w;               // [T][k]
};
int launch_sort_rows(const RowsArgs& a, hipStream_t stream);
int launch_combine_rows(const RowsArgs& a, hipStream_t stream);
int launch_combine_rows_backward(const RowsArgs& a, hipStream_t stream);

// Rows in bf16 or fp32 times 4-bit matrices (matvec.hip).
struct MatvecArgs {
  ProductArgs p;            // a: rows of dtype; a_sc unused; N rows of [gate | up] with swiglu
  int fmt, dtype;           // fmt 1 NVFP4, 4 MXFP4; dtype 0 bf16, 1 fp32
  const float* gs;          // NVFP4: matrix m of group g at gs[g gs_stride + m]
  int gs_group, gs_stride;  // matrices of N / gs_group rows in a group
  int swiglu;               // out [M][N / 2]
  int cap_form;
  float cap;
};
int launch_group_matvec(const MatvecArgs& a, hipStream_t stream);

// The S split-K planes of router logits added in split order, as the top-k
// adds them: z [T][E].
int launch_router_logits_sum(const float* zpart, int T, int E, float* z, hipStream_t stream);

}  // namespace moe
