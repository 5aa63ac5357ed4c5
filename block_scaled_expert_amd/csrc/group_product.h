// The grouped MXFP4 product on gfx950's scaled matrix cores: arguments and
// the pieces its kernels share.
//
//   out[r][n] = sum_k A[src(r)][k] W[g(r)][n][k]
//
// for rows r in [offsets[g], offsets[g+1]).  Both operands are E2M1 codes
// with an E8M0 scale per 32 of k; v_mfma_scale_f32_16x16x128_f8f6f4 takes the
// codes and the scales as they are stored and accumulates in fp32, so no
// operand is expanded.  Operand layout (checked on the device by the parity
// tests): lane l holds row l % 16 and the 32 consecutive k of block l / 16 (16
// bytes), and its scale byte applies to that block.  Accumulator register q
// of lane l is out[4 (l / 16) + q][l % 16].
#pragma once

#include "moe_common.h"
#include "launch.h"

namespace moe {

// 128 of k: codes of one 16-row operand and its scale (low byte).
struct Frag {
  v4u q;
  uint32_t sc;
};

__device__ inline v4f mma4(const Frag& a, const Frag& b, v4f c) {
  const v8i av = v8i{(int)a.q.x, (int)a.q.y, (int)a.q.z, (int)a.q.w, 0, 0, 0, 0};
  const v8i bv = v8i{(int)b.q.x, (int)b.q.y, (int)b.q.z, (int)b.q.w, 0, 0, 0, 0};
  // 4, 4: both operands E2M1
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, 0, (int)a.sc, 0, (int)b.sc);
}

// Rows [lo, hi) of group g, clamped to the M rows of the call whatever the
// device-side offsets hold.
__device__ inline void group_rows(const ProductArgs& p, int g, int& lo, int& hi) {
  lo = min(max(p.offsets[g], 0), p.M);
  hi = min(max(p.offsets[g + 1], lo), p.M);
}

// Source row of row r, -1 for a row id outside A (its output is zero).
__device__ inline int source_row(const ProductArgs& p, int r) {
  if (p.row_ids == nullptr) return r < p.a_rows ? r : -1;
  const int id = p.row_ids[r];
  const int s = id / p.id_div;
  return id >= 0 && s < p.a_rows ? s : -1;
}

__device__ inline void store_out(const ProductArgs& p, size_t i, float v) {
  if (p.out_f32) static_cast<float*>(p.out)[i] = v;
  else static_cast<__bf16*>(p.out)[i] = (__bf16)v;   // to nearest even; inf and NaN kept
}

}  // namespace moe
