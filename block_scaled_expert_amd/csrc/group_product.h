// The grouped MXFP4 product on gfx950's scaled matrix cores: the pieces its
// kernels share.
//
//   out[r][n] = sum_k A[src(r)][k] W[g(r)][n][k]
//
// for rows r in [offsets[g], offsets[g+1]).  Both operands are E2M1 codes
// with an E8M0 scale per 32 of k; v_mfma_scale_f32_16x16x128_f8f6f4 takes the
// codes and the scales as they are stored and accumulates in fp32, so no
// operand is expanded.  Operand layout (checked on the device by the parity
// tests): lane l holds row l % 16 and one block of 32 k (16 bytes) in lane
// group l / 16, and one byte of its scale register applies to that block.
// Accumulator register q of lane l is out[4 (l / 16) + q][l % 16].
//
// The sum over k does not care which blocks meet in one instruction as long
// as both operands agree.  A chunk is kU instructions (128 kU of k) in which
// lane group b takes the kU consecutive blocks kU b .. kU b + kU - 1 of the
// chunk's 4 kU: a lane's codes are then 16 kU contiguous bytes, and its kU
// scales are one aligned load whose byte j the j-th instruction selects, with
// no arithmetic on scales at all.
#pragma once

#include "moe_common.h"
#include "launch.h"

namespace moe {

constexpr int kU = 2;                // instructions per chunk
constexpr int kChunkK = 128 * kU;    // k of a chunk
constexpr int kChunkBlocks = 4 * kU; // scale blocks of a chunk

// One chunk of a 16-row operand.
struct Frag {
  v4u q[kU];
  uint16_t sc;   // as loaded: widening it here would wait for the load
};

// Buffer view of `bytes` bytes at a uniform address: loads outside it return
// zero and touch no memory, so ends of rows and tiles need no branches.
typedef __amdgpu_buffer_rsrc_t Buf;
__device__ inline Buf make_buf(const uint8_t* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, (int)bytes, 0x00027000);
}
constexpr uint32_t kNowhere = 0x80000000u;   // an offset outside every view (views are below 2 GiB)

__device__ inline v4u buf16(Buf b, uint32_t off) {
  return __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(b, (int)off, 0, 2));
}

template <int J>
__device__ inline v4f mma4(const Frag& a, const Frag& b, v4f c) {
  const v8i av = v8i{(int)a.q[J].x, (int)a.q[J].y, (int)a.q[J].z, (int)a.q[J].w, 0, 0, 0, 0};
  const v8i bv = v8i{(int)b.q[J].x, (int)b.q[J].y, (int)b.q[J].z, (int)b.q[J].w, 0, 0, 0, 0};
  // 4, 4: both operands E2M1; J: the scale registers' byte
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, J, (int)a.sc, J, (int)b.sc);
}

// Work items are (group, tile of TM rows) pairs in group order.  Finds item
// `item`: every wave of the workgroup works it out for itself, lane l counting
// the tiles of the PER groups PER l .. (PER * 64 >= G), so that it costs one
// round of loads and a wave scan.  Offsets are clamped to the M rows of the
// call whatever the device array holds.  False: there are fewer items.
struct Item {
  int g, row0, rows;
};
template <int TM, int PER>
__device__ inline bool find_item_n(const ProductArgs& p, int item, Item& it) {
  const int lane = threadIdx.x & 63, g0 = PER * lane;
  int at[PER + 1], n = 0;
#pragma unroll
  for (int i = 0; i <= PER; i++) at[i] = p.offsets[min(g0 + i, p.G)];
#pragma unroll
  for (int i = 0; i <= PER; i++) at[i] = min(max(at[i], 0), p.M);
#pragma unroll
  for (int i = 0; i < PER; i++) n += (max(at[i + 1] - at[i], 0) + TM - 1) / TM;
  int end = n;                                  // inclusive scan over the lanes
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(end, o, kWave);
    end += lane >= o ? v : 0;
  }
  const uint64_t past = __ballot(end > item);
  if (past == 0) return false;
  const int owner = __builtin_ctzll(past);
  int left = item - (end - n), g = 0, row0 = 0, rows = 0;   // of the owner's lane
#pragma unroll
  for (int i = 0; i < PER; i++) {
    const int len = max(at[i + 1] - at[i], 0), tiles = (len + TM - 1) / TM;
    if (left >= 0 && left < tiles) {
      g = g0 + i;
      row0 = at[i] + left * TM;
      rows = min(TM, len - left * TM);
    }
    left -= tiles;
  }
  it.g = __builtin_amdgcn_readlane(g, owner);
  it.row0 = __builtin_amdgcn_readlane(row0, owner);
  it.rows = __builtin_amdgcn_readlane(rows, owner);
  return true;
}
template <int TM>
__device__ inline bool find_item(const ProductArgs& p, int item, Item& it) {
  if (p.G <= 64) return find_item_n<TM, 1>(p, item, it);
  if (p.G <= 512) return find_item_n<TM, 8>(p, item, it);
  return find_item_n<TM, 16>(p, item, it);
}
// Upper bound of the items of a call.
template <int TM>
inline int max_items(const ProductArgs& p) {
  const long n = p.G + (long)p.M / TM;
  return (int)(n < p.M ? n : p.M);
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
