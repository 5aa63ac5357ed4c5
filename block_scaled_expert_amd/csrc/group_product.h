// The grouped MXFP4 product on gfx950's scaled matrix cores: the pieces its
// kernels share.
//
//   out[r][n] = sum_k A[src(r)][k] W[g(r)][n][k]
//
// for rows r in [offsets[g], offsets[g+1]).  Both operands are E2M1 codes
// with an E8M0 scale per 32 of k; the scaled f8f6f4 instructions take the codes
// and the scales as they are stored and accumulate in fp32, so no operand is
// expanded.  What both kernels share is how the work is handed out (Item) and
// the views of memory; the tile kernel's instruction is in its own file.
//
// The streaming kernel uses v_mfma_scale_f32_16x16x128_f8f6f4.  Operand layout
// (checked on the device by the parity tests): lane l holds row l % 16 and one
// block of 32 k (16 bytes) in lane group l / 16, and one byte of its scale
// register applies to that block.
// Accumulator register q of lane l is out[4 (l / 16) + q][l % 16].
//
// The sum over k does not care which blocks meet in one instruction as long
// as both operands agree.  A chunk is kU instructions (128 kU of k) in which
// lane group b takes the kU consecutive blocks kU b .. kU b + kU - 1 of the
// chunk's 4 kU: a lane's codes are then 16 kU contiguous bytes, and its kU
// scales are one aligned load whose byte j the j-th instruction selects, with
// no arithmetic on scales at all.
#pragma once

#include "operators.h"

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
  // the wave's lanes agree on both; saying so keeps the view in scalar registers
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)a);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<uint8_t*>((uint64_t)hi << 32 | lo), 0,
                                           __builtin_amdgcn_readfirstlane((int)bytes), 0x00027000);
}
constexpr uint32_t kNowhere = 0x80000000u;   // an offset outside every view (views are below 2 GiB)

// NT: non-temporal, for bytes that are read once.
template <bool NT>
__device__ inline v4u buf16(Buf b, uint32_t off) {
  return __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(b, (int)off, 0, NT ? 2 : 0));
}

template <int J>
__device__ inline v4f mma4(const Frag& a, const Frag& b, v4f c) {
  const v8i av = v8i{(int)a.q[J].x, (int)a.q[J].y, (int)a.q[J].z, (int)a.q[J].w, 0, 0, 0, 0};
  const v8i bv = v8i{(int)b.q[J].x, (int)b.q[J].y, (int)b.q[J].z, (int)b.q[J].w, 0, 0, 0, 0};
  // 4, 4: both operands E2M1; J: the scale registers' byte
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, J, (int)a.sc, J, (int)b.sc);
}

// One chunk of 16 weight rows as loaded: lane (r, b) = (l % 16, l / 16) holds
// block 2 b + r / 8 of row r % 8 in q[0] and of row 8 + r % 8 in q[1]; sc is
// row r's own.
struct RawW {
  v4u q[2];
  uint16_t sc;
  uint8_t sc1;   // odd block counts: the second scale on its own
};

// Lanes r and r ^ 8 exchange what the other needs (a rotation by 8 within 16
// lanes, written to half of them): q[j] becomes block 2 b + j of row r.
template <bool ODD>
__device__ inline void operand_w(const RawW& w, Frag& f) {
  static_assert(kU == 2, "two loads, two halves");
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int x = (int)w.q[0][i], y = (int)w.q[1][i];
    f.q[0][i] = (uint32_t)__builtin_amdgcn_update_dpp(x, y, 0x128, 0xF, 0xC, false);   // row_ror:8 into lanes 8..15
    f.q[1][i] = (uint32_t)__builtin_amdgcn_update_dpp(y, x, 0x128, 0xF, 0x3, false);   // into lanes 0..7
  }
  f.sc = ODD ? (uint16_t)(w.sc | w.sc1 << 8) : w.sc;
}

// What a lane's loads of 16 weight rows start from: its piece of a line, its
// byte offsets among codes and scales.
struct WLane {
  int at, b, nb, row8;
  uint32_t off, soff;
  __device__ WLane(int r, int b_, int row_bytes, int nb_)
      : at(2 * b_ + (r >> 3)), b(b_), nb(nb_), row8(8 * row_bytes), off((r & 7) * row_bytes + 16 * (2 * b_ + (r >> 3))),
        soff(r * nb_ + kU * b_) {}
};

// Chunk c of the 16 rows whose codes and scales start `base` and `sbase` bytes
// into the views; nothing is loaded unless `on`.  ODD: rows of an odd number
// of scale blocks, whose last chunk ends inside a pair of scales (they are
// then loaded one by one).
template <bool ODD, bool NT>
__device__ inline void load_raw(RawW& W, Buf wq, Buf ws, const WLane& l, bool on, uint32_t base, uint32_t sbase, int c) {
  const int blk = kChunkBlocks * c;
  const uint32_t off = on && blk + l.at < l.nb ? l.off + base + 16 * blk : kNowhere;
  W.q[0] = buf16<NT>(wq, off);
  W.q[1] = buf16<NT>(wq, off + l.row8);
  const uint32_t so = l.soff + sbase + blk;
  const bool s0 = on && blk + kU * l.b < l.nb;
  if constexpr (ODD) {
    W.sc = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(ws, (int)(s0 ? so : kNowhere), 0, 0);
    W.sc1 = __builtin_amdgcn_raw_buffer_load_b8(ws, (int)(on && blk + kU * l.b + 1 < l.nb ? so + 1 : kNowhere), 0, 0);
  } else {
    W.sc = __builtin_amdgcn_raw_buffer_load_b16(ws, (int)(s0 ? so : kNowhere), 0, 0);
  }
}

// A workgroup's work: TM rows (a tile) of one group and one of the nx column
// slices.  The hardware hands workgroups to the 8 XCDs in turn, each with its
// own L2, so XCD x takes the x-th eighth of the items.  They are numbered
// group by group; in a group, up to kPanelTiles tiles of one slice follow each
// other, then come the next slices: what runs on an XCD side by side shares
// weight slices, and a panel's rows of A stay in its L2 for all slices.
// Every wave finds the item for itself, lane l counting the tiles of the PER
// groups PER l .. (PER * 64 >= G): one round of loads and a wave scan.
// Offsets are clamped to the M rows of the call whatever the device array
// holds.  False: there are fewer items.
struct Item {
  int g, row0, rows, bx;
};
constexpr int kPanelTiles = 8;
__device__ inline int clamped_offset(const ProductArgs& p, int i) { return min(max(p.offsets[i], 0), p.M); }
// hw: the workgroup's number.
template <int TM, int PER>
__device__ inline bool find_item_n(const ProductArgs& p, int nx, int hw, Item& it) {
  const int lane = threadIdx.x & 63, g0 = PER * lane;
  int at[PER + 1], n = 0;
#pragma unroll
  for (int i = 0; i <= PER; i++) at[i] = clamped_offset(p, min(g0 + i, p.G));
#pragma unroll
  for (int i = 0; i < PER; i++) n += (max(at[i + 1] - at[i], 0) + TM - 1) / TM;
  int end = n;                                  // inclusive scan over the lanes
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(end, o, kWave);
    end += lane >= o ? v : 0;
  }
  const int items = __builtin_amdgcn_readlane(end, 63) * nx;
  if (hw >= items) return false;
  const int xcd = hw % 8, L = xcd * (items / 8) + min(xcd, items % 8) + hw / 8;
  const int owner = __builtin_ctzll(__ballot(end > L / nx));
  int left = L - (end - n) * nx, g = 0, at0 = 0, len = 0, in = 0;   // meant for the owner's lane
#pragma unroll
  for (int i = 0; i < PER; i++) {
    const int l = max(at[i + 1] - at[i], 0), size = (l + TM - 1) / TM * nx;
    if (left >= 0 && left < size) {
      g = g0 + i;
      at0 = at[i];
      len = l;
      in = left;
    }
    left -= size;
  }
  it.g = __builtin_amdgcn_readlane(g, owner);
  at0 = __builtin_amdgcn_readlane(at0, owner);
  len = __builtin_amdgcn_readlane(len, owner);
  in = __builtin_amdgcn_readlane(in, owner);
  const int tiles = (len + TM - 1) / TM, panel = in / (kPanelTiles * nx), rest = in - panel * (kPanelTiles * nx);
  const int width = min(kPanelTiles, tiles - kPanelTiles * panel);
  it.bx = rest / width;
  const int tile = kPanelTiles * panel + rest - it.bx * width;
  it.row0 = at0 + tile * TM;
  it.rows = min(TM, len - tile * TM);
  return true;
}
template <int TM>
__device__ inline bool find_item(const ProductArgs& p, int nx, int hw, Item& it) {
  if (p.G <= 64) return find_item_n<TM, 1>(p, nx, hw, it);
  if (p.G <= 512) return find_item_n<TM, 8>(p, nx, hw, it);
  return find_item_n<TM, 16>(p, nx, hw, it);
}
// Upper bound of the tiles of a call.
inline int max_tiles(const ProductArgs& p, int tm) {
  const long n = p.G + (long)p.M / tm;
  return (int)(n < p.M ? n : p.M);
}

// Many rows per group (group_product_tile.hip).
int launch_product_tile(const ProductArgs& p, hipStream_t stream);

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
