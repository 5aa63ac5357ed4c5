// Grouped MXFP4 product, many rows per group (prefill, expert-parallel shares,
// plain matrix products): the time is the matrix cores', if they can be fed.
//
// Work: one workgroup of MW x NW waves per (group, BM of its rows, BN weight
// rows); a wave owns 16 SM rows x 16 SN weight rows.  Both operands go through
// LDS.  The operand layout wants 16 bytes of each of 16 rows per instruction,
// and a load in that pattern costs the vector cache one access per lane: 17
// bytes per clock and CU measured, against 62 where each 4 lanes share a
// 64-byte piece.  So the loads take a half step (k 128, 64 bytes) of 16 rows per
// wave, row after row, and the rearrangement is left to LDS, whose 16-byte
// columns are permuted by row so that both sides are free of bank conflicts.
//
// Pipeline, in half steps h: loads of h + 4 go to registers (ring of 2), h + 2
// goes from there to LDS (4 slots), h is multiplied; one barrier every two.
// Scales: 16 bytes (4 half steps) of a row per load, double-buffered, turned
// so that a lane's 4 bytes are one word whose byte the instruction selects.
//
// The weights are the instruction's first operand and the rows of A its
// second, so a lane's 4 accumulator registers are 4 consecutive columns of one
// row of out, stored together.
#include "group_product.h"

#include <type_traits>

namespace moe {

namespace {

constexpr int kHalf = 4;                 // blocks of a half step

// 16-byte column of LDS that holds block b of row `row` (rows of 64 bytes): 16
// rows of one block fall on 16 different columns of the 256-byte bank line.
__device__ inline int column(int row, int b) { return b ^ ((row >> 2) & 3); }

template <int MW, int NW, int SM, int SN>
struct Tile {
  static constexpr int sm = SM, sn = SN, nw = NW;
  static constexpr int BM = 16 * SM * MW, BN = 16 * SN * NW, T = 64 * MW * NW;
  static constexpr int PA = BM * 4 / T, PW = BN * 4 / T;   // 16-byte pieces a thread loads per half step
  static constexpr int kSlot = (BM + BN) * 64, kScale = (BM + BN) * 16;
  static constexpr int kLds = 4 * kSlot + 2 * kScale;
  static_assert(PA * T == BM * 4 && PW * T == BN * 4 && T >= BM + BN, "every thread has whole pieces");
};

}  // namespace

// 4 x 4 bytes transposed: word b of the result holds byte b of every word.
__device__ inline v4u transpose_bytes(v4u v) {
  const uint32_t t0 = __builtin_amdgcn_perm(v[1], v[0], 0x05010400), t1 = __builtin_amdgcn_perm(v[1], v[0], 0x07030602);
  const uint32_t u0 = __builtin_amdgcn_perm(v[3], v[2], 0x05010400), u1 = __builtin_amdgcn_perm(v[3], v[2], 0x07030602);
  return v4u{__builtin_amdgcn_perm(u0, t0, 0x05040100), __builtin_amdgcn_perm(u0, t0, 0x07060302),
             __builtin_amdgcn_perm(u1, t1, 0x05040100), __builtin_amdgcn_perm(u1, t1, 0x07060302)};
}

// The tile's work of one wave whose rows fill NSUB of its SM sub-tiles.  Waves
// of a workgroup may run different NSUB: the barriers are the same in all.
template <typename C, int NSUB>
__device__ __forceinline__ void product_tile(const ProductArgs& p, const Item& it, uint8_t* lds, const int* src,
                                             int wave) {
  constexpr int SM = C::sm, SN = C::sn;
  const int tid = threadIdx.x, lane = tid & 63;
  const int nb = p.K / 32, halves = (nb + kHalf - 1) / kHalf, row_bytes = p.K / 2;
  const int n0 = it.bx * C::BN, wrows = min(C::BN, p.N - n0);
  const size_t wr0 = (size_t)it.g * p.N + n0;
  const Buf wq = make_buf(p.w + wr0 * row_bytes, wrows * row_bytes);         // rows past N read zeros

  // loading: thread t takes piece t % 4 of rows t / 4 + i T / 4; rows of A past
  // the tile repeat its first row (their outputs are not stored)
  const int lrow = tid >> 2, lb = tid & 3;
  const uint8_t* aq[C::PA];
#pragma unroll
  for (int i = 0; i < C::PA; i++) aq[i] = p.a + (size_t)max(src[lrow + i * (C::T / 4)], 0) * row_bytes;
  const uint32_t woff = lrow * row_bytes;
  struct Stage {
    v4u a[C::PA], w[C::PW];
  };
  auto load = [&](int h, Stage& s) {
    const int blk = kHalf * h + lb;
    const size_t ao = 16 * (size_t)min(blk, nb - 1);     // past the end of k: any codes, the weights are zero there
    const uint32_t wo = blk < nb ? woff + 16 * blk : kNowhere;
#pragma unroll
    for (int i = 0; i < C::PA; i++) s.a[i] = *reinterpret_cast<const v4u*>(aq[i] + ao);
#pragma unroll
    for (int i = 0; i < C::PW; i++) s.w[i] = buf16<false>(wq, wo + i * (C::T / 4) * row_bytes);
  };
  auto store = [&](int slot, const Stage& s) {
    uint8_t* t = lds + slot * C::kSlot;
#pragma unroll
    for (int i = 0; i < C::PA + C::PW; i++) {
      const int row = lrow + i * (C::T / 4);
      *reinterpret_cast<v4u*>(t + row * 64 + 16 * column(row, lb)) = i < C::PA ? s.a[i] : s.w[i - C::PA];
    }
  };
  // scales: thread t < BM + BN takes row t (of A, then of W), 16 blocks at a time; past the end of k zeros
  const uint8_t* scr = p.a_sc;
  if (tid < C::BM) scr = p.a_sc + (size_t)max(src[tid], 0) * nb;
  else if (tid < C::BM + C::BN) scr = p.w_sc + (wr0 + min(tid - C::BM, wrows - 1)) * nb;
  auto load_scales = [&](int q) {
    v4u v = v4u{0, 0, 0, 0};
    const int b0 = 16 * q, left = nb - b0;
    if (left >= 16) {
      __builtin_memcpy(&v, scr + b0, 16);
    } else {
      for (int j = 0; j < left; j++) v[j >> 2] |= (uint32_t)scr[b0 + j] << (8 * (j & 3));
    }
    return v;
  };
  uint8_t* const sc_lds = lds + 4 * C::kSlot;
  auto store_scales = [&](int buf, v4u v) {
    if (tid < C::BM + C::BN) *reinterpret_cast<v4u*>(sc_lds + buf * C::kScale + 16 * tid) = transpose_bytes(v);
  };

  // multiplying: this wave's rows and columns
  const int wm = wave / C::nw, wn = wave % C::nw, r = lane & 15, b = lane >> 4;
  const int nw = n0 + 16 * SN * wn;
  const int arow = 16 * SM * wm + r, brow = C::BM + 16 * SN * wn + r;   // (a sub-tile is 16 rows: the same columns)
  const int aoff = arow * 64 + 16 * column(r, b), boff = brow * 64 + 16 * column(r, b);
  const int asc = arow * 16 + 4 * b, bsc = brow * 16 + 4 * b;

  v4f acc[NSUB > 0 ? NSUB : 1][SN];
#pragma unroll
  for (int i = 0; i < NSUB; i++)
#pragma unroll
    for (int c = 0; c < SN; c++) acc[i][c] = v4f{0, 0, 0, 0};

  int wsc[SN], asv[NSUB > 0 ? NSUB : 1];                 // scale words of a pass
  auto compute = [&](auto J) {                           // half step J of a pass, slot J
    constexpr int j = decltype(J)::value;
    const uint8_t* t = lds + j * C::kSlot;
    v4u w[SN];
#pragma unroll
    for (int c = 0; c < SN; c++) w[c] = *reinterpret_cast<const v4u*>(t + boff + 1024 * c);
#pragma unroll
    for (int i = 0; i < NSUB; i++) {
      const v4u a = *reinterpret_cast<const v4u*>(t + aoff + 1024 * i);
#pragma unroll
      for (int c = 0; c < SN; c++) acc[i][c] = mma_codes<j>(w[c], wsc[c], a, asv[i], acc[i][c]);
    }
  };

  Stage st[2];
  load(0, st[0]);
  load(1, st[1]);
  v4u sc = load_scales(0);
  store(0, st[0]);
  load(2, st[0]);
  store(1, st[1]);
  load(3, st[1]);
  store_scales(0, sc);
  lds_barrier();
  // h: 4 half steps per pass, slot and scale byte group h % 4, register set h % 2
  for (int h0 = 0, sb = 0; h0 < halves; h0 += 4, sb ^= 1) {
    sc = load_scales(h0 / 4 + 1);
    if constexpr (NSUB > 0) {
      const uint8_t* s = sc_lds + sb * C::kScale;
#pragma unroll
      for (int c = 0; c < SN; c++) wsc[c] = *reinterpret_cast<const int*>(s + bsc + 256 * c);
#pragma unroll
      for (int i = 0; i < NSUB; i++) asv[i] = *reinterpret_cast<const int*>(s + asc + 256 * i);
    }
    auto half_step = [&](auto J) {
      constexpr int j = decltype(J)::value;
      if constexpr (NSUB > 0) {
        if (h0 + j < halves) compute(J);
      }
      store((j + 2) & 3, st[j & 1]);                     // half step h0 + j + 2
      load(h0 + j + 4, st[j & 1]);
      if constexpr (j == 1) lds_barrier();
      if constexpr (j == 3) {
        store_scales(sb ^ 1, sc);
        lds_barrier();
      }
    };
    half_step(std::integral_constant<int, 0>{});
    half_step(std::integral_constant<int, 1>{});
    half_step(std::integral_constant<int, 2>{});
    half_step(std::integral_constant<int, 3>{});
  }

  // register q of lane (r, b), tile (i, c): row 16 i + r of the wave's, column 16 c + 4 b + q
  const bool wide = p.N % 4 == 0;
#pragma unroll
  for (int i = 0; i < NSUB; i++) {
    const int m = 16 * SM * wm + 16 * i + r;
    if (m >= it.rows) continue;
    const bool zero = src[m] < 0;
#pragma unroll
    for (int c = 0; c < SN; c++) {
      const int n = nw + 16 * c + 4 * b;
      const v4f v = zero ? v4f{0, 0, 0, 0} : acc[i][c];
      const size_t at = (size_t)(it.row0 + m) * p.N + n;
      if (wide) {
        if (n < p.N) store_out4(p, at, v);
      } else {
#pragma unroll
        for (int q = 0; q < 4; q++)
          if (n + q < p.N) store_out(p, at + q, v[q]);
      }
    }
  }
}

template <int MW, int NW, int SM, int SN>
__global__ __launch_bounds__(64 * MW * NW, 2) void k_product_tile(ProductArgs p) {
  typedef Tile<MW, NW, SM, SN> C;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  int* const src = reinterpret_cast<int*>(lds + C::kLds);                    // [BM]
  Item it;
  if (!find_item<C::BM>(p, (p.N + C::BN - 1) / C::BN, it)) return;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  if (tid < C::BM) src[tid] = tid < it.rows ? source_row(p, it.row0 + tid) : -1;
  __syncthreads();
  // bodies for fewer rows (a group's last tile is usually partial) leave out
  // the reads and instructions of sub-tiles without rows
  const int wm = wave / NW, nw = it.bx * C::BN + 16 * SN * (wave % NW);
  const int rows = nw < p.N ? it.rows - 16 * SM * wm : 0;
  if (rows <= 0) product_tile<C, 0>(p, it, lds, src, wave);
  else if (rows <= 4 * SM) product_tile<C, SM / 4>(p, it, lds, src, wave);
  else if (rows <= 8 * SM) product_tile<C, SM / 2>(p, it, lds, src, wave);
  else if (rows <= 12 * SM) product_tile<C, 3 * SM / 4>(p, it, lds, src, wave);
  else product_tile<C, SM>(p, it, lds, src, wave);
}

template <int MW, int NW, int SM, int SN>
static void launch_tile(const ProductArgs& p, hipStream_t stream) {
  typedef Tile<MW, NW, SM, SN> C;
  const dim3 grid((unsigned)max_tiles(p, C::BM) * ceil_div(p.N, C::BN));
  hipLaunchKernelGGL((k_product_tile<MW, NW, SM, SN>), grid, dim3(C::T), C::kLds + 4 * C::BM, stream, p);
}

int launch_product_tile(const ProductArgs& p, hipStream_t stream) {
  // the large tile where it still gives most CUs (256) a workgroup
  const long tiles = ceil_div(p.M, 256) > p.G ? ceil_div(p.M, 256) : p.G;
  if (tiles * ceil_div(p.N, 256) >= 192) launch_tile<2, 4, 8, 4>(p, stream);
  else launch_tile<2, 2, 4, 2>(p, stream);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace moe
