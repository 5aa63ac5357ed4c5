// Grouped MXFP4 product, many rows per group (prefill, expert-parallel shares,
// plain matrix products): the time is the matrix cores', if they can be fed.
//
// Work: one workgroup of MW x NW waves per (group, BM of its rows, BN weight
// rows); a wave owns 32 SM rows x 32 SN weight rows on
// v_mfma_scale_f32_32x32x64_f8f6f4 (measured from registers: 9.4 PFLOP/s; the
// 16x16x128 form of the same product 4.1 to 5.4).  Both operands go through
// LDS.  The operand layout wants 16 bytes of each of 32 rows per instruction,
// and a load in that pattern costs the vector cache one access per lane: 17
// bytes per clock and CU measured, against 47 to 62 where each 4 lanes share a
// 64-byte piece.  So the loads take a half step (k 128, 64 bytes) of 16 rows per
// wave, row after row, and LDS does the rearrangement.
//
// Pipeline, in half steps h: after h's products the loads of h + 2 go out,
// straight to LDS (3 slots), and arrive while h + 1 is multiplied; one barrier a
// half step, passed with the youngest half step's loads still on their way.  Scales: 16 bytes (4 half steps, a pass) of a row
// per load, through registers, turned so that a lane's 8 bytes are two words
// whose bytes the instructions select.  The large tile is 4 waves of 128 x 64
// (199 registers, 78 KiB of LDS), so that two workgroups share a CU and one
// multiplies while the other starts, ends or waits.
//
// Measured (48 groups, 16384 rows x 4608 x 4608): bf16 out 292 us, 2.4
// PFLOP/s; fp32 out, what the layer's gate/up takes, 309; bf16 with the operands going to LDS through registers 307; 256 x 256
// tiles of 8 waves 293, 128 x 128 of 4 335; with the weights brought to operand
// order in registers instead of through LDS 310.  No unit is near its rate.
// Without the loads it takes 184, with loads that all hit a cache 251, without
// the products 274, without the outputs 269, without the scales 278: the parts
// of a half step overlap little, and two workgroups a CU, all that registers
// and LDS hold, do not fill the gaps.
//
// The rows of A are the instruction's first operand and the weights its second,
// so 32 lanes of a store hold consecutive columns of one row of out: 2 cache
// accesses an instruction, where 4 columns a lane (the other order) took 64.
#include "group_product.h"

#include <type_traits>

namespace moe {

namespace {

constexpr int kHalf = 4;                 // blocks of a half step

// 16-byte column of LDS that holds block b of row `row` (rows of 64 bytes): the
// operand's 32 rows read at 110 bytes per clock this way, at 67 in plain order.
__device__ inline int column(int row, int b) { return b ^ ((row >> 2) & 3); }

typedef __attribute__((address_space(3))) uint8_t Lds;
typedef __attribute__((address_space(1))) uint8_t Glb;

// A barrier after which all but the N youngest loads of every wave have arrived.
template <int N>
__device__ inline void loads_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | (N >> 4) << 14);   // vmcnt(N) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

typedef float v16f __attribute__((ext_vector_type(16)));
typedef unsigned v2u __attribute__((ext_vector_type(2)));

// 32 x 32 x 64: lane l holds row l % 32 and block l / 32 of the two; J: the scale words' byte.
// Register q of lane l is out[8 (q / 4) + 4 (l / 32) + q % 4][l % 32].
template <int J>
__device__ inline v16f mma32(v4u a, uint32_t asc, v4u b, uint32_t bsc, v16f c) {
  const v8i av = v8i{(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const v8i bv = v8i{(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, J, (int)asc, J, (int)bsc);
}

template <int MW, int NW, int SM, int SN>
struct Tile {
  static constexpr int sm = SM, sn = SN, nw = NW;
  static constexpr int BM = 32 * SM * MW, BN = 32 * SN * NW, T = 64 * MW * NW;
  static constexpr int PA = BM * 4 / T, PW = BN * 4 / T;   // 16-byte pieces a thread loads per half step
  static constexpr int kSlot = (BM + BN) * 64, kScale = (BM + BN) * 16;
  static constexpr int kLds = 3 * kSlot + kScale;
  static constexpr int R = (BM + BN + T - 1) / T;                            // scale rows it loads per pass
  static_assert(PA * T == BM * 4 && PW * T == BN * 4 && T >= BM, "every thread has whole pieces");
};

}  // namespace

// The 16 scale bytes of a pass: even blocks, then odd ones.
__device__ inline v4u split_scales(v4u v) {
  return v4u{__builtin_amdgcn_perm(v[1], v[0], 0x06040200), __builtin_amdgcn_perm(v[3], v[2], 0x06040200),
             __builtin_amdgcn_perm(v[1], v[0], 0x07050301), __builtin_amdgcn_perm(v[3], v[2], 0x07050301)};
}

// The wave's outputs.  Register 4 k + q of lane (r, b), tile (i, c): row 32 i + 8
// k + 4 b + q of the wave's, column 32 c + r.  Offsets are relative to the
// item's first row; the view ends with its last one, so rows past it are dropped.
template <typename C, bool F32, int NSUB, int NS>
__device__ __forceinline__ void store_tile(const ProductArgs& p, const Item& it, const int* src, int wave,
                                           v16f (&acc)[NS][C::sn]) {
  constexpr int kEl = F32 ? 4 : 2;
  const int lane = threadIdx.x & 63, r = lane & 31, b = lane >> 5;
  const int n = it.bx * C::BN + 32 * C::sn * (wave % C::nw) + r, m0 = 32 * C::sm * (wave / C::nw) + 4 * b;
  const Buf out = make_buf(static_cast<const uint8_t*>(p.out) + (size_t)it.row0 * p.N * kEl, (uint32_t)it.rows * p.N * kEl);
  uint32_t at[C::sn];
#pragma unroll
  for (int c = 0; c < C::sn; c++) at[c] = n + 32 * c < p.N ? ((uint32_t)m0 * p.N + n + 32 * c) * kEl : kNowhere;
  // whether a row of the wave's has its source outside A (its output is zero)
  bool bad = false;
#pragma unroll
  for (int i = 0; i < NSUB; i++) {
    const int m = m0 - 4 * b + 32 * i + r;
    bad |= m < it.rows && src[m] < 0;
  }
  bad = __any(bad);
#pragma unroll
  for (int i = 0; i < NSUB; i++)
#pragma unroll
    for (int q = 0; q < 16; q++) {
      const int dm = 32 * i + 8 * (q / 4) + q % 4;
      const uint32_t row = (uint32_t)dm * p.N * kEl;   // below 2^29, so an offset from kNowhere stays outside
      bool zero = false;
      if (bad) zero = m0 + dm < it.rows && src[m0 + dm] < 0;
#pragma unroll
      for (int c = 0; c < C::sn; c++) {
        const float v = zero ? 0.0f : acc[i][c][q];
        if constexpr (F32) __builtin_amdgcn_raw_buffer_store_b32(f_bits(v), out, (int)(at[c] + row), 0, 0);
        else __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (__bf16)v), out, (int)(at[c] + row), 0, 0);
      }
      __builtin_amdgcn_sched_barrier(0);   // one row at a time: the accumulators leave no registers for more
    }
}

// The tile's work of one wave whose rows fill NSUB of its SM sub-tiles.  Waves
// of a workgroup may run different NSUB: the barriers are the same in all.
template <typename C, bool F32, int NSUB>
__device__ __forceinline__ void product_tile(const ProductArgs& p, const Item& it, uint8_t* lds, const int* src,
                                             int wave) {
  constexpr int SM = C::sm, SN = C::sn;
  const int tid = threadIdx.x, lane = tid & 63;
  const int nb = p.K / 32, halves = (nb + kHalf - 1) / kHalf, row_bytes = p.K / 2;
  const int n0 = it.bx * C::BN, wrows = min(C::BN, p.N - n0);
  const size_t wr0 = (size_t)it.g * p.N + n0;
  const Buf wq = make_buf(p.w + wr0 * row_bytes, wrows * row_bytes);         // rows past N read zeros

  // loading, straight to LDS: a wave's load fills 1 KiB, 16 rows of 64 bytes, so
  // the lane's place says which block it takes.  Rows of A past the tile repeat
  // its first row (their outputs are not stored)
  const int lrow = tid >> 2, lb = column(tid >> 2, tid & 3);
  const uint8_t* aq[C::PA];
#pragma unroll
  for (int i = 0; i < C::PA; i++) aq[i] = p.a + (size_t)max(src[lrow + i * (C::T / 4)], 0) * row_bytes;
  const uint32_t woff = lrow * row_bytes;
  auto load = [&](int h, int slot) {
    const int blk = kHalf * h + lb;
    const size_t ao = 16 * (size_t)min(blk, nb - 1);     // past the end of k: any codes, the weights are zero there
    const uint32_t wo = blk < nb ? woff + 16 * blk : kNowhere;
    Lds* const dst = (Lds*)(lds + slot + wave * 1024);
#pragma unroll
    for (int i = 0; i < C::PA; i++) __builtin_amdgcn_global_load_lds((const Glb*)(aq[i] + ao), dst + i * C::T * 16, 16, 0, 0);
#pragma unroll
    for (int i = 0; i < C::PW; i++)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(wq, dst + (C::PA + i) * C::T * 16, 16,
                                               (int)(wo + i * (C::T / 4) * row_bytes), 0, 0, 0);
  };
  // scales: thread t takes rows t, t + T .. (of A, then of W), 16 blocks at a time; past the end of k zeros
  const uint8_t* scr[C::R];
#pragma unroll
  for (int i = 0; i < C::R; i++) {
    const int row = tid + i * C::T;
    scr[i] = row < C::BM ? p.a_sc + (size_t)max(src[row], 0) * nb
                         : p.w_sc + (wr0 + min(row - C::BM, wrows - 1)) * nb;
  }
  struct Scales {
    v4u v[C::R];
  };
  auto load_scales = [&](int q, Scales& s) {
    const int b0 = 16 * q, left = nb - b0;
    if (left >= 16) {
#pragma unroll
      for (int i = 0; i < C::R; i++) __builtin_memcpy(&s.v[i], scr[i] + b0, 16);
    } else {
#pragma unroll
      for (int i = 0; i < C::R; i++) {
        s.v[i] = v4u{0, 0, 0, 0};
        for (int j = 0; j < left; j++) s.v[i][j >> 2] |= (uint32_t)scr[i][b0 + j] << (8 * (j & 3));
      }
    }
  };
  uint8_t* const sc_lds = lds + 3 * C::kSlot;
  auto store_scales = [&](const Scales& s) {
#pragma unroll
    for (int i = 0; i < C::R; i++)
      if (tid + i * C::T < C::BM + C::BN) *reinterpret_cast<v4u*>(sc_lds + 16 * (tid + i * C::T)) = split_scales(s.v[i]);
  };

  // multiplying: this wave's rows and columns
  const int wm = wave / C::nw, wn = wave % C::nw, r = lane & 31, b = lane >> 5;
  const int nw = n0 + 32 * SN * wn;
  const int arow = 32 * SM * wm + r, brow = C::BM + 32 * SN * wn + r;
  const int aoff[2] = {arow * 64 + 16 * column(r, b), arow * 64 + 16 * column(r, 2 + b)};
  const int boff[2] = {brow * 64 + 16 * column(r, b), brow * 64 + 16 * column(r, 2 + b)};
  const int asc = arow * 16 + 8 * b, bsc = brow * 16 + 8 * b;

  v16f acc[NSUB > 0 ? NSUB : 1][SN];
#pragma unroll
  for (int i = 0; i < NSUB; i++)
#pragma unroll
    for (int c = 0; c < SN; c++)
#pragma unroll
      for (int q = 0; q < 16; q++) acc[i][c][q] = 0.0f;

  v2u wsc[SN], asv[NSUB > 0 ? NSUB : 1];                 // scale words of a pass
  auto compute = [&](auto J, const uint8_t* t) {         // half step J of a pass, in slot t
    constexpr int j = decltype(J)::value;
#pragma unroll
    for (int u = 0; u < 2; u++) {
      v4u w[SN];
#pragma unroll
      for (int c = 0; c < SN; c++) w[c] = *reinterpret_cast<const v4u*>(t + boff[u] + 2048 * c);
#pragma unroll
      for (int i = 0; i < NSUB; i++) {
        const v4u a = *reinterpret_cast<const v4u*>(t + aoff[u] + 2048 * i);
#pragma unroll
        for (int c = 0; c < SN; c++) {
          if (u == 0) acc[i][c] = mma32<2 * (j & 1)>(a, asv[i][j / 2], w[c], wsc[c][j / 2], acc[i][c]);
          else acc[i][c] = mma32<2 * (j & 1) + 1>(a, asv[i][j / 2], w[c], wsc[c][j / 2], acc[i][c]);
        }
      }
    }
  };

  Scales sc;
  load_scales(0, sc);
  load(0, 0);
  store_scales(sc);
  load(1, C::kSlot);
  loads_barrier<C::PA + C::PW>();
  int slot = 0, free_slot = 2 * C::kSlot;                // of half steps h and h + 2
  auto next_slot = [&](int s) { return s == 2 * C::kSlot ? 0 : s + C::kSlot; };
  // 4 half steps per pass: scale bytes by h % 4
  for (int h0 = 0; h0 < halves; h0 += 4) {
    if constexpr (NSUB > 0) {
#pragma unroll
      for (int c = 0; c < SN; c++) wsc[c] = *reinterpret_cast<const v2u*>(sc_lds + bsc + 512 * c);
#pragma unroll
      for (int i = 0; i < NSUB; i++) asv[i] = *reinterpret_cast<const v2u*>(sc_lds + asc + 512 * i);
    }
    auto half_step = [&](auto J) {
      constexpr int j = decltype(J)::value;
      if constexpr (j == 0) load_scales(h0 / 4 + 1, sc);
      if constexpr (j == 3) store_scales(sc);            // read at the start of the pass
      if constexpr (NSUB > 0) {
        if (h0 + j < halves) compute(J, lds + slot);
      }
      load(h0 + j + 2, free_slot);
      loads_barrier<C::PA + C::PW>();                     // half step h0 + j + 1 is in LDS
      slot = next_slot(slot);
      free_slot = next_slot(free_slot);
    };
    half_step(std::integral_constant<int, 0>{});
    half_step(std::integral_constant<int, 1>{});
    half_step(std::integral_constant<int, 2>{});
    half_step(std::integral_constant<int, 3>{});
  }
  loads_barrier<0>();                                      // none may still be on its way when the LDS is given up
  store_tile<C, F32, NSUB>(p, it, src, wave, acc);
}

template <int MW, int NW, int SM, int SN, bool F32>
__global__ __launch_bounds__(64 * MW * NW, SM * SN > 4 ? 2 : 4) void k_product_tile(ProductArgs p) {
  typedef Tile<MW, NW, SM, SN> C;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  int* const src = reinterpret_cast<int*>(lds + C::kLds);                    // [BM]
  Item it;
  if (!find_item<C::BM>(p, (p.N + C::BN - 1) / C::BN, blockIdx.x, it)) return;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  if (tid < C::BM) src[tid] = tid < it.rows ? source_row(p, it.row0 + tid) : -1;
  __syncthreads();
  // bodies for fewer rows (a group's last tile is usually partial) leave out
  // the reads and instructions of sub-tiles without rows
  const int wm = wave / NW, nw = it.bx * C::BN + 32 * SN * (wave % NW);
  const int rows = nw < p.N ? it.rows - 32 * SM * wm : 0;
  if (rows <= 0) product_tile<C, F32, 0>(p, it, lds, src, wave);
  else if (rows <= 32) product_tile<C, F32, 1>(p, it, lds, src, wave);
  else if (SM == 2 || rows <= 64) product_tile<C, F32, 2>(p, it, lds, src, wave);
  else if (rows <= 96) product_tile<C, F32, SM - 1>(p, it, lds, src, wave);
  else product_tile<C, F32, SM>(p, it, lds, src, wave);
}

template <int MW, int NW, int SM, int SN>
static void launch_tile(const ProductArgs& p, hipStream_t stream) {
  typedef Tile<MW, NW, SM, SN> C;
  const dim3 grid((unsigned)max_tiles(p, C::BM) * ceil_div(p.N, C::BN));
  const size_t bytes = C::kLds + 4 * C::BM;
  if (p.out_f32) hipLaunchKernelGGL((k_product_tile<MW, NW, SM, SN, true>), grid, dim3(C::T), bytes, stream, p);
  else hipLaunchKernelGGL((k_product_tile<MW, NW, SM, SN, false>), grid, dim3(C::T), bytes, stream, p);
}

int launch_product_tile(const ProductArgs& p, hipStream_t stream) {
  // the large tile where it still gives most CUs (256) a workgroup: one group of N 4608, K 4608, us large /
  // small: 512 rows 26/19, 1024 28/31, 2048 45/51, 4096 72/95
  const long tiles = ceil_div(p.M, 128) > p.G ? ceil_div(p.M, 128) : p.G;
  if (tiles * ceil_div(p.N, 256) >= 192) launch_tile<1, 4, 4, 2>(p, stream);
  else launch_tile<2, 2, 2, 1>(p, stream);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace moe
