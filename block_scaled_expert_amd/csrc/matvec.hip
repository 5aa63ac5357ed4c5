// Grouped product of bf16 or fp32 rows and 4-bit matrices, for the few rows an
// expert has in decoding:
//
//   out[r][n] = sum_k x[src(r)][k] W[g(r)][n][k],   W = code * block scale (* gs)
//
// or, over the gate and up halves of W, the capped SwiGLU of both.
//
// The time is that of streaming the weights of the groups that have rows, so
// they go the way of k_product_stream: whole 128-byte lines of 8 rows straight
// to registers, a ring of chunks that runs on from tile to tile.  What could
// keep the stream from its rate is the work on each weight, so there is as
// little of it as can be:
//  - codes become bf16 two an instruction (E2M1 values are exact there), under
//    MXFP4 times the block's power of two in the same instruction;
//  - the products run on v_mfma_f32_4x4x4_16b: a lane multiplies its own codes
//    (4 of k) with 4 rows of x, and nothing meets another lane's until the tile
//    is done.  So lanes may hold codes of any row and block, as they were loaded,
//    and an NVFP4 block's scale is applied to its 4 sums instead of its 16 codes
//    (0.75 vector instructions a weight; widening and scaling each code for
//    16x16x32 took 2, and 612 us where this took 556).  Until then the codes are
//    kept 2^-7 smaller (kSmaller), so that 16 products of 6 and the largest x stay
//    in fp32's range; powers of two change no rounding above its least numbers;
//  - scales are loaded four chunks at a time (Scales).
// x, in bf16, waits in LDS; an fp32 x as three bf16 parts whose sum it is.
// Products are exact and sums fp32; gs is applied to the sums.  A row's bits do
// not depend on which other rows its group or call has, but follow the sizes of
// the call: which kernel takes it, and how many waves share the chunks (KS).
//
// Measured (us; TB/s of the weights in use): 64 tokens' gate/up with SwiGLU, 512
// rows over 283 of 384 groups of 4608 x 4608, NVFP4 518 to 551 on different
// machines (6.1 to 6.5), MXFP4 540; one token's gate/up, 8 groups, 23.5 (4.1).
// With more rows, or fp32 rows (three times the products and x reads), the
// kernel of matvec_wide.hip is ahead.
#include "matvec.h"

namespace moe {

namespace {

// Of NVFP4's codes until the sums of a tile are done: 16 * 6 < 2^7.
constexpr float kSmaller = 0x1p-7f;

__device__ inline v4s lo4(v8s v) { return v4s{v[0], v[1], v[2], v[3]}; }
__device__ inline v4s hi4(v8s v) { return v4s{v[4], v[5], v[6], v[7]}; }

// Lane (r, b) of 16 x 4: the sums over the lanes that agree modulo 8, of value
// b of s[0] where r < 8 and of s[1] elsewhere.
__device__ inline float lanes_by_8(const v4f (&s)[2], int r) {
  float k[4];
#pragma unroll
  for (int m = 0; m < 4; m++) {
    const float away = r < 8 ? s[1][m] : s[0][m];
    k[m] = (r < 8 ? s[0][m] : s[1][m]) +
           bits_f((uint32_t)__builtin_amdgcn_update_dpp(0, (int)f_bits(away), 0x128, 0xF, 0xF, false));   // row_ror:8
  }
  // values 0, 1 to the lower half of the lanes, 2, 3 to the upper; then the odd ones to odd rows
  float h[2];
#pragma unroll
  for (int m = 0; m < 2; m++) {
    const auto w = __builtin_amdgcn_permlane32_swap(f_bits(k[m]), f_bits(k[m + 2]), false, false);
    h[m] = bits_f(w[0]) + bits_f(w[1]);
  }
  const auto w = __builtin_amdgcn_permlane16_swap(f_bits(h[0]), f_bits(h[1]), false, false);
  return bits_f(w[0]) + bits_f(w[1]);
}

}  // namespace

// F32: x in fp32.  GLU: the upper half of the waves takes the up rows of the
// columns that the lower half takes the gate rows of.  WHOLE: K is a multiple of
// a chunk.  NQ: quads of x rows of an item.  KS sets of WC waves take every KS-th
// chunk each; with KS > 1 an item is one tile, and all of x fits in LDS.
template <int FMT, bool F32, bool GLU, bool WHOLE, int NQ>
__global__ __launch_bounds__(512) void k_matvec(MatvecArgs a, int NT, int WC, int KS, int lds_bytes) {
  constexpr int PF = 3, PLANES = F32 ? 3 : 1, kRows = 4 * NQ;   // PF 4: 1-2% slower, 6: 3-4%
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ int src[kRows];
  __shared__ float up[GLU ? 2 : 1][4][NQ][64];      // sums of up rows on their way to the gate's waves
  __shared__ Item item;
  const ProductArgs& p = a.p;
  const int width = GLU ? p.N / 2 : p.N;            // columns of out
  const int cols = GLU ? 8 * WC : 16 * WC;          // of a tile

  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  if (wave == 0) {                                  // one wave looks for the item
    Item it;
    if (!find_item<kRows>(p, (width + cols * NT - 1) / (cols * NT), blockIdx.x, it)) it.rows = 0;
    if (lane == 0) item = it;
  }
  lds_barrier();
  const int rows = __builtin_amdgcn_readfirstlane(item.rows);
  if (rows == 0) return;
  const int g = __builtin_amdgcn_readfirstlane(item.g), m0 = __builtin_amdgcn_readfirstlane(item.row0);
  const int n0 = __builtin_amdgcn_readfirstlane(item.bx) * cols * NT;

  const int r = lane & 15, b = lane >> 4;
  const int part = wave / WC, col = wave - part * WC;   // of the chunks, of the tile's columns
  const int half = GLU && 2 * col >= WC ? 1 : 0, pair = GLU ? col - half * (WC / 2) : col;
  const int nb = p.K / 32, chunks = (nb + kChunkBlocks - 1) / kChunkBlocks;
  const int mine = (chunks - part + KS - 1) / KS;   // chunks part, part + KS, ..
  const int tiles = min(NT, (width - n0 + cols - 1) / cols);
  const int row_bytes = p.K / 2, sc_bytes = nb * (FMT == 1 ? 2 : 1);
  // this wave's weight rows nw + cols t ..; rows past the width read zeros
  const int nw = n0 + 16 * pair;
  const int wrows = max(min(cols * NT - 16 * pair, width - nw), 0);
  const size_t wr0 = (size_t)g * p.N + (size_t)half * width + min(nw, width - 1);
  const Buf wq = make_buf(p.w + wr0 * row_bytes, wrows * row_bytes);
  const Buf ws = make_buf(p.w_sc + wr0 * sc_bytes, wrows * sc_bytes);
  const WLane wl(r, b, row_bytes, nb);

  if (tid < kRows) src[tid] = tid < rows ? source_row(p, m0 + tid) : -1;
  Chunk<FMT> ring[PF];
  int lt = mine > 0 ? 0 : tiles, li = 0;            // the chunk that is loaded next
  auto load_next = [&](Chunk<FMT>& W) {
    load_chunk<FMT, WHOLE>(W, wq, ws, wl, lt < tiles, (uint32_t)lt * (cols * row_bytes), (uint32_t)(cols * lt + r) * nb,
                           part + KS * li);
    if (++li == mine) {
      li = 0;
      lt++;
    }
  };
  Scales<FMT> sc;
  int st = lt, sn = 0;                              // the four chunks whose scales are loaded next
  auto load_scales = [&]() {
    sc.load(ws, st < tiles && sn + b < mine, (uint32_t)(cols * st + r) * chunks + part + KS * (sn + b));
    if ((sn += 4) >= mine) {
      sn = 0;
      st++;
    }
  };
  if constexpr (WHOLE) load_scales();
#pragma unroll
  for (int j = 0; j < PF; j++) load_next(ring[j]);

  const Panels pan(lds_bytes, PLANES, rows, chunks);
  const int panel = pan.size, stride = pan.stride, plane = pan.plane;
  const bool one = pan.n == 1;
  lds_barrier();                                    // src is written
  if (one) {
    stage_x<F32, WHOLE>(p, src, rows, 0, chunks, lds, stride, plane);
    lds_barrier();
  }
  // lane (r, b) of quad k has x row 4 k + r % 4 and the block of 32 that it has codes of;
  // past the item its last row; a row's outputs depend on that row alone
  int x_at[NQ];
#pragma unroll
  for (int k = 0; k < NQ; k++) x_at[k] = min(4 * k + (r & 3), rows - 1) * stride + 128 * b + 64 * (r >> 3);

  v4f acc[NQ][2];                                   // of weight rows r % 8 and 8 + r % 8
  auto clear = [&]() {
#pragma unroll
    for (int k = 0; k < NQ; k++) acc[k][0] = acc[k][1] = v4f{0, 0, 0, 0};
  };
  clear();
  // lane (r, b) puts out weight row r and x rows b, 4 + b, ..
  auto finish = [&](int t) {
    const int n = nw + cols * t + r;
    float v[NQ];
#pragma unroll
    for (int k = 0; k < NQ; k++) {
      if (4 * k >= rows) continue;
      v[k] = lanes_by_8(acc[k], r);
      if constexpr (FMT == 1)
        v[k] = v[k] * (1.0f / kSmaller) *
               a.gs[(size_t)g * a.gs_stride + (half * width + min(n, width - 1)) / (p.N / a.gs_group)];
    }
    if constexpr (GLU) {                            // two tiles' worth of room: one barrier a tile
      if (half)
#pragma unroll
        for (int k = 0; k < NQ; k++) up[t & 1][pair][k][lane] = v[k];
      lds_barrier();
      if (half) return;
    }
    if (n >= width) return;
#pragma unroll
    for (int k = 0; k < NQ; k++) {
      const int m = 4 * k + b;
      if (m < rows) {
        float o = v[k];
        if constexpr (GLU) o = glu_of(o, up[t & 1][pair][k][lane], a);
        o = src[m] < 0 ? 0.0f : o;
        const size_t i = (size_t)(m0 + m) * width + n;
        if (p.out_f32) static_cast<float*>(p.out)[i] = o;
        else static_cast<__bf16*>(p.out)[i] = (__bf16)o;   // to nearest even
      }
    }
  };
  int t = mine > 0 ? 0 : tiles, i = 0, xc = part;   // tile, chunk of mine, chunk within the panel
  while (t < tiles) {
#pragma unroll
    for (int j = 0; j < PF; j++) {
      if (t < tiles) {
        if (!one && xc == 0) {                      // KS is 1: every wave is at the same chunk
          lds_barrier();                            // the last panel has been read
          stage_x<F32, WHOLE>(p, src, rows, i, min(panel, chunks - i), lds, stride, plane);
          lds_barrier();
        }
        if constexpr (WHOLE) {
          if (i % 4 == 0) {
            sc.take(b);
            load_scales();
          }
        }
        // this lane's block of 32: its scales in weight rows r % 8 and 8 + r % 8
        const uint32_t own = WHOLE ? sc.pop() : ring[j].sc;
        const uint32_t other = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)own, 0x128, 0xF, 0xF, false);   // row_ror:8
        constexpr int kHalf = FMT == 1 ? 16 : 8;
        const uint32_t s0 = r < 8 ? own : other >> kHalf, s1 = r < 8 ? other : own >> kHalf;
        const uint8_t* const xp = lds + 2 * kChunkK * xc;
#pragma unroll
        for (int e = 0; e < 2; e++) {               // 16 of k: an NVFP4 block
          v8s w[2][2];
          float scale[2];
#pragma unroll
          for (int y = 0; y < 2; y++) {
            const uint32_t s = y == 0 ? s0 : s1;
            scale[y] = FMT == 4 ? bits_f((s & 0xFFu) << 23)
                                : e == 0 ? __builtin_amdgcn_cvt_f32_fp8(s, 0) : __builtin_amdgcn_cvt_f32_fp8(s, 1);
#pragma unroll
            for (int q = 0; q < 2; q++) w[y][q] = widen(ring[j].q[y][2 * e + q], FMT == 4 ? scale[y] : kSmaller);
          }
#pragma unroll
          for (int k = 0; k < NQ; k++) {
            if (k > 0 && 4 * k >= rows) continue;
            v8s x[PLANES][2];
#pragma unroll
            for (int d = 0; d < PLANES; d++)
#pragma unroll
              for (int q = 0; q < 2; q++) x[d][q] = *reinterpret_cast<const v8s*>(xp + x_at[k] + d * plane + 32 * e + 16 * q);
#pragma unroll
            for (int y = 0; y < 2; y++) {
              v4f c = FMT == 4 ? acc[k][y] : v4f{0, 0, 0, 0};
#pragma unroll
              for (int q = 0; q < 2; q++)
#pragma unroll
                for (int d = PLANES - 1; d >= 0; d--) {
                  c = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(lo4(x[d][q]), lo4(w[y][q]), c, 0, 0, 0);
                  c = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(hi4(x[d][q]), hi4(w[y][q]), c, 0, 0, 0);
                }
              if constexpr (FMT == 4) {
                acc[k][y] = c;
              } else {
#pragma unroll
                for (int m = 0; m < 4; m++) acc[k][y][m] = fmaf(scale[y], c[m], acc[k][y][m]);
              }
            }
          }
        }
        xc = !one && xc + 1 == panel ? 0 : xc + KS;
        if (++i == mine) {                          // the tile is done
          if (KS == 1) {
            finish(t);
            clear();
          }
          i = 0;
          xc = part;
          t++;
        }
      }
      load_next(ring[j]);
    }
  }
  if (KS > 1) {                                     // the parts' sums, in order
    v4f* const red = reinterpret_cast<v4f*>(lds);   // [KS - 1][WC][NQ][2][64]
    lds_barrier();                                  // x has been read
    if (part > 0)
#pragma unroll
      for (int k = 0; k < NQ; k++)
#pragma unroll
        for (int y = 0; y < 2; y++) red[((((part - 1) * WC + col) * NQ + k) * 2 + y) * 64 + lane] = acc[k][y];
    lds_barrier();
    if (part > 0) return;
    for (int e = 0; e < KS - 1; e++)
#pragma unroll
      for (int k = 0; k < NQ; k++)
#pragma unroll
        for (int y = 0; y < 2; y++) acc[k][y] += red[(((e * WC + col) * NQ + k) * 2 + y) * 64 + lane];
    finish(0);
  }
}

// Rows of an item: 8.  With 16 the registers for their sums cost 2 to 5% where
// groups have 1 to 4 rows; with 4 groups of 4 rows on average took 499 us where
// 8 take 416.
constexpr int kQuads = 2;

// Waves of a workgroup and LDS, by tiles (64 columns of 8 rows at most).  A CU has
// 160 KiB of LDS; SwiGLU's exchange takes 4 beside x.
//  - up to 10240, 4 waves and 36 KiB, three or four workgroups a CU: with 8 waves
//    and 74 KiB the same work is handed out in larger pieces, which took 84 us
//    instead of 68 for 4 tokens' gate/up, 229 instead of 219 for 16;
//  - above, 8 waves and 74 KiB, in which 8 rows of k 4608 fit: where groups have
//    more than 3 rows, 4 waves bring x in again for every tile (1536 rows down
//    in fp32 624 us instead of 553, gate/up 882 instead of 842).  At 76 KiB only
//    one workgroup with SwiGLU fits a CU: 64 tokens' gate/up 582 us instead of 551,
//    with fp32 rows 767 instead of 686.
//    Also where fp32 rows take several panels, unless most groups are empty and
//    the others have a row each (16 rows of one group of 16384 x 4608 32.6 us
//    instead of 40.0, 64 of 4 of 2048 x 2048 16.5 instead of 18.5; one token's
//    gate/up in fp32 31.8 instead of 28.1);
//  - up to 256, where all of x fits, two sets of 2 waves share the chunks, up to
//    128 four sets: there are not enough columns to go round (4608 x 4608, one
//    row: 8.7 us instead of 11.8; 16384 columns 12.9 instead of 13.7; 4 rows in
//    fp32 11.4 instead of 20.3).  8 fp32 rows fit as two items of 4, in sets of 4
//    waves where one workgroup fills a CU's LDS (13.3 instead of 28.0 as one item,
//    25.4 in sets of 2);
//  - up to 512 (256) otherwise, what x needs up to 74 (150) KiB, as two workgroups
//    of 4 waves a CU (one) leave it: 8 fp32 rows, 16384 x 4608, 28.3 us instead of 32.0.
constexpr long kMostLds = 150 * 1024;
template <int FMT, bool F32, bool GLU, bool WHOLE, int NQ>
static void launch_rows(const MatvecArgs& a, hipStream_t stream) {
  const int width = GLU ? a.p.N / 2 : a.p.N, items = max_tiles(a.p, 4 * NQ), chunks = ceil_div(a.p.K, kChunkK);
  const long tiles = (long)ceil_div(width, GLU ? 32 : 64) * items;
  const int most = a.p.M < 4 * NQ ? a.p.M : 4 * NQ;   // rows of an item at most
  const long need = (long)(F32 ? 3 : 1) * most * (2 * kChunkK * chunks + 16);
  const bool panels = F32 && need > 36 * 1024 && 4L * a.p.M > a.p.G;
  int WC = tiles > 10240 || panels ? 8 : 4, KS = 1, lds = (WC == 8 ? 74 : 36) * 1024;
  // tiles a workgroup takes in turn, so that there remain about 1024 workgroups (2 to 4 a CU)
  const long nt = tiles * 4 / WC / 1024;
  const int NT = (int)(nt < 1 ? 1 : nt > 4 ? 4 : nt);
  if (tiles <= 256 && need <= kMostLds && chunks > 1) {
    KS = tiles <= 128 && chunks > 3 ? 4 : 2;
    WC = KS == 2 && need > 74 * 1024 ? 4 : 2;         // one workgroup a CU: as many as tiles
    const int red = (KS - 1) * WC * NQ * 2048;
    lds = need > red ? (int)need : red;
  } else if (tiles <= 512 && need > lds) {
    const long room = tiles <= (WC == 8 ? 512 : 256) ? kMostLds : 74 * 1024;
    lds = (int)(need < room ? need : room);
  }
  const dim3 grid((unsigned)items * ceil_div(width, (GLU ? 8 : 16) * WC * NT));
  hipLaunchKernelGGL((k_matvec<FMT, F32, GLU, WHOLE, NQ>), grid, dim3(64 * WC * KS), lds, stream, a, NT, WC, KS, lds);
}
template <int FMT, bool F32, bool GLU, bool WHOLE>
static void launch_one(const MatvecArgs& a, hipStream_t stream) {
  if constexpr (F32) {                                // items of 4 rows, if that brings the sets of waves about
    const int width = GLU ? a.p.N / 2 : a.p.N;
    const long row = 3L * (2 * kChunkK * ceil_div(a.p.K, kChunkK) + 16);
    if (a.p.M > 4 && row * (a.p.M < 8 ? a.p.M : 8) > kMostLds && 4 * row <= kMostLds &&
        (long)ceil_div(width, GLU ? 32 : 64) * max_tiles(a.p, 4) <= 256) {
      launch_rows<FMT, F32, GLU, WHOLE, 1>(a, stream);
      return;
    }
  }
  launch_rows<FMT, F32, GLU, WHOLE, kQuads>(a, stream);
}
template <int FMT, bool F32, bool GLU>
static void launch_whole(const MatvecArgs& a, hipStream_t stream) {
  if (a.p.K % kChunkK == 0) launch_one<FMT, F32, GLU, true>(a, stream);
  else launch_one<FMT, F32, GLU, false>(a, stream);
}
template <int FMT>
static void launch_fmt(const MatvecArgs& a, hipStream_t stream) {
  if (a.dtype == 1) {
    if (a.swiglu) launch_whole<FMT, true, true>(a, stream);
    else launch_whole<FMT, true, false>(a, stream);
  } else {
    if (a.swiglu) launch_whole<FMT, false, true>(a, stream);
    else launch_whole<FMT, false, false>(a, stream);
  }
}

// By the mean group, and by tiles of 64 columns of 16 rows (fewer leave CUs idle
// there).  us, quads / wide, 4608 x 4608 NVFP4 bf16: 64 rows of one group 24.8/29.6
// (360 tiles), 96 of 8 groups 47.0/44.1 (1008), 16384 columns 16 rows 21.9/30.0
// (512), 32 rows 30.2/30.1 (768), 64 rows 55.9/40.7.  384 groups, mean 1.3, 2.7, 4, 5
// rows: 4608 x 2304 NVFP4 bf16 285/312, 418/435, 419/428, 453/438, fp32 344/373,
// 480/491, 576/512, 650/534; MXFP4 bf16 254/251, 370/369, 376/355, 405/367, fp32
// 317/284, 443/375, 537/405, 606/428 (0.7: 216/195).  4608 x 4608 with SwiGLU:
// NVFP4 bf16 514/565, 709/748, 762/768, 817/792, fp32 681/716, 953/944, 1128/992,
// 1276/1029; MXFP4 bf16 504/501, 669/663, 720/680, 771/706, fp32 633/561, 905/742.
// Those rows lie spread over the groups, which is what the host has to take them
// for: 64 rows that all lie in one of 384 groups come in items of 8 (55.9 us at
// 16384 columns, where items of 16 take 40.7).
static bool wide_rows(const MatvecArgs& a) {
  const long tiles = (long)max_tiles(a.p, 16) * ceil_div(a.swiglu ? a.p.N / 2 : a.p.N, a.swiglu ? 32 : 64);
  const long M = a.p.M, G = a.p.G;
  if (tiles < 768) return false;
  if (a.fmt == 4) return a.dtype == 1 ? 2 * M > G : M > G;
  return a.dtype == 1 ? M > 2 * G : M > 4 * G;
}

int launch_group_matvec(const MatvecArgs& a, hipStream_t stream) {
  if (a.p.M <= 0) return 0;
  if (wide_rows(a)) return launch_matvec_wide(a, stream);
  if (a.fmt == 1) launch_fmt<1>(a, stream);
  else launch_fmt<4>(a, stream);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace moe
