// The grouped product of bf16 or fp32 rows and 4-bit matrices for more rows, or
// fp32 rows: on v_mfma_f32_16x16x32_bf16, 16 rows of x at a time.
//
// There the 4x4x4 instructions of matvec.hip would be the limit: their time grows
// with every 4 rows, and each quad reads x from LDS anew.  Here codes are brought
// to operand order first (operand_w) and widened with their scale (MXFP4 in the
// conversion; NVFP4 in fp32, exact: 2 vector instructions a weight), 16 rows cost
// what one does, and a wave uses each piece of x for two tiles of 16 weight rows
// (SwiGLU: the gate and up rows of the same columns).  The rest is as there.
//
// Measured (us; TB/s of the weights in use): 1536 rows over 377 groups of 4608 x
// 2304 MXFP4, fp32 431 (5.0), bf16 407 (5.3); with one tile a wave fp32 took 560.
// 3000 rows of 384 groups NVFP4 bf16 521, 4600 590; 64 rows of one group of 16384
// x 4608 NVFP4 40.7 (four items, the weights from L2 in three), MXFP4 32.3.
#include "matvec.h"

namespace moe {

namespace {

// The same times an E4M3 scale: at most 6 significant bits, exact.
typedef float v2f __attribute__((ext_vector_type(2)));
__device__ inline v8bf widen_scaled(uint32_t w, float scale) {
  const v2f a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
  const v2f c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
  const v2bf e = __builtin_convertvector((v2f{a[0] * scale, a[1] * scale}), v2bf);
  const v2bf f = __builtin_convertvector((v2f{b[0] * scale, b[1] * scale}), v2bf);
  const v2bf g = __builtin_convertvector((v2f{c[0] * scale, c[1] * scale}), v2bf);
  const v2bf h = __builtin_convertvector((v2f{d[0] * scale, d[1] * scale}), v2bf);
  return v8bf{e[0], e[1], f[0], f[1], g[0], g[1], h[0], h[1]};
}
}  // namespace

template <int FMT, bool F32, bool GLU, bool WHOLE>
__global__ __launch_bounds__(512) void k_matvec_wide(MatvecArgs a, int NT, int WC, int lds_bytes) {
  constexpr int PF = 2, PLANES = F32 ? 3 : 1, kRows = 16;   // PF 3: up to 2% slower, 4: 7%
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ int src[kRows];
  __shared__ Item item;
  const ProductArgs& p = a.p;
  const int width = GLU ? p.N / 2 : p.N;            // columns of out
  const int cols = GLU ? 16 * WC : 32 * WC;         // of a tile

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
  const int nb = p.K / 32, chunks = (nb + kChunkBlocks - 1) / kChunkBlocks;
  const int tiles = min(NT, (width - n0 + cols - 1) / cols);
  const int row_bytes = p.K / 2, sc_bytes = nb * (FMT == 1 ? 2 : 1);
  // this wave's weight rows nw + cols t .. of both its tiles (GLU: gate and up rows of
  // the same columns; else 16 columns further on); rows past the width read zeros
  const int nw = n0 + (GLU ? 16 : 32) * wave;
  Buf wq[2], ws[2];
#pragma unroll
  for (int h = 0; h < 2; h++) {
    const int first = nw + (GLU ? 0 : 16 * h);
    const int wrows = max(min(cols * NT - (first - n0), width - first), 0);
    const size_t at = (size_t)g * p.N + (size_t)(GLU ? h * width : 0) + min(first, width - 1);
    wq[h] = make_buf(p.w + at * row_bytes, wrows * row_bytes);
    ws[h] = make_buf(p.w_sc + at * sc_bytes, wrows * sc_bytes);
  }
  const WLane wl(r, b, row_bytes, nb);

  if (tid < kRows) src[tid] = tid < rows ? source_row(p, m0 + tid) : -1;
  Chunk<FMT> ring[PF][2];
  int lt = 0, li = 0;                               // the chunk that is loaded next
  auto load_next = [&](Chunk<FMT> (&W)[2]) {
#pragma unroll
    for (int h = 0; h < 2; h++)
      load_chunk<FMT, WHOLE>(W[h], wq[h], ws[h], wl, lt < tiles, (uint32_t)lt * (cols * row_bytes),
                             (uint32_t)(cols * lt + r) * nb, li);
    if (++li == chunks) {
      li = 0;
      lt++;
    }
  };
  Scales<FMT> sc[2];
  int st = 0, sn = 0;                               // the four chunks whose scales are loaded next
  auto load_scales = [&]() {
#pragma unroll
    for (int h = 0; h < 2; h++) sc[h].load(ws[h], st < tiles && sn + b < chunks, (uint32_t)(cols * st + r) * chunks + sn + b);
    if ((sn += 4) >= chunks) {
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
  // rows past the item read its last one; a row's outputs depend on that row alone
  const uint8_t* const x_lane = lds + min(r, rows - 1) * stride + 128 * b;

  v4f acc[2];                                       // weight row r, x rows 4 b ..
  acc[0] = acc[1] = v4f{0, 0, 0, 0};
  auto put = [&](int m, int n, float v) {
    v = src[m] < 0 ? 0.0f : v;
    const size_t i = (size_t)(m0 + m) * width + n;
    if (p.out_f32) static_cast<float*>(p.out)[i] = v;
    else static_cast<__bf16*>(p.out)[i] = (__bf16)v;   // to nearest even
  };
  auto finish = [&](int t) {
#pragma unroll
    for (int h = 0; h < (GLU ? 1 : 2); h++) {
      const int n = nw + cols * t + 16 * h + r;
      if (n >= width) continue;
      float gs[2] = {1.0f, 1.0f};
      if constexpr (FMT == 1) {
        const float* const of = a.gs + (size_t)g * a.gs_stride;
        gs[0] = of[n / (p.N / a.gs_group)];
        if constexpr (GLU) gs[1] = of[(width + n) / (p.N / a.gs_group)];
      }
#pragma unroll
      for (int q = 0; q < 4; q++) {
        const int m = 4 * b + q;
        if (m >= rows) continue;
        if constexpr (GLU) put(m, n, glu_of(acc[0][q] * gs[0], acc[1][q] * gs[1], a));
        else put(m, n, acc[h][q] * gs[0]);
      }
    }
  };
  int t = 0, i = 0, xc = 0;                         // tile, chunk, chunk within the panel
  while (t < tiles) {
#pragma unroll
    for (int j = 0; j < PF; j++) {
      if (t < tiles) {
        if (!one && xc == 0) {                      // every wave is at the same chunk
          lds_barrier();                            // the last panel has been read
          stage_x<F32, WHOLE>(p, src, rows, i, min(panel, chunks - i), lds, stride, plane);
          lds_barrier();
        }
        Frag f[2];
        uint32_t scw[2];
        if constexpr (WHOLE) {
          if (i % 4 == 0) {
            sc[0].take(b);
            sc[1].take(b);
            load_scales();
          }
        }
#pragma unroll
        for (int h = 0; h < 2; h++) {
          scw[h] = WHOLE ? sc[h].pop() : ring[j][h].sc;
          RawW raw;
          raw.q[0] = ring[j][h].q[0];
          raw.q[1] = ring[j][h].q[1];
          raw.sc = 0;
          operand_w<false>(raw, f[h]);
        }
        const uint8_t* const xp = x_lane + 2 * kChunkK * xc;
#pragma unroll
        for (int u = 0; u < kU; u++) {
#pragma unroll
          for (int q = 0; q < 4; q++) {
            v8bf x[PLANES];
#pragma unroll
            for (int d = 0; d < PLANES; d++) x[d] = *reinterpret_cast<const v8bf*>(xp + d * plane + 64 * u + 16 * q);
#pragma unroll
            for (int h = 0; h < 2; h++) {
              const uint32_t s = scw[h];
              v8bf w;
              if constexpr (FMT == 4) {
                w = __builtin_bit_cast(v8bf, widen(f[h].q[u][q], bits_f((s >> (8 * u) & 0xFFu) << 23)));
              } else {
                const float scale = u == 0 ? (q < 2 ? __builtin_amdgcn_cvt_f32_fp8(s, 0) : __builtin_amdgcn_cvt_f32_fp8(s, 1))
                                           : (q < 2 ? __builtin_amdgcn_cvt_f32_fp8(s, 2) : __builtin_amdgcn_cvt_f32_fp8(s, 3));
                w = widen_scaled(f[h].q[u][q], scale);
              }
#pragma unroll
              for (int d = PLANES - 1; d >= 0; d--) acc[h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[d], w, acc[h], 0, 0, 0);
            }
          }
        }
        xc = !one && xc + 1 == panel ? 0 : xc + 1;
        if (++i == chunks) {                        // the tile is done
          finish(t);
          acc[0] = acc[1] = v4f{0, 0, 0, 0};
          i = xc = 0;
          t++;
        }
      }
      load_next(ring[j]);
    }
  }
}

template <int FMT, bool F32, bool GLU>
static void launch_one(const MatvecArgs& a, hipStream_t stream) {
  const int width = GLU ? a.p.N / 2 : a.p.N, items = max_tiles(a.p, 16);
  const long tiles = (long)ceil_div(width, GLU ? 32 : 64) * items;
  // 8 waves and 76 KiB where there are enough tiles, and for fp32 rows, whose panels
  // 8 waves share (64 rows of 8 groups of 4608 x 2304 29.9 us, with 4 waves and 36
  // KiB 49.5); else 4, and 76 KiB as long as every workgroup has a place (bf16, 4608
  // x 4608 with SwiGLU: 42.4 instead of 44.4).  Up to two tiles in turn.
  const int WC = F32 || tiles > 2048 ? 8 : 4, lds = (WC == 8 || tiles <= 1024 ? 76 : 36) * 1024;
  const int NT = tiles * 2 / WC / 1024 >= 2 ? 2 : 1;
  const dim3 grid((unsigned)items * ceil_div(width, (GLU ? 16 : 32) * WC * NT)), block(64 * WC);
  if (a.p.K % kChunkK == 0) hipLaunchKernelGGL((k_matvec_wide<FMT, F32, GLU, true>), grid, block, lds, stream, a, NT, WC, lds);
  else hipLaunchKernelGGL((k_matvec_wide<FMT, F32, GLU, false>), grid, block, lds, stream, a, NT, WC, lds);
}
template <int FMT>
static void launch_fmt(const MatvecArgs& a, hipStream_t stream) {
  if (a.dtype == 1) {
    if (a.swiglu) launch_one<FMT, true, true>(a, stream);
    else launch_one<FMT, true, false>(a, stream);
  } else {
    if (a.swiglu) launch_one<FMT, false, true>(a, stream);
    else launch_one<FMT, false, false>(a, stream);
  }
}

int launch_matvec_wide(const MatvecArgs& a, hipStream_t stream) {
  if (a.fmt == 1) launch_fmt<1>(a, stream);
  else launch_fmt<4>(a, stream);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace moe
