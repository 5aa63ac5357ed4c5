// Grouped product of bf16 or fp32 rows and 4-bit matrices, for the few rows an
// expert has in decoding:
//
//   out[r][n] = sum_k x[src(r)][k] W[g(r)][n][k],   W = code * block scale (* gs)
//
// or, over the gate and up halves of W, the capped SwiGLU of both.
//
// The time is that of streaming the weights of the groups that have rows, so
// the weights go the way of k_product_stream: whole 128-byte lines of 8 rows
// straight to registers, two rows' halves exchanged there, a ring of chunks that
// runs on from tile to tile.  A lane then holds 64 consecutive codes of a row.
// They become bf16 in registers, exactly: an E2M1 value times a power of two
// (MXFP4, one instruction for two), or times an E4M3 value (NVFP4: at most 6
// significant bits).  x, in bf16, waits in LDS; an fp32 x as three bf16 parts
// whose sum it is, so every product is exact and the sums are fp32.  gs is
// applied to the sums.
#include "group_product.h"

namespace moe {

namespace {

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef float v2f __attribute__((ext_vector_type(2)));

constexpr int kRows = 16;                 // rows of an item
constexpr int kLdsBytes = 37 * 1024;      // of x: 4 rows of k 4608 in bf16; four workgroups a CU

// Codes of two blocks of 32 per lane, as loaded (RawW's order), and, unless
// scales come in fours of chunks (Scales), row r's scales of them.
template <int FMT>
struct Chunk {
  v4u q[2];
  uint32_t sc;     // MXFP4: 2 bytes, NVFP4: 4
};

// WHOLE: rows of whole chunks.  Otherwise the row may end inside a chunk, and
// scales are loaded block by block.
template <int FMT, bool WHOLE>
__device__ inline void load_chunk(Chunk<FMT>& W, Buf wq, Buf ws, const WLane& l, bool on, uint32_t base, uint32_t srow, int c) {
  const int blk = kChunkBlocks * c;
  const uint32_t off = on && (WHOLE || blk + l.at < l.nb) ? l.off + base + 16 * blk : kNowhere;
  W.q[0] = buf16<true>(wq, off);
  W.q[1] = buf16<true>(wq, off + l.row8);
  if constexpr (!WHOLE) {
    constexpr int S = FMT == 1 ? 2 : 1;      // scale bytes of a block
    const uint32_t so = S * (srow + blk + kU * l.b);
    const uint32_t at0 = on && blk + kU * l.b < l.nb ? so : kNowhere, at1 = on && blk + kU * l.b + 1 < l.nb ? so + S : kNowhere;
    if constexpr (FMT == 1) {
      const uint32_t a = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(ws, (int)at0, 0, 0);
      const uint32_t b = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(ws, (int)at1, 0, 0);
      W.sc = a | b << 16;
    } else {
      const uint32_t a = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(ws, (int)at0, 0, 0);
      const uint32_t b = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(ws, (int)at1, 0, 0);
      W.sc = a | b << 8;
    }
  }
}

// Scales of four chunks of 16 rows at a time.  One by one they are 16 (NVFP4)
// or 8 bytes of a line per row and chunk, and fetching 16 lines for them costs
// as much as the codes' 16: 512 rows over 283 groups of 4608 x 4608 NVFP4 took
// 732 us that way, 549 with no scales loaded at all.  Here lane (r, b) loads row
// r's scales of chunk b (16 or 8 bytes), and swaps between the four rows of
// lanes hand lane (r, b) what it needs of each chunk.
template <int FMT>
struct Scales {
  v4u next;            // as loaded; MXFP4 uses two words
  uint32_t now[4];     // of the chunks to come, the nearest first

  // chunks c .. c + 3 of the rows that start at row srow; nw: a row's bytes of a chunk
  __device__ inline void load(Buf ws, int r, int b, int chunks, bool on, uint32_t row, int c) {
    constexpr int kBytes = FMT == 1 ? 16 : 8;
    const uint32_t off = on && c + b < chunks ? kBytes * (row * chunks + c + b) : kNowhere;
    if constexpr (FMT == 1) {
      next = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(ws, (int)off, 0, 0));
    } else {
      typedef unsigned v2u __attribute__((ext_vector_type(2)));
      const v2u w = __builtin_bit_cast(v2u, __builtin_amdgcn_raw_buffer_load_b64(ws, (int)off, 0, 0));
      next[0] = w[0];
      next[1] = w[1];
    }
  }
  __device__ inline void take(int b) {
    if constexpr (FMT == 1) {
      // 4 x 4 words across the rows of lanes: halves, then neighbours
      const auto a = __builtin_amdgcn_permlane32_swap(next[0], next[2], false, false);
      const auto c = __builtin_amdgcn_permlane32_swap(next[1], next[3], false, false);
      const auto e = __builtin_amdgcn_permlane16_swap(a[0], c[0], false, false);
      const auto f = __builtin_amdgcn_permlane16_swap(a[1], c[1], false, false);
      now[0] = e[0];
      now[1] = e[1];
      now[2] = f[0];
      now[3] = f[1];
    } else {
      // lanes b = 0, 1 share a chunk's first word, 2, 3 its second
      const auto a = __builtin_amdgcn_permlane32_swap(next[0], next[1], false, false);
      const auto e = __builtin_amdgcn_permlane16_swap(a[0], a[0], false, false);
      const auto f = __builtin_amdgcn_permlane16_swap(a[1], a[1], false, false);
      const int half = 16 * (b & 1);
      now[0] = e[0] >> half;
      now[1] = e[1] >> half;
      now[2] = f[0] >> half;
      now[3] = f[1] >> half;
    }
  }
  __device__ inline uint32_t pop() {
    const uint32_t s = now[0];
    now[0] = now[1];
    now[1] = now[2];
    now[2] = now[3];
    return s;
  }
};

// Eight codes (low nibble first) as bf16.  MXFP4: scale is 2^(byte - 127), of
// which the conversion takes the exponent (255 gives NaN).
template <int FMT>
__device__ inline v8bf widen(uint32_t w, float scale) {
  if constexpr (FMT == 4) {
    const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
    const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
    return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
  } else {
    const v2f a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
    const v2f c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
    const v2bf e = __builtin_convertvector((v2f{a[0] * scale, a[1] * scale}), v2bf);
    const v2bf f = __builtin_convertvector((v2f{b[0] * scale, b[1] * scale}), v2bf);
    const v2bf g = __builtin_convertvector((v2f{c[0] * scale, c[1] * scale}), v2bf);
    const v2bf h = __builtin_convertvector((v2f{d[0] * scale, d[1] * scale}), v2bf);
    return v8bf{e[0], e[1], f[0], f[1], g[0], g[1], h[0], h[1]};
  }
}

// x as hi + mid + lo, each a bf16 (the upper 16 bits of what is left); inf and
// NaN in hi alone.
__device__ inline void split3(float x, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  if (!(fabsf(x) < INFINITY)) {
    hi = __builtin_bit_cast(uint16_t, (__bf16)x);
    mid = lo = 0;
    return;
  }
  const uint32_t h = f_bits(x) & 0xFFFF0000u;
  const float r = x - bits_f(h);
  const uint32_t m = f_bits(r) & 0xFFFF0000u;
  hi = h >> 16;
  mid = m >> 16;
  lo = f_bits(r - bits_f(m)) >> 16;
}

}  // namespace

// F32: x in fp32.  GLU: tiles of 16 gate and the 16 matching up rows a wave.
// WHOLE: K is a multiple of a chunk.
template <int FMT, bool F32, bool GLU, bool WHOLE>
__global__ __launch_bounds__(256, 4) void k_matvec(MatvecArgs a, int NT) {
  constexpr int WT = GLU ? 2 : 1, PF = GLU ? 3 : 6, PLANES = F32 ? 3 : 1;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ int src[kRows];
  const ProductArgs& p = a.p;
  const int width = GLU ? p.N / 2 : p.N;            // columns of out

  Item it;
  if (!find_item<kRows>(p, (width + 64 * NT - 1) / (64 * NT), blockIdx.x, it)) return;
  const int g = it.g, m0 = it.row0, rows = it.rows, n0 = it.bx * 64 * NT;

  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int r = lane & 15, b = lane >> 4;
  const int nb = p.K / 32, chunks = (nb + kChunkBlocks - 1) / kChunkBlocks;
  const int tiles = min(NT, (width - n0 + 63) / 64);
  const int row_bytes = p.K / 2, sc_bytes = nb * (FMT == 1 ? 2 : 1);
  // this wave's weight rows nw + 64 t ..; rows past the width read zeros
  const int nw = n0 + 16 * wave;
  const int wrows = max(min(64 * NT - 16 * wave, width - nw), 0);
  Buf wq[WT], ws[WT];
#pragma unroll
  for (int h = 0; h < WT; h++) {
    const size_t at = (size_t)g * p.N + (size_t)h * width + min(nw, width - 1);
    wq[h] = make_buf(p.w + at * row_bytes, wrows * row_bytes);
    ws[h] = make_buf(p.w_sc + at * sc_bytes, wrows * sc_bytes);
  }
  const WLane wl(r, b, row_bytes, nb);

  if (tid < kRows) src[tid] = tid < rows ? source_row(p, m0 + tid) : -1;
  Chunk<FMT> ring[PF][WT];
  int lt = 0, lc = 0;                               // the chunk that is loaded next
  auto load_next = [&](Chunk<FMT> (&W)[WT]) {
#pragma unroll
    for (int h = 0; h < WT; h++)
      load_chunk<FMT, WHOLE>(W[h], wq[h], ws[h], wl, lt < tiles, (uint32_t)lt * (64 * row_bytes),
                             (uint32_t)(64 * lt + r) * nb, lc);
    if (++lc == chunks) {
      lc = 0;
      lt++;
    }
  };
  Scales<FMT> sc[WT];
  int st = 0, sn = 0;                               // the four chunks whose scales are loaded next
  auto load_scales = [&]() {
#pragma unroll
    for (int h = 0; h < WT; h++) sc[h].load(ws[h], r, b, chunks, st < tiles, 64 * st + r, sn);
    if ((sn += 4) >= chunks) {
      sn = 0;
      st++;
    }
  };
  if constexpr (WHOLE) load_scales();
#pragma unroll
  for (int j = 0; j < PF; j++) load_next(ring[j]);

  // x in panels of as many chunks as the item's rows leave room for; rows are
  // 16 bytes apart beyond a multiple of 512, which spreads them over the banks
  const int most = max((kLdsBytes / (PLANES * rows) - 16) / (2 * kChunkK), 1);
  const int panels = (chunks + most - 1) / most, panel = (chunks + panels - 1) / panels;
  const int stride = 2 * kChunkK * panel + 16, plane = stride * rows;
  auto stage_x = [&](int p0, int pn) {
    const int pieces = pn * (kChunkK / 8);          // of 8 k
    for (int i = tid; i < rows * pieces; i += 256) {
      const int row = i / pieces, q = i - row * pieces, k = kChunkK * p0 + 8 * q, s = max(src[row], 0);
      v4u hi = v4u{0, 0, 0, 0}, mid = hi, lo = hi;
      if (k < p.K) {                                // zeros past the end of k
        if constexpr (F32) {
          const v4f* x = reinterpret_cast<const v4f*>(reinterpret_cast<const float*>(p.a) + (size_t)s * p.K + k);
          const v4f u = x[0], v = x[1];
#pragma unroll
          for (int j = 0; j < 4; j++) {
            uint32_t h0, m0_, l0, h1, m1, l1;
            split3(j < 2 ? u[2 * j] : v[2 * j - 4], h0, m0_, l0);
            split3(j < 2 ? u[2 * j + 1] : v[2 * j - 3], h1, m1, l1);
            hi[j] = h0 | h1 << 16;
            mid[j] = m0_ | m1 << 16;
            lo[j] = l0 | l1 << 16;
          }
        } else {
          hi = *reinterpret_cast<const v4u*>(reinterpret_cast<const uint16_t*>(p.a) + (size_t)s * p.K + k);
        }
      }
      uint8_t* const to = lds + row * stride + 16 * q;
      *reinterpret_cast<v4u*>(to) = hi;
      if constexpr (F32) {
        *reinterpret_cast<v4u*>(to + plane) = mid;
        *reinterpret_cast<v4u*>(to + 2 * plane) = lo;
      }
    }
  };
  lds_barrier();                                    // src is written
  const bool one = panels == 1;
  if (one) {
    stage_x(0, chunks);
    lds_barrier();
  }
  // rows past the item read its last one; a row's outputs depend on that row alone
  const uint8_t* const mine = lds + min(r, rows - 1) * stride + 128 * b;

  v4f acc[WT];
#pragma unroll
  for (int h = 0; h < WT; h++) acc[h] = v4f{0, 0, 0, 0};
  int t = 0, c = 0, pc = 0;                         // tile, chunk, chunk within the panel
  while (t < tiles) {
#pragma unroll
    for (int j = 0; j < PF; j++) {
      if (t < tiles) {
        if (!one && pc == 0) {                      // every wave is at the same chunk
          lds_barrier();                            // the last panel has been read
          stage_x(c, min(panel, chunks - c));
          lds_barrier();
        }
        if constexpr (WHOLE) {
          if (c % 4 == 0) {
#pragma unroll
            for (int h = 0; h < WT; h++) sc[h].take(b);
            load_scales();
          }
        }
        RawW raw;
        Frag f[WT];
        uint32_t scw[WT];
#pragma unroll
        for (int h = 0; h < WT; h++) scw[h] = WHOLE ? sc[h].pop() : ring[j][h].sc;
#pragma unroll
        for (int h = 0; h < WT; h++) {
          raw.q[0] = ring[j][h].q[0];
          raw.q[1] = ring[j][h].q[1];
          raw.sc = 0;
          operand_w<false>(raw, f[h]);
        }
#pragma unroll
        for (int u = 0; u < kU; u++) {
#pragma unroll
          for (int q = 0; q < 4; q++) {
            v8bf x[PLANES];
#pragma unroll
            for (int e = 0; e < PLANES; e++)
              x[e] = *reinterpret_cast<const v8bf*>(mine + e * plane + 2 * kChunkK * pc + 64 * u + 16 * q);
#pragma unroll
            for (int h = 0; h < WT; h++) {
              const uint32_t sc = scw[h];
              const float scale = FMT == 4 ? bits_f((sc >> (8 * u) & 0xFFu) << 23)
                                           : u == 0 ? (q < 2 ? __builtin_amdgcn_cvt_f32_fp8(sc, 0) : __builtin_amdgcn_cvt_f32_fp8(sc, 1))
                                                    : (q < 2 ? __builtin_amdgcn_cvt_f32_fp8(sc, 2) : __builtin_amdgcn_cvt_f32_fp8(sc, 3));
              const v8bf wv = widen<FMT>(f[h].q[u][q], scale);
#pragma unroll
              for (int e = PLANES - 1; e >= 0; e--) acc[h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[e], wv, acc[h], 0, 0, 0);
            }
          }
        }
        pc = pc + 1 == panel ? 0 : pc + 1;
        if (++c == chunks) {                        // the tile is done
          const int n = nw + 64 * t + r;
          if (n < width) {
            float gs[WT];
#pragma unroll
            for (int h = 0; h < WT; h++)
              gs[h] = FMT == 1 ? a.gs[(size_t)g * a.gs_stride + (h * width + n) / (p.N / a.gs_group)] : 1.0f;
#pragma unroll
            for (int q = 0; q < 4; q++) {
              const int m = 4 * b + q;
              if (m < rows) {
                float v = acc[0][q] * gs[0];
                if constexpr (GLU) v = cap_swiglu(v, acc[1][q] * gs[1], a.cap_form, a.cap, 1.0f / a.cap);
                v = src[m] < 0 ? 0.0f : v;
                const size_t i = (size_t)(m0 + m) * width + n;
                if (p.out_f32) static_cast<float*>(p.out)[i] = v;
                else static_cast<__bf16*>(p.out)[i] = (__bf16)v;   // to nearest even
              }
            }
          }
#pragma unroll
          for (int h = 0; h < WT; h++) acc[h] = v4f{0, 0, 0, 0};
          c = pc = 0;
          t++;
        }
      }
      load_next(ring[j]);
    }
  }
}

template <int FMT, bool F32, bool GLU, bool WHOLE>
static void launch_one(const MatvecArgs& a, hipStream_t stream) {
  const int width = GLU ? a.p.N / 2 : a.p.N;
  const long nt = (long)ceil_div(width, 64) * max_tiles(a.p, kRows) / 4096;
  const int NT = (int)(nt < 1 ? 1 : nt > 4 ? 4 : nt);
  const dim3 grid((unsigned)max_tiles(a.p, kRows) * ceil_div(width, 64 * NT));
  hipLaunchKernelGGL((k_matvec<FMT, F32, GLU, WHOLE>), grid, dim3(256), kLdsBytes, stream, a, NT);
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

int launch_group_matvec(const MatvecArgs& a, hipStream_t stream) {
  if (a.p.M <= 0) return 0;
  if (a.fmt == 1) launch_fmt<1>(a, stream);
  else launch_fmt<4>(a, stream);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace moe
