// What the two kernels of the grouped product of bf16 or fp32 rows and 4-bit
// matrices share: how the weights and their scales come in, how codes widen, and
// x in LDS.
#pragma once

#include "group_product.h"

namespace moe {

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

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

  // this lane's chunk: number `at` of the view's, row after row
  __device__ inline void load(Buf ws, bool on, uint32_t at) {
    constexpr int kBytes = FMT == 1 ? 16 : 8;
    const uint32_t off = on ? kBytes * at : kNowhere;
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

// Eight codes (low nibble first) as bf16, times the power of two in scale's
// exponent (an E8M0 byte moved there: 255 gives NaN).
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
__device__ inline v8s widen(uint32_t w, float scale) {
  const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
  const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
  return __builtin_bit_cast(v8s, v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]});
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

// Chunks p0 .. p0 + pn - 1 of the item's rows of x to LDS, zeros past the end of
// k: a wave takes 512 k (64 pieces of 8) of a row at a time.  fp32: three planes.
template <bool F32, bool WHOLE>
__device__ inline void stage_x(const ProductArgs& p, const int* src, int rows, int p0, int pn, uint8_t* lds, int stride,
                               int plane) {
  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6, runs = (pn + 1) / 2;
  int row = threadIdx.x >> 6, run = 0;
  for (;; row += waves) {
    while (row >= rows) {
      row -= rows;
      run++;
    }
    if (run >= runs) break;
    const int q = 64 * run + lane, k = kChunkK * p0 + 8 * q, s = max(src[row], 0);
    if (q >= pn * (kChunkK / 8)) continue;
    v4u hi = v4u{0, 0, 0, 0}, mid = hi, lo = hi;
    if (WHOLE || k < p.K) {
      if constexpr (F32) {
        const v4f* x = reinterpret_cast<const v4f*>(reinterpret_cast<const float*>(p.a) + (size_t)s * p.K + k);
        const v4f u = x[0], v = x[1];
#pragma unroll
        for (int j = 0; j < 4; j++) {
          uint32_t h0, m0, l0, h1, m1, l1;
          split3(j < 2 ? u[2 * j] : v[2 * j - 4], h0, m0, l0);
          split3(j < 2 ? u[2 * j + 1] : v[2 * j - 3], h1, m1, l1);
          hi[j] = h0 | h1 << 16;
          mid[j] = m0 | m1 << 16;
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
}

// Panels of x: as many chunks as the item's rows leave room for in LDS.  Rows
// are 16 bytes apart beyond a multiple of 512, which spreads them over the banks.
struct Panels {
  int n, size, stride, plane;
  __device__ Panels(int lds_bytes, int planes, int rows, int chunks) {
    const int most = max((lds_bytes / (planes * rows) - 16) / (2 * kChunkK), 1);
    n = (chunks + most - 1) / most;
    size = (chunks + n - 1) / n;
    stride = 2 * kChunkK * size + 16;
    plane = stride * rows;
  }
};

// The capped SwiGLU, NaN kept: cap_swiglu's hard cap takes the cap instead.
__device__ inline float glu_of(float g, float u, const MatvecArgs& a) {
  const float h = cap_swiglu(g, u, a.cap_form, a.cap, 1.0f / a.cap);
  return g == g && u == u ? h : g + u;
}

// More rows per group (matvec_wide.hip).
int launch_matvec_wide(const MatvecArgs& a, hipStream_t stream);

}  // namespace moe
