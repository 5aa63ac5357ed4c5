// Rows of bf16 or fp32 elements, eight consecutive ones per lane, and sums
// over a wavefront: what the norm and the sorted rows share.
#pragma once

#include "moe_common.h"

namespace moe {

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef float v2f __attribute__((ext_vector_type(2)));

// Sum over the wavefront, the same in every lane: within each row of 16 lanes
// by DPP (neighbours, pairs, half rows, rows), then the four rows.  One fixed
// order, and a third of the latency of exchanges through LDS.
template <int CTRL>
__device__ inline float dpp_plus(float v) {
  return v + bits_f((uint32_t)__builtin_amdgcn_update_dpp(0, (int)f_bits(v), CTRL, 0xF, 0xF, false));
}
__device__ inline float lane_value(float v, int l) {
  return bits_f((uint32_t)__builtin_amdgcn_readlane((int)f_bits(v), l));
}
__device__ inline float wave_total(float v) {
  v = dpp_plus<0xB1>(v);    // quad_perm [1,0,3,2]
  v = dpp_plus<0x4E>(v);    // quad_perm [2,3,0,1]
  v = dpp_plus<0x141>(v);   // row_half_mirror
  v = dpp_plus<0x140>(v);   // row_mirror
  return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}
// Sum over the workgroup's waves through `red` (one float a wave); every thread
// calls it, and `red` may be written again after the next barrier.
__device__ inline float group_total(float v, float* red) {
  v = wave_total(v);
  const int waves = blockDim.x >> 6;
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  lds_barrier();
  float s = red[0];
  for (int i = 1; i < waves; i++) s += red[i];
  return s;
}

// fp32 -> bf16 pair, to nearest even, inf and NaN kept.
__device__ inline uint32_t bf16_pair(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{a, b}), v2bf));
}
__device__ inline uint16_t bf16_bits(float a) { return __builtin_bit_cast(uint16_t, (__bf16)a); }

// A value as type T holds it.
template <typename T>
__device__ inline float stored(float v);
template <>
__device__ inline float stored<float>(float v) {
  return v;
}
template <>
__device__ inline float stored<uint16_t>(float v) {
  return (float)(__bf16)v;
}

// Eight elements as loaded; widening them waits for the load.
template <typename T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
  v4u w;
  __device__ inline void get(float (&v)[8]) const {
#pragma unroll
    for (int j = 0; j < 4; j++) {
      v[2 * j] = bits_f(w[j] << 16);
      v[2 * j + 1] = bits_f(w[j] & 0xFFFF0000u);
    }
  }
};
template <>
struct Raw8<float> {
  v4f a, b;
  __device__ inline void get(float (&v)[8]) const {
#pragma unroll
    for (int j = 0; j < 4; j++) {
      v[j] = a[j];
      v[4 + j] = b[j];
    }
  }
};

// 16 bytes at an address that is a multiple of 16, or of the element's size alone.
template <typename T, bool FULL>
struct Wide;
template <>
struct Wide<uint16_t, true> {
  typedef v4u V;
};
template <>
struct Wide<uint16_t, false> {
  typedef v4u V __attribute__((aligned(2)));
};
template <>
struct Wide<float, true> {
  typedef v4f V;
};
template <>
struct Wide<float, false> {
  typedef v4f V __attribute__((aligned(4)));
};

// NT: the hint for bytes that are used once (see kStreamBytes).  fp32 does
// without: a lane's 32 bytes are two accesses, and the hint gives the line away
// between them.  With it and without, 16384 tokens of 4608: the norm of bf16 x and
// an fp32 stream 176 and 167 us, its gradient 235 and 228; the combine of 8 fp32
// rows a token 551 and 492, its gradients 1101 and 1000; with one of the 8 rows
// here 86 and 90, 158 and 151.
template <bool FULL, bool NT>
__device__ inline void load8(Raw8<uint16_t>& r, const uint16_t* p) {
  const auto* q = reinterpret_cast<const typename Wide<uint16_t, FULL>::V*>(p);
  r.w = NT ? __builtin_nontemporal_load(q) : *q;
}
template <bool FULL, bool NT>
__device__ inline void load8(Raw8<float>& r, const float* p) {
  const auto* q = reinterpret_cast<const typename Wide<float, FULL>::V*>(p);
  r.a = *q;
  r.b = q[1];
}
template <bool FULL, bool NT>
__device__ inline void store8(uint16_t* p, const Raw8<uint16_t>& r) {
  auto* q = reinterpret_cast<typename Wide<uint16_t, FULL>::V*>(p);
  if constexpr (NT) __builtin_nontemporal_store(r.w, q);
  else *q = r.w;
}
template <bool FULL, bool NT>
__device__ inline void store8(float* p, const Raw8<float>& r) {
  auto* q = reinterpret_cast<typename Wide<float, FULL>::V*>(p);
  q[0] = r.a;
  q[1] = r.b;
}
__device__ inline void set(Raw8<uint16_t>& r, const float* v) {
  r.w = v4u{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])};
}
__device__ inline void set(Raw8<float>& r, const float* v) {
  r.a = v4f{v[0], v[1], v[2], v[3]};
  r.b = v4f{v[4], v[5], v[6], v[7]};
}
__device__ inline float widen1(uint16_t h) { return bf16_to_f32(h); }
__device__ inline float widen1(float f) { return f; }
__device__ inline void set1(uint16_t& h, float f) { h = bf16_bits(f); }
__device__ inline void set1(float& h, float f) { h = f; }

// The part of a row of `cols` elements that a thread holds: pieces of 8
// elements at thread, thread + threads, .. (CH of them, from piece `from` on)
// and, unless FULL, one of the cols % 8 elements behind the last whole piece.
// FULL: cols is a multiple of 8 and rows are 16-byte aligned; else they need only
// be aligned to their elements.  Loads past the row read its last piece or
// element, so that none sits under a branch; what they return is finite where the
// row is and not used.
template <bool FULL, int CH>
struct Span {
  static constexpr int N = 8 * CH + (FULL ? 0 : 1);
  template <typename T>
  struct Raw {
    Raw8<T> c[CH];
    T t;
  };
  int c0, step, n8, rem, cols;

  __device__ Span(int cols_, int threads, int from = 0)
      : c0(from + (int)threadIdx.x), step(threads), n8(cols_ / 8), rem(FULL || from > 0 ? 0 : cols_ % 8), cols(cols_) {}
  // Whether element k of the thread's N lies in the row.
  __device__ bool has(int k) const { return k < 8 * CH ? c0 + step * (k / 8) < n8 : (int)threadIdx.x < rem; }
  __device__ int piece(int i) const { return c0 + step * i; }

  template <bool NT = false, typename T>
  __device__ void load(Raw<T>& r, const T* row) const {
    if (FULL || n8 > 0) {
#pragma unroll
      for (int i = 0; i < CH; i++) load8<FULL, NT>(r.c[i], row + 8 * min(piece(i), n8 - 1));
    } else {
      const float zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < CH; i++) set(r.c[i], zero);
    }
    if constexpr (!FULL) r.t = row[min(8 * n8 + (int)threadIdx.x, cols - 1)];
  }
  template <typename T>
  __device__ void get(const Raw<T>& r, float (&v)[N]) const {
#pragma unroll
    for (int i = 0; i < CH; i++) {
      float u[8];
      r.c[i].get(u);
#pragma unroll
      for (int e = 0; e < 8; e++) v[8 * i + e] = u[e];
    }
    if constexpr (!FULL) v[8 * CH] = widen1(r.t);
  }
  template <typename T>
  __device__ void set_raw(Raw<T>& r, const float (&v)[N]) const {
#pragma unroll
    for (int i = 0; i < CH; i++) set(r.c[i], v + 8 * i);
    if constexpr (!FULL) set1(r.t, v[8 * CH]);
  }
  template <bool NT = false, typename T>
  __device__ void store(T* row, const Raw<T>& r) const {
#pragma unroll
    for (int i = 0; i < CH; i++)
      if (piece(i) < n8) store8<FULL, NT>(row + 8 * piece(i), r.c[i]);
    if constexpr (!FULL)
      if ((int)threadIdx.x < rem) row[8 * n8 + (int)threadIdx.x] = r.t;
  }
  template <bool NT = false, typename T>
  __device__ void put(T* row, const float (&v)[N]) const {
    Raw<T> r;
    set_raw(r, v);
    store<NT>(row, r);
  }
};

// Waves of a workgroup that holds a row in pieces of 8, at most `per` a thread:
// the fewest, up to 16 (at least 8 threads for the elements behind the pieces).
inline int row_waves(int cols, int per) {
  const int n = ceil_div(cols / 8, 64L * per);
  return n < 1 ? 1 : n < 16 ? n : 16;
}
// Pieces of a thread then, as the kernels are built for them.
inline int row_pieces(int cols, int waves) {
  const int n = ceil_div(cols / 8, 64L * waves);
  return n < 1 ? 1 : n > 4 ? 8 : n;
}
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// CALL with the constant CH = n, of 1, 2, 3, 4 and 8.
#define MOE_ROW_PIECES(n, CALL) \
  switch (n) {                  \
    case 1: { constexpr int CH = 1; CALL; } break; \
    case 2: { constexpr int CH = 2; CALL; } break; \
    case 3: { constexpr int CH = 3; CALL; } break; \
    case 4: { constexpr int CH = 4; CALL; } break; \
    default: { constexpr int CH = 8; CALL; } break; \
  }

}  // namespace moe
