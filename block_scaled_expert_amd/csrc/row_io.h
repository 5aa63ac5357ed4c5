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

template <bool NT, typename T>
__device__ inline T get_nt(const T* p) {
  if constexpr (NT) return __builtin_nontemporal_load(p);
  else return *p;
}
template <bool NT, typename T>
__device__ inline void put_nt(T* p, T v) {
  if constexpr (NT) __builtin_nontemporal_store(v, p);
  else *p = v;
}

// Elements 8 c .. 8 c + 7 of a row of `cols`.  VEC: 16-byte accesses (cols a
// multiple of 8, rows 16-byte aligned), else one element at a time.  Loads of
// chunks or elements past the row read its last ones, so none sits under a
// branch; what they return is not used.
template <bool VEC, bool NT = false>
__device__ inline void load_raw8(Raw8<uint16_t>& r, const uint16_t* row, int c, int cols) {
  if constexpr (VEC) {
    r.w = get_nt<NT>(reinterpret_cast<const v4u*>(row) + min(c, cols / 8 - 1));
  } else {
#pragma unroll
    for (int j = 0; j < 4; j++)
      r.w[j] = (uint32_t)row[min(8 * c + 2 * j, cols - 1)] | (uint32_t)row[min(8 * c + 2 * j + 1, cols - 1)] << 16;
  }
}
template <bool VEC, bool NT = false>
__device__ inline void load_raw8(Raw8<float>& r, const float* row, int c, int cols) {
  if constexpr (VEC) {
    const v4f* p = reinterpret_cast<const v4f*>(row) + 2 * min(c, cols / 8 - 1);
    r.a = get_nt<NT>(p);
    r.b = get_nt<NT>(p + 1);
  } else {
#pragma unroll
    for (int j = 0; j < 4; j++) {
      r.a[j] = row[min(8 * c + j, cols - 1)];
      r.b[j] = row[min(8 * c + 4 + j, cols - 1)];
    }
  }
}
// Element e of chunk c lies in the row.
template <bool VEC>
__device__ inline bool in_row(int c, int e, int cols) {
  return VEC ? 8 * c < cols : 8 * c + e < cols;
}
template <bool VEC, bool NT = false>
__device__ inline void store8(uint16_t* row, int c, int cols, const float (&v)[8]) {
  if constexpr (VEC) {
    if (8 * c < cols)
      put_nt<NT>(reinterpret_cast<v4u*>(row) + c,
                 v4u{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])});
  } else {
#pragma unroll
    for (int j = 0; j < 8; j++)
      if (8 * c + j < cols) row[8 * c + j] = bf16_bits(v[j]);
  }
}
template <bool VEC, bool NT = false>
__device__ inline void store8(float* row, int c, int cols, const float (&v)[8]) {
  if constexpr (VEC) {
    if (8 * c < cols) {
      v4f* p = reinterpret_cast<v4f*>(row) + 2 * c;
      put_nt<NT>(p, v4f{v[0], v[1], v[2], v[3]});
      put_nt<NT>(p + 1, v4f{v[4], v[5], v[6], v[7]});
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; j++)
      if (8 * c + j < cols) row[8 * c + j] = v[j];
  }
}

// Waves of a workgroup that takes a row in pieces of 8 elements a lane, `per`
// pieces a lane at most: the fewest, up to 16.
inline int row_waves(int cols, int per) {
  const int n = ceil_div(ceil_div(cols, 8), 64L * per);
  return n < 16 ? n : 16;
}
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace moe
