// MXFP4: E2M1 codes (two per byte, element 2i in the low nibble) with one
// E8M0 scale per 32 consecutive elements of a row.  Encoding, decoding, and
// the capped SwiGLU that feeds the down product, encoded in the same pass.
//
//   X = 2^clamp(floor(log2 amax) - 2, -127, 127)   (2 = E2M1's largest exponent; 2^-127 for a zero block)
//   code = E2M1(v / X), round to nearest even, saturating at 6; a NaN element encodes as +0
//
// v / X is exact (X is a power of two), so codes and scales are bit-identical
// to the definition.  Rows hold whole blocks, so a contiguous matrix is one
// flat run of blocks and the row length plays no part.
//
// HBM-bound: every input byte is read once, every output byte written once,
// with the lanes of a wavefront on consecutive 16-byte pieces.  Measured: 16384
// x 4608 bf16 encoded in 27.3 us (7.0 TB/s), decoded to fp32 in 47.7 (7.2); 8 x
// 2304 x 4608 fp32 encoded in 70.8 (5.4), decoded in 53.8 (7.2); 64 x 4608 bf16
// in 2.7 each, a launch's own time.
#include "operators.h"

namespace moe {

namespace {

// Maximum over aligned groups of 4 lanes (quad_perm DPP: swap neighbours,
// swap pairs).
__device__ inline float quad_max(float v) {
  const int a = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0xB1, 0xF, 0xF, false);
  v = fmaxf(v, __builtin_bit_cast(float, a));
  const int b = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x4E, 0xF, 0xF, false);
  return fmaxf(v, __builtin_bit_cast(float, b));
}

// NT: the hint for bytes that are used once (see kStreamBytes).
template <bool NT = false>
__device__ inline void load8(const uint16_t* p, float (&v)[8]) {
  const v4u* q = reinterpret_cast<const v4u*>(p);
  const v4u w = NT ? __builtin_nontemporal_load(q) : *q;
#pragma unroll
  for (int j = 0; j < 4; j++) {
    v[2 * j] = bits_f(w[j] << 16);
    v[2 * j + 1] = bits_f(w[j] & 0xFFFF0000u);
  }
}
template <bool NT = false>
__device__ inline void load8(const float* p, float (&v)[8]) {
  const v4f* q = reinterpret_cast<const v4f*>(p);
  const v4f a = NT ? __builtin_nontemporal_load(q) : q[0], b = NT ? __builtin_nontemporal_load(q + 1) : q[1];
#pragma unroll
  for (int j = 0; j < 4; j++) {
    v[j] = a[j];
    v[4 + j] = b[j];
  }
}

// This lane's 8 elements of a block held by 4 consecutive lanes: the codes
// as one word; E is the block's exponent.
__device__ inline uint32_t encode8(float (&v)[8], int& E) {
  float am = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; i++) am = fmaxf(am, fabsf(v[i]));   // a NaN is passed over
  E = mxfp4_exponent(quad_max(am));
#pragma unroll
  for (int i = 0; i < 8; i++) v[i] = v[i] == v[i] ? v[i] : 0.0f;
  return e2m1_pack8(v, pow2f(-E));                           // -E in [-126, 127]
}

}  // namespace

constexpr int kEncUnroll = 2;   // loads in flight per lane (16384 x 4608 bf16 to codes and back: 81 us; 4: 85, 8: 91)

// n elements (a multiple of 32), 8 per lane and pass.
template <typename InT, bool NT>
__global__ __launch_bounds__(256) void k_mxfp4_encode(const InT* __restrict__ x, long n, uint8_t* __restrict__ codes,
                                                      uint8_t* __restrict__ scales) {
  constexpr long kPass = 256 * 8 * kEncUnroll;
  for (long base = blockIdx.x * kPass + 8 * threadIdx.x; base < n; base += gridDim.x * kPass) {
    float v[kEncUnroll][8];
#pragma unroll
    for (int u = 0; u < kEncUnroll; u++) {
      const long i = base + u * 2048;
      if (i < n) load8<NT>(x + i, v[u]);
    }
#pragma unroll
    for (int u = 0; u < kEncUnroll; u++) {
      const long i = base + u * 2048;
      if (i >= n) continue;   // the 4 lanes of a block leave together
      int E;
      const uint32_t w = encode8(v[u], E);
      *reinterpret_cast<uint32_t*>(codes + i / 2) = w;
      if ((threadIdx.x & 3) == 0) scales[i / 32] = (uint8_t)(E + 127);
    }
  }
}

// fp32 values: 4 per lane and pass (one 16-byte store).
template <bool NT>
__global__ __launch_bounds__(256) void k_mxfp4_decode(const uint8_t* __restrict__ codes,
                                                      const uint8_t* __restrict__ scales, long n,
                                                      float* __restrict__ out) {
  constexpr long kPass = 256 * 4 * kEncUnroll;
  for (long base = blockIdx.x * kPass + 4 * threadIdx.x; base < n; base += gridDim.x * kPass) {
    uint32_t w[kEncUnroll];
    int e[kEncUnroll];
#pragma unroll
    for (int u = 0; u < kEncUnroll; u++) {
      const long i = base + u * 1024;
      w[u] = 0;
      e[u] = 0;
      if (i < n) {
        w[u] = *reinterpret_cast<const uint16_t*>(codes + i / 2);
        e[u] = (int)scales[i / 32] - 127;
      }
    }
#pragma unroll
    for (int u = 0; u < kEncUnroll; u++) {
      const long i = base + u * 1024;
      if (i >= n) continue;
      v4f o;
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const uint32_t c = (w[u] >> (4 * j)) & 15u, m = c & 7u;
        // magnitude from the fields: subnormal 0 / 0.5, else (1 + m/2) 2^(e-1)
        const float mag = m < 2 ? 0.5f * (float)m : bits_f(((m >> 1) + 126u) << 23 | (m & 1u) << 22);
        const float v = __builtin_amdgcn_ldexpf((c & 8u) ? -mag : mag, e[u]);
        o[j] = e[u] == 128 ? __builtin_nanf("") : v;   // byte 255 is E8M0's NaN, as in the product
      }
      if constexpr (NT) __builtin_nontemporal_store(o, reinterpret_cast<v4f*>(out + i));
      else *reinterpret_cast<v4f*>(out + i) = o;
    }
  }
}

// h = capped SwiGLU of rows [g | u] (fp32, 2F wide, the gate/up product),
// encoded: 8 columns per lane, 4 lanes per block.  Row count on the device, so
// the grid covers every pair of the call.  Measured: about 16384 local rows of
// F 2304 (of 131072 pairs) 105 us, 3.1 TB/s, where 322 MB take 62 at a copy's
// rate: seven of eight workgroups only leave, and the second of a row has 32 of
// 256 lanes at work.  512 rows 5 us.
__global__ __launch_bounds__(256) void k_swiglu_mxfp4(const float* __restrict__ gu, const int* __restrict__ rows_dev,
                                                      int F, int form, float cap, float inv_c,
                                                      uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const int row = blockIdx.x, c = (blockIdx.y * 256 + threadIdx.x) * 8;
  if (row >= *rows_dev || c >= F) return;   // F is a multiple of 32: the 4 lanes of a block leave together
  const float* r = gu + (size_t)row * 2 * F;
  float g[8], u[8];
  load8(r + c, g);
  load8(r + F + c, u);
  cap_swiglu_n(g, u, form, cap, inv_c);
  int E;
  const uint32_t w = encode8(g, E);
  const size_t i = (size_t)row * F + c;
  *reinterpret_cast<uint32_t*>(codes + i / 2) = w;
  if ((threadIdx.x & 3) == 0) scales[i / 32] = (uint8_t)(E + 127);
}

// Workgroups for n elements at `per` a pass; beyond 2^20 they loop.
static unsigned pass_grid(long n, long per) {
  const long g = (n + per - 1) / per;
  return (unsigned)(g < (1L << 20) ? g : (1L << 20));
}

int launch_mxfp4_encode(int dtype, const void* x, long n, uint8_t* codes, uint8_t* scales, hipStream_t stream) {
  if (n <= 0) return 0;
  const dim3 grid(pass_grid(n, 2048L * kEncUnroll));
  const bool nt = (size_t)n * (dtype == 0 ? 2 : 4) > kStreamBytes;
#define MOE_ENC(T, NT) \
  hipLaunchKernelGGL((k_mxfp4_encode<T, NT>), grid, dim3(256), 0, stream, (const T*)x, n, codes, scales)
  if (dtype == 0) {
    if (nt) MOE_ENC(uint16_t, true);
    else MOE_ENC(uint16_t, false);
  } else {
    if (nt) MOE_ENC(float, true);
    else MOE_ENC(float, false);
  }
#undef MOE_ENC
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

int launch_mxfp4_decode(const uint8_t* codes, const uint8_t* scales, long n, float* out, hipStream_t stream) {
  if (n <= 0) return 0;
  const dim3 grid(pass_grid(n, 1024L * kEncUnroll));
  if ((size_t)n * 4 > kStreamBytes)
    hipLaunchKernelGGL(k_mxfp4_decode<true>, grid, dim3(256), 0, stream, codes, scales, n, out);
  else
    hipLaunchKernelGGL(k_mxfp4_decode<false>, grid, dim3(256), 0, stream, codes, scales, n, out);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

int launch_swiglu_mxfp4(const float* gu, int rows, const int* rows_dev, int F, int form, float cap, uint8_t* codes,
                        uint8_t* scales, hipStream_t stream) {
  if (rows <= 0) return 0;
  hipLaunchKernelGGL(k_swiglu_mxfp4, dim3(rows, ceil_div(F / 8, 256)), dim3(256), 0, stream, gu, rows_dev, F, form,
                     cap, 1.0f / cap, codes, scales);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace moe
