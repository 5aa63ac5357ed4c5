// Residual addition, root-mean-square norm and the encoding of the normed
// rows in one pass; and the norm's gradient.
//
//   s = x + residual (rounded to the stream's type; x alone without one)
//   r = (mean s^2 + eps)^(-1/2),  y = s r w  (rounded to x's type)
//   codes, scales: of y as stored, as moe_quantize_act gives them
//
// With n = s r and a = dy w (n's mean square is 1 up to eps):
//   ds = r (a - n mean(a n)) + what reaches s from further on
//   dw = sum over rows of dy n
//
// HBM-bound for many rows, launch-bound for few: one workgroup holds a row in
// registers from its only load to its stores.  Sums are taken in a fixed order
// (lane, wave, workgroup; dw: a workgroup's rows, then the workgroups), those of
// squares in 64 bits, the others in fp32.  Measured, 16384 x 4608 (TB/s of what
// has to move): bf16 with MXFP8 codes 113 us (6.0), MXFP4 109 (5.9), NVFP4 110
// (5.9), bf16 x and an fp32 stream 162 (5.6), its gradient 221 (5.5) and 4.1 for
// dw; 64 rows with codes 4.0.  Wide rows: registers go to scratch in the gradient,
// up to 72 bytes a lane above 6144 columns where x or the stream is fp32, up to 76
// above 12288, 300 to 700 above 16384 and 1400 to 1900 above 32768, where the
// forward has 76 to 192 (4000 x 16384 with an fp32 stream 148 and 215 us, 5.3 and
// 4.9; 2000 x 32768 151 and 687, 5.2 and 1.5; 1000 x 65536 230 and 1066, 3.4 and 1.0).
#include "operators.h"
#include "quant_row.h"
#include "row_io.h"

namespace moe {

namespace {

// Largest |v| of aligned groups of N lanes (2 or 4).
template <int N>
__device__ inline float lanes_max(float v) {
  v = fmaxf(v, bits_f((uint32_t)__builtin_amdgcn_update_dpp(0, (int)f_bits(v), 0xB1, 0xF, 0xF, false)));
  if constexpr (N == 4)
    v = fmaxf(v, bits_f((uint32_t)__builtin_amdgcn_update_dpp(0, (int)f_bits(v), 0x4E, 0xF, 0xF, false)));
  return v;
}
__device__ inline float amax8(const float* v) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; i++) m = fmaxf(m, fabsf(v[i]));   // a NaN is passed over
  return m;
}

// This lane's 8 elements of a row as MXFP8 (2) or MXFP4 (4); a block of 32 is 4 lanes'.
template <int FMT>
__device__ inline void encode_mx(float* v, int c, uint8_t* codes, uint8_t* scales, bool on) {
  const float am = lanes_max<4>(amax8(v));
  const int E = FMT == 2 ? mx_exponent(am) : mxfp4_exponent(am);
  const float step = pow2f(-E);
  if constexpr (FMT == 2) {
    const uint32_t lo = e4m3_pack4(__fmul_rn(v[0], step), __fmul_rn(v[1], step), __fmul_rn(v[2], step), __fmul_rn(v[3], step));
    const uint32_t hi = e4m3_pack4(__fmul_rn(v[4], step), __fmul_rn(v[5], step), __fmul_rn(v[6], step), __fmul_rn(v[7], step));
    if (on) reinterpret_cast<uint2*>(codes)[c] = make_uint2(lo, hi);
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = v[i] == v[i] ? v[i] : 0.0f;
    const uint32_t w = e2m1_pack8(v, step);
    if (on) reinterpret_cast<uint32_t*>(codes)[c] = w;
  }
  if (on && (c & 3) == 0) scales[c / 4] = (uint8_t)(E + 127);
}

// The same as NVFP4 under the row's scale gs; a block of 16 is 2 lanes'.
__device__ inline void encode_nv(const float* v, int c, float gs, bool zero_row, uint8_t* codes, uint8_t* scales,
                                 bool on) {
#pragma clang fp contract(off)
  const float ab = lanes_max<2>(amax8(v));
  const uint32_t sc = e4m3_hw(__fdiv_rn(ab, __fmul_rn(6.0f, gs)));
  const float sigma = e4m3_decode(sc);
  uint32_t w = 0;
  if (!zero_row && sigma != 0.0f) {
    const float r = __fdiv_rn(1.0f, __fmul_rn(sigma, gs));
    if (r <= 3.4028235e38f) {
      w = e2m1_pack8(v, r);
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++) w |= e2m1_encode(__fmul_rn(v[i], r)) << (4 * i);
    }
  }
  if (on) {
    reinterpret_cast<uint32_t*>(codes)[c] = w;
    if ((c & 1) == 0) scales[c / 2] = (uint8_t)(zero_row ? 0u : sc);
  }
}

// v[k] = v[k] r w[k] as XT holds it, r = rstd + rest.  With the squares summed in
// 64 bits and the errors of the products carried along, what is rounded to fp32 is
// within 2^-45 of the exact value (e is exact up to its last rounding, 2^-47 of p;
// the sum of the errors likewise), as long as the errors themselves are above
// fp32's least numbers.  Where y lies next to a bf16 step, and its code next to a
// step of the format, both then fall on the definition's side (16384 x 4608 to
// MXFP8: no code off, where 20 to 70 were in plain fp32; the time is the memory's
// still).
template <typename XT, int N>
__device__ inline void normed(float (&v)[N], const float (&w)[N], float rstd, float rest) {
#pragma clang fp contract(off)
#pragma unroll
  for (int k = 0; k < N; k++) {
    const float p = v[k] * rstd, e = fmaf(v[k], rest, fmaf(v[k], rstd, -p));
    const float q = p * w[k], y = q + fmaf(e, w[k], fmaf(p, w[k], -q));
    v[k] = stored<XT>(y == y && q != 0.0f ? y : q);   // inf: q has it, the errors are NaN; zero: q has the sign
  }
}

// Sum of a 64-bit value over the workgroup.  Every thread calls it.
template <int CTRL>
__device__ inline double dpp_plus64(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xF, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, 0xF, 0xF, false);
  return v + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ inline double group_total64(double v, double* red) {
  v = dpp_plus64<0xB1>(v);    // quad_perm [1,0,3,2]
  v = dpp_plus64<0x4E>(v);    // quad_perm [2,3,0,1]
  v = dpp_plus64<0x141>(v);   // row_half_mirror
  v = dpp_plus64<0x140>(v);   // row_mirror
  if ((threadIdx.x & 15) == 0) red[threadIdx.x >> 4] = v;
  lds_barrier();
  double s = red[0];
  for (int i = 1; i < (int)(blockDim.x >> 4); i++) s += red[i];
  return s;
}

__device__ inline float group_amax(float v, float* red) {
  v = wave_max(v);
  const int waves = blockDim.x >> 6;
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  lds_barrier();
  float m = red[0];
  for (int i = 1; i < waves; i++) m = fmaxf(m, red[i]);
  return m;
}

}  // namespace

// One workgroup per row.  RT: the stream's type.  FMT: 0 no codes.
template <typename XT, typename RT, int FMT, bool FULL, int CH, bool NT>
__global__ __launch_bounds__(1024) void k_norm_forward(NormArgs a) {
  __shared__ double sums[64];
  __shared__ float red[16];
  typedef Span<FULL, CH> S;
  const S sp(a.cols, blockDim.x);
  const int cols = a.cols;
  const size_t at = (size_t)blockIdx.x * cols;
  const RT* const res = static_cast<const RT*>(a.res);

  typename S::template Raw<XT> rx;
  typename S::template Raw<RT> rr;
  sp.template load<NT>(rx, static_cast<const XT*>(a.x) + at);
  if (res != nullptr) sp.template load<NT>(rr, res + at);
  float v[S::N];
  double ss = 0.0;
  sp.get(rx, v);
  if (res != nullptr) {
    float u[S::N];
    sp.get(rr, u);
#pragma unroll
    for (int k = 0; k < S::N; k++) v[k] = stored<RT>(v[k] + u[k]);
  }
#pragma unroll
  for (int k = 0; k < S::N; k++) {
    v[k] = sp.has(k) ? v[k] : 0.0f;
    ss = fma((double)v[k], (double)v[k], ss);
  }
  if (a.res_out != nullptr) sp.template put<NT>(static_cast<RT*>(a.res_out) + at, v);
  typename S::template Raw<float> rw;
  sp.load(rw, a.weight);
  const double r = rsqrt(group_total64(ss, sums) * a.inv_cols + (double)a.eps);
  const float rstd = (float)r, rest = (float)(r - (double)rstd);
  if (a.rstd != nullptr && threadIdx.x == 0) a.rstd[blockIdx.x] = rstd;

  float w[S::N];
  sp.get(rw, w);
  normed<XT>(v, w, rstd, rest);
  if (a.y != nullptr) sp.template put<NT>(static_cast<XT*>(a.y) + at, v);

  const size_t row = blockIdx.x;
  if constexpr (FMT == 2 || FMT == 4) {
    uint8_t* const codes = a.codes + row * (FMT == 2 ? cols : cols / 2);
#pragma unroll
    for (int i = 0; i < CH; i++)
      encode_mx<FMT>(v + 8 * i, sp.piece(i), codes, a.scales + row * (cols / 32), sp.has(8 * i));
  }
  if constexpr (FMT == 1) {
    float gs = a.gs_val;
    bool zero_row = false;
    if (a.gs_row) {
      float A = 0.0f;
#pragma unroll
      for (int i = 0; i < CH; i++) A = fmaxf(A, sp.has(8 * i) ? amax8(v + 8 * i) : 0.0f);
      A = group_amax(A, red);
      zero_row = A == 0.0f;
      gs = nvfp4_gs(A);
    }
    if (threadIdx.x == 0) a.row_gs[row] = gs;
#pragma unroll
    for (int i = 0; i < CH; i++)
      encode_nv(v + 8 * i, sp.piece(i), gs, zero_row, a.codes + row * (cols / 2), a.scales + row * (cols / 16),
                sp.has(8 * i));
  }
}

// Rows blockIdx, blockIdx + grid, ..; this workgroup's share of dw stays in
// registers and goes to partial[blockIdx].  AHEAD (up to 8 waves, which leave the
// registers for it): the next row's loads go out before this row's stores,
// behind which they would wait for them (memory operations complete in order):
// 16384 x 4608 with an fp32 stream 241 us instead of 273.
template <typename XT, typename RT, bool FULL, int CH, int TB, bool NT>
__global__ __launch_bounds__(TB) void k_norm_backward(NormGradArgs a) {
  __shared__ float red[2][16];
  typedef Span<FULL, CH> S;
  const S sp(a.cols, blockDim.x);
  const XT* const dy = static_cast<const XT*>(a.dy);
  const RT* const res = static_cast<const RT*>(a.res);
  const RT* const next = static_cast<const RT*>(a.d_res_out);
  constexpr bool AHEAD = TB <= 512;
  float w[S::N], acc[S::N];
  auto fetch_weight = [&]() {
    typename S::template Raw<float> rw;
    sp.load(rw, a.weight);
    sp.get(rw, w);
  };
  if (AHEAD) fetch_weight();
#pragma unroll
  for (int k = 0; k < S::N; k++) acc[k] = 0.0f;

  typename S::template Raw<XT> rdy;
  typename S::template Raw<RT> rs, rn;
  float rstd_raw;
  auto fetch = [&](int t) {
    const size_t at = (size_t)t * a.cols;
    rstd_raw = a.rstd[t];
    sp.template load<NT>(rdy, dy + at);
    sp.template load<NT>(rs, res + at);
    if (next != nullptr) sp.template load<NT>(rn, next + at);
  };
  if (AHEAD) fetch(blockIdx.x);
  int turn = 0;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
    const size_t at = (size_t)t * a.cols;
    if (!AHEAD) {
      fetch(t);
      fetch_weight();
    }
    const float rstd = rstd_raw;
    float n[S::N], g[S::N], d[S::N], dot = 0.0f;
    sp.get(rdy, g);
    sp.get(rs, n);
#pragma unroll
    for (int k = 0; k < S::N; k++) {
      n[k] = sp.has(k) ? n[k] * rstd : 0.0f;
      const float gn = sp.has(k) ? g[k] * n[k] : 0.0f;
      acc[k] += gn;
      dot = fmaf(gn, w[k], dot);
    }
    if (AHEAD) {
      if (next != nullptr) sp.get(rn, d);
      fetch(min(t + (int)gridDim.x, a.T - 1));
    }
    dot = group_total(dot, red[turn]) / (float)a.cols;
#pragma unroll
    for (int k = 0; k < S::N; k++) {
      if (!AHEAD && k == 0 && next != nullptr) sp.get(rn, d);
      const float v = rstd * (g[k] * w[k] - n[k] * dot);
      d[k] = next != nullptr ? v + d[k] : v;
    }
    sp.template put<NT>(static_cast<RT*>(a.d_res) + at, d);
    if (a.dx != nullptr) sp.template put<NT>(static_cast<XT*>(a.dx) + at, d);
  }
  if (a.partial != nullptr) {
    float* const row = a.partial + (size_t)blockIdx.x * a.pitch;
    sp.put(row, acc);
  }
}

// dw: the partial rows added up, 32 columns a workgroup; run r of 128 takes rows
// r, r + 128, .., then 8 threads a column 16 runs each, then one those 8.
__global__ __launch_bounds__(1024) void k_norm_dw(const float* __restrict__ partial, int n, int cols, int pitch,
                                                  float* __restrict__ dw) {
  __shared__ v4f part[128][8];
  const int c = threadIdx.x & 7, run = threadIdx.x >> 3, col = blockIdx.x * 32 + 4 * c;
  v4f s = v4f{0, 0, 0, 0};
  if (col < pitch) {
    const float* p = partial + col;
    int i = run;
    for (; i + 3 * 128 < n; i += 4 * 128) {
      v4f v[4];
#pragma unroll
      for (int j = 0; j < 4; j++) v[j] = *reinterpret_cast<const v4f*>(p + (size_t)(i + 128 * j) * pitch);
#pragma unroll
      for (int j = 0; j < 4; j++) s += v[j];
    }
    for (; i < n; i += 128) s += *reinterpret_cast<const v4f*>(p + (size_t)i * pitch);
  }
  part[run][c] = s;
  __syncthreads();
  if (run < 8)
    for (int i = run + 8; i < 128; i += 8) s += part[i][c];
  __syncthreads();
  if (run < 8) part[run][c] = s;
  __syncthreads();
  if (run == 0) {
    for (int i = 1; i < 8; i++) s += part[i][c];
#pragma unroll
    for (int e = 0; e < 4; e++)
      if (col + e < cols) dw[col + e] = s[e];
  }
}

namespace {

template <typename XT, typename RT, int FMT, bool FULL, bool NT>
void forward_ch(const NormArgs& a, hipStream_t s) {
  const int waves = row_waves(a.cols, 4);
  MOE_ROW_PIECES(row_pieces(a.cols, waves),
                 hipLaunchKernelGGL((k_norm_forward<XT, RT, FMT, FULL, CH, NT>), dim3(a.T), dim3(64 * waves), 0, s, a))
}
template <typename XT, typename RT, bool NT>
void forward_fmt(const NormArgs& a, bool full, hipStream_t s) {
  if (a.fmt == 1) forward_ch<XT, RT, 1, true, NT>(a, s);
  else if (a.fmt == 2) forward_ch<XT, RT, 2, true, NT>(a, s);
  else if (a.fmt == 4) forward_ch<XT, RT, 4, true, NT>(a, s);
  else if (full) forward_ch<XT, RT, 0, true, NT>(a, s);
  else forward_ch<XT, RT, 0, false, NT>(a, s);
}
template <typename XT, typename RT>
void forward_nt(const NormArgs& a, bool full, hipStream_t s) {
  const size_t bytes = (size_t)a.T * a.cols * (sizeof(XT) + sizeof(RT));
  if (bytes > kStreamBytes) forward_fmt<XT, RT, true>(a, full, s);
  else forward_fmt<XT, RT, false>(a, full, s);
}

// Waves of a row's workgroup in the gradient, and workgroups.
int gradient_waves(int cols) { return row_waves(cols, row_waves(cols, 3) <= 8 ? 3 : 2); }
// More of them for short rows, which need more in flight, as long as their partial
// sums stay small: 65536 x 256 took 126 us with 512, 67 with 4096.
int gradient_groups(int T, int cols) {
  const int n = (256 * 4608) / cols;
  const int g = n < 512 ? 512 : n < 4096 ? n : 4096;
  return T < g ? T : g;
}
int partial_pitch(int cols) { return (int)align_up(cols, 8); }

// Pieces of a thread by waves (gradient_waves, row_pieces): up to 4 waves 1 to 3,
// 5 to 8 waves 3, above 2, 3, 4 or 8.
template <typename XT, typename RT, bool FULL, bool NT>
void backward_ch(const NormGradArgs& a, int grid, hipStream_t s) {
  const int waves = gradient_waves(a.cols), pieces = row_pieces(a.cols, waves);
#define MOE_NORM_BACKWARD(CH, TB) \
  hipLaunchKernelGGL((k_norm_backward<XT, RT, FULL, CH, TB, NT>), dim3(grid), dim3(64 * waves), 0, s, a)
  if (waves <= 4) {
    if (pieces == 1) MOE_NORM_BACKWARD(1, 256);
    else if (pieces == 2) MOE_NORM_BACKWARD(2, 256);
    else MOE_NORM_BACKWARD(3, 256);
  } else if (waves <= 8) {
    MOE_NORM_BACKWARD(3, 512);
  } else {
    if (pieces == 2) MOE_NORM_BACKWARD(2, 1024);
    else if (pieces == 3) MOE_NORM_BACKWARD(3, 1024);
    else if (pieces == 4) MOE_NORM_BACKWARD(4, 1024);
    else MOE_NORM_BACKWARD(8, 1024);
  }
#undef MOE_NORM_BACKWARD
}
template <typename XT, typename RT>
void backward_full(const NormGradArgs& a, bool full, int grid, hipStream_t s) {
  const bool nt = (size_t)a.T * a.cols * (sizeof(XT) + sizeof(RT)) > kStreamBytes;
  if (full && nt) backward_ch<XT, RT, true, true>(a, grid, s);
  else if (full) backward_ch<XT, RT, true, false>(a, grid, s);
  else if (nt) backward_ch<XT, RT, false, true>(a, grid, s);
  else backward_ch<XT, RT, false, false>(a, grid, s);
}

}  // namespace

size_t norm_ws_bytes(int T, int cols) {
  return align_up((size_t)gradient_groups(T, cols) * partial_pitch(cols) * 4, 256);
}

int launch_norm_forward(NormArgs a, hipStream_t stream) {
  if (a.T <= 0) return 0;
  a.inv_cols = 1.0 / a.cols;
  const bool full = a.cols % 8 == 0 && aligned16(a.x) && aligned16(a.res) && aligned16(a.res_out) && aligned16(a.y) &&
                    aligned16(a.weight);
  if (a.dtype == 0 && a.res_dtype == 0) forward_nt<uint16_t, uint16_t>(a, full, stream);
  else if (a.dtype == 0) forward_nt<uint16_t, float>(a, full, stream);
  else forward_nt<float, float>(a, full, stream);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

int launch_norm_backward(NormGradArgs a, float* d_weight, void* ws, hipStream_t stream) {
  const bool full = a.cols % 8 == 0 && aligned16(a.dy) && aligned16(a.res) && aligned16(a.d_res_out) &&
                    aligned16(a.weight) && aligned16(a.d_res) && aligned16(a.dx);
  const int grid = gradient_groups(a.T, a.cols);
  a.partial = d_weight == nullptr ? nullptr : static_cast<float*>(ws);
  a.pitch = partial_pitch(a.cols);
  if (a.T > 0) {
    if (a.dtype == 0 && a.res_dtype == 0) backward_full<uint16_t, uint16_t>(a, full, grid, stream);
    else if (a.dtype == 0) backward_full<uint16_t, float>(a, full, grid, stream);
    else backward_full<float, float>(a, full, grid, stream);
  }
  if (d_weight != nullptr)
    hipLaunchKernelGGL(k_norm_dw, dim3(ceil_div(a.cols, 32)), dim3(1024), 0, stream, a.partial, grid, a.cols, a.pitch,
                       d_weight);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace moe
