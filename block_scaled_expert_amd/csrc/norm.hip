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
// HBM-bound for many rows, launch-bound for few: a row is held in registers by
// one workgroup from its only load to its stores.  All sums are fp32 in a fixed
// order (lane, wave, workgroup; dw: a workgroup's rows, then the workgroups).
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
__device__ inline float amax8(const float (&v)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; i++) m = fmaxf(m, fabsf(v[i]));   // a NaN is passed over
  return m;
}

// This lane's 8 elements of a row as MXFP8 (2) or MXFP4 (4); a block of 32 is 4 lanes'.
template <int FMT>
__device__ inline void encode_mx(float (&v)[8], int c, uint8_t* codes, uint8_t* scales, bool on) {
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
__device__ inline void encode_nv(const float (&v)[8], int c, float gs, bool zero_row, uint8_t* codes, uint8_t* scales,
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

// One workgroup per row; lane chunk c = thread + blockDim i, i < CH.  RT: the
// stream's type.  FMT: 0 no codes.
template <typename XT, typename RT, int FMT, bool VEC, int CH>
__global__ __launch_bounds__(1024) void k_norm_forward(NormArgs a) {
  __shared__ float red[2][16];
  const int tid = threadIdx.x, nt = blockDim.x, cols = a.cols;
  const size_t row = blockIdx.x;
  const XT* const x = static_cast<const XT*>(a.x) + row * cols;
  const RT* const res = a.res == nullptr ? nullptr : static_cast<const RT*>(a.res) + row * cols;

  Raw8<XT> rx[CH];
  Raw8<RT> rr[CH];
#pragma unroll
  for (int i = 0; i < CH; i++) load_raw8<VEC>(rx[i], x, tid + nt * i, cols);
  if (res != nullptr) {
#pragma unroll
    for (int i = 0; i < CH; i++) load_raw8<VEC>(rr[i], res, tid + nt * i, cols);
  }
  float v[CH][8], ss = 0.0f;
#pragma unroll
  for (int i = 0; i < CH; i++) {
    const int c = tid + nt * i;
    rx[i].get(v[i]);
    if (res != nullptr) {
      float u[8];
      rr[i].get(u);
#pragma unroll
      for (int e = 0; e < 8; e++) v[i][e] = stored<RT>(v[i][e] + u[e]);
    }
#pragma unroll
    for (int e = 0; e < 8; e++) {
      v[i][e] = in_row<VEC>(c, e, cols) ? v[i][e] : 0.0f;
      ss = fmaf(v[i][e], v[i][e], ss);
    }
    if (a.res_out != nullptr) store8<VEC>(static_cast<RT*>(a.res_out) + row * cols, c, cols, v[i]);
  }
  ss = group_total(ss, red[0]);
  const float rstd = 1.0f / sqrtf(ss / (float)cols + a.eps);
  if (a.rstd != nullptr && tid == 0) a.rstd[row] = rstd;

#pragma unroll
  for (int i = 0; i < CH; i++) {
    const int c = tid + nt * i;
    Raw8<float> rw;
    load_raw8<VEC>(rw, a.weight, c, cols);
    float w[8];
    rw.get(w);
#pragma unroll
    for (int e = 0; e < 8; e++) v[i][e] = stored<XT>(v[i][e] * rstd * w[e]);
    if (a.y != nullptr) store8<VEC>(static_cast<XT*>(a.y) + row * cols, c, cols, v[i]);
  }
  if constexpr (FMT == 2 || FMT == 4) {
    uint8_t* const codes = a.codes + row * (FMT == 2 ? cols : cols / 2);
#pragma unroll
    for (int i = 0; i < CH; i++)
      encode_mx<FMT>(v[i], tid + nt * i, codes, a.scales + row * (cols / 32), 8 * (tid + nt * i) < cols);
  }
  if constexpr (FMT == 1) {
    float gs = a.gs_val;
    bool zero_row = false;
    if (a.gs_row) {
      float A = 0.0f;
#pragma unroll
      for (int i = 0; i < CH; i++) A = fmaxf(A, 8 * (tid + nt * i) < cols ? amax8(v[i]) : 0.0f);
      A = group_amax(A, red[1]);
      zero_row = A == 0.0f;
      gs = nvfp4_gs(A);
    }
    if (tid == 0) a.row_gs[row] = gs;
#pragma unroll
    for (int i = 0; i < CH; i++)
      encode_nv(v[i], tid + nt * i, gs, zero_row, a.codes + row * (cols / 2), a.scales + row * (cols / 16),
                8 * (tid + nt * i) < cols);
  }
}

// Rows blockIdx, blockIdx + grid, ..; this workgroup's share of dw stays in
// registers and goes to partial[blockIdx].
template <typename XT, typename RT, bool VEC, int CH>
__global__ __launch_bounds__(1024) void k_norm_backward(NormGradArgs a) {
  __shared__ float red[2][16];
  const int tid = threadIdx.x, nt = blockDim.x, cols = a.cols;
  float w[CH][8], acc[CH][8];
#pragma unroll
  for (int i = 0; i < CH; i++) {
    Raw8<float> rw;
    load_raw8<VEC>(rw, a.weight, tid + nt * i, cols);
    rw.get(w[i]);
#pragma unroll
    for (int e = 0; e < 8; e++) acc[i][e] = 0.0f;
  }
  int turn = 0;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
    const size_t at = (size_t)t * cols;
    Raw8<XT> rdy[CH];
    Raw8<RT> rs[CH], rn[CH];
#pragma unroll
    for (int i = 0; i < CH; i++) {
      load_raw8<VEC>(rdy[i], static_cast<const XT*>(a.dy) + at, tid + nt * i, cols);
      load_raw8<VEC>(rs[i], static_cast<const RT*>(a.res) + at, tid + nt * i, cols);
    }
    if (a.d_res_out != nullptr) {
#pragma unroll
      for (int i = 0; i < CH; i++) load_raw8<VEC>(rn[i], static_cast<const RT*>(a.d_res_out) + at, tid + nt * i, cols);
    }
    const float rstd = a.rstd[t];
    float n[CH][8], g[CH][8], dot = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; i++) {
      rdy[i].get(g[i]);
      rs[i].get(n[i]);
#pragma unroll
      for (int e = 0; e < 8; e++) {
        const bool in = in_row<VEC>(tid + nt * i, e, cols);
        n[i][e] = in ? n[i][e] * rstd : 0.0f;
        const float gn = in ? g[i][e] * n[i][e] : 0.0f;
        acc[i][e] += gn;
        dot = fmaf(gn, w[i][e], dot);
      }
    }
    dot = group_total(dot, red[turn]) / (float)cols;
#pragma unroll
    for (int i = 0; i < CH; i++) {
      float d[8];
#pragma unroll
      for (int e = 0; e < 8; e++) d[e] = rstd * (g[i][e] * w[i][e] - n[i][e] * dot);
      if (a.d_res_out != nullptr) {
        float u[8];
        rn[i].get(u);
#pragma unroll
        for (int e = 0; e < 8; e++) d[e] += u[e];
      }
      store8<VEC>(static_cast<RT*>(a.d_res) + at, tid + nt * i, cols, d);
      if (a.dx != nullptr) store8<VEC>(static_cast<XT*>(a.dx) + at, tid + nt * i, cols, d);
    }
  }
  if (a.partial != nullptr) {
#pragma unroll
    for (int i = 0; i < CH; i++) store8<VEC>(a.partial + (size_t)blockIdx.x * cols, tid + nt * i, cols, acc[i]);
  }
}

// dw: the partial rows added in order, 32 columns a workgroup, 8 runs of rows.
__global__ __launch_bounds__(256) void k_norm_dw(const float* __restrict__ partial, int n, int cols,
                                                 float* __restrict__ dw) {
  __shared__ float part[8][32];
  const int c = threadIdx.x & 31, run = threadIdx.x >> 5, col = blockIdx.x * 32 + c;
  const int lo = (long)run * n / 8, hi = (long)(run + 1) * n / 8;
  float s = 0.0f;
  for (int i = lo; i < hi; i++) s += col < cols ? partial[(size_t)i * cols + col] : 0.0f;
  part[run][c] = s;
  __syncthreads();
  if (run == 0 && col < cols) {
    for (int i = 1; i < 8; i++) s += part[i][c];
    dw[col] = s;
  }
}

namespace {

constexpr int kRowPieces = 4;   // of 8 elements a lane; 8 in the widest rows

// Pieces a lane has in a workgroup of row_waves.
int row_pieces(int cols, int waves) {
  const int n = ceil_div(ceil_div(cols, 8), 64L * waves);
  return n > 4 ? 8 : n;
}

template <typename XT, typename RT, int FMT, bool VEC>
void forward_ch(const NormArgs& a, hipStream_t s) {
  const int waves = row_waves(a.cols, kRowPieces);
  const dim3 grid(a.T), block(64 * waves);
  switch (row_pieces(a.cols, waves)) {
    case 1: hipLaunchKernelGGL((k_norm_forward<XT, RT, FMT, VEC, 1>), grid, block, 0, s, a); break;
    case 2: hipLaunchKernelGGL((k_norm_forward<XT, RT, FMT, VEC, 2>), grid, block, 0, s, a); break;
    case 3: hipLaunchKernelGGL((k_norm_forward<XT, RT, FMT, VEC, 3>), grid, block, 0, s, a); break;
    case 4: hipLaunchKernelGGL((k_norm_forward<XT, RT, FMT, VEC, 4>), grid, block, 0, s, a); break;
    default: hipLaunchKernelGGL((k_norm_forward<XT, RT, FMT, VEC, 8>), grid, block, 0, s, a); break;
  }
}
template <typename XT, typename RT>
void forward_fmt(const NormArgs& a, bool vec, hipStream_t s) {
  if (a.fmt == 1) forward_ch<XT, RT, 1, true>(a, s);
  else if (a.fmt == 2) forward_ch<XT, RT, 2, true>(a, s);
  else if (a.fmt == 4) forward_ch<XT, RT, 4, true>(a, s);
  else if (vec) forward_ch<XT, RT, 0, true>(a, s);
  else forward_ch<XT, RT, 0, false>(a, s);
}

template <typename XT, typename RT, bool VEC>
void backward_ch(const NormGradArgs& a, int grid, hipStream_t s) {
  const int waves = row_waves(a.cols, kRowPieces);
  const dim3 block(64 * waves);
  switch (row_pieces(a.cols, waves)) {
    case 1: hipLaunchKernelGGL((k_norm_backward<XT, RT, VEC, 1>), dim3(grid), block, 0, s, a); break;
    case 2: hipLaunchKernelGGL((k_norm_backward<XT, RT, VEC, 2>), dim3(grid), block, 0, s, a); break;
    case 3: hipLaunchKernelGGL((k_norm_backward<XT, RT, VEC, 3>), dim3(grid), block, 0, s, a); break;
    case 4: hipLaunchKernelGGL((k_norm_backward<XT, RT, VEC, 4>), dim3(grid), block, 0, s, a); break;
    default: hipLaunchKernelGGL((k_norm_backward<XT, RT, VEC, 8>), dim3(grid), block, 0, s, a); break;
  }
}

// Workgroups of the gradient of T rows.
int gradient_groups(int T) { return T < 1024 ? T : 1024; }

}  // namespace

size_t norm_ws_bytes(int T, int cols) { return align_up((size_t)gradient_groups(T) * cols * 4, 256); }

int launch_norm_forward(const NormArgs& a, hipStream_t stream) {
  if (a.T <= 0) return 0;
  const bool vec = a.cols % 8 == 0 && aligned16(a.x) && aligned16(a.res) && aligned16(a.res_out) && aligned16(a.y) &&
                   aligned16(a.weight);
  if (a.dtype == 0 && a.res_dtype == 0) forward_fmt<uint16_t, uint16_t>(a, vec, stream);
  else if (a.dtype == 0) forward_fmt<uint16_t, float>(a, vec, stream);
  else forward_fmt<float, float>(a, vec, stream);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

int launch_norm_backward(NormGradArgs a, float* d_weight, void* ws, hipStream_t stream) {
  const bool vec = a.cols % 8 == 0 && aligned16(a.dy) && aligned16(a.res) && aligned16(a.d_res_out) &&
                   aligned16(a.weight) && aligned16(a.d_res) && aligned16(a.dx);
  const int grid = gradient_groups(a.T);
  a.partial = d_weight == nullptr ? nullptr : static_cast<float*>(ws);
  if (a.T > 0) {
#define MOE_NORM_BACK(XT, RT)                            \
  do {                                                   \
    if (vec) backward_ch<XT, RT, true>(a, grid, stream); \
    else backward_ch<XT, RT, false>(a, grid, stream);    \
  } while (0)
    if (a.dtype == 0 && a.res_dtype == 0) MOE_NORM_BACK(uint16_t, uint16_t);
    else if (a.dtype == 0) MOE_NORM_BACK(uint16_t, float);
    else MOE_NORM_BACK(float, float);
#undef MOE_NORM_BACK
  }
  if (d_weight != nullptr)
    hipLaunchKernelGGL(k_norm_dw, dim3(ceil_div(a.cols, 32)), dim3(256), 0, stream, a.partial, grid, a.cols, d_weight);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace moe
