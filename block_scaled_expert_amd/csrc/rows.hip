// Token rows to their experts' rows and back, with the gate weights, and the
// gradients of both.  pos[t k + j] is the row of pair (t, j) (moe_dispatch's
// pair_pos), negative where its expert is elsewhere:
//
//   sort      out[pos[t,j]] = x[t]             its gradient  dx[t] = sum_j d_out[pos[t,j]]
//   combine   out[t] = sum_j w[t,j] y[pos[t,j]]
//             its gradients  dy[pos[t,j]] = w[t,j] d_out[t],  dw[t,j] = <d_out[t], y[pos[t,j]]>
//
// HBM-bound: every token's row is read or written once and every expert row
// once, addressed by token (reading by expert row instead would fetch a token
// k times).  A wavefront has one token, so positions and weights are uniform;
// pairs elsewhere are skipped before any load.  Sums are fp32 in slot order.
#include "operators.h"
#include "row_io.h"

namespace moe {

namespace {

// A token's pairs on this GPU: lane j holds slot j's row (and weight).
struct Pairs {
  int pos;
  float w;
  uint64_t on;
  __device__ Pairs(const RowsArgs& a, int t) {
    const int lane = threadIdx.x & 63;
    const bool slot = lane < a.k;
    pos = slot ? a.pos[(size_t)t * a.k + lane] : -1;
    w = slot && a.w != nullptr ? a.w[(size_t)t * a.k + lane] : 1.0f;
    on = __ballot(pos >= 0 && pos < a.M);
  }
  __device__ int row(int j) const { return __builtin_amdgcn_readlane(pos, j); }
  __device__ float weight(int j) const { return lane_value(w, j); }
};
__device__ inline int next_slot(uint64_t& m) {
  const int j = __builtin_ctzll(m);
  m &= m - 1;
  return j;
}

}  // namespace

// One chunk of 8 columns a thread; blockIdx.x token, blockIdx.y run of columns.
template <typename T, bool VEC, bool NT>
__global__ __launch_bounds__(256) void k_sort_rows(RowsArgs a) {
  const int t = blockIdx.x, c = blockIdx.y * blockDim.x + threadIdx.x;
  Raw8<T> r;
  load_raw8<VEC>(r, static_cast<const T*>(a.token) + (size_t)t * a.cols, c, a.cols);
  const Pairs p(a, t);
  float v[8];
  r.get(v);
  for (uint64_t m = p.on; m != 0;) {
    const int j = next_slot(m);
    store8<VEC, NT>(static_cast<T*>(a.rows_out) + (size_t)p.row(j) * a.cols, c, a.cols, v);
  }
}

constexpr int kSlots = 4;   // rows in flight

template <typename YT, typename OT, bool VEC, bool NT>
__global__ __launch_bounds__(256) void k_combine_rows(RowsArgs a) {
  const int t = blockIdx.x, c = blockIdx.y * blockDim.x + threadIdx.x;
  const Pairs p(a, t);
  float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (uint64_t m = p.on; m != 0;) {
    Raw8<YT> r[kSlots];
    float w[kSlots];
    bool on[kSlots];
    int j = 0;
#pragma unroll
    for (int i = 0; i < kSlots; i++) {   // past the last slot: its row again, unused
      on[i] = m != 0;
      if (on[i]) j = next_slot(m);
      w[i] = p.weight(j);
      load_raw8<VEC, NT>(r[i], static_cast<const YT*>(a.rows_in) + (size_t)p.row(j) * a.cols, c, a.cols);
    }
#pragma unroll
    for (int i = 0; i < kSlots; i++) {
      float v[8];
      r[i].get(v);
#pragma unroll
      for (int e = 0; e < 8; e++) acc[e] = on[i] ? fmaf(w[i], v[e], acc[e]) : acc[e];
    }
  }
  store8<VEC>(static_cast<OT*>(a.token_out) + (size_t)t * a.cols, c, a.cols, acc);
}

// One workgroup per token, whose d_out row stays in registers for all its slots.
template <typename YT, typename OT, bool VEC, bool NT, int CH>
__global__ __launch_bounds__(1024) void k_combine_rows_backward(RowsArgs a) {
  __shared__ float part[32][16];
  const int t = blockIdx.x, tid = threadIdx.x, nt = blockDim.x, waves = nt >> 6;
  float d[CH][8];
  {
    Raw8<OT> r[CH];
#pragma unroll
    for (int i = 0; i < CH; i++)
      load_raw8<VEC>(r[i], static_cast<const OT*>(a.token) + (size_t)t * a.cols, tid + nt * i, a.cols);
#pragma unroll
    for (int i = 0; i < CH; i++) {
      r[i].get(d[i]);
#pragma unroll
      for (int e = 0; e < 8; e++) d[i][e] = in_row<VEC>(tid + nt * i, e, a.cols) ? d[i][e] : 0.0f;
    }
  }
  const Pairs p(a, t);
  for (uint64_t m = p.on; m != 0;) {
    const int j = next_slot(m);
    const size_t at = (size_t)p.row(j) * a.cols;
    const float w = p.weight(j);
    if (a.d_w != nullptr) {
      Raw8<YT> r[CH];
#pragma unroll
      for (int i = 0; i < CH; i++)
        load_raw8<VEC, NT>(r[i], static_cast<const YT*>(a.rows_in) + at, tid + nt * i, a.cols);
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < CH; i++) {
        float y[8];
        r[i].get(y);
#pragma unroll
        for (int e = 0; e < 8; e++) dot = in_row<VEC>(tid + nt * i, e, a.cols) ? fmaf(d[i][e], y[e], dot) : dot;
      }
      dot = wave_total(dot);
      if ((tid & 63) == 0) part[j][tid >> 6] = dot;
    }
    if (a.rows_out != nullptr) {
#pragma unroll
      for (int i = 0; i < CH; i++) {
        float g[8];
#pragma unroll
        for (int e = 0; e < 8; e++) g[e] = w * d[i][e];
        store8<VEC, NT>(static_cast<YT*>(a.rows_out) + at, tid + nt * i, a.cols, g);
      }
    }
  }
  if (a.d_w == nullptr) return;
  lds_barrier();
  if (tid < a.k) {
    float s = 0.0f;
    if (p.on >> tid & 1)
      for (int i = 0; i < waves; i++) s += part[tid][i];
    a.d_w[(size_t)t * a.k + tid] = s;
  }
}

namespace {

// Waves of a workgroup whose threads take one chunk of 8 columns each: those
// that leave the fewest idle over the runs of a row.
int column_waves(int cols) {
  const int n = ceil_div(ceil_div(cols, 8), 64);
  int best = 4;
  for (int w = 3; w >= 1; w--)
    if (ceil_div(n, w) * w < ceil_div(n, best) * best) best = w;
  return best;
}
dim3 column_grid(const RowsArgs& a, int waves) {
  return dim3(a.T, ceil_div(ceil_div(a.cols, 8), 64L * waves));
}

template <typename YT, typename OT, bool VEC, bool NT>
void backward_ch(const RowsArgs& a, hipStream_t s) {
  const int waves = row_waves(a.cols, 4), per = ceil_div(ceil_div(a.cols, 8), 64L * waves);
  const dim3 grid(a.T), block(64 * waves);
  switch (per) {
    case 1: hipLaunchKernelGGL((k_combine_rows_backward<YT, OT, VEC, NT, 1>), grid, block, 0, s, a); break;
    case 2: hipLaunchKernelGGL((k_combine_rows_backward<YT, OT, VEC, NT, 2>), grid, block, 0, s, a); break;
    case 3: hipLaunchKernelGGL((k_combine_rows_backward<YT, OT, VEC, NT, 3>), grid, block, 0, s, a); break;
    case 4: hipLaunchKernelGGL((k_combine_rows_backward<YT, OT, VEC, NT, 4>), grid, block, 0, s, a); break;
    default: hipLaunchKernelGGL((k_combine_rows_backward<YT, OT, VEC, NT, 8>), grid, block, 0, s, a); break;
  }
}

// Bytes of the expert rows of a call.
size_t row_bytes(const RowsArgs& a, int dtype) { return (size_t)a.M * a.cols * (dtype == 0 ? 2 : 4); }

}  // namespace

#define MOE_ROWS_BOOL(flag, N, ...)  \
  do {                               \
    if (flag) {                      \
      constexpr bool N = true;       \
      __VA_ARGS__;                   \
    } else {                         \
      constexpr bool N = false;      \
      __VA_ARGS__;                   \
    }                                \
  } while (0)
#define MOE_ROWS_TYPE(dtype, N, ...) \
  do {                               \
    if ((dtype) == 0) {              \
      typedef uint16_t N;            \
      __VA_ARGS__;                   \
    } else {                         \
      typedef float N;               \
      __VA_ARGS__;                   \
    }                                \
  } while (0)

int launch_sort_rows(const RowsArgs& a, hipStream_t s) {
  if (a.T <= 0) return 0;
  const int waves = column_waves(a.cols);
  const bool vec = a.cols % 8 == 0 && aligned16(a.token) && aligned16(a.rows_out);
  const bool nt = row_bytes(a, a.row_dtype) > kStreamBytes;
  MOE_ROWS_TYPE(a.row_dtype, T, MOE_ROWS_BOOL(vec, VEC, MOE_ROWS_BOOL(nt, NT, hipLaunchKernelGGL((k_sort_rows<T, VEC, NT>), column_grid(a, waves), dim3(64 * waves), 0, s, a))));
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

int launch_combine_rows(const RowsArgs& a, hipStream_t s) {
  if (a.T <= 0) return 0;
  const int waves = column_waves(a.cols);
  const bool vec = a.cols % 8 == 0 && aligned16(a.token_out) && aligned16(a.rows_in);
  const bool nt = row_bytes(a, a.row_dtype) > kStreamBytes;
  MOE_ROWS_TYPE(a.row_dtype, YT, MOE_ROWS_TYPE(a.token_dtype, OT, MOE_ROWS_BOOL(vec, VEC, MOE_ROWS_BOOL(nt, NT,
      hipLaunchKernelGGL((k_combine_rows<YT, OT, VEC, NT>), column_grid(a, waves), dim3(64 * waves), 0, s, a)))));
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

int launch_combine_rows_backward(const RowsArgs& a, hipStream_t s) {
  if (a.T <= 0) return 0;
  const bool vec = a.cols % 8 == 0 && aligned16(a.token) && aligned16(a.rows_in) && aligned16(a.rows_out);
  const bool nt = row_bytes(a, a.row_dtype) > kStreamBytes;
  MOE_ROWS_TYPE(a.row_dtype, YT, MOE_ROWS_TYPE(a.token_dtype, OT, MOE_ROWS_BOOL(vec, VEC, MOE_ROWS_BOOL(nt, NT,
      (backward_ch<YT, OT, VEC, NT>(a, s))))));
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace moe
