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
// Measured, 16384 tokens of 4608, 8 slots, us (TB/s of what has to move): all local
// in bf16, sort 282 (4.8), combine 235 (5.8), its gradients 504 (5.1), sort's 234
// (5.8), the four in turn 1300 (5.1); with fp32 expert rows combine 492 (5.2), its
// gradients 1000 (5.1), the four 2055; an eighth local with fp32 expert rows 54, 90
// (5.0), 150 (5.0), 46, the four 326 to 385 on different machines (4.7 to 5.5).
// 64 tokens: sort 2.8 us, combine of fp32 rows 4.2.  For 1024 and more tokens of rows
// off 8 elements or 16 bytes and above 1031 columns, four slots do not fit the
// registers that the combine's bound of 1024 threads leaves: 8 to 408 bytes a lane go
// to scratch; above 32768 columns 40 to 1320 in any rows (its gradients 268 to 492).
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

// blockIdx.x token, blockIdx.y run of columns (one for many tokens).
template <typename T, bool FULL, int CH, bool NT>
__global__ __launch_bounds__(1024) void k_sort_rows(RowsArgs a) {
  typedef Span<FULL, CH> S;
  const int t = blockIdx.x;
  const S sp(a.cols, blockDim.x, blockIdx.y * blockDim.x * CH);
  typename S::template Raw<T> r;
  sp.template load<NT>(r, static_cast<const T*>(a.token) + (size_t)t * a.cols);
  const Pairs p(a, t);
  for (uint64_t m = p.on; m != 0;)
    sp.template store<NT>(static_cast<T*>(a.rows_out) + (size_t)p.row(next_slot(m)) * a.cols, r);
}

// acc += the next n of the slots in m, whose loads go out together (at 3 and 4 pieces
// of fp32 rows the compiler leaves fewer registers than four slots take, and fewer
// are out at a time).
template <int n, bool NT, typename YT, typename S>
__device__ inline void add_slots(const RowsArgs& a, const S& sp, const Pairs& p, uint64_t& m, float (&acc)[S::N]) {
  typename S::template Raw<YT> r[n];
  float w[n];
#pragma unroll
  for (int i = 0; i < n; i++) {
    const int j = next_slot(m);
    w[i] = p.weight(j);
    sp.template load<NT>(r[i], static_cast<const YT*>(a.rows_in) + (size_t)p.row(j) * a.cols);
  }
#pragma unroll
  for (int i = 0; i < n; i++) {
    float v[S::N];
    sp.get(r[i], v);
#pragma unroll
    for (int k = 0; k < S::N; k++) acc[k] = fmaf(w[i], v[k], acc[k]);
  }
}

template <typename YT, typename OT, bool FULL, int CH, bool NT>
__global__ __launch_bounds__(1024) void k_combine_rows(RowsArgs a) {
  typedef Span<FULL, CH> S;
  const int t = blockIdx.x;
  const S sp(a.cols, blockDim.x, blockIdx.y * blockDim.x * CH);
  const Pairs p(a, t);
  float acc[S::N];
#pragma unroll
  for (int k = 0; k < S::N; k++) acc[k] = 0.0f;
  uint64_t m = p.on;
  int left = __builtin_popcountll(m);
  for (; left >= 4; left -= 4) add_slots<4, NT, YT>(a, sp, p, m, acc);
  if (left >= 2) add_slots<2, NT, YT>(a, sp, p, m, acc);
  if (left & 1) add_slots<1, NT, YT>(a, sp, p, m, acc);
  sp.put(static_cast<OT*>(a.token_out) + (size_t)t * a.cols, acc);
}

// One workgroup per token, whose d_out row stays in registers for all its
// slots.  The next slot's row is loaded before this slot's stores (memory
// operations complete in order).
template <typename YT, typename OT, bool FULL, int CH, bool NT>
__global__ __launch_bounds__(1024) void k_combine_rows_backward(RowsArgs a) {
  __shared__ float part[32][16];
  typedef Span<FULL, CH> S;
  const int t = blockIdx.x, tid = threadIdx.x, waves = blockDim.x >> 6;
  const S sp(a.cols, blockDim.x);
  typename S::template Raw<OT> rd;
  sp.template load<NT>(rd, static_cast<const OT*>(a.token) + (size_t)t * a.cols);
  const Pairs p(a, t);
  typedef typename S::template Raw<YT> Row;
  uint64_t m = p.on;
  int j = 0;
  auto fetch = [&](Row& r) {
    j = next_slot(m);
    if (a.d_w != nullptr) sp.template load<NT>(r, static_cast<const YT*>(a.rows_in) + (size_t)p.row(j) * a.cols);
  };
  float d[S::N];
  auto slot = [&](const Row& r, int s) {
    if (a.d_w != nullptr) {
      float y[S::N], dot = 0.0f;
      sp.get(r, y);
#pragma unroll
      for (int k = 0; k < S::N; k++) dot = sp.has(k) ? fmaf(d[k], y[k], dot) : dot;
      dot = wave_total(dot);
      if ((tid & 63) == 0) part[s][tid >> 6] = dot;
    }
    if (a.rows_out != nullptr) {
      const float w = p.weight(s);
      float g[S::N];
#pragma unroll
      for (int k = 0; k < S::N; k++) g[k] = w * d[k];
      sp.template put<NT>(static_cast<YT*>(a.rows_out) + (size_t)p.row(s) * a.cols, g);
    }
  };
  if (m != 0) {
    Row r0, r1;
    fetch(r0);
    sp.get(rd, d);
    for (;;) {
      int s = j;
      if (m == 0) {
        slot(r0, s);
        break;
      }
      fetch(r1);
      slot(r0, s);
      s = j;
      if (m == 0) {
        slot(r1, s);
        break;
      }
      fetch(r0);
      slot(r1, s);
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

// Workgroups of the sort and of the combine: a whole row each for many tokens, so
// that a row's positions are fetched once and there is more in flight behind them
// (16384 tokens of 4608, 8 slots, in whole rows and in runs: combine of bf16 rows
// 235 and 241 us, of fp32 rows 492 and 515, with an eighth local 90 and 92; sort 282
// and 286, its gradient 234 and 240); for few tokens a run of 8 columns a thread, so
// that there are more.
constexpr int kManyTokens = 1024;
struct Shape {
  int waves, pieces, runs;
};
Shape shape_of(const RowsArgs& a) {
  Shape s;
  const int n = ceil_div(a.cols / 8, 64);           // waves at one piece a thread
  if (a.T >= kManyTokens) {
    s.waves = row_waves(a.cols, 4);
    s.pieces = row_pieces(a.cols, s.waves);
    s.runs = 1;
    return s;
  }
  s.waves = 4;                                      // the number that leaves the fewest idle
  for (int w = 3; w >= 1; w--)
    if (ceil_div(n, w) * w < ceil_div(n, s.waves) * s.waves) s.waves = w;
  s.pieces = 1;
  s.runs = n > 0 ? ceil_div(n, s.waves) : 1;
  return s;
}

// Bytes of the expert rows of a call.
size_t row_bytes(const RowsArgs& a) { return (size_t)a.M * a.cols * (a.row_dtype == 0 ? 2 : 4); }

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
  const Shape h = shape_of(a);
  const bool full = a.cols % 8 == 0 && aligned16(a.token) && aligned16(a.rows_out), nt = row_bytes(a) > kStreamBytes;
  MOE_ROWS_TYPE(a.row_dtype, T, MOE_ROWS_BOOL(full, FULL, MOE_ROWS_BOOL(nt, NT, MOE_ROW_PIECES(h.pieces,
      hipLaunchKernelGGL((k_sort_rows<T, FULL, CH, NT>), dim3(a.T, h.runs), dim3(64 * h.waves), 0, s, a)))));
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

int launch_combine_rows(const RowsArgs& a, hipStream_t s) {
  if (a.T <= 0) return 0;
  const Shape h = shape_of(a);
  const bool full = a.cols % 8 == 0 && aligned16(a.token_out) && aligned16(a.rows_in), nt = row_bytes(a) > kStreamBytes;
  MOE_ROWS_TYPE(a.row_dtype, YT, MOE_ROWS_TYPE(a.token_dtype, OT, MOE_ROWS_BOOL(full, FULL, MOE_ROWS_BOOL(nt, NT,
      MOE_ROW_PIECES(h.pieces, hipLaunchKernelGGL((k_combine_rows<YT, OT, FULL, CH, NT>), dim3(a.T, h.runs),
                                                  dim3(64 * h.waves), 0, s, a))))));
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

int launch_combine_rows_backward(const RowsArgs& a, hipStream_t s) {
  if (a.T <= 0) return 0;
  const int waves = row_waves(a.cols, 4);
  const bool full = a.cols % 8 == 0 && aligned16(a.token) && aligned16(a.rows_in) && aligned16(a.rows_out);
  const bool nt = row_bytes(a) > kStreamBytes;
  MOE_ROWS_TYPE(a.row_dtype, YT, MOE_ROWS_TYPE(a.token_dtype, OT, MOE_ROWS_BOOL(full, FULL, MOE_ROWS_BOOL(nt, NT,
      MOE_ROW_PIECES(row_pieces(a.cols, waves), hipLaunchKernelGGL((k_combine_rows_backward<YT, OT, FULL, CH, NT>),
                                                                   dim3(a.T), dim3(64 * waves), 0, s, a))))));
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace moe
