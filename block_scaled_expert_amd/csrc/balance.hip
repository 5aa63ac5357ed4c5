// The router's balance loss: per-expert counts, mean probabilities and the
// loss of each sequence, and the gradient of the router logits.
//
// For a sequence of n tokens (masked ones left out), s = sigmoid(z),
// p_te = s_te / sum_i s_ti, c_e = number of (token, slot) pairs routed to e:
//   P_e = (1/n) sum_t p_te,   L = E / (k n) * sum_e c_e P_e
// The counts carry no gradient, so with g_e = dL * E / (k n^2) * c_e
//   dz_te = p_te (1 - s_te) (g_e - sum_i g_i p_ti)
// and through the gate weights w_j = scale * s_j / sum_i s_i (i over the
// token's slots; v_j = w_j / scale)
//   dz_{id_j} += scale * v_j (1 - s_j) (dw_j - sum_i dw_i v_i)
// or scale * s_j (1 - s_j) dw_j without the normalisation.
//
// The forward reads the logits once and the backward once: HBM-bound at
// large T (16384 x 384 fp32 logits are 25 MB), launch-bound below.  One
// wavefront holds a token's whole row in registers (lane l experts l + 64 i),
// so the sums over experts are lane exchanges.  Sums over tokens are taken
// in a fixed order (registers, then waves, then token chunks); the counts are
// integers, whose atomics commute.  Every run gives the same bits.
#include "moe_common.h"
#include "launch.h"

namespace moe {

namespace {

// e^x for x <= 0, relative error below 2e-7: the hardware's exp2 of x log2(e),
// with the rounding of that product put back to first order.
__device__ inline float exp_neg(float x) {
  x = x < -200.0f ? -200.0f : x;               // e^-200 is 0 in fp32; keeps -inf out of the products
  const float y = x * 1.44269504f;
  const float r = fmaf(x, 1.44269504f, -y) + x * 1.9259630e-8f;
  const float e = __builtin_amdgcn_exp2f(y);
  return fmaf(e * r, 0.693147181f, e);
}

// sigmoid(z) * e^-shift as t, and 1 - sigmoid(z) as c, for shift = min(0, max
// of the row): with shift = 0 the plain sigmoid; a row whose logits are all far
// below zero keeps its proportions, where the sigmoids themselves underflow.
// em = e^shift.
__device__ inline void sig(float z, float shift, float em, float& t, float& c) {
  const bool pos = z >= 0.0f;
  const float e = exp_neg(pos ? -z : z - shift);
  const float r = __builtin_amdgcn_rcpf(1.0f + (pos ? e : e * em));
  t = pos ? r : e * r;
  c = pos ? e * r : r;
}

template <typename T>
__device__ inline float load_z(const T* p);
template <>
__device__ inline float load_z<float>(const float* p) { return *p; }
template <>
__device__ inline float load_z<uint16_t>(const uint16_t* p) { return bf16_to_f32(*p); }

__device__ inline void store_dz(float* p, float v) { *p = v; }
__device__ inline void store_dz(uint16_t* p, float v) { *reinterpret_cast<__bf16*>(p) = (__bf16)v; }

// A token's row: t[i] proportional to sigmoid(z), c[i] = 1 - sigmoid(z) of
// expert lane + 64 i (t = 0 past E), and 1 / sum t (0 for a row whose logits
// are all -inf).
template <int NPER>
struct Row {
  float t[NPER], c[NPER], inv;
  float shift, em;
};

template <int NPER>
__device__ inline void make_row(const float (&z)[NPER], int E, int lane, Row<NPER>& r) {
  float sum = 0.0f;
  r.shift = 0.0f;
  r.em = 1.0f;
#pragma unroll
  for (int i = 0; i < NPER; i++) {
    sig(z[i], 0.0f, 1.0f, r.t[i], r.c[i]);
    if (lane + 64 * i >= E) r.t[i] = 0.0f;
    sum += r.t[i];
  }
  sum = wave_sum(sum);
  if (sum < 1e-12f) {   // uniform; every logit is below -27: shift by their maximum
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NPER; i++)
      if (lane + 64 * i < E) m = fmaxf(m, z[i]);
    m = wave_max(m);
    sum = 0.0f;
    if (m > -INFINITY) {
      r.shift = m;
      r.em = exp_neg(m);
#pragma unroll
      for (int i = 0; i < NPER; i++) {
        sig(z[i], m, r.em, r.t[i], r.c[i]);
        if (lane + 64 * i >= E) r.t[i] = 0.0f;
        sum += r.t[i];
      }
      sum = wave_sum(sum);
    }
  }
  r.inv = sum == 0.0f ? 0.0f : 1.0f / sum;     // a NaN logit makes the row NaN
}

// First token of sequence s, clamped to [0, T] whatever the device array holds.
__device__ inline int bound(const BalanceArgs& a, int s) {
  if (a.bounds == nullptr) return s == 0 ? 0 : a.T;
  return min(max(a.bounds[s], 0), a.T);
}

// The sequence of token t: the largest s with bounds[s] <= t (-1: none).
__device__ inline int seq_of(const BalanceArgs& a, int t) {
  if (a.bounds == nullptr) return 0;
  int lo = -1, hi = a.S;                       // bounds[lo] <= t < bounds[hi], read as sentinels at the ends
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (a.bounds[m] <= t) lo = m;
    else hi = m;
  }
  return lo;
}

// Forward, first launch: workgroup c takes tokens [c C, (c + 1) C) and, for
// every sequence s with tokens there, writes the sums of p and the counts to
// slot c + s (chunks and sequences both advance, so a slot is used once).
struct BalanceWs {
  float* sums;        // [slots][E]
  int32_t* counts;    // [slots][E]
  int32_t* live;      // [slots]
  float* part;        // [S][kFinishCols]: partial losses
  int32_t* ticket;    // [S]
  int chunk, nchunks, slots;
};

constexpr int kMaxE = 1024, kFinishCols = kMaxE / 64;

__host__ __device__ inline int balance_chunk(int T) {
  const int c = (T + 511) / 512;               // about two workgroups per CU
  return c < 16 ? 16 : c;
}

template <typename ZT, int NPER>
__global__ __launch_bounds__(256) void k_balance_part(BalanceArgs a, BalanceWs w) {
  __shared__ float psum[4][64 * NPER];
  __shared__ int32_t hist[64 * NPER];
  __shared__ int32_t nlive[4];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  if (blockIdx.x == 0)                         // the second launch counts its workgroups here
    for (int s = tid; s < a.S; s += 256) w.ticket[s] = 0;
  const int t0 = blockIdx.x * w.chunk, t1 = min(t0 + w.chunk, a.T);
  const ZT* z = static_cast<const ZT*>(a.z);
  int s = max(seq_of(a, t0), 0);
  for (; s < a.S; s++) {
    const int lo = max(bound(a, s), t0), hi = min(bound(a, s + 1), t1);
    if (lo >= t1) break;
    if (lo >= hi) continue;
    for (int e = tid; e < a.E; e += 256) hist[e] = 0;
    __syncthreads();
    float acc[NPER];
#pragma unroll
    for (int i = 0; i < NPER; i++) acc[i] = 0.0f;
    int n = 0;
    for (int t = lo + wave; t < hi; t += 4) {
      if (a.mask != nullptr && a.mask[t] == 0) continue;
      n++;
      float zr[NPER];
#pragma unroll
      for (int i = 0; i < NPER; i++) zr[i] = load_z<ZT>(z + (size_t)t * a.E + min(lane + 64 * i, a.E - 1));
      if (lane < a.k) {
        const int id = a.ids[(size_t)t * a.k + lane];
        if (id >= 0 && id < a.E) atomicAdd(&hist[id], 1);
      }
      Row<NPER> r;
      make_row<NPER>(zr, a.E, lane, r);
#pragma unroll
      for (int i = 0; i < NPER; i++) acc[i] = fmaf(r.t[i], r.inv, acc[i]);
    }
#pragma unroll
    for (int i = 0; i < NPER; i++) psum[wave][lane + 64 * i] = acc[i];
    if (lane == 0) nlive[wave] = n;
    __syncthreads();
    const size_t slot = (size_t)blockIdx.x + s;
    for (int e = tid; e < a.E; e += 256) {
      w.sums[slot * a.E + e] = ((psum[0][e] + psum[1][e]) + psum[2][e]) + psum[3][e];
      w.counts[slot * a.E + e] = hist[e];
    }
    if (tid == 0) w.live[slot] = nlive[0] + nlive[1] + nlive[2] + nlive[3];
    __syncthreads();
  }
}

// Forward, second launch: workgroup (x, s) adds the slots of sequence s for 64
// experts, 16 waves taking every 16th slot; the last of the sequence's
// workgroups to finish adds their partial losses in order.
__global__ __launch_bounds__(1024) void k_balance_finish(BalanceArgs a, BalanceWs w) {
  __shared__ float ps[16][64];
  __shared__ int32_t cs[16][64], ns[16];
  const int s = blockIdx.y, tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int e = blockIdx.x * 64 + lane, ec = min(e, a.E - 1);
  const int lo = bound(a, s), hi = bound(a, s + 1);
  const int c0 = lo / w.chunk, c1 = hi > lo ? (hi - 1) / w.chunk + 1 : c0;   // chunks [c0, c1)
  float p = 0.0f;
  int32_t c = 0, n = 0;
  for (int i = c0 + wave; i < c1; i += 16) {
    const size_t slot = (size_t)i + s;
    p += w.sums[slot * a.E + ec];
    c += w.counts[slot * a.E + ec];
    n += w.live[slot];
  }
  ps[wave][lane] = p;
  cs[wave][lane] = c;
  if (lane == 0) ns[wave] = n;
  __syncthreads();
  if (wave == 0) {
    p = 0.0f;
    c = n = 0;
#pragma unroll
    for (int i = 0; i < 16; i++) {
      p += ps[i][lane];
      c += cs[i][lane];
      n += ns[i];
    }
    const float inv = n > 0 ? 1.0f / (float)n : 0.0f;
    p *= inv;
    if (e < a.E) {
      a.probs[(size_t)s * a.E + e] = p;
      a.counts[(size_t)s * a.E + e] = c;
    }
    const float part = wave_sum(e < a.E ? (float)c * inv * p : 0.0f);
    if (lane == 0) {
      if (blockIdx.x == 0) a.live[s] = n;
      __hip_atomic_store(w.part + s * kFinishCols + blockIdx.x, part, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      const int before = __hip_atomic_fetch_add(w.ticket + s, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
      if (before == (int)gridDim.x - 1) {
        float l = 0.0f;
        for (int x = 0; x < (int)gridDim.x; x++)
          l += __hip_atomic_load(w.part + s * kFinishCols + x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        a.loss[s] = l * ((float)a.E / (float)a.k);
      }
    }
  }
}

// Backward: one wavefront per token, runs of kRun tokens (the counts of a
// sequence are read again only where the sequence changes).
constexpr int kRun = 4;

template <typename ZT, int NPER>
__global__ __launch_bounds__(256) void k_balance_backward(BalanceArgs a) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int t0 = (blockIdx.x * 4 + wave) * kRun;
  const ZT* z = static_cast<const ZT*>(a.z);
  ZT* dz = static_cast<ZT*>(a.dz);
  float g[NPER];
  int s = -2, s_hi = t0;                        // tokens below s_hi belong to s
  bool in_seq = false;
  for (int t = t0; t < min(t0 + kRun, a.T); t++) {
    if (t >= s_hi) {
      s = seq_of(a, t);
      s_hi = s < 0 ? bound(a, 0) : s < a.S ? bound(a, s + 1) : a.T;
      in_seq = s >= 0 && s < a.S && t < s_hi;
      if (s_hi <= t) s_hi = t + 1;              // bounds out of order: look again at the next token
      const float n = in_seq ? (float)a.live[s] : 0.0f;
      const float f = n > 0.0f ? a.d_loss[s] * ((float)a.E / ((float)a.k * n)) / n : 0.0f;
#pragma unroll
      for (int i = 0; i < NPER; i++)
        g[i] = in_seq && lane + 64 * i < a.E ? f * (float)a.counts[(size_t)s * a.E + lane + 64 * i] : 0.0f;
    }
    ZT* out = dz + (size_t)t * a.E;
    if (!in_seq || (a.mask != nullptr && a.mask[t] == 0)) {
#pragma unroll
      for (int i = 0; i < NPER; i++)
        if (lane + 64 * i < a.E) store_dz(out + lane + 64 * i, 0.0f);
      continue;
    }
    const ZT* zt = z + (size_t)t * a.E;
    float zr[NPER];
#pragma unroll
    for (int i = 0; i < NPER; i++) zr[i] = load_z<ZT>(zt + min(lane + 64 * i, a.E - 1));
    Row<NPER> r;
    make_row<NPER>(zr, a.E, lane, r);
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NPER; i++) dot = fmaf(g[i], r.t[i], dot);
    dot = wave_sum(dot) * r.inv;
    float d[NPER];
#pragma unroll
    for (int i = 0; i < NPER; i++) d[i] = r.t[i] * r.inv * r.c[i] * (g[i] - dot);
    if (a.d_w != nullptr) {
      // lane j < k: slot j
      int id = -1;
      float v = 0.0f, c = 0.0f, dw = 0.0f;
      if (lane < a.k) {
        id = a.ids[(size_t)t * a.k + lane];
        if (id < 0 || id >= a.E) id = -1;
        if (id >= 0) dw = a.d_w[(size_t)t * a.k + lane];
      }
      const float zs = id >= 0 ? load_z<ZT>(zt + id) : -INFINITY;
      float gate;
      sig(zs, 0.0f, 1.0f, v, c);
      if (a.norm_topk) {
        float tot = wave_sum(v);
        if (tot < 1e-12f) {                      // uniform: as in make_row, for the token's slots
          const float m = wave_max(zs);
          if (m > -INFINITY) {
            sig(zs, m, exp_neg(m), v, c);
            tot = wave_sum(v);
          }
        }
        v = tot == 0.0f ? 0.0f : v / tot;
        gate = v * c * (dw - wave_sum(dw * v));
      } else {
        gate = v * c * dw;
      }
      gate *= a.routed_scale;
      for (int j = 0; j < a.k; j++) {
        const int idj = __builtin_amdgcn_readlane(id, j);
        const float gj = bits_f(__builtin_amdgcn_readlane((int)f_bits(gate), j));
        if (idj < 0) continue;
#pragma unroll
        for (int i = 0; i < NPER; i++)
          if (idj == lane + 64 * i) d[i] += gj;
      }
    }
#pragma unroll
    for (int i = 0; i < NPER; i++)
      if (lane + 64 * i < a.E) store_dz(out + lane + 64 * i, d[i]);
  }
}

// Adds the S split planes of router logits in split order.
__global__ __launch_bounds__(256) void k_router_logits_sum(const float* __restrict__ zpart, int S, long n,
                                                           float* __restrict__ z) {
  const long i = (long)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float v = zpart[i];
  for (int s = 1; s < S; s++) v += zpart[s * n + i];
  z[i] = v;
}

BalanceWs carve(void* ws, int T, int E, int S) {
  BalanceWs w;
  w.chunk = balance_chunk(T);
  w.nchunks = ceil_div(T, w.chunk);
  w.slots = w.nchunks + S;
  char* p = static_cast<char*>(ws);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    char* q = p + o;
    o = align_up(o + bytes, 256);
    return q;
  };
  w.sums = reinterpret_cast<float*>(take((size_t)w.slots * E * 4));
  w.counts = reinterpret_cast<int32_t*>(take((size_t)w.slots * E * 4));
  w.live = reinterpret_cast<int32_t*>(take((size_t)w.slots * 4));
  w.part = reinterpret_cast<float*>(take((size_t)S * kFinishCols * 4));
  w.ticket = reinterpret_cast<int32_t*>(take((size_t)S * 4));
  return w;
}

}  // namespace

size_t balance_ws_bytes(int T, int E, int S) {
  const size_t slots = (size_t)ceil_div(T, balance_chunk(T)) + S;
  return 2 * align_up(slots * E * 4, 256) + align_up(slots * 4, 256) + align_up((size_t)S * kFinishCols * 4, 256) +
         align_up((size_t)S * 4, 256);
}

// NPER: registers of a lane's row, from the experts
#define MOE_BAL(CALL)                              \
  do {                                             \
    const int nper = ceil_div(a.E, 64);            \
    if (nper <= 1) CALL(1);                        \
    else if (nper <= 2) CALL(2);                   \
    else if (nper <= 4) CALL(4);                   \
    else if (nper <= 6) CALL(6);                   \
    else if (nper <= 8) CALL(8);                   \
    else CALL(16);                                 \
  } while (0)

int launch_balance_forward(const BalanceArgs& a, hipStream_t stream) {
  const BalanceWs w = carve(a.ws, a.T, a.E, a.S);
  const dim3 grid(w.nchunks > 0 ? w.nchunks : 1);   // also clears the tickets
#define MOE_PART(N)                                                                                             \
  do {                                                                                                          \
    if (a.dtype == 0)                                                                                           \
      hipLaunchKernelGGL((k_balance_part<uint16_t, N>), grid, dim3(256), 0, stream, a, w);           \
    else                                                                                                        \
      hipLaunchKernelGGL((k_balance_part<float, N>), grid, dim3(256), 0, stream, a, w);              \
  } while (0)
  MOE_BAL(MOE_PART);
#undef MOE_PART
  hipLaunchKernelGGL(k_balance_finish, dim3(ceil_div(a.E, 64), a.S), dim3(1024), 0, stream, a, w);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

int launch_balance_backward(const BalanceArgs& a, hipStream_t stream) {
  if (a.T <= 0) return 0;
  const dim3 grid(ceil_div(a.T, 4 * kRun));
#define MOE_BACK(N)                                                                                  \
  do {                                                                                               \
    if (a.dtype == 0)                                                                                \
      hipLaunchKernelGGL((k_balance_backward<uint16_t, N>), grid, dim3(256), 0, stream, a);          \
    else                                                                                             \
      hipLaunchKernelGGL((k_balance_backward<float, N>), grid, dim3(256), 0, stream, a);             \
  } while (0)
  MOE_BAL(MOE_BACK);
#undef MOE_BACK
  return hipGetLastError() == hipSuccess ? 0 : -1;
}
#undef MOE_BAL

int launch_router_logits_sum(const float* zpart, int T, int E, float* z, hipStream_t stream) {
  const long n = (long)T * E;
  if (n <= 0) return 0;
  hipLaunchKernelGGL(k_router_logits_sum, dim3(ceil_div(n, 256)), dim3(256), 0, stream, zpart, router_splits(T, E), n,
                     z);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace moe
