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
// large T, launch-bound below.  Measured, 131072 x 384 fp32 and 8 ids a token:
// forward 47 us + 10 for its second launch (4.4 TB/s), backward 76 (5.4 TB/s);
// 16384 tokens 8.6 + 7.2 and 15.6; 64 tokens 6.3 in one launch and 4.4.  bf16
// logits take nearly fp32's time (44 + 10 and 73 at 131072 tokens): half the
// bytes, but as many loads and stores and the same arithmetic an element.  One
// wavefront holds a token's whole row in registers (lane l experts l + 64 i),
// so the sums over experts are lane exchanges.  Sums over tokens are taken
// in a fixed order (registers, then waves, then token chunks); the counts are
// integers, whose atomics commute.  Every run gives the same bits.
#include "operators.h"

namespace moe {

namespace {

// Sum over the wavefront, the same in every lane: within each row of 16 lanes
// by DPP (neighbours, pairs, half rows, rows), then the four rows.  A third of
// the instructions' latency of an exchange through LDS, and one fixed order.
template <int CTRL>
__device__ inline float dpp_add(float v) {
  return v + bits_f((uint32_t)__builtin_amdgcn_update_dpp(0, (int)f_bits(v), CTRL, 0xF, 0xF, false));
}
__device__ inline float row_sum(float v) {
  v = dpp_add<0xB1>(v);    // quad_perm [1,0,3,2]
  v = dpp_add<0x4E>(v);    // quad_perm [2,3,0,1]
  v = dpp_add<0x141>(v);   // row_half_mirror
  return dpp_add<0x140>(v);   // row_mirror
}
__device__ inline float lane_f(float v, int l) { return bits_f((uint32_t)__builtin_amdgcn_readlane((int)f_bits(v), l)); }
__device__ inline float all_sum(float v) {
  v = row_sum(v);
  return (lane_f(v, 0) + lane_f(v, 16)) + (lane_f(v, 32) + lane_f(v, 48));
}
// The same where lanes 32 .. 63 hold zero.
__device__ inline float half_sum(float v) {
  v = row_sum(v);
  return lane_f(v, 0) + lane_f(v, 16);
}

// e^x for x <= 0, relative error below 2e-7: the hardware's exp2 of x log2(e),
// with the rounding of that product put back to first order.  Below -200 (0 in
// fp32) as at -200, which keeps -inf out of the products.
__device__ inline float exp_neg(float x) {
  x = fmaxf(x, -200.0f);
  const float y = x * 1.44269504f;
  const float r = fmaf(x, 1.44269504f, -y) + x * 1.9259630e-8f;
  const float e = __builtin_amdgcn_exp2f(y);
  return fmaf(e * r, 0.693147181f, e);
}

// sigmoid(z) as t and 1 - sigmoid(z) as c.  A NaN gives finite values: rows
// are checked for NaN on their own.
__device__ inline void sig(float z, float& t, float& c) {
  const float e = exp_neg(-fabsf(z));
  const float r = __builtin_amdgcn_rcpf(1.0f + e), er = e * r;
  t = z >= 0.0f ? r : er;
  c = z >= 0.0f ? er : r;
}
// sigmoid(z) e^-shift and 1 - sigmoid(z) for z <= shift <= 0: a row whose logits
// are all far below zero keeps its proportions, where the sigmoids themselves
// underflow.  em = e^shift.
__device__ inline void sig_shifted(float z, float shift, float em, float& t, float& c) {
  const float e = exp_neg(z - shift);
  c = __builtin_amdgcn_rcpf(fmaf(e, em, 1.0f));
  t = e * c;
}

__device__ inline float load_z(const float* p) { return *p; }
__device__ inline float load_z(const uint16_t* p) { return bf16_to_f32(*p); }
template <bool NT, typename T>
__device__ inline void put(T* p, T v) {
  if constexpr (NT) __builtin_nontemporal_store(v, p);
  else *p = v;
}
template <bool NT>
__device__ inline void store_dz(float* p, float v) { put<NT>(p, v); }
template <bool NT>
__device__ inline void store_dz(uint16_t* p, float v) { put<NT>(p, __builtin_bit_cast(uint16_t, (__bf16)v)); }

// A token's row: t[i] proportional to sigmoid(z), c[i] = 1 - sigmoid(z) of
// expert lane + 64 i (t = 0 past E), and 1 / sum t (0 for a row whose logits
// are all -inf, NaN if one is NaN).
template <int NPER>
struct Row {
  float t[NPER], c[NPER], inv;
};

template <int NPER>
__device__ inline void make_row(const float (&z)[NPER], int E, int lane, Row<NPER>& r) {
  float sum = 0.0f;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < NPER; i++) {
    const bool in = lane + 64 * i < E;
    sig(z[i], r.t[i], r.c[i]);
    r.t[i] = in ? r.t[i] : 0.0f;
    nan |= z[i] != z[i];                         // (lanes past E repeat the last expert)
    sum += r.t[i];
  }
  sum = all_sum(sum);
  if (sum < 1e-12f) {                            // uniform; every logit is below -27: shift by their maximum
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NPER; i++) m = fmaxf(m, z[i]);
    m = wave_max(m);
    sum = 0.0f;
    if (m > -INFINITY) {
      const float em = exp_neg(m);
#pragma unroll
      for (int i = 0; i < NPER; i++) {
        sig_shifted(z[i], m, em, r.t[i], r.c[i]);
        if (lane + 64 * i >= E) r.t[i] = 0.0f;
        sum += r.t[i];
      }
      sum = all_sum(sum);
    }
  }
  r.inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  if (__any(nan)) r.inv = __builtin_nanf("");
}

template <typename ZT, int NPER>
__device__ inline void load_row(const ZT* z, int E, int lane, float (&v)[NPER]) {
#pragma unroll
  for (int i = 0; i < NPER; i++) v[i] = load_z(z + min(lane + 64 * i, E - 1));
}

// First token of sequence s, clamped to [0, T] whatever the device array holds.
__device__ inline int bound(const BalanceArgs& a, int s) {
  if (a.bounds == nullptr) return s == 0 ? 0 : a.T;
  return min(max(a.bounds[s], 0), a.T);
}

// The sequence of token t: the largest s with bounds[s] <= t (-1: none).  The
// wave looks at 64 bounds at a time.
__device__ inline int seq_of(const BalanceArgs& a, int t, int lane) {
  if (a.bounds == nullptr) return 0;
  int lo = 0, hi = a.S;                          // the number of bounds <= t is in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 63) / 64, at = lo + lane * step;
    const int n = __popcll(__ballot(at < hi && a.bounds[min(at, a.S)] <= t));
    if (n == 0) break;
    hi = min(hi, lo + n * step);
    lo += (n - 1) * step + 1;
  }
  return lo - 1;
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

constexpr int kMaxE = 1024, kFinishE = 16, kFinishCols = kMaxE / kFinishE;

__host__ __device__ inline int balance_chunk(int T) {
  // at least a token a wave; four workgroups per CU, eight where they then
  // still have 16 tokens (each writes E sums and counts)
  const int c = (T + 1023) / 1024;
  return c < 4 ? 4 : c <= 16 ? c : c < 32 ? 16 : (T + 2047) / 2048;
}

// Tokens a wave adds up in one run of fp32 additions.  Equal logits round the
// same way at every addition: one run over the 8192 tokens that a wave takes at
// T = 2^26 put the mean of 1/5 off by 6.5e-5 of itself.
constexpr int kRun = 256;

template <typename ZT, int NPER>
__global__ __launch_bounds__(256) void k_balance_part(BalanceArgs a, BalanceWs w) {
  __shared__ float psum[4][64 * NPER];
  __shared__ int32_t hist[64 * NPER];
  __shared__ int32_t nlive[4];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  if (blockIdx.x == 0)                         // the second launch counts its workgroups here
    for (int s = tid; s < a.S; s += 256) w.ticket[s] = 0;
  const int t0 = blockIdx.x * w.chunk, t1 = min(t0 + w.chunk, a.T);
  const ZT* z = static_cast<const ZT*>(a.z);
  int s = max(seq_of(a, t0, lane), 0);
  for (; s < a.S; s++) {
    const int lo = max(bound(a, s), t0), hi = min(bound(a, s + 1), t1);
    if (lo >= t1) break;
    if (lo >= hi) continue;
    // the wave's tokens lo + wave, + 4 ..: the next one's logits are on their way while one is worked on
    int t = lo + wave;
    float zr[NPER];
    bool on = false;
    if (t < hi) {
      on = a.mask == nullptr || a.mask[t] != 0;
      load_row<ZT, NPER>(z + (size_t)t * a.E, a.E, lane, zr);
    }
    for (int e = tid; e < a.E; e += 256) hist[e] = 0;
    __syncthreads();
    for (int p = lo * a.k + tid; p < hi * a.k; p += 256) {
      const int id = a.ids[p];
      if (id >= 0 && id < a.E && (a.mask == nullptr || a.mask[p / a.k] != 0)) atomicAdd(&hist[id], 1);
    }
    float acc[NPER];
#pragma unroll
    for (int i = 0; i < NPER; i++) {
      acc[i] = 0.0f;
      psum[wave][lane + 64 * i] = 0.0f;
    }
    int n = 0;
    for (int run = 1; t < hi; t += 4, run++) {
      const int tn = min(t + 4, hi - 1);
      float zn[NPER];
      const bool on_next = a.mask == nullptr || a.mask[tn] != 0;
      load_row<ZT, NPER>(z + (size_t)tn * a.E, a.E, lane, zn);
      if (on) {
        n++;
        Row<NPER> r;
        make_row<NPER>(zr, a.E, lane, r);
#pragma unroll
        for (int i = 0; i < NPER; i++) acc[i] = fmaf(r.t[i], r.inv, acc[i]);
      }
      if (run % kRun == 0) {
#pragma unroll
        for (int i = 0; i < NPER; i++) {
          psum[wave][lane + 64 * i] += acc[i];
          acc[i] = 0.0f;
        }
      }
      on = on_next;
#pragma unroll
      for (int i = 0; i < NPER; i++) zr[i] = zn[i];
    }
#pragma unroll
    for (int i = 0; i < NPER; i++) psum[wave][lane + 64 * i] += acc[i];
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

// Forward in one launch for few tokens: workgroup s takes sequence s whole, its
// W waves a token each in turn, about 1 us a turn at 384 experts and 1.2 at
// 1024.  One sequence of 384 experts, on the GPU: 2.9 us for 8 tokens against
// 7.3 in two launches, 6.4 against 7.4 for 64, 8.4 against 7.9 for 96; 1024
// experts: 12.9 against 8.6 for 64.  Called eagerly the launch saved is 3 us.
// So by tokens times experts, as if one sequence held them all.
inline bool one_launch(const BalanceArgs& a) { return a.T <= 128 && a.T * ceil_div(a.E, 64) <= 384; }

template <int NPER>
constexpr int kOneWaves = NPER > 8 ? 8 : 16;   // (their partial sums stay below 64 KiB of LDS)

template <typename ZT, int NPER>
__global__ __launch_bounds__(64 * kOneWaves<NPER>) void k_balance_one(BalanceArgs a) {
  constexpr int W = kOneWaves<NPER>;
  __shared__ float psum[W][64 * NPER], part[W];
  __shared__ int32_t hist[64 * NPER], nlive[W];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, s = blockIdx.x;
  const int lo = bound(a, s), hi = bound(a, s + 1);
  const ZT* z = static_cast<const ZT*>(a.z);
  int t = lo + wave;
  float zr[NPER];
  bool on = false;
  if (t < hi) {
    on = a.mask == nullptr || a.mask[t] != 0;
    load_row<ZT, NPER>(z + (size_t)t * a.E, a.E, lane, zr);
  }
  for (int e = tid; e < a.E; e += 64 * W) hist[e] = 0;
  __syncthreads();
  for (int p = lo * a.k + tid; p < hi * a.k; p += 64 * W) {
    const int id = a.ids[p];
    if (id >= 0 && id < a.E && (a.mask == nullptr || a.mask[p / a.k] != 0)) atomicAdd(&hist[id], 1);
  }
  float acc[NPER];
#pragma unroll
  for (int i = 0; i < NPER; i++) acc[i] = 0.0f;
  int n = 0;
  for (; t < hi; t += W) {
    const int tn = min(t + W, hi - 1);
    float zn[NPER];
    const bool on_next = a.mask == nullptr || a.mask[tn] != 0;
    load_row<ZT, NPER>(z + (size_t)tn * a.E, a.E, lane, zn);
    if (on) {
      n++;
      Row<NPER> r;
      make_row<NPER>(zr, a.E, lane, r);
#pragma unroll
      for (int i = 0; i < NPER; i++) acc[i] = fmaf(r.t[i], r.inv, acc[i]);
    }
    on = on_next;
#pragma unroll
    for (int i = 0; i < NPER; i++) zr[i] = zn[i];
  }
#pragma unroll
  for (int i = 0; i < NPER; i++) psum[wave][lane + 64 * i] = acc[i];
  if (lane == 0) nlive[wave] = n;
  __syncthreads();
  n = 0;
#pragma unroll
  for (int i = 0; i < W; i++) n += nlive[i];
  const float inv = n > 0 ? 1.0f / (float)n : 0.0f;
  float l = 0.0f;
  for (int e = tid; e < a.E; e += 64 * W) {
    float p = 0.0f;
#pragma unroll
    for (int i = 0; i < W; i++) p += psum[i][e];
    p *= inv;
    a.probs[(size_t)s * a.E + e] = p;
    a.counts[(size_t)s * a.E + e] = hist[e];
    l += (float)hist[e] * inv * p;
  }
  l = all_sum(l);
  if (lane == 0) part[wave] = l;
  __syncthreads();
  if (tid == 0) {
    l = 0.0f;
#pragma unroll
    for (int i = 0; i < W; i++) l += part[i];
    a.live[s] = n;
    a.loss[s] = l * ((float)a.E / (float)a.k);
  }
}

// Forward, second launch: workgroup (x, s) adds the slots of sequence s for
// kFinishE experts, its groups of 16 lanes (64, or 16 for short sequences)
// taking the slots in turn; the last of the sequence's workgroups to finish
// adds their partial losses in order.
__global__ __launch_bounds__(1024) void k_balance_finish(BalanceArgs a, BalanceWs w) {
  __shared__ float ps[16][kFinishE];
  __shared__ int32_t cs[16][kFinishE], ns[16];
  const int s = blockIdx.y, tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int e = blockIdx.x * kFinishE + (lane & 15), ec = min(e, a.E - 1);
  const int lo = bound(a, s), hi = bound(a, s + 1);
  const int c0 = lo / w.chunk, c1 = hi > lo ? (hi - 1) / w.chunk + 1 : c0;   // chunks [c0, c1)
  float p = 0.0f;
  int32_t c = 0, n = 0;
#pragma unroll 8
  for (int i = c0 + (tid >> 4); i < c1; i += (int)blockDim.x / 16) {
    const size_t slot = (size_t)i + s;
    p += w.sums[slot * a.E + ec];
    c += w.counts[slot * a.E + ec];
    n += w.live[slot];
  }
  // the wave's four groups, then the waves
#pragma unroll
  for (int o = 16; o < 64; o <<= 1) {
    p += __shfl_xor(p, o, kWave);
    c += __shfl_xor(c, o, kWave);
    n += __shfl_xor(n, o, kWave);
  }
  if (lane < kFinishE) {
    ps[wave][lane] = p;
    cs[wave][lane] = c;
  }
  if (lane == 0) ns[wave] = n;
  __syncthreads();
  if (wave == 0) {
    p = 0.0f;
    c = n = 0;
    for (int i = 0; i < (int)blockDim.x / 64; i++) {
      p += ps[i][lane & 15];
      c += cs[i][lane & 15];
      n += ns[i];
    }
    const float inv = n > 0 ? 1.0f / (float)n : 0.0f;
    p *= inv;
    const bool mine = lane < kFinishE && e < a.E;
    if (mine) {
      a.probs[(size_t)s * a.E + e] = p;
      a.counts[(size_t)s * a.E + e] = c;
    }
    const float part = all_sum(mine ? (float)c * inv * p : 0.0f);
    int before = 0;
    if (lane == 0) {
      if (blockIdx.x == 0) a.live[s] = n;
      // device-scope store, complete before the ticket is taken: no cache has to be written back
      __hip_atomic_store(w.part + s * kFinishCols + blockIdx.x, part, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0)
      asm volatile("" ::: "memory");
      before = __hip_atomic_fetch_add(w.ticket + s, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (__builtin_amdgcn_readfirstlane(before) == (int)gridDim.x - 1) {
      asm volatile("" ::: "memory");
      float l = 0.0f;
      if (lane < (int)gridDim.x)            // at most kFinishCols = 64
        l = __hip_atomic_load(w.part + s * kFinishCols + lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      l = all_sum(l);
      if (lane == 0) a.loss[s] = l * ((float)a.E / (float)a.k);
    }
  }
}

// Backward: one wavefront works through a run of tokens, the next one's logits,
// ids and weights' gradients on their way while one is worked on.  The counts
// of a sequence are read where the sequence changes.  The gate weights' share
// reaches its experts through a row of LDS per wave.
template <typename ZT, int NPER, bool NT>
__global__ __launch_bounds__(256) void k_balance_backward(BalanceArgs a, int run) {
  __shared__ float gate_row[4][64 * NPER];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int t0 = (blockIdx.x * 4 + wave) * run, t1 = min(t0 + run, a.T);
  const ZT* z = static_cast<const ZT*>(a.z);
  ZT* dz = static_cast<ZT*>(a.dz);
  float* const row = gate_row[wave];
  if (t0 >= t1) return;                         // no barrier follows

  struct Token {
    float z[NPER], dw;
    int id;
    uint8_t on;
  };
  auto load = [&](int t, Token& k) {
    k.on = a.mask == nullptr ? 1 : a.mask[t];
    k.id = -1;
    k.dw = 0.0f;
    if (a.d_w != nullptr && lane < a.k) {
      k.id = a.ids[(size_t)t * a.k + lane];
      k.dw = a.d_w[(size_t)t * a.k + lane];
    }
    load_row<ZT, NPER>(z + (size_t)t * a.E, a.E, lane, k.z);
  };
  Token cur;
  load(t0, cur);
#pragma unroll
  for (int i = 0; i < NPER; i++) row[lane + 64 * i] = 0.0f;

  float g[NPER];
  int s_hi = t0;                                // tokens below s_hi belong to the sequence g is of
  bool in_seq = false;
  for (int t = t0; t < t1; t++) {
    Token next;
    load(min(t + 1, a.T - 1), next);
    if (t >= s_hi) {
      const int s = seq_of(a, t, lane);
      s_hi = s < 0 ? bound(a, 0) : bound(a, s + 1);
      in_seq = s >= 0 && t < s_hi;
      if (s_hi <= t) s_hi = t + 1;              // past every sequence, or bounds out of order: look again
      if (in_seq) {
        const float n = (float)a.live[s];
        const float f = n > 0.0f ? a.d_loss[s] * ((float)a.E / ((float)a.k * n)) / n : 0.0f;
#pragma unroll
        for (int i = 0; i < NPER; i++) g[i] = f * (float)a.counts[(size_t)s * a.E + min(lane + 64 * i, a.E - 1)];
      }
    }
    ZT* out = dz + (size_t)t * a.E;
    float d[NPER];
    if (in_seq && cur.on != 0) {
      Row<NPER> r;
      make_row<NPER>(cur.z, a.E, lane, r);
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < NPER; i++) dot = fmaf(g[i], r.t[i], dot);
      dot = all_sum(dot) * r.inv;
#pragma unroll
      for (int i = 0; i < NPER; i++) d[i] = (r.t[i] * r.inv) * r.c[i] * (g[i] - dot);
      if (a.d_w != nullptr) {
        // lane j < k: slot j (k <= 32)
        const bool in = cur.id >= 0 && cur.id < a.E;
        const float zs = in ? load_z(z + (size_t)t * a.E + cur.id) : -INFINITY, dw = in ? cur.dw : 0.0f;
        float v, c;
        sig(zs, v, c);
        float gate;
        if (a.norm_topk) {
          float tot = half_sum(v);
          if (tot < 1e-12f) {                   // uniform: as in make_row, for the token's slots
            const float m = wave_max(zs);
            if (m > -INFINITY) {
              sig_shifted(zs, m, exp_neg(m), v, c);
              tot = half_sum(v);
            }
          }
          v = tot == 0.0f ? 0.0f : v / tot;
          gate = v * c * (dw - half_sum(dw * v));
        } else {
          gate = v * c * dw;
        }
        if (in) atomicAdd(&row[cur.id], gate * a.routed_scale);
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
#pragma unroll
        for (int i = 0; i < NPER; i++) d[i] += row[lane + 64 * i];
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        if (in) row[cur.id] = 0.0f;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NPER; i++) d[i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < NPER; i++)
      if (lane + 64 * i < a.E) store_dz<NT>(out + lane + 64 * i, d[i]);
    cur = next;
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
  if (one_launch(a)) {
#define MOE_ONE(N)                                                                                            \
  do {                                                                                                        \
    const dim3 block(64 * kOneWaves<N>);                                                                      \
    if (a.dtype == 0) hipLaunchKernelGGL((k_balance_one<uint16_t, N>), dim3(a.S), block, 0, stream, a);       \
    else hipLaunchKernelGGL((k_balance_one<float, N>), dim3(a.S), block, 0, stream, a);                       \
  } while (0)
    MOE_BAL(MOE_ONE);
#undef MOE_ONE
    return hipGetLastError() == hipSuccess ? 0 : -1;
  }
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
  hipLaunchKernelGGL(k_balance_finish, dim3(ceil_div(a.E, kFinishE), a.S), dim3(w.nchunks > 64 * a.S ? 1024 : 256), 0,
                     stream, a, w);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

int launch_balance_backward(const BalanceArgs& a, hipStream_t stream) {
  if (a.T <= 0) return 0;
  // tokens per wave: 32 waves a CU and then longer runs, up to 16
  const int want = a.T / 8192, run = want < 1 ? 1 : want > 16 ? 16 : want;
  const dim3 grid(ceil_div(a.T, 4L * run));
  // logits and gradient beyond the last-level cache: the gradient streams past it (161 -> 145 us for a
  // step over 131072 x 384, whose logits the cache then still holds from the forward)
  const bool nt = 2 * (size_t)a.T * a.E * (a.dtype == 0 ? 2 : 4) > kStreamBytes;
#define MOE_BACK_T(ZT, N)                                                                                \
  do {                                                                                                   \
    if (nt) hipLaunchKernelGGL((k_balance_backward<ZT, N, true>), grid, dim3(256), 0, stream, a, run);   \
    else hipLaunchKernelGGL((k_balance_backward<ZT, N, false>), grid, dim3(256), 0, stream, a, run);     \
  } while (0)
#define MOE_BACK(N)                        \
  do {                                     \
    if (a.dtype == 0) MOE_BACK_T(uint16_t, N); \
    else MOE_BACK_T(float, N);             \
  } while (0)
  MOE_BAL(MOE_BACK);
#undef MOE_BACK
#undef MOE_BACK_T
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
