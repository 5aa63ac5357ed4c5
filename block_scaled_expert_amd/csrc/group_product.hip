// Grouped MXFP4 product, few rows per group (decode, ragged calls): the time
// is that of streaming the weights of the groups that have rows.
//
// Work: one workgroup of 4 waves per (group, 64 weight rows).  The waves split
// k four ways, each loads its weight pieces straight from HBM into matrix
// operands (each weight byte is used by one wave), the partial tiles meet in
// LDS and are added in wave order, so the result does not depend on
// scheduling.  A group without rows costs one pair of offset reads.  A group
// with more than 16 MS rows takes further passes over the same weights, which
// then come from the caches.
#include "group_product.h"

namespace moe {

constexpr int kStep = 128;   // k of one matrix instruction

template <int MS>
struct StreamLds {
  float red[4][16 * MS][64 + 1];
  int src[16 * MS];
};

template <int MS>
__global__ __launch_bounds__(256) void k_product_stream(ProductArgs p) {
  constexpr int TM = 16 * MS, PF = 2;
  __shared__ StreamLds<MS> sm;
  const int g = blockIdx.y, n0 = blockIdx.x * 64;
  int lo, hi;
  group_rows(p, g, lo, hi);
  if (lo >= hi) return;

  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int r = lane & 15, b = lane >> 4;
  const int nb = p.K / 32;                       // scale blocks of a row
  const int steps = (p.K + kStep - 1) / kStep;
  const int s0 = wave * steps / 4, s1 = (wave + 1) * steps / 4;
  const size_t row_bytes = p.K / 2;

  const uint8_t* wrow[4];
  const uint8_t* wsc[4];
#pragma unroll
  for (int c = 0; c < 4; c++) {                  // rows past N read the last row; their columns are not stored
    const size_t n = (size_t)g * p.N + min(n0 + 16 * c + r, p.N - 1);
    wrow[c] = p.w + n * row_bytes;
    wsc[c] = p.w_sc + n * nb;
  }

  for (int m0 = lo; m0 < hi; m0 += TM) {
    const int rows = min(TM, hi - m0);
    if (tid < TM) sm.src[tid] = tid < rows ? source_row(p, m0 + tid) : -1;
    __syncthreads();
    const uint8_t* arow[MS];
    const uint8_t* asc[MS];
#pragma unroll
    for (int i = 0; i < MS; i++) {               // rows past the tile read row 0; they are not stored
      const size_t s = max(sm.src[16 * i + r], 0);
      arow[i] = p.a + s * row_bytes;
      asc[i] = p.a_sc + s * nb;
    }

    v4f acc[MS][4];
#pragma unroll
    for (int i = 0; i < MS; i++)
#pragma unroll
      for (int c = 0; c < 4; c++) acc[i][c] = v4f{0, 0, 0, 0};

    Frag fa[PF][MS], fw[PF][4];
    auto load = [&](int step, Frag (&A)[MS], Frag (&W)[4]) {
      const int blk = 4 * step + b, at = min(blk, nb - 1);
#pragma unroll
      for (int c = 0; c < 4; c++) {
        W[c].q = *reinterpret_cast<const v4u*>(wrow[c] + 16 * (size_t)at);
        W[c].sc = wsc[c][at];
      }
#pragma unroll
      for (int i = 0; i < MS; i++) {
        A[i].q = *reinterpret_cast<const v4u*>(arow[i] + 16 * (size_t)at);
        A[i].sc = asc[i][at];
        // past the last block of a row (k not a multiple of 128) A is zero
        if (blk >= nb) A[i].q = v4u{0, 0, 0, 0};
      }
    };
    if (s0 < s1) {
#pragma unroll
      for (int j = 0; j < PF; j++) load(min(s0 + j, s1 - 1), fa[j], fw[j]);
    }
    for (int s = s0; s < s1; s += PF) {
#pragma unroll
      for (int j = 0; j < PF; j++) {
        if (s + j < s1) {
#pragma unroll
          for (int i = 0; i < MS; i++)
#pragma unroll
            for (int c = 0; c < 4; c++) acc[i][c] = mma4(fa[j][i], fw[j][c], acc[i][c]);
        }
        load(min(s + j + PF, s1 - 1), fa[j], fw[j]);
      }
    }

#pragma unroll
    for (int i = 0; i < MS; i++)
#pragma unroll
      for (int c = 0; c < 4; c++)
#pragma unroll
        for (int q = 0; q < 4; q++) sm.red[wave][16 * i + 4 * b + q][16 * c + r] = acc[i][c][q];
    __syncthreads();
    for (int idx = tid; idx < TM * 64; idx += 256) {
      const int m = idx >> 6, c = idx & 63;
      if (m >= rows || n0 + c >= p.N) continue;
      float v = ((sm.red[0][m][c] + sm.red[1][m][c]) + sm.red[2][m][c]) + sm.red[3][m][c];
      if (sm.src[m] < 0) v = 0.0f;
      store_out(p, (size_t)(m0 + m) * p.N + n0 + c, v);
    }
    __syncthreads();
  }
}

int launch_group_product(const ProductArgs& p, hipStream_t stream) {
  if (p.M <= 0) return 0;
  const dim3 grid(ceil_div(p.N, 64), p.G);
  // rows per pass from the mean group: 16 up to 16 rows, else 32
  if ((long)p.M <= 16L * p.G) hipLaunchKernelGGL(k_product_stream<1>, grid, dim3(256), 0, stream, p);
  else hipLaunchKernelGGL(k_product_stream<2>, grid, dim3(256), 0, stream, p);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace moe
