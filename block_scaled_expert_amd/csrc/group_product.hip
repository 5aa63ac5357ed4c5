// Grouped MXFP4 product, few rows per group (decode, ragged calls): the time
// is that of streaming the weights of the groups that have rows.
//
// Work: one workgroup of 4 waves per (group, 16 of its rows, run of NT tiles
// of 64 weight rows); a wave takes 16 rows of each tile over the whole of k.
// Each weight byte is loaded once, by the wave that uses it, into registers (no LDS on
// that path) through a ring of PF chunks that runs on from tile to tile.  The
// operand wants 64 bytes of each of 16 rows; loaded that way every 128-byte
// line is asked for twice, and the second time it is often gone.  Each load
// takes whole lines of 8 rows instead (RawW), and two rows' halves change
// places in registers before the product (operand_w).  The group's rows of A
// are staged in LDS in operand order once for all tiles.  Sums over k stay in
// one accumulator in k order, so a result depends on nothing but its own
// operands.
//
// Measured: 512 rows over 283 of 384 groups of 4608 x 4608, 559 us (5.7 TB/s of
// all bytes); 1536 over 377 groups of 4608 x 2304, 368 us (5.8); 8 rows of 8
// groups, 22 us (4.1: the start and the end weigh).  Loads in operand order
// took 656 to 670 and 421 to 450, a workgroup per 64 weight rows 628 and 389.
#include "group_product.h"

namespace moe {

constexpr int kPanel = 18;   // chunks of A in LDS at a time (k 4608; 39 KiB per 16 rows)

constexpr int kStreamRows = 16;
constexpr size_t stream_lds(int panel) { return (size_t)panel * (1024 * kU + 64 * 2) + kStreamRows * 4; }

template <int PF, bool ODD>
__global__ __launch_bounds__(256, 4) void k_product_stream(ProductArgs p, int panel, int NT) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  v4u* const lq = reinterpret_cast<v4u*>(lds);                                     // [panel][kU][64]
  uint16_t* const ls = reinterpret_cast<uint16_t*>(lds + (size_t)panel * kU * 1024);   // [panel][64]
  int* const src = reinterpret_cast<int*>(ls + (size_t)panel * 64);                // [kStreamRows]

  Item it;
  if (!find_item<kStreamRows>(p, (p.N + 64 * NT - 1) / (64 * NT), blockIdx.x, it)) return;
  const int g = it.g, m0 = it.row0, rows = it.rows, n0 = it.bx * 64 * NT;

  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int r = lane & 15, b = lane >> 4;
  const int nb = p.K / 32;                          // scale blocks of a row
  const int chunks = (nb + kChunkBlocks - 1) / kChunkBlocks;
  const int tiles = min(NT, (p.N - n0 + 63) / 64);
  const int row_bytes = p.K / 2;
  // this wave's weight rows nw + 64 t ..; rows past N read zeros
  const int nw = n0 + 16 * wave;
  const int wrows = max(min(64 * NT - 16 * wave, p.N - nw), 0);
  const size_t wr0 = (size_t)g * p.N + min(nw, p.N - 1);
  const Buf wq = make_buf(p.w + wr0 * row_bytes, wrows * row_bytes);
  const Buf ws = make_buf(p.w_sc + wr0 * nb, wrows * nb);
  const WLane wl(r, b, row_bytes, nb);

  // chunk c of tile t
  auto load_w = [&](int t, int c, RawW& W) {
    load_raw<ODD, true>(W, wq, ws, wl, t < tiles, (uint32_t)t * (64 * row_bytes), (uint32_t)t * (64 * nb), c);
  };

  if (tid < kStreamRows) src[tid] = tid < rows ? source_row(p, m0 + tid) : -1;
  // the first weights are on their way while the rows of A are fetched
  RawW fw[PF];
  int lt = 0, lc = 0;                               // the chunk that is loaded next
  auto load_next = [&](RawW& W) {
    load_w(lt, lc, W);
    if (++lc == chunks) {
      lc = 0;
      lt++;
    }
  };
#pragma unroll
  for (int j = 0; j < PF; j++) load_next(fw[j]);

  // A's chunks [p0, p0 + pn) to LDS, a 16-byte piece (one block) per thread,
  // zeros past the end of k; rows past the tile are left as they are: a row's
  // outputs depend on that row alone
  auto stage_a = [&](int p0, int pn) {
    const int pb = kChunkBlocks * pn;
#pragma unroll 4
    for (int i = tid; i < rows * pb; i += 256) {
      const int row = i / pb, x = i - row * pb, blk = kChunkBlocks * p0 + x;
      const int s = max(src[row], 0);
      v4u v = v4u{0, 0, 0, 0};
      uint8_t sv = 0;
      if (blk < nb) {
        v = *reinterpret_cast<const v4u*>(p.a + (size_t)s * row_bytes + 16 * (size_t)blk);
        sv = p.a_sc[(size_t)s * nb + blk];
      }
      // block x of the panel: chunk x / 8, lane group (x % 8) / 2, instruction x % 2
      const int c = x / kChunkBlocks, l = row + 16 * (x % kChunkBlocks / kU);
      lq[(c * kU + x % kU) * 64 + l] = v;
      reinterpret_cast<uint8_t*>(ls + c * 64 + l)[x % kU] = sv;
    }
  };
  lds_barrier();                                    // src is written
  const bool one = chunks <= panel;
  if (one) {
    stage_a(0, chunks);
    lds_barrier();
  }

  v4f acc = v4f{0, 0, 0, 0};
  int t = 0, c = 0, pc = 0;                         // tile, chunk, chunk within the panel
  while (t < tiles) {
#pragma unroll
    for (int j = 0; j < PF; j++) {
      if (t < tiles) {
        if (!one && pc == 0) {                      // every wave is at the same chunk
          lds_barrier();                            // the last panel has been read
          stage_a(c, min(panel, chunks - c));
          lds_barrier();
        }
        Frag A, W;
        operand_w<ODD>(fw[j], W);
#pragma unroll
        for (int u = 0; u < kU; u++) A.q[u] = lq[(pc * kU + u) * 64 + lane];
        A.sc = ls[pc * 64 + lane];
        acc = mma4<0>(A, W, acc);
        acc = mma4<1>(A, W, acc);
        pc = pc + 1 == panel ? 0 : pc + 1;
        if (++c == chunks) {                        // the tile is done
          const int n = nw + 64 * t + r;
#pragma unroll
          for (int q = 0; q < 4; q++) {
            const int m = 4 * b + q;
            if (m < rows && n < p.N) store_out(p, (size_t)(m0 + m) * p.N + n, src[m] < 0 ? 0.0f : acc[q]);
          }
          acc = v4f{0, 0, 0, 0};
          c = pc = 0;
          t++;
        }
      }
      load_next(fw[j]);
    }
  }
}

// Tiles of 64 weight rows per workgroup.
static int stream_tiles(const ProductArgs& p) {
  const long nt = (long)ceil_div(p.N, 64) * max_tiles(p, kStreamRows) / 4096;
  return (int)(nt < 1 ? 1 : nt > 4 ? 4 : nt);
}

static void launch_stream(const ProductArgs& p, hipStream_t stream) {
  constexpr int PF = 6;
  const int chunks = ceil_div(p.K, kChunkK), panel = chunks < kPanel ? chunks : kPanel, nt = stream_tiles(p);
  const dim3 grid((unsigned)max_tiles(p, kStreamRows) * ceil_div(p.N, 64 * nt));
  if ((p.K / 32) % 2)
    hipLaunchKernelGGL((k_product_stream<PF, true>), grid, dim3(256), stream_lds(panel), stream, p, panel, nt);
  else
    hipLaunchKernelGGL((k_product_stream<PF, false>), grid, dim3(256), stream_lds(panel), stream, p, panel, nt);
}

// By the mean group.  At few rows the time is the weights' and they come in
// faster without LDS and its barriers; a group past 16 rows streams them twice.
// us, streamed / tiled, for a mean of 1, 4, 8, 12, 16 and 32 rows (random
// sizes): 384 groups of 4608 x 4608 458/522, 745/828, 814/865, 932/886,
// 1215/911, 1284/952; 48 of them 65/88, 101/121, 107/123, 127/123, 165/124,
// 205/130; 384 of 4608 x 2304 214/286, 358/449, 409/461, 458/466, 599/476,
// 642/505.  The mean counts empty groups, so rows that crowd into a few of many
// groups stream all the same: 8 of 384 groups with 480, 64 and 32 rows each (4608
// x 4608, fp32 out) 412/70, 80/27 and 57/22; 121 of them with 30 rows each 533/310.
int launch_group_product(const ProductArgs& p, hipStream_t stream) {
  if (p.M <= 0) return 0;
  if ((long)p.expect > 10L * p.G) return launch_product_tile(p, stream);
  launch_stream(p, stream);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace moe
