// Joins the items that a border of the column line has cut: the kernels that
// took the parts left each row's N, m and z (m in log2 units) in scratch, and
//   m = max m_k,  z = sum z_k 2^(m_k - m),  o = sum N_k 2^(m_k - m) / z,
// the sums in the order of the parts.  A kernel of its own over all SMs: the
// block that finishes last taking them instead cost 20 us for 8 parts of 256
// rows, all from one SM's share of L2, and counters that each call had to
// clear.  It is launched early and waits for the parts, so that its launch
// costs next to nothing.  Few rows over a long cache have many parts, and each
// is a trip to L2: a warp takes a row's m and z, a lane a part, and the threads
// that a block's rows leave over share the parts of a numerator.
#include "paged.cuh"

namespace fl {

constexpr int kPjRows = 32;  // rows a block
constexpr int kPjThreads = 512;
constexpr int kPjParts = 2 * kPgSms;  // an item has at most a part a block

struct PjArgs {
  PgArgs g;
  const PgCut* tile_cuts;  // [kPgSms] or NULL
  const PgCut* row_cuts;   // [2 * kPgSms] or NULL
  const float2* tile_mz;
  const float2* row_mz;
  const float4* tile_n;
  const float4* row_n;
  int row_blocks;          // blocks of the few-row kernel's items come first
};

template <int DH, int BF>
__global__ void __launch_bounds__(kPjThreads) pg_join_kernel(PjArgs a) {
  pg_wait_for_launch_before();
  const PgArgs& g = a.g;
  const bool few = (int)blockIdx.x < a.row_blocks;
  const int i0 = few ? blockIdx.x : blockIdx.x - a.row_blocks;
  const PgCut c = few ? a.row_cuts[i0] : a.tile_cuts[i0 / (kPgTileRows / kPjRows)];
  if (c.parts < 2) return;
  const int first = few ? 0 : (i0 % (kPgTileRows / kPjRows)) * kPjRows;  // row within the slot
  const int rows = c.n * g.G - c.r0;                                     // rows of the item, maybe more than the slot's
  if (first >= rows) return;
  const int slot_rows = few ? kPgFewRows : kPgTileRows;
  const float2* mz_of = (few ? a.row_mz : a.tile_mz);
  const float4* n_of = (few ? a.row_n : a.tile_n);
  // weight of each part in a row, and 1 / z
  __shared__ float s_w[kPjRows][kPjParts + 1];
  __shared__ float s_inv[kPjRows];
  __shared__ float4 s_acc[kPjThreads];
  const int live = min(rows - first, kPjRows);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // part i > 0 lies in its block's first slot
  auto slot = [&](int i) { return (size_t)(i == 0 ? c.slot0 : (c.slot0 & ~1) + 2 * i); };
  for (int r = warp; r < live; r += kPjThreads / 32) {
    float m = -INFINITY, z = 0.f;
    for (int k = lane; k < c.parts; k += 32) m = fmaxf(m, __ldcg(mz_of + slot(k) * slot_rows + first + r).x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    for (int k = lane; k < c.parts; k += 32) {
      const float2 mz = __ldcg(mz_of + slot(k) * slot_rows + first + r);
      // a part that saw nothing of the row has no weight, and no numerator in scratch
      const float w = mz.x == -INFINITY && mz.y == 0.f ? 0.f : ex2(mz.x - m);
      s_w[r][k] = w;
      if (w != 0.f) z += w * mz.y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    if (lane == 0) {
      s_inv[r] = z == 0.f ? 0.f : 1.f / z;
      const int tok = (c.r0 + first + r) / g.G, hq = c.h * g.G + (c.r0 + first + r) - tok * g.G;
      if (g.lse)
        g.lse[(size_t)hq * g.max_tokens + c.q0 + tok] = z == 0.f ? -INFINITY : (m + log2f(z)) * kPgLn2;
    }
  }
  __syncthreads();
  const int items = live * (DH / 4), pass = min(items, kPjThreads), groups = kPjThreads / pass;
  const int group = threadIdx.x / pass;
  for (int base = 0; base < items; base += pass) {
    const int i = base + threadIdx.x - group * pass;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    // the tile kernel's numerators lie [column / 4][row], the few-row kernel's [row][column / 4]
    const int r = few ? i / (DH / 4) : i % live, c4 = few ? i % (DH / 4) : i / live;
    if (group < groups && i < items) {
      const int k1 = c.parts * (group + 1) / groups;
#pragma unroll 8
      for (int k = c.parts * group / groups; k < k1; ++k) {
        const float4 x = __ldcg(n_of + (few ? (slot(k) * kPgFewRows + r) * (DH / 4) + c4
                                            : (slot(k) * (DH / 4) + c4) * kPgTileRows + first + r));
        const float w = s_w[r][k];
        if (w == 0.f) continue;
        acc.x += w * x.x;
        acc.y += w * x.y;
        acc.z += w * x.z;
        acc.w += w * x.w;
      }
    }
    s_acc[threadIdx.x] = acc;
    __syncthreads();
    if (group == 0 && i < items) {
      for (int k = 1; k < groups; ++k) {
        const float4 x = s_acc[k * pass + threadIdx.x];
        acc.x += x.x;
        acc.y += x.y;
        acc.z += x.z;
        acc.w += x.w;
      }
      const int tok = (c.r0 + first + r) / g.G, hq = c.h * g.G + (c.r0 + first + r) - tok * g.G;
      const float inv = s_inv[r];
      *reinterpret_cast<uint2*>(g.o.p + (c.q0 + tok) * g.o.st + hq * g.o.sh + c4 * 4) =
          make_uint2(pg_pack2<BF>(acc.x * inv, acc.y * inv), pg_pack2<BF>(acc.z * inv, acc.w * inv));
    }
    __syncthreads();
  }
}

int launch_pg_join(const PgArgs& g, int dh, int bf16, const PgScratch& ws, bool tiles, cudaStream_t stream) {
  PjArgs a{g, ws.tile_cuts, ws.row_cuts, ws.tile_mz, ws.row_mz, ws.tile_n, ws.row_n, ws.row_cuts ? 2 * kPgSms : 0};
  const int blocks = a.row_blocks + (tiles ? kPgSms * (kPgTileRows / kPjRows) : 0);
  if (blocks == 0) return FLASHLOOP_OK;
  auto go = [&](auto kernel) { return pg_launch_early(kernel, dim3(blocks), kPjThreads, 0, stream, a); };
  if (dh == 128) return bf16 ? go(pg_join_kernel<128, 1>) : go(pg_join_kernel<128, 0>);
  return bf16 ? go(pg_join_kernel<64, 1>) : go(pg_join_kernel<64, 0>);
}

}  // namespace fl
