// Joins the items that a border of the column line has cut: the kernels that
// took the parts left each row's N, m and z (m in log2 units) in scratch, and
//   m = max m_k,  z = sum z_k 2^(m_k - m),  o = sum N_k 2^(m_k - m) / z,
// the sums in an order that the parts alone decide.  A kernel of its own over
// all SMs: the block that finishes last taking them instead cost 20 us for 8
// parts of 256 rows, all from one SM's share of L2, and counters that each call
// had to clear.  It is launched early and waits for the parts.  What it costs are
// three dependent trips to L2 (the record, m and z, N) and the numerators' bytes:
// every lane has several loads under way, and the threads that few rows leave
// over share the parts.  3 to 5 us behind the few-row kernel, 8 us for the 148
// cuts of two chunks of 1000 rows (37 MB of numerators).
#include "paged.cuh"

namespace fl {

constexpr int kPjThreads = 512;
constexpr int kPjWarps = kPjThreads / 32;
constexpr int kPjRows = 64;           // rows of a tile item a block takes

struct PjArgs {
  PgArgs g;
  const PgCut* cuts;  // of the tile kernel, four blocks each, or of the few-row kernel, a block each
  const float2* mz;
  const float4* n;
};

// The weight of a part in a row: none if it saw nothing of it (it has no numerator in scratch either).
__device__ __forceinline__ float pj_weight(const float2& mz, float m) {
  return mz.x == -INFINITY && mz.y == 0.f ? 0.f : mz.y != mz.y ? mz.y : ex2(mz.x - m);
}

template <int BF>
__device__ __forceinline__ void pj_put(const PgArgs& g, const PgCut& c, int r, int c4, const float4& acc, float inv) {
  const int tok = g.by_g(c.r0 + r), hq = c.h * g.G + (c.r0 + r) - tok * g.G;
  *reinterpret_cast<uint2*>(g.o.p + (c.q0 + tok) * g.o.st + hq * g.o.sh + c4 * 4) =
      make_uint2(pg_pack2<BF>(acc.x * inv, acc.y * inv), pg_pack2<BF>(acc.z * inv, acc.w * inv));
}

__device__ __forceinline__ void pj_axpy(float4& acc, float w, const float4& x) {
  if (w == 0.f) return;
  acc.x += w * x.x;
  acc.y += w * x.y;
  acc.z += w * x.z;
  acc.w += w * x.w;
}

// FEW: the parts are the few-row kernel's.
template <int DH, int BF, int FEW>
__global__ void __launch_bounds__(kPjThreads) pg_join_kernel(PjArgs a) {
  constexpr int kC4 = DH / 4;
  constexpr int kRows = FEW ? kPgFewRows : kPjRows, kSlotRows = FEW ? kPgFewRows : kPgTileRows;
  constexpr int kShare = kSlotRows / kRows;                // blocks an item
  constexpr int kParts = FEW ? 2 * kPgSms : kPgSms;        // at most a part a block
  __shared__ float s_w[kRows * (kParts + 1)];              // weights [row][part]
  __shared__ float s_inv[kRows];                           // 1 / z
  __shared__ float4 s_acc[FEW ? kPjThreads : 1];
  pg_wait_for_launch_before();
  const PgArgs& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PgCut c = a.cuts[blockIdx.x / kShare];
  if (c.parts < 2) return;
  const int first = (blockIdx.x % kShare) * kRows;
  const int live = min(min(c.n * g.G - c.r0, kSlotRows) - first, kRows);
  if (live <= 0) return;
  const int pitch = c.parts | 1;
  // part i > 0 lies in its block's first slot
  auto slot = [&](int i) { return (size_t)(i == 0 ? c.slot0 : (c.slot0 & ~1) + 2 * i); };
  const float2* mz_of = a.mz + first;
  // rows' weights: `lanes` lanes a row, as many as there are parts or a warp
  const int lanes = c.parts > 16 ? 32 : c.parts > 8 ? 16 : c.parts > 4 ? 8 : 4;
  for (int r0 = 0; r0 < live; r0 += kPjWarps * (32 / lanes)) {
    const int r = r0 + warp * (32 / lanes) + lane / lanes, k0 = lane % lanes;
    const bool on = r < live;
    float m = -INFINITY, z = 0.f;
    for (int k = k0; on && k < c.parts; k += lanes) m = fmaxf(m, __ldcg(mz_of + slot(k) * kSlotRows + r).x);
    for (int o = lanes / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    for (int k = k0; on && k < c.parts; k += lanes) {
      const float2 mz = __ldcg(mz_of + slot(k) * kSlotRows + r);
      const float w = pj_weight(mz, m);
      s_w[r * pitch + k] = w;
      if (w != 0.f) z += w * mz.y;
    }
    for (int o = lanes / 2; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    if (on && k0 == 0) {
      s_inv[r] = z == 0.f ? 0.f : 1.f / z;
      const int tok = g.by_g(c.r0 + first + r), hq = c.h * g.G + (c.r0 + first + r) - tok * g.G;
      if (g.lse)
        g.lse[(size_t)hq * g.max_tokens + c.q0 + tok] = z == 0.f ? -INFINITY : (m + log2f(z)) * kPgLn2;
    }
  }
  __syncthreads();
  if (!FEW) {
    // numerators [column / 4][row]: four of a thread at a time
    constexpr int kPer = kPjRows * kC4 / kPjThreads;
    const int r = threadIdx.x % kPjRows, q0 = threadIdx.x / kPjRows;
    if (r >= live) return;
    const float4* n = a.n + (size_t)q0 * kPgTileRows + first + r;
    float4 acc[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int k = 0; k < c.parts; ++k) {
      const float4* nk = n + slot(k) * kC4 * kPgTileRows;
      float4 x[kPer];
#pragma unroll
      for (int e = 0; e < kPer; ++e) x[e] = __ldcg(nk + (size_t)e * (kPjThreads / kPjRows) * kPgTileRows);
      const float w = s_w[r * pitch + k];
#pragma unroll
      for (int e = 0; e < kPer; ++e) pj_axpy(acc[e], w, x[e]);
    }
    const float inv = s_inv[r];
#pragma unroll
    for (int e = 0; e < kPer; ++e) pj_put<BF>(g, c, first + r, q0 + e * (kPjThreads / kPjRows), acc[e], inv);
    return;
  }
  // numerators [row][column / 4]: as many groups of threads as the rows leave share the parts
  const int items = live * kC4, pass = min(items, kPjThreads), groups = kPjThreads / pass;
  const int group = threadIdx.x / pass;
  for (int base = 0; base < items; base += pass) {
    const int i = base + threadIdx.x - group * pass, r = i / kC4, c4 = i % kC4;
    const bool on = group < groups && i < items;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (on) {
      const int k1 = c.parts * (group + 1) / groups;
#pragma unroll 8
      for (int k = c.parts * group / groups; k < k1; ++k)
        pj_axpy(acc, s_w[r * pitch + k], __ldcg(a.n + (slot(k) * kPgFewRows + r) * kC4 + c4));
    }
    s_acc[threadIdx.x] = acc;
    __syncthreads();
    if (on && group == 0) {
      for (int k = 1; k < groups; ++k) pj_axpy(acc, 1.f, s_acc[k * pass + threadIdx.x]);
      pj_put<BF>(g, c, r, c4, acc, s_inv[r]);
    }
    __syncthreads();
  }
}

int launch_pg_join(const PgArgs& g, int dh, int bf16, const PgScratch& ws, cudaStream_t stream) {
  if (!ws.tile_cuts && !ws.row_cuts) return FLASHLOOP_OK;
  const bool few = ws.row_cuts != nullptr;  // a call's scratch is one kernel's
  const PjArgs a = few ? PjArgs{g, ws.row_cuts, ws.row_mz, ws.row_n} : PjArgs{g, ws.tile_cuts, ws.tile_mz, ws.tile_n};
  const int blocks = few ? 2 * kPgSms : kPgSms * (kPgTileRows / kPjRows);
  auto go = [&](auto kernel) { return pg_launch_early(kernel, dim3(blocks), kPjThreads, 0, stream, a); };
  if (few) {
    if (dh == 128) return bf16 ? go(pg_join_kernel<128, 1, 1>) : go(pg_join_kernel<128, 0, 1>);
    return bf16 ? go(pg_join_kernel<64, 1, 1>) : go(pg_join_kernel<64, 0, 1>);
  }
  if (dh == 128) return bf16 ? go(pg_join_kernel<128, 1, 0>) : go(pg_join_kernel<128, 0, 0>);
  return bf16 ? go(pg_join_kernel<64, 1, 0>) : go(pg_join_kernel<64, 0, 0>);
}

}  // namespace fl
