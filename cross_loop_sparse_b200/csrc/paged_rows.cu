// Attention of few packed rows over many columns (mma.sync, one warp a column
// slice): the decode form of the paged attention, and the plain path of every
// other call.
//
// The rows of a request and key head are packed token-major, r = token * G +
// (query head within the group), so that the G heads that share a key head
// read it once.  A block takes RT = 16 * MT packed rows and streams the
// columns in stages of 64, 16 to each of its four warps; a warp keeps its own
// ring of asynchronous copies, running maximum, sum and numerator over its
// columns, so that nothing synchronises the warps until they are joined at
// the end.  With m the running reference (log2 units, raised only when a
// score exceeds it by 8, which bounds a probability by 2^8),
//   p = 2^(s - m), z = sum p, N = sum p v, o = N / z, lse = (m + log2 z) ln 2.
// Scores, sums and N are float32; p is rounded to the values' type, since the
// matrix product takes one type.
#include <type_traits>

#include "paged.cuh"

namespace fl {

constexpr int kPrThreads = 128;
constexpr int kPrCols = 64;  // columns a stage, 16 a warp
constexpr float kPrRescale = 8.f;

template <int DH, int MT>
struct PrCfg {
  static constexpr int kRows = 16 * MT;
  static constexpr int kTile = 16 * DH * 2;  // bytes of a warp's K (or V) slice of a stage
  static constexpr int kStages = 3;
  static constexpr int kWarpRing = kStages * 2 * kTile;
  static constexpr int kPitch = DH + 8;  // floats, of the joined numerators
  static constexpr int kJoin = 4 * kRows * (kPitch + 2) * 4;
  static constexpr int kSmem = 4 * kWarpRing > kJoin ? 4 * kWarpRing : kJoin;
};

template <int DH, int BF, int MT>
__global__ void __launch_bounds__(kPrThreads) pg_rows_kernel(PgArgs g) {
  using C = PrCfg<DH, MT>;
  constexpr int kPieces = DH / 8;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.z, h = blockIdx.y, r0 = blockIdx.x * C::kRows;
  const PgSeq s = pg_seq(g, b);
  const int rows = s.n * g.G;
  if (r0 >= rows) return;
  const int shift = g.table ? g.shift : 31;
  const int off = s.L - s.n;                                      // row i sees j <= off + i
  const int ncols = max(0, off + (min(rows, r0 + C::kRows) - 1) / g.G + 1);  // of the tile's last row
  const int free_cols = off + r0 / g.G + 1;                       // columns that every row sees
  uint8_t* ring = smem + warp * C::kWarpRing;

  // queries: the A fragments of every k step
  uint32_t qa[MT][DH / 16][4];
  int lim[MT][2];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int r = r0 + mt * 16 + hf * 8 + (lane >> 2);
      const int tok = r / g.G;
      lim[mt][hf] = r < rows ? off + tok : -1;
      const uint16_t* src = g.q.p + (s.q0 + (r < rows ? tok : 0)) * g.q.st +
                            (long long)(h * g.G + (r < rows ? r - tok * g.G : 0)) * g.q.sh + (lane & 3) * 2;
#pragma unroll
      for (int ks = 0; ks < DH / 16; ++ks) {
        qa[mt][ks][hf] = r < rows ? *reinterpret_cast<const uint32_t*>(src + ks * 16) : 0u;
        qa[mt][ks][2 + hf] = r < rows ? *reinterpret_cast<const uint32_t*>(src + ks * 16 + 8) : 0u;
      }
    }

  const int stages = (ncols + kPrCols - 1) / kPrCols;
  // the page of this warp's slice of stages [32 i, 32 i + 32): lane l holds stage 32 i + l
  auto pages_of = [&](int st) -> int {
    const int col = st * kPrCols + warp * 16;
    if (col >= ncols) return -1;
    if (!g.table) return 0;
    const int page = g.table[(size_t)b * g.max_blocks + (col >> shift)];
    if (page < 0 || page >= g.n_pages) {
      set_error(g.err, FLASHLOOP_DEVERR_INDEX);
      return -1;
    }
    return page;
  };
  int pages = pages_of(lane), pages_next = pages_of(32 + lane);
  const long long row0 = g.table ? 0 : s.q0;
  auto load = [&](int st) {
    if (st < stages) {
      if ((st & 31) == 0 && st > 0) {
        pages = pages_next;
        pages_next = pages_of(st + 32 + lane);
      }
      const int page = __shfl_sync(0xffffffffu, pages, st & 31);
      const int c0 = st * kPrCols + warp * 16;
      const int in0 = g.table ? (c0 & ((1 << shift) - 1)) : c0;
      uint8_t* dst = ring + (st % C::kStages) * 2 * C::kTile;
      const uint16_t* kb = g.k.p + (page > 0 ? page : 0) * g.k.sp + (row0 + in0) * g.k.st + h * g.k.sh;
      const uint16_t* vb = g.v.p + (page > 0 ? page : 0) * g.v.sp + (row0 + in0) * g.v.st + h * g.v.sh;
#pragma unroll
      for (int it = 0; it < 16 * kPieces / 32; ++it) {
        const int i = it * 32 + lane, row = i / kPieces, c = i % kPieces;
        const int bytes = (page >= 0 && c0 + row < ncols) ? 16 : 0;  // the rest reads as zero
        const uint32_t at = row * DH * 2 + ((c ^ (row & 7)) << 4);
        cp_async16(dst + at, bytes ? kb + row * g.k.st + c * 8 : g.k.p, bytes);
        cp_async16(dst + C::kTile + at, bytes ? vb + row * g.v.st + c * 8 : g.v.p, bytes);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < C::kStages - 1; ++i) load(i);

  float o[MT][DH / 8][4];
  float m[MT][2], z[MT][2];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
    for (int n = 0; n < DH / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[mt][n][e] = 0.f;
    m[mt][0] = m[mt][1] = -INFINITY;
    z[mt][0] = z[mt][1] = 0.f;
  }

  for (int st = 0; st < stages; ++st) {
    load(st + C::kStages - 1);
    cp_async_wait<C::kStages - 1>();
    __syncwarp();
    const uint8_t* kt = ring + (st % C::kStages) * 2 * C::kTile;
    const uint8_t* vt = kt + C::kTile;
    const int c0 = st * kPrCols + warp * 16;
    float sc[MT][2][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 8; ++e) sc[mt][e >> 2][e & 3] = 0.f;
#pragma unroll
    for (int ks = 0; ks < DH / 16; ++ks) {
      // matrices: columns 0-7 / 8-15 (bit 4 of the lane) x k halves (bit 3)
      uint32_t kb[4];
      const int row = (lane & 7) + ((lane >> 4) << 3), c = ks * 2 + ((lane >> 3) & 1);
      ldmatrix_x4(kb, kt + row * DH * 2 + ((c ^ (row & 7)) << 4));
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        pg_mma<BF>(sc[mt][0], qa[mt][ks], kb[0], kb[1]);
        pg_mma<BF>(sc[mt][1], qa[mt][ks], kb[2], kb[3]);
      }
    }
    uint32_t pa[MT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int col = c0 + n * 8 + (lane & 3) * 2 + (e & 1);
          float x = sc[mt][n][e] * g.scale_log2;
          if (c0 + 16 > free_cols && col > lim[mt][e >> 1]) x = -INFINITY;
          sc[mt][n][e] = x;
          mx[e >> 1] = fmaxf(mx[e >> 1], x);
        }
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        mx[hf] = fmaxf(mx[hf], __shfl_xor_sync(0xffffffffu, mx[hf], 1));
        mx[hf] = fmaxf(mx[hf], __shfl_xor_sync(0xffffffffu, mx[hf], 2));
      }
      const bool up0 = mx[0] > m[mt][0] + kPrRescale, up1 = mx[1] > m[mt][1] + kPrRescale;
      if (__any_sync(0xffffffffu, up0 || up1)) {
        const float f0 = up0 ? ex2(m[mt][0] - mx[0]) : 1.f, f1 = up1 ? ex2(m[mt][1] - mx[1]) : 1.f;
        if (up0) m[mt][0] = mx[0];
        if (up1) m[mt][1] = mx[1];
        z[mt][0] *= f0;
        z[mt][1] *= f1;
#pragma unroll
        for (int n = 0; n < DH / 8; ++n) {
          o[mt][n][0] *= f0;
          o[mt][n][1] *= f0;
          o[mt][n][2] *= f1;
          o[mt][n][3] *= f1;
        }
      }
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const float ref = m[mt][hf] == -INFINITY ? 0.f : m[mt][hf];
          const float p0 = ex2(sc[mt][n][2 * hf] - ref), p1 = ex2(sc[mt][n][2 * hf + 1] - ref);
          z[mt][hf] += p0 + p1;
          pa[mt][n * 2 + hf] = pg_pack2<BF>(p0, p1);
        }
    }
#pragma unroll
    for (int n2 = 0; n2 < DH / 16; ++n2) {
      // matrices: k 0-7 / 8-15 (bit 3 of the lane) x n halves (bit 4)
      uint32_t vb[4];
      const int row = (lane & 7) + (((lane >> 3) & 1) << 3), c = n2 * 2 + (lane >> 4);
      ldmatrix_x4_trans(vb, vt + row * DH * 2 + ((c ^ (row & 7)) << 4));
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        pg_mma<BF>(o[mt][2 * n2], pa[mt], vb[0], vb[1]);
        pg_mma<BF>(o[mt][2 * n2 + 1], pa[mt], vb[2], vb[3]);
      }
    }
    __syncwarp();
  }
  cp_async_wait<0>();

  // join the four warps
  __syncthreads();
  float* so = reinterpret_cast<float*>(smem);           // [4][rows][pitch]
  float* sm = so + 4 * C::kRows * C::kPitch;            // [4][rows]
  float* sz = sm + 4 * C::kRows;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      float zz = z[mt][hf];
      zz += __shfl_xor_sync(0xffffffffu, zz, 1);
      zz += __shfl_xor_sync(0xffffffffu, zz, 2);
      const int r = mt * 16 + hf * 8 + (lane >> 2);
      if ((lane & 3) == 0) {
        sm[warp * C::kRows + r] = m[mt][hf];
        sz[warp * C::kRows + r] = zz;
      }
      float* d = so + (warp * C::kRows + r) * C::kPitch + (lane & 3) * 2;
#pragma unroll
      for (int n = 0; n < DH / 8; ++n)
        *reinterpret_cast<float2*>(d + n * 8) = make_float2(o[mt][n][2 * hf], o[mt][n][2 * hf + 1]);
    }
  __syncthreads();
  for (int i = threadIdx.x; i < C::kRows * (DH / 4); i += kPrThreads) {
    const int r = i / (DH / 4), c = (i % (DH / 4)) * 4;
    if (r0 + r >= rows) break;
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < 4; ++w) mm = fmaxf(mm, sm[w * C::kRows + r]);
    float zz = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float mw = sm[w * C::kRows + r];
      if (mw == -INFINITY && sz[w * C::kRows + r] == 0.f) continue;  // saw nothing
      const float f = ex2(mw - mm);
      const float4 x = *reinterpret_cast<const float4*>(so + (w * C::kRows + r) * C::kPitch + c);
      zz += f * sz[w * C::kRows + r];
      acc.x += f * x.x;
      acc.y += f * x.y;
      acc.z += f * x.z;
      acc.w += f * x.w;
    }
    const int tok = (r0 + r) / g.G, hq = h * g.G + (r0 + r) - tok * g.G;
    const float inv = zz == 0.f ? 0.f : 1.f / zz;
    uint2 out = make_uint2(pg_pack2<BF>(acc.x * inv, acc.y * inv), pg_pack2<BF>(acc.z * inv, acc.w * inv));
    *reinterpret_cast<uint2*>(g.o.p + (s.q0 + tok) * g.o.st + hq * g.o.sh + c) = out;
    if (g.lse && c == 0)
      g.lse[(size_t)hq * g.max_tokens + s.q0 + tok] = zz == 0.f ? -INFINITY : (mm + log2f(zz)) * kPgLn2;
  }
}

int launch_pg_rows(const PgArgs& g, int dh, int bf16, cudaStream_t stream) {
  const long long rows = (long long)g.max_new * g.G;
  auto go = [&](auto kernel, int rt, int smem) -> int {
    FL_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    kernel<<<dim3((unsigned)((rows + rt - 1) / rt), g.Hk, g.B), kPrThreads, smem, stream>>>(g);
    return launch_status();
  };
  auto pick = [&](auto dhc) -> int {
    constexpr int DH = decltype(dhc)::value;
    if (rows <= 16) {
      if (bf16) return go(pg_rows_kernel<DH, 1, 1>, 16, PrCfg<DH, 1>::kSmem);
      return go(pg_rows_kernel<DH, 0, 1>, 16, PrCfg<DH, 1>::kSmem);
    }
    if (bf16) return go(pg_rows_kernel<DH, 1, 2>, 32, PrCfg<DH, 2>::kSmem);
    return go(pg_rows_kernel<DH, 0, 2>, 32, PrCfg<DH, 2>::kSmem);
  };
  if (dh == 128) return pick(std::integral_constant<int, 128>{});
  return pick(std::integral_constant<int, 64>{});
}

}  // namespace fl
