// Attention of few packed rows over many columns (mma.sync, one warp a column
// slice): decode steps, and small prompts and chunks whose rows would leave most
// of the tile kernel's tiles empty.
//
// The rows of a request and key head are packed token-major, r = token * G +
// (query head within the group), so that the G heads that share a key head
// read it once.  A block takes RT = 16 * MT packed rows and streams the
// columns in stages of 64, 16 to each of its four warps; a warp keeps its own
// ring of asynchronous copies, running maximum, sum and numerator over its
// columns, so that nothing synchronises the warps until they are joined at
// the end.  With m the running reference (log2 units, see PgRef),
//   p = 2^(s - m), z = sum p, N = sum p v, o = N / z, lse = (m + log2 z) ln 2.
// Scores, sums and N are float32.  The matrix product takes p in the values'
// type.  Up to 16 packed rows, what that rounding drops is multiplied with V too,
// so that the rounding of o alone is left: up to 8 rows in the places of rows 8
// to 15, at no cost, up to 16 in products of their own (16 contexts of 16384
// tokens, 16 heads a key head: 95 to 98 us).  With more rows, whose products
// bound the kernel, p is rounded, which makes the error sqrt(2) times as large.
//
// Bound by HBM: a column costs 4 * head_dim bytes and few instructions (8 contexts
// of 32768 tokens, 16 heads of 128: 306 to 314 us by card, 6.8 to 7.0 TB/s; with 32
// packed rows a key head 100 us for 537 MB, 5.4 TB/s, where eight warps an SM cannot
// hide two tiles' products).  With
// scratch, the stages of all requests and key heads are one line that is cut
// into equal lengths, one a block and two blocks an SM, so that requests of any
// mix of lengths load the SMs alike; what a border cuts leaves float32 N, m and z
// in scratch, which another kernel joins.  Short tables need no cut and no
// scratch: a block a request, key head and row tile.
#include <type_traits>

#include "paged.cuh"

namespace fl {

constexpr int kPrThreads = 128;
constexpr int kPrCols = 64;  // columns a stage, 16 a warp

template <int DH, int MT>
struct PrCfg {
  static constexpr int kRows = 16 * MT;
  static constexpr int kTile = 16 * DH * 2;  // bytes of a warp's K (or V) slice of a stage
  // 128 KB an SM on their way are enough for HBM, and more are slower: 8 contexts of 32768 tokens
  // take 308 us with 2 stages of 16 heads of 128 and 320 with 3 on one card, 98 us with 3 stages of
  // 8 heads of 64, 99 with 2, 102 with 4 and 104 with 6
  static constexpr int kStages = DH == 128 ? 2 : 3;
  static constexpr int kWarpRing = kStages * 2 * kTile;
  static constexpr int kPitch = DH + 8;  // floats, of the joined numerators
  static constexpr int kJoin = 4 * kRows * (kPitch + 2) * 4;
  static constexpr int kSmem = 4 * kWarpRing > kJoin ? 4 * kWarpRing : kJoin;
};

constexpr int kPrMinUnits = 4;  // units a block takes at least when the line is cut
// Units of an item beside its stages: what starting and joining it costs, as
// much as some stages do.  Without them a block that gets dozens of short
// requests ends long after the others.
constexpr int kPrStart = 6;

struct PrArgs {
  PgArgs g;
  PgCut* cuts;      // [grid]; NULL: blocks take whole row tiles
  float2* part_mz;  // [2 * grid, 32]
  float4* part_n;   // [2 * grid, 32, DH / 4]
};

// Columns [c0, c1) of the rows from r0 on of one request and key head.
struct PrItem {
  int b, h, q0, n, L, r0, c0, c1;
  int slot, parts;  // scratch slot, number of parts of the whole item (1 = this is all)
};

// LO: what the rounding of p to the values' type drops goes through the product
// with V too, in the place of rows 8 to 15 (1) or in a product of its own (2).
//
// True, with nothing written, if a numerator is not finite and some row does not see all of the
// item's columns: zero times a value that is not finite may have got there.  The item is then taken
// AGAIN, with such values of those columns as zeros in the product and added where they are seen.
// (Looking the values over before the product instead took prompts of 300 tokens from 8.0 to 8.7 us.)
template <int DH, int BF, int MT, int LO, bool AGAIN>
__device__ __forceinline__ bool pr_item(const PrArgs& a, const PrItem& s, uint8_t* smem) {
  using C = PrCfg<DH, MT>;
  constexpr int kPieces = DH / 8;
  constexpr int kHalves = LO == 1 ? 1 : 2;  // eights of rows that a tile's are
  const PgArgs& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = s.b, h = s.h, r0 = s.r0;
  const int rows = s.n * g.G;
  const int shift = g.table ? g.shift : 31;
  const int off = s.L - s.n;                 // row i sees j <= off + i
  const int free_cols = off + g.by_g(r0) + 1;  // columns that every row sees
  const int ncols = s.c1;
  uint8_t* ring = smem + warp * C::kWarpRing;

  // queries: the A fragments of every k step
  uint32_t qa[MT][DH / 16][4];
  int lim[MT][2];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int r = r0 + mt * 16 + hf * 8 + (lane >> 2);
      const int tok = g.by_g(r);
      lim[mt][hf] = r < rows ? off + tok : -1;
      const uint16_t* src = g.q.p + (s.q0 + (r < rows ? tok : 0)) * g.q.st +
                            (long long)(h * g.G + (r < rows ? r - tok * g.G : 0)) * g.q.sh + (lane & 3) * 2;
#pragma unroll
      for (int ks = 0; ks < DH / 16; ++ks) {
        qa[mt][ks][hf] = r < rows ? *reinterpret_cast<const uint32_t*>(src + ks * 16) : 0u;
        qa[mt][ks][2 + hf] = r < rows ? *reinterpret_cast<const uint32_t*>(src + ks * 16 + 8) : 0u;
      }
    }

  const int stages = ncols > s.c0 ? (ncols - s.c0 + kPrCols - 1) / kPrCols : 0;
  // the page of this warp's slice of stages [32 i, 32 i + 32): lane l holds stage 32 i + l
  auto pages_of = [&](int st) -> int {
    const int col = s.c0 + st * kPrCols + warp * 16;
    if (st >= stages || col >= ncols) return -1;
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
  // A lane brings 16 bytes of every kStep-th row of K and of V, beginning with row `up`; row r's
  // 16-byte piece c lies at place c ^ (r & 7), so that ldmatrix's eight rows fall on all banks.
  // The addresses advance by a constant a copy (computed anew for each of them, with a check a
  // row, issuing took 530 to 1380 cycles a stage, as much as everything else); the last columns
  // and bad pages take the checks.
  constexpr int kStep = 32 / kPieces;
  const int up = lane / kPieces, piece = lane % kPieces;
  const uint32_t to = smem_u32(ring) + up * (DH * 2);
  const uint16_t* k_lane = g.k.p + h * g.k.sh + (row0 + up) * g.k.st + piece * 8;
  const uint16_t* v_lane = g.v.p + h * g.v.sh + (row0 + up) * g.v.st + piece * 8;
  const long long k_step = kStep * g.k.st, v_step = kStep * g.v.st;
  auto load = [&](int st) {
    if (st < stages) {
      if ((st & 31) == 0 && st > 0) {
        pages = pages_next;
        pages_next = pages_of(st + 32 + lane);
      }
      const int page = __shfl_sync(0xffffffffu, pages, st & 31);
      const int c0 = s.c0 + st * kPrCols + warp * 16;
      const int in0 = g.table ? (c0 & ((1 << shift) - 1)) : c0;
      const uint32_t dst = to + (st % C::kStages) * 2 * C::kTile;
      const uint16_t* ks = k_lane + (page > 0 ? page : 0) * g.k.sp + in0 * g.k.st;
      const uint16_t* vs = v_lane + (page > 0 ? page : 0) * g.v.sp + in0 * g.v.st;
      if (page >= 0 && c0 + 16 <= ncols) {
#pragma unroll
        for (int it = 0; it < 16 / kStep; ++it) {
          const uint32_t at = dst + it * kStep * DH * 2 + ((piece ^ ((it * kStep + up) & 7)) << 4);
          cp_async16_to(at, ks);
          cp_async16_to(at + C::kTile, vs);
          ks += k_step;
          vs += v_step;
        }
      } else {
#pragma unroll 1
        for (int it = 0; it < 16 / kStep; ++it) {
          const uint32_t at = dst + it * kStep * DH * 2 + ((piece ^ ((it * kStep + up) & 7)) << 4);
          const int bytes = (page >= 0 && c0 + it * kStep + up < ncols) ? 16 : 0;  // the rest reads as zero
          cp_async16_to(at, bytes ? ks : g.k.p, bytes);
          cp_async16_to(at + C::kTile, bytes ? vs : g.v.p, bytes);
          ks += k_step;
          vs += v_step;
        }
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < C::kStages; ++i) load(i);

  float o[MT][DH / 8][4], ol[MT][LO == 2 ? DH / 8 : 1][4];
  float m[MT][2], z[MT][2];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
    for (int n = 0; n < DH / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[mt][n][e] = ol[mt][LO == 2 ? n : 0][e] = 0.f;
    m[mt][0] = m[mt][1] = -INFINITY;
    z[mt][0] = z[mt][1] = 0.f;
  }

  for (int st = 0; st < stages; ++st) {
    cp_async_wait<C::kStages - 1>();
    __syncwarp();
    const uint8_t* kt = ring + (st % C::kStages) * 2 * C::kTile;
    uint8_t* vt = ring + (st % C::kStages) * 2 * C::kTile + C::kTile;
    const int c0 = s.c0 + st * kPrCols + warp * 16;
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
    uint32_t pa[MT][4], lo[MT][4];
    if (c0 + 16 > free_cols) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2 * kHalves; ++e)
            if (c0 + n * 8 + (lane & 3) * 2 + (e & 1) > lim[mt][e >> 1]) sc[mt][n][e] = -INFINITY;
      if (AGAIN) {
        for (int i = max(0, free_cols - c0) * kPieces + lane; i < 16 * kPieces; i += 32) {
          uint4* at = reinterpret_cast<uint4*>(vt + i * 16);
          const uint4 x = *at;
          *at = make_uint4(pg_finite_part<BF>(x.x), pg_finite_part<BF>(x.y), pg_finite_part<BF>(x.z), pg_finite_part<BF>(x.w));
        }
        __syncwarp();
      }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int hf = 0; hf < kHalves; ++hf) {
        mx[hf] = fmaxf(fmaxf(sc[mt][0][2 * hf], sc[mt][0][2 * hf + 1]), fmaxf(sc[mt][1][2 * hf], sc[mt][1][2 * hf + 1]));
        mx[hf] = fmaxf(mx[hf], __shfl_xor_sync(0xffffffffu, mx[hf], 1));
        mx[hf] = fmaxf(mx[hf], __shfl_xor_sync(0xffffffffu, mx[hf], 2)) * g.scale_log2;
      }
      const bool up0 = mx[0] > m[mt][0] + PgRef<BF>::kRise, up1 = mx[1] > m[mt][1] + PgRef<BF>::kRise;
      if (__any_sync(0xffffffffu, up0 || up1)) {
        mx[0] -= PgRef<BF>::kLift;
        mx[1] -= PgRef<BF>::kLift;
        const float f0 = up0 ? ex2(m[mt][0] - mx[0]) : 1.f;
        const float f1 = LO == 1 ? f0 : up1 ? ex2(m[mt][1] - mx[1]) : 1.f;
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
          if (LO == 2) {
            ol[mt][n][0] *= f0;
            ol[mt][n][1] *= f0;
            ol[mt][n][2] *= f1;
            ol[mt][n][3] *= f1;
          }
        }
      }
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int hf = 0; hf < kHalves; ++hf) {
          const float ref = m[mt][hf] == -INFINITY ? 0.f : m[mt][hf];
          const float p0 = ex2(fmaf(sc[mt][n][2 * hf], g.scale_log2, -ref));
          const float p1 = ex2(fmaf(sc[mt][n][2 * hf + 1], g.scale_log2, -ref));
          z[mt][hf] += p0 + p1;
          pa[mt][n * 2 + hf] = pg_pack2<BF>(p0, p1);
          if (LO) {
            const float2 h = pg_unpack2<BF>(pa[mt][n * 2 + hf]);
            (LO == 1 ? pa[mt][n * 2 + 1] : lo[mt][n * 2 + hf]) = pg_pack2<BF>(p0 - h.x, p1 - h.y);
          }
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
        if (LO == 2) {
          pg_mma<BF>(ol[mt][2 * n2], lo[mt], vb[0], vb[1]);
          pg_mma<BF>(ol[mt][2 * n2 + 1], lo[mt], vb[2], vb[3]);
        }
      }
    }
    __syncwarp();
    load(st + C::kStages);
  }
  cp_async_wait<0>();

  const bool look = !AGAIN && ncols > free_cols;
  bool odd = false;
  if (look) {
    float t[4] = {0.f, 0.f, 0.f, 0.f};  // zeros, or NaN
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int n = 0; n < DH / 8; ++n)
#pragma unroll
        for (int e = 0; e < 2 * kHalves; ++e) t[e] = fmaf(o[mt][n][e], 0.f, t[e]);
    odd = !((t[0] + t[1]) + (t[2] + t[3]) == 0.f);
  }

  // join the four warps
  __syncthreads();
  float* so = reinterpret_cast<float*>(smem);           // [4][rows][pitch]
  float* sm = so + 4 * C::kRows * C::kPitch;            // [4][rows]
  float* sz = sm + 4 * C::kRows;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int hf = 0; hf < kHalves; ++hf) {
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
      {
        float2 x = make_float2(o[mt][n][2 * hf], o[mt][n][2 * hf + 1]);
        if (LO) {  // an infinite value gives an infinite product with p, and one of any sign, or none, with the rest
          const float2 l = LO == 1 ? make_float2(o[mt][n][2], o[mt][n][3]) : make_float2(ol[mt][n][2 * hf], ol[mt][n][2 * hf + 1]);
          if (isfinite(l.x)) x.x += l.x;
          if (isfinite(l.y)) x.y += l.y;
        }
        *reinterpret_cast<float2*>(d + n * 8) = x;
      }
    }
  if (!look) __syncthreads();
  else if (__syncthreads_or(odd)) return true;
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
    if (AGAIN) {
      const int end = min(off + g.by_g(r0 + r) + 1, ncols);
#pragma unroll 1
      for (int j = max(free_cols, s.c0); j < end; ++j) {
        const uint16_t* v = g.v.p + h * g.v.sh + c;
        if (g.table) {
          const int page = g.table[(size_t)b * g.max_blocks + (j >> shift)];
          if (page < 0 || page >= g.n_pages) continue;
          v += page * g.v.sp + (j & ((1 << shift) - 1)) * g.v.st;
        } else {
          v += (row0 + j) * g.v.st;
        }
        if (pg_not_finite<BF>(v[0])) acc.x += pg_unpack2<BF>(v[0]).x;
        if (pg_not_finite<BF>(v[1])) acc.y += pg_unpack2<BF>(v[1]).x;
        if (pg_not_finite<BF>(v[2])) acc.z += pg_unpack2<BF>(v[2]).x;
        if (pg_not_finite<BF>(v[3])) acc.w += pg_unpack2<BF>(v[3]).x;
      }
    }
    if (s.parts > 1) {
      const size_t at = (size_t)s.slot * kPgFewRows + r;
      __stcg(a.part_n + at * (DH / 4) + c / 4, acc);
      if (c == 0) __stcg(a.part_mz + at, make_float2(mm, zz));
      continue;
    }
    const int tok = g.by_g(r0 + r), hq = h * g.G + (r0 + r) - tok * g.G;
    const float inv = zz == 0.f ? 0.f : 1.f / zz;
    *reinterpret_cast<uint2*>(g.o.p + (s.q0 + tok) * g.o.st + hq * g.o.sh + c) =
        make_uint2(pg_pack2<BF>(acc.x * inv, acc.y * inv), pg_pack2<BF>(acc.z * inv, acc.w * inv));
    if (g.lse && c == 0)
      g.lse[(size_t)hq * g.max_tokens + s.q0 + tok] = zz == 0.f ? -INFINITY : (mm + log2f(zz)) * kPgLn2;
  }
  return false;
}
template <int DH, int BF, int MT, int LO>
__device__ __forceinline__ void pr_take(const PrArgs& a, const PrItem& it, uint8_t* smem) {
  if (pr_item<DH, BF, MT, LO, false>(a, it, smem)) pr_item<DH, BF, MT, LO, true>(a, it, smem);
}

// Units of a row tile of request s (a request whose rows see nothing still has them written), and
// the request's row tiles of one key head.
__device__ __forceinline__ int pr_units(const PgSeq& s) { return kPrStart + max(1, (s.L + kPrCols - 1) / kPrCols); }
__device__ __forceinline__ int pr_tiles(const PgArgs& g, const PgSeq& s) {
  return (s.n * g.G + kPgFewRows - 1) / kPgFewRows;
}

// By the rows of the request: up to 16 do half of a 32-row tile's products.  The kernel of 16-row
// tiles takes requests of any number of rows.
template <int DH, int BF, int MT>
__device__ __forceinline__ void pr_one(const PrArgs& a, const PrItem& it, uint8_t* smem) {
  const int rows = it.n * a.g.G;
  if (rows <= 8) pr_take<DH, BF, 1, 1>(a, it, smem);
  else if (MT == 1 || rows <= 16) pr_take<DH, BF, 1, 2>(a, it, smem);
  else pr_take<DH, BF, MT, 0>(a, it, smem);
}

template <int DH, int BF, int MT>
__global__ void __launch_bounds__(kPrThreads) pg_rows_kernel(PrArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_b;
  __shared__ long long s_sum[kPrThreads / 32], s_at;
  pg_wait_for_launch_before();
  pg_launch_next();
  const PgArgs& g = a.g;
  if (a.cuts == nullptr) {
    const PgSeq q = pg_seq(g, blockIdx.z);
    const int rows = q.n * g.G, r0 = (gridDim.x - 1 - blockIdx.x) * PrCfg<DH, MT>::kRows;  // long ones first
    if (r0 >= rows) return;
    const int seen = q.L - q.n + g.by_g(min(rows, r0 + PrCfg<DH, MT>::kRows) - 1) + 1;  // by the tile's last row
    PrItem it{(int)blockIdx.z, (int)blockIdx.y, q.q0, q.n, q.L, r0, 0, max(0, seen), 0, 1};
    pr_one<DH, BF, MT>(a, it, smem);
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // a thread's request of the chunk at b0, and sums over the chunk: inclusive and whole
  PgSeq q;
  long long mine, incl, whole;
  auto chunk = [&](int b0) {
    q = {0, 0, 0};
    if (b0 + tid < g.B) q = pg_seq(g, b0 + tid);
    incl = (long long)pr_units(q) * pr_tiles(g, q);
    mine = incl;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    __syncthreads();
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    whole = 0;
#pragma unroll
    for (int w = 0; w < kPrThreads / 32; ++w) {
      if (w < warp) incl += s_sum[w];
      whole += s_sum[w];
    }
  };
  long long total = 0;
  for (int b0 = 0; b0 < g.B; b0 += kPrThreads) {
    chunk(b0);
    total += whole;
  }
  total *= g.Hk;
  if (tid == 0) a.cuts[blockIdx.x].parts = 0;
  const long long per = max((long long)kPrMinUnits, pg_div(total + gridDim.x - 1, gridDim.x));
  long long x = blockIdx.x * per;
  const long long x1 = min(total, x + per);
  if (x >= x1) return;
  // the request that holds x
  long long base = 0;
  for (int b0 = 0; b0 < g.B; b0 += kPrThreads) {
    if (g.B > kPrThreads) chunk(b0);
    const long long first = base + (incl - mine) * g.Hk;
    if (x >= first && x < base + incl * g.Hk) {
      s_b = b0 + tid;
      s_at = first;
    }
    base += whole * g.Hk;
    if (x < base) break;
  }
  __syncthreads();
  int b = s_b;
  long long at = s_at;  // the request's first unit
  while (x < x1) {
    q = pg_seq(g, b);
    const int u = pr_units(q), tiles = pr_tiles(g, q);
    const long long next = at + (long long)u * tiles * g.Hk;
    while (x < x1 && x < next) {
      PrItem it{};
      it.b = b;
      const int idx = (int)pg_div(x - at, u);  // key head by key head, the row tiles of one next to each other
      it.h = idx / tiles;
      it.r0 = (idx - it.h * tiles) * kPgFewRows;
      it.q0 = q.q0;
      it.n = q.n;
      it.L = q.L;
      const long long u1 = at + (long long)(idx + 1) * u, end = min(u1, x1);
      const long long s0 = u1 - u + kPrStart;  // its first stage
      if (end <= s0) {  // the next block has its stages
        x = end;
        break;
      }
      it.c0 = (int)max(0ll, x - s0) * kPrCols;
      const int last = min(q.n * g.G, it.r0 + kPgFewRows) - 1;  // its last row, which sees the most
      it.c1 = max(0, min(q.L - q.n + g.by_g(last) + 1, (int)(end - s0) * kPrCols));
      const long long fc = pg_div(s0, per), lc = pg_div(u1 - 1, per);
      it.parts = (int)(lc - fc) + 1;
      // the first item of a block has its slot 0, the last, if it goes on behind the block, slot 1
      it.slot = blockIdx.x * 2 + (fc == blockIdx.x && s0 != fc * per);
      if (it.parts > 1 && fc == blockIdx.x && tid == 0)
        a.cuts[blockIdx.x] = PgCut{it.parts, it.slot, it.h, it.q0, it.n, it.r0, {0, 0}};
      pr_one<DH, BF, MT>(a, it, smem);
      __syncthreads();  // shared memory goes to the next item
      x = end;
    }
    at = next;
    ++b;
  }
}

int launch_pg_rows(const PgArgs& g, int dh, int bf16, const PgScratch& ws, cudaStream_t stream) {
  PrArgs a{g, ws.row_cuts, ws.row_mz, ws.row_n};
  const long long rows = (long long)g.max_new * g.G;
  // Whole tiles of 16 rows if every SM gets one at most: a stage of 16 is shorter (4 prompts of 100
  // tokens, 4 heads of 128: 5.0 us against 7.9), but two blocks of 16 on an SM take longer than one
  // of 32 (16 of 128 tokens, 4 heads of 64: 8.3 against 6.2).
  const long long tiles16 = (long long)g.max_tokens * g.Hq / 16 + (long long)(g.B < g.max_tokens ? g.B : g.max_tokens) * g.Hk / 2;
  const bool narrow = rows <= 16 || (!a.cuts && tiles16 <= kPgSms);
  auto go = [&](auto kernel, int rt, int smem) -> int {
    FL_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    dim3 grid((unsigned)((rows + rt - 1) / rt), g.Hk, g.B);
    if (a.cuts) grid = dim3(2 * kPgSms);  // each leaves a record
    return pg_launch_early(kernel, grid, kPrThreads, smem, stream, a);
  };
  auto pick = [&](auto dhc) -> int {
    constexpr int DH = decltype(dhc)::value;
    if (narrow) {
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
