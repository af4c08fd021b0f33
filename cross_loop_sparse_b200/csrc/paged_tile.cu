// Attention of many packed rows over many columns (tcgen05): packed prompts
// and chunks of new tokens over a paged cache.
//
// The rows of a request and key head are packed token-major, r = token * G +
// (query head within the group): grouped heads fill a tile with rows that
// read the same keys.  Work item: one request, key head and pair of 128-row
// tiles A, B, over a range of 128-column tiles; A and B share every K / V
// tile.  Per row, with s the scores in log2 units and m a reference raised
// only by leaps (see PgRef),
//   p = 2^(s - m), z = sum p, N = sum p v, o = N / z, lse = (m + log2 z) ln 2;
// scores, z and N in float32, p rounded to the values' type because the
// matrix product takes one type for both operands.
//
// Shared memory: the pair's queries (2 x 128 x DH) and a ring of K / V slots of
// 128 columns (K-major K tiles; V as it lies in memory, MN-major), all in the
// 128-byte swizzle.  K and V come by TMA: one box of 128 tokens of packed rows
// or of a page, or one box a page where pages are smaller.  Boxes of pages
// behind the request's end start outside the tensor and fill with zeros.  The
// V rows that some row of the pair does not see are looked over before the tile
// is handed on, since 0 * NaN would reach that row: those that no row sees are
// cleared, and what is not finite of the others is set to zero and added to the
// numerators of the rows that see it when they are written back.  A prompt of 32768
// tokens x 16 heads takes 4156 us with that and 4124 without, 20 prompts of 700
// tokens x 32 heads 137 and 130; by the row warps instead of the loads' 144.
// TMEM (512 columns): N_A, N_B, then the tiles' 128-column scores; the P of a
// 64-column half is written over the half's first 32 score columns and feeds
// that half's P.V from TMEM.  The next tile's scores of a half are issued right
// behind that P.V, so that they are there when the rows have done the other
// half.  A score MMA is 64 wide for this: it takes 48 cycles a k step where 32
// would do (it reads the queries for half as many columns, and shared memory
// gives 128 bytes a clock), but 128-wide ones, at their full rate, leave the rows
// waiting for a whole P.V and score MMA a tile: 4.1 ms against 3.5 ms for a
// prompt of 32768 tokens x 16 heads on a cool card (at its power cap this one takes 4.2).
//
// Roles (16 warps): 0-3 / 4-7 rows of tile A / B, one thread a row; 8-11
// queries of the next item and write-back of the last, while the row warps take
// the next one's exponentials; 12 TMEM and K / V loads (lane = page of a tile);
// 13 / 14 MMA issue of tile A / B; 15 work items.
//
// What bounds it, a pair of 128-column tiles: the MMAs take 2560 cycles (1536
// scores, 1024 P.V), the exponentials 2300 (MUFU gives 16 a clock; a row thread's
// other instructions fit beside them), and a pair takes 3450 as they meet.
// Exponentials by polynomial on the FMA units were no gain at any share: two
// warps a scheduler cannot keep both units fed (1101 cycles a half with a quarter
// of them against 1166 without, alone, and a slower kernel).
//
// Work: without scratch (prompts) an item is a whole row pair, dealt to and fro
// from a list that begins with the longest.  With scratch (paged) the column
// tiles of all items are one line that is cut into equal lengths, one a block,
// so that few rows over a long cache still use every SM; an item cut by a
// border leaves float32 N, m and z in scratch, which another kernel joins.
//
// Every wait is bounded; one that gives up sets FLASHLOOP_DEVERR_TIMEOUT, and the
// block unwinds.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <type_traits>

#include "paged.cuh"
#include "tc_util.cuh"

namespace fl {

constexpr int kPtRows = 128;
constexpr int kPtPair = 2 * kPtRows;
constexpr int kPtCols = 128;
constexpr int kPtThreads = 512;
constexpr int kPtWarpQ = 8, kPtWarpTma = 12, kPtWarpMma = 13, kPtWarpSched = 15;
constexpr int kPtRegsRows = 192, kPtRegsRest = 64;  // of the 65536 registers: 256 threads of each
constexpr int kPtReaders = 15;   // arrivals that free a work item's slot: 8 + 4 + 1 + 2 warps
constexpr int kPtMinUnits = 4;   // units a block takes at least when the line is cut
constexpr int kPtStart = 2;      // units of an item beside its column tiles: what starting and writing it costs

template <int DH>
struct PtCfg {
  static constexpr int kQChunk = kPtRows * 128;
  static constexpr int kQBytes = kPtRows * DH * 2;
  static constexpr int kChunk = kPtCols * 128;  // 128 tokens x 64 elements
  static constexpr int kSlotBytes = kPtCols * DH * 2;
  static constexpr int kStages = DH == 128 ? 5 : 8;
  static constexpr int kRingOff = 2 * kQBytes;
  static constexpr int kBarOff = kRingOff + kStages * kSlotBytes;
  static constexpr int kInvOff = kBarOff + 512;  // 1 / z of both tiles' rows
  static constexpr int kSmem = 1024 + kInvOff + 2 * kPtRows * 4;
  static_assert(kSmem <= 232448, "shared memory per block");
};

struct PtItem {
  int valid, b, h, q0, n, L, r0;
  int t0, t1;            // column tiles
  int slot, parts;       // scratch slot, number of parts of the whole item (1 = this is all)
  int odd;               // set by the loads: V rows that not every row sees held values that are not finite
};

struct PtArgs {
  PgArgs g;
  int box_shift;  // tokens of a TMA box: 1 << box_shift
  PgCut* cuts;      // [grid]; NULL: items are whole
  float2* part_mz;  // [2 * grid, 256]
  float4* part_n;   // [2 * grid, DH / 4, 256]
};

__device__ __forceinline__ int pt_pairs(const PtArgs& a, int n) {
  return (n * a.g.G + kPtPair - 1) / kPtPair;
}
// Column tiles that the rows before packed row `end` see.
__device__ __forceinline__ int pt_tiles(int n, int L, const PgArgs& g, int end) {
  const int f = L - n + g.by_g(min(end, n * g.G) - 1) + 1;
  return f > 0 ? (f + kPtCols - 1) / kPtCols : 0;
}
// Units of pair p on the line that is cut; a pair that sees no column still has its rows written.
__device__ __forceinline__ int pt_units(int n, int L, const PgArgs& g, int p) {
  return kPtStart + max(1, pt_tiles(n, L, g, (p + 1) * kPtPair));
}

// First of np pairs with at least `units` column tiles (they grow with the pair); np if none.
__device__ __forceinline__ int pt_first_pair(int n, int L, int G, int np, int units) {
  const long long x = (long long)(units - 1) * kPtCols - (L - n);  // its last row's position, at least
  if (units <= 1 || x <= 0) return 0;
  if (x > n - 1) return np;
  return (int)min((long long)np - 1, (x * G + kPtPair) / kPtPair - 1);
}

// Warp 15: cuts the work into items.  `emit` returns false when the block ends.
template <typename Emit>
__device__ __forceinline__ void pt_schedule(const PtArgs& a, int lane, Emit emit) {
  const PgArgs& g = a.g;
  const int G = g.G;
  constexpr unsigned kAll = 0xffffffffu;
  // lane's request of the chunk at b0, and its pairs
  PgSeq s;
  int np;
  auto chunk = [&](int b0) {
    s = {0, 0, 0};
    if (b0 + lane < g.B) s = pg_seq(g, b0 + lane);
    np = pt_pairs(a, s.n);
  };
  if (a.cuts == nullptr) {
    // whole items, dealt out to and fro (block c takes items c, 2 grid - 1 - c, 2 grid + c, ...) from
    // a list that begins with the longest: those of 2^c column tiles and more, c falling, and
    // within a class and request the last rows first
    long long item = blockIdx.x, round = 0, base = 0;
    int loaded = -1;
    for (int cls = 31 - __clz(max(1, (g.max_new + kPtCols - 1) / kPtCols)); cls >= 0; --cls) {
      for (int b0 = 0; b0 < g.B; b0 += 32) {
        if (loaded != b0) chunk(b0);
        loaded = b0;
        const int p0 = pt_first_pair(s.n, s.L, G, np, 1 << cls), p1 = pt_first_pair(s.n, s.L, G, np, 2 << cls);
        const long long mine = (long long)(p1 - p0) * g.Hk;
        long long end = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long y = __shfl_up_sync(kAll, end, o);
          if (lane >= o) end += y;
        }
        const long long total = __shfl_sync(kAll, end, 31);
        while (item < base + total) {
          const int src = __ffs(__ballot_sync(kAll, base + end > item)) - 1;
          const int idx = (int)(item - base - __shfl_sync(kAll, end - mine, src));
          PtItem it{};
          it.valid = 1;
          it.b = b0 + src;
          it.h = idx % g.Hk;
          it.q0 = __shfl_sync(kAll, s.q0, src);
          it.n = __shfl_sync(kAll, s.n, src);
          it.L = __shfl_sync(kAll, s.L, src);
          it.r0 = (__shfl_sync(kAll, p1, src) - 1 - idx / g.Hk) * kPtPair;
          it.t1 = pt_tiles(it.n, it.L, g, it.r0 + kPtPair);
          it.parts = 1;
          if (!emit(it)) return;
          ++round;
          item = round * gridDim.x + ((round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
        }
        base += total;
      }
    }
    return;
  }
  // column tiles of one key head of the lane's request (of the chunk loaded last)
  auto head_units = [&]() -> long long {
    long long u = 0;
    if (np <= 8)
      for (int p = 0; p < np; ++p) u += pt_units(s.n, s.L, g, p);
    unsigned big = __ballot_sync(kAll, np > 8);
    while (big) {
      const int src = __ffs(big) - 1;
      big &= big - 1;
      const int n_p = __shfl_sync(kAll, np, src), n = __shfl_sync(kAll, s.n, src), L = __shfl_sync(kAll, s.L, src);
      long long v = 0;
      for (int p = lane; p < n_p; p += 32) v += pt_units(n, L, g, p);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
      if (lane == src) u = v;
    }
    return u;
  };
  long long total = 0, hu = 0;
  for (int b0 = 0; b0 < g.B; b0 += 32) {
    chunk(b0);
    hu = head_units();
    long long u = hu * g.Hk;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) u += __shfl_xor_sync(kAll, u, o);
    total += u;
  }
  if (lane == 0) a.cuts[blockIdx.x].parts = 0;
  const long long per = max((long long)kPtMinUnits, pg_div(total + gridDim.x - 1, gridDim.x));
  long long x = blockIdx.x * per;
  const long long x1 = min(total, x + per);
  long long base = 0;
  for (int b0 = 0; b0 < g.B && x < x1; b0 += 32) {
    if (g.B > 32) {
      chunk(b0);
      hu = head_units();
    }
    const long long mine = hu * g.Hk;
    long long end = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(kAll, end, o);
      if (lane >= o) end += y;
    }
    const long long chunk_total = __shfl_sync(kAll, end, 31);
    while (x < x1 && x < base + chunk_total) {
      const int src = __ffs(__ballot_sync(kAll, base + end > x)) - 1;
      const int n_p = __shfl_sync(kAll, np, src);
      const long long head = __shfl_sync(kAll, hu, src);
      const long long b_at = base + __shfl_sync(kAll, end - mine, src);  // the request's first unit
      PtItem it{};
      it.valid = 1;
      it.b = b0 + src;
      it.q0 = __shfl_sync(kAll, s.q0, src);
      it.n = __shfl_sync(kAll, s.n, src);
      it.L = __shfl_sync(kAll, s.L, src);
      it.h = (int)pg_div(x - b_at, head);
      long long at = b_at + it.h * head;  // the head's first unit; pairs follow, long rows first
      // the pair that holds x: prefix sums over 32 pairs at a time
      for (int i0 = 0; i0 < n_p; i0 += 32) {
        const int i = i0 + lane;
        const int u = i < n_p ? pt_units(it.n, it.L, g, n_p - 1 - i) : 0;
        int e = u;  // 32 pairs' units fit
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(kAll, e, o);
          if (lane >= o) e += y;
        }
        const unsigned hit = __ballot_sync(kAll, at + e > x);
        if (hit == 0) {
          at += __shfl_sync(kAll, e, 31);
          continue;
        }
        const int hl = __ffs(hit) - 1;
        const long long u1 = at + __shfl_sync(kAll, e, hl), end = min(u1, x1);
        const long long s0 = u1 - __shfl_sync(kAll, u, hl) + kPtStart;  // its first column tile
        it.r0 = (n_p - 1 - (i0 + hl)) * kPtPair;
        it.t0 = (int)max(0ll, x - s0);
        it.t1 = (int)(end - s0);
        const long long fc = pg_div(s0, per), lc = pg_div(u1 - 1, per);
        it.parts = (int)(lc - fc) + 1;
        // the first item of a block has its slot 0, the last, if it goes on behind the block, slot 1
        it.slot = blockIdx.x * 2 + (fc == blockIdx.x && s0 != fc * per);
        x = end;
        if (end <= s0) break;  // the next block has its column tiles
        if (it.parts > 1 && fc == blockIdx.x && lane == 0)
          a.cuts[blockIdx.x] = PgCut{it.parts, it.slot, it.h, it.q0, it.n, it.r0, {0, 0}};
        break;
      }
      if (it.t1 <= 0) continue;
      // a pair that sees no column has one unit and no tiles
      it.t1 = min(it.t1, pt_tiles(it.n, it.L, g, it.r0 + kPtPair));
      if (!emit(it)) return;
    }
    base += chunk_total;
  }
}

// Columns that every row of the item's pair sees.
__device__ __forceinline__ int pt_seen_by_all(const PtItem& it, const PgArgs& g) {
  return max(0, it.L - it.n + g.by_g(it.r0) + 1);
}

// Columns that its last row sees.
__device__ __forceinline__ int pt_seen_by_some(const PtItem& it, const PgArgs& g) {
  return it.L - it.n + g.by_g(min(it.r0 + kPtPair, it.n * g.G) - 1) + 1;
}

// Column tiles of the item that tile x (0 = A, 1 = B) reads, from t0 on.
__device__ __forceinline__ int pt_mine(const PtItem& it, const PgArgs& g, int x) {
  const int first = it.r0 + x * kPtRows;
  if (first >= it.n * g.G) return 0;
  return max(0, min(it.t1, pt_tiles(it.n, it.L, g, first + kPtRows)) - it.t0);
}

// Registers move from the warpgroups of the other roles to the rows', which
// hold a whole row of scores: the shares sum to what the block launched with.
template <int N>
__device__ __forceinline__ void pt_regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void pt_regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}
static_assert(256 * kPtRegsRows + 256 * kPtRegsRest <= kPtThreads * 128, "registers of the block");

// Columns from nvalid on count as -inf.
__device__ __forceinline__ void pt_mask(uint32_t (&s)[32], int nvalid) {
#pragma unroll
  for (int e = 0; e < 32; ++e)
    if (e >= nvalid) s[e] = 0xff800000u;
}

template <int DH, int BF>
__global__ void __launch_bounds__(kPtThreads, 1)
pg_tile_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, PtArgs a) {
  using C = PtCfg<DH>;
  constexpr uint32_t kIdescS = f16_idesc(128, 64, BF);
  constexpr uint32_t kIdescPV = f16_idesc(128, DH, BF) | kIdescBMnMajor;
  constexpr uint32_t kColS = 256;  // tile x: scores at 256 + 128 x, numerator at x * DH
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* kv_full = bars;                  // [stages] a slot's bytes landed
  uint64_t* kv_empty = bars + C::kStages;    // [stages] both issuers done with the slot
  uint64_t* s_full = bars + 2 * C::kStages;  // [x * 2 + half] scores of a half column tile in TMEM
  uint64_t* p_full = s_full + 4;             // [x * 2 + half] P of a half written (4 warps)
  uint64_t* pv0_done = p_full + 4;           // [x] the item's last first-half P.V completed
  uint64_t* acc_full = pv0_done + 2;         // [x] the item's last P.V completed
  uint64_t* inv_full = acc_full + 2;         // [x] the item's 1 / z written (4 warps)
  uint64_t* n_free = inv_full + 2;           // [x] the numerator has been read (4 warps)
  uint64_t* q_full = n_free + 2;             // [x] queries stored (128 threads)
  uint64_t* q_empty = q_full + 2;            // [x] the item's score MMAs completed
  uint64_t* item_full = q_empty + 2;         // [2]
  uint64_t* item_empty = item_full + 2;      // [2]
  uint64_t* tail = item_empty + 2;           // [1] bytes of a V tile whose last rows are cleared
  uint64_t* fin = tail + 1;                  // [1] every MMA of both issuers completed
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(fin + 1);
  PtItem* items = reinterpret_cast<PtItem*>(tmem_slot + 4);  // [2]
  static_assert((2 * C::kStages + 26) * 8 + 16 + 2 * sizeof(PtItem) <= 512, "barriers");
  uint8_t* ring = smem + C::kRingOff;
  float* inv_of = reinterpret_cast<float*>(smem + C::kInvOff);  // [x][row]
  const PgArgs& g = a.g;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 2);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], kPtRows / 32);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&pv0_done[x], 1);
      mbar_init(&acc_full[x], 1);
      mbar_init(&inv_full[x], kPtRows / 32);
      mbar_init(&n_free[x], kPtRows / 32);
      mbar_init(&q_full[x], kPtRows);
      mbar_init(&q_empty[x], 1);
      mbar_init(&item_full[x], 1);
      mbar_init(&item_empty[x], kPtReaders);
    }
    mbar_init(tail, 1);
    mbar_init(fin, 2);
    fence_mbar_init();
  }
  if (warp == kPtWarpTma) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  pg_wait_for_launch_before();
  pg_launch_next();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // a role whose wait gave up stops arriving, so that the others' waits give up in turn
  auto fail = [&]() { set_error(g.err, kDevErrTimeout); };
  // whole-warp wait
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (!__all_sync(0xffffffffu, mbar_wait_sleep(bar, parity))) {
      fail();
      return false;
    }
    return true;
  };
  // the warp's next item; false at the end
  auto next_item = [&](uint32_t k, PtItem& it) -> bool {
    if (!wait_warp(&item_full[k & 1], (k >> 1) & 1)) return false;
    it = items[k & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(&item_empty[k & 1]);
    return it.valid != 0;
  };

  if (warp == kPtWarpSched) {
    // ------------------------------------------------------------ work items
    pt_regs_dec<kPtRegsRest>();
    uint32_t k = 0;
    bool ok = true;
    auto emit = [&](const PtItem& it) -> bool {
      if (!wait_warp(&item_empty[k & 1], ((k >> 1) & 1) ^ 1)) return ok = false;
      if (lane == 0) {
        items[k & 1] = it;
        mbar_arrive(&item_full[k & 1]);
      }
      ++k;
      __syncwarp();
      return true;
    };
    pt_schedule(a, lane, emit);
    if (ok) emit(PtItem{});
  } else if (warp == kPtWarpTma) {
    // ------------------------------------------------------------ K / V loads
    pt_regs_dec<kPtRegsRest>();
    if (lane < 2) asm volatile("prefetch.tensormap [%0];\n" ::"l"(lane ? &tm_v : &tm_k) : "memory");
    const int box = 1 << a.box_shift, boxes = kPtCols >> a.box_shift;
    uint32_t seq = 0, tails = 0;
    bool ok = true;
    PtItem it;
    for (uint32_t k = 0; ok && next_item(k, it); ++k) {
      const int nt = max(pt_mine(it, g, 0), pt_mine(it, g, 1));
      // lane l's page and first token in it, of box l of column tile t
      auto page_of = [&](int t) -> int {
        if (!g.table) return 0;
        const int col = t * kPtCols + lane * box;
        if (lane >= boxes || col >= it.L) return g.n_pages;  // outside the tensor: zeros
        const int page = g.table[(size_t)it.b * g.max_blocks + (col >> g.shift)];
        if (page < 0 || page >= g.n_pages) {
          set_error(g.err, FLASHLOOP_DEVERR_INDEX);
          return g.n_pages;
        }
        return page;
      };
      int page = nt > 0 ? page_of(it.t0) : 0;
      for (int i = 0; i < nt && ok; ++i) {
        const int t = it.t0 + i;
        const int next = i + 1 < nt ? page_of(t + 1) : 0;
        const int col = t * kPtCols + lane * box;
        const int y = g.table ? (col & ((1 << g.shift) - 1)) : it.q0 + col;
        // the tile's rows that all of the pair's rows see, and those that some do
        const int from = max(0, pt_seen_by_all(it, g) - t * kPtCols);
        const int held = min(pt_seen_by_some(it, g) - t * kPtCols, kPtCols);
        for (int kv = 0; kv < 2; ++kv, ++seq) {
          const int slot = seq % C::kStages;
          const uint32_t ph = (seq / C::kStages) & 1;
          if (!wait_warp(&kv_empty[slot], ph ^ 1)) {
            ok = false;
            break;
          }
          uint8_t* st = ring + slot * C::kSlotBytes;
          const bool clear = kv == 1 && from < kPtCols;
          uint64_t* bar = clear ? tail : &kv_full[slot];
          if (lane == 0) mbar_arrive_expect_tx(bar, C::kSlotBytes);
          __syncwarp();
          if (lane < boxes) {
#pragma unroll
            for (int c = 0; c < DH / 64; ++c)
              tma_load_4d(st + c * C::kChunk + lane * box * 128, kv ? &tm_v : &tm_k, c * 64, y, it.h, page, bar);
          }
          if (clear) {
            if (!wait_warp(tail, tails & 1)) {
              ok = false;
              break;
            }
            ++tails;
            PgFinite<BF> finite;
#pragma unroll 4
            for (int j = from * 8 + lane; j < held * 8; j += 32) {
#pragma unroll
              for (int c = 0; c < DH / 64; ++c) finite.add(*reinterpret_cast<const uint4*>(st + c * C::kChunk + j * 16));
            }
            if (__any_sync(0xffffffffu, !finite.all())) {
              for (int j = from * 8 + lane; j < held * 8; j += 32) {
#pragma unroll
                for (int c = 0; c < DH / 64; ++c) {
                  uint4* at = reinterpret_cast<uint4*>(st + c * C::kChunk + j * 16);
                  const uint4 v = *at;
                  *at = make_uint4(pg_finite_part<BF>(v.x), pg_finite_part<BF>(v.y), pg_finite_part<BF>(v.z), pg_finite_part<BF>(v.w));
                }
              }
              // the item's place is the write-back's until it has read it, which waits for this tile's product
              if (lane == 0) items[k & 1].odd = 1;
            }
            for (int j = held * 8 + lane; j < kPtCols * 8; j += 32) {
#pragma unroll
              for (int c = 0; c < DH / 64; ++c) *reinterpret_cast<uint4*>(st + c * C::kChunk + j * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&kv_full[slot]);
          }
        }
        page = next;
      }
    }
    // never leave with a copy in flight: wait (bounded) for the last load of every slot
    for (uint32_t i = seq > C::kStages ? seq - C::kStages : 0; i < seq; ++i)
      (void)mbar_wait(&kv_full[i % C::kStages], (i / C::kStages) & 1);
    __syncwarp();
  } else if (warp == kPtWarpMma || warp == kPtWarpMma + 1) {
    // ------------------------------------------------------------ MMA issue, one thread per tile
    pt_regs_dec<kPtRegsRest>();
    if (lane == 0) {
      const int x = warp - kPtWarpMma;
      uint32_t seq = 0, u = 0;  // slots so far, column tiles of this tile so far
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        if (!mbar_wait_sleep(bar, parity)) {
          fail();
          ok = false;
          return false;
        }
        tc_fence_after();
        return true;
      };
      auto slot_of = [&](uint32_t s) { return (int)(s % C::kStages); };
      auto par_of = [&](uint32_t s) { return (s / C::kStages) & 1u; };
      const uint32_t q = smem_u32(smem + x * C::kQBytes);
      const uint32_t scol = tmem + kColS + 128u * x;
      auto issue_s = [&](int slot, int hf) {
        const uint32_t kt = smem_u32(ring + slot * C::kSlotBytes) + hf * 64 * 128;
#pragma unroll
        for (int ks = 0; ks < DH / 16; ++ks)
          umma_f16(scol + 64u * hf, sw128_kmajor_desc(q + (ks >> 2) * C::kQChunk + (ks & 3) * 32),
                   sw128_kmajor_desc(kt + (ks >> 2) * C::kChunk + (ks & 3) * 32), kIdescS, ks > 0);
      };
      auto issue_pv = [&](int slot, int hf, bool acc) {
        const uint32_t v = smem_u32(ring + slot * C::kSlotBytes) + hf * 64 * 128;
        const uint32_t d = tmem + (uint32_t)(x * DH), pcol = scol + 64u * hf;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          umma_f16_ts(d, pcol + ks * 8, sw128_mnmajor_desc(v + ks * 2048, C::kChunk), kIdescPV,
                      (acc || ks > 0) ? 1u : 0u);
      };
      // a slot this tile does not read: released once its load has landed
      auto skip = [&](uint32_t s) -> bool {
        if (!wait(&kv_full[slot_of(s)], par_of(s))) return false;
        mbar_arrive(&kv_empty[slot_of(s)]);
        return true;
      };
      for (uint32_t k = 0; ok; ++k) {
        if (!wait(&item_full[k & 1], (k >> 1) & 1)) break;
        const PtItem it = items[k & 1];
        mbar_arrive(&item_empty[k & 1]);
        if (!it.valid) break;
        const int mine[2] = {pt_mine(it, g, 0), pt_mine(it, g, 1)};
        const int my = mine[x], nt = max(mine[0], mine[1]);
        if (!wait(&q_full[x], k & 1)) break;
        const uint32_t base = seq;
        if (my > 0) {
          if (!wait(&kv_full[slot_of(base)], par_of(base))) break;
          for (int hf = 0; hf < 2; ++hf) {
            issue_s(slot_of(base), hf);
            umma_commit(&s_full[2 * x + hf]);
          }
          if (my == 1) umma_commit(&q_empty[x]);
          umma_commit(&kv_empty[slot_of(base)]);
          if (k > 0 && !wait(&n_free[x], (k - 1) & 1)) break;
        } else {
          umma_commit(&q_empty[x]);
          if (nt > 0 && !skip(base)) break;
        }
        // A tile's V and the next tile's K are waited for before its P, and slots are given
        // back behind the next scores: between a P and those lies MMA issue alone.
        for (int t = 0; t < my && ok; ++t, ++u) {
          const uint32_t vs = base + 2 * t + 1, ks = vs + 1;
          const bool more = t + 1 < my;
          if (!wait(&kv_full[slot_of(vs)], par_of(vs))) break;
          if (more && !wait(&kv_full[slot_of(ks)], par_of(ks))) break;
          for (int hf = 0; hf < 2; ++hf) {
            if (!wait(&p_full[2 * x + hf], u & 1)) break;
            issue_pv(slot_of(vs), hf, t > 0 || hf > 0);
            if (more) {
              issue_s(slot_of(ks), hf);
              umma_commit(&s_full[2 * x + hf]);
            } else {
              umma_commit(hf ? &acc_full[x] : &pv0_done[x]);
            }
          }
          if (!ok) break;
          umma_commit(&kv_empty[slot_of(vs)]);
          if (more) {
            umma_commit(&kv_empty[slot_of(ks)]);
            if (t + 2 == my) umma_commit(&q_empty[x]);
          }
        }
        // slots of column tiles that the other tile alone reads
        for (uint32_t s = base + (my > 0 ? 2 * my : 1); ok && s < base + 2 * nt; ++s) skip(s);
        if (!ok) break;
        if (my == 0) {
          if (k > 0 && !wait(&n_free[x], (k - 1) & 1)) break;
          umma_commit(&acc_full[x]);
        }
        seq = base + 2 * nt;
      }
      // every MMA issued has completed before TMEM is released
      umma_commit(fin);
      (void)mbar_wait(fin, 0);
    }
  } else if (warp >= kPtWarpQ) {
    // ------------------------------------------------------------ queries and write-back
    pt_regs_dec<kPtRegsRest>();
    constexpr int kPieces = DH / 8;
    const int quarter = warp - kPtWarpQ, row = quarter * 32 + lane;
    // To the numerators of tile x in TMEM: the values that the loads' warp took out of the item's V tiles.
    // One channel at a time: the write-back is longer where this takes more registers.
    auto add_odd = [&](const PtItem& it, int x, uint32_t nbase) {
      const int r = it.r0 + x * kPtRows + row;
      const int end = r < it.n * g.G ? it.L - it.n + g.by_g(r) + 1 : 0;  // columns that the row sees
      const int stop = min(pt_seen_by_some(it, g), it.t1 * kPtCols);
#pragma unroll 1
      for (int j = max(pt_seen_by_all(it, g), it.t0 * kPtCols); j < stop; ++j) {
        const uint16_t* v = g.v.p + it.h * g.v.sh;
        if (g.table) {
          const int page = g.table[(size_t)it.b * g.max_blocks + (j >> g.shift)];
          if (page < 0 || page >= g.n_pages) continue;
          v += page * g.v.sp + (j & ((1 << g.shift) - 1)) * g.v.st;
        } else {
          v += (long long)(it.q0 + j) * g.v.st;
        }
#pragma unroll 1
        for (int c = lane; c < DH; c += 32) {
          unsigned odd = __ballot_sync(0xffffffffu, pg_not_finite<BF>(v[c]));
          while (odd) {
            const int e = c - lane + __ffs(odd) - 1;
            odd &= odd - 1;
            uint32_t w;
            tmem_ld1(nbase + e, w);
            tmem_wait_ld();
            if (j < end) w = __float_as_uint(__uint_as_float(w) + pg_unpack2<BF>(v[e]).x);
            __syncwarp();
            tmem_st1(nbase + e, w);
            tmem_wait_st();
          }
        }
      }
    };
    // The rows of item k, once both tiles' P.V and 1 / z are there: o = N / z, or N to scratch.
    auto write_back = [&](uint32_t k) -> bool {
      const PtItem& it = items[k & 1];
#pragma unroll 1
      for (int x = 0; x < 2; ++x) {
        const int my = pt_mine(it, g, x);
        const int r = it.r0 + x * kPtRows + row;
        const bool live = r < it.n * g.G;
        const int tok = g.by_g(r);
        uint16_t* od = g.o.p + (live ? (it.q0 + tok) * g.o.st + (long long)(it.h * g.G + r - tok * g.G) * g.o.sh : 0);
        float4* part = a.part_n + (size_t)it.slot * (DH / 4) * kPtPair + x * kPtRows + row;
        const bool whole = it.parts == 1;
        const uint32_t nbase = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(x * DH);
        if (!wait_warp(&acc_full[x], k & 1) || !wait_warp(&inv_full[x], k & 1)) return false;
        tc_fence_after();
        const float inv = inv_of[x * kPtRows + row];
        if (my > 0 && it.odd) add_odd(it, x, nbase);
#pragma unroll 1
        for (int cc = 0; cc < DH; cc += 16) {
          uint32_t w[16];
          if (my > 0) {
            tmem_ld16(nbase + cc, w);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = 0u;
          }
          if (cc + 16 == DH) {  // the numerator is free for the next item's
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&n_free[x]);
          }
          if (whole && live) {
            uint32_t h[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
              h[e] = pg_pack2<BF>(__uint_as_float(w[2 * e]) * inv, __uint_as_float(w[2 * e + 1]) * inv);
            if (g.o32) {
              st_global_v8(od + cc, h);
            } else {
              *reinterpret_cast<uint4*>(od + cc) = make_uint4(h[0], h[1], h[2], h[3]);
              *reinterpret_cast<uint4*>(od + cc + 8) = make_uint4(h[4], h[5], h[6], h[7]);
            }
          } else if (live && my > 0) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              __stcg(part + (cc / 4 + e) * kPtPair, make_float4(__uint_as_float(w[4 * e]), __uint_as_float(w[4 * e + 1]),
                                                               __uint_as_float(w[4 * e + 2]), __uint_as_float(w[4 * e + 3])));
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&item_empty[k & 1]);
      return true;
    };
    for (uint32_t k = 0;; ++k) {
      if (!wait_warp(&item_full[k & 1], (k >> 1) & 1)) break;
      const PtItem& it = items[k & 1];  // kept until its write-back
      if (!it.valid) {
        if (k > 0) (void)write_back(k - 1);
        break;
      }
      const int rows = it.n * g.G;
      // a warp brings 32 rows of a tile, 16 bytes a lane; lane l knows where row l lies
      auto bring = [&](int x) {
        const int mine = it.r0 + x * kPtRows + (warp - kPtWarpQ) * 32 + lane;
        const uint16_t* at = nullptr;
        if (mine < rows) {
          const int tok = g.by_g(mine);
          at = g.q.p + (it.q0 + tok) * g.q.st + (long long)(it.h * g.G + mine - tok * g.G) * g.q.sh;
        }
        const unsigned long long mine_at = reinterpret_cast<unsigned long long>(at);
        const int c = lane % kPieces;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          const int from = i * (32 / kPieces) + lane / kPieces, row = (warp - kPtWarpQ) * 32 + from;
          const unsigned long long src = __shfl_sync(0xffffffffu, mine_at, from);
          cp_async16(smem + x * C::kQBytes + (c >> 3) * C::kQChunk + row * 128 + (((c & 7) ^ (row & 7)) << 4),
                     src ? reinterpret_cast<const uint16_t*>(src) + c * 8 : g.q.p, src ? 16 : 0);
        }
        cp_async_commit();
      };
      auto hand_on = [&](int x) {
        fence_proxy_async_smem();
        mbar_arrive(&q_full[x]);
      };
      if (k > 0 && !wait_warp(&q_empty[0], (k - 1) & 1)) break;
      bring(0);
      // tile B's with them, if its place is free already
      const bool both = k == 0 || __all_sync(0xffffffffu, mbar_try_wait(&q_empty[1], (k - 1) & 1));
      if (both) {
        bring(1);
        cp_async_wait<1>();
        hand_on(0);
      } else {
        cp_async_wait<0>();
        hand_on(0);
        if (!wait_warp(&q_empty[1], (k - 1) & 1)) break;
        bring(1);
      }
      cp_async_wait<0>();
      hand_on(1);
      if (k > 0 && !write_back(k - 1)) break;
    }
  } else {
    // ------------------------------------------------------------ rows
    pt_regs_inc<kPtRegsRows>();
    const int x = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t sbase = tmem + lane_base + kColS + 128u * x;
    const uint32_t nbase = tmem + lane_base + (uint32_t)(x * DH);
    const uint64_t scale2 = f2_pack(g.scale_log2, g.scale_log2);
    uint32_t u = 0, full = 0;  // column tiles of this tile, and items with some, so far
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      if (!wait_warp(bar, parity)) {
        ok = false;
        return false;
      }
      tc_fence_after();
      return true;
    };
    for (uint32_t k = 0; ok; ++k) {
      // the item's slot is kept until the write-back has read it: the column loop needs the registers
      if (!wait(&item_full[k & 1], (k >> 1) & 1)) break;
      const PtItem& it = items[k & 1];
      auto release = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&item_empty[k & 1]);
      };
      if (!it.valid) {
        release();
        break;
      }
      const int my = pt_mine(it, g, x);
      // columns of the item's that the row sees; a row behind the last one computes on zero queries and is not written
      int seen = 0x7fffffff;
      {
        const int r = it.r0 + x * kPtRows + row;
        if (r < it.n * g.G) seen = it.L - it.n + g.by_g(r) + 1 - it.t0 * kPtCols;
      }
      float m_ref = -INFINITY, z = 0.f;
      for (int t = 0; t < my && ok; ++t, ++u) {
#pragma unroll 1
        for (int hf = 0; hf < 2; ++hf) {
          if (!wait(&s_full[2 * x + hf], u & 1)) break;
          const uint32_t at = sbase + 64u * hf;
          const int nvalid = seen - t * kPtCols - hf * 64;
          uint32_t s0[32], s1[32];
          tmem_ld32(at, s0);
          tmem_ld32(at + 32, s1);
          tmem_wait_ld();
          if (__any_sync(0xffffffffu, nvalid < 64)) {
            pt_mask(s0, nvalid);
            pt_mask(s1, nvalid - 32);
          }
          // The exponentials are taken on the reference as it is, beside the maximum that says
          // whether it will do: one score in thousands of tiles says no, and they are taken again.
          // (An item's first ones always are: making them wait for the maximum made every other
          // half 5% slower, since the two no longer run beside each other.)
          uint32_t pk[32];
          uint64_t za[2];
          auto exps = [&]() {
            const float mr = m_ref == -INFINITY ? 0.f : m_ref;
            const uint64_t neg = f2_pack(-mr, -mr);
            za[0] = za[1] = 0ull;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const uint32_t a0 = e < 16 ? s0[(2 * e) & 31] : s1[(2 * e) & 31], a1 = e < 16 ? s0[(2 * e + 1) & 31] : s1[(2 * e + 1) & 31];
              float p0, p1;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(a0), __uint_as_float(a1)), scale2, neg), p0, p1);
              p0 = ex2(p0);
              p1 = ex2(p1);
              za[e & 1] = f2_add(za[e & 1], f2_pack(p0, p1));
              pk[e] = pg_pack2<BF>(p0, p1);
            }
          };
          exps();
          const float mx = fmaxf(max32(s0), max32(s1)) * g.scale_log2;
          const bool need = mx > m_ref + PgRef<BF>::kRise;
          if (__any_sync(0xffffffffu, need)) {
            // raise it: z and the numerator so far scale by 2^(old - new) once the last P.V has
            // completed; the scores that were issued behind it say so
            const float f = need ? ex2(m_ref - (mx - PgRef<BF>::kLift)) : 1.f;
            uint64_t* behind = hf == 0 ? &s_full[2 * x + 1] : t + 1 < my ? &s_full[2 * x] : &pv0_done[x];
            const uint32_t phase = hf == 0 ? u : t + 1 < my ? u + 1 : full;
            if ((t > 0 || hf > 0) && !wait(behind, phase & 1)) break;
            if (t > 0 || hf > 0) {
#pragma unroll 1
              for (int cc = 0; cc < DH; cc += 16) {
                uint32_t w[16];
                tmem_ld16(nbase + cc, w);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * f);
                tmem_st16(nbase + cc, w);
              }
            }
            z *= f;
            if (need) m_ref = mx - PgRef<BF>::kLift;
            exps();
          }
          tmem_st32(at, pk);
          float z0, z1, z2, z3;
          f2_unpack(za[0], z0, z1);
          f2_unpack(za[1], z2, z3);
          z += (z0 + z1) + (z2 + z3);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[2 * x + hf]);
        }
      }
      // the write-back is the query warps': the next item's scores are there already.  They have
      // read the last item's 1 / z when its numerator is free
      if (!ok || (k > 0 && !wait(&n_free[x], (k - 1) & 1))) break;
      full += my > 0;
      const int r = it.r0 + x * kPtRows + row;
      const bool live = r < it.n * g.G;
      if (it.parts > 1) {  // a part: another kernel joins them
        if (live)
          __stcg(a.part_mz + (size_t)it.slot * kPtPair + x * kPtRows + row,
                 make_float2(my > 0 ? m_ref : -INFINITY, my > 0 ? z : 0.f));
      } else {
        inv_of[x * kPtRows + row] = z == 0.f ? 0.f : 1.f / z;
        if (live && g.lse) {
          const int tok = g.by_g(r);
          g.lse[(size_t)(it.h * g.G + r - tok * g.G) * g.max_tokens + it.q0 + tok] =
              z == 0.f ? -INFINITY : (m_ref + log2f(z)) * kPgLn2;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&inv_full[x]);
      release();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kPtWarpTma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

int at_sm_count();

// A 16-bit tensor [d3, d2, d1, DH] (strides in elements) whose boxes are `rows`
// tokens of 64 elements, 128-byte swizzle; what lies outside reads as zero.
static int pt_tmap(CUtensorMap* map, const PgPages& t, int bf16, uint64_t dh, uint64_t tokens, uint64_t heads,
                   uint64_t pages, uint32_t rows) {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    return nullptr;
  }();
  if (fn == nullptr) return FLASHLOOP_ERR_CUDA;
  // a dimension of one has no stride of its own
  const long long sh = heads > 1 ? t.sh : (long long)dh, sp = pages > 1 ? t.sp : (long long)dh;
  const long long st = tokens > 1 ? t.st : (long long)dh;
  cuuint64_t dims[4] = {dh, tokens, heads, pages};
  cuuint64_t strides[3] = {(cuuint64_t)st * 2, (cuuint64_t)sh * 2, (cuuint64_t)sp * 2};
  cuuint32_t box[4] = {64, rows, 1, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                        const_cast<uint16_t*>(t.p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FLASHLOOP_OK : FLASHLOOP_ERR_CUDA;
}

int launch_pg_tile(const PgArgs& g, int dh, int bf16, const PgScratch& ws, cudaStream_t stream) {
  PtArgs a{};
  a.g = g;
  a.box_shift = g.table && g.shift < 7 ? g.shift : 7;
  a.cuts = ws.tile_cuts;
  a.part_mz = ws.tile_mz;
  a.part_n = ws.tile_n;
  const uint64_t tokens = g.table ? 1ull << g.shift : (uint64_t)g.max_tokens;
  const uint64_t pages = g.table ? (uint64_t)g.n_pages : 1;
  const uint32_t rows = 1u << a.box_shift;
  CUtensorMap tk, tv;
  int rc = pt_tmap(&tk, g.k, bf16, dh, tokens, g.Hk, pages, rows);
  if (rc == FLASHLOOP_OK) rc = pt_tmap(&tv, g.v, bf16, dh, tokens, g.Hk, pages, rows);
  if (rc != FLASHLOOP_OK) return rc;
  int grid = kPgSms;  // in a cut, each leaves a record
  if (!a.cuts) {
    grid = at_sm_count();
    const long long items = (long long)g.Hk * (((long long)g.max_tokens * g.G + kPtPair - 1) / kPtPair + g.B);
    if (grid > items) grid = (int)items;
  }
  auto go = [&](auto kernel, int smem) -> int {
    FL_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    return pg_launch_early(kernel, dim3(grid), kPtThreads, smem, stream, tk, tv, a);
  };
  if (dh == 128) {
    if (bf16) return go(pg_tile_kernel<128, 1>, PtCfg<128>::kSmem);
    return go(pg_tile_kernel<128, 0>, PtCfg<128>::kSmem);
  }
  if (bf16) return go(pg_tile_kernel<64, 1>, PtCfg<64>::kSmem);
  return go(pg_tile_kernel<64, 0>, PtCfg<64>::kSmem);
}

}  // namespace fl
