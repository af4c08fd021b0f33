// Block tables, slot maps and cache writes of the many-request operators.
//
// plan: two prefix sums over the requests (new tokens, opened pages), then one
// slot and position a token.  It moves 8 bytes a token and is bound by its
// launch and two or three dependent L2 reads, so one launch does all: every
// block repeats the scan over the requests (a few KB out of L2) and then takes
// its share of the tokens, which needs no exchange between blocks.  64 requests
// of a token each take 3.3 us, 512 with 250 thousand tokens 5.8 us in a graph
// (half as many blocks 7.8, twice as many 7.7).
//
// write: a copy with a gathered destination, bound by HBM.  A thread moves one
// 16-byte piece of a row's K and of its V, so both loads are in flight at once:
// 32768 rows of 16 heads x 128, float32 to bf16, in 124 us, 6.5 TB/s.
#include "paged.cuh"

namespace fl {

constexpr int kPlanThreads = 512;
constexpr int kPlanTokens = 1024;  // tokens a block takes at least

struct PlanArgs {
  int B, T, shift, n_pages, max_blocks, max_free;
  const int32_t* kv;
  const int32_t* add;
  const int32_t* stack;
  const int32_t* n_free;
  int32_t* table;
  int32_t* cu;
  int32_t* kv_out;
  int32_t* slot;
  int32_t* pos;
  int32_t* n_free_out;
  int32_t* err;
};

__device__ __forceinline__ int plan_blocks(int len, int shift) {
  return (int)(((long long)len + (1 << shift) - 1) >> shift);
}

// Exclusive sums over the block of two counts at once, both below 2^31: (tokens, pages), and over all of it.
__device__ __forceinline__ int2 plan_scan(int tokens, int pages, unsigned long long (&s_warp)[kPlanThreads / 32], int2& all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned long long mine = (unsigned long long)pages << 32 | (unsigned)tokens;
  unsigned long long sum = mine, before = 0, total = 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += y;
  }
  if (lane == 31) s_warp[warp] = sum;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w == warp) before = total;
    total += s_warp[w];
  }
  before += sum - mine;
  all = make_int2((int)(unsigned)total, (int)(total >> 32));
  return make_int2((int)(unsigned)before, (int)(before >> 32));
}

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(PlanArgs g) {
  __shared__ int s_start[kPlanThreads], s_open[kPlanThreads], s_kv[kPlanThreads];
  __shared__ unsigned long long s_warp[kPlanThreads / 32];
  __shared__ ulonglong2 s_sums[kPlanThreads / 32];  // tokens and pages of a warp's requests
  __shared__ int s_bad[kPlanThreads / 32];
  const int tid = threadIdx.x;
  pg_wait_for_launch_before();
  pg_launch_next();
  const int n_free = *g.n_free;
  int kv0 = 0, n0 = 0;  // of the first chunk's request
  // totals first: the call appends everything or nothing
  unsigned long long tn = 0, to = 0;
  int bad = 0;
  {
    for (int b = tid; b < g.B; b += kPlanThreads) {
      const int kv = g.kv[b], n = g.add[b];
      if (b == tid) {
        kv0 = kv;
        n0 = n;
      }
      if (kv < 0 || n < 0) {
        bad |= FLASHLOOP_DEVERR_INDEX;
        continue;
      }
      const long long end = ((long long)kv + n + (1 << g.shift) - 1) >> g.shift;
      if (end > g.max_blocks) bad |= 16;  // more blocks than the table has
      tn += n;
      to += end - plan_blocks(kv, g.shift);
    }
    auto sum = [&](int lanes) {
#pragma unroll
      for (int o = lanes / 2; o > 0; o >>= 1) {
        tn += __shfl_xor_sync(0xffffffffu, tn, o);
        to += __shfl_xor_sync(0xffffffffu, to, o);
        bad |= __shfl_xor_sync(0xffffffffu, bad, o);
      }
    };
    const int warp = tid >> 5, lane = tid & 31;
    sum(32);
    if (lane == 0) {
      s_sums[warp] = make_ulonglong2(tn, to);
      s_bad[warp] = bad;
    }
    __syncthreads();
    const int from = lane % (kPlanThreads / 32);
    tn = s_sums[from].x;
    to = s_sums[from].y;
    bad = s_bad[from];
    sum(kPlanThreads / 32);
  }
  int code = 0;
  if ((bad & FLASHLOOP_DEVERR_INDEX) || n_free < 0 || n_free > g.max_free) code = FLASHLOOP_DEVERR_INDEX;
  else if (bad || tn > (unsigned long long)g.T || to > (unsigned long long)n_free)
    code = FLASHLOOP_DEVERR_CAPACITY;
  const int total = code ? 0 : (int)tn;
  if (blockIdx.x == 0 && tid == 0) {
    if (code) set_error(g.err, code);
    g.cu[g.B] = total;
    *g.n_free_out = code ? n_free : n_free - (int)to;
  }
  const int share = (g.T + gridDim.x - 1) / gridDim.x;
  const int t0 = min(g.T, (int)min((long long)blockIdx.x * share, (long long)g.T)), t1 = min(g.T, t0 + share);
  for (int t = max(t0, total) + tid; t < t1; t += kPlanThreads) {
    g.slot[t] = -1;
    g.pos[t] = 0;
  }
  if (code) {
    if (blockIdx.x == 0)
      for (int b = tid; b < g.B; b += kPlanThreads) {
        g.cu[b] = 0;
        g.kv_out[b] = g.kv[b];
      }
    return;
  }
  int base = 0, opened = 0;  // of the requests before this chunk
  for (int b0 = 0; b0 < g.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    const int kv = b0 == 0 ? kv0 : b < g.B ? g.kv[b] : 0, n = b0 == 0 ? n0 : b < g.B ? g.add[b] : 0;
    const int old = plan_blocks(kv, g.shift);
    const int open = plan_blocks(kv + n, g.shift) - old;
    int2 chunk;
    const int2 before = plan_scan(n, open, s_warp, chunk);
    const int start = base + before.x;
    s_start[tid] = start;
    s_open[tid] = opened + before.y - old;  // block i of the request takes stack entry n_free - 1 - (this + i)
    s_kv[tid] = kv;
    if (blockIdx.x == 0 && b < g.B) {
      g.cu[b] = start;
      g.kv_out[b] = kv + n;
    }
    __syncthreads();
    const int end = min(t1, base + chunk.x);
    for (int t = max(t0, base) + tid; t < end; t += kPlanThreads) {
      int lo = 0, hi = min(kPlanThreads, g.B - b0);  // last request of the chunk that starts at or before t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_start[mid] <= t) lo = mid;
        else hi = mid;
      }
      const int pos = s_kv[lo] + (t - s_start[lo]);
      const int blk = pos >> g.shift, in = pos & ((1 << g.shift) - 1);
      int32_t* entry = g.table + (size_t)(b0 + lo) * g.max_blocks + blk;
      int page;
      if (blk >= plan_blocks(s_kv[lo], g.shift)) {  // opened by this call; its first token enters it
        page = g.stack[n_free - 1 - (s_open[lo] + blk)];
        if (in == 0) *entry = page;
      } else {
        page = *entry;
      }
      const bool good = page >= 0 && page < g.n_pages;
      if (!good) set_error(g.err, FLASHLOOP_DEVERR_INDEX);
      g.slot[t] = good ? (page << g.shift) + in : -1;
      g.pos[t] = pos;
    }
    base += chunk.x;
    opened += chunk.y;
    __syncthreads();
    // the other blocks only need the requests of their own tokens
    if (blockIdx.x != 0 && base >= t1) break;
  }
}

int launch_paged_plan(const flashloop_paged_params* p, int shift, const int32_t* kv_lens, const int32_t* new_lens,
                      const int32_t* free_pages, int free_capacity, const int32_t* n_free, int32_t* table, int32_t* cu,
                      int32_t* kv_lens_out, int32_t* slot_map, int32_t* positions, int32_t* n_free_out, int32_t* err,
                      cudaStream_t stream) {
  PlanArgs g{p->batch, p->max_tokens, shift, p->n_pages, p->max_blocks,
             free_capacity < p->n_pages ? free_capacity : p->n_pages, kv_lens, new_lens, free_pages, n_free,
             table, cu, kv_lens_out, slot_map, positions, n_free_out, err};
  int grid = (p->max_tokens + kPlanTokens - 1) / kPlanTokens;
  if (grid > 148) grid = 148;
  if (grid < 1) grid = 1;
  return pg_launch_early(paged_plan_kernel, dim3(grid), kPlanThreads, 0, stream, g);
}

// ---------------------------------------------------------------------------
// cache writes
// ---------------------------------------------------------------------------
struct WriteArgs {
  const void* k;
  const void* v;
  long long kst, ksh, vst, vsh;  // source strides in elements
  uint16_t* kc;
  uint16_t* vc;
  long long kcp, kct, kch, vcp, vct, vch;  // cache strides
  const int32_t* slot;
  int T, Hk, shift, n_pages;
  int32_t* err;
};

// Eight elements as 16-bit words: a copy, or float32 rounded to nearest even.  Read once, through
// coherent loads: the kernel in front may still be writing the rows when this one starts, and a
// load of the read-only path could move before the wait for its end.
template <int SRC32, int BF>
__device__ __forceinline__ uint4 write_load(const void* base, long long off, bool& range) {
  if (!SRC32) return *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + off);
  const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(base) + off);
  const float4 a = s[0], b = s[1];
  if (!BF) {
    const float m = fmaxf(fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(a.z), fabsf(a.w))),
                          fmaxf(fmaxf(fabsf(b.x), fabsf(b.y)), fmaxf(fabsf(b.z), fabsf(b.w))));
    // 65520 is the first value that rounds to infinity; infinities themselves are not reported
    if (m >= 65520.f) {
      const float e[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) range = range || (fabsf(e[i]) >= 65520.f && fabsf(e[i]) <= 3.402823466e38f);
    }
  }
  return make_uint4(pg_pack2<BF>(a.x, a.y), pg_pack2<BF>(a.z, a.w), pg_pack2<BF>(b.x, b.y), pg_pack2<BF>(b.z, b.w));
}

template <int DH, int SRC32, int BF>
__global__ void __launch_bounds__(256) paged_kv_write_kernel(WriteArgs g) {
  constexpr int kPieces = DH / 8;
  const int per_token = g.Hk * kPieces;
  const long long total = (long long)g.T * per_token;
  const long long slots = (long long)g.n_pages << g.shift;
  bool range = false;
  pg_wait_for_launch_before();
  pg_launch_next();
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const int t = (int)(i / per_token), r = (int)(i - (long long)t * per_token);
    const int h = r / kPieces, c = (r % kPieces) * 8;
    const int slot = g.slot[t];
    const uint4 k = write_load<SRC32, BF>(g.k, t * g.kst + h * g.ksh + c, range);
    const uint4 v = write_load<SRC32, BF>(g.v, t * g.vst + h * g.vsh + c, range);
    if (slot < 0 || slot >= slots) {
      range = false;  // a skipped row reports its slot only
      if (slot != -1) set_error(g.err, FLASHLOOP_DEVERR_INDEX);
      continue;
    }
    if (range) {
      set_error(g.err, FLASHLOOP_DEVERR_RANGE);
      range = false;
    }
    const long long page = slot >> g.shift, in = slot & ((1 << g.shift) - 1);
    *reinterpret_cast<uint4*>(g.kc + page * g.kcp + in * g.kct + h * g.kch + c) = k;
    *reinterpret_cast<uint4*>(g.vc + page * g.vcp + in * g.vct + h * g.vch + c) = v;
  }
}

int launch_paged_kv_write(const flashloop_paged_params* p, int shift, const flashloop_rows* k, const flashloop_rows* v,
                          int src32, const int32_t* slot_map, const flashloop_pages* kc, const flashloop_pages* vc,
                          int32_t* err, cudaStream_t stream) {
  WriteArgs g{k->data, v->data, k->stride_token, k->stride_head, v->stride_token, v->stride_head,
              static_cast<uint16_t*>(kc->data), static_cast<uint16_t*>(vc->data), kc->stride_page, kc->stride_token,
              kc->stride_head, vc->stride_page, vc->stride_token, vc->stride_head, slot_map, p->max_tokens,
              p->n_kv_heads, shift, p->n_pages, err};
  const long long total = (long long)p->max_tokens * p->n_kv_heads * (p->head_dim / 8);
  long long blocks = (total + 255) / 256;
  const int grid = (int)(blocks > 148 * 16 ? 148 * 16 : blocks);
  const int bf = p->dtype == FLASHLOOP_DTYPE_BF16;
  auto go = [&](auto kernel) { return pg_launch_early(kernel, dim3(grid), 256, 0, stream, g); };
  if (p->head_dim == 128) {
    if (!src32) return go(paged_kv_write_kernel<128, 0, 1>);
    return bf ? go(paged_kv_write_kernel<128, 1, 1>) : go(paged_kv_write_kernel<128, 1, 0>);
  }
  if (!src32) return go(paged_kv_write_kernel<64, 0, 1>);
  return bf ? go(paged_kv_write_kernel<64, 1, 1>) : go(paged_kv_write_kernel<64, 1, 0>);
}

}  // namespace fl
