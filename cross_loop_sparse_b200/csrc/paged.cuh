// Shared declarations of the many-request operators (packed prompts, paged
// cache): the kernels' arguments and what a request's lengths mean.
#pragma once

#include "common.cuh"
#include "mma_util.cuh"

namespace fl {

constexpr float kPgLog2e = 1.4426950408889634f;
constexpr float kPgLn2 = 0.6931471805599453f;

struct PgRows {  // 16-bit rows [token, head, head_dim]
  uint16_t* p;
  long long st, sh;
};
struct PgPages {  // 16-bit pages [page, token, head, head_dim]; packed rows are one page without a table
  const uint16_t* p;
  long long sp, st, sh;
};

// Division by the group, whose size is no constant: for 0 <= x < 2^31 and d > 1,
// x / d = (x * mul) >> (32 + shift) with mul = ceil(2^(32 + shift) / d) and
// 2^(shift + 1) >= d, since the error of mul adds less than x / 2^31 <= 1 / d steps.
struct PgDiv {
  uint32_t mul;  // 0: d is 1
  int shift;
  __device__ __forceinline__ int operator()(int x) const { return mul ? (int)(__umulhi((uint32_t)x, mul) >> shift) : x; }
};
inline PgDiv pg_divide_by(int d) {
  if (d <= 1) return {0, 0};
  int log = 0;
  while ((1ll << log) < d) ++log;
  return {(uint32_t)(((1ull << (31 + log)) + d - 1) / d), log - 1};
}

struct PgArgs {
  int B, Hq, Hk, G, max_tokens, max_new;
  PgDiv by_g;                      // x / G
  int shift, n_pages, max_blocks;  // page_size = 1 << shift
  const int32_t* table;            // NULL: keys and values are packed rows
  const int32_t* kv_lens;          // NULL: a request's cached length is its number of rows
  const int32_t* cu;
  PgRows q, o;
  PgPages k, v;
  float* lse;
  int32_t* err;
  float scale_log2;  // scale * log2(e) > 0: scores in log2 units
  int o32;           // rows of o begin on 32 bytes: whole sectors are written
};

// Request b: rows [q0, q0 + n) and L columns; n = 0 for one that the call
// skips (bad lengths are reported).  Row i sees the columns j <= L - n + i.
struct PgSeq {
  int q0, n, L;
};
__device__ __forceinline__ PgSeq pg_seq(const PgArgs& g, int b) {
  PgSeq s;
  const int c0 = g.cu[b], c1 = g.cu[b + 1];
  s.q0 = c0;
  s.n = c1 - c0;
  s.L = g.kv_lens ? g.kv_lens[b] : s.n;
  bool bad = c0 < 0 || c1 < c0 || c1 > g.max_tokens || s.n > g.max_new || s.L < 0;
  if (g.table) bad = bad || (long long)s.L > ((long long)g.max_blocks << g.shift);
  if (bad) {
    set_error(g.err, FLASHLOOP_DEVERR_INDEX);
    s.q0 = s.n = s.L = 0;
  }
  return s;
}

// a / b, in 32 bits where both fit (a 64-bit division is a hundred instructions).
__device__ __forceinline__ long long pg_div(long long a, long long b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

// bf16 / fp16 as a template parameter: BF = 1 bf16, 0 fp16.
template <int BF>
__device__ __forceinline__ uint32_t pg_pack2(float lo, float hi) {
  if (BF) {
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
  }
  return pack_half2(lo, hi);
}
template <int BF>
__device__ __forceinline__ float2 pg_unpack2(uint32_t x) {
  if (BF) return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&x));
  return __half22float2(*reinterpret_cast<__half2*>(&x));
}
template <int BF>
__device__ __forceinline__ void pg_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (BF) mma_bf16(d, a, b0, b1);
  else mma_f16(d, a, b0, b1);
}

// The running reference of the exponentials p = 2^(s - m) is raised when a score exceeds it by kRise,
// to kLift below that score.  A probability is then at most 2^kRise, and the row's largest at least
// 2^kLift.  In fp16, whose numbers end at 2^16 and lose bits below 2^-14, the lift keeps all bits of
// probabilities down to 2^-21 of the largest, where they would go at 2^-14 without: a row whose
// first key draws nearly all of its weight to a value of zero is the sum of those.  bf16 has the range.
template <int BF>
struct PgRef {
  static constexpr float kLift = BF ? 0.f : 7.f, kRise = 8.f + kLift;
};

// Values that are not finite.  A row's probability of a column that it does not see is zero, and zero
// times infinity or NaN would reach the row through the product.  So the values that are not finite
// of columns that some row of a tile does not see are zeros in the product, and are added to the
// numerators of the rows that see them.
//
// Looks over pairs of values: x * 0 is zero, or NaN for what is not finite.  Four sums, so that a
// 16-byte piece's products do not wait for one another.
template <int BF>
struct PgFinite {
  uint32_t sum[4] = {0u, 0u, 0u, 0u};
  static __device__ __forceinline__ uint32_t fma0(uint32_t x, uint32_t acc) {
    if (BF) {
      const __nv_bfloat162 r = __hfma2(*reinterpret_cast<__nv_bfloat162*>(&x), __float2bfloat162_rn(0.f), *reinterpret_cast<__nv_bfloat162*>(&acc));
      return *reinterpret_cast<const uint32_t*>(&r);
    }
    const __half2 r = __hfma2(*reinterpret_cast<__half2*>(&x), __float2half2_rn(0.f), *reinterpret_cast<__half2*>(&acc));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  __device__ __forceinline__ void add(const uint4& x) {
    sum[0] = fma0(x.x, sum[0]);
    sum[1] = fma0(x.y, sum[1]);
    sum[2] = fma0(x.z, sum[2]);
    sum[3] = fma0(x.w, sum[3]);
  }
  __device__ __forceinline__ bool all() const { return ((sum[0] | sum[1] | sum[2] | sum[3]) & 0x7fff7fffu) == 0; }
};
template <int BF>
__device__ __forceinline__ bool pg_not_finite(uint32_t bits) {  // of one value
  constexpr uint32_t kExp = BF ? 0x7f80u : 0x7c00u;
  return (bits & kExp) == kExp;
}
// The pair with zeros for what is not finite.
template <int BF>
__device__ __forceinline__ uint32_t pg_finite_part(uint32_t x) {
  return (pg_not_finite<BF>(x) ? 0u : x & 0xffffu) | (pg_not_finite<BF>(x >> 16) ? 0u : x & 0xffff0000u);
}

// The scratch of the paged attention.  A block that takes a cut of the column
// line holds at most two items that are not whole, the first and the last, and
// at most one whose part 0 it has; of that one it leaves a record.
constexpr int kPgSms = 148;        // blocks of the tile kernel at most; the few-row kernel runs two an SM
constexpr int kPgTileRows = 256;   // rows of a slot of the tile kernel
struct PgCut {
  int parts, slot0;    // parts < 2: no item to join
  int h, q0, n, r0;    // key head, the request's first row and rows, first packed row
  int pad[2];
};
struct PgScratch {
  PgCut* tile_cuts;  // [kPgSms]
  float2* tile_mz;   // [2 * kPgSms, 256] (m, z)
  float4* tile_n;    // [2 * kPgSms, head_dim / 4, 256]
  PgCut* row_cuts;   // [2 * kPgSms]; NULL: the few-row kernel takes whole requests
  float2* row_mz;    // [4 * kPgSms, 32]
  float4* row_n;     // [4 * kPgSms, 32, head_dim / 4]
  size_t total;
};

// Every kernel of these operators is launched when the one before it in the
// stream ends or has all of its blocks under way and says so, and waits for that
// one's end before it reads or writes global memory: its launch, its barriers'
// set-up and its tensor memory are ready by then.  All threads wait, so that the
// end of a kernel is also the end of all before it.  A step of 4 layers of cache
// write and attention over 1000 tokens takes 54 us instead of 71, a short prompt
// 8 instead of 10.3, outside a graph.
__device__ __forceinline__ void pg_launch_next() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }
__device__ __forceinline__ void pg_wait_for_launch_before() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
template <typename Kernel, typename... Args>
inline int pg_launch_early(Kernel kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? FLASHLOOP_OK : FLASHLOOP_ERR_CUDA;
}

// Rows of a slot of the few-row kernel, its largest row tile.
constexpr int kPgFewRows = 32;

// Tables of at most this many columns are not cut: whole requests are a few
// microseconds' work, and a cut costs a second kernel.
constexpr int kPgShort = 512;

int launch_pg_rows(const PgArgs& g, int dh, int bf16, const PgScratch& ws, cudaStream_t stream);
int launch_pg_tile(const PgArgs& g, int dh, int bf16, const PgScratch& ws, cudaStream_t stream);
int launch_pg_join(const PgArgs& g, int dh, int bf16, const PgScratch& ws, cudaStream_t stream);

}  // namespace fl
