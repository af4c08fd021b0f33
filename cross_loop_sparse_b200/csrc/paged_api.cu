// C entry points of the many-request operators (see include/flashloop.h):
// argument checks and launches.
#include <math.h>

#include "paged.cuh"

namespace fl {

int check_device_arch();
int launch_paged_plan(const flashloop_paged_params*, int, const int32_t*, const int32_t*, const int32_t*, int,
                      const int32_t*, int32_t*, int32_t*, int32_t*, int32_t*, int32_t*, int32_t*, int32_t*,
                      cudaStream_t);
int launch_paged_kv_write(const flashloop_paged_params*, int, const flashloop_rows*, const flashloop_rows*, int,
                          const int32_t*, const flashloop_pages*, const flashloop_pages*, int32_t*, cudaStream_t);

static int pg_shift(int page_size) {
  for (int s = 4; s <= 8; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

// Bounds that leave the kernels' 32-bit sums a tile's or a grid stride's room.
constexpr long long kPgMaxTokens = 1ll << 30, kPgMaxColumns = 0x7fff0000ll, kPgMaxRows = 0x7fff0000ll;

// Sizes that every call reads.
static int pg_check_sizes(const flashloop_paged_params* p) {
  if (!p) return FLASHLOOP_ERR_INVALID_ARG;
  if (p->batch < 0 || p->max_tokens < 0 || p->max_new < 1) return FLASHLOOP_ERR_INVALID_ARG;
  if (p->batch > 65535 || p->max_tokens > kPgMaxTokens) return FLASHLOOP_ERR_UNSUPPORTED;
  return FLASHLOOP_OK;
}

static int pg_check_pages(const flashloop_paged_params* p) {
  if (pg_shift(p->page_size) < 0) return FLASHLOOP_ERR_UNSUPPORTED;
  if (p->n_pages < 1 || p->max_blocks < 1) return FLASHLOOP_ERR_INVALID_ARG;
  if ((long long)p->n_pages * p->page_size > 0x7fffffffll || (long long)p->max_blocks * p->page_size > kPgMaxColumns)
    return FLASHLOOP_ERR_UNSUPPORTED;
  return FLASHLOOP_OK;
}

static int pg_check_heads(const flashloop_paged_params* p, bool queries) {
  if (p->n_kv_heads < 1) return FLASHLOOP_ERR_INVALID_ARG;
  if (p->head_dim != 64 && p->head_dim != 128) return FLASHLOOP_ERR_UNSUPPORTED;
  if (p->dtype != FLASHLOOP_DTYPE_BF16 && p->dtype != FLASHLOOP_DTYPE_FP16) return FLASHLOOP_ERR_UNSUPPORTED;
  if (p->n_kv_heads > 65535) return FLASHLOOP_ERR_UNSUPPORTED;
  if (!queries) return FLASHLOOP_OK;
  if (p->n_heads < 1 || p->n_heads % p->n_kv_heads != 0) return FLASHLOOP_ERR_INVALID_ARG;
  if ((long long)p->max_tokens * p->n_heads > kPgMaxRows) return FLASHLOOP_ERR_UNSUPPORTED;  // packed rows
  if (!isfinite(p->scale * kPgLog2e) || !(p->scale > 0.f)) return FLASHLOOP_ERR_INVALID_ARG;
  return FLASHLOOP_OK;
}

// Address and strides multiples of 16 bytes; strides not negative.
static bool pg_aligned(const void* ptr, long long a, long long b, long long c, int elem) {
  if (!ptr || (reinterpret_cast<uintptr_t>(ptr) & 15) != 0) return false;
  const long long s[3] = {a, b, c};
  for (long long x : s)
    if (x < 0 || x >= (1ll << 36) || (x * elem) % 16 != 0) return false;
  return true;
}
static bool pg_ok(const flashloop_rows* r, int elem) {
  return r && pg_aligned(r->data, r->stride_token, r->stride_head, 0, elem);
}
static bool pg_ok(const flashloop_pages* c) {
  return c && pg_aligned(c->data, c->stride_page, c->stride_token, c->stride_head, 2);
}

static PgRows pg_rows(const flashloop_rows* r) {
  return {static_cast<uint16_t*>(r->data), r->stride_token, r->stride_head};
}
static PgPages pg_pages(const flashloop_pages* c) {
  return {static_cast<const uint16_t*>(c->data), c->stride_page, c->stride_token, c->stride_head};
}

// TMA takes no stride of zero (rows that a caller broadcast); the few-row
// kernel's own loads do, whatever the number of rows.
static bool pg_tma_ok(const PgArgs& g, int pages) {
  for (const PgPages* t : {&g.k, &g.v})
    if (t->st == 0 || (g.Hk > 1 && t->sh == 0) || (pages > 1 && t->sp == 0)) return false;
  return true;
}

// The tile kernel's roles wait for one another for up to an item's time, and its
// waits give up after about a second: items of this many columns take 250 ms.
// The few-row kernel waits for nothing.
constexpr long long kPgTileColumns = 1ll << 24;

// Which kernel takes a call whose requests see at most `cols` columns, by the
// call's bounds alone: estimates of both times in microseconds, fitted to both
// kernels' times over 35 shapes.  A block of the few-row kernel takes a stage of
// 64 columns for 32 packed rows (two blocks an SM), one of the tile kernel 128
// columns for 256 rows; to start and, where the column line is cut, to join has a
// price for each.  Some of those times (few-row / tile kernel):
//   prompts   24 rows, 2 heads a key head, of 16 tokens: 7.2 / 8.5
//             1 x 512 tokens, 4 heads: 13.8 / 15.0     1 x 1024, 8 heads: 27.0 / 22.7
//             4 x 512, 16 heads: 48.7 / 17.4           64 x 64, 16 heads: 56 / 18.7
//   chunks    12 rows x 8 heads a key head over 2219: 18.1 / 20.7
//             128 rows x 4 over 4096, 8 key heads: 49.4 / 31.9
//             63 single rows and one of 64 over 8000 each, 32 heads: 389 / 447
static bool pg_tiles(const flashloop_paged_params* p, long long cols, bool paged) {
  const long long most = p->max_new < p->max_tokens ? p->max_new : p->max_tokens;
  if (most * (p->n_heads / p->n_kv_heads) <= kPgFewRows || cols > kPgTileColumns) return false;
  auto over = [](double a, double b) { return a > b ? a : b; };
  const double rows = (double)p->max_tokens * p->n_heads;
  const double requests = p->batch < p->max_tokens ? p->batch : p->max_tokens;
  const double starts = requests * p->n_kv_heads / 2;  // row tiles that a request does not fill
  const double few = rows / kPgFewRows + starts, tiles = rows / kPgTileRows + starts;
  const double stages = (double)((cols + 63) / 64), units = (double)((cols + 127) / 128);
  const double stage = p->head_dim == 128 ? 1.4 : 0.6, unit = p->head_dim == 128 ? 1.9 : 1.6;
  const double blocks = 2 * kPgSms, sms = kPgSms;
  if (!paged) {  // whole items; a prompt's row tiles see half of its columns on average
    const double few_us = over(3.0 + stage * stages, few / blocks * (7.5 + stage / 2 * stages));
    return over(7.0 + unit * units, tiles / sms * (7.0 + unit / 2 * units)) < few_us;
  }
  const double hbm = requests * (double)cols * p->n_kv_heads * p->head_dim * 4 / 6.5e6;
  const double few_us = cols <= kPgShort ? over(3.0 + stage * stages, few / blocks * (7.5 + stage * stages))
                                         : 9.0 + over(1.2 * stage * over(4.0, few * (stages + 6) / blocks), 1.15 * hbm);
  return 18.0 + over(1.05 * unit * over(4.0, tiles * (units + 2) / sms), 1.35 * hbm) < few_us;
}
static bool pg_tiles(const flashloop_paged_params* p) {
  return pg_tiles(p, (long long)p->max_blocks * p->page_size, true);
}

// Offsets depend on the shape alone.
static PgScratch pg_scratch(const flashloop_paged_params* p, void* base) {
  PgScratch w{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align256(off + bytes);
    return at;
  };
  const size_t slots = 2 * kPgSms, row_slots = 4 * kPgSms, dh = (size_t)p->head_dim;
  if (pg_tiles(p)) {
    w.tile_cuts = ws_ptr<PgCut>(base, take(kPgSms * sizeof(PgCut)));
    w.tile_mz = ws_ptr<float2>(base, take(slots * kPgTileRows * sizeof(float2)));
    w.tile_n = ws_ptr<float4>(base, take(slots * kPgTileRows * dh * sizeof(float)));
  } else if ((long long)p->max_blocks * p->page_size > kPgShort) {
    w.row_cuts = ws_ptr<PgCut>(base, take(2 * kPgSms * sizeof(PgCut)));
    w.row_mz = ws_ptr<float2>(base, take(row_slots * kPgFewRows * sizeof(float2)));
    w.row_n = ws_ptr<float4>(base, take(row_slots * kPgFewRows * dh * sizeof(float)));
  }
  w.total = off;
  return w;
}

static PgArgs pg_args(const flashloop_paged_params* p, const flashloop_rows* q, const int32_t* cu,
                      const flashloop_rows* o, float* lse, int32_t* err) {
  PgArgs g{};
  g.B = p->batch;
  g.Hq = p->n_heads;
  g.Hk = p->n_kv_heads;
  g.G = p->n_heads / p->n_kv_heads;
  g.by_g = pg_divide_by(g.G);
  g.max_tokens = p->max_tokens;
  g.max_new = p->max_new < p->max_tokens ? p->max_new : p->max_tokens;
  g.cu = cu;
  g.q = pg_rows(q);
  g.o = pg_rows(o);
  g.lse = lse;
  g.err = err;
  g.scale_log2 = p->scale * kPgLog2e;
  g.o32 = (reinterpret_cast<uintptr_t>(o->data) & 31) == 0 && o->stride_token % 16 == 0 && o->stride_head % 16 == 0;
  return g;
}

}  // namespace fl

using namespace fl;

extern "C" {

int flashloop_paged_plan(const flashloop_paged_params* p, const int32_t* kv_lens, const int32_t* new_lens,
                         const int32_t* free_pages, int32_t free_capacity, const int32_t* n_free,
                         int32_t* block_table, int32_t* cu, int32_t* kv_lens_out, int32_t* slot_map,
                         int32_t* positions, int32_t* n_free_out, int32_t* err_word, void* stream) {
  int rc = pg_check_sizes(p);
  if (rc == FLASHLOOP_OK) rc = pg_check_pages(p);
  if (rc != FLASHLOOP_OK) return rc;
  if (!n_free || !cu || !n_free_out || free_capacity < 0 || (free_capacity > 0 && !free_pages))
    return FLASHLOOP_ERR_INVALID_ARG;
  if (p->batch > 0 && (!kv_lens || !new_lens || !block_table || !kv_lens_out)) return FLASHLOOP_ERR_INVALID_ARG;
  if (p->max_tokens > 0 && (!slot_map || !positions)) return FLASHLOOP_ERR_INVALID_ARG;
  // every block reads the lengths while block 0 writes the new ones
  if (n_free == n_free_out) return FLASHLOOP_ERR_INVALID_ARG;
  if (p->batch > 0 && kv_lens_out < kv_lens + p->batch && kv_lens < kv_lens_out + p->batch)
    return FLASHLOOP_ERR_INVALID_ARG;
  if (p->batch > 0 && kv_lens_out < new_lens + p->batch && new_lens < kv_lens_out + p->batch)
    return FLASHLOOP_ERR_INVALID_ARG;
  rc = check_device_arch();
  if (rc != FLASHLOOP_OK) return rc;
  return launch_paged_plan(p, pg_shift(p->page_size), kv_lens, new_lens, free_pages, free_capacity, n_free, block_table,
                           cu, kv_lens_out, slot_map, positions, n_free_out, err_word,
                           reinterpret_cast<cudaStream_t>(stream));
}

int flashloop_paged_kv_write(const flashloop_paged_params* p, const flashloop_rows* k, const flashloop_rows* v,
                             int32_t src_dtype, const int32_t* slot_map, const flashloop_pages* k_cache,
                             const flashloop_pages* v_cache, int32_t* err_word, void* stream) {
  int rc = pg_check_sizes(p);
  if (rc == FLASHLOOP_OK) rc = pg_check_pages(p);
  if (rc == FLASHLOOP_OK) rc = pg_check_heads(p, false);
  if (rc != FLASHLOOP_OK) return rc;
  if (src_dtype != FLASHLOOP_DTYPE_FP32 && src_dtype != p->dtype) return FLASHLOOP_ERR_UNSUPPORTED;
  if (!pg_ok(k_cache) || !pg_ok(v_cache)) return FLASHLOOP_ERR_INVALID_ARG;
  if (p->max_tokens == 0) return FLASHLOOP_OK;
  const int elem = src_dtype == FLASHLOOP_DTYPE_FP32 ? 4 : 2;
  if (!pg_ok(k, elem) || !pg_ok(v, elem) || !slot_map) return FLASHLOOP_ERR_INVALID_ARG;
  rc = check_device_arch();
  if (rc != FLASHLOOP_OK) return rc;
  return launch_paged_kv_write(p, pg_shift(p->page_size), k, v, elem == 4, slot_map, k_cache, v_cache, err_word,
                               reinterpret_cast<cudaStream_t>(stream));
}

int flashloop_prompt_attn(const flashloop_paged_params* p, const flashloop_rows* q, const flashloop_rows* k,
                          const flashloop_rows* v, const int32_t* cu, const flashloop_rows* o, float* lse,
                          int32_t* err_word, void* stream) {
  int rc = pg_check_sizes(p);
  if (rc == FLASHLOOP_OK) rc = pg_check_heads(p, true);
  if (rc != FLASHLOOP_OK) return rc;
  if (p->batch == 0 || p->max_tokens == 0) return FLASHLOOP_OK;
  if (!pg_ok(q, 2) || !pg_ok(k, 2) || !pg_ok(v, 2) || !pg_ok(o, 2) || !cu) return FLASHLOOP_ERR_INVALID_ARG;
  rc = check_device_arch();
  if (rc != FLASHLOOP_OK) return rc;
  PgArgs g = pg_args(p, q, cu, o, lse, err_word);
  g.k = {static_cast<const uint16_t*>(k->data), 0, k->stride_token, k->stride_head};
  g.v = {static_cast<const uint16_t*>(v->data), 0, v->stride_token, v->stride_head};
  const int bf16 = p->dtype == FLASHLOOP_DTYPE_BF16;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!pg_tiles(p, g.max_new, false) || !pg_tma_ok(g, 1)) return launch_pg_rows(g, p->head_dim, bf16, PgScratch{}, s);
  return launch_pg_tile(g, p->head_dim, bf16, PgScratch{}, s);
}

size_t flashloop_paged_attn_workspace_bytes(const flashloop_paged_params* p) {
  if (pg_check_sizes(p) != FLASHLOOP_OK || pg_check_pages(p) != FLASHLOOP_OK ||
      pg_check_heads(p, true) != FLASHLOOP_OK)
    return 0;
  const size_t n = pg_scratch(p, nullptr).total;
  return n > 0 ? n : 16;
}

int flashloop_paged_attn(const flashloop_paged_params* p, const flashloop_rows* q, const flashloop_pages* k_cache,
                         const flashloop_pages* v_cache, const int32_t* block_table, const int32_t* kv_lens,
                         const int32_t* cu, const flashloop_rows* o, float* lse, void* workspace,
                         size_t workspace_bytes, int32_t* err_word, void* stream) {
  int rc = pg_check_sizes(p);
  if (rc == FLASHLOOP_OK) rc = pg_check_pages(p);
  if (rc == FLASHLOOP_OK) rc = pg_check_heads(p, true);
  if (rc != FLASHLOOP_OK) return rc;
  if (!pg_ok(k_cache) || !pg_ok(v_cache)) return FLASHLOOP_ERR_INVALID_ARG;
  if (p->batch == 0 || p->max_tokens == 0) return FLASHLOOP_OK;
  if (!pg_ok(q, 2) || !pg_ok(o, 2) || !block_table || !kv_lens || !cu) return FLASHLOOP_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15) != 0 ||
      workspace_bytes < flashloop_paged_attn_workspace_bytes(p))
    return FLASHLOOP_ERR_INVALID_ARG;
  rc = check_device_arch();
  if (rc != FLASHLOOP_OK) return rc;
  PgArgs g = pg_args(p, q, cu, o, lse, err_word);
  g.shift = pg_shift(p->page_size);
  g.n_pages = p->n_pages;
  g.max_blocks = p->max_blocks;
  g.table = block_table;
  g.kv_lens = kv_lens;
  g.k = pg_pages(k_cache);
  g.v = pg_pages(v_cache);
  const int bf16 = p->dtype == FLASHLOOP_DTYPE_BF16;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const PgScratch ws = pg_scratch(p, workspace);
  if (pg_tiles(p) && !pg_tma_ok(g, p->n_pages)) return launch_pg_rows(g, p->head_dim, bf16, PgScratch{}, s);
  rc = pg_tiles(p) ? launch_pg_tile(g, p->head_dim, bf16, ws, s) : launch_pg_rows(g, p->head_dim, bf16, ws, s);
  return rc != FLASHLOOP_OK ? rc : launch_pg_join(g, p->head_dim, bf16, ws, s);
}

}  // extern "C"
