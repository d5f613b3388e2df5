// What the host sides of the paged key/value cache operators share (cs_kv.cu, cs_kv4.cu): the
// plan, checks of batches and rows, launches.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>

#include "../../include/cs_kv.h"
#include "cs_kv_rows.cuh"
#include "cs_tune.h"  // cs_fail

// A failure of the CUDA runtime that the call reports itself: the runtime keeps no last error,
// which would fail the next check of whoever calls it after us.
inline cs_status cuda_failed(const char* what, cudaError_t e) {
  cudaGetLastError();
  return cs_fail(CS_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

#define KV_CUDA(call)                                          \
  do {                                                         \
    const cudaError_t e_ = (call);                             \
    if (e_ != cudaSuccess) return cuda_failed(#call, e_);      \
  } while (0)

struct cs_kv_s {
  cs_kv_desc d{};
  int device = 0, num_sms = 0;
  uint32_t* ctrl = nullptr;  // error words, then the counters
  size_t ctrl_words = 0;
  float* part = nullptr;    // pieces of items that several CTAs share
  float4* other = nullptr;  // halves of items inside a CTA
  cskv::Split* splits = nullptr;
  uint8_t* mend = nullptr;  // rows to be computed again
  float* flat_o = nullptr;  // desc.shared: the prefix's output and log-sum-exp
  // copies of a cache (its address is put in by each call): a whole page's slots of a
  // head, and 16 slots
  CUtensorMap page_map, slots_map;
  CUtensorMap codes_map;  // of a cache's codes: a whole page's slots of a head
  bool error_latched = false;
  bool four_ready = false;  // the kernels of caches in 4 bits have their shared memory
};

namespace {

constexpr int kMaxSeqs = 8192;
constexpr int kMaxKeys = 1 << 22;

// The plan's device is current while a call of it runs.
struct DeviceGuard {
  int was = -1;
  bool ok = true;
  explicit DeviceGuard(int device) {
    int cur = -1;
    ok = cudaGetDevice(&cur) == cudaSuccess;
    if (ok && cur != device) {
      ok = cudaSetDevice(device) == cudaSuccess;
      was = cur;
    }
    if (!ok) cudaGetLastError();
  }
  ~DeviceGuard() {
    if (was >= 0) cudaSetDevice(was);
  }
};

// The factor of the scores for exponents in base 2.
inline float scale_log2(const cs_kv_desc& d) {
  const double scale = d.scale > 0.0f ? d.scale : 1.0 / std::sqrt(static_cast<double>(d.head_dim));
  return static_cast<float>(scale * 1.4426950408889634);
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Row stride of a token-indexed tensor `width` wide: the default, or what the caller gave.
inline cs_status row_stride(const char* name, long long given, long long width, long long* stride) {
  *stride = given == 0 ? width : given;
  if (*stride < width || *stride % 8 != 0 || *stride > (1ll << 32))
    return cs_fail(CS_ERR_INVALID_ARG, "%s=%lld (0, or a multiple of 8 from %lld on)", name, given, width);
  return CS_OK;
}

// Whether two sets of `rows` rows (16-bit elements) share one: rows of one pitch may lie
// side by side in a wider buffer.
inline bool rows_overlap(const void* a, long long a_stride, long long a_width, const void* b, long long b_stride, long long b_width,
                  int rows) {
  const char *a0 = static_cast<const char*>(a), *b0 = static_cast<const char*>(b);
  const char *a1 = a0 + 2 * ((rows - 1) * a_stride + a_width), *b1 = b0 + 2 * ((rows - 1) * b_stride + b_width);
  if (rows < 1 || a1 <= b0 || b1 <= a0) return false;
  if (a_stride != b_stride || rows == 1) return true;
  const long long pitch = 2 * a_stride;
  const long long off = ((b0 - a0) % pitch + pitch) % pitch;  // of b's rows inside a's pitch
  return off < 2 * a_width || off + 2 * b_width > pitch;
}

// Whether one of `rows` rows (16-bit elements) shares bytes with a contiguous range.
inline bool rows_over(const void* a, long long stride, long long width, int rows, const void* range, long long bytes) {
  if (!range || bytes <= 0) return false;
  const long long pitch = 2 * stride, from = static_cast<const char*>(range) - static_cast<const char*>(a);
  const long long r = from >= 0 ? from / pitch : -1;  // the last row that begins at or before the range
  if (r >= 0 && r < rows && from < r * pitch + 2 * width) return true;
  return r + 1 < rows && (r + 1) * pitch < from + bytes;
}

inline bool ranges_overlap(const void* a, long long a_bytes, const void* b, long long b_bytes) {
  return rows_over(a, a_bytes / 2, a_bytes / 2, 1, b, b_bytes);
}

inline cs_status check_batch(const cs_kv_s* p, const cs_kv_batch* b) {
  if (!b) return cs_fail(CS_ERR_INVALID_ARG, "batch is NULL");
  if (b->tokens < 0 || b->tokens > p->d.max_tokens)
    return cs_fail(CS_ERR_INVALID_ARG, "tokens=%d (the plan holds %d)", b->tokens, p->d.max_tokens);
  if (b->seqs < 0 || b->seqs > p->d.max_seqs)
    return cs_fail(CS_ERR_INVALID_ARG, "seqs=%d (the plan holds %d)", b->seqs, p->d.max_seqs);
  if (b->max_q < 1) return cs_fail(CS_ERR_INVALID_ARG, "max_q=%d", b->max_q);
  if (b->table_cols < 0 || static_cast<long long>(b->table_cols) * p->d.page_size > kMaxKeys)
    return cs_fail(CS_ERR_INVALID_ARG, "table_cols=%d (at most %d keys)", b->table_cols, kMaxKeys);
  if (b->tokens > 0 && b->seqs > 0 && (!b->cu_q || !b->kv_lens || (!b->page_table && b->table_cols > 0)))
    return cs_fail(CS_ERR_INVALID_ARG, "cu_q, kv_lens and page_table are required");
  return CS_OK;
}

inline cskv::Batch device_batch(const cs_kv_s* p, const cs_kv_batch* b) {
  const cs_kv_desc& d = p->d;
  cskv::Batch B{};
  B.cu_q = b->cu_q;
  B.kv_lens = b->kv_lens;
  B.table = b->page_table;
  B.tokens = b->tokens;
  B.seqs = b->seqs;
  B.max_q = b->max_q;
  B.table_cols = b->table_cols;
  B.heads = d.heads;
  B.kv_heads = d.kv_heads;
  B.group = d.heads / d.kv_heads;
  B.page_size = d.page_size;
  B.page_shift = __builtin_ctz(static_cast<unsigned>(d.page_size));
  B.num_pages = d.num_pages;
  B.page_stride = static_cast<long long>(d.page_size) * d.kv_heads * d.head_dim;
  B.slot_stride = d.cache_layout == CS_KV_TOKEN ? static_cast<long long>(d.kv_heads) * d.head_dim : d.head_dim;
  B.head_stride = d.cache_layout == CS_KV_TOKEN ? d.head_dim : static_cast<long long>(d.page_size) * d.head_dim;
  B.ctrl = p->ctrl;
  return B;
}

// A launch that may be scheduled while the preceding grid drains: every kernel
// here waits for that grid (griddepcontrol.wait) before it touches global memory.
inline cs_status launch(const void* fn, dim3 grid, int threads, int smem, void* params, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[] = {params};
  const cudaError_t e = cudaLaunchKernelExC(&cfg, fn, args);
  if (e != cudaSuccess) return cuda_failed("kernel launch", e);
  return CS_OK;
}

struct Driver {
  PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  PFN_cuTensorMapReplaceAddress_v12000 replace = nullptr;
};

inline const Driver& driver() {
  static Driver d;
  static std::once_flag once;
  std::call_once(once, [] {
    auto entry = [](const char* name) {
      void* f = nullptr;
      cudaDriverEntryPointQueryResult q;
      const bool ok = cudaGetDriverEntryPointByVersion(name, &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
                      q == cudaDriverEntryPointSuccess;
      if (!ok) cudaGetLastError();
      return ok ? f : nullptr;
    };
    d.encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(entry("cuTensorMapEncodeTiled"));
    d.replace = reinterpret_cast<PFN_cuTensorMapReplaceAddress_v12000>(entry("cuTensorMapReplaceAddress"));
  });
  return d;
}

inline cs_status encode(CUtensorMap* map, int bf16, const void* ptr, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                 const cuuint32_t* box, const char* name) {
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  const CUresult r = driver().encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank,
                         const_cast<void*>(ptr), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return cs_fail(CS_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d) for %s", static_cast<int>(r), name);
  return CS_OK;
}

// States of pieces: the tensor-core kernel's are larger than the rows kernel's.
inline size_t part_floats(const cs_kv_desc& d, int num_sms) {
  static_assert(4 * 2 * cskv::ROWS * (64 + 4) <= 4 * 128 * (64 + 8), "workspace");
  return static_cast<size_t>(num_sms) * 4 * 128 * (d.head_dim + 8);
}

// Counters of one phase: one for each CTA of the largest kernel for few rows.
constexpr int kRowsCtas = 4;
static_assert(cskv::ROWS_CTAS <= kRowsCtas, "counters");
inline int arrival_words(const cs_kv_s* p) { return p->num_sms * kRowsCtas; }

// Rows of one key head that n new tokens have.
inline int rows_of(const cskv::AttnP& k, long long n) {
  const long long tokens = n < k.b.tokens ? n : k.b.tokens;
  return static_cast<int>(tokens * k.b.group);
}

inline cs_status begin(cs_kv_s* p, const cs_kv_batch* b) {
  if (!p) return cs_fail(CS_ERR_INVALID_ARG, "plan is NULL");
  if (p->error_latched) return cs_fail(CS_ERR_NEEDS_RESET, "plan holds a device error; call cs_kv_reset");
  return check_batch(p, b);
}

// A contiguous part of a cache.
struct Held {
  const void* at;
  long long bytes;
};

// The arguments of attention but the cache itself, whose parts are `held`.
inline cs_status check_attn_rows(const cs_kv_s* p, const cs_kv_batch* b, const void* q, long long given_q_stride, void* out,
                                 long long given_out_stride, float* lse, const Held* held, int parts, cskv::AttnP& k) {
  const cs_kv_desc& d = p->d;
  const long long width = static_cast<long long>(d.heads) * d.head_dim;
  long long q_stride = 0;
  cs_status s;
  if ((s = row_stride("q_stride", given_q_stride, width, &q_stride)) != CS_OK) return s;
  if ((s = row_stride("out_stride", given_out_stride, width, &k.out_stride)) != CS_OK) return s;
  if (b->tokens == 0) return CS_OK;
  if (!q || !out) return cs_fail(CS_ERR_INVALID_ARG, "q and out are required");
  if (!aligned16(q) || !aligned16(out)) return cs_fail(CS_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
  if (rows_overlap(q, q_stride, width, out, k.out_stride, width, b->tokens))
    return cs_fail(CS_ERR_INVALID_ARG, "out overlaps q");
  const long long lse_bytes = 4ll * b->tokens * d.heads;
  for (int i = 0; i < parts; ++i)
    if (rows_over(out, k.out_stride, width, b->tokens, held[i].at, held[i].bytes))
      return cs_fail(CS_ERR_INVALID_ARG, "out overlaps a cache");
  bool over = rows_over(out, k.out_stride, width, b->tokens, lse, lse_bytes) || rows_over(q, q_stride, width, b->tokens, lse, lse_bytes);
  for (int i = 0; i < parts; ++i) over = over || ranges_overlap(held[i].at, held[i].bytes, lse, lse_bytes);
  if (over) return cs_fail(CS_ERR_INVALID_ARG, "lse overlaps another argument");
  k.b = device_batch(p, b);
  // a window as long as any sequence hides nothing
  k.c.window = d.window >= kMaxKeys ? 0 : d.window;
  k.c.sinks = k.c.window == 0 ? 0 : d.sinks < kMaxKeys ? d.sinks : kMaxKeys;
  k.c.item_cost = 1;
  k.out = out;
  k.lse = lse;
  k.scale_log2 = scale_log2(d);
  k.part = p->part;
  k.other = p->other;
  k.splits = p->splits;
  k.num_splits = p->num_sms;
  k.mend = p->mend;
  k.arrivals = p->ctrl + cskv::CTRL_COUNTERS;
  k.q_raw = q;
  k.q_stride = q_stride;
  k.out_wide = reinterpret_cast<uintptr_t>(out) % 32 == 0 && k.out_stride % 16 == 0;
  return CS_OK;
}

// The arguments of an append but the cache itself; the rows' strides in elements.
inline cs_status check_append_rows(const cs_kv_s* p, const cs_kv_batch* b, const cs_kv_append_args* a, const Held* held, int parts,
                                   long long* qkv_stride, long long* q_stride) {
  const cs_kv_desc& d = p->d;
  cs_status s;
  if (b->tokens > 0 && (!a->qkv || !a->q_out)) return cs_fail(CS_ERR_INVALID_ARG, "qkv and q_out are required");
  if (!aligned16(a->qkv) || !aligned16(a->q_out)) return cs_fail(CS_ERR_INVALID_ARG, "qkv and q_out must be 16-byte aligned");
  const long long q_width = static_cast<long long>(d.heads) * d.head_dim;
  const long long width = q_width + 2ll * d.kv_heads * d.head_dim;
  if ((s = row_stride("qkv_stride", a->qkv_stride, width, qkv_stride)) != CS_OK) return s;
  if ((s = row_stride("q_stride", a->q_stride, q_width, q_stride)) != CS_OK) return s;
  if (!(a->q_out == a->qkv && (*q_stride == *qkv_stride || b->tokens == 1)) &&
      rows_overlap(a->qkv, *qkv_stride, width, a->q_out, *q_stride, q_width, b->tokens))
    return cs_fail(CS_ERR_INVALID_ARG, "q_out overlaps qkv without being its Q part");
  if (d.rotary_dim > 0) {
    if (!a->rope || a->rope_rows < 1) return cs_fail(CS_ERR_INVALID_ARG, "rope is required (rotary_dim=%d)", d.rotary_dim);
    if (!aligned16(a->rope)) return cs_fail(CS_ERR_INVALID_ARG, "rope must be 16-byte aligned");
  }
  for (int i = 0; i < parts; ++i) {
    for (int j = 0; j < i; ++j)
      if (ranges_overlap(held[i].at, held[i].bytes, held[j].at, held[j].bytes))
        return cs_fail(CS_ERR_INVALID_ARG, "k_cache and v_cache, or parts of one of them, overlap");
  }
  for (int i = 0; i < parts; ++i)
    if (rows_over(a->q_out, *q_stride, q_width, b->tokens, held[i].at, held[i].bytes) ||
        rows_over(a->qkv, *qkv_stride, width, b->tokens, held[i].at, held[i].bytes))
      return cs_fail(CS_ERR_INVALID_ARG, "qkv or q_out overlaps a cache");
  return CS_OK;
}

inline cs_status map_caches(cskv::AttnP& k, const CUtensorMap& like) {
  k.k = like;
  k.v = like;
  auto replace = driver().replace;
  if (replace(&k.k, const_cast<void*>(k.k_raw)) != CUDA_SUCCESS || replace(&k.v, const_cast<void*>(k.v_raw)) != CUDA_SUCCESS)
    return cs_fail(CS_ERR_CUDA, "cuTensorMapReplaceAddress failed");
  return CS_OK;
}

// The kernels of a call with at most `max_rows` rows per key head, and the maps of their caches' copies.
struct Kernels {
  const void *rows, *attn, *join;
  // few rows: keys of a tile; CTAs of a key head where items go by heads, or 0; fewest units of a CTA; items of up to
  // `uncut` tiles stay whole if that gives a CTA up to `spare` tiles more
  int rows_shift, head_ctas, least, uncut, spare;
  int rows_grid, rows_smem, attn_smem, attn_threads;
  const CUtensorMap *rows_map, *attn_map;  // nullptr: read through pointers
};

// Few rows: do items stay whole?  With as many tiles as the page table (or the window) lets an item have, and one a
// sequence and head: the longest CTA's tiles against those of equal ranges.  That says nothing of batches of long and short
// items, where a CTA may get nearly an item's tiles more than an equal range, so items that may be long are cut.
inline bool rows_uncut(const cskv::AttnP& k, const Kernels& use, const cs_kv_desc& d) {
  const int tile = 1 << k.c.shift;
  long long keys = static_cast<long long>(k.b.table_cols) * d.page_size;
  if (k.c.window > 0) keys = std::min<long long>(keys, k.c.window + k.c.per_item + tile + (k.c.sinks + tile - 1) / tile * tile);
  const long long tiles = std::max<long long>(1, (keys + tile - 1) / tile), units = tiles + k.c.item_cost;
  const long long seqs = std::min(k.b.seqs, k.b.tokens);
  const long long ctas = use.head_ctas ? use.head_ctas : use.rows_grid, items = use.head_ctas ? seqs : seqs * d.kv_heads;
  return !k.c.flat && tiles <= use.uncut && (items + ctas - 1) / ctas * units * ctas - items * units <= use.spare * ctas;
}

inline cs_status run_attention(cs_kv_s* p, cskv::AttnP& k, const Kernels& use, int max_rows, cudaStream_t st) {
  const cs_kv_desc& d = p->d;
  const bool bf16 = d.dtype == CS_BF16;
  k.head_groups = d.cache_layout == CS_KV_HEAD ? d.page_size / 8 : 0;
  cs_status s;
  if (max_rows <= cskv::ROWS) {
    k.c.per_item = cskv::ROWS / k.b.group;
    k.c.shift = use.rows_shift;
    k.c.head_ctas = use.head_ctas;
    k.c.least = use.least;
    if (rows_uncut(k, use, d)) k.c.whole = 1;
    if (use.rows_map && (s = map_caches(k, *use.rows_map)) != CS_OK) return s;
    s = launch(use.rows, dim3(use.rows_grid), cskv::ROWS_THREADS, use.rows_smem, &k, st);
    if (s != CS_OK || max_rows <= k.b.group || k.c.flat) return s;
    k.num_splits = 0;  // rows of several tokens: some may have to be mended
    s = launch(use.join, dim3(p->num_sms), cskv::JOIN_THREADS, 0, &k, st);
    k.num_splits = p->num_sms;
    return s;
  }
  k.per_tile = 128 / k.b.group;
  k.c.per_item = 2 * k.per_tile;
  k.c.shift = 7;
  k.c.least = 1;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d.head_dim), static_cast<cuuint64_t>(d.heads),
                              static_cast<cuuint64_t>(k.b.tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d.head_dim) * 2, static_cast<cuuint64_t>(k.q_stride) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(k.b.group), static_cast<cuuint32_t>(k.per_tile)};
  s = encode(&k.q, bf16, k.q_raw, 3, dims, strides, box, "q");
  if (s == CS_OK && use.attn_map) s = map_caches(k, *use.attn_map);
  if (s != CS_OK) return s;
  // Cutting items evens out the load, and costs about 9 tiles' time: the pieces' stores and
  // their joining.  Not cutting them leaves up to half an item more on a CTA, and CTAs idle
  // when there are fewer items than CTAs.  So short items stay whole.  Measured, cut and
  // whole, 12 heads of 128: 10 prompts of 512 tokens 36 and 24 us, 3 of 1024 39 and 24 us,
  // 5 of 2500 105 and 99 us, 2 of 4000 (32 tiles) both 109 us, one of 1500 27 and 29 us.
  // The longest item is that of the longest keys that the page table has room for.
  const int tile = 1 << k.c.shift;
  long long keys = k.c.flat ? k.c.flat_len : static_cast<long long>(k.b.table_cols) * d.page_size;
  if (k.c.window > 0) keys = std::min<long long>(keys, k.c.window + k.c.per_item + tile + (k.c.sinks + tile - 1) / tile * tile);
  const long long longest = (keys + tile - 1) / tile;
  const long long items = static_cast<long long>((k.b.tokens + k.c.per_item - 1) / k.c.per_item) * d.kv_heads;
  const long long idle = std::max<long long>(0, p->num_sms - items);
  if (!k.c.flat && longest <= 24 && longest * idle <= 5 * p->num_sms) {
    k.c.whole = 1;
    k.num_splits = 0;
  }
  if ((s = launch(use.attn, dim3(p->num_sms), use.attn_threads, use.attn_smem, &k, st)) != CS_OK) return s;
  return launch(use.join, dim3((k.c.whole ? 1 : cskv::JOIN_CTAS) * p->num_sms), cskv::JOIN_THREADS, 0, &k, st);
}

// All tokens of the batch over a prefix, then every sequence's own keys, which join it; use(rows): the
// kernels for that many rows per key head.
template <typename Use>
cs_status run_shared(cs_kv_s* p, cskv::AttnP& k, const cs_kv_batch* b, const int32_t* prefix_pages, int prefix_len, Use use,
                     cudaStream_t st) {
  if (prefix_len > 0) {
    k.flat_o = p->flat_o;
    k.flat_lse = p->flat_o + static_cast<size_t>(p->d.max_tokens) * p->d.heads * p->d.head_dim;
    k.pages = prefix_pages;
    k.c.flat = 1;
    k.c.flat_len = prefix_len;
    const int rows = rows_of(k, b->seqs * static_cast<long long>(b->max_q));
    const cs_status s = run_attention(p, k, use(rows), rows, st);
    if (s != CS_OK) return s;
    k.c.flat = 0;
    k.part += part_floats(p->d, p->num_sms);  // the rows kernel does not wait for the prefix's phase
    k.arrivals += arrival_words(p);
  }
  const int rows = rows_of(k, b->max_q);
  return run_attention(p, k, use(rows), rows, st);
}

inline cs_status check_prefix(const cs_kv_s* p, const int32_t* prefix_pages, int prefix_len) {
  if (!p->d.shared) return cs_fail(CS_ERR_INVALID_ARG, "the plan was made without desc.shared");
  if (prefix_len < 0 || prefix_len > kMaxKeys) return cs_fail(CS_ERR_INVALID_ARG, "prefix_len=%d (0..%d)", prefix_len, kMaxKeys);
  if (!prefix_pages && prefix_len > 0) return cs_fail(CS_ERR_INVALID_ARG, "prefix_pages is NULL");
  return CS_OK;
}

// Whether an attention chain's plan and a cache's plan make a layer.
inline cs_status check_layer(cs_chain_t chain, const cs_kv_s* p, const cs_kv_batch* b, cs_chain_info& info) {
  const cs_status s = cs_chain_query(chain, &info);
  if (s != CS_OK) return s;
  const cs_chain_desc& cd = *cs_chain_desc_of(chain);
  if (cd.kind != CS_CHAIN_ATTN) return cs_fail(CS_ERR_INVALID_ARG, "chain is not an attention chain");
  if (cs_chain_device_of(chain) != p->device)
    return cs_fail(CS_ERR_INVALID_ARG, "the chain's plan is on device %d, the cache's on device %d", cs_chain_device_of(chain), p->device);
  const cs_kv_desc& d = p->d;
  if (d.dtype != cd.dtype || d.heads != cd.heads || d.kv_heads != cd.heads || d.head_dim != 128)
    return cs_fail(CS_ERR_INVALID_ARG, "the plans differ: dtype %d/%d, heads %d/%d, kv_heads %d, head_dim %d", cd.dtype, d.dtype,
                   cd.heads, d.heads, d.kv_heads, d.head_dim);
  if (b->tokens != cd.M) return cs_fail(CS_ERR_INVALID_ARG, "batch has %d tokens, the chain M=%d", b->tokens, cd.M);
  // a stage that runs alone does not advance the epoch that its split tiles count by
  if (info.split_k[0] != 1 || info.split_k[2] != 1 || info.sk_units != 0)
    return cs_fail(CS_ERR_UNSUPPORTED, "the chain's plan splits K (make it with split_k = 1 and sk_tiles = -1)");
  return CS_OK;
}

}  // namespace
