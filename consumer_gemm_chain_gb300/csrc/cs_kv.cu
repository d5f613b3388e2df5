// Host side of the paged key/value cache operators (include/cs_kv.h): plans,
// argument checks, launches and status.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>
#include <new>

#include "../../include/cs_kv.h"
#include "cs_kv_rows.cuh"
#include "cs_tune.h"  // cs_fail

// A failure of the CUDA runtime that the call reports itself: the runtime keeps no last error,
// which would fail the next check of whoever calls it after us.
static cs_status cuda_failed(const char* what, cudaError_t e) {
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
  bool error_latched = false;
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
float scale_log2(const cs_kv_desc& d) {
  const double scale = d.scale > 0.0f ? d.scale : 1.0 / std::sqrt(static_cast<double>(d.head_dim));
  return static_cast<float>(scale * 1.4426950408889634);
}

cs_status validate(const cs_kv_desc* d) {
  if (!d) return cs_fail(CS_ERR_INVALID_ARG, "desc is NULL");
  if (d->dtype != CS_F16 && d->dtype != CS_BF16) return cs_fail(CS_ERR_INVALID_ARG, "bad dtype %d", d->dtype);
  if (d->heads < 1 || d->heads > 1024) return cs_fail(CS_ERR_INVALID_ARG, "heads=%d (1..1024)", d->heads);
  if (d->kv_heads < 1 || d->heads % d->kv_heads != 0)
    return cs_fail(CS_ERR_INVALID_ARG, "kv_heads=%d does not divide heads=%d", d->kv_heads, d->heads);
  if (d->heads / d->kv_heads > 128)
    return cs_fail(CS_ERR_UNSUPPORTED, "%d query heads per key head (at most 128)", d->heads / d->kv_heads);
  if (d->head_dim != 64 && d->head_dim != 128) return cs_fail(CS_ERR_UNSUPPORTED, "head_dim=%d (64 or 128)", d->head_dim);
  if (d->page_size != 16 && d->page_size != 32 && d->page_size != 64 && d->page_size != 128)
    return cs_fail(CS_ERR_UNSUPPORTED, "page_size=%d (16, 32, 64 or 128)", d->page_size);
  if (d->num_pages < 1 || d->num_pages > (1 << 27)) return cs_fail(CS_ERR_INVALID_ARG, "num_pages=%d (1..2^27)", d->num_pages);
  if (d->cache_layout != CS_KV_TOKEN && d->cache_layout != CS_KV_HEAD)
    return cs_fail(CS_ERR_INVALID_ARG, "bad cache_layout %d", d->cache_layout);
  if (d->max_tokens < 1 || d->max_tokens > (1 << 20))
    return cs_fail(CS_ERR_INVALID_ARG, "max_tokens=%d (1..2^20)", d->max_tokens);
  if (d->max_seqs < 1 || d->max_seqs > kMaxSeqs) return cs_fail(CS_ERR_INVALID_ARG, "max_seqs=%d (1..%d)", d->max_seqs, kMaxSeqs);
  if (d->rotary_dim < 0 || d->rotary_dim > d->head_dim || d->rotary_dim % 16 != 0)
    return cs_fail(CS_ERR_INVALID_ARG, "rotary_dim=%d (a multiple of 16 up to head_dim)", d->rotary_dim);
  if (d->rotary_pairing != CS_KV_HALF && d->rotary_pairing != CS_KV_ADJACENT)
    return cs_fail(CS_ERR_INVALID_ARG, "bad rotary_pairing %d", d->rotary_pairing);
  if (d->window < 0) return cs_fail(CS_ERR_INVALID_ARG, "window=%d", d->window);
  if (d->sinks < 0) return cs_fail(CS_ERR_INVALID_ARG, "sinks=%d", d->sinks);
  if (!(d->scale >= 0.0f) || std::isinf(scale_log2(*d)))
    return cs_fail(CS_ERR_INVALID_ARG, "scale=%g (positive and below 2.35e38, or 0 for 1/sqrt(head_dim))", d->scale);
  if (d->shared != 0 && d->shared != 1) return cs_fail(CS_ERR_INVALID_ARG, "shared=%d (0 or 1)", d->shared);
  if (d->shared && d->window > 0) return cs_fail(CS_ERR_UNSUPPORTED, "a shared prefix is built without a window");
  if (static_cast<long long>(d->num_pages) * d->kv_heads * (d->page_size / 8) >= (1ll << 31))
    return cs_fail(CS_ERR_UNSUPPORTED, "num_pages=%d times %d heads is more than the copies can address", d->num_pages, d->kv_heads);
  if (d->num_sms < 0) return cs_fail(CS_ERR_INVALID_ARG, "num_sms=%d", d->num_sms);
  return CS_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Row stride of a token-indexed tensor `width` wide: the default, or what the caller gave.
cs_status row_stride(const char* name, long long given, long long width, long long* stride) {
  *stride = given == 0 ? width : given;
  if (*stride < width || *stride % 8 != 0 || *stride > (1ll << 32))
    return cs_fail(CS_ERR_INVALID_ARG, "%s=%lld (0, or a multiple of 8 from %lld on)", name, given, width);
  return CS_OK;
}

// Whether two sets of `rows` rows (16-bit elements) share one: rows of one pitch may lie
// side by side in a wider buffer.
bool rows_overlap(const void* a, long long a_stride, long long a_width, const void* b, long long b_stride, long long b_width,
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
bool rows_over(const void* a, long long stride, long long width, int rows, const void* range, long long bytes) {
  if (!range || bytes <= 0) return false;
  const long long pitch = 2 * stride, from = static_cast<const char*>(range) - static_cast<const char*>(a);
  const long long r = from >= 0 ? from / pitch : -1;  // the last row that begins at or before the range
  if (r >= 0 && r < rows && from < r * pitch + 2 * width) return true;
  return r + 1 < rows && (r + 1) * pitch < from + bytes;
}

long long cache_bytes(const cs_kv_desc& d) {
  return 2ll * d.num_pages * d.page_size * d.kv_heads * d.head_dim;
}

cs_status check_batch(const cs_kv_s* p, const cs_kv_batch* b) {
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

cskv::Batch device_batch(const cs_kv_s* p, const cs_kv_batch* b) {
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
cs_status launch(const void* fn, dim3 grid, int threads, int smem, void* params, cudaStream_t stream) {
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

cs_status check_caches(const void* k, const void* v) {
  if (!k || !v) return cs_fail(CS_ERR_INVALID_ARG, "k_cache and v_cache are required");
  if (!aligned16(k) || !aligned16(v)) return cs_fail(CS_ERR_INVALID_ARG, "the caches must be 16-byte aligned");
  return CS_OK;
}

struct Driver {
  PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  PFN_cuTensorMapReplaceAddress_v12000 replace = nullptr;
};

const Driver& driver() {
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

cs_status encode(CUtensorMap* map, int bf16, const void* ptr, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                 const cuuint32_t* box, const char* name) {
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  const CUresult r = driver().encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank,
                         const_cast<void*>(ptr), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return cs_fail(CS_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d) for %s", static_cast<int>(r), name);
  return CS_OK;
}

// A cache as [8-slot group][head][64-dimension half][slot of the group][64]: one box is
// some slots of a page, of one head.  In the HEAD layout heads are part of the groups' order.
cs_status encode_cache(const cs_kv_desc& d, const cskv::Batch& B, CUtensorMap* map, const void* ptr, int slots) {
  const bool head = d.cache_layout == CS_KV_HEAD;
  const cuuint64_t groups = static_cast<cuuint64_t>(d.num_pages) * (d.page_size / 8);
  const cuuint64_t dims[5] = {64, 8, static_cast<cuuint64_t>(d.head_dim / 64), head ? 1 : static_cast<cuuint64_t>(d.kv_heads),
                              head ? groups * d.kv_heads : groups};
  const cuuint64_t slot = static_cast<cuuint64_t>(B.slot_stride) * 2;
  const cuuint64_t strides[4] = {slot, 128, static_cast<cuuint64_t>(B.head_stride) * 2, 8 * slot};
  const cuuint32_t box[5] = {64, 8, static_cast<cuuint32_t>(d.head_dim / 64), 1, static_cast<cuuint32_t>(slots / 8)};
  return encode(map, d.dtype == CS_BF16, ptr, 5, dims, strides, box, "a cache");
}

cs_status map_caches(cskv::AttnP& k, const CUtensorMap& like) {
  k.k = like;
  k.v = like;
  auto replace = driver().replace;
  if (replace(&k.k, const_cast<void*>(k.k_raw)) != CUDA_SUCCESS || replace(&k.v, const_cast<void*>(k.v_raw)) != CUDA_SUCCESS)
    return cs_fail(CS_ERR_CUDA, "cuTensorMapReplaceAddress failed");
  return CS_OK;
}

cs_status check_attn(const cs_kv_s* p, const cs_kv_batch* b, const cs_kv_attn_args* a, cskv::AttnP& k) {
  if (!a) return cs_fail(CS_ERR_INVALID_ARG, "args is NULL");
  const cs_kv_desc& d = p->d;
  const long long width = static_cast<long long>(d.heads) * d.head_dim;
  std::memset(&k, 0, sizeof(k));
  cs_status s = check_caches(a->k_cache, a->v_cache);
  if (s != CS_OK) return s;
  long long q_stride = 0;
  if ((s = row_stride("q_stride", a->q_stride, width, &q_stride)) != CS_OK) return s;
  if ((s = row_stride("out_stride", a->out_stride, width, &k.out_stride)) != CS_OK) return s;
  if (b->tokens == 0) return CS_OK;
  if (!a->q || !a->out) return cs_fail(CS_ERR_INVALID_ARG, "q and out are required");
  if (!aligned16(a->q) || !aligned16(a->out)) return cs_fail(CS_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
  if (rows_overlap(a->q, q_stride, width, a->out, k.out_stride, width, b->tokens))
    return cs_fail(CS_ERR_INVALID_ARG, "out overlaps q");
  const long long bytes = cache_bytes(d), lse_bytes = 4ll * b->tokens * d.heads;
  if (rows_over(a->out, k.out_stride, width, b->tokens, a->k_cache, bytes) ||
      rows_over(a->out, k.out_stride, width, b->tokens, a->v_cache, bytes))
    return cs_fail(CS_ERR_INVALID_ARG, "out overlaps a cache");
  if (rows_over(a->out, k.out_stride, width, b->tokens, a->lse, lse_bytes) ||
      rows_over(a->q, q_stride, width, b->tokens, a->lse, lse_bytes) ||
      rows_over(a->k_cache, bytes / 2, bytes / 2, 1, a->lse, lse_bytes) ||
      rows_over(a->v_cache, bytes / 2, bytes / 2, 1, a->lse, lse_bytes))
    return cs_fail(CS_ERR_INVALID_ARG, "lse overlaps another argument");
  k.b = device_batch(p, b);
  // a window as long as any sequence hides nothing
  k.c.window = d.window >= kMaxKeys ? 0 : d.window;
  k.c.sinks = k.c.window == 0 ? 0 : d.sinks < kMaxKeys ? d.sinks : kMaxKeys;
  k.c.item_cost = 1;
  k.out = a->out;
  k.lse = a->lse;
  k.scale_log2 = scale_log2(d);
  k.part = p->part;
  k.other = p->other;
  k.splits = p->splits;
  k.num_splits = p->num_sms;
  k.mend = p->mend;
  k.arrivals = p->ctrl + cskv::CTRL_COUNTERS;
  k.q_raw = a->q;
  k.k_raw = a->k_cache;
  k.v_raw = a->v_cache;
  k.q_stride = q_stride;
  k.out_wide = reinterpret_cast<uintptr_t>(a->out) % 32 == 0 && k.out_stride % 16 == 0;
  return CS_OK;
}

const void* join_kernel(const cs_kv_desc& d) {
  if (d.dtype == CS_BF16)
    return d.head_dim == 128 ? (const void*)cskv::cs_kv_join_kernel<__nv_bfloat16, 128>
                             : (const void*)cskv::cs_kv_join_kernel<__nv_bfloat16, 64>;
  return d.head_dim == 128 ? (const void*)cskv::cs_kv_join_kernel<__half, 128> : (const void*)cskv::cs_kv_join_kernel<__half, 64>;
}

const void* rows_kernel(const cs_kv_desc& d) {
  if (d.dtype == CS_BF16)
    return d.head_dim == 128 ? (const void*)cskv::cs_kv_rows_kernel<__nv_bfloat16, 128>
                             : (const void*)cskv::cs_kv_rows_kernel<__nv_bfloat16, 64>;
  return d.head_dim == 128 ? (const void*)cskv::cs_kv_rows_kernel<__half, 128> : (const void*)cskv::cs_kv_rows_kernel<__half, 64>;
}

int rows_smem(const cs_kv_desc& d) {
  return d.head_dim == 128 ? sizeof(cskv::RowsShared<128>) + 1024 : sizeof(cskv::RowsShared<64>) + 1024;
}

// States of pieces: the tensor-core kernel's are larger than the rows kernel's.
size_t part_floats(const cs_kv_desc& d, int num_sms) {
  static_assert(cskv::ROWS_CTAS * 2 * cskv::ROWS * (64 + 4) <= 4 * 128 * (64 + 8), "workspace");
  return static_cast<size_t>(num_sms) * 4 * 128 * (d.head_dim + 8);
}

int rows_grid(const cs_kv_s* p) {
  return p->num_sms * cskv::ROWS_CTAS;
}

template <typename T, int D>
const void* attn_kernel_of(bool window) {
  return window ? (const void*)cskv::cs_kv_attn_kernel<T, D, true> : (const void*)cskv::cs_kv_attn_kernel<T, D, false>;
}

const void* attn_kernel(const cs_kv_desc& d, int* smem) {
  *smem = d.head_dim == 128 ? cskv::AttnShape<128>::SMEM : cskv::AttnShape<64>::SMEM;
  const bool window = d.window > 0 && d.window < kMaxKeys;
  if (d.dtype == CS_BF16)
    return d.head_dim == 128 ? attn_kernel_of<__nv_bfloat16, 128>(window) : attn_kernel_of<__nv_bfloat16, 64>(window);
  return d.head_dim == 128 ? attn_kernel_of<__half, 128>(window) : attn_kernel_of<__half, 64>(window);
}

cs_status run_attention(cs_kv_s* p, cskv::AttnP& k, int max_rows, cudaStream_t st) {
  const cs_kv_desc& d = p->d;
  const bool bf16 = d.dtype == CS_BF16;
  k.head_groups = d.cache_layout == CS_KV_HEAD ? d.page_size / 8 : 0;
  cs_status s;
  if (max_rows <= cskv::ROWS) {
    k.c.per_item = cskv::ROWS / k.b.group;
    k.c.shift = cskv::ROWS_SHIFT;
    if ((s = map_caches(k, p->slots_map)) != CS_OK) return s;
    s = launch(rows_kernel(d), dim3(rows_grid(p)), cskv::ROWS_THREADS, rows_smem(d), &k, st);
    if (s != CS_OK || max_rows <= k.b.group || k.c.flat) return s;
    k.num_splits = 0;  // rows of several tokens: some may have to be mended
    s = launch(join_kernel(d), dim3(p->num_sms), cskv::JOIN_THREADS, 0, &k, st);
    k.num_splits = p->num_sms;
    return s;
  }
  k.per_tile = 128 / k.b.group;
  k.c.per_item = 2 * k.per_tile;
  k.c.shift = 7;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d.head_dim), static_cast<cuuint64_t>(d.heads),
                              static_cast<cuuint64_t>(k.b.tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d.head_dim) * 2, static_cast<cuuint64_t>(k.q_stride) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(k.b.group), static_cast<cuuint32_t>(k.per_tile)};
  s = encode(&k.q, bf16, k.q_raw, 3, dims, strides, box, "q");
  if (s == CS_OK) s = map_caches(k, p->page_map);
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
  int smem = 0;
  const void* fn = attn_kernel(d, &smem);
  if ((s = launch(fn, dim3(p->num_sms), cskv::ATTN_THREADS, smem, &k, st)) != CS_OK) return s;
  return launch(join_kernel(d), dim3((k.c.whole ? 1 : cskv::JOIN_CTAS) * p->num_sms), cskv::JOIN_THREADS, 0, &k, st);
}

cs_status check_append(const cs_kv_s* p, const cs_kv_batch* b, const cs_kv_append_args* a, cskv::AppendP& k) {
  if (!a) return cs_fail(CS_ERR_INVALID_ARG, "args is NULL");
  const cs_kv_desc& d = p->d;
  std::memset(&k, 0, sizeof(k));
  cs_status s = check_caches(a->k_cache, a->v_cache);
  if (s != CS_OK) return s;
  if (b->tokens > 0 && (!a->qkv || !a->q_out)) return cs_fail(CS_ERR_INVALID_ARG, "qkv and q_out are required");
  if (!aligned16(a->qkv) || !aligned16(a->q_out)) return cs_fail(CS_ERR_INVALID_ARG, "qkv and q_out must be 16-byte aligned");
  const long long q_width = static_cast<long long>(d.heads) * d.head_dim;
  const long long width = q_width + 2ll * d.kv_heads * d.head_dim;
  if ((s = row_stride("qkv_stride", a->qkv_stride, width, &k.qkv_stride)) != CS_OK) return s;
  if ((s = row_stride("q_stride", a->q_stride, q_width, &k.q_stride)) != CS_OK) return s;
  if (!(a->q_out == a->qkv && (k.q_stride == k.qkv_stride || b->tokens == 1)) &&
      rows_overlap(a->qkv, k.qkv_stride, width, a->q_out, k.q_stride, q_width, b->tokens))
    return cs_fail(CS_ERR_INVALID_ARG, "q_out overlaps qkv without being its Q part");
  if (d.rotary_dim > 0) {
    if (!a->rope || a->rope_rows < 1) return cs_fail(CS_ERR_INVALID_ARG, "rope is required (rotary_dim=%d)", d.rotary_dim);
    if (!aligned16(a->rope)) return cs_fail(CS_ERR_INVALID_ARG, "rope must be 16-byte aligned");
  }
  const long long bytes = cache_bytes(d);
  if (rows_over(a->k_cache, bytes / 2, bytes / 2, 1, a->v_cache, bytes))
    return cs_fail(CS_ERR_INVALID_ARG, "k_cache and v_cache overlap");
  for (const void* cache : {a->k_cache, a->v_cache})
    if (rows_over(a->q_out, k.q_stride, q_width, b->tokens, cache, bytes) ||
        rows_over(a->qkv, k.qkv_stride, width, b->tokens, cache, bytes))
      return cs_fail(CS_ERR_INVALID_ARG, "qkv or q_out overlaps a cache");
  k.b = device_batch(p, b);
  k.qkv = static_cast<const uint4*>(a->qkv);
  k.q_out = static_cast<uint4*>(a->q_out);
  k.k_cache = static_cast<uint4*>(a->k_cache);
  k.v_cache = static_cast<uint4*>(a->v_cache);
  k.rope = reinterpret_cast<const float4*>(a->rope);
  k.positions = a->positions;
  k.qkv_stride >>= 3;
  k.q_stride >>= 3;
  k.rope_rows = a->rope_rows;
  k.rotary_dim = d.rotary_dim;
  k.half = d.rotary_pairing == CS_KV_HALF;
  k.head_chunks = d.head_dim / 8;
  k.units = (d.heads + 2 * d.kv_heads) * (d.head_dim / 16);
  return CS_OK;
}

cs_status run_append(const cs_kv_s* p, cskv::AppendP& k, cudaStream_t st) {
  if (k.b.tokens == 0 || k.b.seqs == 0) return CS_OK;
  // The lookups of a block's tokens go side by side, so several tokens cost one chain of
  // them; but not before there are two blocks an SM, and not beyond four or five rounds of
  // a block's threads.  Measured, one token a block and by this rule: 19743 tokens of 384
  // units 83 and 74 us, 1962 of 144 units 6.9 and 5.6 us; 253 of 640 units 4.1 us, two a block 4.6.
  const int wanted = std::min(k.b.tokens / (2 * p->num_sms), 1152 / k.units);
  k.tokens_per_block = std::max(1, std::min(wanted, cskv::APPEND_MAX_TOKENS));
  const dim3 grid((k.b.tokens + k.tokens_per_block - 1) / k.tokens_per_block);
  const void* fn = p->d.dtype == CS_BF16 ? (const void*)cskv::cs_kv_append_kernel<__nv_bfloat16>
                                         : (const void*)cskv::cs_kv_append_kernel<__half>;
  return launch(fn, grid, cskv::APPEND_THREADS, 0, &k, st);
}

// Rows of one key head that n new tokens have.
int rows_of(const cskv::AttnP& k, long long n) {
  const long long tokens = n < k.b.tokens ? n : k.b.tokens;
  return static_cast<int>(tokens * k.b.group);
}

cs_status begin(cs_kv_s* p, const cs_kv_batch* b) {
  if (!p) return cs_fail(CS_ERR_INVALID_ARG, "plan is NULL");
  if (p->error_latched) return cs_fail(CS_ERR_NEEDS_RESET, "plan holds a device error; call cs_kv_reset");
  return check_batch(p, b);
}

void free_plan(cs_kv_s* p) {
  cudaFree(p->ctrl);
  cudaFree(p->part);
  cudaFree(p->other);
  cudaFree(p->splits);
  cudaFree(p->mend);
  cudaFree(p->flat_o);
  delete p;
}

}  // namespace

extern "C" {

int cs_kv_abi_version(void) { return CS_KV_ABI_VERSION; }

cs_status cs_kv_desc_init(cs_kv_desc* d) {
  if (!d) return cs_fail(CS_ERR_INVALID_ARG, "desc is NULL");
  std::memset(d, 0, sizeof(*d));
  d->dtype = CS_F16;
  d->head_dim = 128;
  d->page_size = 16;
  return CS_OK;
}

cs_status cs_kv_plan(const cs_kv_desc* desc, cs_kv_t* out) {
  if (!out) return cs_fail(CS_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  cs_status s = validate(desc);
  if (s != CS_OK) return s;
  int dev = 0, sms = 0, major = 0, minor = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_failed("no CUDA device available", e);
  cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  if (major * 10 + minor != 103)
    return cs_fail(CS_ERR_UNSUPPORTED, "device is sm_%d%d; this library is built for sm_103a only", major, minor);
  cs_kv_s* p = new (std::nothrow) cs_kv_s();
  if (!p) return cs_fail(CS_ERR_OOM, "host allocation failed");
  p->d = *desc;
  p->device = dev;
  p->num_sms = desc->num_sms > 0 && desc->num_sms < sms ? desc->num_sms : sms;
  if (p->num_sms > cskv::JOIN_THREADS) p->num_sms = cskv::JOIN_THREADS;
  p->ctrl_words = cskv::CTRL_COUNTERS + (p->d.shared ? 2 : 1) * static_cast<size_t>(rows_grid(p));
  int smem = 0;
  const void* fn = attn_kernel(p->d, &smem);
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
      cudaFuncSetAttribute(rows_kernel(p->d), cudaFuncAttributeMaxDynamicSharedMemorySize, rows_smem(p->d)) != cudaSuccess) {
    cudaGetLastError();
    free_plan(p);
    return cs_fail(CS_ERR_CUDA, "the attention kernels need %d bytes of shared memory", smem);
  }
  const size_t part = (desc->shared ? 2 : 1) * part_floats(*desc, p->num_sms) * 4;
  const size_t other = static_cast<size_t>(p->num_sms) * (desc->head_dim / 4 + 1) * 128 * 16;
  const size_t rows = static_cast<size_t>(desc->max_tokens) * desc->heads;
  const size_t flat = rows * (desc->head_dim + 1) * 4;
  if (cudaMalloc(reinterpret_cast<void**>(&p->ctrl), p->ctrl_words * 4) != cudaSuccess ||
      cudaMalloc(reinterpret_cast<void**>(&p->part), part) != cudaSuccess ||
      cudaMalloc(reinterpret_cast<void**>(&p->other), other) != cudaSuccess ||
      cudaMalloc(reinterpret_cast<void**>(&p->mend), rows) != cudaSuccess ||
      cudaMalloc(reinterpret_cast<void**>(&p->splits), p->num_sms * sizeof(cskv::Split)) != cudaSuccess ||
      (desc->shared && cudaMalloc(reinterpret_cast<void**>(&p->flat_o), flat) != cudaSuccess)) {
    cudaGetLastError();
    free_plan(p);
    return cs_fail(CS_ERR_OOM, "cudaMalloc of the plan's workspace failed");
  }
  if (cudaMemset(p->ctrl, 0, p->ctrl_words * 4) != cudaSuccess || cudaMemset(p->mend, 0, rows) != cudaSuccess ||
      cudaDeviceSynchronize() != cudaSuccess) {
    cudaGetLastError();
    free_plan(p);
    return cs_fail(CS_ERR_CUDA, "clearing the plan's workspace failed");
  }
  if (!driver().encode || !driver().replace) s = cs_fail(CS_ERR_CUDA, "the driver has no tensor maps (too old?)");
  const cs_kv_batch none{};
  const cskv::Batch geometry = device_batch(p, &none);
  if (s == CS_OK) s = encode_cache(p->d, geometry, &p->page_map, p->part, p->d.page_size);
  if (s == CS_OK) s = encode_cache(p->d, geometry, &p->slots_map, p->part, 16);
  if (s != CS_OK) {
    free_plan(p);
    return s;
  }
  *out = p;
  return CS_OK;
}

cs_status cs_kv_destroy(cs_kv_t p) {
  if (!p) return CS_OK;
  DeviceGuard g(p->device);
  if (cudaDeviceSynchronize() != cudaSuccess) cudaGetLastError();
  free_plan(p);
  return CS_OK;
}

cs_status cs_kv_append(cs_kv_t p, const cs_kv_batch* b, const cs_kv_append_args* a, void* stream) {
  cs_status s = begin(p, b);
  if (s != CS_OK) return s;
  cskv::AppendP k;
  if ((s = check_append(p, b, a, k)) != CS_OK) return s;
  DeviceGuard g(p->device);
  if (!g.ok) return cs_fail(CS_ERR_CUDA, "cannot select the plan's device");
  return run_append(p, k, static_cast<cudaStream_t>(stream));
}

cs_status cs_kv_attention(cs_kv_t p, const cs_kv_batch* b, const cs_kv_attn_args* a, void* stream) {
  cs_status s = begin(p, b);
  if (s != CS_OK) return s;
  cskv::AttnP k;
  if ((s = check_attn(p, b, a, k)) != CS_OK) return s;
  DeviceGuard g(p->device);
  if (!g.ok) return cs_fail(CS_ERR_CUDA, "cannot select the plan's device");
  if (b->tokens == 0 || b->seqs == 0) return CS_OK;
  return run_attention(p, k, rows_of(k, b->max_q), static_cast<cudaStream_t>(stream));
}

cs_status cs_kv_attention_shared(cs_kv_t p, const cs_kv_batch* b, const int32_t* prefix_pages, int prefix_len,
                                 const cs_kv_attn_args* a, void* stream) {
  cs_status s = begin(p, b);
  if (s != CS_OK) return s;
  if (!p->d.shared) return cs_fail(CS_ERR_INVALID_ARG, "the plan was made without desc.shared");
  if (prefix_len < 0 || prefix_len > kMaxKeys) return cs_fail(CS_ERR_INVALID_ARG, "prefix_len=%d (0..%d)", prefix_len, kMaxKeys);
  if (!prefix_pages && prefix_len > 0) return cs_fail(CS_ERR_INVALID_ARG, "prefix_pages is NULL");
  cskv::AttnP k;
  if ((s = check_attn(p, b, a, k)) != CS_OK) return s;
  DeviceGuard g(p->device);
  if (!g.ok) return cs_fail(CS_ERR_CUDA, "cannot select the plan's device");
  if (b->tokens == 0 || b->seqs == 0) return CS_OK;
  if (prefix_len > 0) {
    // all tokens of the batch over the prefix; then every sequence's own keys, which join it
    k.flat_o = p->flat_o;
    k.flat_lse = p->flat_o + static_cast<size_t>(p->d.max_tokens) * p->d.heads * p->d.head_dim;
    k.pages = prefix_pages;
    k.c.flat = 1;
    k.c.flat_len = prefix_len;
    if ((s = run_attention(p, k, rows_of(k, b->seqs * static_cast<long long>(b->max_q)), static_cast<cudaStream_t>(stream))) != CS_OK) return s;
    k.c.flat = 0;
    k.part += part_floats(p->d, p->num_sms);  // the rows kernel does not wait for the prefix's phase
    k.arrivals += rows_grid(p);
  }
  return run_attention(p, k, rows_of(k, b->max_q), static_cast<cudaStream_t>(stream));
}

cs_status cs_attn_cached_forward(cs_chain_t chain, cs_kv_t p, const cs_kv_batch* b, const cs_attn_args* args,
                                 const cs_kv_append_args* append_args, void* stream) {
  cs_status s = begin(p, b);
  if (s != CS_OK) return s;
  if (!chain || !args || !append_args) return cs_fail(CS_ERR_INVALID_ARG, "chain, args and append are required");
  cs_chain_info info;
  if ((s = cs_chain_query(chain, &info)) != CS_OK) return s;
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
  cs_kv_append_args ap = *append_args;
  ap.qkv = info.intermediate[0];
  ap.q_out = info.intermediate[0];
  ap.qkv_stride = ap.q_stride = 3ll * cd.F;
  cs_kv_attn_args at;
  std::memset(&at, 0, sizeof(at));
  at.q = info.intermediate[0];
  at.q_stride = 3ll * cd.F;
  at.k_cache = ap.k_cache;
  at.v_cache = ap.v_cache;
  at.out = info.intermediate[1];
  // what can be refused is, before any stage has run
  cskv::AppendP ak;
  cskv::AttnP k;
  if ((s = check_append(p, b, &ap, ak)) != CS_OK || (s = check_attn(p, b, &at, k)) != CS_OK) return s;
  DeviceGuard g(p->device);
  if (!g.ok) return cs_fail(CS_ERR_CUDA, "cannot select the plan's device");
  if ((s = cs_chain_forward_stage(chain, args, 0, stream)) != CS_OK) return s;
  if (b->seqs > 0) {
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if ((s = run_append(p, ak, st)) != CS_OK) return s;
    if ((s = run_attention(p, k, rows_of(k, b->max_q), st)) != CS_OK) return s;
  }
  return cs_chain_forward_stage(chain, args, 2, stream);
}

cs_status cs_kv_status(cs_kv_t p) {
  if (!p) return cs_fail(CS_ERR_INVALID_ARG, "plan is NULL");
  DeviceGuard g(p->device);
  uint32_t w[3];
  KV_CUDA(cudaMemcpy(w, p->ctrl, sizeof(w), cudaMemcpyDeviceToHost));
  if (w[cskv::CTRL_ERROR] == 0) return CS_OK;
  p->error_latched = true;
  const cs_status code = static_cast<cs_status>(w[cskv::CTRL_ERROR]);
  const uint32_t i = w[cskv::CTRL_INDEX];
  switch (w[cskv::CTRL_WHAT]) {
    case cskv::WHAT_LENGTHS:
      return cs_fail(code, "cu_q or kv_lens of sequence %u does not fit the call", i);
    case cskv::WHAT_PAGE:
      return cs_fail(code, "a page of sequence %u (%u: of the prefix) is not in the pool", i, 0xFFFFFFFFu);
    case cskv::WHAT_POSITION:
      return cs_fail(code, "the position of token %u has no row in rope", i);
    default:
      return cs_fail(code, "a wait inside a kernel ran out (at %u)", i);
  }
}

cs_status cs_kv_reset(cs_kv_t p) {
  if (!p) return cs_fail(CS_ERR_INVALID_ARG, "plan is NULL");
  DeviceGuard g(p->device);
  KV_CUDA(cudaDeviceSynchronize());
  KV_CUDA(cudaMemset(p->ctrl, 0, p->ctrl_words * 4));
  KV_CUDA(cudaMemset(p->mend, 0, static_cast<size_t>(p->d.max_tokens) * p->d.heads));
  KV_CUDA(cudaDeviceSynchronize());
  p->error_latched = false;
  return CS_OK;
}

}  // extern "C"
