// Host side of the paged key/value cache operators (include/cs_kv.h): plans,
// argument checks, launches and status.
#include <new>

#include "cs_kv_host.cuh"

namespace {

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

cs_status check_caches(const void* k, const void* v) {
  if (!k || !v) return cs_fail(CS_ERR_INVALID_ARG, "k_cache and v_cache are required");
  if (!aligned16(k) || !aligned16(v)) return cs_fail(CS_ERR_INVALID_ARG, "the caches must be 16-byte aligned");
  return CS_OK;
}

long long cache_bytes(const cs_kv_desc& d) {
  return 2ll * d.num_pages * d.page_size * d.kv_heads * d.head_dim;
}

cs_status check_attn(const cs_kv_s* p, const cs_kv_batch* b, const cs_kv_attn_args* a, cskv::AttnP& k) {
  if (!a) return cs_fail(CS_ERR_INVALID_ARG, "args is NULL");
  std::memset(&k, 0, sizeof(k));
  const cs_status s = check_caches(a->k_cache, a->v_cache);
  if (s != CS_OK) return s;
  const long long bytes = cache_bytes(p->d);
  const Held held[2] = {{a->k_cache, bytes}, {a->v_cache, bytes}};
  k.k_raw = a->k_cache;
  k.v_raw = a->v_cache;
  return check_attn_rows(p, b, a->q, a->q_stride, a->out, a->out_stride, a->lse, held, 2, k);
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

Kernels kernels(const cs_kv_s* p) {
  Kernels u;
  u.rows = rows_kernel(p->d);
  u.attn = attn_kernel(p->d, &u.attn_smem);
  u.attn_threads = cskv::ATTN_THREADS;
  u.join = join_kernel(p->d);
  u.rows_grid = p->num_sms * cskv::ROWS_CTAS;
  u.rows_shift = cskv::ROWS_SHIFT;
  u.head_ctas = 0;
  u.least = 1;
  u.uncut = 0;
  u.spare = 0;
  u.rows_smem = rows_smem(p->d);
  u.rows_map = &p->slots_map;
  u.attn_map = &p->page_map;
  return u;
}

cs_status check_append(const cs_kv_s* p, const cs_kv_batch* b, const cs_kv_append_args* a, cskv::AppendP& k) {
  if (!a) return cs_fail(CS_ERR_INVALID_ARG, "args is NULL");
  const cs_kv_desc& d = p->d;
  std::memset(&k, 0, sizeof(k));
  cs_status s = check_caches(a->k_cache, a->v_cache);
  if (s != CS_OK) return s;
  const long long bytes = cache_bytes(d);
  const Held held[2] = {{a->k_cache, bytes}, {a->v_cache, bytes}};
  if ((s = check_append_rows(p, b, a, held, 2, &k.qkv_stride, &k.q_stride)) != CS_OK) return s;
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
  p->ctrl_words = cskv::CTRL_COUNTERS + (p->d.shared ? 2 : 1) * static_cast<size_t>(arrival_words(p));
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
  return run_attention(p, k, kernels(p), rows_of(k, b->max_q), static_cast<cudaStream_t>(stream));
}

cs_status cs_kv_attention_shared(cs_kv_t p, const cs_kv_batch* b, const int32_t* prefix_pages, int prefix_len,
                                 const cs_kv_attn_args* a, void* stream) {
  cs_status s = begin(p, b);
  if (s != CS_OK) return s;
  if ((s = check_prefix(p, prefix_pages, prefix_len)) != CS_OK) return s;
  cskv::AttnP k;
  if ((s = check_attn(p, b, a, k)) != CS_OK) return s;
  DeviceGuard g(p->device);
  if (!g.ok) return cs_fail(CS_ERR_CUDA, "cannot select the plan's device");
  if (b->tokens == 0 || b->seqs == 0) return CS_OK;
  return run_shared(p, k, b, prefix_pages, prefix_len, [&](int) { return kernels(p); }, static_cast<cudaStream_t>(stream));
}

cs_status cs_attn_cached_forward(cs_chain_t chain, cs_kv_t p, const cs_kv_batch* b, const cs_attn_args* args,
                                 const cs_kv_append_args* append_args, void* stream) {
  cs_status s = begin(p, b);
  if (s != CS_OK) return s;
  if (!chain || !args || !append_args) return cs_fail(CS_ERR_INVALID_ARG, "chain, args and append are required");
  cs_chain_info info;
  if ((s = check_layer(chain, p, b, info)) != CS_OK) return s;
  const cs_chain_desc& cd = *cs_chain_desc_of(chain);
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
    if ((s = run_attention(p, k, kernels(p), rows_of(k, b->max_q), st)) != CS_OK) return s;
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
