// Host side of the paged key/value cache held in 4 bits (include/cs_kv4.h): argument
// checks and launches.
#include "../../include/cs_kv4.h"
#include "cs_kv4_append.cuh"
#include "cs_kv4_rows.cuh"
#include "cs_kv_host.cuh"

namespace {

static_assert(cskv::ROWS4_CTAS<64, 1> <= kRowsCtas && cskv::ROWS4_CTAS<128, 1> <= kRowsCtas, "counters and pieces");

long long code_bytes(const cs_kv_desc& d) {
  return static_cast<long long>(d.num_pages) * d.page_size * d.kv_heads * d.head_dim / 2;
}
long long scale_bytes(const cs_kv_desc& d) { return code_bytes(d) / (cskv::GROUP4 / 2); }

// The parts of the caches that are used, K's and V's.
struct Parts {
  Held held[4];
  int count = 0;
};

cs_status add_cache(const cs_kv_desc& d, const char* name, const cs_kv4_cache& c, Parts& parts) {
  if (!c.codes || !c.scales) return cs_fail(CS_ERR_INVALID_ARG, "the codes and scales of %s are required", name);
  if (!aligned16(c.codes) || !aligned16(c.scales))
    return cs_fail(CS_ERR_INVALID_ARG, "the codes and scales of %s must be 16-byte aligned", name);
  parts.held[parts.count++] = {c.codes, code_bytes(d)};
  parts.held[parts.count++] = {c.scales, scale_bytes(d)};
  return CS_OK;
}

cs_status add_caches(const cs_kv_desc& d, const cs_kv4_cache& k, const cs_kv4_cache& v, Parts& parts) {
  const cs_status s = add_cache(d, "k", k, parts);
  return s != CS_OK ? s : add_cache(d, "v", v, parts);
}

template <typename T, int D, int NT>
const void* rows_kernel_of(bool by_head) {
  return by_head ? (const void*)cskv::cs_kv4_rows_kernel<T, D, NT, true> : (const void*)cskv::cs_kv4_rows_kernel<T, D, NT, false>;
}

template <typename T, int D>
Kernels kernels_of(const cs_kv_s* p, int max_rows) {
  const bool window = p->d.window > 0 && p->d.window < kMaxKeys, narrow = max_rows <= 8;
  Kernels u;
  u.rows_grid = p->num_sms * (narrow ? cskv::ROWS4_CTAS<D, 1> : cskv::ROWS4_CTAS<D, 2>);
  // with the heads' rows side by side, and at least eight CTAs for each, by heads
  const bool by_head = p->d.cache_layout == CS_KV_TOKEN && p->d.kv_heads > 1 && u.rows_grid >= 8 * p->d.kv_heads;
  u.head_ctas = by_head ? u.rows_grid / p->d.kv_heads : 0;
  u.rows = narrow ? rows_kernel_of<T, D, 1>(by_head) : rows_kernel_of<T, D, 2>(by_head);
  u.attn = window ? (const void*)cskv::cs_kv_attn_kernel<T, D, true, true> : (const void*)cskv::cs_kv_attn_kernel<T, D, false, true>;
  u.join = (const void*)cskv::cs_kv_join_kernel<T, D, true>;
  // Ranges of one, two and four tiles at least: one token over 16000 keys 35.8, 34.4 and 31.0 us, 128 of them over 100
  // keys 19.9, 20.0 and 23.1.
  u.least = 2;
  // Whole items save the pieces' stores and joins, and load the CTAs less evenly.  Measured, whole and cut, 32 / 8 heads of 128,
  // keys of each sequence between the numbers given: 57 sequences (a CTA each) 1..500 16.7 and 18.0 us, 250..500 19.8 and
  // 19.8, 1..760 18.7 and 20.8, 380..760 24.7 and 23.0, 510..1020 28.5 and 24.9, one of 1020 beside 1..100 14.6 and 12.4, one of
  // 32000 beside 500 277 and 30; 114 of them 1..500 25.7 and 26.2, 250..500 29.7 and 29.2, 510..1020 43.5 and 40.8; 6
  // sequences of 250 7.2 and 8.7, 50 of 250..500 14.4 and 18.3.  40 / 8 heads of 64, 76 sequences: 1..500 15.3 and 16.4, 510..1020
  // 26.6 and 23.6.  So up to four tiles, where whole costs at most 2 %.
  u.uncut = 4;
  u.spare = 3;
  u.rows_shift = cskv::ROWS4_SHIFT;
  u.rows_smem = sizeof(cskv::Rows4Shared<D>);
  u.attn_smem = cskv::AttnShape<D, true>::SMEM;
  u.attn_threads = cskv::ATTN_THREADS_OF<true>;
  u.rows_map = nullptr;
  u.attn_map = &p->codes_map;
  return u;
}

Kernels kernels(const cs_kv_s* p, int max_rows) {
  if (p->d.dtype == CS_BF16)
    return p->d.head_dim == 128 ? kernels_of<__nv_bfloat16, 128>(p, max_rows) : kernels_of<__nv_bfloat16, 64>(p, max_rows);
  return p->d.head_dim == 128 ? kernels_of<__half, 128>(p, max_rows) : kernels_of<__half, 64>(p, max_rows);
}

// A cache's codes as [8-slot group][head][slot of the group][head_dim / 2 bytes]: one box is a page's slots of a
// head.  In the HEAD layout heads are part of the groups' order.
cs_status encode_codes(const cs_kv_s* p, CUtensorMap* map) {
  const cs_kv_desc& d = p->d;
  const cs_kv_batch none{};
  const cskv::Batch B = device_batch(p, &none);
  const bool head = d.cache_layout == CS_KV_HEAD;
  const cuuint64_t groups = static_cast<cuuint64_t>(d.num_pages) * (d.page_size / 8), width = d.head_dim / 2;
  const cuuint64_t dims[4] = {width, 8, head ? 1 : static_cast<cuuint64_t>(d.kv_heads), head ? groups * d.kv_heads : groups};
  const cuuint64_t slot = static_cast<cuuint64_t>(B.slot_stride) / 2;
  const cuuint64_t strides[3] = {slot, static_cast<cuuint64_t>(B.head_stride) / 2, 8 * slot};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(width), 8, 1, static_cast<cuuint32_t>(d.page_size / 8)}, ones[4] = {1, 1, 1, 1};
  const CUresult r = driver().encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, p->part, dims, strides, box, ones,
                                     CU_TENSOR_MAP_INTERLEAVE_NONE, width == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B,
                                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return cs_fail(CS_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d) for a cache's codes", static_cast<int>(r));
  return CS_OK;
}

// Once for a plan, on its device: the shared memory of its kernels, and the map of its copies.
cs_status make_ready(cs_kv_s* p) {
  if (p->four_ready) return CS_OK;
  const cs_status s = encode_codes(p, &p->codes_map);
  if (s != CS_OK) return s;
  for (int rows : {1, 16}) {
    const Kernels u = kernels(p, rows);
    cudaError_t e = cudaFuncSetAttribute(u.rows, cudaFuncAttributeMaxDynamicSharedMemorySize, u.rows_smem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(u.attn, cudaFuncAttributeMaxDynamicSharedMemorySize, u.attn_smem);
    if (e != cudaSuccess) return cuda_failed("shared memory of the attention kernels", e);
  }
  p->four_ready = true;
  return CS_OK;
}

cs_status check_attn4(const cs_kv_s* p, const cs_kv_batch* b, const cs_kv4_attn_args* a, cskv::AttnP& k) {
  if (!a) return cs_fail(CS_ERR_INVALID_ARG, "args is NULL");
  std::memset(&k, 0, sizeof(k));
  Parts parts;
  cs_status s = add_caches(p->d, a->k, a->v, parts);
  if (s != CS_OK) return s;
  k.k_raw = a->k.codes;
  k.v_raw = a->v.codes;
  k.k_scales = static_cast<const uint8_t*>(a->k.scales);
  k.v_scales = static_cast<const uint8_t*>(a->v.scales);
  return check_attn_rows(p, b, a->q, a->q_stride, a->out, a->out_stride, a->lse, parts.held, parts.count, k);
}

void fill_places(const cs_kv_s* p, const cs_kv_batch* b, const cs_kv4_cache& k, const cs_kv4_cache& v, cskv::Four4P& f) {
  f.b = device_batch(p, b);
  f.k_codes = static_cast<uint8_t*>(k.codes);
  f.v_codes = static_cast<uint8_t*>(v.codes);
  f.k_scales = static_cast<uint8_t*>(k.scales);
  f.v_scales = static_cast<uint8_t*>(v.scales);
  f.head_chunks = p->d.head_dim / 8;
  f.head_shift = p->d.head_dim == 128 ? 4 : 3;
}

cs_status check_append4(const cs_kv_s* p, const cs_kv_batch* b, const cs_kv4_append_args* a, cskv::Four4P& f) {
  if (!a) return cs_fail(CS_ERR_INVALID_ARG, "args is NULL");
  const cs_kv_desc& d = p->d;
  std::memset(&f, 0, sizeof(f));
  Parts parts;
  cs_status s = add_caches(d, a->k, a->v, parts);
  if (s != CS_OK) return s;
  cs_kv_append_args rows{};
  rows.qkv = a->qkv;
  rows.qkv_stride = a->qkv_stride;
  rows.q_out = a->q_out;
  rows.q_stride = a->q_stride;
  rows.rope = a->rope;
  rows.rope_rows = a->rope_rows;
  if ((s = check_append_rows(p, b, &rows, parts.held, parts.count, &f.qkv_stride, &f.q_stride)) != CS_OK) return s;
  fill_places(p, b, a->k, a->v, f);
  f.qkv = static_cast<const uint4*>(a->qkv);
  f.q_out = static_cast<uint4*>(a->q_out);
  f.rope = reinterpret_cast<const float4*>(a->rope);
  f.positions = a->positions;
  f.qkv_stride >>= 3;
  f.q_stride >>= 3;
  f.rope_rows = a->rope_rows;
  f.rotary_dim = d.rotary_dim;
  f.half = d.rotary_pairing == CS_KV_HALF;
  f.units = 2 * d.kv_heads * f.head_chunks;
  f.q_units = d.heads * (f.head_chunks / 2);
  return CS_OK;
}

// A token's values are shared out to eight warps, or fewer once there are more than eight times as many of them as the SMs hold: each
// of a token's warps looks its place up.
cs_status run_places(const cs_kv_s* p, const void* fn, cskv::Four4P& f, cudaStream_t st) {
  if (f.b.tokens == 0 || f.b.seqs == 0) return CS_OK;
  constexpr int WARPS = cskv::FOUR_THREADS / 32;
  f.warps_shift = 3;
  while (f.warps_shift > 0 && (static_cast<long long>(f.b.tokens) << f.warps_shift) > 8ll * 48 * p->num_sms) --f.warps_shift;
  const dim3 grid(static_cast<unsigned>(((static_cast<long long>(f.b.tokens) << f.warps_shift) + WARPS - 1) / WARPS));
  return launch(fn, grid, cskv::FOUR_THREADS, 0, &f, st);
}

cs_status run_append4(const cs_kv_s* p, cskv::Four4P& f, cudaStream_t st) {
  const void* fn = p->d.dtype == CS_BF16 ? (const void*)cskv::cs_kv4_append_kernel<__nv_bfloat16>
                                         : (const void*)cskv::cs_kv4_append_kernel<__half>;
  return run_places(p, fn, f, st);
}

cs_status check_read4(const cs_kv_s* p, const cs_kv_batch* b, const cs_kv4_read_args* a, cskv::Four4P& f) {
  if (!a) return cs_fail(CS_ERR_INVALID_ARG, "args is NULL");
  const cs_kv_desc& d = p->d;
  std::memset(&f, 0, sizeof(f));
  const long long width = static_cast<long long>(d.kv_heads) * d.head_dim;
  cs_status s;
  if (b->tokens > 0 && !a->k_out && !a->v_out) return cs_fail(CS_ERR_INVALID_ARG, "k_out or v_out is required");
  if (!aligned16(a->k_out) || !aligned16(a->v_out)) return cs_fail(CS_ERR_INVALID_ARG, "k_out and v_out must be 16-byte aligned");
  Parts parts;
  if (a->k_out && (s = add_cache(d, "k", a->k, parts)) != CS_OK) return s;
  if (a->v_out && (s = add_cache(d, "v", a->v, parts)) != CS_OK) return s;
  if ((s = row_stride("k_stride", a->k_stride, width, &f.k_stride)) != CS_OK) return s;
  if ((s = row_stride("v_stride", a->v_stride, width, &f.v_stride)) != CS_OK) return s;
  if (a->k_out && a->v_out && rows_overlap(a->k_out, f.k_stride, width, a->v_out, f.v_stride, width, b->tokens))
    return cs_fail(CS_ERR_INVALID_ARG, "k_out overlaps v_out");
  for (int i = 0; i < parts.count; ++i)
    if ((a->k_out && rows_over(a->k_out, f.k_stride, width, b->tokens, parts.held[i].at, parts.held[i].bytes)) ||
        (a->v_out && rows_over(a->v_out, f.v_stride, width, b->tokens, parts.held[i].at, parts.held[i].bytes)))
      return cs_fail(CS_ERR_INVALID_ARG, "k_out or v_out overlaps a cache");
  fill_places(p, b, a->k, a->v, f);
  f.k_out = static_cast<uint4*>(a->k_out);
  f.v_out = static_cast<uint4*>(a->v_out);
  f.k_stride >>= 3;
  f.v_stride >>= 3;
  f.wide = ((reinterpret_cast<uintptr_t>(a->k_out) | reinterpret_cast<uintptr_t>(a->v_out)) % 32 == 0) && (f.k_stride | f.v_stride) % 2 == 0;
  f.units = ((a->k_out ? 1 : 0) + (a->v_out ? 1 : 0)) * d.kv_heads * (f.head_chunks / 2);
  return CS_OK;
}

}  // namespace

extern "C" {

cs_status cs_kv4_append(cs_kv_t p, const cs_kv_batch* b, const cs_kv4_append_args* a, void* stream) {
  cs_status s = begin(p, b);
  if (s != CS_OK) return s;
  cskv::Four4P f;
  if ((s = check_append4(p, b, a, f)) != CS_OK) return s;
  DeviceGuard g(p->device);
  if (!g.ok) return cs_fail(CS_ERR_CUDA, "cannot select the plan's device");
  return run_append4(p, f, static_cast<cudaStream_t>(stream));
}

cs_status cs_kv4_read(cs_kv_t p, const cs_kv_batch* b, const cs_kv4_read_args* a, void* stream) {
  cs_status s = begin(p, b);
  if (s != CS_OK) return s;
  cskv::Four4P f;
  if ((s = check_read4(p, b, a, f)) != CS_OK) return s;
  DeviceGuard g(p->device);
  if (!g.ok) return cs_fail(CS_ERR_CUDA, "cannot select the plan's device");
  const void* fn = p->d.dtype == CS_BF16 ? (const void*)cskv::cs_kv4_read_kernel<__nv_bfloat16>
                                         : (const void*)cskv::cs_kv4_read_kernel<__half>;
  return run_places(p, fn, f, static_cast<cudaStream_t>(stream));
}

cs_status cs_kv4_attention(cs_kv_t p, const cs_kv_batch* b, const cs_kv4_attn_args* a, void* stream) {
  cs_status s = begin(p, b);
  if (s != CS_OK) return s;
  cskv::AttnP k;
  if ((s = check_attn4(p, b, a, k)) != CS_OK) return s;
  DeviceGuard g(p->device);
  if (!g.ok) return cs_fail(CS_ERR_CUDA, "cannot select the plan's device");
  if (b->tokens == 0 || b->seqs == 0) return CS_OK;
  if ((s = make_ready(p)) != CS_OK) return s;
  const int rows = rows_of(k, b->max_q);
  return run_attention(p, k, kernels(p, rows), rows, static_cast<cudaStream_t>(stream));
}

cs_status cs_kv4_attention_shared(cs_kv_t p, const cs_kv_batch* b, const int32_t* prefix_pages, int prefix_len,
                                  const cs_kv4_attn_args* a, void* stream) {
  cs_status s = begin(p, b);
  if (s != CS_OK) return s;
  if ((s = check_prefix(p, prefix_pages, prefix_len)) != CS_OK) return s;
  cskv::AttnP k;
  if ((s = check_attn4(p, b, a, k)) != CS_OK) return s;
  DeviceGuard g(p->device);
  if (!g.ok) return cs_fail(CS_ERR_CUDA, "cannot select the plan's device");
  if (b->tokens == 0 || b->seqs == 0) return CS_OK;
  if ((s = make_ready(p)) != CS_OK) return s;
  return run_shared(p, k, b, prefix_pages, prefix_len, [&](int rows) { return kernels(p, rows); }, static_cast<cudaStream_t>(stream));
}

cs_status cs_attn_cached4_forward(cs_chain_t chain, cs_kv_t p, const cs_kv_batch* b, const cs_attn_args* args,
                                  const cs_kv4_append_args* append_args, void* stream) {
  cs_status s = begin(p, b);
  if (s != CS_OK) return s;
  if (!chain || !args || !append_args) return cs_fail(CS_ERR_INVALID_ARG, "chain, args and append are required");
  cs_chain_info info;
  if ((s = check_layer(chain, p, b, info)) != CS_OK) return s;
  cs_kv4_append_args ap = *append_args;
  ap.qkv = info.intermediate[0];
  ap.q_out = info.intermediate[0];
  ap.qkv_stride = ap.q_stride = 3ll * p->d.heads * p->d.head_dim;
  cs_kv4_attn_args at{};
  at.q = info.intermediate[0];
  at.q_stride = ap.qkv_stride;
  at.k = ap.k;
  at.v = ap.v;
  at.out = info.intermediate[1];
  // what can be refused is, before any stage has run
  cskv::Four4P f;
  cskv::AttnP k;
  if ((s = check_append4(p, b, &ap, f)) != CS_OK || (s = check_attn4(p, b, &at, k)) != CS_OK) return s;
  DeviceGuard g(p->device);
  if (!g.ok) return cs_fail(CS_ERR_CUDA, "cannot select the plan's device");
  if ((s = make_ready(p)) != CS_OK) return s;
  if ((s = cs_chain_forward_stage(chain, args, 0, stream)) != CS_OK) return s;
  if (b->seqs > 0) {
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int rows = rows_of(k, b->max_q);
    if ((s = run_append4(p, f, st)) != CS_OK) return s;
    if ((s = run_attention(p, k, kernels(p, rows), rows, st)) != CS_OK) return s;
  }
  return cs_chain_forward_stage(chain, args, 2, stream);
}

}  // extern "C"
