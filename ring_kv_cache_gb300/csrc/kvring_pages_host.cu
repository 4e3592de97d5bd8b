// Host side of the paged cache: argument checks, buffer carving, TMA maps
// and launches.  As on the ring's side, every entry point only enqueues work
// (kvring_pages_create alone waits, for its own set-up) and none allocates
// device memory.
#include <cmath>
#include <cstring>
#include <new>

#include "kvring_pages.cuh"

struct kvring_pages {
  kvring_pages_config cfg;
  kvr::PagesDev dev;
  CUtensorMap tmK, tmV;   // [L * num_pages * Hkv][P][d] in boxes of a page, or 128 rows of one
  const void* buf;        // the caller's, layout.total bytes
  size_t bytes;
  int sm_count;
  int device;
  int max_new, requests;  // of the last plan: bound on new tokens per request, requests (they pick kernels only)
  unsigned long long wait_ns;
  int debug_stall;
};

namespace {

constexpr size_t kAlign = 256;
constexpr unsigned long long kDefaultWaitNs = 1000000000ull;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool config_ok(const kvring_pages_config* c) {
  if (!c) return false;
  if (c->num_kv_heads < 1 || c->num_q_heads < 1 || c->num_q_heads > 4096) return false;
  if (c->num_q_heads % c->num_kv_heads != 0 || c->num_q_heads / c->num_kv_heads > 64) return false;
  if (c->head_dim != 64 && c->head_dim != 128) return false;
  if (c->num_layers < 1 || c->num_layers > 1024) return false;
  const int P = c->page_size;
  if (P != 16 && P != 32 && P != 64 && P != 128 && P != 256) return false;
  if (c->num_pages < 1 || (int64_t)c->num_pages * c->num_kv_heads * P >= (int64_t)1 << 31) return false;
  if ((int64_t)c->num_layers * c->num_pages * c->num_kv_heads >= ((int64_t)1 << 31) - 1) return false;
  if (c->max_requests < 1 || c->max_requests > kvr::kMaxRows) return false;
  if (c->max_pages_per_request < 1 || (int64_t)c->max_pages_per_request * P > (1 << 24)) return false;
  if (c->max_tokens < 1 || c->max_tokens > (1 << 20)) return false;
  if (c->cache_dtype != KVRING_CACHE_E4M3 && c->cache_dtype != KVRING_CACHE_BF16) return false;
  if (c->rope_pairing != KVRING_ROPE_ADJACENT && c->rope_pairing != KVRING_ROPE_HALVES) return false;
  if (c->reserved != 0) return false;
  return c->rope_base > 0.0 && std::isfinite(c->rope_base);
}

struct Plan {
  kvring_pages_layout pub;
  size_t table, part_o, part_ml, tickets, few_o, few_ml;
  size_t cache_bytes;   // of K, and of V
};

Plan plan_for(const kvring_pages_config* c) {
  Plan p{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = (off + bytes + kAlign - 1) & ~(kAlign - 1);
    return at;
  };
  const size_t esz = c->cache_dtype == KVRING_CACHE_E4M3 ? 1 : 2, D = (size_t)c->head_dim, R = (size_t)c->max_requests;
  const size_t W = (size_t)c->max_pages_per_request, T = (size_t)c->max_tokens;
  p.cache_bytes = (size_t)c->num_layers * c->num_pages * c->num_kv_heads * c->page_size * D * esz;
  p.pub.k_cache = take(p.cache_bytes);
  p.pub.v_cache = take(p.cache_bytes);
  p.pub.scales = take((size_t)c->num_layers * 4 * c->num_kv_heads * 4);
  p.pub.lengths = take(R * 4);
  p.pub.tables = take(R * W * 4);
  p.pub.free_pages = take((size_t)c->num_pages * 4);
  p.pub.state = take(kvr::PST_WORDS_ALLOC * 4);
  p.pub.step_rows = take(R * 4);
  p.pub.step_cu = take((R + 1) * 4);
  p.pub.step_lengths = take(R * 4);
  p.pub.positions = take(T * 4);
  p.pub.slots = take(T * 4);
  p.table = take(W * c->page_size * D * 4);
  p.part_o = take((size_t)2 * kvr::kPagedMaxCtas * kvr::kPartRows * D * 4);
  p.part_ml = take((size_t)2 * kvr::kPagedMaxCtas * kvr::kPartRows * 8);
  p.tickets = take((size_t)3 * kvr::kPagedMaxCtas * 4);   // two per CTA, and one of the other kernel
  p.few_o = take((size_t)2 * kvr::kPagedMaxCtas * kvr::kFewRows * D * 4);
  p.few_ml = take((size_t)2 * kvr::kPagedMaxCtas * kvr::kFewRows * 8);
  p.pub.total = off;
  return p;
}

bool on_device(const kvring_pages* h) {
  int cur = -1;
  return cudaGetDevice(&cur) == cudaSuccess && cur == h->device;
}

kvring_status cuda_status(cudaError_t e) { return e == cudaSuccess ? KVRING_OK : KVRING_ERR_CUDA; }

// The pool of one kind (K or V, every layer) as [pages x heads][P][d]: boxes
// of a page's rows (at most 128), 64 columns (128 bytes) wide for bf16, whole
// rows for E4M3, in the swizzle the attention kernels read.
bool make_pool_map(CUtensorMap* m, void* base, const kvring_pages_config* c) {
  auto fn = kvr::encode_tiled();
  if (!fn) return false;
  const bool e4m3 = c->cache_dtype == KVRING_CACHE_E4M3;
  const cuuint64_t D = (cuuint64_t)c->head_dim, P = (cuuint64_t)c->page_size, esz = e4m3 ? 1 : 2;
  const cuuint64_t dims[3] = {D, P, (cuuint64_t)c->num_layers * c->num_pages * c->num_kv_heads};
  const cuuint64_t strides[2] = {D * esz, P * D * esz};
  const cuuint32_t box[3] = {e4m3 ? (cuuint32_t)D : 64u, P < 128 ? (cuuint32_t)P : 128u, 1u};
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  const CUtensorMapSwizzle sw = e4m3 && D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  return fn(m, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Queries [n][Hq][d] with a token stride, in boxes of 64 columns x the query
// heads of one key/value head x the tokens of a row group (128 rows at most).
bool make_query_map(CUtensorMap* m, const void* q, int64_t stride, int n, const kvring_pages_config& c) {
  auto fn = kvr::encode_tiled();
  if (!fn) return false;
  const int G = c.num_q_heads / c.num_kv_heads;
  const cuuint64_t D = (cuuint64_t)c.head_dim;
  const cuuint64_t dims[3] = {D, (cuuint64_t)c.num_q_heads, (cuuint64_t)n};
  const cuuint64_t strides[2] = {D * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64u, (cuuint32_t)G, (cuuint32_t)(kvr::kTile / G)};
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Launch under the library's record of written caller buffers: the cache's own,
// from which a caller may pass on what a plan made (a ring's attention reads its
// query positions before it waits), and the call's output.
template <typename F>
kvring_status recorded(const kvring_pages* h, cudaStream_t s, F launch, const void* a = nullptr, size_t an = 0) {
  return kvr::launch_recorded(
      s, [](void* ctx) { return (*static_cast<F*>(ctx))(); }, &launch, a, an, h->buf, h->bytes);
}

bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + bn && y < x + an;
}

}  // namespace

extern "C" {

kvring_status kvring_pages_get_layout(const kvring_pages_config* cfg, kvring_pages_layout* out) {
  if (!out) return KVRING_ERR_INVALID_ARG;
  std::memset(out, 0, sizeof *out);
  if (!config_ok(cfg)) return KVRING_ERR_INVALID_ARG;
  *out = plan_for(cfg).pub;
  return KVRING_OK;
}

kvring_status kvring_pages_create(const kvring_pages_config* cfg, void* dev_buf, size_t bytes, void* stream,
                                  kvring_pages_t** out) {
  if (!out) return KVRING_ERR_INVALID_ARG;
  *out = nullptr;
  if (!config_ok(cfg) || !dev_buf || !aligned(dev_buf, kAlign)) return KVRING_ERR_INVALID_ARG;
  const Plan p = plan_for(cfg);
  if (bytes < p.pub.total) return KVRING_ERR_CAPACITY;
  int dev = 0, major = 0, minor = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return KVRING_ERR_CUDA;
  cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (major != 10 || minor != 3) return KVRING_ERR_UNSUPPORTED;   // built for sm_103a only
  cudaPointerAttributes pa;
  if (cudaPointerGetAttributes(&pa, dev_buf) != cudaSuccess || pa.type != cudaMemoryTypeDevice || pa.device != dev)
    return KVRING_ERR_INVALID_ARG;
  kvring_pages* h = new (std::nothrow) kvring_pages();
  if (!h) return KVRING_ERR_INVALID_ARG;
  h->cfg = *cfg;
  h->device = dev;
  h->buf = dev_buf;
  h->bytes = p.pub.total;
  h->sm_count = sms < 1 ? 1 : (sms > kvr::kPagedMaxCtas ? kvr::kPagedMaxCtas : sms);
  h->max_new = cfg->max_tokens;
  h->requests = cfg->max_requests;
  h->wait_ns = kDefaultWaitNs;
  h->debug_stall = 0;
  uint8_t* b = static_cast<uint8_t*>(dev_buf);
  auto ints = [&](size_t off) { return reinterpret_cast<int32_t*>(b + off); };
  kvr::PagesDev& d = h->dev;
  d.k = b + p.pub.k_cache;
  d.v = b + p.pub.v_cache;
  d.scales = reinterpret_cast<float*>(b + p.pub.scales);
  d.lens = ints(p.pub.lengths);
  d.tables = ints(p.pub.tables);
  d.free_pages = ints(p.pub.free_pages);
  d.state = ints(p.pub.state);
  d.rows = ints(p.pub.step_rows);
  d.cu = ints(p.pub.step_cu);
  d.klen = ints(p.pub.step_lengths);
  d.pos = ints(p.pub.positions);
  d.slots = ints(p.pub.slots);
  d.table = reinterpret_cast<const float*>(b + p.table);
  d.part_o = reinterpret_cast<float*>(b + p.part_o);
  d.part_ml = reinterpret_cast<float*>(b + p.part_ml);
  d.tickets = ints(p.tickets);
  d.few_tickets = d.tickets + 2 * kvr::kPagedMaxCtas;
  d.few_o = reinterpret_cast<float*>(b + p.few_o);
  d.few_ml = reinterpret_cast<float*>(b + p.few_ml);
  d.Hq = cfg->num_q_heads;
  d.Hkv = cfg->num_kv_heads;
  d.D = cfg->head_dim;
  d.L = cfg->num_layers;
  d.P = cfg->page_size;
  d.logP = 0;
  while ((1 << d.logP) < d.P) ++d.logP;
  d.num_pages = cfg->num_pages;
  d.R = cfg->max_requests;
  d.W = cfg->max_pages_per_request;
  d.max_tokens = cfg->max_tokens;
  d.e4m3 = cfg->cache_dtype == KVRING_CACHE_E4M3;
  d.halves = cfg->rope_pairing == KVRING_ROPE_HALVES;
  double theta[64] = {};
  for (int i = 0; i < d.D / 2; ++i) theta[i] = std::pow(cfg->rope_base, (-2.0 * i) / (double)d.D);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  kvring_status st = KVRING_OK;
  if (!make_pool_map(&h->tmK, d.k, cfg) || !make_pool_map(&h->tmV, d.v, cfg)) st = KVRING_ERR_UNSUPPORTED;
  if (st == KVRING_OK) st = cuda_status(kvr::pages_prepare());
  if (st == KVRING_OK) st = cuda_status(kvr::paged_few_prepare());
  if (st == KVRING_OK) st = cuda_status(kvr::paged_chunk_prepare());
  // everything but the caches and the workspace's partial rows starts as zeros
  if (st == KVRING_OK) st = cuda_status(cudaMemsetAsync(b + p.pub.scales, 0, p.table - p.pub.scales, s));
  if (st == KVRING_OK) st = cuda_status(cudaMemsetAsync(d.tickets, 0, 3 * kvr::kPagedMaxCtas * 4, s));
  if (st == KVRING_OK)
    st = recorded(h, s, [&] {
      const cudaError_t e = kvr::launch_pages_table(d, reinterpret_cast<float*>(b + p.table), theta, s);
      return e == cudaSuccess ? kvr::launch_pages_reset(d, d.num_pages, true, s) : e;
    });
  if (st == KVRING_OK) st = cuda_status(cudaStreamSynchronize(s));
  if (st != KVRING_OK) {
    delete h;
    return st;
  }
  *out = h;
  return KVRING_OK;
}

kvring_status kvring_pages_destroy(kvring_pages_t* h) {
  delete h;
  return KVRING_OK;
}

kvring_status kvring_pages_restore(kvring_pages_t* h, const int32_t* lengths, const int32_t* tables,
                                   const int32_t* free_pages, int32_t n_free, void* stream) {
  if (!h || !lengths || !tables || (n_free > 0 && !free_pages) || n_free < 0 || n_free > h->cfg.num_pages)
    return KVRING_ERR_INVALID_ARG;
  if (!aligned(lengths, 4) || !aligned(tables, 4) || !aligned(free_pages, 4) || !on_device(h))
    return KVRING_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const kvr::PagesDev& d = h->dev;
  // the cache's own arrays stay where they are; other parts of its buffer would
  // be copied over one another
  struct Copy {
    int32_t* to;
    const int32_t* from;
    size_t bytes;
  } copies[3] = {{d.lens, lengths, (size_t)d.R * 4},
                 {d.tables, tables, (size_t)d.R * d.W * 4},
                 {d.free_pages, free_pages, (size_t)n_free * 4}};
  for (Copy& c : copies) {
    if (c.from == c.to) c.bytes = 0;
    if (c.bytes && overlap(c.from, c.bytes, h->buf, h->bytes)) return KVRING_ERR_INVALID_ARG;
  }
  return recorded(h, s, [&] {
    cudaError_t e = cudaSuccess;
    for (const Copy& c : copies)
      if (e == cudaSuccess && c.bytes) e = cudaMemcpyAsync(c.to, c.from, c.bytes, cudaMemcpyDeviceToDevice, s);
    return e == cudaSuccess ? kvr::launch_pages_reset(d, n_free, false, s) : e;
  });
}

kvring_status kvring_pages_set_scales(kvring_pages_t* h, int32_t layer, const float* sk, const float* sv,
                                      void* stream) {
  if (!h || !sk || !sv || !aligned(sk, 4) || !aligned(sv, 4) || layer < 0 || layer >= h->cfg.num_layers ||
      !on_device(h))
    return KVRING_ERR_INVALID_ARG;
  if (!h->dev.e4m3) return KVRING_ERR_UNSUPPORTED;   // a bf16 cache has no scales
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return recorded(h, s, [&] { return kvr::launch_pages_scales(h->dev, layer, sk, sv, s); });
}

kvring_status kvring_pages_plan(kvring_pages_t* h, const int32_t* rows, const int32_t* new_tokens, int32_t n,
                                int32_t num_tokens, int32_t max_new, void* stream) {
  if (!h || !new_tokens || !aligned(new_tokens, 4) || (rows && !aligned(rows, 4)) || n < 1 || num_tokens < 1 ||
      max_new < 1 || !on_device(h))
    return KVRING_ERR_INVALID_ARG;
  if (n > h->cfg.max_requests || num_tokens > h->cfg.max_tokens) return KVRING_ERR_CAPACITY;
  // what the plan writes while it reads them
  const uint8_t* steps = reinterpret_cast<const uint8_t*>(h->dev.rows);
  const size_t step_bytes = static_cast<const uint8_t*>(h->buf) + h->bytes - steps;
  if (overlap(new_tokens, (size_t)n * 4, steps, step_bytes) || (rows && overlap(rows, (size_t)n * 4, steps, step_bytes)))
    return KVRING_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (max_new > num_tokens) max_new = num_tokens;
  const kvring_status st =
      recorded(h, s, [&] { return kvr::launch_pages_plan(h->dev, rows, new_tokens, n, num_tokens, max_new, s); });
  if (st == KVRING_OK) {
    h->max_new = max_new;
    h->requests = n;
  }
  return st;
}

kvring_status kvring_pages_commit(kvring_pages_t* h, void* stream) {
  if (!h || !on_device(h)) return KVRING_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return recorded(h, s, [&] { return kvr::launch_pages_commit(h->dev, s); });
}

kvring_status kvring_pages_release(kvring_pages_t* h, const int32_t* rows, int32_t n, void* stream) {
  if (!h || !rows || !aligned(rows, 4) || n < 1 || !on_device(h)) return KVRING_ERR_INVALID_ARG;
  if (n > h->cfg.max_requests) return KVRING_ERR_CAPACITY;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return recorded(h, s, [&] { return kvr::launch_pages_release(h->dev, rows, n, s); });
}

kvring_status kvring_pages_write(kvring_pages_t* h, int32_t layer, const void* q, const void* k, const void* v,
                                 int64_t qs, int64_t ks, int64_t vs, const void* qw, const void* kw, float eps,
                                 void* q_out, int32_t n, void* stream) {
  if (!h || !q || !k || !v || !q_out || layer < 0 || layer >= h->cfg.num_layers || n < 1 || !on_device(h))
    return KVRING_ERR_INVALID_ARG;
  const void* ptrs[6] = {q, k, v, q_out, qw, kw};
  for (const void* p : ptrs)
    if (!aligned(p, 16)) return KVRING_ERR_INVALID_ARG;
  const int64_t D = h->cfg.head_dim, qrow = h->cfg.num_q_heads * D, krow = h->cfg.num_kv_heads * D;
  const int64_t most = (int64_t)1 << 40;
  if (qs % 8 || ks % 8 || vs % 8 || qs < qrow || ks < krow || vs < krow || qs > most || ks > most || vs > most)
    return KVRING_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return KVRING_ERR_INVALID_ARG;
  if (n > h->cfg.max_tokens) return KVRING_ERR_CAPACITY;
  const size_t out_bytes = (size_t)n * qrow * 2;
  auto bytes = [&](int64_t stride, int64_t row) { return ((size_t)(n - 1) * stride + row) * 2; };
  if (overlap(q_out, out_bytes, q, bytes(qs, qrow)) || overlap(q_out, out_bytes, k, bytes(ks, krow)) ||
      overlap(q_out, out_bytes, v, bytes(vs, krow)) || overlap(q_out, out_bytes, h->buf, h->bytes))
    return KVRING_ERR_INVALID_ARG;
  for (const void* p : {qw, kw})
    if (p && overlap(q_out, out_bytes, p, (size_t)D * 2)) return KVRING_ERR_INVALID_ARG;
  kvr::PagesWrite w{};
  w.q = static_cast<const uint16_t*>(q);
  w.k = static_cast<const uint16_t*>(k);
  w.v = static_cast<const uint16_t*>(v);
  w.q_stride = qs;
  w.k_stride = ks;
  w.v_stride = vs;
  w.qw = static_cast<const uint16_t*>(qw);
  w.kw = static_cast<const uint16_t*>(kw);
  w.q_out = static_cast<uint16_t*>(q_out);
  w.eps = eps;
  w.T = n;
  w.layer = layer;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return recorded(h, s, [&] { return kvr::launch_pages_write(h->dev, w, h->sm_count, s); }, q_out, out_bytes);
}

kvring_status kvring_pages_attention(kvring_pages_t* h, int32_t layer, const void* q, int64_t q_stride, void* out,
                                     int32_t n, int32_t causal, int32_t window, float scale, void* stream) {
  if (!h || !q || !out || !aligned(q, 16) || !aligned(out, 16) || layer < 0 || layer >= h->cfg.num_layers || n < 1 ||
      !on_device(h))
    return KVRING_ERR_INVALID_ARG;
  const int64_t row = (int64_t)h->cfg.num_q_heads * h->cfg.head_dim;
  if (q_stride % 8 || q_stride < row || q_stride > (int64_t)1 << 40) return KVRING_ERR_INVALID_ARG;
  if ((causal != 0 && causal != 1) || window < 0 || (window > 0 && !causal)) return KVRING_ERR_INVALID_ARG;
  if (!(scale >= 0.f) || !std::isfinite(scale)) return KVRING_ERR_INVALID_ARG;
  if (n > h->cfg.max_tokens) return KVRING_ERR_CAPACITY;
  const size_t out_bytes = (size_t)n * row * 2;
  if (overlap(out, out_bytes, q, ((size_t)(n - 1) * q_stride + row) * 2) || overlap(out, out_bytes, h->buf, h->bytes))
    return KVRING_ERR_INVALID_ARG;
  kvr::PagedAttn a{};
  a.q = static_cast<const uint16_t*>(q);
  a.out = static_cast<uint16_t*>(out);
  a.q_stride = q_stride;
  a.T = n;
  a.layer = layer;
  a.causal = causal;
  a.window = window;
  a.sm_log2 = 1.4426950408889634f * (scale > 0.f ? scale : 1.0f / sqrtf((float)h->cfg.head_dim));
  // (a product that overflows, or underflows to 0, is no factor for a mask)
  if (!std::isfinite(a.sm_log2)) return KVRING_ERR_INVALID_ARG;
  if (a.sm_log2 < 1e-30f) a.sm_log2 = 1e-30f;
  a.ctas = h->sm_count;
  a.wait_ns = h->wait_ns;
  a.debug_stall = h->debug_stall;
  // Which kernel takes a request: up to kFewRows query rows (tokens x G) the
  // one for few rows, beyond that the one for chunks.  One kernel alone when
  // the plan's bound, or its single request, leaves nothing for the other;
  // that one then takes every request, whatever the device's lengths are.
  const int G = h->cfg.num_q_heads / h->cfg.num_kv_heads;
  const int64_t rows = (int64_t)h->max_new * G;
  const bool chunk = rows > kvr::kFewRows, few = !chunk || (h->requests > 1 && G <= kvr::kFewRows);
  CUtensorMap tmQ;
  if (chunk && !make_query_map(&tmQ, q, q_stride, n, h->cfg)) return KVRING_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return recorded(h, s, [&] {
    cudaError_t e = cudaSuccess;
    if (chunk) {
      a.min_rows = few ? kvr::kFewRows : 0;
      a.max_rows = INT32_MAX;
      a.min_tiles = 8;
      e = kvr::launch_paged_chunk(h->dev, &tmQ, &h->tmK, &h->tmV, a, s);
    }
    if (few && e == cudaSuccess) {
      a.min_rows = 0;
      a.max_rows = chunk ? kvr::kFewRows : INT32_MAX;
      a.min_tiles = 2;
      a.beside = chunk;
      e = kvr::launch_paged_few(h->dev, &h->tmK, &h->tmV, a, s);
    }
    return e;
  }, out, out_bytes);
}

kvring_status kvring_pages_debug_set_wait(kvring_pages_t* h, int64_t limit_ns, int32_t stall) {
  if (!h || limit_ns < 1000 || limit_ns > 60000000000ll || (stall != 0 && stall != 1)) return KVRING_ERR_INVALID_ARG;
  h->wait_ns = (unsigned long long)limit_ns;
  h->debug_stall = stall;
  return KVRING_OK;
}

}  // extern "C"
