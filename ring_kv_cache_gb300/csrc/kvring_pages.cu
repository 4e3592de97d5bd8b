// The paged cache's step bookkeeping (plan, commit, release) and its write
// (head norms, RoPE, quantisation into the pages).
//
// All kernels wait for the preceding kernel on the stream
// (griddepcontrol.wait) before they read anything, and let the next one
// start right after that.
#include <type_traits>

#include "kvring_pages.cuh"

namespace kvr {
namespace {

constexpr int kPlanThreads = 512;

__device__ __forceinline__ void set_error(const PagesDev& p, unsigned bits) {
  atomicOr(reinterpret_cast<unsigned*>(p.state + PST_ERROR), bits);
}

// Exclusive block scan of one 64-bit value per thread (blockDim.x a multiple
// of 32, at most 1024); *total gets the sum.  `ws` holds 33 words.
__device__ __forceinline__ unsigned long long block_scan(unsigned long long v, unsigned long long* ws,
                                                         unsigned long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  unsigned long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) ws[warp] = x;
  __syncthreads();
  if (warp == 0) {
    unsigned long long s = lane < nw ? ws[lane] : 0ull;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xFFFFFFFFu, s, o);
      if (lane >= o) s += y;
    }
    ws[lane] = s;
  }
  __syncthreads();
  *total = ws[nw - 1];
  const unsigned long long before = warp ? ws[warp - 1] : 0ull;
  __syncthreads();
  return before + x - v;
}

// Last index i of [0, n) with a[i] <= x (a ascending, a[0] <= x).
__device__ __forceinline__ int last_at_most(const int32_t* a, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// ------------------------------------------------------------------ plan ---
// Every block makes the sums over all requests for itself (a few thousand
// words at most, in one pass with one block scan of tokens and pages packed
// in 64 bits), so no block waits for another and the plan is one launch; a
// block then writes its share of the token maps and of the table entries.
// Bound by latency: 4.5 us for 48 requests and as many tokens, 6.7 us for 1,000
// requests with 65,536 tokens (0.6 MB).
// Tokens take 34 bits (4,096 requests x 2^20 tokens), pages 30.
constexpr int kTokBits = 34;

__global__ void __launch_bounds__(kPlanThreads)
    k_pages_plan(const PagesDev p, const int32_t* rows, const int32_t* nt, int B, int T, int max_new) {
  extern __shared__ int32_t sm_plan[];
  __shared__ unsigned long long ws[33];
  __shared__ unsigned s_err;
  int32_t* s_len = sm_plan;
  int32_t* s_row = s_len + B;
  int32_t* s_cu = s_row + B;          // [B + 1]
  int32_t* s_off = s_cu + B + 1;      // [B + 1]
  unsigned* s_seen = reinterpret_cast<unsigned*>(s_off + B + 1);   // [ceil(R / 32)]
  for (int i = threadIdx.x; i < (p.R + 31) / 32; i += kPlanThreads) s_seen[i] = 0u;
  if (threadIdx.x == 0) s_err = 0u;
  griddep_wait();
  griddep_launch_dependents();
  __syncthreads();
  int nfree = __ldcg(p.state + PST_FREE);
  unsigned long long carry = 0;
  for (int base = 0; base < B; base += kPlanThreads) {
    const int i = base + threadIdx.x;
    unsigned long long v = 0;
    if (i < B) {
      int row = rows ? __ldcg(rows + i) : i;
      int n = __ldcg(nt + i);
      unsigned err = 0;
      int len = 0;
      if (row < 0 || row >= p.R) {
        err |= KVRING_PAGES_ERR_ROW;
        row = -1;
      } else {
        if (atomicOr(s_seen + (row >> 5), 1u << (row & 31)) & (1u << (row & 31))) err |= KVRING_PAGES_ERR_ROW;
        len = __ldcg(p.lens + row);
        if (len < 0) {
          err |= KVRING_PAGES_ERR_LENGTH;
          len = 0;
        }
      }
      if (n < 0 || n > max_new || n > T) {
        err |= KVRING_PAGES_ERR_TOKENS;
        n = 0;
      }
      if ((long long)len + n > (long long)p.W * p.P) err |= KVRING_PAGES_ERR_LENGTH;
      if (err) {
        atomicOr(&s_err, err);
        n = 0;
      }
      const int pages = ((len + n + p.P - 1) >> p.logP) - ((len + p.P - 1) >> p.logP);
      v = (unsigned long long)n | ((unsigned long long)pages << kTokBits);
      s_len[i] = len;
      s_row[i] = row;
    }
    unsigned long long total;
    const unsigned long long at = carry + block_scan(v, ws, &total);
    if (i < B) {
      // (a sum beyond 31 bits is one beyond T: refused below)
      s_cu[i] = (int32_t)(at & 0x7FFFFFFFull);
      s_off[i] = (int32_t)(at >> kTokBits);
    }
    carry += total;
  }
  const unsigned long long tokens64 = carry & ((1ull << kTokBits) - 1);
  const int taken = (int)(carry >> kTokBits);
  nfree = nfree < 0 ? 0 : (nfree > p.num_pages ? p.num_pages : nfree);
  if (threadIdx.x == 0) {
    s_cu[B] = (int32_t)(tokens64 & 0x7FFFFFFFull);
    s_off[B] = taken;
    if (tokens64 > (unsigned long long)T) s_err |= KVRING_PAGES_ERR_TOKENS;
    if (taken > nfree) s_err |= KVRING_PAGES_ERR_PAGES;
  }
  __syncthreads();
  const bool bad = s_err != 0u;
  const int tokens = bad ? 0 : (int)tokens64;
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i < B; i += kPlanThreads) {
      p.rows[i] = s_row[i];
      p.cu[i] = bad ? 0 : s_cu[i];
      p.klen[i] = bad ? s_len[i] : s_len[i] + s_cu[i + 1] - s_cu[i];
    }
    // (only an attention whose waits gave up leaves tickets behind)
    for (int i = threadIdx.x; i < 3 * kPagedMaxCtas; i += kPlanThreads) p.tickets[i] = 0;
    if (threadIdx.x == 0) {
      p.cu[B] = tokens;
      p.state[PST_PLANNED] = 1;
      p.state[PST_REQUESTS] = bad ? 0 : B;
      p.state[PST_TOKENS] = tokens;
      p.state[PST_TAKEN] = bad ? 0 : taken;
      if (bad) set_error(p, s_err);
    }
  }
  auto page_ok = [&](int id) { return id >= 0 && id < p.num_pages; };
  const int nthreads = gridDim.x * kPlanThreads, tid = blockIdx.x * kPlanThreads + threadIdx.x;
  if (!bad) {
    for (int j = tid; j < taken; j += nthreads) {
      const int b = last_at_most(s_off, B, j);
      const int w = ((s_len[b] + p.P - 1) >> p.logP) + (j - s_off[b]);
      const int id = __ldcg(p.free_pages + nfree - 1 - j);
      if (!page_ok(id)) set_error(p, KVRING_PAGES_ERR_TABLE);
      p.tables[(size_t)s_row[b] * p.W + w] = page_ok(id) ? id : -1;
    }
  }
  // token maps, four tokens per thread
  for (int t0 = 4 * tid; t0 < T; t0 += 4 * nthreads) {
    int pos[4], slot[4];
    int b = t0 < tokens ? last_at_most(s_cu, B, t0) : B, w_last = -1, id = -1;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int t = t0 + e;
      pos[e] = 0;
      slot[e] = -1;
      if (t < tokens) {
        while (t >= s_cu[b + 1]) {
          ++b;
          w_last = -1;
        }
        pos[e] = s_len[b] + t - s_cu[b];
        const int w = pos[e] >> p.logP;
        if (w != w_last) {
          const int have = (s_len[b] + p.P - 1) >> p.logP;
          id = w < have ? __ldcg(p.tables + (size_t)s_row[b] * p.W + w)
                        : __ldcg(p.free_pages + nfree - 1 - (s_off[b] + w - have));
          if (!page_ok(id)) {
            set_error(p, KVRING_PAGES_ERR_TABLE);
            id = -1;
          }
          w_last = w;
        }
        if (id >= 0) slot[e] = (id << p.logP) + (pos[e] & (p.P - 1));
      }
    }
    if (t0 + 4 <= T) {
      *reinterpret_cast<int4*>(p.pos + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      *reinterpret_cast<int4*>(p.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (t0 + e < T) {
          p.pos[t0 + e] = pos[e];
          p.slots[t0 + e] = slot[e];
        }
    }
  }
}

__global__ void __launch_bounds__(kPlanThreads) k_pages_commit(const PagesDev p) {
  griddep_wait();
  griddep_launch_dependents();
  const int planned = __ldcg(p.state + PST_PLANNED), B = __ldcg(p.state + PST_REQUESTS);
  const int nfree = __ldcg(p.state + PST_FREE), taken = __ldcg(p.state + PST_TAKEN);
  __syncthreads();
  if (!planned) {
    if (threadIdx.x == 0) set_error(p, KVRING_PAGES_ERR_COMMIT);
    return;
  }
  for (int i = threadIdx.x; i < B; i += kPlanThreads) p.lens[__ldcg(p.rows + i)] = __ldcg(p.klen + i);
  if (threadIdx.x == 0) {
    p.state[PST_FREE] = nfree - taken;
    p.state[PST_PLANNED] = 0;
  }
}

// Ends requests.  A page id that the pool does not have is reported and not put
// back: on the stack it would go to the next request.
__global__ void __launch_bounds__(kPlanThreads) k_pages_release(const PagesDev p, const int32_t* rows, int B) {
  extern __shared__ int32_t sm_plan[];
  __shared__ unsigned long long ws[33];
  __shared__ unsigned s_err;
  int32_t* s_row = sm_plan;
  int32_t* s_n = s_row + B;     // [B] pages of each row
  int32_t* s_off = s_n + B;     // [B] those that go back, then the sums before
  unsigned* s_seen = reinterpret_cast<unsigned*>(s_off + B);
  for (int i = threadIdx.x; i < (p.R + 31) / 32; i += kPlanThreads) s_seen[i] = 0u;
  if (threadIdx.x == 0) s_err = 0u;
  griddep_wait();
  griddep_launch_dependents();
  __syncthreads();
  for (int i = threadIdx.x; i < B; i += kPlanThreads) {
    const int row = __ldcg(rows + i);
    int n = 0;
    if (row < 0 || row >= p.R || (atomicOr(s_seen + (row >> 5), 1u << (row & 31)) & (1u << (row & 31)))) {
      atomicOr(&s_err, KVRING_PAGES_ERR_ROW);
    } else {
      const int len = __ldcg(p.lens + row);
      if (len < 0 || (long long)len > (long long)p.W * p.P) atomicOr(&s_err, KVRING_PAGES_ERR_LENGTH);
      else n = (len + p.P - 1) >> p.logP;
    }
    s_row[i] = row;
    s_n[i] = n;
  }
  __syncthreads();
  const int lane = threadIdx.x & 31;
  auto page_ok = [&](int id) { return id >= 0 && id < p.num_pages; };
  // one warp per request, a lane per table entry
  unsigned foreign = 0;
  for (int b = threadIdx.x >> 5; b < B; b += kPlanThreads / 32) {
    const int n = s_n[b];
    int back = 0;
    for (int w = lane; w - lane < n; w += 32) {
      const bool ok = w < n && page_ok(__ldcg(p.tables + (size_t)s_row[b] * p.W + w));
      if (w < n && !ok) foreign = KVRING_PAGES_ERR_TABLE;
      back += __popc(__ballot_sync(0xFFFFFFFFu, ok));
    }
    if (lane == 0) s_off[b] = back;
  }
  __syncthreads();
  unsigned long long carry = 0;
  for (int base = 0; base < B; base += kPlanThreads) {
    const int i = base + threadIdx.x;
    unsigned long long total;
    const unsigned long long at = carry + block_scan(i < B ? (unsigned long long)s_off[i] : 0ull, ws, &total);
    if (i < B) s_off[i] = (int32_t)at;
    carry += total;
  }
  const int nfree = __ldcg(p.state + PST_FREE);
  if (threadIdx.x == 0) {
    // more pages than the pool holds: the tables are not this cache's
    if (nfree < 0 || (unsigned long long)nfree + carry > (unsigned long long)p.num_pages)
      s_err |= KVRING_PAGES_ERR_PAGES;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    p.state[PST_PLANNED] = 0;
    p.state[PST_REQUESTS] = 0;
    p.state[PST_TOKENS] = 0;
    p.state[PST_TAKEN] = 0;
    if (s_err) set_error(p, s_err);
    else p.state[PST_FREE] = nfree + (int)carry;
  }
  if (s_err) return;
  if (foreign) set_error(p, foreign);
  for (int b = threadIdx.x >> 5; b < B; b += kPlanThreads / 32) {
    const int n = s_n[b];
    int32_t* row = p.tables + (size_t)s_row[b] * p.W;
    int32_t* to = p.free_pages + nfree + s_off[b];
    for (int w = lane; w - lane < n; w += 32) {
      const int id = w < n ? __ldcg(row + w) : -1;
      const unsigned back = __ballot_sync(0xFFFFFFFFu, page_ok(id));
      if (page_ok(id)) to[__popc(back & ((1u << lane) - 1))] = id;
      if (w < n) row[w] = -1;
      to += __popc(back);
    }
    if (lane == 0) p.lens[s_row[b]] = 0;
  }
}

// The state words after create (fill: every page free, rows empty) or
// restore (the free list and tables have been copied in).
__global__ void k_pages_reset(const PagesDev p, int n_free, int fill) {
  griddep_wait();
  const size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x, n = (size_t)gridDim.x * blockDim.x;
  if (fill) {
    for (size_t k = i; k < (size_t)p.num_pages; k += n) p.free_pages[k] = p.num_pages - 1 - (int)k;
    for (size_t k = i; k < (size_t)p.R * p.W; k += n) p.tables[k] = -1;
    for (size_t k = i; k < (size_t)p.L * 4 * p.Hkv; k += n) p.scales[k] = 1.0f;
  }
  if (i < PST_WORDS_ALLOC && (fill || i != PST_ERROR)) p.state[i] = i == PST_FREE ? n_free : 0;
}

__global__ void k_pages_scales(const PagesDev p, int layer, const float* sk, const float* sv) {
  griddep_wait();
  griddep_launch_dependents();
  float* dst = p.scales + (size_t)layer * 4 * p.Hkv;
  for (int h = threadIdx.x; h < p.Hkv; h += blockDim.x) {
    const float k = __ldcg(sk + h), v = __ldcg(sv + h);   // (past L1, as everywhere: see the write)
    dst[h] = k;
    dst[p.Hkv + h] = v;
    dst[2 * p.Hkv + h] = 1.0f / k;
    dst[3 * p.Hkv + h] = 1.0f / v;
  }
}

struct Thetas {
  double t[64];
};
// cos and sin of position * theta_i in 64 bits, rounded once.
__global__ void k_pages_table(float* table, const Thetas th, int half, size_t n) {
  for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (size_t)gridDim.x * blockDim.x) {
    double s, c;
    sincos((double)(i / half) * th.t[i % half], &s, &c);
    reinterpret_cast<float2*>(table)[i] = make_float2((float)c, (float)s);
  }
}

// --------------------------------------------------------- 3-D positions ---
__device__ __forceinline__ bool coords_ok(const PagesDev& p, const int (&xyz)[3]) {
  const unsigned n = (unsigned)p.max_pos;
  return (unsigned)xyz[0] < n && (unsigned)xyz[1] < n && (unsigned)xyz[2] < n;
}
// cos and sin of a pair, from the row of its section's coordinate.
template <int D>
__device__ __forceinline__ float2 turn_of(const PagesDev& p, const int (&xyz)[3], int pair) {
  const int row = pair < p.pt ? xyz[0] : (pair < p.pt + p.py ? xyz[1] : xyz[2]);
  return __ldg(reinterpret_cast<const float2*>(p.table) + (size_t)row * (D / 2) + pair);
}

// ----------------------------------------------------------------- write ---
// y = x rsqrt(mean x^2 + eps) w, rotated; one rounding at the end.  Bound by
// HBM: each bf16 head row is read once and its result written once.
//
// D/8 lanes hold a head row, 8 values each, so the sum of squares is a
// shuffle reduction; a lane's values are four whole rotation pairs in either
// pairing (adjacent: one 16-byte chunk; halves: 8 bytes of each half), so the
// rotation needs no exchange and both pairings read the same 32 bytes of the
// cos/sin row.  Norm weight and rotation make one 2 x 2 matrix per pair,
// r (x0 w0 c - x1 w1 s, x0 w0 s + x1 w1 c), formed once per token for the
// queries and once for the keys and kept for all heads: with the weights
// applied separately the kernel was bound by issuing instructions (153 per
// warp and head row).  A block takes the tokens of one warp (2 or 4) and its
// four warps walk the heads; loads of a batch of heads go out together,
// those of the first batch and of the first key and value before anything
// else is known.  Measured (GB300): 16,384 tokens, 32/8 heads x 128, bf16 cache,
// 411 MB: 65.2 us, 6.3 TB/s (93 % of the copy rate); 757 tokens of 40 heads into
// an E4M3 cache, 39 MB: 8.5 us; nine tokens: 1.9 us.
// Blocks of four warps with batches of four, eight on an SM: eight warps with
// batches of two take 73.5 us (a finished warp's place stays empty until the
// block's last is done), two warps with batches of four 66.8 us.
constexpr int kWriteWarps = 4;
constexpr int kWriteBatch = 4;

// AXES: 3-D positions: each pair's cos and sin from the row of its own coordinate,
// once per token.  KV false: the queries alone, of the kernel that writes blocks with
// scales.  bx: the block of tokens.
template <int D, bool E4M3, bool HALVES, bool AXES, bool KV>
__device__ __forceinline__ void write_tokens(const PagesDev& p, const PagesWrite& w, const int bx) {
  constexpr int LPR = D / 8, TPW = 32 / LPR;
  const int lane = threadIdx.x & 31, c = lane % LPR;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0);   // (uniform, and known to be)
  const int t = bx * TPW + lane / LPR;
  const int e0 = HALVES ? 4 * c : 8 * c;            // the lane's first 4 values
  const int e1 = HALVES ? D / 2 + 4 * c : 8 * c + 4;
  const bool mine = t < w.T;
  const int gw = blockIdx.y * kWriteWarps + warp, step = kWriteWarps * gridDim.y;
  auto widen = [](uint4 v, float (&x)[8]) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  };
  // (past L1: the rows may have been written by a kernel that still ran when
  // this one started)
  auto load = [&](const uint16_t* row) -> uint4 {
    if constexpr (HALVES) {
      const uint2 a = __ldcg(reinterpret_cast<const uint2*>(row + e0));
      const uint2 b = __ldcg(reinterpret_cast<const uint2*>(row + e1));
      return make_uint4(a.x, a.y, b.x, b.y);
    } else {
      return __ldcg(reinterpret_cast<const uint4*>(row + e0));
    }
  };
  const uint16_t* q = w.q + (mine ? (long long)t * w.q_stride : 0);
  const uint16_t* k = w.k + (mine ? (long long)t * w.k_stride : 0);
  const uint16_t* v = w.v + (mine ? (long long)t * w.v_stride : 0);
  const float* inv = p.scales + ((size_t)w.layer * 4 + 2) * p.Hkv;
  uint4 raw[kWriteBatch], kraw, vraw;
  float inv_k = 1.0f, inv_v = 1.0f;
  auto load_q = [&](int h0) {
#pragma unroll
    for (int i = 0; i < kWriteBatch; ++i)
      if (h0 + i * step < p.Hq) raw[i] = load(q + (h0 + i * step) * D);
  };
  auto load_kv = [&](int h) {
    kraw = load(k + h * D);
    vraw = load(v + h * D);
    if constexpr (E4M3) {
      inv_k = __ldcg(inv + h);
      inv_v = __ldcg(inv + p.Hkv + h);
    }
  };
  griddep_wait();
  griddep_launch_dependents();
  // Everything that depends on nothing else is asked for at once; only the
  // cos/sin row waits, for the position.  Key/value heads are dealt out from
  // the other end, so that warps without a query head take them first.
  const int hk0 = step - 1 - gw;
  load_q(gw);
  if constexpr (KV) {
    if (hk0 < p.Hkv) load_kv(hk0);
  }
  int tokens = __ldcg(p.state + PST_TOKENS);
  int slot = mine ? __ldcg(p.slots + t) : -1;
  int pos = mine && !AXES ? __ldcg(p.pos + t) : 0;
  int xyz[3] = {0, 0, 0};
  if constexpr (AXES) {
    if (mine) {
#pragma unroll
      for (int i = 0; i < 3; ++i) xyz[i] = __ldcg(w.coords + 3 * (size_t)t + i);
    }
  }
  const uint4 one = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);   // bf16 ones
  const uint4 gq = w.qw ? load(w.qw) : one, gk = w.kw ? load(w.kw) : one;
  tokens = tokens < w.T ? tokens : w.T;
  if (bx * TPW >= tokens) return;
  bool valid = t < tokens;
  if (!valid) {
    slot = -1;
    pos = 0;
  }
  float4 cs0, cs1;
  if constexpr (!AXES) {
    cs0 = __ldg(reinterpret_cast<const float4*>(p.table + (size_t)pos * D + 8 * c));
    cs1 = __ldg(reinterpret_cast<const float4*>(p.table + (size_t)pos * D + 8 * c + 4));
  } else {
    if (!coords_ok(p, xyz)) {
      if (valid) set_error(p, KVRING_PAGES_ERR_POSITION);
      valid = false;
      slot = -1;
      xyz[0] = xyz[1] = xyz[2] = 0;
    }
    float2 cs[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) cs[e] = turn_of<D>(p, xyz, 4 * c + e);
    cs0 = make_float4(cs[0].x, cs[0].y, cs[1].x, cs[1].y);
    cs1 = make_float4(cs[2].x, cs[2].y, cs[3].x, cs[3].y);
  }
  // pair e: values lo(e), hi(e) of the lane's eight
  auto lo = [](int e) { return HALVES ? e : 2 * e; };
  auto hi = [](int e) { return HALVES ? 4 + e : 2 * e + 1; };
  float m[4][4];
  auto matrix = [&](uint4 g4) {
    float g[8];
    widen(g4, g);
    const float cc[4] = {cs0.x, cs0.z, cs1.x, cs1.z}, ss[4] = {cs0.y, cs0.w, cs1.y, cs1.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      m[e][0] = g[lo(e)] * cc[e];
      m[e][1] = -g[hi(e)] * ss[e];
      m[e][2] = g[lo(e)] * ss[e];
      m[e][3] = g[hi(e)] * cc[e];
    }
  };
  auto turn = [&](uint4 r4, bool norm, float (&x)[8]) {
    widen(r4, x);
    float r = 1.0f;
    if (norm) {
      float sq = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sq = fmaf(x[e], x[e], sq);
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) sq += __shfl_xor_sync(0xFFFFFFFFu, sq, o);
      r = rsqrtf(sq * (1.0f / D) + w.eps);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = x[lo(e)] * r, b = x[hi(e)] * r;   // (scaled first: huge rows stay finite)
      x[lo(e)] = a * m[e][0] + b * m[e][1];
      x[hi(e)] = a * m[e][2] + b * m[e][3];
    }
  };
  auto store_bf16 = [&](uint16_t* dst, const float (&x)[8]) {
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat162 b2 = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
      o[e] = *reinterpret_cast<const uint32_t*>(&b2);
    }
    if constexpr (HALVES) {
      *reinterpret_cast<uint2*>(dst + e0) = make_uint2(o[0], o[1]);
      *reinterpret_cast<uint2*>(dst + e1) = make_uint2(o[2], o[3]);
    } else {
      *reinterpret_cast<uint4*>(dst + e0) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  };
  auto store_cache = [&](uint8_t* cache, size_t row, const float (&x)[8], float s) {
    if constexpr (E4M3) {
      const uint32_t a = f32x2_to_e4m3x2(x[0] * s, x[1] * s) | ((uint32_t)f32x2_to_e4m3x2(x[2] * s, x[3] * s) << 16);
      const uint32_t b = f32x2_to_e4m3x2(x[4] * s, x[5] * s) | ((uint32_t)f32x2_to_e4m3x2(x[6] * s, x[7] * s) << 16);
      uint8_t* dst = cache + row * D;
      if constexpr (HALVES) {
        *reinterpret_cast<uint32_t*>(dst + e0) = a;
        *reinterpret_cast<uint32_t*>(dst + e1) = b;
      } else {
        *reinterpret_cast<uint2*>(dst + e0) = make_uint2(a, b);
      }
    } else {
      store_bf16(reinterpret_cast<uint16_t*>(cache) + row * D, x);
    }
  };
  matrix(gq);
  uint16_t* q_out = w.q_out + (size_t)t * p.Hq * D;
  for (int h0 = gw; h0 < p.Hq; h0 += kWriteBatch * step) {
    if (h0 != gw) load_q(h0);
#pragma unroll
    for (int i = 0; i < kWriteBatch; ++i) {
      const int h = h0 + i * step;
      if (h >= p.Hq) break;   // (the same for the whole warp)
      float x[8];
      turn(raw[i], w.qw != nullptr, x);
      if (valid) store_bf16(q_out + h * D, x);
    }
  }
  if constexpr (!KV) return;
  if (hk0 >= p.Hkv) return;
  matrix(gk);
  // row of (page, head 0, offset) in the layer's caches; heads are P rows apart
  const size_t row0 =
      (((size_t)w.layer * p.num_pages + (slot >> p.logP)) * p.Hkv << p.logP) + (slot & (p.P - 1));
  for (int h = hk0; h < p.Hkv; h += step) {
    if (h != hk0) load_kv(h);
    float x[8];
    turn(kraw, w.kw != nullptr, x);
    const size_t row = row0 + ((size_t)h << p.logP);
    if (slot >= 0) store_cache(p.k, row, x, inv_k);
    widen(vraw, x);
    if (slot >= 0) store_cache(p.v, row, x, inv_v);
  }
}

template <int D, bool E4M3, bool HALVES, bool AXES>
__global__ void __launch_bounds__(kWriteWarps * 32, 8) k_pages_write(const PagesDev p, const PagesWrite w) {
  write_tokens<D, E4M3, HALVES, AXES, true>(p, w, blockIdx.x);
}

// ------------------------------------------- write into blocks with scales ---
// Keys and values into an E4M3 cache whose blocks of 16 tokens have a scale
// 2^e each:  e = least with amax <= 448 2^e over the step's tokens of the block,
// not below the block's so far where it holds tokens; those are then rounded
// again, code * 2^(e_old - e_new).  Powers of two, so that neither a value's
// division by its scale nor a code's move to a larger one rounds, but for the one
// rounding to E4M3's step (a code that has moved loses bits only among the
// subnormals): a scale of amax / 448 itself would use the top binade better by less than
// one step in 16 and round every code again with each growth.
//
// Bound by HBM as the write above, and by issue.  A run is the step's tokens with
// consecutive slots of one block; four warps hold a run's rows, four each, and a
// head's keys and values, until their sizes are known, so each value is read
// once, and a block's codes leave as whole lines.  Runs begin anywhere, so a
// group of 16 consecutive tokens of the step owns those that begin in it: up to
// 16 runs (single tokens) and up to 31 tokens, of which the first 16 and a last
// run of up to 16 make two turns at most (mostly one).  Sizes of rows are
// exchanged through shared memory, one barrier per turn and head; every warp takes the
// maximum over the runs by shuffles, a lane per row of keys and of values.
// cos/sin rows of the group's tokens lie in shared memory for the block's heads.  Blocks that
// take the queries (the write's code above) lie between those of keys and values.
// Measured (GB300): 16,384 tokens, 32/8 heads x 128, 377 MB: 70.7 us, 5.3 TB/s; 757 tokens of
// 40 heads 12.8 us (1.26 waves), 48 single tokens of 10 heads 3.3 us, with half of their blocks
// moved to larger scales by each call 7 us.  (A warp for a whole run, 64 values a thread and 168
// registers: 80, 16.2 and, no block moved, 7.2 us; queries by warps of that shape as well 111, 19.0
// and 7.6 us.)
constexpr int kBlockWarps = kWriteWarps;
constexpr int kBlocksPerSm = 7;   // (16,384 tokens: 82, 75.7, 70.7, 69.9 us with 5, 6, 7, 8)
constexpr int kBlockHeads = 2;    // of a block of keys and values (77 us, 78 with four, 82 with one, all at six blocks)

__device__ __forceinline__ int block_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u);   // 448 = 1.75 x 2^8
  return min(max(e, kMinExp), kMaxExp);
}
__device__ __forceinline__ float power(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }   // 2^e

template <int D, bool HALVES, bool AXES>
__global__ void __launch_bounds__(kBlockWarps * 32, kBlocksPerSm) k_pages_write_blocks(const PagesDev p, const PagesWrite w) {
  constexpr int B = KVRING_SCALE_BLOCK;
  // Blocks of queries and of keys and values in turn, as many of the former as 16
  // tokens take, so that the one's arithmetic runs beside the other's copies.
  constexpr int kQueries = B / (32 / (D / 8));
  const int per = w.kv_blocks + kQueries, group = blockIdx.x / per, unit = blockIdx.x % per;
  if (unit >= w.kv_blocks) {
    write_tokens<D, false, HALVES, AXES, false>(p, w, group * kQueries + unit - w.kv_blocks);
    return;
  }
  static_assert(B == 16, "a turn is one block");
  constexpr int LPR = D / 8, TPW = 32 / LPR;         // lanes of a row, rows of a warp's access
  constexpr int RPW = B / kBlockWarps, IT = RPW / TPW;   // rows of a warp, accesses for them
  constexpr int kOld = 15 * 16 / kBlockWarps;        // a warp's share of what blocks may have held before
  __shared__ __align__(16) float s_cs[32][D];        // cos, sin of the window's tokens
  __shared__ float s_max[2][2][B];                   // sizes of rows, of keys and values, two turns in turn
  __shared__ uint32_t s_old[kBlockWarps][kOld];      // rows of the layer's cache to be rounded again
  __shared__ uint8_t s_run[kBlockWarps][kOld];       // and the first row of the run that they are of
  const int lane = threadIdx.x & 31, c = lane % LPR, sub = lane / LPR;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0);
  const int e0 = HALVES ? 4 * c : 8 * c, e1 = HALVES ? D / 2 + 4 * c : 8 * c + 4;
  griddep_wait();
  griddep_launch_dependents();
  // The window: lane i looks at token 16 g - 1 + i.
  const int t_lane = group * B - 1 + lane;
  int tokens = __ldcg(p.state + PST_TOKENS);
  int slot = t_lane >= 0 && t_lane < w.T ? __ldcg(p.slots + t_lane) : -1;
  tokens = tokens < w.T ? tokens : w.T;
  if (t_lane >= tokens) slot = -1;
  const int prev = __shfl_up_sync(0xFFFFFFFFu, slot, 1);
  const bool follows = lane > 0 && slot >= 0 && slot == prev + 1 && (slot & (B - 1)) != 0;
  const unsigned cont = __ballot_sync(0xFFFFFFFFu, follows);
  const unsigned lead = __ballot_sync(0xFFFFFFFFu, slot >= 0 && !follows) & 0x1FFFEu;
  if (lead == 0) return;   // (the same in every warp)
  const int f = __ffs(lead) - 1, last = 31 - __clz(lead);
  // end of the last run: the first lane behind `last` that does not follow
  const unsigned stops = ~cont & ~((2u << last) - 1);
  const int end = stops ? __ffs(stops) - 1 : 32;
  // lanes that belong to a run of this group
  const unsigned members = (lead | cont) & (0xFFFFFFFFu << f) & (end == 32 ? 0xFFFFFFFFu : (1u << end) - 1);
  const bool member = members >> lane & 1u;
  bool stored = member;
  // cos and sin of the members' tokens
  int at[3] = {0, 0, 0};
  if (member) {
    if constexpr (AXES) {
#pragma unroll
      for (int i = 0; i < 3; ++i) at[i] = __ldcg(w.coords + 3 * (size_t)t_lane + i);
      if (!coords_ok(p, at)) {
        set_error(p, KVRING_PAGES_ERR_POSITION);
        stored = false;
        at[0] = at[1] = at[2] = 0;
      }
    } else {
      at[0] = __ldcg(p.pos + t_lane);
    }
  }
  const unsigned store_mask = __ballot_sync(0xFFFFFFFFu, stored);
  auto widen = [](uint4 v, float (&x)[8]) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  };
  auto load = [&](const uint16_t* row) -> uint4 {
    if constexpr (HALVES) {
      const uint2 a = __ldcg(reinterpret_cast<const uint2*>(row + e0));
      const uint2 b = __ldcg(reinterpret_cast<const uint2*>(row + e1));
      return make_uint4(a.x, a.y, b.x, b.y);
    } else {
      return __ldcg(reinterpret_cast<const uint4*>(row + e0));
    }
  };
  // The rows of a turn, `base` its first lane: whole runs, at most 16.
  auto rows_of = [&](int base) { return end - base > 16 ? last - base : end - base; };
  const int row0 = warp * RPW + sub;                 // this lane's rows of a turn: row0 + i * TPW
  uint4 kr[IT], vr[IT];
  auto fetch = [&](int h, int base) {
    const unsigned live = (store_mask >> base) & ((1u << rows_of(base)) - 1);
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int r = row0 + i * TPW;
      kr[i] = vr[i] = make_uint4(0u, 0u, 0u, 0u);
      if (live >> r & 1u) {
        const long long t = (long long)group * B - 1 + base + r;
        kr[i] = load(w.k + t * w.k_stride + h * D);
        vr[i] = load(w.v + t * w.v_stride + h * D);
      }
    }
  };
  int h = unit * gridDim.y + blockIdx.y, base = f;
  const int step = w.kv_blocks * gridDim.y;
  if (h < p.Hkv) fetch(h, base);
  {
    constexpr int kRows = 32 / kBlockWarps, kPart = D / 64;   // rows of a warp, pairs of a lane
    float2 v[kRows][kPart];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int i = f + j * kBlockWarps + warp;
      const int xyz[3] = {__shfl_sync(0xFFFFFFFFu, at[0], i & 31), __shfl_sync(0xFFFFFFFFu, at[1], i & 31),
                          __shfl_sync(0xFFFFFFFFu, at[2], i & 31)};
      if (i < end) {
#pragma unroll
        for (int k = 0; k < kPart; ++k)
          v[j][k] = AXES ? turn_of<D>(p, xyz, lane + 32 * k)
                         : __ldg(reinterpret_cast<const float2*>(p.table) + (size_t)xyz[0] * (D / 2) + lane + 32 * k);
      }
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int i = f + j * kBlockWarps + warp;
      if (i < end) {
#pragma unroll
        for (int k = 0; k < kPart; ++k) reinterpret_cast<float2*>(s_cs[i])[lane + 32 * k] = v[j][k];
      }
    }
  }
  float gk[8];
  if (w.kw) {
    widen(load(w.kw), gk);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) gk[e] = 1.0f;
  }
  const size_t layer0 = (size_t)w.layer * p.num_pages * p.Hkv << p.logP;   // the layer's first row of the cache
  // row [page][head 0][offset] of this lane's token
  const uint32_t row_lane =
      member ? ((uint32_t)(slot >> p.logP) * (uint32_t)p.Hkv << p.logP) + (uint32_t)(slot & (p.P - 1)) : 0u;
  __syncthreads();
  auto size_of = [&](const float (&x)[8]) {          // of a row, in all its lanes
    float m = 0.f;                                   // (a maximum passes over NaN)
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[e]));
    if (m == INFINITY) {                             // of the others
      m = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[e]) < INFINITY ? fabsf(x[e]) : 0.f);
    }
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    return m;
  };
  auto size_of_bf16 = [&](uint4 v) {                 // the same of a row as it came
    const uint32_t u[4] = {v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu, v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu};
    uint32_t m2 = __vmaxu2(__vmaxu2(u[0], u[1]), __vmaxu2(u[2], u[3]));
    uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
    if (m >= 0x7F80u) {
      m = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t y = u[e >> 1] >> (16 * (e & 1)) & 0xFFFFu;
        m = max(m, y < 0x7F80u ? y : 0u);
      }
    }
    float f = __uint_as_float(m << 16);
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) f = fmaxf(f, __shfl_xor_sync(0xFFFFFFFFu, f, o));
    return f;
  };
  int place = 0;
  while (h < p.Hkv) {
    const int n = rows_of(base);
    const unsigned here = (members >> base) & ((1u << n) - 1);
    const unsigned firsts = (lead >> base) & here, live = (store_mask >> base) & here;
    // Lanes r and 16 + r: row r of the turn, of keys and of values; its run's first row
    // and the row behind its last.
    const int r = lane & 15;
    const uint32_t row_r = __shfl_sync(0xFFFFFFFFu, row_lane, (base + r) & 31) + ((uint32_t)h << p.logP);
    const int slot_r = __shfl_sync(0xFFFFFFFFu, slot, (base + r) & 31);
    const unsigned upto = firsts & ((2u << r) - 1), behind = (firsts | ~here) & ~((2u << r) - 1);
    const int from = upto ? 31 - __clz(upto) : 0;
    const int to = __ffs(behind) - 1;                // (here has at most 16 bits: there is one)
    const int held = (slot_r & (B - 1)) - (r - from);   // tokens the block held before
    uint8_t* scale = (lane < 16 ? p.ks : p.vs) + ((layer0 + row_r) >> 4);
    int old = 0;
    if ((here >> r & 1u) && held > 0) old = __ldcg(scale);
    float x[IT][8];
    uint4 values[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int k = row0 + i * TPW;
      const float mv = size_of_bf16(vr[i]);
      values[i] = vr[i];
      widen(kr[i], x[i]);
      float rs = 1.0f;
      if (w.kw) {
        float sq = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) sq = fmaf(x[i][e], x[i][e], sq);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) sq += __shfl_xor_sync(0xFFFFFFFFu, sq, o);
        rs = rsqrtf(sq * (1.0f / D) + w.eps);
      }
      const float* cs = s_cs[(base + k) & 31] + 8 * c;
      const float4 a = *reinterpret_cast<const float4*>(cs), b = *reinterpret_cast<const float4*>(cs + 4);
      const float cc[4] = {a.x, a.z, b.x, b.z}, ss[4] = {a.y, a.w, b.y, b.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int lo = HALVES ? e : 2 * e, hi = HALVES ? 4 + e : 2 * e + 1;
        const float u = x[i][lo] * rs * gk[lo], v = x[i][hi] * rs * gk[hi];   // (scaled first: huge rows stay finite)
        x[i][lo] = u * cc[e] - v * ss[e];
        x[i][hi] = u * ss[e] + v * cc[e];
      }
      const float mk = size_of(x[i]);                // (of anything in a row that is none)
      if (c == 0) {
        const bool is = live >> k & 1u;
        s_max[place][0][k] = is ? mk : 0.f;
        s_max[place][1][k] = is ? mv : 0.f;
      }
    }
    // the next turn's values, or the next head's, on their way
    const bool more = base + n < end;
    const int h_next = more ? h : h + step, base_next = more ? base + n : f;
    if (h_next < p.Hkv) fetch(h_next, base_next);
    __syncthreads();
    // maximum over the run: up to its last row, then back from there
    float m = s_max[place][lane >> 4][r];
    place ^= 1;
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) {
      const float y = __shfl_up_sync(0xFFFFFFFFu, m, o, 16);
      if (r - o >= from) m = fmaxf(m, y);
    }
    m = __shfl_sync(0xFFFFFFFFu, m, to - 1, 16);
    old = min(max(old, kMinExp), kMaxExp);
    const int need = block_exponent(m), exp = held > 0 ? max(need, old) : need;
    const float inv = power(127 - exp);              // 2^-(exp - 127)
    const bool first = (here >> r & 1u) && r == from;
    // (a run of skipped tokens alone leaves its block's scale, as its codes)
    if (warp == 0 && first && (live >> from & ((1u << (to - from)) - 1))) *scale = (uint8_t)exp;
    uint8_t *kc = p.k + layer0 * D, *vc = p.v + layer0 * D;
    auto store = [&](uint8_t* dst, const float (&y)[8], float s) {
      const uint32_t a = f32x2_to_e4m3x2(y[0] * s, y[1] * s) | ((uint32_t)f32x2_to_e4m3x2(y[2] * s, y[3] * s) << 16);
      const uint32_t b = f32x2_to_e4m3x2(y[4] * s, y[5] * s) | ((uint32_t)f32x2_to_e4m3x2(y[6] * s, y[7] * s) << 16);
      if constexpr (HALVES) {
        *reinterpret_cast<uint32_t*>(dst + e0) = a;
        *reinterpret_cast<uint32_t*>(dst + e1) = b;
      } else {
        *reinterpret_cast<uint2*>(dst + e0) = make_uint2(a, b);
      }
    };
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int k = row0 + i * TPW;
      const float sk = __shfl_sync(0xFFFFFFFFu, inv, k), sv = __shfl_sync(0xFFFFFFFFu, inv, 16 + k);
      const size_t row = (size_t)__shfl_sync(0xFFFFFFFFu, row_r, k) * D;
      if (live >> k & 1u) {
        store(kc + row, x[i], sk);
        widen(values[i], x[i]);
        store(vc + row, x[i], sv);
      }
    }
    // Tokens from before in blocks that move to a larger scale: every warp takes
    // every fourth row, its share in a list, so that they are on their way at once.
    const unsigned grown = __ballot_sync(0xFFFFFFFFu, first && held > 0 && exp > old);
    const float ratio = power(old - exp);
    for (int kind = 0; kind < 2; ++kind) {
      if ((grown >> (16 * kind) & 0xFFFFu) == 0) continue;
      const int mine = grown >> (16 * kind + r) & 1u ? held : 0;   // (both halves of the warp alike)
      int sum = mine;
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, sum, o, 16);
        if (r >= o) sum += y;
      }
      const int total = __shfl_sync(0xFFFFFFFFu, sum, 15);
      __syncwarp();
      if (lane < 16) {
        for (int i = 0; i < mine; ++i) {
          const int k = sum - mine + i;
          if (k % kBlockWarps == warp) {
            s_old[warp][k / kBlockWarps] = row_r - held + i;
            s_run[warp][k / kBlockWarps] = (uint8_t)r;
          }
        }
      }
      __syncwarp();
      const int count = (total - warp + kBlockWarps - 1) / kBlockWarps;
      uint8_t* cache = kind ? vc : kc;
      constexpr int G = 4;                           // accesses on their way
#pragma unroll 1
      for (int i0 = 0; i0 < count; i0 += G * TPW) {
        uint2 v[G];
#pragma unroll
        for (int i = 0; i < G; ++i) {
          const int k = i0 + i * TPW + sub;
          if (k < count) v[i] = __ldcg(reinterpret_cast<const uint2*>(cache + (size_t)s_old[warp][k] * D) + c);
        }
#pragma unroll
        for (int i = 0; i < G; ++i) {
          const int k = i0 + i * TPW + sub;
          const float s = __shfl_sync(0xFFFFFFFFu, ratio, 16 * kind + (k < count ? s_run[warp][k] : 0));
          if (k >= count) continue;
          uint32_t o[2];
          const uint32_t in[2] = {v[i].x, v[i].y};
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 lo = e4m3x2_to_f32x2((uint16_t)in[e]), hi = e4m3x2_to_f32x2((uint16_t)(in[e] >> 16));
            o[e] = f32x2_to_e4m3x2(lo.x * s, lo.y * s) | ((uint32_t)f32x2_to_e4m3x2(hi.x * s, hi.y * s) << 16);
          }
          reinterpret_cast<uint2*>(cache + (size_t)s_old[warp][k] * D)[c] = make_uint2(o[0], o[1]);
        }
      }
    }
    h = h_next;
    base = base_next;
  }
}

size_t plan_smem(const PagesDev& p, int B) { return (size_t)(4 * B + 2) * 4 + (size_t)((p.R + 31) / 32) * 4; }

}  // namespace

cudaError_t pages_prepare() {
  const int most = (4 * kMaxRows + 2) * 4 + kMaxRows / 8;
  cudaError_t e = cudaFuncSetAttribute(k_pages_plan, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(k_pages_release, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  return e;
}

cudaError_t launch_pages_table(const PagesDev& p, float* table, const double* theta, cudaStream_t s) {
  Thetas th{};
  for (int i = 0; i < p.D / 2; ++i) th.t[i] = theta[i];
  const size_t n = (size_t)p.max_pos * (p.D / 2);
  const size_t blocks = (n + 255) / 256;
  k_pages_table<<<(unsigned)(blocks < 4096 ? blocks : 4096), 256, 0, s>>>(table, th, p.D / 2, n);
  return cudaGetLastError();
}

cudaError_t launch_pages_reset(const PagesDev& p, int n_free, bool fill, cudaStream_t s) {
  return launch_pdl(k_pages_reset, dim3(fill ? 256 : 1), dim3(256), 0, s, p, n_free, fill ? 1 : 0);
}

cudaError_t launch_pages_scales(const PagesDev& p, int layer, const float* sk, const float* sv, cudaStream_t s) {
  return launch_pdl(k_pages_scales, dim3(1), dim3(256), 0, s, p, layer, sk, sv);
}

cudaError_t launch_pages_plan(const PagesDev& p, const int32_t* rows, const int32_t* nt, int B, int T, int max_new,
                              cudaStream_t s) {
  const int blocks = (T + 4 * kPlanThreads - 1) / (4 * kPlanThreads);
  return launch_pdl(k_pages_plan, dim3(blocks < 1 ? 1 : (blocks > 64 ? 64 : blocks)), dim3(kPlanThreads),
                    plan_smem(p, B), s, p, rows, nt, B, T, max_new);
}

cudaError_t launch_pages_commit(const PagesDev& p, cudaStream_t s) {
  return launch_pdl(k_pages_commit, dim3(1), dim3(kPlanThreads), 0, s, p);
}

cudaError_t launch_pages_release(const PagesDev& p, const int32_t* rows, int B, cudaStream_t s) {
  return launch_pdl(k_pages_release, dim3(1), dim3(kPlanThreads), plan_smem(p, B), s, p, rows, B);
}

static cudaError_t launch_write_blocks(const PagesDev& p, PagesWrite w, int sm_count, cudaStream_t s) {
  const int groups = (w.T + KVRING_SCALE_BLOCK - 1) / KVRING_SCALE_BLOCK;
  w.kv_blocks = (p.Hkv + kBlockHeads - 1) / kBlockHeads;
  const int blocks = groups * (w.kv_blocks + KVRING_SCALE_BLOCK / (256 / p.D));
  // few tokens: split the heads over blocks too, until every SM has what it holds
  const int heads = (p.Hq + kWriteWarps - 1) / kWriteWarps, most = heads > kBlockHeads ? heads : kBlockHeads;
  int split = (kBlocksPerSm * sm_count + blocks - 1) / blocks;
  split = split < 1 ? 1 : (split > most ? most : split);
  const dim3 grid((unsigned)blocks, (unsigned)split), block(kBlockWarps * 32);
  auto go = [&](auto kernel) { return launch_pdl(kernel, grid, block, 0, s, p, w); };
  if (p.D == 128) {
    if (p.pt) return p.halves ? go(k_pages_write_blocks<128, true, true>) : go(k_pages_write_blocks<128, false, true>);
    return p.halves ? go(k_pages_write_blocks<128, true, false>) : go(k_pages_write_blocks<128, false, false>);
  }
  if (p.pt) return p.halves ? go(k_pages_write_blocks<64, true, true>) : go(k_pages_write_blocks<64, false, true>);
  return p.halves ? go(k_pages_write_blocks<64, true, false>) : go(k_pages_write_blocks<64, false, false>);
}

cudaError_t launch_pages_write(const PagesDev& p, const PagesWrite& w, int sm_count, cudaStream_t s) {
  if (p.ks) return launch_write_blocks(p, w, sm_count, s);
  const int tpw = 32 / (p.D / 8), blocks = (w.T + tpw - 1) / tpw;
  const int htot = p.Hq + 2 * p.Hkv, most = (htot + kWriteWarps - 1) / kWriteWarps;
  // few tokens: split the heads over blocks too, until every SM has the eight
  // blocks that it holds
  int split = (8 * sm_count + blocks - 1) / blocks;
  split = split < 1 ? 1 : (split > most ? most : split);
  const dim3 grid((unsigned)blocks, (unsigned)split), block(kWriteWarps * 32);
  auto go = [&](auto kernel) { return launch_pdl(kernel, grid, block, 0, s, p, w); };
  // a kernel by head size, pairing and positions
  auto pick = [&](auto e4m3) {
    constexpr bool E = decltype(e4m3)::value;
    if (p.D == 128) {
      if (p.pt) return p.halves ? go(k_pages_write<128, E, true, true>) : go(k_pages_write<128, E, false, true>);
      return p.halves ? go(k_pages_write<128, E, true, false>) : go(k_pages_write<128, E, false, false>);
    }
    if (p.pt) return p.halves ? go(k_pages_write<64, E, true, true>) : go(k_pages_write<64, E, false, true>);
    return p.halves ? go(k_pages_write<64, E, true, false>) : go(k_pages_write<64, E, false, false>);
  };
  return p.e4m3 ? pick(std::true_type{}) : pick(std::false_type{});
}

}  // namespace kvr
