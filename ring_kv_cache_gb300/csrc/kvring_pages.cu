// The paged cache's step bookkeeping (plan, commit, release) and its write
// (head norms, RoPE, quantisation into the pages).
//
// All kernels wait for the preceding kernel on the stream
// (griddepcontrol.wait) before they read anything, and let the next one
// start right after that.
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

template <int D, bool E4M3, bool HALVES>
__global__ void __launch_bounds__(kWriteWarps * 32, 8)
    k_pages_write(const PagesDev p, const PagesWrite w) {
  constexpr int LPR = D / 8, TPW = 32 / LPR;
  const int lane = threadIdx.x & 31, c = lane % LPR;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0);   // (uniform, and known to be)
  const int t = blockIdx.x * TPW + lane / LPR;
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
  if (hk0 < p.Hkv) load_kv(hk0);
  int tokens = __ldcg(p.state + PST_TOKENS);
  int slot = mine ? __ldcg(p.slots + t) : -1;
  int pos = mine ? __ldcg(p.pos + t) : 0;
  const uint4 one = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);   // bf16 ones
  const uint4 gq = w.qw ? load(w.qw) : one, gk = w.kw ? load(w.kw) : one;
  tokens = tokens < w.T ? tokens : w.T;
  if (blockIdx.x * TPW >= tokens) return;
  const bool valid = t < tokens;
  if (!valid) {
    slot = -1;
    pos = 0;
  }
  const float4 cs0 = __ldg(reinterpret_cast<const float4*>(p.table + (size_t)pos * D + 8 * c));
  const float4 cs1 = __ldg(reinterpret_cast<const float4*>(p.table + (size_t)pos * D + 8 * c + 4));
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
  const size_t n = (size_t)p.W * p.P * (p.D / 2);
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

cudaError_t launch_pages_write(const PagesDev& p, const PagesWrite& w, int sm_count, cudaStream_t s) {
  const int tpw = 32 / (p.D / 8), blocks = (w.T + tpw - 1) / tpw;
  const int htot = p.Hq + 2 * p.Hkv, most = (htot + kWriteWarps - 1) / kWriteWarps;
  // few tokens: split the heads over blocks too, until every SM has the eight
  // blocks that it holds
  int split = (8 * sm_count + blocks - 1) / blocks;
  split = split < 1 ? 1 : (split > most ? most : split);
  const dim3 grid((unsigned)blocks, (unsigned)split), block(kWriteWarps * 32);
  auto go = [&](auto kernel) { return launch_pdl(kernel, grid, block, 0, s, p, w); };
  if (p.D == 128) {
    if (p.e4m3) return p.halves ? go(k_pages_write<128, true, true>) : go(k_pages_write<128, true, false>);
    return p.halves ? go(k_pages_write<128, false, true>) : go(k_pages_write<128, false, false>);
  }
  if (p.e4m3) return p.halves ? go(k_pages_write<64, true, true>) : go(k_pages_write<64, true, false>);
  return p.halves ? go(k_pages_write<64, false, true>) : go(k_pages_write<64, false, false>);
}

}  // namespace kvr
