// Attention over the paged cache for requests with few query rows: single
// tokens, drafts, short chunks (up to 16 rows a unit, a row being one query
// head of one token).
//
//   out[r] = sum_j softmax_j(s_rj) V[j],  s_rj = scale q[r] . K[j]
// by one pass over the keys with a running maximum m and sum l per row
// (log2 units): m' = max(m, max_j s_rj), p = 2^(s - m'),
// l' = l 2^(m - m') + sum p, O' = O 2^(m - m') + p V.
//
// Bound by HBM: every cached key and value of the request is read once per
// key/value head (all its query heads share the tile), and with at most 16
// rows the arithmetic is a small part of the tensor rate.  So the design is
// about keeping copies in flight: one CTA per SM whose producer warp streams
// page pieces by TMA into a ring of shared-memory slots (about 190 KB), and
// about evenness: the (request, row tile, key/value head, 128-token tile)
// space is flattened and cut into equal contiguous ranges, one per CTA, from
// the lengths on the device, so ragged batches and a single long request
// both load every SM alike.  A unit (request, row tile, head) that lies in
// several ranges leaves partial (m, l, O) in the workspace; the last CTA to
// arrive (one ticket per unit) merges the parts in range order, so results
// do not depend on arrival.
//
// The matrix products use mma.sync (m16n8k16): with 16 rows a tile of
// 128 tokens needs 32 instructions per warp, far from any limit, and a
// register fragment lets the row tile be 16 high where tcgen05 has 64 or
// 128 rows.  Each warp takes 16 of a tile's tokens through both
// products with a running (m, l, O) of its own: the score fragment is the
// probability operand as it stands, and nothing is exchanged between warps
// before the unit's end, where their states are merged in shared memory.
// (With the columns of O split over the warps instead, and the probabilities
// passed through shared memory, two barriers per tile bounded the kernel over
// an E4M3 cache: 310 MB in 88 us.)
//
// E4M3 tiles are read as 16-bit pairs by ldmatrix and widened in registers
// to f16, exactly.  For the scores four consecutive bytes of a key become
// the pair (k, k+1) and (k+8, k+9) of a k = 16 step, so the queries are
// stored with that permutation of each 16 columns.  For the values the
// transposed load gives two tokens x two columns; a byte permute makes the
// token pairs, the even columns forming one n = 8 tile and the odd ones the
// other.  Queries become f16 after scaling each row by a power of two into
// [1, 2) at its largest value: bf16's 8 significant bits fit f16's 11, and
// what the row's small values lose is below 2^-25 of its largest.
//
// Measured (GB300): 128 decoding requests of 7,000 tokens on average, 32/8
// heads x 128, bf16, 3.67 GB: 544 us, 6.75 TB/s (the copy rate is 6.80); the
// same in E4M3 321 us, 5.7 TB/s, bound by the latency of each warp's chain of
// widening and products; six requests of up to 32,000 tokens in pages of 16, 10 heads, E4M3,
// four tokens each, 310 MB: 65 us (61 us in pages of 64); one request of 700
// tokens: 10 us, latency.
#include "kvring_pages.cuh"


namespace kvr {
namespace {

constexpr int kGroups = 8;       // groups of 16 tokens of a tile
constexpr int kRows = kFewRows;  // query rows of a unit
constexpr int kSmemMost = 232448;

template <int D, bool E4M3>
struct FewLayout {
  // Consumer warps.  They take the 16-token groups in turn.  Eight keep up
  // with HBM over a bf16 cache; an E4M3 tile is there in half the time and
  // takes more instructions (1.83 GB: 370 us with 8 warps, 354 with 11, 381
  // with 15, which leaves them 128 registers).
  static constexpr int kWarps = E4M3 ? 11 : 8;
  static constexpr int kConsumers = kWarps * 32;
  static constexpr int kThreads = kConsumers + 32;
  static constexpr int kSlot = kTile * D * (E4M3 ? 1 : 2); // one K or V tile
  static constexpr int kQ = 0;                             // offsets behind the slots
  static constexpr int kO = kQ + kRows * D * 2;               // float [warps][4 rows][D]: the merge of the warps
  static constexpr int kMl = kO + kWarps * 4 * D * 4;      // float2 [warps][kRows]: their offsets and sums
  static constexpr int kRow = kMl + kWarps * kRows * 8;       // int lo, hi; float factor; pad: [kRows][4]
  static constexpr int kMisc = kRow + kRows * 16;
  static constexpr int kFixed = kMisc + 512;
  static constexpr int kRoom = (kSmemMost - 1024 - kFixed) / kSlot;
  static constexpr int kSlots = kRoom > 16 ? 16 : kRoom;
  static constexpr int kBytes = 1024 + kSlots * kSlot + kFixed;
  static_assert(kSlots >= 4, "two tiles in flight");
};

// What a unit of a request needs to know.
struct Req {
  int q0, nq, klen;    // first token, tokens (that the tensors hold), length
  int pos0;            // position of the first token
  int nrows, nrt;      // query rows, row tiles
  int lo, hi;          // tokens any row sees: [lo, hi)
  int t0, nt;          // their tiles
  int row;             // of the block tables
};

struct FewMisc {
  uint64_t full[16];
  uint64_t empty[16];
  unsigned long long ws[16];
  long long total;
  long long base;    // tiles before the request the CTA starts in
  Req rq;            // that request
  int b0;
  int parts;         // CTAs that have a range
  int abort;
  int last;
};

// Keeps the accumulator type of the two element types in one place.
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm2t(uint32_t (&r)[2], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr) : "memory");
}
template <int N>
__device__ __forceinline__ void sync_consumers_n() {
  asm volatile("bar.sync 1, %0;" ::"n"(N) : "memory");
}

// The words of the step that describe request b.
struct ReqWords {
  int q0, end, klen, row;
};
__device__ __forceinline__ ReqWords load_words(const PagesDev& p, int b) {
  return ReqWords{__ldcg(p.cu + b), __ldcg(p.cu + b + 1), __ldcg(p.klen + b), __ldcg(p.rows + b)};
}

__device__ __forceinline__ Req make_req(const PagedAttn& a, const ReqWords& w, int G) {
  Req r;
  r.q0 = w.q0;
  r.row = w.row;
  r.klen = w.klen;
  r.pos0 = r.klen - (w.end - r.q0);
  r.nq = (w.end < a.T ? w.end : a.T) - r.q0;
  if (r.nq < 0) r.nq = 0;
  r.nrows = r.nq * G;
  const long long all = (long long)(w.end - r.q0) * G;
  if (all <= a.min_rows || all > a.max_rows || r.klen <= 0) r.nrows = 0;
  r.nrt = (r.nrows + kRows - 1) / kRows;
  r.hi = r.klen;
  r.lo = 0;
  if (a.window > 0) {
    const int lo = r.pos0 + 1 - a.window;
    r.lo = lo > 0 ? lo : 0;
  }
  r.t0 = r.lo / kTile;
  r.nt = r.nrows ? (r.hi + kTile - 1) / kTile - r.t0 : 0;
  return r;
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(FewLayout<D, E4M3>::kThreads, 1)
    k_paged_few(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const PagesDev p,
                const PagedAttn a) {
  using L = FewLayout<D, E4M3>;
  constexpr int kWarps = L::kWarps, kConsumers = L::kConsumers, kFewThreads = L::kThreads;
  auto sync_consumers = [] { sync_consumers_n<kConsumers>(); };
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(sm);
  uint8_t* fix = sm + L::kSlots * L::kSlot;
  const uint32_t fbase = sbase + L::kSlots * L::kSlot;
  FewMisc* misc = reinterpret_cast<FewMisc*>(fix + L::kMisc);
  volatile int* abort = &misc->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.Hq / p.Hkv;
  auto full = [&](int s) { return smem_u32(&misc->full[s]); };
  auto empty = [&](int s) { return smem_u32(&misc->empty[s]); };
  if (threadIdx.x == 0) {
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
    for (int s = 0; s < L::kSlots; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), kWarps);   // every consumer warp, those without a group of the tile too
    }
    misc->abort = 0;
    mbar_fence_init();
  }
  // Behind the chunk kernel of the same call this one starts as soon as that
  // kernel has seen its own predecessors done, works beside it (on other
  // requests, with tickets and workspace of its own) and waits for it at the
  // end, so that what follows waits for both.
  if (!a.beside) griddep_wait();
  griddep_launch_dependents();

  // ------------------------------------------------- this CTA's range
  // Each thread sums the tiles (of one head) of its requests, then one block
  // scan.  The words of the first requests are asked for together with the
  // request count (the arrays are max_requests long).
  const ReqWords ahead = load_words(p, (int)threadIdx.x < p.R ? threadIdx.x : 0);
  const int B = __ldcg(p.state + PST_REQUESTS);
  {
    const int per = (B + kFewThreads - 1) / kFewThreads;
    const int i0 = threadIdx.x * per, i1 = i0 + per < B ? i0 + per : B;
    auto req_of = [&](int i) { return make_req(a, per == 1 ? ahead : load_words(p, i), G); };
    unsigned long long mine = 0;
    for (int i = i0; i < i1; ++i) {
      const Req r = req_of(i);
      mine += (unsigned long long)r.nrt * (unsigned)r.nt;
    }
    unsigned long long x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) misc->ws[warp] = x;
    __syncthreads();
    unsigned long long before = 0, total = 0;
    for (int w = 0; w < kFewThreads / 32; ++w) {
      if (w < warp) before += misc->ws[w];
      total += misc->ws[w];
    }
    total *= (unsigned)p.Hkv;
    before = (before + x - mine) * (unsigned)p.Hkv;
    mine *= (unsigned)p.Hkv;
    // as many ranges as there are CTAs, unless they would be shorter than
    // min_tiles: below that a range's start-up and the merge cost more
    unsigned long long parts = total / (unsigned)a.min_tiles;
    parts = parts < 1 ? 1 : (parts > gridDim.x ? gridDim.x : parts);
    const unsigned long long start = blockIdx.x < parts ? total * blockIdx.x / parts : total;
    if (mine && start >= before && start < before + mine) {   // exactly one thread, unless total is 0
      int i = i0;
      for (; i < i1; ++i) {
        misc->rq = req_of(i);
        const unsigned long long n = (unsigned long long)misc->rq.nrt * (unsigned)misc->rq.nt * (unsigned)p.Hkv;
        if (start < before + n) break;
        before += n;
      }
      misc->b0 = i;
      misc->base = (long long)before;
    }
    if (threadIdx.x == 0) {
      misc->total = (long long)total;
      misc->parts = (int)parts;
    }
    __syncthreads();
  }
  const long long total = misc->total;
  const long long parts = misc->parts;
  const long long start = total * blockIdx.x / parts, stop = total * (blockIdx.x + 1) / parts;
  if (blockIdx.x >= parts || start >= stop) {
    if (a.beside) griddep_wait();
    return;
  }

  // The walk over units, the same in the producer and the consumers.
  int b = misc->b0;
  Req rq = misc->rq;
  long long x = start;                       // next tile of the flattened space
  long long ubase;                           // first tile of the current unit
  int rt, h;
  {
    const long long in_b = start - misc->base;
    const int u = (int)(in_b / rq.nt);
    rt = u / p.Hkv;
    h = u % p.Hkv;
    ubase = misc->base + (long long)u * rq.nt;
  }
  auto next_unit = [&]() {                   // x has reached the unit's end
    ubase += rq.nt;
    if (++h < p.Hkv) return;
    h = 0;
    if (++rt < rq.nrt) return;
    rt = 0;
    do rq = make_req(a, load_words(p, ++b), G);
    while (rq.nt == 0);                      // (some request follows: x < stop)
  };

  if (warp == kWarps) {
    // --------------------------------------------------------- producer
    const int box_rows = p.P < kTile ? p.P : kTile;
    const int nbox = kTile / box_rows;       // page pieces of a tile
    constexpr int kHalves = E4M3 ? 1 : D / 64;   // 64-column atoms of a bf16 tile
    const uint32_t box_bytes = (uint32_t)(box_rows * (E4M3 ? D : 128));
    const long long layer0 = (long long)a.layer * p.num_pages;
    const int none = p.L * p.num_pages * p.Hkv;   // past the map: reads as zeros
    int n = 0;                               // slots filled so far
    bool stopped = a.debug_stall;            // a wait gave up (or test support: nothing is copied)
    while (x < stop && !stopped) {
      long long ue = ubase + rq.nt;
      const int32_t* tab = p.tables + (size_t)rq.row * p.W;
      ue = ue < stop ? ue : stop;
      // A lane per page piece (8 at most), kind and 64-column half reads its
      // page id, a tile ahead, and waits for its slot.  With small pages it is
      // the copies' issue that takes the time (16 of 2 KB, one kind after the
      // other from 8 lanes, held a 16-token-page E4M3 cache to 4.3 TB/s).  Where
      // a piece is one copy the elected thread issues them all: lanes move
      // their operands to uniform registers in turn (128 decoding requests, E4M3
      // in 16-token pages: 346 -> 331 us; d = 64 in bf16: 296 -> 293 us).  Where
      // it is two, the lanes do (d = 128 in bf16: 543 us, 548 from one thread).
      const int box = lane & 7, kv = (lane >> 3) & 1, hf = lane >> 4;
      int tile = rq.t0 + (int)(x - ubase);
      auto page_of = [&](int t) -> int {
        const int tok = t * kTile + box * box_rows;
        if (box >= nbox || hf >= kHalves || tok >= rq.hi || tok + box_rows <= rq.lo) return -2;   // nothing any row sees
        return __ldcg(tab + (tok >> p.logP));
      };
      int page = page_of(tile);
      for (; x < ue; ++x, ++tile, n += 2) {
        const int ahead = x + 1 < ue ? page_of(tile + 1) : -2;
        const unsigned there = __ballot_sync(0xFFFFFFFFu, page != -2) & 0xFFu;
        const int row0 = (tile * kTile + box * box_rows) & (p.P - 1);
        const bool ok = page >= 0 && page < p.num_pages;
        if (page != -2 && !ok) atomicOr(reinterpret_cast<unsigned*>(p.state + PST_ERROR), KVRING_PAGES_ERR_TABLE);
        const int c2 = ok ? (int)((layer0 + page) * p.Hkv + h) : none;
        const int mine = n + kv, s = mine % L::kSlots;
        stopped = !__all_sync(0xFFFFFFFFu, mbar_wait_bounded(empty(s), ((mine / L::kSlots) & 1) ^ 1, abort, a.wait_ns));
        if (stopped) break;
        if constexpr (kHalves == 1) {
          int c2s[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) c2s[i] = __shfl_sync(0xFFFFFFFFu, c2, i);
          const int row_0 = __shfl_sync(0xFFFFFFFFu, row0, 0);   // (of the others 0: whole pages)
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int sk = (n + k) % L::kSlots;
              mbar_arrive_expect_tx(full(sk), (uint32_t)__popc(there) * box_bytes);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (there >> i & 1)
                  tma_load_3d(sbase + sk * L::kSlot + i * box_bytes, k ? &tmV : &tmK, 0, i == 0 ? row_0 : 0, c2s[i],
                              full(sk));
            }
          }
          __syncwarp();
        } else {
          if (box == 0 && hf == 0) mbar_arrive_expect_tx(full(s), (uint32_t)__popc(there) * kHalves * box_bytes);
          __syncwarp();
          if (page != -2)
            tma_load_3d(sbase + s * L::kSlot + hf * (kTile * 128) + box * box_bytes, kv ? &tmV : &tmK, hf * 64, row0, c2,
                        full(s));
        }
        page = ahead;
      }
      if (x < stop && !stopped) next_unit();
    }
    // every copy lands before the CTA may exit
    volatile int none_aborted = 0;
    for (int i = n - L::kSlots < 0 ? 0 : n - L::kSlots; i < n; ++i)
      mbar_wait_bounded(full(i % L::kSlots), (i / L::kSlots) & 1, &none_aborted, a.wait_ns);
    if (a.beside) griddep_wait();
    return;
  }

  // ----------------------------------------------------------- consumers
  // A wait that gives up raises the abort flag; from then on nobody waits
  // and the rest of the range runs through on whatever the slots hold, so
  // every barrier is still met and every ticket still drawn.
  int s = 0;                                            // the next slot, and its barrier's phase
  uint32_t phase = 0;
  auto wait_full = [&]() {
    if (!mbar_try_wait(full(s), phase) && !*abort) mbar_wait_bounded(full(s), phase, abort, a.wait_ns);
  };
  auto next_slot = [&]() {
    if (++s == L::kSlots) {
      s = 0;
      phase ^= 1u;
    }
  };
  // The slot back to the producer: behind this warp's reads of it, with the fence
  // between them and the next copy, which is of the other proxy.
  auto give_back = [&]() {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(empty(s));
    next_slot();
  };
  const int g = lane >> 2, c = lane & 3;
  float* s_o = reinterpret_cast<float*>(fix + L::kO);
  float2* s_ml = reinterpret_cast<float2*>(fix + L::kMl);
  int4* s_row = reinterpret_cast<int4*>(fix + L::kRow);
  const uint32_t sQ = fbase + L::kQ;
  const float* sc = p.scales + (size_t)a.layer * 4 * p.Hkv;
  constexpr int kChunksQ = D / 8;                       // 16-byte chunks of a query row
  auto load_q = [&](int ks, uint32_t (&qa)[4]) {
    const int r = lane & 15;
    ldsm4(qa, sQ + r * (D * 2) + (((2 * ks + (lane >> 4)) ^ (r & 7)) << 4));
  };
  auto pack = [](float lo, float hi) {
    if constexpr (E4M3) {
      return f32x2_to_f16x2(lo, hi);
    } else {
      const __nv_bfloat162 b2 = __floats2bfloat162_rn(lo, hi);
      return *reinterpret_cast<const uint32_t*>(&b2);
    }
  };
  auto bf2 = [](float lo, float hi) {
    const __nv_bfloat162 b2 = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b2);
  };
  while (x < stop) {
    const long long uend = ubase + rq.nt;
    const long long ue = uend < stop ? uend : stop;
    const int r0 = rt * kRows;
    const int rows = rq.nrows - r0 < kRows ? rq.nrows - r0 : kRows;
    // ---- queries and row data into shared memory
    sync_consumers();                                    // the previous unit is done with it
    const float scale_k = E4M3 ? __ldcg(sc + h) : 1.0f;
    for (int i = threadIdx.x; i < kRows * kChunksQ; i += kConsumers) {
      const int r = i / kChunksQ, ch = i % kChunksQ;
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows) {
        const int row = r0 + r, tok = rq.q0 + row / G, head = h * G + row % G;
        w = __ldcg(reinterpret_cast<const uint4*>(a.q + (long long)tok * a.q_stride + (size_t)head * D) + ch);
      }
      float fac = a.sm_log2;
      if constexpr (E4M3) {
        // the row's largest exponent, over the lanes that hold the row
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
        uint32_t em = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) em = max(em, max((u[e] >> 7) & 0xFFu, (u[e] >> 23) & 0xFFu));
#pragma unroll
        for (int o = kChunksQ / 2; o > 0; o >>= 1) em = max(em, __shfl_xor_sync(0xFFFFFFFFu, em, o));
        float up, down;
        query_factor(em, up, down);
        // (at least 1e-30: a factor that underflows would make NaN of what is
        // masked, and such scores are all alike anyway)
        fac = fmaxf(fac * scale_k * up, 1e-30f);
        uint32_t hq[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          hq[e] = f32x2_to_f16x2(__uint_as_float(u[e] << 16) * down, __uint_as_float(u[e] & 0xFFFF0000u) * down);
        // columns 8 (ch & 1) + 0..7 of a group of 16: pair (4j, 4j+1) to place
        // 2j, pair (4j+2, 4j+3) to place 2j + 8
        const uint32_t rowb = sQ + r * (D * 2);
        const int j0 = 2 * (ch & 1), cb = ch & ~1;
        auto put = [&](int place, uint32_t v) {          // place: even column of the 16
          const int k = cb + (place >> 3);
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(rowb + ((uint32_t)(k ^ (r & 7)) << 4) + (place & 7) * 2), "r"(v)
                       : "memory");
        };
        put(2 * j0, hq[0]);
        put(2 * j0 + 8, hq[1]);
        put(2 * j0 + 2, hq[2]);
        put(2 * j0 + 10, hq[3]);
      } else {
        *reinterpret_cast<uint4*>(fix + L::kQ + r * (D * 2) + ((ch ^ (r & 7)) << 4)) = w;
      }
      if (ch == 0) {
        int lo = 0, hi = 0;
        if (r < rows) {
          const int pos = rq.pos0 + (r0 + r) / G;
          hi = a.causal ? pos + 1 : rq.klen;
          lo = a.window > 0 && pos + 1 - a.window > 0 ? pos + 1 - a.window : 0;
        }
        s_row[r] = make_int4(lo, hi, __float_as_int(fac), 0);
      }
    }
    sync_consumers();
    uint32_t qreg[D / 16][4];
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) load_q(ks, qreg[ks]);
    float m_run[2], l_run[2], fac[2];                    // offsets, sums, factors of rows g and 8 + g
    float acc[D / 8][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      m_run[i] = -INFINITY;
      l_run[i] = 0.f;
      fac[i] = __int_as_float(s_row[8 * i + g].z);
    }
#pragma unroll
    for (int k = 0; k < D / 8; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[k][e] = 0.f;
    // tokens that every row of the unit sees: tiles inside need no mask
    const int all_hi = s_row[0].y, all_lo = s_row[rows - 1].x;

    int group = warp;                                    // this warp's group of the tile, if below kGroups
    for (int tile = rq.t0 + (int)(x - ubase); x < ue; ++x, ++tile, group += group < kGroups ? kWarps - kGroups : -kGroups) {
      const int tok0 = tile * kTile + group * 16;        // this warp's tokens
      // ---- scores
      wait_full();
      if (kWarps > kGroups && group >= kGroups) {
        // another's tile: waited for and given back like an own one, so that
        // no slot is filled again before every warp has seen it full (its
        // barrier then never is two phases ahead of a waiting warp)
        give_back();
        wait_full();
        give_back();
        continue;
      }
      float sc_[2][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) sc_[0][e] = sc_[1][e] = 0.f;
      const uint32_t sK = sbase + s * L::kSlot;
      auto score_step = [&](int ks, uint32_t b0, uint32_t b1, uint32_t b2, uint32_t b3) {
        mma16816<E4M3>(sc_[0], qreg[ks], b0, b1);
        mma16816<E4M3>(sc_[1], qreg[ks], b2, b3);
      };
      if constexpr (!E4M3) {
        const int tok = group * 16 + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t kb[4];
          const int ch = 2 * ks + ((lane >> 3) & 1);
          ldsm4(kb, sK + (ch >> 3) * (kTile * 128) + tok * 128 + (((ch & 7) ^ (tok & 7)) << 4));
          score_step(ks, kb[0], kb[1], kb[2], kb[3]);
        }
      } else {
        const int tok = group * 16 + (lane & 15);
#pragma unroll
        for (int k2 = 0; k2 < D / 32; ++k2) {
          uint32_t kb[4];
          ldsm4(kb, D == 128 ? (sK + tok * 128 + ((tok & 7) << 4)) ^ ((2 * k2 + (lane >> 4)) << 4)
                             : sK + swz_offset(tok, 2 * k2 + (lane >> 4), D));
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t b[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) e4m3x4_to_f16x4(kb[2 * half + e], b[2 * e], b[2 * e + 1]);
            score_step(2 * k2 + half, b[0], b[1], b[2], b[3]);
          }
        }
      }
      give_back();
      // ---- probabilities, in the layout of the next product's operand
      const bool masked = tok0 < all_lo || tok0 + 16 > all_hi;
      uint32_t pa[4];
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) {
        if (8 * hr >= rows) {                            // no such rows (the same for all threads)
          pa[hr] = pa[2 + hr] = 0u;
          continue;
        }
        const float f = fac[hr];
        if (masked) {
          const int4 ri = s_row[8 * hr + g];
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int tok = tok0 + nt * 8 + 2 * c + e;
              if (tok < ri.x || tok >= ri.y) sc_[nt][2 * hr + e] = -INFINITY;
            }
        }
        // (rounded before the maximum is taken away, so that the largest
        // gives exactly 0 whatever its size)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          sc_[nt][2 * hr] *= f;
          sc_[nt][2 * hr + 1] *= f;
        }
        float mx = fmaxf(fmax3(sc_[0][2 * hr], sc_[0][2 * hr + 1], sc_[1][2 * hr]), sc_[1][2 * hr + 1]);
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
        float& mr = m_run[hr];
        // What a row keeps, and what its parts are merged by, is the offset that
        // scores are taken relative to: the maximum less the shift.  (Compared as
        // a difference, so that it holds for scores whose steps are coarser than
        // the shift too; at the start, where mr is -inf, for anything but -inf.)
        const bool need = mx - mr > kRaise + kShift<E4M3>;
        const float m = need ? mx - kShift<E4M3> : mr, mu = m == -INFINITY ? 0.f : m;   // nothing seen yet: p = 2^-inf = 0
        if (__any_sync(0xFFFFFFFFu, need)) {
          const float alpha = ex2_approx(mr - mu);
          l_run[hr] *= alpha;
#pragma unroll
          for (int k = 0; k < D / 8; ++k) {
            acc[k][2 * hr] *= alpha;
            acc[k][2 * hr + 1] *= alpha;
          }
        }
        mr = m;
        float sum = 0.f;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const float p0 = ex2_approx(sc_[nt][2 * hr] - mu), p1 = ex2_approx(sc_[nt][2 * hr + 1] - mu);
          sum += p0 + p1;
          pa[2 * nt + hr] = pack(p0, p1);
        }
        l_run[hr] += sum;
      }
      // ---- values
      wait_full();
      const uint32_t sV = sbase + s * L::kSlot;
      // 16 columns (two column tiles) of the warp's 16 tokens; columns of an
      // E4M3 cache as 16 ch + 2 n + (0, 1) for column n of the two tiles
      auto load_v = [&](int ch2, uint32_t (&vb)[4]) {    // ch2: 16-column group
        const int tok = group * 16 + (lane & 15);
        if constexpr (!E4M3) {
          const int ch = 2 * ch2 + (lane >> 4);
          ldsm4t(vb, sV + (ch >> 3) * (kTile * 128) + tok * 128 + (((ch & 7) ^ (tok & 7)) << 4));
        } else {
          uint32_t vr[2];
          ldsm2t(vr, D == 128 ? (sV + tok * 128 + ((tok & 7) << 4)) ^ (ch2 << 4) : sV + swz_offset(tok, ch2, D));
          // (token, column) 00 01 10 11 in the bytes of vr: token pairs per column
#pragma unroll
          for (int e = 0; e < 2; ++e) e4m3x4_to_f16x4(__byte_perm(vr[e], 0u, 0x3120), vb[e], vb[2 + e]);
        }
      };
      // values of tokens outside [lo, hi) to zeros
      auto hide = [&](uint32_t (&vb)[4], int lo, int hi) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int tok = tok0 + 8 * (e & 1) + 2 * c;    // tokens tok, tok + 1 in the halves
          vb[e] &= (tok >= lo && tok < hi ? 0xFFFFu : 0u) | (tok + 1 >= lo && tok + 1 < hi ? 0xFFFF0000u : 0u);
        }
      };
      if (!masked) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t vb[4];
          load_v(k, vb);
          mma16816<E4M3>(acc[2 * k], pa, vb[0], vb[1]);
          mma16816<E4M3>(acc[2 * k + 1], pa, vb[2], vb[3]);
        }
      } else {
        // What no row sees may hold anything and becomes zeros.  What some
        // row sees may hold infinities or NaN that must not reach the others
        // (0 x inf): then one product per row, over that row's tokens only.
        bool wild = false;
#pragma unroll 1
        for (int k = 0; k < D / 16; ++k) {
          uint32_t vb[4];
          load_v(k, vb);
          hide(vb, rq.lo, rq.hi);
          constexpr uint32_t kExp = E4M3 ? 0x7C00u : 0x7F80u;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            wild = wild || (vb[e] & kExp) == kExp || ((vb[e] >> 16) & kExp) == kExp;
        }
        wild = __any_sync(0xFFFFFFFFu, wild);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t vb[4];
          load_v(k, vb);
          hide(vb, rq.lo, rq.hi);
          if (!wild) {
            mma16816<E4M3>(acc[2 * k], pa, vb[0], vb[1]);
            mma16816<E4M3>(acc[2 * k + 1], pa, vb[2], vb[3]);
          } else {
#pragma unroll 1
            for (int r = 0; r < kRows; ++r) {
              const int4 ri = s_row[r];
              uint32_t wb[4] = {vb[0], vb[1], vb[2], vb[3]};
              hide(wb, ri.x, ri.y);
              float t0[4] = {0.f, 0.f, 0.f, 0.f}, t1[4] = {0.f, 0.f, 0.f, 0.f};
              mma16816<E4M3>(t0, pa, wb[0], wb[1]);
              mma16816<E4M3>(t1, pa, wb[2], wb[3]);
#pragma unroll
              for (int e = 0; e < 4; ++e) {              // e >> 1: the thread's row g or g + 8
                if (8 * (e >> 1) + g == r) {
                  acc[2 * k][e] += t0[e];
                  acc[2 * k + 1][e] += t1[e];
                }
              }
            }
          }
        }
      }
      give_back();
    }

    // ---- end of the unit, or of this CTA's part of it: merge the warps
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float l = l_run[i];
      l += __shfl_xor_sync(0xFFFFFFFFu, l, 1);
      l += __shfl_xor_sync(0xFFFFFFFFu, l, 2);
      if (c == 0) s_ml[warp * kRows + 8 * i + g] = make_float2(m_run[i], l);
    }
    sync_consumers();
    const bool whole = ubase >= start && uend <= stop;
    const float scale_v = E4M3 ? __ldcg(sc + p.Hkv + h) : 1.0f;
    auto out_row = [&](int r) -> uint16_t* {
      const int row = r0 + r;
      return a.out + ((size_t)(rq.q0 + row / G) * p.Hq + h * G + row % G) * D;
    };
    const int part = 2 * blockIdx.x + (ubase < start ? 0 : 1);
    auto row_max = [&](int r) {
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_ml[w * kRows + r].x);
      return m;
    };
    // four rows at a time: every warp's O, scaled to the common maximum, into
    // shared memory, then each thread adds them for two columns
#pragma unroll
    for (int q4 = 0; q4 < kRows / 4; ++q4) {
      if (4 * q4 >= rows) break;
      const int hr = q4 >> 1;                            // which of the thread's rows
      if ((g >> 2) == (q4 & 1)) {
        const int r = 4 * q4 + (g & 3);
        const float m = row_max(r), f = ex2_approx(m_run[hr] - (m == -INFINITY ? 0.f : m));
        float* o = s_o + (warp * 4 + (g & 3)) * D;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const float v0 = acc[2 * k][2 * hr] * f, v1 = acc[2 * k][2 * hr + 1] * f;
          const float v2 = acc[2 * k + 1][2 * hr] * f, v3 = acc[2 * k + 1][2 * hr + 1] * f;
          if constexpr (E4M3) {
            *reinterpret_cast<float4*>(o + 16 * k + 4 * c) = make_float4(v0, v2, v1, v3);
          } else {
            *reinterpret_cast<float2*>(o + 16 * k + 2 * c) = make_float2(v0, v1);
            *reinterpret_cast<float2*>(o + 16 * k + 8 + 2 * c) = make_float2(v2, v3);
          }
        }
      }
      sync_consumers();
      for (int k = threadIdx.x; k < 4 * (D / 2); k += kConsumers) {
        const int rr = k / (D / 2), d2 = k % (D / 2), r = 4 * q4 + rr;
        if (r >= rows) break;
        float2 o = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float2 v = *reinterpret_cast<const float2*>(s_o + (w * 4 + rr) * D + 2 * d2);
          o.x += v.x;
          o.y += v.y;
        }
        const float m = row_max(r), mu = m == -INFINITY ? 0.f : m;
        float l = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) l += s_ml[w * kRows + r].y * ex2_approx(s_ml[w * kRows + r].x - mu);
        if (whole) {
          const float inv = l > 0.f || l != l ? scale_v / l : 0.f;
          *reinterpret_cast<uint32_t*>(out_row(r) + 2 * d2) = bf2(o.x * inv, o.y * inv);
        } else {
          *reinterpret_cast<float2*>(p.few_o + ((size_t)part * kFewRows + r) * D + 2 * d2) = o;
          if (d2 == 0)
            *reinterpret_cast<float2*>(p.few_ml + ((size_t)part * kFewRows + r) * 2) = make_float2(m, l);
        }
      }
      sync_consumers();
    }
    if (!whole) {
      // CTAs whose ranges hold a tile of this unit: owner(t) is the last CTA
      // whose range starts at or before tile t
      const int first = (int)(((ubase + 1) * parts - 1) / total), last = (int)((uend * parts - 1) / total);
      __threadfence();
      sync_consumers();
      if (threadIdx.x == 0) {
        const int old = atomicAdd(p.few_tickets + first, 1);
        misc->last = old == last - first;
        if (misc->last) p.few_tickets[first] = 0;
      }
      sync_consumers();
      if (misc->last) {
        __threadfence();
        for (int k = threadIdx.x; k < rows * (D / 4); k += kConsumers) {
          const int r = k / (D / 4), d4 = k % (D / 4);
          auto slot = [&](int cta) { return (size_t)(2 * cta + (cta == first ? 1 : 0)) * kFewRows + r; };
          float m = -INFINITY, l = 0.f;
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int c0 = first; c0 <= last; c0 += 8) {     // eight parts' loads in flight at a time
            float2 ml[8];
            float4 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int cta = c0 + i <= last ? c0 + i : last;
              ml[i] = __ldcg(reinterpret_cast<const float2*>(p.few_ml + slot(cta) * 2));
              v[i] = __ldcg(reinterpret_cast<const float4*>(p.few_o + slot(cta) * D) + d4);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if (c0 + i > last) break;
              const float mn = fmaxf(m, ml[i].x), mu = mn == -INFINITY ? 0.f : mn;
              const float wa = ex2_approx(m - mu), wb = ex2_approx(ml[i].x - mu);
              l = l * wa + ml[i].y * wb;
              o.x = o.x * wa + v[i].x * wb;
              o.y = o.y * wa + v[i].y * wb;
              o.z = o.z * wa + v[i].z * wb;
              o.w = o.w * wa + v[i].w * wb;
              m = mn;
            }
          }
          const float inv = l > 0.f || l != l ? scale_v / l : 0.f;
          *reinterpret_cast<uint2*>(out_row(r) + 4 * d4) = make_uint2(bf2(o.x * inv, o.y * inv), bf2(o.z * inv, o.w * inv));
        }
      }
    }
    if (x < stop) next_unit();
  }
  if (threadIdx.x == 0 && *abort)
    atomicOr(reinterpret_cast<unsigned*>(p.state + PST_ERROR), KVRING_PAGES_ERR_TIMEOUT);
  if (a.beside) griddep_wait();
}

template <int D, bool E4M3>
cudaError_t prepare_one() {
  return cudaFuncSetAttribute(k_paged_few<D, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              FewLayout<D, E4M3>::kBytes);
}
template <int D, bool E4M3>
cudaError_t go(const PagesDev& p, const CUtensorMap* tmK, const CUtensorMap* tmV, const PagedAttn& a, cudaStream_t s) {
  return launch_pdl(k_paged_few<D, E4M3>, dim3((unsigned)a.ctas), dim3(FewLayout<D, E4M3>::kThreads),
                    FewLayout<D, E4M3>::kBytes, s, *tmK, *tmV, p, a);
}

}  // namespace

cudaError_t paged_few_prepare() {
  cudaError_t e = prepare_one<128, true>();
  if (e == cudaSuccess) e = prepare_one<128, false>();
  if (e == cudaSuccess) e = prepare_one<64, true>();
  if (e == cudaSuccess) e = prepare_one<64, false>();
  return e;
}

cudaError_t launch_paged_few(const PagesDev& p, const CUtensorMap* tmK, const CUtensorMap* tmV, const PagedAttn& a,
                             cudaStream_t s) {
  if (p.D == 128) return p.e4m3 ? go<128, true>(p, tmK, tmV, a, s) : go<128, false>(p, tmK, tmV, a, s);
  return p.e4m3 ? go<64, true>(p, tmK, tmV, a, s) : go<64, false>(p, tmK, tmV, a, s);
}

}  // namespace kvr
