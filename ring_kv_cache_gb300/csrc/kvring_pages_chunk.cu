// Attention over the paged cache for requests with many query rows (chunks
// of a prompt, whole frames), on the tcgen05 tensor cores.
//
//   out[r] = sum_j softmax_j(s_rj) V[j],  s_rj = scale q[r] . K[j]
// in one pass over the keys with a running maximum per row, raised only when
// a tile's maximum exceeds it by more than 8 (log2 units): then and only then
// is the accumulator rescaled.  Probabilities are rounded once, to the 16-bit
// type of the values' operand (f16 over an E4M3 cache, else bf16), and the
// normaliser sums them unrounded in fp32.
//
// Bound by the tensor cores: 4 rows keys d operations against
// 2 keys d cached values per 256 rows.  A unit is 256 query rows of one
// request and key/value head, a row being one query head of one token, so
// all query heads of a key/value head share its tiles and the causal
// diagonal is as fine as the tokens of a unit; two row groups of 128 take
// turns on the tensor cores: while one group's scores are turned into
// probabilities, the other's products run.  Per 128-token tile and group:
//   S_g = Q_g K^T  (kind::f16, both operands from shared memory)
//   O_g += P_g V   (P from TMEM; V MN-major from shared memory, as the TMA
//                   wrote it)
// P_g lies over S_g in TMEM, so the scores of the next tile follow P_g V of
// this one.  At d = 128: S_0, S_1, O_0, O_1, 128 columns each.  At d = 64 the
// products are half as long and there is room for four streams of 128 columns,
// each row group's tiles cut into two halves of 64 tokens with softmax warps and
// sums of their own, added at the unit's end, and for two units' queries in
// shared memory.  (With whole tiles in two streams, probabilities in columns of
// their own and each tile's scores computed while the tile before is turned into
// probabilities, 2,048 queries over 32,768 tokens take 555 us instead of 470: eight
// softmax warps are too few to keep the exponentials busy.)
//
// The (request, row tile, head, key tile) space is flattened and cut into
// one contiguous range per CTA, as in the kernel for few rows; units cut by a
// range's border leave partial (m, l, O) in the workspace and the last CTA to
// arrive merges them in range order.
//
// Warps: 0-7 softmax (group = warp / 4, thread = row), 8 copies (walks the
// units, writes their descriptors into a small queue, TMA), 9 (and 10 at
// d = 64) the MMA issuers, the rest helpers: over an E4M3 cache they widen each landed tile, exactly, to
// f16 (K and V); over a bf16 cache they only touch tiles at the borders of
// what a request may read, whose values at other places become zeros.
//
// A value that some rows of a unit see and others do not may be infinite or
// NaN, and 0 x inf in the product would carry it into the rows that do not.
// So the helpers, in tiles with a mask, put zeros in the place of such
// values and mark the unit, and the rows that do see them add them to their
// sums at the end (p inf = inf, p NaN = NaN for any probability).
//
// Queries over an E4M3 cache: f16 after scaling each row by a power of two
// into [1, 2) at its largest value (bf16's 8 significant bits fit f16's 11).
//
// Every wait, those between the threads of a group included, is an mbarrier
// wait with a limit; after one gives up nobody waits any more, every warp
// leaves at its next unit, copies and MMAs in flight are drained, TMEM is
// freed and KVRING_PAGES_ERR_TIMEOUT is set.  Tickets that were then not
// drawn are cleared by the next plan.
//
// Measured (GB300): 4,096 queries behind 12,288 cached tokens, causal, 32/8
// heads x 128, bf16: 605 to 622 us in a graph, 629 us a call among others, 1,530
// to 1,590 TFLOP/s (81 to 84 % of the library product's 1,884, 90 to 94 % of what
// that keeps up for seconds); 757
// queries over 5,788 E4M3 tokens, 40 heads, all seen: 84 us (1,070 TFLOP/s; 120
// units on 152 SMs, so nearly all are split); 11 chunks of up to 900 tokens,
// window 1,500, 20/4 heads x 64: 80 to 87 us.  At d = 128 a tile takes what a
// group's chain does (softmax 1,550 cycles, then its two products behind the
// other group's, 1,230), at d = 64 the issue of the softmax warps (59 % of the
// slots; exponentials 44 %, ALU 42 %, tensor pipe 43 %).
#include <type_traits>

#include "kvring_pages.cuh"


namespace kvr {
namespace {

constexpr int kUnitQueue = 4;
// A unit's start and end cost about as much as this many of its tiles (its
// queries' way to the tensor cores, the last probabilities' and the results'
// way out); ranges are cut by tiles plus this.
constexpr int kUnitCost = 3;      // (8,192 causal queries: 404, 372, 372, 380 us with 2, 3, 4, 6)
constexpr int kTileBits = 40;     // of the sums over requests: places in the low bits, units above
constexpr int kChunkSmem = 232448;
// Tiles whose blocks' exponents are kept.  When a tile's are written its slot for
// keys is free, so the helpers are through the entry kRaws before, whose slot the
// MMAs of the entry kSlots before that have left: the values of the tile seven
// before (four at d = 128) have been multiplied, so its exponents have been read.
constexpr int kExpTiles = 8;

template <int D, bool E4M3, bool BLK>
struct ChunkLayout {
  // Streams: a row group's 128 rows, and at d = 64 half of each tile's tokens.
  static constexpr int kHalves = D == 128 ? 1 : 2;               // token halves of a tile
  static constexpr int kStreams = 2 * kHalves;
  static constexpr int kCols = kTile / kHalves;                  // tokens of a stream's tile
  static constexpr int kIssuers = kHalves;                       // MMA-issuing threads, two streams each
  static constexpr int kSoftWarps = 4 * kStreams;
  static constexpr int kSoftThreads = 32 * kSoftWarps;
  static constexpr int kWarpCopy = kSoftWarps, kWarpIssue = kSoftWarps + 1;
  // Over an E4M3 cache the helpers are a warpgroup of their own (with idle
  // warps before them), so that registers can move between warpgroups.
  static constexpr int kWarpHelp = E4M3 ? kSoftWarps + 4 : kWarpIssue + kIssuers;
  static constexpr int kHelpers = E4M3 ? 4 : kSoftWarps + 4 - kWarpHelp;   // warps
  static constexpr int kThreads = 32 * (kWarpHelp + kHelpers);
  // Registers per thread after the split (0: none): the sum over all threads
  // stays that of the launch (128 x 512, 96 x 640, 80 x 768).  Over blocks each of
  // a tile's eight has a factor and an exponent in registers beside the scores (4,096
  // queries behind 12,288: 730 us with 176, 699 with 192, 719 with 200).
  static constexpr int kRegsSoft = D == 128 ? (E4M3 ? (BLK ? 192 : 176) : 0) : (E4M3 ? 96 : 104);
  static constexpr int kRegsRest = D == 128 ? (E4M3 ? (BLK ? 64 : 80) : 0) : (E4M3 ? 48 : 64);
  static constexpr int kAtom = kTile * 128;                      // 128 rows x 64 16-bit columns
  static constexpr int kAtoms = D / 64;
  static constexpr int kQGroup = kAtoms * kAtom;
  static constexpr int kSlot = kAtoms * kAtom;                   // one 16-bit K or V tile
  static constexpr int kRaw = E4M3 ? kTile * D : 0;              // one E4M3 tile
  static constexpr int kSlots = D == 128 ? (E4M3 ? 3 : 5) : (E4M3 ? 7 : 9);
  static constexpr int kRaws = E4M3 ? (D == 128 ? 4 : 5) : 0;
  static constexpr int kQBufs = D == 128 ? 1 : 2;                // units whose queries fit
  // TMEM columns of stream i: scores (the probabilities over them), sums
  static constexpr uint32_t col_s(int i) { return 128 * i; }
  static constexpr uint32_t col_o(int i) { return D == 128 ? 256 + 128 * i : 128 * i + 64; }
  static constexpr int kQ = 0;
  static constexpr int kKV = kQBufs * 2 * kQGroup;
  static constexpr int kRawAt = kKV + kSlots * kSlot;
  static constexpr int kMisc = kRawAt + kRaws * kRaw;
  static constexpr int kMiscBytes = BLK ? 1280 : 1536;
  static constexpr int kMl = kMisc + kMiscBytes;                 // float2 [2][2][halves][128]: their maxima and sums, by unit parity
  // float [tiles][3][8], a tile in turn: 2^e_k, e_v and 2^-e_v of its blocks (BLK)
  static constexpr int kExp = kMl + (kHalves > 1 ? 4 * kHalves * kTile * 8 : 0);
  static constexpr int kBytes = 1024 + kExp + (BLK ? kExpTiles * 96 : 0);
  static_assert(kBytes <= kChunkSmem, "fits one CTA per SM");
};

// One unit, or the part of it in this CTA's range.
struct Unit {
  int q_tok;       // first token in q and out
  int pos0;        // its position
  int ntok;        // tokens of the unit
  int klen;        // the request's length
  int vlo, vhi;    // tokens any row of the unit sees: [vlo, vhi)
  int tile0, ntile;
  int h;
  int whole;       // all of its tiles are this CTA's
  int part;        // workspace slot, if not
  int first, last; // the CTAs that share it
  int end;         // no unit follows
  int table;       // the request's row of the block tables
  int wild;        // a masked tile holds values that are not finite
  int n0;          // this CTA's tiles before it
};

// The words of the step that describe a request, and what follows from them.
struct ChunkWords {
  int q0, end, klen, row;
};
__device__ __forceinline__ ChunkWords load_chunk_words(const PagesDev& p, int b) {
  return ChunkWords{__ldcg(p.cu + b), __ldcg(p.cu + b + 1), __ldcg(p.klen + b), __ldcg(p.rows + b)};
}
struct ChunkReq {
  int q0, nq, klen, pos0, nrt, row;
};
__device__ __forceinline__ ChunkReq make_chunk_req(const PagedAttn& a, const ChunkWords& w, int G, int tpu) {
  ChunkReq r;
  r.q0 = w.q0;
  r.row = w.row;
  r.klen = w.klen;
  r.pos0 = r.klen - (w.end - r.q0);
  r.nq = (w.end < a.T ? w.end : a.T) - r.q0;
  const long long rows = (long long)(w.end - r.q0) * G;
  if (r.nq < 0 || r.klen <= 0 || rows <= a.min_rows || rows > a.max_rows) r.nq = 0;
  r.nrt = (r.nq + tpu - 1) / tpu;
  return r;
}
struct ChunkMisc {
  uint64_t u_full[kUnitQueue], u_empty[kUnitQueue];
  uint64_t q_full[2], q_ready[2], q_empty[2];
  // of a stream: scores there, probabilities there, its last product done
  // (pv), its sums read
  uint64_t s_full[4], p_full[4], pv[4], o_free[4];
  // ring slots: the copy landed (bf16 only), the helpers are done with it,
  // its MMAs have read it; and the E4M3 tiles before they are widened
  uint64_t full[11], ready[11], empty[11], raw_full[6], raw_empty[6];
  uint64_t p_half[4];   // the first half of the probabilities there
  uint64_t exps[kExpTiles];   // a tile's exponents there
  uint64_t done[2], grp[2];
  unsigned long long ws[24];
  long long total, base;
  Unit u[kUnitQueue];
  ChunkReq rq;   // the request the CTA starts in
  uint32_t tmem;
  int b0, rt0, parts, abort, last[2];
};
static_assert(sizeof(ChunkMisc) <= ChunkLayout<128, true, true>::kMiscBytes, "misc block");

// The key tiles [t0, t0 + nt) of row tile rt.
__device__ __forceinline__ int chunk_tiles(const PagedAttn& a, const ChunkReq& r, int rt, int tpu, int* t0) {
  const int i0 = rt * tpu, i1 = i0 + tpu < r.nq ? i0 + tpu : r.nq;
  const int hi = a.causal ? r.pos0 + i1 : r.klen;
  int lo = a.window > 0 ? r.pos0 + i0 + 1 - a.window : 0;
  lo = lo > 0 ? lo : 0;
  *t0 = lo / kTile;
  return (hi + kTile - 1) / kTile - *t0;
}

__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                           uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "mov.b64 da, {%1, %2};\n\t"
      "mov.b64 db, {%3, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc)
      : "memory");
}
// idesc of kind::f16: bf16 operands have type code 1, f16 code 0.
__host__ __device__ constexpr uint32_t idesc_16(int M, int N, bool b_mn_major, bool bf16) {
  return idesc_f16(M, N, b_mn_major) | (bf16 ? (1u << 7) | (1u << 10) : 0u);
}

// 32 fp32 values to bf16 in a row of the output: whole 32-byte sectors where
// the output is aligned for them.
__device__ __forceinline__ void store_row32(uint16_t* dst, const float (&x)[32], bool out32) {
  uint32_t w[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const __nv_bfloat162 b2 = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
    w[e] = *reinterpret_cast<const uint32_t*>(&b2);
  }
  if (out32) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + 16 * k), "r"(w[8 * k]),
                   "r"(w[8 * k + 1]), "r"(w[8 * k + 2]), "r"(w[8 * k + 3]), "r"(w[8 * k + 4]), "r"(w[8 * k + 5]),
                   "r"(w[8 * k + 6]), "r"(w[8 * k + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      *reinterpret_cast<uint4*>(dst + 8 * k) = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
  }
}

// Eight 16-bit values w = *at of a masked tile: zeros where no row may read, zeros in
// the place of infinities and NaN (EXP: the exponent fields, ONE: their lowest
// bits, so that the sum carries into bit 15 where a field is all ones).
// Returns whether there were any of the latter.
template <uint32_t EXP, uint32_t ONE>
__device__ __forceinline__ uint32_t clean_values(uint4* at, uint4 w, bool inside) {
  auto wild = [](uint32_t x) { return ((x & EXP) + ONE) & 0x80008000u; };
  const uint32_t b = inside ? wild(w.x) | wild(w.y) | wild(w.z) | wild(w.w) : 0u;
  if (!inside) {
    *at = make_uint4(0u, 0u, 0u, 0u);
  } else if (b) {
    auto clean = [&](uint32_t& x) { x &= ~((wild(x) >> 15) * 0xFFFFu); };
    clean(w.x);
    clean(w.y);
    clean(w.z);
    clean(w.w);
    *at = w;
  }
  return b;
}

// BLK: an E4M3 cache with a scale 2^e per 16 tokens.  As in the kernel for few rows the
// values' exponent joins the score before the maximum is taken, and the
// normaliser's sums of 16 take it back; a block's 16 columns have a factor and an offset
// of their own in the multiply-add that makes the exponentials' arguments, so a tile
// costs eight factors, offsets and sums more per row: a frame of 757 over 5,788 tokens 94 us, 4,096
// queries behind 12,288 699 us (with scales per head and the same scores 93 and 688).
// Measured and slower: the codes brought to one exponent per tile by the helpers
// (779 us: the groups wait for them), factors read again from shared memory where they
// are used (812 us), pairs of them kept (832 us).
template <int D, bool E4M3, bool BLK>
__global__ void __launch_bounds__(ChunkLayout<D, E4M3, BLK>::kThreads, 1)
    k_paged_chunk(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const PagesDev p, const PagedAttn a) {
  static_assert(E4M3 || !BLK, "block scales are of E4M3 codes");
  using L = ChunkLayout<D, E4M3, BLK>;
  // Probabilities handed over in two parts, so that the first half's product
  // runs beside the second half's exponentials: over an E4M3 cache a gain (757
  // queries over 5,788 tokens, 40 heads: 86.4 -> 83.8 us), over a bf16 one, whose
  // scores wait for no helper, a loss (4,096 behind 12,288: 611 -> 630 us).
  constexpr bool kTwo = D == 128 && E4M3;
  constexpr int kThreads = L::kThreads, kHelpThreads = 32 * L::kHelpers;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(sm);
  ChunkMisc* misc = reinterpret_cast<ChunkMisc*>(sm + L::kMisc);
  volatile int* abort = &misc->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.Hq / p.Hkv, TG = kTile / G, tpu = 2 * TG;   // tokens of a group, of a unit
  auto bar = [](uint64_t& b) { return smem_u32(&b); };
  auto wait = [&](uint64_t& b, uint32_t parity) {
    if (!mbar_try_wait(smem_u32(&b), parity) && !*abort) mbar_wait_bounded(smem_u32(&b), parity, abort, a.wait_ns);
  };
  if (threadIdx.x == 0) {
    prefetch_tensormap(&tmQ);
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
    for (int i = 0; i < kUnitQueue; ++i) {
      mbar_init(bar(misc->u_full[i]), 1);
      mbar_init(bar(misc->u_empty[i]), L::kSoftWarps + L::kIssuers + L::kHelpers);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(bar(misc->q_full[g]), 1);
      mbar_init(bar(misc->q_ready[g]), L::kSoftThreads);
      mbar_init(bar(misc->q_empty[g]), L::kIssuers);
    }
    for (int i = 0; i < L::kStreams; ++i) {
      mbar_init(bar(misc->s_full[i]), 1);
      mbar_init(bar(misc->p_full[i]), 4);
      mbar_init(bar(misc->p_half[i]), 4);
      mbar_init(bar(misc->pv[i]), 1);
      mbar_init(bar(misc->o_free[i]), 4 * L::kHalves);
    }
    for (int i = 0; i < L::kSlots; ++i) {
      mbar_init(bar(misc->full[i]), 1);
      mbar_init(bar(misc->empty[i]), L::kIssuers);
      mbar_init(bar(misc->ready[i]), E4M3 ? kHelpThreads : L::kHelpers);
    }
    for (int i = 0; i < L::kRaws; ++i) {
      mbar_init(bar(misc->raw_full[i]), 1);
      mbar_init(bar(misc->raw_empty[i]), kHelpThreads);
    }
    for (int i = 0; i < kExpTiles; ++i) mbar_init(bar(misc->exps[i]), 1);
    for (int g = 0; g < 2; ++g) mbar_init(bar(misc->done[g]), 1);
    for (int g = 0; g < 2; ++g) mbar_init(bar(misc->grp[g]), kTile * L::kHalves);
    misc->abort = 0;
    mbar_fence_init();
  }
  griddep_wait();
  griddep_launch_dependents();

  // ------------------------------------------------- this CTA's range
  // (the words of the first requests are asked for together with their count)
  const ChunkWords first_words = load_chunk_words(p, (int)threadIdx.x < p.R ? threadIdx.x : 0);
  const int B = __ldcg(p.state + PST_REQUESTS);
  {
    const int per = (B + kThreads - 1) / kThreads;
    const int i0 = threadIdx.x * per, i1 = i0 + per < B ? i0 + per : B;
    auto req_of = [&](int i) { return make_chunk_req(a, per == 1 ? first_words : load_chunk_words(p, i), G, tpu); };
    unsigned long long mine = 0;
    int t0;
    for (int i = i0; i < i1; ++i) {
      const ChunkReq r = req_of(i);
      for (int rt = 0; rt < r.nrt; ++rt) mine += (unsigned)(kUnitCost + chunk_tiles(a, r, rt, tpu, &t0));
      mine += (unsigned long long)r.nrt << kTileBits;
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
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += misc->ws[w];
      total += misc->ws[w];
    }
    constexpr unsigned long long kTiles = (1ull << kTileBits) - 1;
    const unsigned long long units = (total >> kTileBits) * (unsigned)p.Hkv;
    total = (total & kTiles) * (unsigned)p.Hkv;
    before = ((before + x - mine) & kTiles) * (unsigned)p.Hkv;
    mine = (mine & kTiles) * (unsigned)p.Hkv;
    // a range per CTA; shorter than min_tiles only where that keeps as many
    // ranges as there are units
    unsigned long long parts = total / (unsigned)a.min_tiles;
    parts = parts > units ? parts : units;
    parts = parts < 1 ? 1 : (parts > gridDim.x ? gridDim.x : parts);
    const unsigned long long start = blockIdx.x < parts ? total * blockIdx.x / parts : total;
    if (mine && start >= before && start < before + mine) {   // exactly one thread, unless total is 0
      bool found = false;
      for (int i = i0; i < i1 && !found; ++i) {
        const ChunkReq r = req_of(i);
        for (int rt = 0; rt < r.nrt; ++rt) {
          const unsigned long long n = (unsigned long long)(kUnitCost + chunk_tiles(a, r, rt, tpu, &t0)) * (unsigned)p.Hkv;
          if (start < before + n) {
            misc->b0 = i;
            misc->rq = r;
            misc->rt0 = rt;
            misc->base = (long long)before;
            found = true;
            break;
          }
          before += n;
        }
      }
    }
    if (threadIdx.x == 0) {
      misc->total = (long long)total;
      misc->parts = (int)parts;
    }
    __syncthreads();
  }
  const long long total = misc->total, parts = misc->parts;
  const long long start = total * blockIdx.x / parts, stop = total * (blockIdx.x + 1) / parts;
  if (blockIdx.x >= parts || start >= stop) return;
  if (warp == L::kWarpIssue) {
    tmem_alloc(smem_u32(&misc->tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc->tmem;
  // whether a tile holds tokens outside [vlo, vhi), or tokens that some row
  // of the unit does not see
  auto edge_tile = [&](const Unit& u, int j) {
    const int t = (u.tile0 + j) * kTile;
    const int seen = a.causal ? u.pos0 + 1 : u.klen;                 // every row sees up to here
    const int from = a.window > 0 ? u.pos0 + u.ntok - a.window : 0;  // and from here
    return t + kTile > seen || t < from;
  };

  if (warp >= L::kSoftWarps) {
    if constexpr (L::kRegsRest) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::kRegsRest ? L::kRegsRest : 24));
  if (warp == L::kWarpCopy) {
    // ------------------------------------------------------------ copies
    const int box_rows = p.P < kTile ? p.P : kTile, nbox = kTile / box_rows;
    constexpr int kBoxes = E4M3 ? 1 : L::kAtoms;
    const uint32_t box_bytes = (uint32_t)(box_rows * (E4M3 ? D : 128));
    const long long layer0 = (long long)a.layer * p.num_pages;
    const int none = p.L * p.num_pages * p.Hkv;
    constexpr int kRing = E4M3 ? L::kRaws : L::kSlots;
    uint64_t* full = E4M3 ? misc->raw_full : misc->full;
    uint64_t* empty = E4M3 ? misc->raw_empty : misc->empty;
    constexpr int kRingAt = E4M3 ? L::kRawAt : L::kKV, kRingSize = E4M3 ? L::kRaw : L::kSlot;
    bool stopped = a.debug_stall;
    int b = misc->b0, rt = misc->rt0, t0;
    ChunkReq rq = misc->rq;
    int nt = chunk_tiles(a, rq, rt, tpu, &t0);
    int h = (int)((start - misc->base) / (nt + kUnitCost));
    long long ubase = misc->base + (long long)h * (nt + kUnitCost), x = start;   // x: next place of the range
    int n = 0, nu = 0, nq = 0;   // ring entries filled, units begun, query copies issued
    auto try_wait = [&](uint64_t& br, uint32_t parity) {
      const bool ok = !stopped && !*abort && mbar_wait_bounded(smem_u32(&br), parity, abort, a.wait_ns);
      stopped = !__all_sync(0xFFFFFFFFu, ok);
    };
    for (;;) {
      // the unit's tiles lie at [t_at, uend) of the flattened space
      const long long t_at = ubase + kUnitCost, uend = t_at + nt;
      const bool end = x >= stop;
      const long long from = x > t_at ? x : t_at, ue = uend < stop ? uend : stop;
      const int tile0 = t0 + (int)(from - t_at), ntile = (int)(ue - from);
      const int i0 = rt * tpu, ntok = rq.nq - i0 < tpu ? rq.nq - i0 : tpu;
      if (end || ntile > 0) {
      const int uq = nu % kUnitQueue;
      try_wait(misc->u_empty[uq], ((nu / kUnitQueue) & 1) ^ 1);
      if (stopped && (nu > 0 || !a.debug_stall)) break;
      if (lane == 0) {
        Unit& u = misc->u[uq];
        u.end = end;
        u.q_tok = rq.q0 + i0;
        u.pos0 = rq.pos0 + i0;
        u.ntok = ntok;
        u.klen = rq.klen;
        const int lo = rq.pos0 + i0 + 1 - a.window;
        u.vlo = a.window > 0 && lo > 0 ? lo : 0;
        u.vhi = a.causal ? rq.pos0 + i0 + ntok : rq.klen;
        u.tile0 = tile0;
        u.ntile = ntile;
        u.h = h;
        u.table = rq.row;
        u.wild = 0;
        u.n0 = n >> 1;
        u.whole = ntile == nt;
        // the CTAs whose ranges hold a tile of this unit (the owner of place x
        // is the last CTA whose range starts at or before x)
        u.first = (int)(((t_at + 1) * parts - 1) / total);
        u.last = (int)((uend * parts - 1) / total);
        u.part = 2 * blockIdx.x + (u.first == (int)blockIdx.x ? 1 : 0);
        mbar_arrive(bar(misc->u_full[uq]));
      }
      __syncwarp();
      if (end) break;
      const int32_t* tab = p.tables + (size_t)rq.row * p.W;
      const int hi_u = a.causal ? rq.pos0 + i0 + ntok : rq.klen;   // what the unit's rows see
      int lo_u = a.window > 0 ? rq.pos0 + i0 + 1 - a.window : 0;
      lo_u = lo_u > 0 ? lo_u : 0;
      auto page_of = [&](int t) -> int {
        const int tok = t * kTile + lane * box_rows;
        if (lane >= nbox || tok >= hi_u || tok + box_rows <= lo_u) return -2;
        return __ldcg(tab + (tok >> p.logP));
      };
      int page = page_of(tile0);
      // The exponents of K and V of 16 tokens, block `lane` of the tile: their page is that
      // of the piece they lie in.  Asked for a tile ahead, and not looked at before (any
      // use would wait here).
      struct Exps {
        int k, v;
      };
      auto exps_of = [&](int t, int pg) -> Exps {
        const int id = __shfl_sync(0xFFFFFFFFu, pg, (lane & 7) * KVRING_SCALE_BLOCK / box_rows);
        if (lane >= 8 || id < 0 || id >= p.num_pages) return Exps{127, 127};
        const int tok = (t * kTile + lane * KVRING_SCALE_BLOCK) & (p.P - 1);
        const size_t at = ((size_t)(layer0 + id) * p.Hkv + h << p.logP >> 4) + (tok >> 4);
        return Exps{__ldcg(p.ks + at), __ldcg(p.vs + at)};
      };
      int page2 = -2;
      Exps exps{}, exps2{};
      if constexpr (BLK) {
        page2 = ntile > 1 ? page_of(tile0 + 1) : -2;
        exps = exps_of(tile0, page);
      }
      for (int j = 0; j < ntile && !stopped; ++j) {
        const int tile = tile0 + j;
        int ahead;
        if constexpr (BLK) {
          ahead = page2;
          page2 = j + 2 < ntile ? page_of(tile + 2) : -2;
          if (j + 1 < ntile) exps2 = exps_of(tile + 1, ahead);
        } else {
          ahead = j + 1 < ntile ? page_of(tile + 1) : -2;
        }
        const unsigned there = __ballot_sync(0xFFFFFFFFu, page != -2);
        const int row0 = (tile * kTile + lane * box_rows) & (p.P - 1);
        const bool ok = page >= 0 && page < p.num_pages;
        if (page != -2 && !ok) atomicOr(reinterpret_cast<unsigned*>(p.state + PST_ERROR), KVRING_PAGES_ERR_TABLE);
        const int c2 = ok ? (int)((layer0 + page) * p.Hkv + h) : none;
        for (int kv = 0; kv < 2 && !stopped; ++kv, ++n) {
          const int s = n % kRing;
          try_wait(empty[s], ((n / kRing) & 1) ^ 1);
          if (stopped) break;
          if (lane == 0) mbar_arrive_expect_tx(bar(full[s]), (uint32_t)__popc(there) * kBoxes * box_bytes);
          __syncwarp();
          if (page != -2) {
            const uint32_t dst = sbase + kRingAt + s * kRingSize + lane * box_bytes;
#pragma unroll
            for (int c = 0; c < kBoxes; ++c)
              tma_load_3d(dst + c * L::kAtom, kv ? &tmV : &tmK, c * 64, row0, c2, bar(full[s]));
          }
          if constexpr (BLK) {
            if (kv == 0) {
              const int at = (n >> 1) % kExpTiles;
              if (lane < 8) {
                auto within = [](int e) { return e < kMinExp ? kMinExp : (e > kMaxExp ? kMaxExp : e); };
                const int ek = within(exps.k), ev = within(exps.v);
                float* e = reinterpret_cast<float*>(sm + L::kExp) + 24 * at + lane;
                e[0] = __uint_as_float((uint32_t)ek << 23);
                e[8] = (float)(ev - 127);
                e[16] = __uint_as_float((uint32_t)(254 - ev) << 23);
              }
              __syncwarp();
              if (lane == 0) mbar_arrive(bar(misc->exps[at]));
              exps = exps2;
            }
          }
          // the queries behind the unit's first keys: their place is free
          // once the previous unit's last scores have been computed
          if (j == 0 && kv == 0) {
            const int qb = nu % L::kQBufs;
            try_wait(misc->q_empty[qb], ((nu / L::kQBufs) & 1) ^ 1);
            if (stopped) {
              ++n;
              break;
            }
            if (lane == 0) {
              const int ng = ntok > TG ? 2 : 1;
              mbar_arrive_expect_tx(bar(misc->q_full[qb]), (uint32_t)(ng * L::kAtoms * TG * G * 128));
              for (int g = 0; g < ng; ++g)
#pragma unroll
                for (int c = 0; c < L::kAtoms; ++c)
                  tma_load_3d(sbase + L::kQ + (2 * qb + g) * L::kQGroup + c * L::kAtom, &tmQ, c * 64, h * G,
                              rq.q0 + i0 + g * TG, bar(misc->q_full[qb]));
              // the next unit's queries on their way into L2, if it is of the
              // same request
              const bool next_h = h + 1 < p.Hkv;
              if (uend < stop && (next_h || rt + 1 < rq.nrt))
                for (int g = 0; g < 2; ++g)
#pragma unroll
                  for (int c = 0; c < L::kAtoms; ++c)
                    tma_prefetch_3d(&tmQ, c * 64, next_h ? (h + 1) * G : 0, rq.q0 + i0 + (next_h ? 0 : tpu) + g * TG);
            }
            ++nq;
            __syncwarp();
          }
        }
        page = ahead;
      }
      ++nu;
      }
      x = ue;
      if (x < stop) {
        ubase = uend;
        if (++h == p.Hkv) {
          h = 0;
          if (++rt >= rq.nrt) {
            rt = 0;
            do rq = make_chunk_req(a, load_chunk_words(p, ++b), G, tpu);
            while (rq.nrt == 0);
          }
          nt = chunk_tiles(a, rq, rt, tpu, &t0);
        }
      }
    }
    // every copy lands before the CTA may exit
    volatile int no_abort = 0;
    for (int i = n - kRing < 0 ? 0 : n - kRing; i < n; ++i)
      mbar_wait_bounded(bar(full[i % kRing]), (i / kRing) & 1, &no_abort, a.wait_ns);
    for (int i = nq - L::kQBufs < 0 ? 0 : nq - L::kQBufs; i < nq; ++i)
      mbar_wait_bounded(bar(misc->q_full[i % L::kQBufs]), (i / L::kQBufs) & 1, &no_abort, a.wait_ns);
  } else if (warp >= L::kWarpIssue && warp < L::kWarpIssue + L::kIssuers) {
    // ------------------------------------------------- MMA issuers
    // One thread issues for two streams: both row groups at d = 128 (with a
    // thread for each, their products interleave: 612 -> 655 us), the two token
    // halves of a group at d = 64.  Commits are few and none lies between a
    // product and the next scores.
    if (elect_one()) {
      const int who = warp - L::kWarpIssue;
      constexpr uint32_t idesc_qk = idesc_16(128, L::kCols, false, !E4M3), idesc_pv = idesc_16(128, D, true, !E4M3);
      const uint64_t dq = smem_desc(sbase + L::kQ, 16, 1024, 2u), dk = smem_desc(sbase + L::kKV, 16, 1024, 2u);
      const uint64_t dv = smem_desc(sbase + L::kKV, (uint32_t)L::kAtom, 1024, 2u);
      constexpr uint32_t kSlotStep = L::kSlot >> 4, kQStep = L::kQGroup >> 4, kAtomStep = L::kAtom >> 4;
      constexpr uint32_t kHalfStep = L::kCols * 128 >> 4;   // a half's rows of a K or V tile
      const uint32_t q_lo = (uint32_t)dq, q_hi = (uint32_t)(dq >> 32);
      const uint32_t k_lo = (uint32_t)dk, k_hi = (uint32_t)(dk >> 32), v_lo = (uint32_t)dv, v_hi = (uint32_t)(dv >> 32);
      int n = 0;   // slots so far
      auto slot_ready = [&](int i) { wait(misc->ready[i % L::kSlots], (i / L::kSlots) & 1); };
      // i: 0 or 1 of this thread's streams
      auto qk = [&](int i, int slot, uint32_t q_at) {
        const int g = L::kHalves == 1 ? i : who;
        const uint32_t k_at = k_lo + slot * kSlotStep + (L::kHalves == 1 ? 0 : i * kHalfStep);
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_f16_ss(tmem + L::col_s(2 * who + i), q_at + g * kQStep + (kk >> 2) * kAtomStep + 2 * (kk & 3), q_hi,
                     k_at + (kk >> 2) * kAtomStep + 2 * (kk & 3), k_hi, idesc_qk, kk != 0);
        mma_commit(bar(misc->s_full[2 * who + i]));
      };
      auto pv = [&](int i, int slot, bool first, int k0, int k1) {
        const uint32_t v_at = v_lo + slot * kSlotStep + (L::kHalves == 1 ? 0 : i * kHalfStep);
        tc_fence_after();
#pragma unroll
        for (int kk = k0; kk < k1; ++kk)
          mma_f16_ts_w(tmem + L::col_o(2 * who + i), tmem + L::col_s(2 * who + i) + 8 * kk, v_at + kk * 128, v_hi,
                       idesc_pv, (!first || kk > 0) ? 1u : 0u);
      };
      auto free_slot = [&](int slot) { mma_commit(bar(misc->empty[slot])); };
      int np[2] = {0, 0}, no[2] = {0, 0};   // each stream's products and units so far
      for (int nu = 0;; ++nu) {
        const int uq = nu % kUnitQueue;
        wait(misc->u_full[uq], (nu / kUnitQueue) & 1);
        const Unit u = misc->u[uq];
        if (u.end || *abort) break;
        const int qb = nu % L::kQBufs;
        const uint32_t q_at = q_lo + 2 * qb * kQStep;
        wait(E4M3 ? misc->q_ready[qb] : misc->q_full[qb], (nu / L::kQBufs) & 1);
        const bool second = u.ntok > TG;    // the second row group has rows
        const int ns = L::kHalves == 1 ? (second ? 2 : 1) : (who == 0 || second ? 2 : 0);
        if (ns == 0) {
          // no rows for this group: pass everything on as it comes
          mbar_arrive(bar(misc->q_empty[qb]));
          for (const int stop_n = n + 2 * u.ntile; n < stop_n; ++n) {
            slot_ready(n);
            mbar_arrive(bar(misc->empty[n % L::kSlots]));
          }
        } else {
          slot_ready(n);
          for (int i = 0; i < ns; ++i) qk(i, n % L::kSlots, q_at);
          free_slot(n % L::kSlots);
          if (u.ntile == 1) mma_commit(bar(misc->q_empty[qb]));
          for (int j = 0; j < u.ntile; ++j, n += 2) {
            const bool more = j + 1 < u.ntile;
            for (int i = 0; i < ns; ++i) {
              const int st = 2 * who + i;
              if (i == 0) slot_ready(n + 1);
              if constexpr (kTwo) {
                wait(misc->p_half[st], np[i] & 1);
                if (j == 0) wait(misc->o_free[st], (no[i]++ & 1) ^ 1);
                pv(i, (n + 1) % L::kSlots, j == 0, 0, L::kCols / 32);
                wait(misc->p_full[st], np[i]++ & 1);
                pv(i, (n + 1) % L::kSlots, false, L::kCols / 32, L::kCols / 16);
              } else {
                wait(misc->p_full[st], np[i]++ & 1);
                if (j == 0) wait(misc->o_free[st], (no[i]++ & 1) ^ 1);
                pv(i, (n + 1) % L::kSlots, j == 0, 0, L::kCols / 16);
              }
              // (the next scores' commit tells the softmax of this product
              // too, except behind the last tile)
              if (!more) {
                mma_commit(bar(misc->pv[st]));
              } else {
                if (i == 0) slot_ready(n + 2);
                qk(i, (n + 2) % L::kSlots, q_at);
              }
            }
            free_slot((n + 1) % L::kSlots);
            if (more) free_slot((n + 2) % L::kSlots);
            if (j + 2 == u.ntile) mma_commit(bar(misc->q_empty[qb]));
          }
        }
        mbar_arrive(bar(misc->u_empty[uq]));
      }
      // every MMA issued above has finished before TMEM is freed
      uint64_t& done = misc->done[who];
      mma_commit(bar(done));
      volatile int no_abort = 0;
      mbar_wait_bounded(bar(done), 0, &no_abort, a.wait_ns);
    }
    __syncwarp();
  } else if (warp >= L::kWarpHelp) {
    // ------------------------------------------------------------ helpers
    const int ht = threadIdx.x - 32 * L::kWarpHelp;
    int n = 0;
    for (int nu = 0;; ++nu) {
      const int uq = nu % kUnitQueue;
      wait(misc->u_full[uq], (nu / kUnitQueue) & 1);
      const Unit u = misc->u[uq];
      if (__any_sync(0xFFFFFFFFu, u.end || *abort)) break;
      if constexpr (E4M3) {
        // E4M3 tile [128 tokens][d] (128- or 64-byte swizzle) to f16 atoms
        // [128 tokens][64] (128-byte swizzle); task i: token i / CPR, 16
        // values i % CPR
        constexpr int CPR = D / 16, PER = kTile * CPR / kHelpThreads;
        for (int j = 0; j < 2 * u.ntile; ++j, ++n) {
          const int rs = n % L::kRaws, s = n % L::kSlots;
          wait(misc->raw_full[rs], (n / L::kRaws) & 1);
          const uint8_t* src = sm + L::kRawAt + rs * L::kRaw;
          uint4 w[PER];
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            const int k = ht + i * kHelpThreads;
            w[i] = *reinterpret_cast<const uint4*>(src + swz_offset(k / CPR, k % CPR, D));
          }
          wait(misc->empty[s], ((n / L::kSlots) & 1) ^ 1);
          uint8_t* dst = sm + L::kKV + s * L::kSlot;
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            const int k = ht + i * kHelpThreads, row = k / CPR, c = k % CPR;
            const uint32_t wi[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
            uint32_t hv[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) e4m3x4_to_f16x4(wi[e], hv[2 * e], hv[2 * e + 1]);
            uint8_t* atom = dst + (c >> 2) * L::kAtom;
            *reinterpret_cast<uint4*>(atom + swz_offset(row, 2 * (c & 3), 128)) = make_uint4(hv[0], hv[1], hv[2], hv[3]);
            *reinterpret_cast<uint4*>(atom + swz_offset(row, 2 * (c & 3) + 1, 128)) =
                make_uint4(hv[4], hv[5], hv[6], hv[7]);
          }
          if ((j & 1) && edge_tile(u, j >> 1)) {   // this thread's values again
            uint32_t bad = 0;
#pragma unroll 1
            for (int k = 2 * ht; k < 2 * kTile * CPR; k += 2 * kHelpThreads) {
              const int row = (k >> 1) / CPR, c = (k >> 1) % CPR, tok = (u.tile0 + (j >> 1)) * kTile + row;
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                uint4* at = reinterpret_cast<uint4*>(dst + (c >> 2) * L::kAtom + swz_offset(row, 2 * (c & 3) + e, 128));
                bad |= clean_values<0x7C007C00u, 0x04000400u>(at, *at, tok >= u.vlo && tok < u.vhi);
              }
            }
            if (bad) *const_cast<volatile int*>(&misc->u[uq].wild) = 1;
          }
          // (the E4M3 tile goes back only now: every value read from it is in
          // use, and the fence stands between the reads and the next copy, which
          // is of the other proxy)
          fence_proxy_async_smem();
          mbar_arrive(bar(misc->ready[s]));
          mbar_arrive(bar(misc->raw_empty[rs]));
        }
      } else {
        // every landed tile passes through the helpers, nearly always untouched
        for (int j = 0; j < 2 * u.ntile; ++j, ++n) {
          const int s = n % L::kSlots;
          wait(misc->full[s], (n / L::kSlots) & 1);
          if ((j & 1) && edge_tile(u, j >> 1)) {
            uint8_t* v = sm + L::kKV + s * L::kSlot;
            const int t = (u.tile0 + (j >> 1)) * kTile;
            uint32_t bad = 0;
            constexpr int kBatch = 8;   // loads in flight
#pragma unroll 1
            for (int k0 = ht; k0 < kTile * L::kAtoms * 8; k0 += kBatch * kHelpThreads) {
              uint4 w[kBatch];
#pragma unroll
              for (int i = 0; i < kBatch; ++i) w[i] = *reinterpret_cast<uint4*>(v + 16 * (k0 + i * kHelpThreads));
#pragma unroll
              for (int i = 0; i < kBatch; ++i) {
                const int k = k0 + i * kHelpThreads, tok = t + ((k >> 3) & (kTile - 1));
                bad |= clean_values<0x7F807F80u, 0x00800080u>(reinterpret_cast<uint4*>(v + 16 * k), w[i],
                                                              tok >= u.vlo && tok < u.vhi);
              }
            }
            if (bad) *const_cast<volatile int*>(&misc->u[uq].wild) = 1;
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(misc->ready[s]));
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(misc->u_empty[uq]));
    }
  }
  } else {
    if constexpr (L::kRegsSoft) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(L::kRegsSoft ? L::kRegsSoft : 24));
    // ------------------------------------------------------------ softmax
    const int st = warp >> 2, g = st / L::kHalves, half = st % L::kHalves, row = threadIdx.x & (kTile - 1);
    const int ri = row / G, head = row % G;            // the row's token in its group, its query head
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tS = trow + L::col_s(st), tO = trow + L::col_o(st);
    const bool speaks = half == 0 && row == 0;         // one thread of the group
    const float* sc = p.scales + (size_t)a.layer * 4 * p.Hkv;
    int syncs = 0;
    auto sync_group = [&]() {
      mbar_arrive(bar(misc->grp[g]));
      wait(misc->grp[g], syncs++ & 1);
      __syncwarp();
    };
    int nt_done = 0, nu_done = 0;   // this group's tiles and units so far
    const bool out32 = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;   // 32-byte stores
    for (int nu = 0;; ++nu) {
      const int uq = nu % kUnitQueue;
      wait(misc->u_full[uq], (nu / kUnitQueue) & 1);
      const Unit& u = misc->u[uq];
      if (__any_sync(0xFFFFFFFFu, u.end || *abort)) break;
      const bool active = g == 0 || u.ntok > TG;
      const int tok = g * TG + ri;
      const bool live = ri < TG && tok < u.ntok;
      float f_row = a.sm_log2;
      if constexpr (E4M3) {
        const int qb = nu % L::kQBufs;
        wait(misc->q_full[qb], (nu / L::kQBufs) & 1);
        // this row's queries, in place: D / 8 chunks of 16 bytes
        uint8_t* qg = sm + L::kQ + (2 * qb + g) * L::kQGroup;
        auto chunk_at = [&](int c) {
          return reinterpret_cast<uint4*>(qg + (c >> 3) * L::kAtom + swz_offset(row, c & 7, 128));
        };
        uint32_t em = 0;
        if (live) {
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {
            const uint4 w = *chunk_at(c);
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) em = max(em, max((ww[e] >> 7) & 0xFFu, (ww[e] >> 23) & 0xFFu));
          }
        }
        if (L::kHalves > 1) sync_group();              // (both halves' threads have read the row)
        if (live) {
          float up, down;
          query_factor(em, up, down);
          // (at least 1e-30: a factor that underflows would make NaN of what is
          // masked, and such scores are all alike anyway)
          f_row = fmaxf(f_row * (BLK ? 1.0f : __ldcg(sc + u.h)) * up, 1e-30f);
          if constexpr (BLK) f_row = fminf(f_row, kMostFactor);
#pragma unroll
          for (int i = 0; i < D / 8 / L::kHalves; ++i) {
            uint4* at = chunk_at(half * (D / 8 / L::kHalves) + i);
            const uint4 w = *at;
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              o[e] = f32x2_to_f16x2(__uint_as_float(ww[e] << 16) * down, __uint_as_float(ww[e] & 0xFFFF0000u) * down);
            *at = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(bar(misc->q_ready[qb]));
      }
      if (active) {
        // what this row sees, and what every row of the group sees
        const int pos = u.pos0 + tok;
        const int hi = live ? (a.causal ? pos + 1 : u.klen) : 0;
        const int lo = a.window > 0 && pos + 1 - a.window > 0 ? pos + 1 - a.window : 0;
        const int ntok_g = u.ntok - g * TG < TG ? u.ntok : (g + 1) * TG;
        const int all_hi = a.causal ? u.pos0 + g * TG + 1 : u.klen;
        const int all_lo = a.window > 0 ? u.pos0 + ntok_g - a.window : 0;
        const int ntile = u.ntile;
        // (a row that is none keeps a factor of 0 and asks for nothing; over blocks its maximum
        // is that of the values' exponents, which asks once where one is beyond kRaise)
        float m_run = live ? -INFINITY : 0.f, ell = 0.f;
        if (!live) f_row = 0.f;
        // (nothing seen yet: 2^-inf = 0)
        float moff = kShift<E4M3>;
        // (over an E4M3 cache a score is at most 4 x 448 x 128 < 2^18, so the
        // factor tells)
        bool huge = E4M3 && !BLK && __any_sync(0xFFFFFFFFu, f_row > 8.0f);
        // 32 scores to probabilities, as pairs of the 16-bit type; their sum
        // is added to lsum
        auto probabilities = [&](const uint32_t (&s32)[32], uint32_t* pw, float moff, float2& lsum) {
          const float2 fr2 = make_float2(f_row, f_row), mo2 = make_float2(moff, moff);
          float2 e[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 x =
                __ffma2_rn(make_float2(__uint_as_float(s32[2 * i]), __uint_as_float(s32[2 * i + 1])), fr2, mo2);
            e[i] = make_float2(ex2_approx(x.x), ex2_approx(x.y));
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if constexpr (E4M3) {
              pw[i] = f32x2_to_f16x2(e[i].x, e[i].y);
            } else {
              const __nv_bfloat162 b2 = __floats2bfloat162_rn(e[i].x, e[i].y);
              pw[i] = *reinterpret_cast<const uint32_t*>(&b2);
            }
          }
#pragma unroll
          for (int w = 8; w > 0; w >>= 1)
#pragma unroll
            for (int i = 0; i < w; ++i) e[i] = __fadd2_rn(e[i], e[i + w]);
          lsum = __fadd2_rn(lsum, e[0]);
        };
        // The same for 32 columns of two blocks: factors, offsets and weights of
        // their sums are theirs (e: their place among the tile's exponents).
        auto block_probabilities = [&](const uint32_t (&s32)[32], uint32_t* pw, const float* fr_b, const float* ev_b,
                                       const float* over_b, float moff, float2& lsum) {
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const float fr = fr_b[b], mo = moff + ev_b[b], over = over_b[b];
            const float2 fr2 = make_float2(fr, fr), mo2 = make_float2(mo, mo);
            float2 y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 x = __ffma2_rn(
                  make_float2(__uint_as_float(s32[16 * b + 2 * i]), __uint_as_float(s32[16 * b + 2 * i + 1])), fr2, mo2);
              y[i] = make_float2(ex2_approx(x.x), ex2_approx(x.y));
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) pw[8 * b + i] = f32x2_to_f16x2(y[i].x, y[i].y);
#pragma unroll
            for (int w = 4; w > 0; w >>= 1)
#pragma unroll
              for (int i = 0; i < w; ++i) y[i] = __fadd2_rn(y[i], y[i + w]);
            lsum = __ffma2_rn(y[0], make_float2(over, over), lsum);
          }
        };
        // Scores so large that factor x score, not rounded in the fused
        // multiply-add, may lie well above its rounding, the maximum: the
        // differences of the rounded ones (for the largest exactly 0) go in
        // the scores' place, over the factor.  From the first such tile on
        // the unit's tiles take the loop below that always does this.
        auto differences = [&](uint32_t (&sr)[L::kCols]) {
          const float mu = m_run == -INFINITY ? 0.f : m_run, over = 1.0f / f_row;
#pragma unroll
          for (int c = 0; c < L::kCols; ++c)
            sr[c] = __float_as_uint((__fmul_rn(__uint_as_float(sr[c]), f_row) - mu) * over);
          moff = kShift<E4M3>;
        };
        constexpr int kBlk = L::kCols / 16;   // blocks of a stream's tile
        // (over blocks: the whole difference, for a factor of 1 and no offset)
        auto block_differences = [&](uint32_t (&sr)[L::kCols], float (&fr)[kBlk], float (&ev)[kBlk]) {
          const float mu = m_run == -INFINITY ? 0.f : m_run;
#pragma unroll
          for (int c = 0; c < L::kCols; ++c)
            sr[c] = __float_as_uint(__fadd_rn(__fmul_rn(__uint_as_float(sr[c]), fr[c >> 4]), ev[c >> 4]) - mu);
#pragma unroll
          for (int b = 0; b < kBlk; ++b) {
            fr[b] = 1.0f;
            ev[b] = 0.f;
          }
          moff = kShift<E4M3>;
        };
        int j = 0;
        auto tile = [&](auto slow_tag) {
          constexpr bool slow = decltype(slow_tag)::value;
          [[maybe_unused]] float fr[kBlk], ev[kBlk];   // factors and exponents of the tile's blocks (BLK)
          const int n = u.n0 + j;
          [[maybe_unused]] const float* exps = reinterpret_cast<const float*>(sm + L::kExp) + 24 * (n % kExpTiles) + half * kBlk;
          if constexpr (BLK) {        // (there long before the scores are)
            wait(misc->exps[n % kExpTiles], (n / kExpTiles) & 1);
#pragma unroll
            for (int b = 0; b < kBlk; b += 4) {
              const float4 k4 = *reinterpret_cast<const float4*>(exps + b), v4 = *reinterpret_cast<const float4*>(exps + 8 + b);
              fr[b] = f_row * k4.x, fr[b + 1] = f_row * k4.y, fr[b + 2] = f_row * k4.z, fr[b + 3] = f_row * k4.w;
              ev[b] = v4.x, ev[b + 1] = v4.y, ev[b + 2] = v4.z, ev[b + 3] = v4.w;
            }
          }
          wait(misc->s_full[st], nt_done & 1);
          __syncwarp();
          tc_fence_after();
          const int t = (u.tile0 + j) * kTile + half * L::kCols;
          const bool masked = t + L::kCols > all_hi || t < all_lo;
          uint32_t sr[L::kCols];
#pragma unroll
          for (int c = 0; c < L::kCols / 32; ++c) tmem_ld32(tS + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(sr + 32 * c));
          tmem_wait_ld();
          if (masked) {
            const int vh = hi - t, vl = lo - t;
#pragma unroll
            for (int w = 0; w < L::kCols / 32; ++w) {
              const int h = vh - 32 * w, l = vl - 32 * w;
              uint32_t seen = h >= 32 ? 0xFFFFFFFFu : (h <= 0 ? 0u : (1u << h) - 1);
              if (l > 0) seen &= l >= 32 ? 0u : ~0u << l;
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!(seen >> c & 1u)) sr[32 * w + c] = __float_as_uint(-INFINITY);
            }
          }
          float tmax;
          if constexpr (BLK) {
            float w[kBlk];
#pragma unroll
            for (int b = 0; b < kBlk; ++b) {
              auto v = [&](int i) { return __uint_as_float(sr[16 * b + i]); };
              const float a0 = fmax3(v(0), v(1), v(2)), a1 = fmax3(v(3), v(4), v(5)), a2 = fmax3(v(6), v(7), v(8));
              const float a3 = fmax3(v(9), v(10), v(11)), a4 = fmax3(v(12), v(13), v(14));
              // (rounded as block_differences does, so that the largest gives exactly 0)
              w[b] = __fadd_rn(__fmul_rn(fmax3(fmax3(a0, a1, a2), fmax3(a3, a4, v(15)), a4), fr[b]), ev[b]);
            }
#pragma unroll
            for (int k = kBlk / 2; k > 0; k >>= 1)
#pragma unroll
              for (int i = 0; i < k; ++i) w[i] = fmaxf(w[i], w[i + k]);
            tmax = w[0];
          } else {
            float mx[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) mx[k] = fmaxf(__uint_as_float(sr[2 * k]), __uint_as_float(sr[2 * k + 1]));
#pragma unroll
            for (int i = 1; i < L::kCols / 16; ++i)
#pragma unroll
              for (int k = 0; k < 8; ++k)
                mx[k] = fmax3(mx[k], __uint_as_float(sr[16 * i + 2 * k]), __uint_as_float(sr[16 * i + 2 * k + 1]));
            tmax = f_row * fmaxf(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], fmax3(mx[5], mx[6], mx[7])));
          }
          const bool need = tmax > m_run + kRaise || (m_run == -INFINITY && tmax > m_run);
          const float m_new = need ? tmax : m_run;
          if (__any_sync(0xFFFFFFFFu, need)) {
            // S(j) complete means that P V(j - 1), issued before it, is, too
            if (j > 0) {
              const float alpha = need ? ex2_approx(m_run - m_new) : 1.0f;
#pragma unroll 1
              for (int c = 0; c < D / 16; ++c) {
                uint32_t rr[16];
                tmem_ld_n<16>(tO + 16 * c, rr);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                  const float2 y = __fmul2_rn(make_float2(__uint_as_float(rr[i]), __uint_as_float(rr[i + 1])),
                                              make_float2(alpha, alpha));
                  rr[i] = __float_as_uint(y.x);
                  rr[i + 1] = __float_as_uint(y.y);
                }
                tmem_st16(tO + 16 * c, rr);
              }
              ell *= alpha;
            }
            m_run = m_new;
            moff = kShift<E4M3> - (m_run == -INFINITY ? 0.f : m_run);
            if constexpr (!slow && (!E4M3 || BLK)) {
              huge = __any_sync(0xFFFFFFFFu, fabsf(moff) > 0x1p20f);
              if (huge) {
                if constexpr (BLK) block_differences(sr, fr, ev);
                else differences(sr);
              }
            }
          }
          if constexpr (slow) {
            if constexpr (BLK) block_differences(sr, fr, ev);
            else differences(sr);
          }
          float2 lsum = make_float2(0.f, 0.f);
#pragma unroll
          for (int c = 0; c < L::kCols / 32; ++c) {
            uint32_t pw[16];
            if constexpr (BLK)
              block_probabilities(*reinterpret_cast<uint32_t(*)[32]>(sr + 32 * c), pw, fr + 2 * c, ev + 2 * c, exps + 16 + 2 * c,
                                  moff, lsum);
            else
              probabilities(*reinterpret_cast<uint32_t(*)[32]>(sr + 32 * c), pw, moff, lsum);
            tmem_st16(tS + 16 * c, pw);
            if constexpr (kTwo) {
              if (c + 1 == L::kCols / 64) {
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(misc->p_half[st]));
              }
            }
          }
          ell += lsum.x + lsum.y;
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(misc->p_full[st]));
          ++nt_done;
        };
        for (; j < ntile && !huge; ++j) tile(std::false_type{});
        for (; j < ntile; ++j) tile(std::true_type{});
        // ------------------------------------------------------- epilogue
        // Both halves' sums count from here on: w_half their weights, m_run
        // and ell those of the row.  A half's threads write half the columns.
        float w_half[2] = {1.0f, 1.0f};
        if constexpr (L::kHalves > 1) {
          // (two places in turn: a half may be through the next unit's tiles
          // before the other has read this one's, but not through its exchange)
          float2* ml = reinterpret_cast<float2*>(sm + L::kMl) + (2 * (nu_done & 1) + g) * 2 * kTile + row;
          ml[half * kTile] = make_float2(m_run, ell);
          sync_group();
          const float2 a0 = ml[0], a1 = ml[kTile];
          m_run = fmaxf(a0.x, a1.x);
          const float mu = m_run == -INFINITY ? 0.f : m_run;
          w_half[0] = ex2_approx(a0.x - mu);
          w_half[1] = ex2_approx(a1.x - mu);
          ell = a0.y * w_half[0] + a1.y * w_half[1];
        }
#pragma unroll
        for (int i = 0; i < L::kHalves; ++i) wait(misc->pv[g * L::kHalves + i], nu_done & 1);
        ++nu_done;
        __syncwarp();
        tc_fence_after();
        constexpr int kC = D / 32 / L::kHalves;        // 32-column groups of this thread
        const int c_first = half * kC;
        const float scale_v = E4M3 && !BLK ? __ldcg(sc + p.Hkv + u.h) : 1.0f;
        const float inv = ell > 0.f || ell != ell ? scale_v / ell : 0.f;   // (of the row, both halves)
        const bool whole = u.whole;
        const int first = u.first, last = u.last;
        uint16_t* o16 = a.out + ((size_t)(u.q_tok + tok) * p.Hq + u.h * G + head) * D;
        // Partial rows lie column group by column group, [D/4][128 rows] of
        // four floats, so that a warp writes and reads whole lines; their
        // (maximum, sum) in part_ml.
        auto slot_of = [&](int cta) { return (size_t)(2 * cta + (cta == first ? 1 : 0)) * kPartRows + g * kTile; };
        int* ticket = p.tickets + 2 * first + g;
        // The CTA whose part is the last to be done merges: at once, with its
        // own accumulator, if the others' parts are all there already, else
        // all from the workspace.
        bool merge_now = false;
        if (!whole) {
          if (speaks) misc->last[g] = ld_acquire_gpu(ticket) == last - first;
          sync_group();
          merge_now = misc->last[g];
        }
        // Parts are always taken in range order (this CTA's own, where it
        // still has it, from registers), so the result does not depend on
        // who merges.
        float m_all = 0.f, iv_all = 0.f;
        auto ml_of = [&](int cta) {
          if (merge_now && cta == (int)blockIdx.x) return make_float2(m_run, ell);
          return __ldcg(reinterpret_cast<const float2*>(p.part_ml + (slot_of(cta) + row) * 2));
        };
        auto weigh = [&]() {
          float m = -INFINITY, l = 0.f;
#pragma unroll 4
          for (int cta = first; cta <= last; ++cta) {
            const float2 ml = ml_of(cta);
            const float mn = fmaxf(m, ml.x), mu = mn == -INFINITY ? 0.f : mn;
            l = l * ex2_approx(m - mu) + ml.y * ex2_approx(ml.x - mu);
            m = mn;
          }
          m_all = m == -INFINITY ? 0.f : m;
          iv_all = l > 0.f || l != l ? scale_v / l : 0.f;
        };
        auto merge_columns = [&](int c, const uint32_t (&own)[32]) {
          float x[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) x[k] = 0.f;
#pragma unroll 2
          for (int cta = first; cta <= last; ++cta) {
            const float4* src = reinterpret_cast<const float4*>(p.part_o + slot_of(cta) * D) + row;
            const bool mine = merge_now && cta == (int)blockIdx.x;
            float4 v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
              v[k] = mine ? make_float4(__uint_as_float(own[4 * k]), __uint_as_float(own[4 * k + 1]),
                                        __uint_as_float(own[4 * k + 2]), __uint_as_float(own[4 * k + 3]))
                          : __ldcg(src + (8 * c + k) * kTile);
            const float w = ex2_approx(ml_of(cta).x - m_all) * iv_all;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              x[4 * k] = fmaf(v[k].x, w, x[4 * k]);
              x[4 * k + 1] = fmaf(v[k].y, w, x[4 * k + 1]);
              x[4 * k + 2] = fmaf(v[k].z, w, x[4 * k + 2]);
              x[4 * k + 3] = fmaf(v[k].w, w, x[4 * k + 3]);
            }
          }
          if (live) store_row32(o16 + 32 * c, x, out32);
        };
        if (merge_now) {
          __threadfence();
          if (speaks) *ticket = 0;
          weigh();
        }
        const bool is_wild = *const_cast<const volatile int*>(&u.wild);
        float4* o32 = reinterpret_cast<float4*>(p.part_o + ((size_t)u.part * kPartRows + g * kTile) * D) + row;
#pragma unroll 1
        for (int c = c_first; c < c_first + kC; ++c) {
          uint32_t rr[32];
          __syncwarp();
          if constexpr (L::kHalves == 1) {
            tmem_ld32(tO + 32 * c, rr);
            tmem_wait_ld();
          } else {
            uint32_t r1[32];
            tmem_ld32(trow + L::col_o(2 * g) + 32 * c, rr);
            tmem_ld32(trow + L::col_o(2 * g + 1) + 32 * c, r1);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k)
              rr[k] = __float_as_uint(__uint_as_float(rr[k]) * w_half[0] + __uint_as_float(r1[k]) * w_half[1]);
          }
          if (is_wild && live) {
            // the values that are not finite among those this row sees
            for (int j = 0; j < ntile; ++j) {
              if (!edge_tile(u, j)) continue;
              const int t = (u.tile0 + j) * kTile;
              for (int k = lo > t ? lo : t; k < hi && k < t + kTile; ++k) {
                const int page = __ldcg(p.tables + (size_t)u.table * p.W + (k >> p.logP));
                if (page < 0 || page >= p.num_pages) continue;
                const size_t at =
                    (((((size_t)a.layer * p.num_pages + page) * p.Hkv + u.h) << p.logP) + (k & (p.P - 1))) * D + 32 * c;
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                  const float x = E4M3 ? e4m3x2_to_f32x2(p.v[at + e]).x
                                       : __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(p.v)[at + e] << 16);
                  if (!isfinite(x)) rr[e] = __float_as_uint(__uint_as_float(rr[e]) + x);
                }
              }
            }
          }
          if (!whole && !merge_now) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              o32[(8 * c + k) * kTile] = make_float4(__uint_as_float(rr[4 * k]), __uint_as_float(rr[4 * k + 1]),
                                                     __uint_as_float(rr[4 * k + 2]), __uint_as_float(rr[4 * k + 3]));
          } else if (merge_now) {
            merge_columns(c, rr);
          } else if (live) {
            float x[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k] = __uint_as_float(rr[k]) * inv;
            store_row32(o16 + 32 * c, x, out32);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
#pragma unroll
          for (int i = 0; i < L::kHalves; ++i) mbar_arrive(bar(misc->o_free[g * L::kHalves + i]));
        }
        if (!whole && !merge_now) {
          if (half == 0) *reinterpret_cast<float2*>(p.part_ml + ((size_t)u.part * kPartRows + g * kTile + row) * 2) =
              make_float2(m_run, ell);
          __threadfence();
          sync_group();
          if (speaks) {
            misc->last[g] = atomicAdd(ticket, 1) == last - first;
            if (misc->last[g]) *ticket = 0;
          }
          sync_group();
          if (misc->last[g]) {
            __threadfence();
            weigh();
            const uint32_t none[32] = {};
#pragma unroll 1
            for (int c = c_first; c < c_first + kC; ++c) merge_columns(c, none);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(misc->u_empty[uq]));
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == L::kWarpIssue) tmem_dealloc(tmem, 512);
  if (threadIdx.x == 0 && *abort)
    atomicOr(reinterpret_cast<unsigned*>(p.state + PST_ERROR), KVRING_PAGES_ERR_TIMEOUT);
}

template <int D, bool E4M3, bool BLK>
cudaError_t prepare_one() {
  using L = ChunkLayout<D, E4M3, BLK>;
  // the register split must fit what a block is launched with, or the warps
  // that ask for more would wait for ever
  cudaFuncAttributes at;
  const cudaError_t e = cudaFuncGetAttributes(&at, k_paged_chunk<D, E4M3, BLK>);
  if (e != cudaSuccess) return e;
  if (L::kRegsSoft && at.numRegs * L::kThreads <
                          L::kRegsSoft * L::kSoftThreads + L::kRegsRest * (L::kThreads - L::kSoftThreads))
    return cudaErrorInvalidConfiguration;
  return cudaFuncSetAttribute(k_paged_chunk<D, E4M3, BLK>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              ChunkLayout<D, E4M3, BLK>::kBytes);
}
template <int D, bool E4M3, bool BLK>
cudaError_t go(const PagesDev& p, const CUtensorMap* tmQ, const CUtensorMap* tmK, const CUtensorMap* tmV,
               const PagedAttn& a, cudaStream_t s) {
  return launch_pdl(k_paged_chunk<D, E4M3, BLK>, dim3((unsigned)a.ctas), dim3(ChunkLayout<D, E4M3, BLK>::kThreads),
                    ChunkLayout<D, E4M3, BLK>::kBytes, s, *tmQ, *tmK, *tmV, p, a);
}

}  // namespace

cudaError_t paged_chunk_prepare() {
  cudaError_t e = prepare_one<128, true, false>();
  if (e == cudaSuccess) e = prepare_one<128, true, true>();
  if (e == cudaSuccess) e = prepare_one<128, false, false>();
  if (e == cudaSuccess) e = prepare_one<64, true, false>();
  if (e == cudaSuccess) e = prepare_one<64, true, true>();
  if (e == cudaSuccess) e = prepare_one<64, false, false>();
  return e;
}

cudaError_t launch_paged_chunk(const PagesDev& p, const CUtensorMap* tmQ, const CUtensorMap* tmK,
                               const CUtensorMap* tmV, const PagedAttn& a, cudaStream_t s) {
  if (p.D == 128) {
    if (p.ks) return go<128, true, true>(p, tmQ, tmK, tmV, a, s);
    return p.e4m3 ? go<128, true, false>(p, tmQ, tmK, tmV, a, s) : go<128, false, false>(p, tmQ, tmK, tmV, a, s);
  }
  if (p.ks) return go<64, true, true>(p, tmQ, tmK, tmV, a, s);
  return p.e4m3 ? go<64, true, false>(p, tmQ, tmK, tmV, a, s) : go<64, false, false>(p, tmQ, tmK, tmV, a, s);
}

}  // namespace kvr
