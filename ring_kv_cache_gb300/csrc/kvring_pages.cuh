// Device-side view of a paged cache and the launchers of its kernels.
#pragma once

#include "kvring_internal.cuh"

namespace kvr {

// State words beyond the public ones (KVRING_PAGES_STATE_*).
enum : int {
  PST_FREE = KVRING_PAGES_STATE_FREE,
  PST_ERROR = KVRING_PAGES_STATE_ERROR,
  PST_PLANNED = KVRING_PAGES_STATE_PLANNED,
  PST_REQUESTS = KVRING_PAGES_STATE_REQUESTS,
  PST_TOKENS = KVRING_PAGES_STATE_TOKENS,
  PST_TAKEN = KVRING_PAGES_STATE_TAKEN,
  PST_WORDS_ALLOC = 16,
};

constexpr int kMaxRows = 4096;       // rows of the block tables
constexpr int kPagedMaxCtas = 160;   // CTAs of an attention launch (workspace slots: two each)
constexpr int kPartRows = 256;       // query rows of a workspace slot of the chunk kernel
// Query rows of a unit of the kernel for few rows, one m = 16 tile, and the most
// a request may have for it.  Beyond, the chunk kernel takes the request:
// requests of 16 to 32 rows take 173 us so, and took 324 us with two m = 16 tiles
// per warp (64 requests of up to 8,192 tokens, 32/8 heads x 128, bf16; E4M3 178
// and 346); requests of 8 to 16 rows 166 us there and 161 us here (136 and 131).
constexpr int kFewRows = 16;

// Both attention kernels raise a row's running maximum only when a score exceeds
// it by more than kRaise (log2 units), so that sums are rescaled about once per
// unit and not in every other tile, and probabilities carry 2^kShift relative to
// it.  Over an E4M3 cache they become f16: the largest is then 2^15, and those down to
// 2^-21 of the maximum stay normal numbers.  Over a bf16 cache the probabilities,
// which become bf16, are at most 2^-24, so that the sums of 2^24 tokens' weighted
// values stay finite as long as the values are; what a row weighs with less than 2^-94 of
// its maximum counts as 0.
constexpr float kRaise = 8.0f;
template <bool E4M3>
constexpr float kShift = E4M3 ? 7.0f : -32.0f;

struct PagesDev {
  uint8_t* k;             // [L][num_pages][Hkv][P][D]
  uint8_t* v;
  float* scales;          // [L][4][Hkv]
  int32_t* lens;          // [R]
  int32_t* tables;        // [R][W]
  int32_t* free_pages;    // [num_pages]
  int32_t* state;         // [PST_WORDS_ALLOC]
  int32_t* rows;          // [R] the step's rows
  int32_t* cu;            // [R + 1]
  int32_t* klen;          // [R]
  int32_t* pos;           // [max_tokens]
  int32_t* slots;         // [max_tokens]
  const float* table;     // [max_pos][D/2][2] fp32 (cos, sin)
  float* part_o;          // [2 * kPagedMaxCtas][kPartRows x D] attention partials, laid out by the kernel
  float* part_ml;         // [2 * kPagedMaxCtas][kPartRows][2] their running maxima and sums
  int32_t* tickets;       // [2 * kPagedMaxCtas] arrivals per split unit (0 between calls)
  float* few_o;           // the same of the kernel for few rows: [2 * kPagedMaxCtas][kFewRows][D]
  float* few_ml;          // [2 * kPagedMaxCtas][kFewRows][2]
  int32_t* few_tickets;   // [kPagedMaxCtas]; behind `tickets`
  int Hq, Hkv, D, L, P, logP, num_pages, R, W, max_tokens;
  int e4m3;               // cache type
  int halves;             // rotation pairs (i, i + d/2)
  uint8_t* ks;            // [L][num_pages][Hkv][P/16] exponents of block scales (NULL: scales per head)
  uint8_t* vs;
  int pt, py;             // 3-D RoPE: pairs of t and y (pt = 0: 1-D)
  int max_pos;            // rows of `table`: W * P, or as many as coordinates go
};

// Exponents (biased by 127) that a block's scale may have; others are read as the
// nearest of these.  With both products' range in mind: a weight 2^(score + e - m)
// that counts is never lost beside the normaliser's 2^(score - m).
constexpr int kMinExp = 127 - 40, kMaxExp = 127 + 40;
// The most a query row's factor may be over blocks.  A raw score is below 4 x 448 x 128 <
// 2^18 (f16 queries, codes), so with a key's scale of 2^40 it stays below 2^127: scores, and
// the differences of two, are finite.  (With 2^87 the factor alone was: raw scores from 2 on over
// the largest scale made inf, and inf - inf NaN.)  Rows beyond are read with this factor: their
// scores keep their order, and two that fp32 tells apart beside a raw score of 1 differ by
// 2^69 2^-40 2^-24 = 2^5 at least, over the smallest scale, so such a row is one-hot all the same.
constexpr float kMostFactor = 0x1p69f;

struct PagedAttn {
  const uint16_t* q;
  uint16_t* out;
  long long q_stride;     // elements between tokens
  int T;                  // tokens of q and out
  int layer;
  int causal, window;
  float sm_log2;          // softmax scale * log2(e)
  int min_rows, max_rows; // a kernel takes requests with min_rows < rows <= max_rows (rows = tokens * G)
  int ctas;
  int min_tiles;          // a CTA's range holds at least this many tiles
  unsigned long long wait_ns;
  int debug_stall;
  int beside;             // the kernel for few rows runs beside the chunk kernel of the same call
};

cudaError_t pages_prepare();
cudaError_t launch_pages_table(const PagesDev& p, float* table, const double* theta_host, cudaStream_t s);
cudaError_t launch_pages_reset(const PagesDev& p, int n_free, bool fill, cudaStream_t s);
cudaError_t launch_pages_scales(const PagesDev& p, int layer, const float* sk, const float* sv, cudaStream_t s);
cudaError_t launch_pages_plan(const PagesDev& p, const int32_t* rows, const int32_t* nt, int B, int T, int max_new,
                              cudaStream_t s);
cudaError_t launch_pages_commit(const PagesDev& p, cudaStream_t s);
cudaError_t launch_pages_release(const PagesDev& p, const int32_t* rows, int B, cudaStream_t s);

struct PagesWrite {
  const uint16_t *q, *k, *v;
  long long q_stride, k_stride, v_stride;
  const uint16_t *qw, *kw;
  uint16_t* q_out;
  const int32_t* coords;  // [T][3], 3-D RoPE
  float eps;
  int T, layer;
  int kv_blocks;          // blocks of keys and values per 16 tokens (block scales)
};
cudaError_t launch_pages_write(const PagesDev& p, const PagesWrite& w, int sm_count, cudaStream_t s);

// Attention: few query rows per request (units of 16 rows) ...
cudaError_t paged_few_prepare();
cudaError_t launch_paged_few(const PagesDev& p, const CUtensorMap* tmK, const CUtensorMap* tmV, const PagedAttn& a,
                             cudaStream_t s);

// ... and many (chunks).
cudaError_t paged_chunk_prepare();
cudaError_t launch_paged_chunk(const PagesDev& p, const CUtensorMap* tmQ, const CUtensorMap* tmK,
                               const CUtensorMap* tmV, const PagedAttn& a, cudaStream_t s);

// Four E4M3 codes (low byte first) to two f16 pairs, exactly.
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=&r"(lo), "=r"(hi)
      : "r"(w));
}

// The power of two that a query row is divided by on its way to f16, and its
// inverse, from the row's largest exponent field: its largest value then lies in [1, 2) (in [2, 4) for the
// last exponent, whose factor's inverse would not be a normal number).
// Infinities and NaN (255) keep a factor of 1 and stay what they are, and so does a
// row of zeros.
__device__ __forceinline__ void query_factor(uint32_t em, float& up, float& down) {
  const bool plain = em == 0 || em == 255;
  const uint32_t e = min(em, 253u);
  up = plain ? 1.0f : __uint_as_float(e << 23);
  down = plain ? 1.0f : __uint_as_float((254u - e) << 23);
}

// One launch with the programmatic-stream-serialisation attribute.
template <typename... KP, typename... A>
inline cudaError_t launch_pdl(void (*kernel)(KP...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KP>(args)...);
}

// Defined with the ring's host code: the record of caller buffers written by
// kernels that may still run (see kvring_host.cu).  Runs `launch` under its
// lock and records the written ranges.
kvring_status launch_recorded(cudaStream_t s, cudaError_t (*launch)(void*), void* ctx, const void* a, size_t a_bytes,
                              const void* b, size_t b_bytes);
typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encode_tiled();

}  // namespace kvr
