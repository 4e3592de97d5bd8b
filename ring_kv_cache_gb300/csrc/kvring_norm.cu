// The step between two blocks of a transformer: the block's output (normed,
// gated, scaled) joins the residual stream, and the stream's norm, modulated,
// is the next block's input.
//
//   u  = y, or norm_p(y) * w_p
//   h' = h + residual_scale * gate[r] * u
//   x  = norm(h') * w * (1 + scale[r]) + shift[r]
//   rms(z) = z / sqrt(mean z^2 + eps), layer(z) = (z - mean z) / sqrt(var z + eps)
// Everything between reading and the one rounding of h' and of x is fp32 (x comes
// from the unrounded h'); a variance is summed from the differences, in a
// second pass over the registers, since E[z^2] - E[z]^2 would cancel.
//
// Bound by HBM: h and y are read once, h' and x written once.  A row's values stay
// in the registers of the threads that share it, eight per 16-byte load, so a norm
// costs one exchange (two for a layer norm).  The tables' rows come from L1, where
// the rows of an SM find them (a session's tokens lie together).  Measured (GB300):
// 16,384 rows of 5,120, bf16, post norm, gate, 16 rows of fp32 tables, 672 MB: 130 us,
// 5.2 TB/s; the instructions of a row's start and sums and the trips to L1 for 71 KB
// of tables and weight per row take what is left.  757 rows of 5,120, fp32 stream: 8.8 us; nine
// rows of 1,280: 2.0 us.  Measured and slower: persistent blocks with rows ahead in
// shared memory (cp.async), the tables from L1 (283 us: shared memory takes L1's
// room) or held in registers (208 us: eight columns a thread, 534 instructions a warp
// and row).
#include <cmath>
#include <type_traits>

#include "kvring_pages.cuh"

namespace kvr {
namespace {

struct NormDev {
  const void* h;
  const uint16_t* y;
  const void *gate, *scale, *shift;
  const int32_t* index;
  const uint16_t *post_w, *w;
  void* h_out;
  uint16_t* x_out;
  long long h_stride, y_stride, ho_stride, x_stride, mod_stride;
  int n, vecs;          // rows, groups of eight columns
  int mods, mods_f32;   // rows of the modulation tables, their type
  int post, norm;       // KVRING_NORM_*
  bool h_wide, ho_wide, m_wide;   // fp32 rows aligned to 32 bytes
  float eps, alpha, inv_width;
};

// Eight columns as four pairs: Blackwell multiplies and adds fp32 two at a time.
using Pairs = float2[4];
__device__ __forceinline__ void widen8(uint4 v, Pairs& x) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
}
__device__ __forceinline__ uint4 narrow8(const Pairs& x) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b2 = __floats2bfloat162_rn(x[i].x, x[i].y);
    o[i] = *reinterpret_cast<const uint32_t*>(&b2);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
// Eight columns of a row of either type, as they lie in memory.  fp32: one
// 32-byte access, so that a warp's lies in whole lines; two of 16 where the
// row is not aligned for it.  CACHED: tables, which other rows of the SM read too,
// through L1; else past it.  (Tables may be what the kernel before wrote, and L1 may hold
// lines of them from before that: all reads lie behind griddepcontrol.wait, which makes the
// memory operations of the kernels before visible, L1's lines included.)
template <bool F32>
struct Raw8;
template <>
struct Raw8<true> {
  float x[8];
  template <bool CACHED>
  __device__ __forceinline__ void load(const void* base, long long at, bool wide) {
    const float* p = static_cast<const float*>(base) + at;
    if (wide) {
      if constexpr (CACHED)
        asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
                     : "l"(p));
      else
        asm volatile("ld.global.cg.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
                     : "l"(p));
    } else {
      const float4* p4 = reinterpret_cast<const float4*>(p);
      const float4 a = CACHED ? p4[0] : __ldcg(p4), b = CACHED ? p4[1] : __ldcg(p4 + 1);
      x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
      x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
  }
  __device__ __forceinline__ void widen(Pairs& y) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = make_float2(x[2 * e], x[2 * e + 1]);
  }
};
template <>
struct Raw8<false> {
  uint4 v;
  template <bool CACHED>
  __device__ __forceinline__ void load(const void* base, long long at, bool) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at);
    v = CACHED ? *p : __ldcg(p);
  }
  __device__ __forceinline__ void widen(Pairs& x) const { widen8(v, x); }
};

constexpr int kRowWarps = 4;   // rows of a block where a warp is enough for one

// T threads share a row, NV groups of eight columns each (FULL: exactly).  F32,
// M32: the stream's and the tables' type.
template <int NV, bool FULL, bool F32, bool M32>
__global__ void __launch_bounds__(NV < 4 ? 1024 : (NV == 4 ? 512 : 416), 1)
    k_residual_norm(const NormDev a, const int T) {
  __shared__ float4 s_sum[4][8];
  const bool one_warp = T == 32;                 // then a block holds several rows
  const int tid = one_warp ? threadIdx.x & 31 : threadIdx.x, lane = threadIdx.x & 31;
  const int row = one_warp ? blockIdx.x * kRowWarps + (threadIdx.x >> 5) : blockIdx.x;
  if (!one_warp) {
    if (threadIdx.x < 32) reinterpret_cast<float4*>(s_sum)[threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
    __syncthreads();
  }
  int round = 0;
  // (a place of its own for each of the at most four sums of a row)
  auto sum_row = [&](float v) -> float {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (!one_warp) {
      if (lane == 0) reinterpret_cast<float*>(s_sum[round])[threadIdx.x >> 5] = v;
      __syncthreads();
      v = 0.f;
      for (int w = 0; w < T; w += 128) {
        const float4 p = s_sum[round][w >> 7];
        v += (p.x + p.y) + (p.z + p.w);
      }
      ++round;
    }
    return v;
  };
  griddep_wait();
  griddep_launch_dependents();
  if (row >= a.n) return;   // (whole warps, and no block-wide sum where a block has several rows)
  const int r = a.index ? __ldcg(a.index + row) : (a.mods > 1 ? row : 0);
  // A warp's groups lie side by side, so that their addresses differ by constants.
  const int v0 = (tid >> 5) * (32 * NV) + lane;
  auto each = [&](auto f) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (FULL || v0 + 32 * i < a.vecs) f(i, v0 + 32 * i);
  };
  Raw8<F32> hr[NV];
  uint4 yr[NV];
  Pairs z[NV];
  if (a.y) {
    const uint4* y = reinterpret_cast<const uint4*>(a.y + row * a.y_stride);
    each([&](int i, int v) { yr[i] = __ldcg(y + v); });
  }
  each([&](int i, int v) { hr[i].template load<false>(a.h, row * a.h_stride + 8 * v, a.h_wide); });
  const bool known = r >= 0 && r < a.mods;
  const long long mrow = known ? (long long)r * a.mod_stride : 0;
  const float nan = __int_as_float(0x7FFFFFFF);
  // z = f(z, table), every load on its way before the first value is used (no store
  // lies between, over which none would be moved).  Only here, behind the sums: the
  // tables are near, and the registers hold no more (five groups of a bf16 stream: 116
  // registers instead of 128 and spills, 130 us instead of 137; of an fp32 one, with
  // fp32 tables and places left empty, 128 and 8 bytes of spills).
  auto with_table = [&](const void* base, auto m32, long long at, bool wide, auto f) {
    Raw8<decltype(m32)::value> t[NV];
    each([&](int i, int v) { t[i].template load<true>(base, at + 8 * v, wide); });
    each([&](int i, int) {
      Pairs g;
      t[i].widen(g);
#pragma unroll
      for (int e = 0; e < 4; ++e) z[i][e] = f(z[i][e], g[e]);
    });
  };
  using Mods = std::integral_constant<bool, M32>;
  using Bf16 = std::false_type;
  auto times = [](float2 x, float2 y) { return __fmul2_rn(x, y); };
  // 1 / sqrt(mean square + eps), after the mean is taken away (layer); places
  // behind the row's end hold zeros
  auto standard = [&](int kind) -> float {
    if (kind == KVRING_NORM_LAYER) {
      float2 s = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) s = __fadd2_rn(s, z[i][e]);
      const float mean = sum_row(s.x + s.y) * -a.inv_width;
      each([&](int i, int) {
#pragma unroll
        for (int e = 0; e < 4; ++e) z[i][e] = __fadd2_rn(z[i][e], make_float2(mean, mean));
      });
    }
    float2 q = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) q = __ffma2_rn(z[i][e], z[i][e], q);
    return rsqrtf(sum_row(q.x + q.y) * a.inv_width + a.eps);
  };
  if constexpr (!FULL) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) z[i][e] = make_float2(0.f, 0.f);
  }
  if (a.y) {
    each([&](int i, int) { widen8(yr[i], z[i]); });
    float f = a.post != KVRING_NORM_NONE ? standard(a.post) : 1.0f;
    if (a.post_w) with_table(a.post_w, Bf16{}, 0, false, times);
    if (a.gate) with_table(a.gate, Mods{}, mrow, a.m_wide, times);
    f = known ? f * a.alpha : nan;
    each([&](int i, int) {
      Pairs h;
      hr[i].widen(h);
#pragma unroll
      for (int e = 0; e < 4; ++e) z[i][e] = __ffma2_rn(z[i][e], make_float2(f, f), h[e]);
    });
    if (a.h_out) {
      each([&](int i, int v) {
        if constexpr (F32) {
          float* p = static_cast<float*>(a.h_out) + row * a.ho_stride + 8 * v;
          if (a.ho_wide) {
            asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(z[i][0].x), "f"(z[i][0].y),
                         "f"(z[i][1].x), "f"(z[i][1].y), "f"(z[i][2].x), "f"(z[i][2].y), "f"(z[i][3].x), "f"(z[i][3].y)
                         : "memory");
          } else {
            reinterpret_cast<float4*>(p)[0] = make_float4(z[i][0].x, z[i][0].y, z[i][1].x, z[i][1].y);
            reinterpret_cast<float4*>(p)[1] = make_float4(z[i][2].x, z[i][2].y, z[i][3].x, z[i][3].y);
          }
        } else {
          reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.h_out) + row * a.ho_stride)[v] = narrow8(z[i]);
        }
      });
    }
  } else {
    each([&](int i, int) { hr[i].widen(z[i]); });
  }
  if (a.norm == KVRING_NORM_NONE) return;
  float f = standard(a.norm);
  if (!known) f = nan;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) z[i][e] = __fmul2_rn(z[i][e], make_float2(f, f));
  if (a.w) with_table(a.w, Bf16{}, 0, false, times);
  if (a.scale) with_table(a.scale, Mods{}, mrow, a.m_wide, [](float2 x, float2 y) { return __ffma2_rn(x, y, x); });
  if (a.shift) with_table(a.shift, Mods{}, mrow, a.m_wide, [](float2 x, float2 y) { return __fadd2_rn(x, y); });
  uint4* o = reinterpret_cast<uint4*>(a.x_out + row * a.x_stride);
  each([&](int i, int v) { o[v] = narrow8(z[i]); });
}

template <int NV, bool FULL>
cudaError_t go(const NormDev& d, bool f32, int T, cudaStream_t s) {
  const int rows = T == 32 ? kRowWarps : 1;   // of a block
  const dim3 grid((unsigned)((d.n - 1) / rows + 1)), block((unsigned)(T * rows));
  if (f32)
    return d.mods_f32 ? launch_pdl(k_residual_norm<NV, FULL, true, true>, grid, block, 0, s, d, T)
                      : launch_pdl(k_residual_norm<NV, FULL, true, false>, grid, block, 0, s, d, T);
  return d.mods_f32 ? launch_pdl(k_residual_norm<NV, FULL, false, true>, grid, block, 0, s, d, T)
                    : launch_pdl(k_residual_norm<NV, FULL, false, false>, grid, block, 0, s, d, T);
}

// Few rows: as many groups of eight columns as 1,024 threads on each of this card's 152 SMs take at
// one a thread.  (bf16 rows of 5,120: 150 rows 3.3 us, 243, the last below the border, 5.3 us, 244,
// with five, 3.7 us: above one wave of the former the border could lie lower.)
constexpr long long kFewGroups = 152 * 1024;

cudaError_t launch_residual_norm(const NormDev& d, bool f32, cudaStream_t s) {
  // Groups of eight columns a thread.  Few rows: one, for latency (9 rows of 1,280:
  // 2.0 us, with five 2.4).  Else many, for a row's fixed instructions are then
  // shared by more columns (16,384 bf16 rows of 5,120, one: 287 us, two: 153, four:
  // 154, five: 130; 757 fp32 rows, whose groups take more registers, two and
  // four: 8.8, five: 9.4), unless fewer leave fewer places empty.
  auto threads = [&](int nv) { return (d.vecs + 32 * nv - 1) / (32 * nv) * 32; };
  int nv = f32 ? 4 : 5;
  for (int k : {f32 ? 5 : 4, 2})
    if (threads(k) * k < threads(nv) * nv) nv = k;
  if (d.vecs <= 1024 && (long long)d.n * d.vecs <= kFewGroups) nv = 1;
  const int T = threads(nv);
  const bool full = d.vecs == T * nv;
  switch (nv) {
    case 1: return full ? go<1, true>(d, f32, T, s) : go<1, false>(d, f32, T, s);
    case 2: return full ? go<2, true>(d, f32, T, s) : go<2, false>(d, f32, T, s);
    case 4: return full ? go<4, true>(d, f32, T, s) : go<4, false>(d, f32, T, s);
    default: return full ? go<5, true>(d, f32, T, s) : go<5, false>(d, f32, T, s);
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The bytes of n rows of `width` elements.
struct Span {
  const void* p;
  size_t bytes;
};
Span rows_of(const void* p, int64_t n, int64_t stride, int64_t width, int64_t size) {
  return Span{p, p ? (size_t)(((n - 1) * stride + width) * size) : 0};
}
bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
}

}  // namespace
}  // namespace kvr

extern "C" kvring_status kvring_residual_norm(const kvring_norm_config* c, const void* h, const void* y,
                                              const void* gate, const void* scale, const void* shift,
                                              const int32_t* mod_index, const void* post_weight, const void* weight,
                                              void* h_out, void* x_out, void* stream) {
  using namespace kvr;
  auto type_ok = [](int t) { return t == KVRING_OUT_F32 || t == KVRING_OUT_BF16; };
  auto norm_ok = [](int k) { return k >= KVRING_NORM_NONE && k <= KVRING_NORM_LAYER; };
  if (!c || !h || c->num_tokens < 1 || c->width < 8 || c->width % 8 || c->width > KVRING_NORM_MAX_WIDTH ||
      !type_ok(c->stream_dtype) || !type_ok(c->mod_dtype) || !norm_ok(c->post_norm) || !norm_ok(c->norm) ||
      c->reserved != 0)
    return KVRING_ERR_INVALID_ARG;
  if (!(c->eps >= 0.f) || !std::isfinite(c->eps) || !std::isfinite(c->residual_scale)) return KVRING_ERR_INVALID_ARG;
  const bool tables = gate || scale || shift;
  // what the call would compute from, or into, and what it would not
  if (!y && (h_out || gate || post_weight || c->post_norm != KVRING_NORM_NONE)) return KVRING_ERR_INVALID_ARG;
  if (y && !h_out && !x_out) return KVRING_ERR_INVALID_ARG;
  if (post_weight && c->post_norm == KVRING_NORM_NONE) return KVRING_ERR_INVALID_ARG;
  if ((c->norm == KVRING_NORM_NONE) != (x_out == nullptr)) return KVRING_ERR_INVALID_ARG;
  if (c->norm == KVRING_NORM_NONE && (weight || scale || shift)) return KVRING_ERR_INVALID_ARG;
  if (tables ? c->mod_rows < 1 : mod_index != nullptr) return KVRING_ERR_INVALID_ARG;
  if (tables && !mod_index && c->mod_rows != 1 && c->mod_rows != c->num_tokens) return KVRING_ERR_INVALID_ARG;
  for (const void* p : {h, y, gate, scale, shift, post_weight, weight, (const void*)h_out, (const void*)x_out})
    if (!aligned16(p)) return KVRING_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(mod_index) & 3) return KVRING_ERR_INVALID_ARG;
  const int64_t n = c->num_tokens, w = c->width, most = (int64_t)1 << 28;
  auto stride_ok = [&](const void* p, int64_t s, int64_t rows) {
    return !p || (s % 8 == 0 && s <= most && (s >= w || (rows == 1 && s >= 0)));
  };
  if (!stride_ok(h, c->h_stride, n) || !stride_ok(y, c->y_stride, n) || !stride_ok(h_out, c->h_out_stride, n) ||
      !stride_ok(x_out, c->x_out_stride, n) || !stride_ok(tables ? h : nullptr, c->mod_stride, c->mod_rows))
    return KVRING_ERR_INVALID_ARG;
  const int64_t hs = c->stream_dtype == KVRING_OUT_F32 ? 4 : 2, ms = c->mod_dtype == KVRING_OUT_F32 ? 4 : 2;
  const Span in_h = rows_of(h, n, c->h_stride, w, hs), out_h = rows_of(h_out, n, c->h_out_stride, w, hs);
  const Span out_x = rows_of(x_out, n, c->x_out_stride, w, 2);
  const int64_t m = tables ? c->mod_rows : 1;
  const Span inputs[] = {rows_of(y, n, c->y_stride, w, 2),      rows_of(gate, m, c->mod_stride, w, ms),
                         rows_of(scale, m, c->mod_stride, w, ms), rows_of(shift, m, c->mod_stride, w, ms),
                         rows_of(post_weight, 1, w, w, 2),      rows_of(weight, 1, w, w, 2),
                         Span{mod_index, mod_index ? (size_t)n * 4 : 0}};
  // the stream may be updated in place; nothing else may lie over a result
  const bool in_place = h_out == h && (c->h_out_stride == c->h_stride || n == 1);
  if ((!in_place && overlap(out_h, in_h)) || overlap(out_x, in_h) || overlap(out_x, out_h)) return KVRING_ERR_INVALID_ARG;
  for (const Span& in : inputs)
    if (overlap(out_h, in) || overlap(out_x, in)) return KVRING_ERR_INVALID_ARG;
  NormDev d{};
  d.h = h;
  d.y = static_cast<const uint16_t*>(y);
  d.gate = gate;
  d.scale = scale;
  d.shift = shift;
  d.index = mod_index;
  d.post_w = static_cast<const uint16_t*>(post_weight);
  d.w = static_cast<const uint16_t*>(weight);
  d.h_out = h_out;
  d.x_out = static_cast<uint16_t*>(x_out);
  d.h_stride = c->h_stride;
  d.y_stride = c->y_stride;
  d.ho_stride = c->h_out_stride;
  d.x_stride = c->x_out_stride;
  d.mod_stride = c->mod_stride;
  d.n = c->num_tokens;
  d.vecs = c->width / 8;
  // fp32 rows of 32-byte groups (strides are multiples of them)
  auto wide = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31) == 0; };
  d.h_wide = wide(h);
  d.ho_wide = wide(h_out);
  d.m_wide = wide(gate) && wide(scale) && wide(shift);
  d.mods = tables ? c->mod_rows : 1;
  d.mods_f32 = c->mod_dtype == KVRING_OUT_F32;
  d.post = c->post_norm;
  d.norm = c->norm;
  d.eps = c->eps;
  d.alpha = c->residual_scale;
  d.inv_width = 1.0f / (float)c->width;
  struct Ctx {
    const NormDev* d;
    bool f32;
    cudaStream_t s;
  } ctx{&d, c->stream_dtype == KVRING_OUT_F32, static_cast<cudaStream_t>(stream)};
  return launch_recorded(
      ctx.s, [](void* p) {
        const Ctx* x = static_cast<const Ctx*>(p);
        return launch_residual_norm(*x->d, x->f32, x->s);
      }, &ctx, h_out, out_h.bytes, x_out, out_x.bytes);
}
