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
// costs one exchange (two for a layer norm).
#include <cmath>

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
  float eps, alpha, inv_width;
};

__device__ __forceinline__ void widen8(uint4 v, float (&x)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 narrow8(const float (&x)[8]) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b2 = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    o[i] = *reinterpret_cast<const uint32_t*>(&b2);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
// Eight values of a table of either type.
__device__ __forceinline__ void table8(const void* base, long long at, bool f32, float (&x)[8]) {
  if (f32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    const float4 a = p[0], b = p[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    widen8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at), x);
  }
}

// T threads share a row, NV groups of eight columns each; F32: the stream's type.
template <int T, int NV, bool F32>
__global__ void __launch_bounds__(T < 128 ? 128 : T) k_residual_norm(const NormDev a) {
  constexpr int kRows = T < 128 ? 128 / T : 1;   // rows of a block
  __shared__ float s_sum[4][T / 32];
  const int tid = threadIdx.x % T, lane = threadIdx.x & 31;
  const int row = blockIdx.x * kRows + (kRows > 1 ? (int)threadIdx.x / T : 0);
  int round = 0;
  auto sum_row = [&](float v) -> float {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if constexpr (T > 32) {   // (a place for each of the at most four sums of a row)
      if (lane == 0) s_sum[round][tid >> 5] = v;
      __syncthreads();
      v = 0.f;
#pragma unroll
      for (int w = 0; w < T / 32; ++w) v += s_sum[round][w];
      ++round;
    }
    return v;
  };
  griddep_wait();
  griddep_launch_dependents();
  if (row >= a.n) return;   // (whole warps, and no block-wide sum where a block has several rows)
  const int r = a.index ? __ldcg(a.index + row) : (a.mods > 1 ? row : 0);
  const bool known = r >= 0 && r < a.mods;
  const long long mrow = known ? (long long)r * a.mod_stride : 0;
  float z[NV][8], u[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = i * T + tid;
#pragma unroll
    for (int e = 0; e < 8; ++e) z[i][e] = u[i][e] = 0.f;
    if (v >= a.vecs) continue;
    if constexpr (F32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.h) + row * a.h_stride) + 2 * v;
      const float4 b = __ldcg(p), c = __ldcg(p + 1);
      z[i][0] = b.x, z[i][1] = b.y, z[i][2] = b.z, z[i][3] = b.w;
      z[i][4] = c.x, z[i][5] = c.y, z[i][6] = c.z, z[i][7] = c.w;
    } else {
      widen8(__ldcg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.h) + row * a.h_stride) + v), z[i]);
    }
    if (a.y) widen8(__ldcg(reinterpret_cast<const uint4*>(a.y + row * a.y_stride) + v), u[i]);
  }
  // x - mean (layer) and 1 / sqrt(mean square + eps) of a row
  auto standard = [&](float (&x)[NV][8], int kind) -> float {
    if (kind == KVRING_NORM_LAYER) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) s += x[i][e];
      const float mean = sum_row(s) * a.inv_width;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i * T + tid < a.vecs) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[i][e] -= mean;
        }
    }
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) q = fmaf(x[i][e], x[i][e], q);
    return rsqrtf(sum_row(q) * a.inv_width + a.eps);
  };
  if (a.y) {
    const float f = a.post != KVRING_NORM_NONE ? standard(u, a.post) : 1.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = i * T + tid;
      if (v >= a.vecs) continue;
      float g[8];
      if (a.post_w) {
        widen8(reinterpret_cast<const uint4*>(a.post_w)[v], g);
#pragma unroll
        for (int e = 0; e < 8; ++e) u[i][e] *= g[e];
      }
      if (a.gate) {
        table8(a.gate, mrow + 8 * v, a.mods_f32, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) u[i][e] *= g[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) z[i][e] = fmaf(u[i][e] * f, a.alpha, z[i][e]);
      if (!known) {
#pragma unroll
        for (int e = 0; e < 8; ++e) z[i][e] = __int_as_float(0x7FFFFFFF);
      }
      if (!a.h_out) continue;
      if constexpr (F32) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(a.h_out) + row * a.ho_stride) + 2 * v;
        p[0] = make_float4(z[i][0], z[i][1], z[i][2], z[i][3]);
        p[1] = make_float4(z[i][4], z[i][5], z[i][6], z[i][7]);
      } else {
        reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.h_out) + row * a.ho_stride)[v] = narrow8(z[i]);
      }
    }
  }
  if (a.norm == KVRING_NORM_NONE) return;
  const float f = standard(z, a.norm);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = i * T + tid;
    if (v >= a.vecs) continue;
    float g[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) z[i][e] *= f;
    if (a.w) {
      widen8(reinterpret_cast<const uint4*>(a.w)[v], g);
#pragma unroll
      for (int e = 0; e < 8; ++e) z[i][e] *= g[e];
    }
    if (a.scale) {
      table8(a.scale, mrow + 8 * v, a.mods_f32, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) z[i][e] *= 1.0f + g[e];
    }
    if (a.shift) {
      table8(a.shift, mrow + 8 * v, a.mods_f32, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) z[i][e] += g[e];
    }
    if (!known) {
#pragma unroll
      for (int e = 0; e < 8; ++e) z[i][e] = __int_as_float(0x7FFFFFFF);
    }
    reinterpret_cast<uint4*>(a.x_out + row * a.x_stride)[v] = narrow8(z[i]);
  }
}

template <int T, int NV>
cudaError_t go(const NormDev& d, bool f32, cudaStream_t s) {
  constexpr int kRows = T < 128 ? 128 / T : 1;
  const dim3 grid((unsigned)((d.n - 1) / kRows + 1)), block(T < 128 ? 128 : T);
  return f32 ? launch_pdl(k_residual_norm<T, NV, true>, grid, block, 0, s, d)
             : launch_pdl(k_residual_norm<T, NV, false>, grid, block, 0, s, d);
}

cudaError_t launch_residual_norm(const NormDev& d, bool f32, cudaStream_t s) {
  if (d.vecs <= 32) return go<32, 1>(d, f32, s);
  if (d.vecs <= 96) return go<32, 3>(d, f32, s);
  if (d.vecs <= 160) return go<32, 5>(d, f32, s);
  if (d.vecs <= 384) return go<128, 3>(d, f32, s);
  if (d.vecs <= 640) return go<128, 5>(d, f32, s);
  if (d.vecs <= 1280) return go<256, 5>(d, f32, s);
  return go<512, 4>(d, f32, s);
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
  const int64_t n = c->num_tokens, w = c->width, most = (int64_t)1 << 32;
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
