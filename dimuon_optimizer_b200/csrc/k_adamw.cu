// AdamW over many tensors in one launch, moments in fp32 or in 8 bits.
//
// Per element (include/dimuon.h): m' = b1 m + (1 - b1) g, v' = b2 v + (1 - b2) g^2,
// W' = (1 - lr wd) W - lr (m' / bc1) / (sqrt(v' / bc2) + eps).  One pass: every
// operand is read once and written once (bf16 weights and gradients: 22 bytes
// per element with fp32 moments, 10.1 with 8-bit ones), so HBM bounds it.
#include <cuda_fp8.h>

#include "dm_common.cuh"
#include "dm_many.h"

namespace dm {
namespace {

constexpr int THREADS = 256;

__device__ __forceinline__ bool finite_f(float x) {
  return (__float_as_uint(x) & 0x7fffffffu) < 0x7f800000u;
}

// What one tensor's update needs besides its data.
struct Coef {
  float gs;            // gradient scale
  float b1, c1, b2, c2, eps;
  float isb2;          // 1 / sqrt(1 - b2^t)
  float step;          // lr / (1 - b1^t)
  float decay;         // 1 - lr wd
  uint32_t step_key;
  bool skip;
};

// Reads the step's device values; the status word is written by one thread
// of a host-counted step (adamw_scalars has written it otherwise).
__device__ __forceinline__ Coef coefficients(const AdamwHead& h, float lr_mult, float decay_mult) {
  Coef c;
  c.gs = h.grad_scale ? *h.grad_scale : 1.f;
  const float lr0 = h.lr_dev ? *h.lr_dev : h.lr;
  const AdamwScalars sc = h.dev ? *h.dev : h.sc;
  c.skip = h.dev ? sc.skip != 0 : !(finite_f(c.gs) && finite_f(lr0));
  c.b1 = h.b1; c.c1 = h.c1; c.b2 = h.b2; c.c2 = h.c2; c.eps = h.eps;
  const float lr = lr0 * lr_mult;
  c.step = lr * sc.inv_bc1;
  c.decay = fmaf(-lr, h.wd * decay_mult, 1.f);
  c.isb2 = sc.inv_sqrt_bc2;
  c.step_key = sc.step_key;
  if (h.write_status && blockIdx.x == 0 && threadIdx.x == 0)
    *h.status = c.skip ? ST_NONFINITE : ST_OK;
  return c;
}

// The moments, each product and sum rounded to fp32 by itself: the
// stochastic rounding of the 8-bit form compares these bits with its noise,
// so their value is part of the operator's definition.
__device__ __forceinline__ void moments(const Coef& c, float g, float& m, float& v) {
  g = __fmul_rn(g, c.gs);
  m = __fadd_rn(__fmul_rn(m, c.b1), __fmul_rn(g, c.c1));
  v = __fadd_rn(__fmul_rn(v, c.b2), __fmul_rn(__fmul_rn(g, g), c.c2));
}

// The new weight; square root and division are the approximate ones (2 ulp:
// they touch the update only, which is lr / |W| of the weight).
__device__ __forceinline__ float updated(const Coef& c, float w, float m, float v) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  const float d = fmaf(r, c.isb2, c.eps);
  return fmaf(w, c.decay, -c.step * __fdividef(m, d));
}

// ---------------------------------------------------------------------------
// fp32 moments.  A thread takes 8 consecutive elements; group k of a tensor
// covers elements 8k - shift .. 8k - shift + 7, so that whole groups are
// 32-byte aligned in fp32 (16 in bf16) whatever the tensor's offset.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void adamw32_elem(void* W, const void* G, float* M, float* V, int wdt,
                                             int gdt, int64_t e, const Coef& c) {
  float m = M[e], v = V[e];
  moments(c, ld_elem(G, e, gdt), m, v);
  const float w = updated(c, ld_elem(W, e, wdt), m, v);
  M[e] = m;
  V[e] = v;
  st_elem(W, e, wdt, w);
}

template <int N>
__global__ void __launch_bounds__(THREADS) adamw32_step(const __grid_constant__ Adamw32Params<N> p) {
  const int tile = blockIdx.x;
  const int t = find_group(p.starts, p.h.count, tile);
  const Coef c = coefficients(p.h, p.lr_mult[t], p.decay_mult[t]);
  if (c.skip) return;
  const int flags = p.flags[t];
  const int wdt = flags & MF_W_FP32 ? DT_FP32 : DT_BF16, gdt = flags & MF_G_FP32 ? DT_FP32 : DT_BF16;
  const int64_t n = p.n[t];
  void* W = p.W[t];
  const void* G = p.G[t];
  float* M = p.M[t];
  float* V = p.V[t];
  const int64_t base = (int64_t)(tile - p.starts[t]) * ADAMW32_TILE;
  if (!(flags & MF_VEC)) {
    for (int q = 0; q < 8; ++q) {
      const int64_t e = base + q * THREADS + threadIdx.x;
      if (e < n) adamw32_elem(W, G, M, V, wdt, gdt, e, c);
    }
    return;
  }
  const int64_t e = base + threadIdx.x * 8 - ((flags >> MF_SHIFT_BIT) & 7);
  if (e < 0 || e + 8 > n) {
    for (int q = 0; q < 8; ++q)
      if (e + q >= 0 && e + q < n) adamw32_elem(W, G, M, V, wdt, gdt, e + q, c);
    return;
  }
  float g[8], m[8], v[8], w[8];
  ld8(G, e, gdt, g);
  ld8(M, e, DT_FP32, m);
  ld8(V, e, DT_FP32, v);
  ld8(W, e, wdt, w);
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    moments(c, g[q], m[q], v[q]);
    w[q] = updated(c, w[q], m[q], v[q]);
  }
  st8(M, e, DT_FP32, m);
  st8(V, e, DT_FP32, v);
  st8(W, e, wdt, w);
}

// ---------------------------------------------------------------------------
// 8-bit moments.  A thread takes 16 consecutive elements, so 8 threads of a
// warp share the scale of a block of 128.
// ---------------------------------------------------------------------------
// Smallest power of two s >= 2^-110 with the magnitude of `bits` <= 1.75 2^top s,
// and its inverse; NaN for a non-finite magnitude.
__device__ __forceinline__ void block_scale(uint32_t bits, int top, float& s, float& inv) {
  const int e = max((int)((bits + 0x1FFFFFu) >> 23) - top, 17);
  s = bits < 0x7f800000u ? __uint_as_float((uint32_t)e << 23) : __uint_as_float(0x7fffffffu);
  inv = __uint_as_float((uint32_t)(254 - e) << 23);
}

// Code of x >= 0 (x at most the format's largest value) with MAN mantissa bits
// and exponent bias BIAS.  The bits of an fp32 number below the code's last
// place are its remainder, so adding noise there and cutting off rounds up
// with the remainder's probability.  Below the least normal number L, x + L
// lies on the spacing of the subnormal codes.
template <int MAN, int BIAS>
__device__ __forceinline__ uint32_t encode(float x, uint32_t noise) {
  constexpr float L = BIAS == 7 ? 0.015625f : 6.103515625e-05f;  // 2^(1 - BIAS)
  const bool small = x < L;
  const float y = small ? x + L : x;
  const uint32_t off = (uint32_t)((127 - BIAS) << MAN) + (small ? (1u << MAN) : 0u);
  return ((__float_as_uint(y) + noise) >> (23 - MAN)) - off;
}

__device__ __forceinline__ uint32_t group_max(uint32_t v) {  // over 8 neighbouring lanes
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

template <int N>
__global__ void __launch_bounds__(THREADS) adamw8_step(const __grid_constant__ Adamw8Params<N> p) {
  const int tile = blockIdx.x;
  const int t = find_group(p.starts, p.h.count, tile);
  const Coef c = coefficients(p.h, p.lr_mult[t], p.decay_mult[t]);
  if (c.skip) return;
  const int flags = (int)(p.n_flags[t] & 0xff);
  const int64_t n = p.n_flags[t] >> 8;
  const int wdt = flags & MF_W_FP32 ? DT_FP32 : DT_BF16, gdt = flags & MF_G_FP32 ? DT_FP32 : DT_BF16;
  void* W = p.W[t];
  const void* G = p.G[t];
  uint8_t* M = reinterpret_cast<uint8_t*>(p.M[t]);
  uint8_t* V = reinterpret_cast<uint8_t*>(p.V[t]);
  const int64_t e = (int64_t)(tile - p.starts[t]) * ADAMW8_TILE + threadIdx.x * 16;
  const int64_t blk = e / 128;
  const bool full = (flags & MF_VEC) && e + 16 <= n;
  const int cnt = e >= n ? 0 : (int)min((int64_t)16, n - e);

  float g[16], w[16], m[16], v[16];
  uint32_t cm[4] = {0, 0, 0, 0}, cv[4] = {0, 0, 0, 0};
  float s1 = 0.f, s2 = 0.f;
  if (cnt) {
    s1 = p.S1[t][blk];
    s2 = p.S2[t][blk];
  }
  if (full) {
    *reinterpret_cast<uint4*>(cm) = *reinterpret_cast<const uint4*>(M + e);
    *reinterpret_cast<uint4*>(cv) = *reinterpret_cast<const uint4*>(V + e);
    ld8(G, e, gdt, g);
    ld8(G, e + 8, gdt, g + 8);
    ld8(W, e, wdt, w);
    ld8(W, e + 8, wdt, w + 8);
  } else {
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      g[q] = w[q] = 0.f;
      if (q < cnt) {
        cm[q / 4] |= (uint32_t)M[e + q] << (8 * (q % 4));
        cv[q / 4] |= (uint32_t)V[e + q] << (8 * (q % 4));
        g[q] = ld_elem(G, e + q, gdt);
        w[q] = ld_elem(W, e + q, wdt);
      }
    }
  }
  uint32_t top1 = 0, top2 = 0;
#pragma unroll
  for (int q = 0; q < 16; q += 2) {
    const uint32_t a = cm[q / 4] >> (8 * (q % 4)), b = cv[q / 4] >> (8 * (q % 4));
    const float2 fm = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)a, __NV_E4M3)));
    const float2 fv = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)b, __NV_E5M2)));
    m[q] = fm.x * s1;
    m[q + 1] = fm.y * s1;
    v[q] = fv.x * s2;
    v[q + 1] = fv.y * s2;
#pragma unroll
    for (int i = q; i < q + 2; ++i) {
      if (i >= cnt) { m[i] = v[i] = 0.f; }  // behind the tensor's end (g = 0 there)
      moments(c, g[i], m[i], v[i]);
      w[i] = updated(c, w[i], m[i], v[i]);
      top1 = max(top1, __float_as_uint(m[i]) & 0x7fffffffu);
      top2 = max(top2, __float_as_uint(v[i]) & 0x7fffffffu);
    }
  }
  top1 = group_max(top1);
  top2 = group_max(top2);
  float i1, i2;
  block_scale(top1, 8, s1, i1);
  block_scale(top2, 15, s2, i2);
  const uint64_t group = (uint64_t)e >> 4;
  const uint32_t key = many_mix(many_mix(c.step_key + p.index[t]) + (uint32_t)(group >> 32));
  const uint32_t h0 = many_mix(key ^ (uint32_t)group);
#pragma unroll
  for (int q = 0; q < 4; ++q) cm[q] = cv[q] = 0;
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    uint32_t h = (h0 + (uint32_t)q * MANY_GOLDEN) * 0x7FEB352Du;
    h = (h ^ (h >> 15)) * 0x846CA68Bu;
    h ^= h >> 16;
    const uint32_t a = encode<3, 7>(fabsf(m[q]) * i1, (h >> 16) << 4) |
                       (__float_as_uint(m[q]) >> 31 << 7);
    uint32_t b = encode<2, 15>(v[q] * i2, (h & 0xffffu) << 5);
    if (v[q] > 0.f && b == 0) b = 1;
    cm[q / 4] |= (a & 0xffu) << (8 * (q % 4));
    cv[q / 4] |= (b & 0xffu) << (8 * (q % 4));
  }
  if (full) {
    *reinterpret_cast<uint4*>(M + e) = *reinterpret_cast<const uint4*>(cm);
    *reinterpret_cast<uint4*>(V + e) = *reinterpret_cast<const uint4*>(cv);
    st8(W, e, wdt, w);
    st8(W, e + 8, wdt, w + 8);
  } else {
#pragma unroll
    for (int q = 0; q < 16; ++q)
      if (q < cnt) {
        M[e + q] = (uint8_t)(cm[q / 4] >> (8 * (q % 4)));
        V[e + q] = (uint8_t)(cv[q / 4] >> (8 * (q % 4)));
        st_elem(W, e + q, wdt, w[q]);
      }
  }
  if (cnt && (threadIdx.x & 7) == 0) {
    p.S1[t][blk] = s1;
    p.S2[t][blk] = s2;
  }
}

// ---------------------------------------------------------------------------
// Step counted on the device: one thread looks at the device values, counts
// the step and leaves what depends on it in the workspace.
// ---------------------------------------------------------------------------
__global__ void adamw_scalars(const AdamwScalarsParams p) {
  const bool skip = (p.grad_scale && !finite_f(*p.grad_scale)) || (p.lr_dev && !finite_f(*p.lr_dev));
  *p.status = skip ? ST_NONFINITE : ST_OK;
  p.out->skip = skip;
  if (skip) return;
  const int64_t t = *p.counter + 1;
  *p.counter = t;
  p.out->inv_bc1 = (float)(1.0 / (1.0 - pow(p.b1, (double)t)));
  p.out->inv_sqrt_bc2 = (float)(1.0 / sqrt(1.0 - pow(p.b2, (double)t)));
  p.out->step_key = many_mix(p.seed + MANY_GOLDEN * (uint32_t)t);
}

}  // namespace

template <int N>
cudaError_t launch_adamw32(const Adamw32Params<N>& p, int tiles, cudaStream_t s) {
  adamw32_step<N><<<tiles, THREADS, 0, s>>>(p);
  return cudaGetLastError();
}
template <int N>
cudaError_t launch_adamw8(const Adamw8Params<N>& p, int tiles, cudaStream_t s) {
  adamw8_step<N><<<tiles, THREADS, 0, s>>>(p);
  return cudaGetLastError();
}
cudaError_t launch_adamw_scalars(const AdamwScalarsParams& p, cudaStream_t s) {
  adamw_scalars<<<1, 1, 0, s>>>(p);
  return cudaGetLastError();
}
template cudaError_t launch_adamw32(const Adamw32Params<MANY_SMALL>&, int, cudaStream_t);
template cudaError_t launch_adamw32(const Adamw32Params<MANY_MAX>&, int, cudaStream_t);
template cudaError_t launch_adamw8(const Adamw8Params<MANY_SMALL>&, int, cudaStream_t);
template cudaError_t launch_adamw8(const Adamw8Params<MANY_MAX>&, int, cudaStream_t);

}  // namespace dm
