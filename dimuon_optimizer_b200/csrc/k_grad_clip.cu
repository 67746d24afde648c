// Euclidean norm of many gradients together and clipping by it
// (include/dimuon.h, dm_grad_clip): a norm pass that leaves one fp64 partial
// sum per CTA, and a second pass whose CTAs add the partials in their order
// (the same bits in every CTA, on every run) and write the clipped
// gradients; without outputs one CTA of the second kind writes the result.
// Bound by HBM: 2 bytes per element (bf16), and once more with its output.
#include "dm_common.cuh"
#include "dm_many.h"

namespace dm {
namespace {

constexpr int THREADS = 256;

// Sum of squares of 16 values: fp32 while it stays in range, else (rare) in
// fp64, so that gradients of 1e30 or 1e-30 have a norm as well.
__device__ __forceinline__ double sumsq16(const float v[16]) {
  float s = 0.f;
#pragma unroll
  for (int q = 0; q < 16; ++q) s = fmaf(v[q], v[q], s);
  if (s > 1e-24f && s < 1e37f) return (double)s;
  float top = 0.f;
#pragma unroll
  for (int q = 0; q < 16; ++q) top = fmaxf(top, fabsf(v[q]));
  if (s == 0.f && top == 0.f) return 0.0;
  double d = 0.0;
#pragma unroll
  for (int q = 0; q < 16; ++q) d += (double)v[q] * (double)v[q];
  return d;
}

template <int N>
__global__ void __launch_bounds__(THREADS) grad_sumsq(const __grid_constant__ ClipParams<N> p) {
  __shared__ double red[32];
  double acc = 0.0;
  for (int tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
    const int t = find_group(p.starts, p.count, tile);
    const int flags = p.flags[t], gdt = flags & MF_G_FP32 ? DT_FP32 : DT_BF16;
    const int64_t n = p.n[t];
    const int64_t base = (int64_t)(tile - p.starts[t]) * CLIP_TILE;
    float v[16];
    const int64_t e = base + threadIdx.x * 16 - ((flags >> MF_SHIFT_BIT) & 7);
    if ((flags & MF_VEC) && e >= 0 && e + 16 <= n) {
      ld8(p.G[t], e, gdt, v);
      ld8(p.G[t], e + 8, gdt, v + 8);
    } else if (flags & MF_VEC) {
#pragma unroll
      for (int q = 0; q < 16; ++q)
        v[q] = e + q >= 0 && e + q < n ? ld_elem(p.G[t], e + q, gdt) : 0.f;
    } else {
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const int64_t i = base + q * THREADS + threadIdx.x;
        v[q] = i < n ? ld_elem(p.G[t], i, gdt) : 0.f;
      }
    }
    acc += sumsq16(v);
  }
  acc = block_sum_d(acc, red);
  if (threadIdx.x == 0) p.part[blockIdx.x] = acc;
}

// The norm and the coefficient from all partials, in one order.
__device__ __forceinline__ float coefficient(const double* part, int n, float max_norm,
                                             float* result, int* status, double* red) {
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += THREADS) s += part[i];
  const double norm = sqrt(block_sum_d(s, red));
  const bool ok = (float)norm <= 3.402823466e38f;  // finite in fp32
  const float coef = !ok ? __uint_as_float(0x7fffffffu)
                         : norm > (double)max_norm ? (float)((double)max_norm / norm) : 1.f;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    result[0] = (float)norm;
    result[1] = coef;
    *status = ok ? ST_OK : ST_NONFINITE;
  }
  return coef;
}

template <int N>
__global__ void __launch_bounds__(THREADS) grad_write(const __grid_constant__ ClipParams<N> p) {
  __shared__ double red[32];
  const float c = coefficient(p.part, p.n_part, p.max_norm, p.result, p.status, red);
  if (!(c == c)) return;
  for (int tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
    const int t = find_group(p.starts, p.count, tile);
    const void* G = p.G[t];
    void* out = p.out[t];
    if (c == 1.f && G == out) continue;
    const int flags = p.flags[t], gdt = flags & MF_G_FP32 ? DT_FP32 : DT_BF16,
              odt = flags & MF_W_FP32 ? DT_FP32 : DT_BF16;
    const int64_t n = p.n[t];
    const int64_t base = (int64_t)(tile - p.starts[t]) * CLIP_TILE;
    const int64_t e = base + threadIdx.x * 16 - ((flags >> MF_SHIFT_BIT) & 7);
    if ((flags & MF_VEC) && e >= 0 && e + 16 <= n) {
      float v[16];
      ld8(G, e, gdt, v);
      ld8(G, e + 8, gdt, v + 8);
#pragma unroll
      for (int q = 0; q < 16; ++q) v[q] *= c;
      st8(out, e, odt, v);
      st8(out, e + 8, odt, v + 8);
    } else if (flags & MF_VEC) {
      for (int q = 0; q < 16; ++q)
        if (e + q >= 0 && e + q < n) st_elem(out, e + q, odt, ld_elem(G, e + q, gdt) * c);
    } else {
      for (int q = 0; q < 16; ++q) {
        const int64_t i = base + q * THREADS + threadIdx.x;
        if (i < n) st_elem(out, i, odt, ld_elem(G, i, gdt) * c);
      }
    }
  }
}

__global__ void __launch_bounds__(THREADS) grad_finish(const __grid_constant__ ClipParams<MANY_SMALL> p) {
  __shared__ double red[32];
  coefficient(p.part, p.n_part, p.max_norm, p.result, p.status, red);
}

}  // namespace

template <int N>
cudaError_t launch_grad_sumsq(const ClipParams<N>& p, int grid, cudaStream_t s) {
  grad_sumsq<N><<<grid, THREADS, 0, s>>>(p);
  return cudaGetLastError();
}
template <int N>
cudaError_t launch_grad_write(const ClipParams<N>& p, int grid, cudaStream_t s) {
  grad_write<N><<<grid, THREADS, 0, s>>>(p);
  return cudaGetLastError();
}
cudaError_t launch_grad_finish(const ClipParams<MANY_SMALL>& p, cudaStream_t s) {
  grad_finish<<<1, THREADS, 0, s>>>(p);
  return cudaGetLastError();
}
template cudaError_t launch_grad_sumsq(const ClipParams<MANY_SMALL>&, int, cudaStream_t);
template cudaError_t launch_grad_sumsq(const ClipParams<MANY_MAX>&, int, cudaStream_t);
template cudaError_t launch_grad_write(const ClipParams<MANY_SMALL>&, int, cudaStream_t);
template cudaError_t launch_grad_write(const ClipParams<MANY_MAX>&, int, cudaStream_t);

}  // namespace dm
