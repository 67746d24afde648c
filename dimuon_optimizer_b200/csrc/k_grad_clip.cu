// Euclidean norm of many gradients together and clipping by it
// (include/dimuon.h, dm_grad_clip).
//
// A norm pass leaves one fp64 partial sum per CTA; the CTAs of a second pass
// each add the partials in their order (the same bits in every CTA, on every
// run) and write the clipped gradients, last tiles first, since those are the
// ones L2 may still hold.  Without outputs one CTA writes the result.
//
// Bound by HBM.  The norm of 268 M bf16 values takes 80 us (6.7 TB/s, 1.02 of
// the measured copy; 127 us with 16 elements in flight per thread, 80 with 64
// in bf16 and 32 in fp32 and four CTAs per SM).  100 M fp32 values clipped
// into bf16 take 152 us: read twice and written once that is 6.6 TB/s.  What
// was tried beyond: L2 eviction hints that keep the norm pass's last 64 MB
// (153 us); short lists in one launch of one cluster, with the sums exchanged
// through distributed shared memory (98 vectors of 768: 5.2 us on the device, two
// launches 4.3; a call takes 11.5 to 13.6 us, most of it the host's two
// launches, and by that measure the two forms were not compared).
#include "dm_common.cuh"
#include "dm_many.h"

namespace dm {
namespace {

constexpr int THREADS = 256;
constexpr int GROUP = 16;  // elements of one thread's access: 32 bytes in bf16, twice that in fp32

template <int DT>
__device__ __forceinline__ char* elem_ptr(const void* p, int64_t e) {
  return const_cast<char*>(reinterpret_cast<const char*>(p)) + e * (DT == DT_BF16 ? 2 : 4);
}

// 16 elements as they lie in memory.
template <int DT>
struct Raw {
  static constexpr int WORDS = DT == DT_BF16 ? 8 : 16;
  uint32_t w[WORDS];
  __device__ __forceinline__ void load(const void* p) {
#pragma unroll
    for (int i = 0; i < WORDS; i += 8)
      asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3]), "=r"(w[i + 4]),
                     "=r"(w[i + 5]), "=r"(w[i + 6]), "=r"(w[i + 7])
                   : "l"(reinterpret_cast<const char*>(p) + 4 * i));
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int q = 0; q < WORDS; ++q) w[q] = 0;
  }
  __device__ __forceinline__ float operator[](int q) const {
    if (DT == DT_BF16)
      return __uint_as_float(q & 1 ? w[(q / 2) % WORDS] & 0xffff0000u : w[(q / 2) % WORDS] << 16);
    return __uint_as_float(w[q % WORDS]);
  }
};

// Sum of squares: fp32 while it stays in range, else (rare) in fp64, so that
// gradients of 1e30 or 1e-30 have a norm as well.
template <int DT>
__device__ __forceinline__ double sumsq(const Raw<DT>& x) {
  float a = 0.f, b = 0.f;
#pragma unroll
  for (int q = 0; q < 16; q += 2) {
    a = fmaf(x[q], x[q], a);
    b = fmaf(x[q + 1], x[q + 1], b);
  }
  const float s = a + b;
  if (s > 1e-30f && s < 1e37f) return (double)s;
  uint32_t any = 0;
#pragma unroll
  for (int q = 0; q < Raw<DT>::WORDS; ++q) any |= x.w[q];
  if ((any & (DT == DT_BF16 ? 0x7fff7fffu : 0x7fffffffu)) == 0) return 0.0;
  double d = 0.0;
#pragma unroll
  for (int q = 0; q < 16; ++q) d += (double)x[q] * (double)x[q];
  return d;
}

// A tile: K groups of 16 elements for each of the CTA's threads, THREADS apart.
// Elements lo <= i < hi of it are the tensor's (lo > 0 where the tile begins
// before it, which it does to lie on a multiple of 16 elements).  B groups
// are in flight at a time.
struct Tile {
  int64_t first;
  int lo, hi;
};
template <int TILE, int N>
__device__ __forceinline__ Tile tile_of(const ClipParams<N>& p, int t, int tile) {
  Tile x;
  x.first = (int64_t)(tile - p.starts[t]) * TILE - ((p.flags[t] >> MF_SHIFT_BIT) & 15);
  x.lo = x.first < 0 ? (int)-x.first : 0;
  x.hi = (int)min(p.n[t] - x.first, (int64_t)TILE);
  return x;
}
__device__ __forceinline__ bool whole(const Tile& x, int e) { return e >= x.lo && e + GROUP <= x.hi; }
__device__ __forceinline__ bool cut(const Tile& x, int e) {
  return !whole(x, e) && e + GROUP > x.lo && e < x.hi;
}

template <int DT, int K, int B>
__device__ __forceinline__ double tile_sumsq(const void* G, const Tile& t) {
  const char* base = elem_ptr<DT>(G, t.first);
  double acc = 0.0;
#pragma unroll 1
  for (int e = threadIdx.x * GROUP; e < K * THREADS * GROUP; e += B * THREADS * GROUP) {
    Raw<DT> x[B];
#pragma unroll
    for (int k = 0; k < B; ++k) {
      const int f = e + k * THREADS * GROUP;
      x[k].clear();
      if (whole(t, f)) x[k].load(elem_ptr<DT>(base, f));
    }
#pragma unroll
    for (int k = 0; k < B; ++k) acc += sumsq(x[k]);
  }
  if (t.lo > 0 || t.hi < K * THREADS * GROUP)  // an end of the tensor: its cut groups
    for (int e = threadIdx.x * GROUP; e < t.hi; e += THREADS * GROUP)
      if (cut(t, e))
        for (int i = max(e, t.lo); i < min(e + GROUP, t.hi); ++i) {
          const double v = ld_elem(base, i, DT);
          acc += v * v;
        }
  return acc;
}

__device__ __forceinline__ void st16(void* out, int odt, const float v[16]) {
  uint32_t w[16];
  if (odt == DT_BF16) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * q], v[2 * q + 1]);
      w[q] = *reinterpret_cast<const uint32_t*>(&h);
    }
  } else {
#pragma unroll
    for (int q = 0; q < 16; ++q) w[q] = __float_as_uint(v[q]);
  }
#pragma unroll
  for (int i = 0; i < 16; i += 8) {
    if (i == 8 && odt == DT_BF16) break;
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                     reinterpret_cast<char*>(out) + 4 * i),
                 "r"(w[i]), "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[i + 4]),
                 "r"(w[i + 5]), "r"(w[i + 6]), "r"(w[i + 7])
                 : "memory");
  }
}

// The tile times c into the output; `vec`: gradient and output share their offset.
template <int DT, int ODT, int K, int B>
__device__ __forceinline__ void tile_write(const void* G, void* out, const Tile& t, bool vec, float c) {
  const char* base = elem_ptr<DT>(G, t.first);
  char* dst = elem_ptr<ODT>(out, t.first);
  if (!vec) {  // another offset than the gradient's: element by element, eight in flight
    for (int i = threadIdx.x; i < t.hi; i += 8 * THREADS) {
      float v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = i + q * THREADS < t.hi ? ld_elem(base, i + q * THREADS, DT) : 0.f;
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (i + q * THREADS < t.hi) st_elem(dst, i + q * THREADS, ODT, v[q] * c);
    }
    return;
  }
#pragma unroll 1
  for (int e = threadIdx.x * GROUP; e < K * THREADS * GROUP; e += B * THREADS * GROUP) {
    Raw<DT> x[B];
#pragma unroll
    for (int k = 0; k < B; ++k)
      if (whole(t, e + k * THREADS * GROUP)) x[k].load(elem_ptr<DT>(base, e + k * THREADS * GROUP));
#pragma unroll
    for (int k = 0; k < B; ++k) {
      float v[16];
#pragma unroll
      for (int q = 0; q < 16; ++q) v[q] = x[k][q] * c;
      if (whole(t, e + k * THREADS * GROUP)) st16(elem_ptr<ODT>(dst, e + k * THREADS * GROUP), ODT, v);
    }
  }
  if (t.lo > 0 || t.hi < K * THREADS * GROUP)
    for (int e = threadIdx.x * GROUP; e < t.hi; e += THREADS * GROUP)
      if (cut(t, e))
        for (int i = max(e, t.lo); i < min(e + GROUP, t.hi); ++i)
          st_elem(dst, i, ODT, ld_elem(base, i, DT) * c);
}

template <int N>
__global__ void __launch_bounds__(THREADS, 4) grad_sumsq(const __grid_constant__ ClipParams<N> p) {
  __shared__ double red[32];
  double acc = 0.0;
  for (int tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
    const int t = find_group(p.starts, p.count, tile);
    const Tile x = tile_of<CLIP_TILE>(p, t, tile);
    acc += p.flags[t] & MF_G_FP32 ? tile_sumsq<DT_FP32, CLIP_GROUPS, (CLIP_GROUPS + 1) / 2>(p.G[t], x)
                                  : tile_sumsq<DT_BF16, CLIP_GROUPS, CLIP_GROUPS>(p.G[t], x);
  }
  acc = block_sum_d(acc, red);
  if (threadIdx.x == 0) p.part[blockIdx.x] = acc;
}

// The coefficient from the sum of squares; one thread of the launch writes
// the result and the status.
__device__ __forceinline__ float coefficient(double sum, float max_norm, float* result, int* status,
                                             bool writer) {
  const double norm = sqrt(sum);
  const bool ok = (float)norm <= 3.402823466e38f;  // finite in fp32
  const float coef = !ok ? __uint_as_float(0x7fffffffu)
                         : norm > (double)max_norm ? (float)((double)max_norm / norm) : 1.f;
  if (writer) {
    result[0] = (float)norm;
    result[1] = coef;
    *status = ok ? ST_OK : ST_NONFINITE;
  }
  return coef;
}

__device__ __forceinline__ double sum_partials(const double* part, int n, double* red) {
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += THREADS) s += part[i];
  return block_sum_d(s, red);
}

template <int N, int DT, int ODT>
__global__ void __launch_bounds__(THREADS, 3) grad_write(const __grid_constant__ ClipParams<N> p) {
  __shared__ double red[32];
  const float c = coefficient(sum_partials(p.part, p.n_part, red), p.max_norm, p.result, p.status,
                              blockIdx.x == 0 && threadIdx.x == 0);
  if (!(c == c)) return;
  for (int tile = p.tiles - 1 - blockIdx.x; tile >= 0; tile -= gridDim.x) {
    const int t = find_group(p.starts, p.count, tile);
    if (c == 1.f && p.G[t] == p.out[t]) continue;
    tile_write<DT, ODT, CLIP_GROUPS, DT == DT_FP32 ? (CLIP_GROUPS + 1) / 2 : CLIP_GROUPS>(
        p.G[t], p.out[t], tile_of<CLIP_TILE>(p, t, tile), (p.flags[t] & MF_VEC) != 0, c);
  }
}

__global__ void __launch_bounds__(THREADS) grad_finish(const double* part, int n_part, float max_norm,
                                                       float* result, int* status) {
  __shared__ double red[32];
  coefficient(sum_partials(part, n_part, red), max_norm, result, status, threadIdx.x == 0);
}

}  // namespace

template <int N>
cudaError_t launch_grad_sumsq(const ClipParams<N>& p, int grid, cudaStream_t s) {
  grad_sumsq<N><<<grid, THREADS, 0, s>>>(p);
  return cudaGetLastError();
}
template <int N>
cudaError_t launch_grad_write(const ClipParams<N>& p, int gdt, int odt, int grid, cudaStream_t s) {
  if (gdt == DT_BF16 && odt == DT_BF16)
    grad_write<N, DT_BF16, DT_BF16><<<grid, THREADS, 0, s>>>(p);
  else if (gdt == DT_BF16)
    grad_write<N, DT_BF16, DT_FP32><<<grid, THREADS, 0, s>>>(p);
  else if (odt == DT_BF16)
    grad_write<N, DT_FP32, DT_BF16><<<grid, THREADS, 0, s>>>(p);
  else
    grad_write<N, DT_FP32, DT_FP32><<<grid, THREADS, 0, s>>>(p);
  return cudaGetLastError();
}
cudaError_t launch_grad_finish(const double* part, int n_part, float max_norm, float* result,
                               int* status, cudaStream_t s) {
  grad_finish<<<1, THREADS, 0, s>>>(part, n_part, max_norm, result, status);
  return cudaGetLastError();
}
template cudaError_t launch_grad_sumsq(const ClipParams<MANY_SMALL>&, int, cudaStream_t);
template cudaError_t launch_grad_sumsq(const ClipParams<MANY_MID>&, int, cudaStream_t);
template cudaError_t launch_grad_sumsq(const ClipParams<MANY_MAX>&, int, cudaStream_t);
template cudaError_t launch_grad_write(const ClipParams<MANY_SMALL>&, int, int, int, cudaStream_t);
template cudaError_t launch_grad_write(const ClipParams<MANY_MID>&, int, int, int, cudaStream_t);
template cudaError_t launch_grad_write(const ClipParams<MANY_MAX>&, int, int, int, cudaStream_t);

}  // namespace dm
