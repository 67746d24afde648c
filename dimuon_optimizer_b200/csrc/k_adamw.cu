// AdamW over many tensors in one launch, moments in fp32 or in 8 bits.
//
// Per element (include/dimuon.h): m' = b1 m + (1 - b1) g, v' = b2 v + (1 - b2) g^2,
// W' = (1 - lr wd) W - lr (m' / bc1) / (sqrt(v' / bc2) + eps).  One pass: every
// operand is read once and written once (bf16 weights and gradients: 22 bytes
// per element with fp32 moments, 10.1 with 8-bit ones), so HBM bounds it.
#include <cuda_fp8.h>

#include "dimuon.h"
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
  float inv_bc1;       // 1 / (1 - b1^t)
  float lr, wd;        // without the tensor's multipliers
  uint32_t step_key;
  bool skip;
};

// Reads the step's device values; the status word is written by one thread
// of a host-counted step (adamw_scalars has written it otherwise).
__device__ __forceinline__ Coef coefficients(const AdamwHead& h) {
  Coef c;
  c.gs = h.grad_scale ? *h.grad_scale : 1.f;
  c.lr = h.lr_dev ? *h.lr_dev : h.lr;
  const AdamwScalars sc = h.dev ? *h.dev : h.sc;
  c.skip = h.dev ? sc.skip != 0 : !(finite_f(c.gs) && finite_f(c.lr));
  c.b1 = h.b1; c.c1 = h.c1; c.b2 = h.b2; c.c2 = h.c2; c.eps = h.eps;
  c.wd = h.wd;
  c.inv_bc1 = sc.inv_bc1;
  c.isb2 = sc.inv_sqrt_bc2;
  c.step_key = sc.step_key;
  if (h.write_status && blockIdx.x == 0 && threadIdx.x == 0)
    *h.status = c.skip ? ST_NONFINITE : ST_OK;
  return c;
}

// Two fp32 numbers in one 64-bit register pair, for the packed fp32
// instructions: half the issue slots of the separate ones, the same rounding.
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ float2 split(F2 x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 mul2_rz(F2 a, F2 b) {  // rounded towards zero
  F2 r;
  asm("mul.rz.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
// A sum of two products that stay rounded: as two separate additions, because
// the assembler joins a packed product and a packed sum into one packed
// multiply-add, their .rn and --fmad=false notwithstanding (it costs 1.5 %).
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  const float2 x = split(a), y = split(b);
  return f2(__fadd_rn(x.x, y.x), __fadd_rn(x.y, y.y));
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
// Largest of |a|, |b|, |c|; NaN if any is.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// FLUSH takes subnormal numbers for zero: one instruction instead of four, for an eps next to
// which their square roots vanish.
template <bool FLUSH>
__device__ __forceinline__ float sqrt_approx(float x) {
  float r;
  if (FLUSH)
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  else
    asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_ftz(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

template <int DT>
__device__ __forceinline__ void* elem_ptr(const void* p, int64_t e) {
  return const_cast<char*>(reinterpret_cast<const char*>(p)) + e * (DT == DT_BF16 ? 2 : 4);
}

// ---------------------------------------------------------------------------
// fp32 moments.  A thread takes 8 consecutive elements at a time; group k of a
// tensor covers elements 8k - shift .. 8k - shift + 7, so that whole groups lie
// on 32-byte boundaries in fp32 (16 in bf16) whatever the tensor's offset.
// ---------------------------------------------------------------------------
// The step for two elements.  The moments' products and sums are rounded one
// by one, as in the 8-bit form (there they are part of its definition); square
// root and reciprocal are the approximate ones (2^-23: they touch the update only).
struct Step {
  F2 gs, b1, c1, b2, c2, isb2, eps, nstep, decay;
};
__device__ __forceinline__ void update2(const Step& s, F2 g, F2& m, F2& v, F2& w) {
  g = mul2(g, s.gs);
  m = add2(mul2(m, s.b1), mul2(g, s.c1));
  v = add2(mul2(v, s.b2), mul2(mul2(g, g), s.c2));
  const float2 f = split(v), d = split(fma2(f2(sqrt_approx<false>(f.x), sqrt_approx<false>(f.y)), s.isb2, s.eps));
  w = fma2(mul2(m, s.nstep), f2(rcp_ftz(d.x), rcp_ftz(d.y)), mul2(w, s.decay));
}

// 8 elements as pairs.
template <int DT>
__device__ __forceinline__ void ld4x2(const void* p, F2 x[4]) {
  if (DT == DT_BF16) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int q = 0; q < 4; ++q)
      x[q] = f2(__uint_as_float(w[q] << 16), __uint_as_float(w[q] & 0xffff0000u));
  } else {
    asm volatile("ld.global.v4.b64 {%0, %1, %2, %3}, [%4];"
                 : "=l"(x[0].v), "=l"(x[1].v), "=l"(x[2].v), "=l"(x[3].v)
                 : "l"(p));
  }
}
template <int DT>
__device__ __forceinline__ void st4x2(void* p, const F2 x[4]) {
  if (DT == DT_BF16) {
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 f = split(x[q]);
      const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
      w[q] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    asm volatile("st.global.v4.b64 [%0], {%1, %2, %3, %4};" ::"l"(p), "l"(x[0].v), "l"(x[1].v),
                 "l"(x[2].v), "l"(x[3].v)
                 : "memory");
  }
}

// Bound by HBM: 262 M elements (bf16 weights and gradients, 22 bytes each) take
// 834 us, 6.93 TB/s or 1.06 of the measured copy; 448 tensors of 32768 fp32
// elements 63 us (1.00).  What made the difference were accesses of 32 bytes
// per thread (16 bytes at a stride of 32 before: 924 and 70 us) and types fixed
// per launch; one pass per CTA (2, 4, 8 passes: 849, 859, 875 us).
template <int N, int WDT, int GDT>
__global__ void __launch_bounds__(THREADS) adamw32_step(const __grid_constant__ Adamw32Params<N> p) {
  const int tile = blockIdx.x;
  const int t = find_group(p.starts, p.h.count, tile);
  const Coef c = coefficients(p.h);
  if (c.skip) return;
  const int flags = p.flags[t];
  // the CTA's elements, counted from its first group (which may begin before the tensor)
  const int64_t first = (int64_t)(tile - p.starts[t]) * ADAMW32_TILE - ((flags >> MF_SHIFT_BIT) & 7);
  const int left = (int)min(p.n[t] - first, (int64_t)ADAMW32_TILE);
  const int lo = first < 0 ? (int)-first : 0;
  const void* G = elem_ptr<GDT>(p.G[t], first);
  void* W = elem_ptr<WDT>(p.W[t], first);
  float* M = p.M[t] + first;
  float* V = p.V[t] + first;
  const float lr = c.lr * p.lr_mult[t];
  const Step s = {f2(c.gs), f2(c.b1), f2(c.c1), f2(c.b2), f2(c.c2), f2(c.isb2), f2(c.eps),
                  f2(-(lr * c.inv_bc1)), f2(fmaf(-lr, c.wd * p.decay_mult[t], 1.f))};
  auto one = [&](uint32_t e) {
    F2 m = f2(M[e]), v = f2(V[e]), w = f2(ld_elem(W, e, WDT));
    update2(s, f2(ld_elem(G, e, GDT)), m, v, w);
    M[e] = split(m).x;
    V[e] = split(v).x;
    st_elem(W, e, WDT, split(w).x);
  };
  if (!(flags & MF_VEC)) {
    for (uint32_t e = threadIdx.x; e < (uint32_t)left; e += THREADS) one(e);
    return;
  }
  const int e = threadIdx.x * 8;
  if (e < lo || e + 8 > left) {  // a group that is not all inside
    for (int i = max(e, lo); i < min(e + 8, left); ++i) one(i);
    return;
  }
  F2 g[4], m[4], v[4], w[4];
  ld4x2<GDT>(elem_ptr<GDT>(G, e), g);
  ld4x2<DT_FP32>(M + e, m);
  ld4x2<DT_FP32>(V + e, v);
  ld4x2<WDT>(elem_ptr<WDT>(W, e), w);
#pragma unroll
  for (int q = 0; q < 4; ++q) update2(s, g[q], m[q], v[q], w[q]);
  st4x2<DT_FP32>(M + e, m);
  st4x2<DT_FP32>(V + e, v);
  st4x2<WDT>(elem_ptr<WDT>(W, e), w);
}

// ---------------------------------------------------------------------------
// 8-bit moments.  A thread takes 16 consecutive elements at a time, so 8
// threads of a warp share the scale of a block of 128.
// ---------------------------------------------------------------------------
// Rounding to codes.  x in units of its code's format, multiplied by 2^-120
// (e4m3) or 2^-112 (e5m2), lies where the fp32 exponent field counts like the
// code's: the code's bits then stand in the fp32 pattern 20 (21) places up, the
// subnormal codes as fp32 subnormals, and the bits below are the remainder.
// Adding noise to them and cutting them off takes the upper neighbour with the
// remainder's probability.  A remainder finer than the subnormal pattern holds
// is cut off, not rounded: the noise counts in 2^-16 of a code's step, so what
// lies below the pattern's last place (2^-20 or 2^-21 of it) decides nothing.
// Two factors, as their product leaves fp32 for large scales.
constexpr float E4M3_TO_BITS = 7.52316384526264e-37f;   // 2^-120
constexpr float E5M2_TO_BITS = 1.925929944387236e-34f;  // 2^-112

// Smallest power of two s >= 2^-110 with the magnitude of `bits` <= 1.75 2^top s,
// and its inverse; NaN for a non-finite magnitude.
__device__ __forceinline__ void block_scale(uint32_t bits, int top, float& s, float& inv) {
  const int e = max((int)((bits + 0x1FFFFFu) >> 23) - top, 17);
  s = bits < 0x7f800000u ? __uint_as_float((uint32_t)e << 23) : __uint_as_float(0x7fffffffu);
  inv = __uint_as_float((uint32_t)(254 - e) << 23);
}

// 1.75 x 2^127, the largest second moment that is stored (the code above it would
// stand for 2^128, which fp32 does not hold).  Larger ones, and one that
// overflowed while the block's first moments did not (a finite gradient above
// 1.8e19, whose square leaves fp32), are held there, so that the block stays
// finite: the scale is that of HELD_BITS, and codes above LARGEST_E5M2 become it.
constexpr uint32_t HELD_BITS = 0x7f600000u;
constexpr uint32_t LARGEST_E5M2 = 0x7b7b7b7bu;  // four codes of 57344

__device__ __forceinline__ uint32_t group_max(uint32_t v) {  // over 8 neighbouring lanes
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// 16 elements of a buffer as they lie in memory: `cnt` of them from element
// e on, zero bits behind; `vec`: all 16, on a 32-byte boundary.
template <int DT>
struct Raw16 {
  static constexpr int WORDS = DT == DT_BF16 ? 8 : 16;
  uint32_t w[WORDS];
  __device__ __forceinline__ void load(const void* p, uint32_t e, int cnt, bool vec) {
    if (vec) {
#pragma unroll
      for (int i = 0; i < WORDS; i += 8)
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3]), "=r"(w[i + 4]),
                       "=r"(w[i + 5]), "=r"(w[i + 6]), "=r"(w[i + 7])
                     : "l"(reinterpret_cast<const char*>(elem_ptr<DT>(p, e)) + 4 * i));
    } else if (DT == DT_BF16) {
      const uint16_t* q = reinterpret_cast<const uint16_t*>(p) + e;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        w[i] = (2 * i < cnt ? (uint32_t)q[2 * i] : 0u) |
               (2 * i + 1 < cnt ? (uint32_t)q[2 * i + 1] << 16 : 0u);
    } else {
      const uint32_t* q = reinterpret_cast<const uint32_t*>(p) + e;
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i % WORDS] = i < cnt ? q[i] : 0u;
    }
  }
  __device__ __forceinline__ F2 pair(int q) const {  // elements 2q, 2q + 1
    if (DT == DT_BF16)
      return f2(__uint_as_float(w[q] << 16), __uint_as_float(w[q] & 0xffff0000u));
    return f2(__uint_as_float(w[(2 * q) % WORDS]), __uint_as_float(w[(2 * q + 1) % WORDS]));
  }
  __device__ __forceinline__ void set(int q, F2 x) {
    const float2 f = split(x);
    if (DT == DT_BF16) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
      w[q] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      w[(2 * q) % WORDS] = __float_as_uint(f.x);
      w[(2 * q + 1) % WORDS] = __float_as_uint(f.y);
    }
  }
  __device__ __forceinline__ void store(void* p, uint32_t e, int cnt, bool vec) const {
    if (vec) {
#pragma unroll
      for (int i = 0; i < WORDS; i += 8)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                         reinterpret_cast<char*>(elem_ptr<DT>(p, e)) + 4 * i),
                     "r"(w[i]), "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[i + 4]),
                     "r"(w[i + 5]), "r"(w[i + 6]), "r"(w[i + 7])
                     : "memory");
    } else if (DT == DT_BF16) {
      uint16_t* q = reinterpret_cast<uint16_t*>(p) + e;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < cnt) q[i] = (uint16_t)(w[i / 2] >> (16 * (i % 2)));
    } else {
      uint32_t* q = reinterpret_cast<uint32_t*>(p) + e;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < cnt) q[i] = w[i % WORDS];
    }
  }
};

// 16 codes, four to a word.
struct Codes16 {
  uint32_t w[4];
  __device__ __forceinline__ void load(const void* p8, uint32_t e, int cnt, bool vec) {
    const uint8_t* p = reinterpret_cast<const uint8_t*>(p8) + e;
    if (vec) {
      *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(p);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (i % 4 == 0) w[i / 4] = 0;
        if (i < cnt) w[i / 4] |= (uint32_t)p[i] << (8 * (i % 4));
      }
    }
  }
  __device__ __forceinline__ void store(void* p8, uint32_t e, int cnt, bool vec) const {
    uint8_t* p = reinterpret_cast<uint8_t*>(p8) + e;
    if (vec) {
      *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(w);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < cnt) p[i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
    }
  }
  __device__ __forceinline__ F2 pair(int q, __nv_fp8_interpretation_t kind) const {
    const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(
        (__nv_fp8x2_storage_t)(w[q / 2] >> (16 * (q % 2))), kind)));
    return f2(f.x, f.y);
  }
  // Byte 3 of the four words.
  __device__ __forceinline__ void gather(int i, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    w[i] = __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
  }
};

// Bound by HBM up to the power limit: 262 M elements (bf16 weights and
// gradients) take 397 us (6.71 TB/s) while the clock stays at 1.96 GHz, and 424 to
// 455 us by the board (0.96 to 0.89 of the measured copy) in a long run, when the
// part reaches its 1000 W and the clock falls to 1.6 GHz: 41.5 instructions per
// element then fill four fifths of the issue slots.  The first form (one
// fp32 operation at a time, separate code for the subnormal codes, one pass
// per CTA) took 88 instructions and 837 us.  Packed fp32 arithmetic, the codes'
// bits by a power-of-two product, the packed fp8 conversions and the test for
// zero codes four at a time brought that down, and accesses of 32 bytes instead of
// 16 by another 7 %.  What follows was measured against each other in long runs.
// A CTA takes four passes, so that finding its tensor and the coefficients
// costs little (2 passes: 466 us, 4: 446, 8: 444, but with 8 152 instead of 142
// us on 448 tensors of 131072 elements); lists of less than 2^24 elements take
// one, as four would leave fewer than 1024 CTAs for the 592 that are resident.  Reading the next
// pass into registers during this one made it twice as slow (128 registers).
// Registers are held to 64, four CTAs per SM; 21 of the 24 forms spill one or
// two of them for that (without the limit 66 to 104 by type: 458 instead of 449
// us, and 182 instead of 173 us with 66 M fp32 weights and gradients).
// FLUSH: see sqrt_approx (447 against 465 us; with fp32 moments the
// instructions are hidden behind HBM, so that form has no such variant).
template <int N, int WDT, int GDT, bool FLUSH>
__global__ void __launch_bounds__(THREADS, 4)
    adamw8_step(const __grid_constant__ Adamw8Params<N> p) {
  const int tile = blockIdx.x;
  const int t = find_group(p.starts, p.h.count, tile);
  const Coef c = coefficients(p.h);
  if (c.skip) return;
  const int64_t n = p.n_flags[t] >> 8;
  const int64_t first = (int64_t)(tile - p.starts[t]) * p.tile_elems;  // of this CTA
  const bool aligned = (p.n_flags[t] & MF_VEC) != 0;
  const int left = (int)min(n - first, (int64_t)p.tile_elems);  // elements of this CTA
  const void* G = elem_ptr<GDT>(p.G[t], first);
  void* W = elem_ptr<WDT>(p.W[t], first);
  uint8_t* M = reinterpret_cast<uint8_t*>(p.M[t]) + first;
  uint8_t* V = reinterpret_cast<uint8_t*>(p.V[t]) + first;
  float* S1 = p.S1[t] + first / DM_ADAMW_BLOCK;
  float* S2 = p.S2[t] + first / DM_ADAMW_BLOCK;
  const uint64_t group = (uint64_t)first >> 4;  // 2^32 groups are whole tiles: one upper half
  const uint32_t key =
      many_mix(many_mix(c.step_key + p.index[t]) + (uint32_t)(group >> 32)) ^ (uint32_t)group;
  const float lr = c.lr * p.lr_mult[t];
  const F2 gs = f2(c.gs), c1 = f2(c.c1), c2 = f2(c.c2), isb2 = f2(c.isb2), eps = f2(c.eps),
           nstep = f2(-(lr * c.inv_bc1)), decay = f2(fmaf(-lr, c.wd * p.decay_mult[t], 1.f));

  for (uint32_t e = threadIdx.x * 16; e - threadIdx.x * 16 < (uint32_t)left; e += ADAMW8_PASS) {
    const int cnt = min(max(left - (int)e, 0), 16);
    const bool vec = aligned && cnt == 16;
    const uint32_t blk = e / DM_ADAMW_BLOCK;
    Raw16<GDT> g;
    Raw16<WDT> w;
    Codes16 cm, cv;
    g.load(G, e, cnt, vec);
    w.load(W, e, cnt, vec);
    cm.load(M, e, cnt, vec);
    cv.load(V, e, cnt, vec);
    float s1 = 0.f, s2 = 0.f;
    if (cnt) {
      s1 = S1[blk];
      s2 = S2[blk];
    }
    // code x scale x beta: the scale is a power of two, so scale x beta is exact and the product
    // is rounded once, as code x scale (exact) times beta
    const F2 sb1 = f2(s1 * c.b1), sb2 = f2(s2 * c.b2);
    F2 m[8], v[8];
    float top1 = 0.f, top2 = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      // products and sums rounded one by one: the rounding below compares these bits with its
      // noise, so their value is part of the operator's definition
      const F2 gq = mul2(g.pair(q), gs);
      m[q] = add2(mul2(cm.pair(q, __NV_E4M3), sb1), mul2(gq, c1));
      v[q] = add2(mul2(cv.pair(q, __NV_E5M2), sb2), mul2(mul2(gq, gq), c2));
      const float2 mf = split(m[q]), vf = split(v[q]);
      top1 = max3_abs(top1, mf.x, mf.y);
      top2 = max3_abs(top2, vf.x, vf.y);
      const float2 d = split(fma2(f2(sqrt_approx<FLUSH>(vf.x), sqrt_approx<FLUSH>(vf.y)), isb2, eps));
      w.set(q, fma2(mul2(m[q], nstep), f2(rcp_ftz(d.x), rcp_ftz(d.y)), mul2(w.pair(q), decay)));
    }
    w.store(W, e, cnt, vec);
    const uint32_t max1 = group_max(__float_as_uint(top1)), max2 = group_max(__float_as_uint(top2));
    const bool held = max2 > HELD_BITS && max2 <= 0x7f800000u && max1 < 0x7f800000u;
    float i1, i2;
    block_scale(max1, 8, s1, i1);
    block_scale(held ? HELD_BITS : max2, 15, s2, i2);
    const uint32_t h0 = many_mix(key ^ e / 16) * 0x7FEB352Du;
    uint32_t zero = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t a[4], b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int q = 4 * k + j;
        const float2 xm = split(mul2_rz(mul2(m[q / 2], f2(i1)), f2(E4M3_TO_BITS)));
        const float2 xv = split(mul2_rz(mul2(v[q / 2], f2(i2)), f2(E5M2_TO_BITS)));
        uint32_t h = h0 + (uint32_t)q * (MANY_GOLDEN * 0x7FEB352Du);
        h = (h ^ (h >> 15)) * 0x846CA68Bu;
        // the hash's last round, h ^= h >> 16, leaves the upper half: noise of the first moment
        // from the upper half, of the second from the lower, each moved to bits 8-23 (16 bits
        // below the code in byte 3)
        const uint32_t n1 = __byte_perm(h, 0, 0x4324), n2 = __byte_perm(h, 0, 0x4104) ^ n1;
        const uint32_t bm = __float_as_uint(q & 1 ? xm.y : xm.x);  // sign, 7 code bits from 20 on
        const uint32_t bv = __float_as_uint(q & 1 ? xv.y : xv.x);  // 8 code bits from 21 on
        a[j] = ((bm << 4) + n1) | (bm & 0x80000000u);
        b[j] = (bv << 3) + n2;
      }
      cm.gather(k, a[0], a[1], a[2], a[3]);
      cv.gather(k, b[0], b[1], b[2], b[3]);
      zero |= (cv.w[k] - 0x01010101u) & ~cv.w[k] & 0x80808080u;
    }
    if (zero) {  // a zero code: a positive second moment takes the least positive one
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const float2 f = split(v[q / 2]);
        if ((q & 1 ? f.y : f.x) > 0.f && (cv.w[q / 4] >> (8 * (q % 4)) & 0xffu) == 0)
          cv.w[q / 4] |= 1u << (8 * (q % 4));
      }
    }
    if (held) {  // an infinite moment gave 0xfc, a finite one above the largest 0x7b or 0x7c
#pragma unroll
      for (int k = 0; k < 4; ++k) cv.w[k] = __vminu4(cv.w[k], LARGEST_E5M2);
    }
    cm.store(M, e, cnt, vec);
    cv.store(V, e, cnt, vec);
    if (cnt && (threadIdx.x & 7) == 0) {
      S1[blk] = s1;
      S2[blk] = s2;
    }
  }
}

// ---------------------------------------------------------------------------
// Step counted on the device: one thread looks at the device values, counts
// the step and leaves what depends on it in the workspace.  Without a counter
// (a host-counted step over no elements) it only writes the status.
// ---------------------------------------------------------------------------
__global__ void adamw_scalars(const AdamwScalarsParams p) {
  const bool skip = (p.grad_scale && !finite_f(*p.grad_scale)) || (p.lr_dev && !finite_f(*p.lr_dev));
  *p.status = skip ? ST_NONFINITE : ST_OK;
  if (!p.counter) return;
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
cudaError_t launch_adamw32(const Adamw32Params<N>& p, int wdt, int gdt, int grid, cudaStream_t s) {
  if (wdt == DT_BF16 && gdt == DT_BF16)
    adamw32_step<N, DT_BF16, DT_BF16><<<grid, THREADS, 0, s>>>(p);
  else if (wdt == DT_BF16)
    adamw32_step<N, DT_BF16, DT_FP32><<<grid, THREADS, 0, s>>>(p);
  else if (gdt == DT_BF16)
    adamw32_step<N, DT_FP32, DT_BF16><<<grid, THREADS, 0, s>>>(p);
  else
    adamw32_step<N, DT_FP32, DT_FP32><<<grid, THREADS, 0, s>>>(p);
  return cudaGetLastError();
}
template <int N, int WDT, int GDT>
void run_adamw8(const Adamw8Params<N>& p, int grid, cudaStream_t s) {
  if (p.h.flush)
    adamw8_step<N, WDT, GDT, true><<<grid, THREADS, 0, s>>>(p);
  else
    adamw8_step<N, WDT, GDT, false><<<grid, THREADS, 0, s>>>(p);
}
template <int N>
cudaError_t launch_adamw8(const Adamw8Params<N>& p, int wdt, int gdt, int grid, cudaStream_t s) {
  if (wdt == DT_BF16 && gdt == DT_BF16)
    run_adamw8<N, DT_BF16, DT_BF16>(p, grid, s);
  else if (wdt == DT_BF16)
    run_adamw8<N, DT_BF16, DT_FP32>(p, grid, s);
  else if (gdt == DT_BF16)
    run_adamw8<N, DT_FP32, DT_BF16>(p, grid, s);
  else
    run_adamw8<N, DT_FP32, DT_FP32>(p, grid, s);
  return cudaGetLastError();
}
cudaError_t launch_adamw_scalars(const AdamwScalarsParams& p, cudaStream_t s) {
  adamw_scalars<<<1, 1, 0, s>>>(p);
  return cudaGetLastError();
}
template cudaError_t launch_adamw32(const Adamw32Params<MANY_SMALL>&, int, int, int, cudaStream_t);
template cudaError_t launch_adamw32(const Adamw32Params<MANY_MID>&, int, int, int, cudaStream_t);
template cudaError_t launch_adamw32(const Adamw32Params<MANY_MAX>&, int, int, int, cudaStream_t);
template cudaError_t launch_adamw8(const Adamw8Params<MANY_SMALL>&, int, int, int, cudaStream_t);
template cudaError_t launch_adamw8(const Adamw8Params<MANY_MID>&, int, int, int, cudaStream_t);
template cudaError_t launch_adamw8(const Adamw8Params<MANY_MAX>&, int, int, int, cudaStream_t);

}  // namespace dm
