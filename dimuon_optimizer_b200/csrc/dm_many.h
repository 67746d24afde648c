// Launch parameters of the many-tensor operators (AdamW, gradient clipping):
// the tensors of one launch travel in the kernel parameters, as arrays per
// field so that 448 of them fit the 32764 bytes.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace dm {

// Tensors per launch.  The parameters are copied at every launch, so shorter
// lists take a smaller block.
constexpr int MANY_SMALL = 24;
constexpr int MANY_MID = 160;
constexpr int MANY_MAX = 448;

// Per-tensor flags: types, and the element offset of the tensor that all its
// buffers share (AdamW: 0..7, from a multiple of 8 elements; clipping: 0..15, from
// a multiple of 16).
enum {
  MF_W_FP32 = 1,     // weight (or out) is fp32, else bf16
  MF_G_FP32 = 2,     // grad is fp32, else bf16
  MF_VEC = 4,        // all buffers share one offset: vector path
  MF_SHIFT_BIT = 4   // bits 4-7: that offset
};

// ------------------------------- AdamW ------------------------------------
constexpr int ADAMW32_TILE = 2048;  // elements per CTA, 8 per thread
constexpr int ADAMW8_PASS = 4096;   // elements a CTA takes at a time, 16 per thread: 8 threads
                                    // share a block's scale

// Values that depend on the step, computed on the host, or by adamw_scalars
// when the step is counted on the device.
struct AdamwScalars {
  float inv_bc1;        // 1 / (1 - beta1^t)
  float inv_sqrt_bc2;   // 1 / sqrt(1 - beta2^t)
  uint32_t step_key;    // hash of (seed, t)
  int32_t skip;         // device mode: a device value was not finite
};

struct AdamwHead {
  int count;
  int write_status;          // host-counted step: block 0 writes the status word
  int flush;                 // eps is so large that the root of a subnormal second moment vanishes
                             // beside it
  float lr, wd, b1, c1, b2, c2, eps;
  AdamwScalars sc;
  const AdamwScalars* dev;   // null: sc above
  const float* lr_dev;
  const float* grad_scale;
  int* status;
};

template <int N>
struct Adamw32Params {
  AdamwHead h;
  void* W[N];
  const void* G[N];
  float* M[N];
  float* V[N];
  int64_t n[N];
  float lr_mult[N], decay_mult[N];
  int starts[N + 1];         // first tile of each tensor
  uint8_t flags[N];
};

template <int N>
struct Adamw8Params {
  AdamwHead h;
  int tile_elems;            // elements per CTA, a multiple of ADAMW8_PASS
  void* W[N];
  const void* G[N];
  void* M[N];
  void* V[N];
  float* S1[N];
  float* S2[N];
  int64_t n_flags[N];        // numel << 8 | flags
  float lr_mult[N], decay_mult[N];
  uint32_t index[N];         // position in the call (part of the rounding's hash)
  int starts[N + 1];
};
static_assert(sizeof(Adamw32Params<MANY_MAX>) <= 32764, "kernel parameter space");
static_assert(sizeof(Adamw8Params<MANY_MAX>) <= 32764, "kernel parameter space");

struct AdamwScalarsParams {
  int64_t* counter;
  const float* lr_dev;
  const float* grad_scale;
  double b1, b2;
  uint32_t seed;
  int* status;
  AdamwScalars* out;
};

template <int N>
cudaError_t launch_adamw32(const Adamw32Params<N>& p, int wdt, int gdt, int grid, cudaStream_t s);
template <int N>
cudaError_t launch_adamw8(const Adamw8Params<N>& p, int wdt, int gdt, int grid, cudaStream_t s);
cudaError_t launch_adamw_scalars(const AdamwScalarsParams& p, cudaStream_t s);

// The 32-bit mixing step of the rounding's hash (host and device): two
// multiply and shift rounds, a bijection.  Shifts and multipliers are the
// published ones of least measured bias for that form (C. Wellons, "Prospecting
// for Hash Functions", 2018).
__host__ __device__ inline uint32_t many_mix(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x7FEB352Du;
  x = (x ^ (x >> 15)) * 0x846CA68Bu;
  return x ^ (x >> 16);
}
constexpr uint32_t MANY_GOLDEN = 0x9E3779B9u;  // 2^32 / golden ratio, odd

// ----------------------------- grad clip ----------------------------------
constexpr int CLIP_GROUPS = 4;                     // 16-element groups of a thread in a tile
constexpr int CLIP_TILE = 256 * 16 * CLIP_GROUPS;  // elements of a tile: one CTA of 256 threads
constexpr int CLIP_MAX_GRID = 1184;                // CTAs of a launch (partial sums of the norm pass)

template <int N>
struct ClipParams {
  int count;
  int tiles;
  int n_part;             // partials of the whole call
  float max_norm;
  double* part;           // this launch's partials (norm pass), or all of them
  float* result;
  int* status;
  const void* G[N];
  void* out[N];
  int64_t n[N];
  int starts[N + 1];
  uint8_t flags[N];       // MF_W_FP32: out is fp32
};
static_assert(sizeof(ClipParams<MANY_MAX>) <= 32764, "kernel parameter space");

template <int N>
cudaError_t launch_grad_sumsq(const ClipParams<N>& p, int grid, cudaStream_t s);
template <int N>
cudaError_t launch_grad_write(const ClipParams<N>& p, int gdt, int odt, int grid, cudaStream_t s);
cudaError_t launch_grad_finish(const double* part, int n_part, float max_norm, float* result,
                               int* status, cudaStream_t s);

}  // namespace dm
