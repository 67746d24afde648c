// Host side of the many-tensor operators declared in include/dimuon.h:
// dm_adamw_step and dm_grad_clip.  Argument checks, the split of the list
// into launches (tensors travel in the kernel parameters) and their tiles.
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>
#include <memory>
#include <vector>

#include "dimuon.h"
#include "dm_internal.h"
#include "dm_many.h"

namespace dm {
namespace {

constexpr size_t HEADER_BYTES = 1024;      // status word at 0, AdamwScalars at 64
constexpr size_t SCALARS_OFFSET = 64;
constexpr int64_t MAX_NUMEL = int64_t(1) << 40;
// From this many elements on, a CTA takes four passes of one tensor (there are
// then 1024 CTAs and more, 6.9 for each SM; both sides measured at adamw8_step).
constexpr int64_t ADAMW8_LONG = int64_t(1) << 24;
// Tiles of one launch: the norm pass steps by its grid, one step past the last tile too.
constexpr int64_t MAX_TILES = (int64_t(1) << 31) - 1 - CLIP_MAX_GRID;

constexpr float EPS_MIN = 0x1p-126f, EPS_MAX = 0x1p125f;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool finite_h(float v) { return std::isfinite(v); }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t elem_size(int32_t dt) { return dt == DM_FP32 ? 4 : 2; }
bool bad_dtype(int32_t dt) { return dt != DM_BF16 && dt != DM_FP32; }

// Element offset of a buffer from the last address whose element number is a multiple of `m`.
int offset_in(const void* p, size_t esz, int m) {
  return (int)(reinterpret_cast<uintptr_t>(p) / esz % m);
}

// Buffer addresses of a call (an open-addressing table), to find those that occur twice.
class AddressSet {
 public:
  explicit AddressSet(size_t count) {
    size_t cap = 16;
    while (cap < 2 * count) cap *= 2;
    slots_.assign(cap, nullptr);
  }
  bool insert(const void* p) {  // false: it is there already
    const size_t i = find(p);
    if (slots_[i]) return false;
    slots_[i] = p;
    return true;
  }
  bool has(const void* p) const { return slots_[find(p)] != nullptr; }

 private:
  size_t find(const void* p) const {  // its slot, or the free one it would take
    const size_t mask = slots_.size() - 1;
    size_t i = (size_t)((reinterpret_cast<uintptr_t>(p) >> 1) * 0x9E3779B97F4A7C15ull >> 20) & mask;
    while (slots_[i] && slots_[i] != p) i = (i + 1) & mask;
    return i;
  }
  std::vector<const void*> slots_;
};

#define DM_CUDA(x)                          \
  do {                                      \
    if ((x) != cudaSuccess) return DM_ERR_CUDA; \
  } while (0)

dm_status_t check_workspace(const void* ws, size_t bytes, size_t need) {
  if (!ws || !aligned(ws, 256) || bytes < need) return DM_ERR_WORKSPACE;
  return DM_OK;
}

// ------------------------------- AdamW ------------------------------------
dm_status_t validate(const dm_adamw_tensor_t* ts, int n, const dm_adamw_hparams_t* hp) {
  if (n < 0 || (n > 0 && !ts) || !hp) return DM_ERR_INVALID_ARG;
  const float scalars[] = {hp->lr, hp->beta1, hp->beta2, hp->eps, hp->weight_decay};
  for (float v : scalars)
    if (!finite_h(v)) return DM_ERR_INVALID_ARG;
  if (hp->beta1 < 0.f || hp->beta1 >= 1.f || hp->beta2 < 0.f || hp->beta2 >= 1.f)
    return DM_ERR_INVALID_ARG;
  // The divisor sqrt(v) + eps is eps where v = 0: it and its reciprocal have to be normal numbers
  // (the kernels' reciprocal takes subnormal ones for zero, and 0 x infinity would be NaN).
  if (hp->eps != 0.f && !(hp->eps >= EPS_MIN && hp->eps <= EPS_MAX)) return DM_ERR_INVALID_ARG;
  if (!hp->step_counter && hp->step < 1) return DM_ERR_INVALID_ARG;
  if (!aligned(hp->step_counter, 8) || !aligned(hp->lr_dev, 4) || !aligned(hp->grad_scale, 4))
    return DM_ERR_INVALID_ARG;
  if (hp->reserved[0] || hp->reserved[1]) return DM_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) {
    const dm_adamw_tensor_t& t = ts[i];
    if (t.numel < 0 || t.numel > MAX_NUMEL || t.reserved0) return DM_ERR_INVALID_ARG;
    if (!finite_h(t.lr_mult) || !finite_h(t.decay_mult)) return DM_ERR_INVALID_ARG;
    if (bad_dtype(t.weight_dtype) || bad_dtype(t.grad_dtype)) return DM_ERR_UNSUPPORTED;
    if (t.state != DM_STATE_FP32 && t.state != DM_STATE_8BIT) return DM_ERR_UNSUPPORTED;
    if (t.numel == 0) continue;
    if (!t.weight || !t.grad || !t.moment1 || !t.moment2) return DM_ERR_INVALID_ARG;
    if (!aligned(t.weight, elem_size(t.weight_dtype)) || !aligned(t.grad, elem_size(t.grad_dtype)))
      return DM_ERR_INVALID_ARG;
    if (t.state == DM_STATE_8BIT) {
      if (!t.scale1 || !t.scale2 || !aligned(t.scale1, 4) || !aligned(t.scale2, 4))
        return DM_ERR_INVALID_ARG;
    } else if (!aligned(t.moment1, 4) || !aligned(t.moment2, 4)) {
      return DM_ERR_INVALID_ARG;
    }
  }
  return DM_OK;
}

// No buffer is written twice, none that is written is a gradient.
bool outputs_distinct(const dm_adamw_tensor_t* ts, int n) {
  AddressSet seen((size_t)n * 5);
  for (int i = 0; i < n; ++i) {
    const dm_adamw_tensor_t& t = ts[i];
    if (t.numel == 0) continue;
    if (!seen.insert(t.weight) || !seen.insert(t.moment1) || !seen.insert(t.moment2)) return false;
    if (t.state == DM_STATE_8BIT && (!seen.insert(t.scale1) || !seen.insert(t.scale2))) return false;
  }
  for (int i = 0; i < n; ++i)
    if (ts[i].numel > 0 && seen.has(ts[i].grad)) return false;
  return true;
}

uint8_t adamw_flags(const dm_adamw_tensor_t& t) {
  const size_t wsz = elem_size(t.weight_dtype), gsz = elem_size(t.grad_dtype);
  int f = (t.weight_dtype == DM_FP32 ? MF_W_FP32 : 0) | (t.grad_dtype == DM_FP32 ? MF_G_FP32 : 0);
  const int s = offset_in(t.weight, wsz, 8);
  if (t.state == DM_STATE_8BIT) {
    if (aligned(t.weight, 32) && aligned(t.grad, 32) && aligned(t.moment1, 16) &&
        aligned(t.moment2, 16))
      f |= MF_VEC;
  } else if (offset_in(t.grad, gsz, 8) == s && offset_in(t.moment1, 4, 8) == s &&
             offset_in(t.moment2, 4, 8) == s) {
    f |= MF_VEC | s << MF_SHIFT_BIT;
  }
  return (uint8_t)f;
}

// Tiles of a tensor in its launch (vector groups start `shift` elements early).
int64_t tile_count(int64_t numel, int flags, int tile) {
  return ceil_div(numel + ((flags >> MF_SHIFT_BIT) & 15), tile);
}

// Launches over the tensors of `order` (indices with work), in that order:
// fill(params, slot, index) for each, then go(params, tiles) per launch.
template <template <int> class Params, class Tiles, class Fill, class Go>
dm_status_t in_launches(const std::vector<int>& order, Tiles tiles_of, Fill fill, Go go) {
  static thread_local Params<MANY_SMALL> small;
  static thread_local Params<MANY_MID> mid;
  static thread_local Params<MANY_MAX> large;
  for (size_t b = 0; b < order.size();) {
    size_t e = b;
    int64_t tiles = 0;
    while (e < order.size() && (int)(e - b) < MANY_MAX) {
      const int64_t k = tiles_of(order[e]);
      if (tiles + k > MAX_TILES) break;
      tiles += k;
      ++e;
    }
    auto run = [&](auto& p) {
      int64_t at = 0;
      for (size_t q = b; q < e; ++q) {
        p.starts[q - b] = (int)at;
        at += tiles_of(order[q]);
        fill(p, (int)(q - b), order[q]);
      }
      p.starts[e - b] = (int)at;
      return go(p, (int)(e - b), (int)at);
    };
    const int count = (int)(e - b);
    const cudaError_t err = count <= MANY_SMALL ? run(small) : count <= MANY_MID ? run(mid) : run(large);
    if (err != cudaSuccess) return DM_ERR_CUDA;
    b = e;
  }
  return DM_OK;
}

dm_status_t adamw_step(const dm_adamw_tensor_t* ts, int n, const dm_adamw_hparams_t* hp, void* ws_v,
                       size_t ws_bytes, cudaStream_t s) {
  dm_status_t st = validate(ts, n, hp);
  if (st != DM_OK) return st;
  st = check_workspace(ws_v, ws_bytes, HEADER_BYTES);
  if (st != DM_OK) return st;
  if (!outputs_distinct(ts, n)) return DM_ERR_INVALID_ARG;
  uint8_t* ws = reinterpret_cast<uint8_t*>(ws_v);
  int* status = reinterpret_cast<int*>(ws);

  AdamwHead h;
  std::memset(&h, 0, sizeof(h));
  h.lr = hp->lr;
  h.wd = hp->weight_decay;
  h.b1 = hp->beta1;
  h.c1 = (float)(1.0 - (double)hp->beta1);
  h.b2 = hp->beta2;
  h.c2 = (float)(1.0 - (double)hp->beta2);
  h.eps = hp->eps;
  // sqrt(2^-126) times the largest 1 / sqrt(1 - beta2^t) below half a place of eps
  h.flush = 0x1p-63 / std::sqrt(1.0 - (double)hp->beta2) <= 0x1p-24 * (double)hp->eps;
  h.lr_dev = hp->lr_dev;
  h.grad_scale = hp->grad_scale;
  h.status = status;
  bool any = false;
  for (int i = 0; i < n; ++i) any = any || ts[i].numel > 0;
  if (hp->step_counter || !any) {  // without elements, too, the status tells of the device values
    AdamwScalarsParams sp;
    sp.counter = hp->step_counter;
    sp.lr_dev = hp->lr_dev;
    sp.grad_scale = hp->grad_scale;
    sp.b1 = hp->beta1;
    sp.b2 = hp->beta2;
    sp.seed = hp->seed;
    sp.status = status;
    sp.out = reinterpret_cast<AdamwScalars*>(ws + SCALARS_OFFSET);
    DM_CUDA(launch_adamw_scalars(sp, s));
    h.dev = sp.out;
  } else {
    const double t = (double)hp->step;
    h.sc.inv_bc1 = (float)(1.0 / (1.0 - std::pow((double)hp->beta1, t)));
    h.sc.inv_sqrt_bc2 = (float)(1.0 / std::sqrt(1.0 - std::pow((double)hp->beta2, t)));
    h.sc.step_key = many_mix(hp->seed + MANY_GOLDEN * (uint32_t)hp->step);
    h.write_status = 1;
  }

  // one launch takes tensors of the same state format and types
  for (int wdt = DM_BF16; wdt <= DM_FP32; ++wdt)
    for (int gdt = DM_BF16; gdt <= DM_FP32; ++gdt) {
      std::vector<int> fp32, eight;
      int64_t elems8 = 0;
      for (int i = 0; i < n; ++i) {
        if (ts[i].numel == 0 || ts[i].weight_dtype != wdt || ts[i].grad_dtype != gdt) continue;
        const bool is8 = ts[i].state == DM_STATE_8BIT;
        (is8 ? eight : fp32).push_back(i);
        if (is8) elems8 += ts[i].numel;
      }
      auto common = [&](auto& p, int q, int i) {
        const dm_adamw_tensor_t& t = ts[i];
        p.W[q] = t.weight;
        p.G[q] = t.grad;
        p.lr_mult[q] = t.lr_mult;
        p.decay_mult[q] = t.decay_mult;
      };
      if (!fp32.empty()) {
        st = in_launches<Adamw32Params>(
            fp32,
            [&](int i) { return tile_count(ts[i].numel, adamw_flags(ts[i]), ADAMW32_TILE); },
            [&](auto& p, int q, int i) {
              common(p, q, i);
              p.M[q] = reinterpret_cast<float*>(ts[i].moment1);
              p.V[q] = reinterpret_cast<float*>(ts[i].moment2);
              p.n[q] = ts[i].numel;
              p.flags[q] = adamw_flags(ts[i]);
            },
            [&](auto& p, int count, int tiles) {
              p.h = h;
              p.h.count = count;
              return launch_adamw32(p, wdt, gdt, tiles, s);
            });
        if (st != DM_OK) return st;
      }
      if (!eight.empty()) {
        const int tile = elems8 >= ADAMW8_LONG ? 4 * ADAMW8_PASS : ADAMW8_PASS;
        st = in_launches<Adamw8Params>(
            eight, [&](int i) { return tile_count(ts[i].numel, 0, tile); },
            [&](auto& p, int q, int i) {
              common(p, q, i);
              p.M[q] = ts[i].moment1;
              p.V[q] = ts[i].moment2;
              p.S1[q] = ts[i].scale1;
              p.S2[q] = ts[i].scale2;
              p.n_flags[q] = ts[i].numel << 8 | adamw_flags(ts[i]);
              p.index[q] = (uint32_t)i;
            },
            [&](auto& p, int count, int tiles) {
              p.h = h;
              p.h.count = count;
              p.tile_elems = tile;
              return launch_adamw8(p, wdt, gdt, tiles, s);
            });
        if (st != DM_OK) return st;
      }
    }
  return DM_OK;
}

// ----------------------------- grad clip ----------------------------------
dm_status_t validate(const dm_grad_t* ts, int n) {
  if (n < 0 || (n > 0 && !ts)) return DM_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) {
    const dm_grad_t& t = ts[i];
    if (t.numel < 0 || t.numel > MAX_NUMEL) return DM_ERR_INVALID_ARG;
    if (bad_dtype(t.grad_dtype) || (t.out && bad_dtype(t.out_dtype))) return DM_ERR_UNSUPPORTED;
    if (t.numel == 0) continue;
    if (!t.grad || !aligned(t.grad, elem_size(t.grad_dtype))) return DM_ERR_INVALID_ARG;
    if (t.out && (!aligned(t.out, elem_size(t.out_dtype)) ||
                  (t.out == t.grad && t.out_dtype != t.grad_dtype)))
      return DM_ERR_INVALID_ARG;
  }
  return DM_OK;
}

uint8_t clip_flags(const dm_grad_t& t, bool with_out) {
  const int s = offset_in(t.grad, elem_size(t.grad_dtype), 16);
  int f = (t.grad_dtype == DM_FP32 ? MF_G_FP32 : 0) | s << MF_SHIFT_BIT | MF_VEC;
  if (with_out) {
    if (t.out_dtype == DM_FP32) f |= MF_W_FP32;
    if (offset_in(t.out, elem_size(t.out_dtype), 16) != s) f &= ~(MF_VEC | 15 << MF_SHIFT_BIT);
  }
  return (uint8_t)f;
}

// Launches of the norm pass, each of which leaves at most CLIP_MAX_GRID partial
// sums (counted with the most tiles that any alignment gives).
int64_t clip_launches(const dm_grad_t* ts, int n) {
  int64_t launches = 0, count = 0, tiles = 0;
  for (int i = 0; i < n; ++i) {
    if (ts[i].numel == 0) continue;
    const int64_t k = tile_count(ts[i].numel, 15 << MF_SHIFT_BIT, CLIP_TILE);
    if (count == 0 || count == MANY_MAX || tiles + k > MAX_TILES) {
      ++launches;
      count = tiles = 0;
    }
    ++count;
    tiles += k;
  }
  return launches;
}

size_t clip_bytes(const dm_grad_t* ts, int n) {
  return HEADER_BYTES + (size_t)clip_launches(ts, n) * CLIP_MAX_GRID * sizeof(double);
}

dm_status_t grad_clip(const dm_grad_t* ts, int n, float max_norm, float* result, void* ws_v,
                      size_t ws_bytes, cudaStream_t s) {
  dm_status_t st = validate(ts, n);
  if (st != DM_OK) return st;
  if (!(max_norm > 0.f) || !result || !aligned(result, 4)) return DM_ERR_INVALID_ARG;
  st = check_workspace(ws_v, ws_bytes, clip_bytes(ts, n));
  if (st != DM_OK) return st;
  std::vector<int> all, with_out[4];  // by the two types
  // an output is written once, and is no gradient but its own, and then of no other tensor
  AddressSet outs((size_t)n), grads((size_t)n), repeated((size_t)n);
  for (int i = 0; i < n; ++i)
    if (ts[i].numel > 0 && !grads.insert(ts[i].grad)) repeated.insert(ts[i].grad);
  for (int i = 0; i < n; ++i) {
    if (ts[i].numel == 0) continue;
    all.push_back(i);
    const void* out = ts[i].out;
    if (!out) continue;
    if (!outs.insert(out) || (grads.has(out) && (out != ts[i].grad || repeated.has(out))))
      return DM_ERR_INVALID_ARG;
    with_out[ts[i].grad_dtype * 2 + ts[i].out_dtype].push_back(i);
  }
  uint8_t* ws = reinterpret_cast<uint8_t*>(ws_v);
  double* part = reinterpret_cast<double*>(ws + HEADER_BYTES);
  int n_part = 0;
  auto pass = [&](const std::vector<int>& order, bool out) {
    auto flags = [&](int i) { return clip_flags(ts[i], out); };
    return in_launches<ClipParams>(
        order,
        [&](int i) { return tile_count(ts[i].numel, flags(i), CLIP_TILE); },
        [&](auto& p, int q, int i) {
          p.G[q] = ts[i].grad;
          p.out[q] = ts[i].out;
          p.n[q] = ts[i].numel;
          p.flags[q] = flags(i);
        },
        [&](auto& p, int count, int tiles) {
          p.count = count;
          p.tiles = tiles;
          p.max_norm = max_norm;
          p.result = result;
          p.status = reinterpret_cast<int*>(ws);
          const int grid = tiles < CLIP_MAX_GRID ? tiles : CLIP_MAX_GRID;
          if (out) {
            p.part = part;
            p.n_part = n_part;
            return launch_grad_write(p, ts[order[0]].grad_dtype, ts[order[0]].out_dtype, grid, s);
          }
          p.part = part + n_part;
          n_part += grid;
          return launch_grad_sumsq(p, grid, s);
        });
  };
  st = pass(all, false);
  if (st != DM_OK) return st;
  bool written = false;
  for (const std::vector<int>& list : with_out) {
    if (list.empty()) continue;
    st = pass(list, true);
    if (st != DM_OK) return st;
    written = true;
  }
  if (written) return DM_OK;
  DM_CUDA(launch_grad_finish(part, n_part, max_norm, result, reinterpret_cast<int*>(ws), s));
  return DM_OK;
}

}  // namespace
}  // namespace dm

extern "C" {

void dm_adamw_default_hparams(dm_adamw_hparams_t* hp) {
  if (!hp) return;
  std::memset(hp, 0, sizeof(*hp));
  hp->lr = 1e-3f;
  hp->beta1 = 0.9f;
  hp->beta2 = 0.999f;
  hp->eps = 1e-8f;
  hp->weight_decay = 0.01f;
  hp->step = 1;
}

dm_status_t dm_adamw_workspace_size(const dm_adamw_tensor_t* tensors, int n,
                                    const dm_adamw_hparams_t* hp, size_t* bytes) {
  if (!bytes) return DM_ERR_INVALID_ARG;
  const dm_status_t st = dm::validate(tensors, n, hp);
  if (st != DM_OK) return st;
  *bytes = dm::HEADER_BYTES;
  return DM_OK;
}

dm_status_t dm_adamw_step(const dm_adamw_tensor_t* tensors, int n, const dm_adamw_hparams_t* hp,
                          void* workspace, size_t workspace_bytes, void* stream) {
  try {
    return dm::adamw_step(tensors, n, hp, workspace, workspace_bytes,
                          reinterpret_cast<cudaStream_t>(stream));
  } catch (...) {
    return DM_ERR_CUDA;
  }
}

dm_status_t dm_grad_clip_workspace_size(const dm_grad_t* tensors, int n, size_t* bytes) {
  if (!bytes) return DM_ERR_INVALID_ARG;
  const dm_status_t st = dm::validate(tensors, n);
  if (st != DM_OK) return st;
  *bytes = dm::clip_bytes(tensors, n);
  return DM_OK;
}

dm_status_t dm_grad_clip(const dm_grad_t* tensors, int n, float max_norm, float* result,
                         void* workspace, size_t workspace_bytes, void* stream) {
  try {
    return dm::grad_clip(tensors, n, max_norm, result, workspace, workspace_bytes,
                         reinterpret_cast<cudaStream_t>(stream));
  } catch (...) {
    return DM_ERR_CUDA;
  }
}

}  // extern "C"
