// optim.hip -- CDNA4 (gfx950) kernels of the operators that follow a
// synchronisation: the global gradient norm and the AdamW step, with 32-bit or
// 8-bit states, over many tensors in one launch each.
#include <hip/hip_runtime.h>

#include "optim.hpp"

namespace ddpb {
namespace {

constexpr int kOptBlock = 256;

#define HIP_OK(expr, what)                                                        \
  do {                                                                            \
    hipError_t e_ = (expr);                                                       \
    if (e_ != hipSuccess) {                                                       \
      *err = std::string(what) + ": " + hipGetErrorString(e_);                    \
      return kErrHip;                                                             \
    }                                                                             \
  } while (0)

// ---------------------------------------------------------------------------
// Four consecutive elements as fp32. Addresses come from device tables, so they
// are cast to address space 1 (else the compiler emits flat accesses). Vectors
// are only assumed to be aligned like their element: gfx950's memory
// instructions take any such address, and bucket views or packed storages put
// tensors at odd offsets.
typedef float v4f __attribute__((ext_vector_type(4)));
typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef __bf16 v4bf __attribute__((ext_vector_type(4)));
typedef _Float16 v4h __attribute__((ext_vector_type(4)));

template <int D> struct Elem;
template <> struct Elem<kF32> {
  typedef float one;
  typedef v4f four __attribute__((aligned(4)));
  typedef v4f raw;
};
template <> struct Elem<kBF16> {
  typedef __bf16 one;
  typedef v4bf four __attribute__((aligned(2)));
  typedef v4bf raw;
};
template <> struct Elem<kF16> {
  typedef _Float16 one;
  typedef v4h four __attribute__((aligned(2)));
  typedef v4h raw;
};

template <typename T>
__device__ __forceinline__ __attribute__((address_space(1))) T* G(uint64_t a) {
  return (__attribute__((address_space(1))) T*)a;
}

// Elements i .. i+3 of the array at `a`, of which `left` (1..4, or more) exist.
template <int D>
__device__ __forceinline__ v4f load4(uint64_t a, int i, int left) {
  typedef typename Elem<D>::one one;
  typedef typename Elem<D>::four four;
  if (left >= 4) return __builtin_convertvector(*G<const four>(a + static_cast<uint64_t>(i) * sizeof(one)), v4f);
  v4f x = {0.0f, 0.0f, 0.0f, 0.0f};
  const auto* p = G<const one>(a) + i;
  if (left > 0) x.x = static_cast<float>(p[0]);
  if (left > 1) x.y = static_cast<float>(p[1]);
  if (left > 2) x.z = static_cast<float>(p[2]);
  return x;
}

// Rounds to nearest even where D has 16 bits: the one rounding a stored
// parameter goes through (its fp32 master, if there is one, keeps the rest).
template <int D>
__device__ __forceinline__ void store4(uint64_t a, int i, int left, v4f x) {
  typedef typename Elem<D>::one one;
  typedef typename Elem<D>::four four;
  typedef typename Elem<D>::raw raw;
  if (left >= 4) {
    *G<four>(a + static_cast<uint64_t>(i) * sizeof(one)) = __builtin_convertvector(x, raw);
    return;
  }
  auto* p = G<one>(a) + i;
  if (left > 0) p[0] = static_cast<one>(x.x);
  if (left > 1) p[1] = static_cast<one>(x.y);
  if (left > 2) p[2] = static_cast<one>(x.z);
}

__device__ __forceinline__ uint32_t load_codes(uint64_t a, int i, int left) {
  typedef uint32_t u1 __attribute__((aligned(1)));
  if (left >= 4) return *G<const u1>(a + static_cast<uint64_t>(i));
  const auto* p = G<const uint8_t>(a) + i;
  uint32_t x = 0;
  if (left > 0) x = p[0];
  if (left > 1) x |= static_cast<uint32_t>(p[1]) << 8;
  if (left > 2) x |= static_cast<uint32_t>(p[2]) << 16;
  return x;
}

__device__ __forceinline__ void store_codes(uint64_t a, int i, int left, uint32_t x) {
  typedef uint32_t u1 __attribute__((aligned(1)));
  if (left >= 4) {
    *G<u1>(a + static_cast<uint64_t>(i)) = x;
    return;
  }
  auto* p = G<uint8_t>(a) + i;
  if (left > 0) p[0] = static_cast<uint8_t>(x);
  if (left > 1) p[1] = static_cast<uint8_t>(x >> 8);
  if (left > 2) p[2] = static_cast<uint8_t>(x >> 16);
}

// ---------------------------------------------------------------------------
// Global norm: n = grad_scale * sqrt(sum g^2), coef = max_norm / n if n >
// max_norm, else 1. Summed in fp64, in an order that only the sizes decide:
// each lane over its elements, each workgroup over its lanes, the workgroup
// that finishes last over all partial sums.

__device__ __forceinline__ double block_sum(double x, double* lds) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  x = lds[0];
#pragma unroll
  for (int w = 1; w < kOptBlock / 64; ++w) x += lds[w];
  return x;
}

template <int D>
__device__ __forceinline__ double tile_squares(const NormTile& t, double acc) {
  for (int i = 4 * threadIdx.x; i < t.len; i += 4 * kOptBlock) {
    const v4f g = load4<D>(t.grad, i, t.len - i);
#pragma unroll
    for (int j = 0; j < 4; ++j) acc = __builtin_fma(static_cast<double>(g[j]), static_cast<double>(g[j]), acc);
  }
  return acc;
}

__global__ __launch_bounds__(kOptBlock) void norm_kernel(const NormTile* __restrict__ tiles, int32_t ntiles,
                                                         double* __restrict__ partials, NormResult* result,
                                                         double max_norm, double grad_scale, int32_t skip_nonfinite) {
  __shared__ double lds[kOptBlock / 64];
  __shared__ bool last;
  double acc = 0.0;
  for (int k = blockIdx.x; k < ntiles; k += gridDim.x) {
    const NormTile t = tiles[k];
    if (t.dtype == kF32) acc = tile_squares<kF32>(t, acc);
    else if (t.dtype == kBF16) acc = tile_squares<kBF16>(t, acc);
    else acc = tile_squares<kF16>(t, acc);
  }
  acc = block_sum(acc, lds);
  if (threadIdx.x == 0) {
    __hip_atomic_store(&partials[blockIdx.x], acc, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    last = __hip_atomic_fetch_add(&result->arrived, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  acc = 0.0;
  for (int k = threadIdx.x; k < static_cast<int>(gridDim.x); k += kOptBlock)
    acc += __hip_atomic_load(&partials[k], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  acc = block_sum(acc, lds);
  if (threadIdx.x == 0) {
    const double n = __builtin_sqrt(acc) * __builtin_fabs(grad_scale);
    result->norm = static_cast<float>(n);
    result->coef = n > max_norm ? static_cast<float>(max_norm / n) : 1.0f;
    result->skip = skip_nonfinite && !__builtin_isfinite(n);
    result->arrived = 0;
  }
}

// ---------------------------------------------------------------------------
// AdamW.

// The 16 + 16 random bits of elements 4 group .. 4 group + 3 (high half: m,
// low half: r), counter-based: multiply and xor-shift rounds over the group's
// index under the step's key, then a short round per element.
__device__ __forceinline__ v4u random_bits(uint64_t group, uint32_t key0, uint32_t key1) {
  uint32_t h = static_cast<uint32_t>(group) * 0x9C8E5A6Du + static_cast<uint32_t>(group >> 32) * 0x7F4A3C15u + key0;
  h ^= h >> 15;
  h *= 0x85D3B2A7u;
  h ^= (h >> 13) ^ key1;
  h *= 0xC5A7E36Bu;
  h ^= h >> 16;
  v4u x;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t y = h + j * 0x6D2B4E95u;
    y ^= y >> 16;
    y *= 0xB5297A4Du;
    x[j] = y ^ (y >> 15);
  }
  return x;
}

// The largest of the 16 lanes of a DPP row, in all of them. Every lane of the
// wave takes part.
template <int ROR>
__device__ __forceinline__ uint32_t row_rotate(uint32_t x) {
  return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x120 + ROR, 0xf, 0xf, true));
}
__device__ __forceinline__ uint32_t row_max(uint32_t x) {
  x = max(x, row_rotate<8>(x));
  x = max(x, row_rotate<4>(x));
  x = max(x, row_rotate<2>(x));
  return max(x, row_rotate<1>(x));
}

__device__ __forceinline__ float as_float(uint32_t x) { return __builtin_bit_cast(float, x); }
__device__ __forceinline__ uint32_t as_bits(float x) { return __builtin_bit_cast(uint32_t, x); }

__device__ __forceinline__ v4f decode4(uint32_t codes, uint32_t scale) {
  const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(codes), false);
  const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(codes), true);
  const float f = as_float(scale << 23);
  return v4f{lo[0] * f, lo[1] * f, hi[0] * f, hi[1] * f};
}

// e4m3 codes of four elements and the scale of their block (the 64 elements of
// the lane's row). The scale is the smallest power of two with max|x| / scale
// <= 448; then |x| / scale is cut to 3 fraction bits after the random bits are
// added below them (below 2^-6, where all steps are 2^-9, 2^-6 is added first
// so that the same cut falls on 2^-9). ROOT: r > 0 keeps at least the smallest
// code, since the step divides by it. Elements that are not finite become NaN
// and do not count for the scale.
template <bool ROOT>
__device__ __forceinline__ uint32_t encode4(v4f x, v4u random, uint32_t* scale) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t a = as_bits(x[j]) & 0x7FFFFFFFu;
    top = max(top, a < 0x7F800000u ? a : 0u);
  }
  top = row_max(top);
  const int s = max(static_cast<int>(top >> 23) + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0) - 8, 1);
  *scale = static_cast<uint32_t>(s);
  const float inv = as_float(static_cast<uint32_t>(254 - s) << 23);
  float z[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t u = ROOT ? (random[j] & 0xFFFFu) << 4 : (random[j] >> 16) << 4;
    const float y = __builtin_fabsf(x[j]) * inv;
    const float low = y < 0.015625f ? 0.015625f : 0.0f;
    float c = as_float((as_bits(y + low) + u) & 0xFFF00000u) - low;
    if (ROOT && y > 0.0f) c = __builtin_fmaxf(c, 0.001953125f);
    c = __builtin_copysignf(c, x[j]);
    z[j] = __builtin_isfinite(x[j]) ? c : __builtin_nanf("");
  }
  int codes = __builtin_amdgcn_cvt_pk_fp8_f32(z[0], z[1], 0, false);
  codes = __builtin_amdgcn_cvt_pk_fp8_f32(z[2], z[3], codes, true);
  return static_cast<uint32_t>(codes);
}

struct AdamwArgs {
  const AdamwTile* tiles;
  const uint64_t* replicas;
  StepScalars* scalars;
  const NormResult* clip;
  const float* lr_device;
  double lr, beta1d, beta2d;
  uint64_t seed;
  float grad_scale, beta1, beta2, one_minus_beta1, one_minus_beta2, eps;
  int32_t ntiles, R, P;
};

template <int PD, int GD, bool MASTER, bool F8>
__global__ __launch_bounds__(kOptBlock) void adamw_kernel(const AdamwArgs a) {
  constexpr int SD = MASTER ? kF32 : PD;
  float gs = a.grad_scale;
  if (a.clip != nullptr) {
    if (a.clip->skip) return;            // every workgroup alike: the step does not count
    gs *= a.clip->coef;
  }
  const StepScalars sc = *a.scalars;
  const double lr = a.lr_device != nullptr ? static_cast<double>(*a.lr_device) : a.lr;
  for (int k = blockIdx.x; k < a.ntiles; k += gridDim.x) {
    const AdamwTile t = a.tiles[k];
    const float decay = static_cast<float>(1.0 - lr * t.lr_scale * t.weight_decay);
    const float rate = static_cast<float>(lr * t.lr_scale * sc.inv_bc1);
    // all lanes of a wave stay in the loop together (row_max), those beyond
    // the end on zeros that are not stored
    for (int i0 = 0; i0 < t.len; i0 += 4 * kOptBlock) {
      const int i = i0 + 4 * static_cast<int>(threadIdx.x);
      const int left = t.len - i;
      v4f w = load4<SD>(t.src, i, left);
      const v4f g = load4<GD>(t.grad, i, left) * gs;
      v4f m, v;
      if constexpr (F8) {
        uint32_t ms = 0, rs = 0;
        if (left > 0) {
          ms = G<const uint8_t>(t.avg_scale)[i / kStateBlock];
          rs = G<const uint8_t>(t.root_scale)[i / kStateBlock];
        }
        m = decode4(load_codes(t.avg, i, left), ms);
        v = decode4(load_codes(t.second, i, left), rs);
        v = v * v;
      } else {
        m = load4<kF32>(t.avg, i, left);
        v = load4<kF32>(t.second, i, left);
      }
      m = m * a.beta1 + g * a.one_minus_beta1;
      v = v * a.beta2 + (g * g) * a.one_minus_beta2;
      v4f r;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        r[j] = __builtin_sqrtf(v[j]);
        w[j] = w[j] * decay - (m[j] / (r[j] * sc.inv_rbc2 + a.eps)) * rate;
      }
      store4<PD>(t.out, i, left, w);
      if constexpr (MASTER) store4<kF32>(t.src, i, left, w);
      for (int rep = 1; rep < a.R; ++rep)
        store4<PD>(a.replicas[static_cast<int64_t>(rep - 1) * a.P + t.var] +
                       static_cast<uint64_t>(t.start) * sizeof(typename Elem<PD>::one),
                   i, left, w);
      if constexpr (F8) {
        const v4u random = random_bits(t.group0 + static_cast<uint64_t>(i >> 2), sc.key0, sc.key1);
        uint32_t ms, rs;
        const uint32_t mc = encode4<false>(m, random, &ms);
        const uint32_t rc = encode4<true>(r, random, &rs);
        store_codes(t.avg, i, left, mc);
        store_codes(t.second, i, left, rc);
        if ((threadIdx.x & 15) == 0 && left > 0) {
          G<uint8_t>(t.avg_scale)[i / kStateBlock] = static_cast<uint8_t>(ms);
          G<uint8_t>(t.root_scale)[i / kStateBlock] = static_cast<uint8_t>(rs);
        }
      } else {
        store4<kF32>(t.avg, i, left, m);
        store4<kF32>(t.second, i, left, v);
      }
    }
  }
  // The workgroup that is done last has seen every other read the scalars: it
  // advances them for the next step.
  __syncthreads();
  if (threadIdx.x == 0 &&
      __hip_atomic_fetch_add(&a.scalars->arrived, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1)
    *a.scalars = step_scalars(sc.done + 1, a.beta1d, a.beta2d, a.seed);
}

// ---------------------------------------------------------------------------

// The handle's device for the duration of a call, the caller's afterwards.
class OnDevice {
 public:
  explicit OnDevice(int device) {
    if (hipGetDevice(&before_) != hipSuccess) before_ = device;
    if (before_ != device) ok_ = hipSetDevice(device) == hipSuccess;
    changed_ = ok_ && before_ != device;
  }
  ~OnDevice() {
    if (changed_) (void)hipSetDevice(before_);
  }
  OnDevice(const OnDevice&) = delete;
  OnDevice& operator=(const OnDevice&) = delete;
  bool ok() const { return ok_; }

 private:
  int before_ = 0;
  bool ok_ = true, changed_ = false;
};

template <int PD, int GD, bool MASTER, bool F8>
void launch_adamw(const AdamwArgs& a, hipStream_t s) {
  const int blocks = a.ntiles > 0 ? a.ntiles : 1;
  hipLaunchKernelGGL((adamw_kernel<PD, GD, MASTER, F8>), dim3(blocks), dim3(kOptBlock), 0, s, a);
}

template <int PD, int GD>
void pick_adamw(const AdamwLaunch& l, const AdamwArgs& a, hipStream_t s) {
  if constexpr (PD != kF32) {
    if (l.master) return l.f8 ? launch_adamw<PD, GD, true, true>(a, s) : launch_adamw<PD, GD, true, false>(a, s);
  }
  return l.f8 ? launch_adamw<PD, GD, false, true>(a, s) : launch_adamw<PD, GD, false, false>(a, s);
}

template <int PD>
void pick_adamw(const AdamwLaunch& l, const AdamwArgs& a, hipStream_t s) {
  if (l.grad_dtype == kF32) return pick_adamw<PD, kF32>(l, a, s);
  if (l.grad_dtype == kBF16) return pick_adamw<PD, kBF16>(l, a, s);
  return pick_adamw<PD, kF16>(l, a, s);
}

class HipOptimDevice final : public OptimDevice {
 public:
  int current(int* device, std::string* err) override {
    HIP_OK(hipGetDevice(device), "hipGetDevice");
    return kOk;
  }

  int upload(int device, void* stream, void* dst, const void* src, size_t bytes, std::string* err) override {
    return copy(device, stream, dst, src, bytes, hipMemcpyHostToDevice, err);
  }

  int download(int device, void* stream, void* dst, const void* src, size_t bytes, std::string* err) override {
    return copy(device, stream, dst, src, bytes, hipMemcpyDeviceToHost, err);
  }

  int norm(const NormLaunch& l, std::string* err) override {
    const OnDevice on(l.device);
    if (!on.ok()) return no_device(err);
    const int blocks = l.ntiles < kNormBlocks ? (l.ntiles > 0 ? l.ntiles : 1) : kNormBlocks;
    hipLaunchKernelGGL(norm_kernel, dim3(blocks), dim3(kOptBlock), 0, static_cast<hipStream_t>(l.stream), l.tiles,
                       l.ntiles, l.partials, l.result, l.max_norm, l.grad_scale, l.skip_nonfinite);
    HIP_OK(hipGetLastError(), "launch norm_kernel");
    return kOk;
  }

  int adamw(const AdamwLaunch& l, std::string* err) override {
    const OnDevice on(l.device);
    if (!on.ok()) return no_device(err);
    AdamwArgs a;
    a.tiles = l.tiles;
    a.replicas = l.replicas;
    a.scalars = l.scalars;
    a.clip = l.clip;
    a.lr_device = l.lr_device;
    a.lr = l.lr;
    a.beta1d = l.beta1;
    a.beta2d = l.beta2;
    a.seed = l.seed;
    a.grad_scale = static_cast<float>(l.grad_scale);
    a.beta1 = static_cast<float>(l.beta1);
    a.beta2 = static_cast<float>(l.beta2);
    a.one_minus_beta1 = static_cast<float>(1.0 - l.beta1);
    a.one_minus_beta2 = static_cast<float>(1.0 - l.beta2);
    a.eps = static_cast<float>(l.eps);
    a.ntiles = l.ntiles;
    a.R = l.R;
    a.P = l.P;
    hipStream_t s = static_cast<hipStream_t>(l.stream);
    if (l.param_dtype == kF32) pick_adamw<kF32>(l, a, s);
    else if (l.param_dtype == kBF16) pick_adamw<kBF16>(l, a, s);
    else pick_adamw<kF16>(l, a, s);
    HIP_OK(hipGetLastError(), "launch adamw_kernel");
    return kOk;
  }

 private:
  static int no_device(std::string* err) {
    *err = "hipSetDevice failed";
    return kErrHip;
  }

  int copy(int device, void* stream, void* dst, const void* src, size_t bytes, hipMemcpyKind kind,
           std::string* err) {
    const OnDevice on(device);
    if (!on.ok()) return no_device(err);
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipStreamCaptureStatus st = hipStreamCaptureStatusNone;
    HIP_OK(hipStreamIsCapturing(s, &st), "hipStreamIsCapturing");
    if (st != hipStreamCaptureStatusNone) {   // the host memory is gone when the graph replays
      *err = "this call cannot be captured into a graph";
      return kErrState;
    }
    HIP_OK(hipMemcpyAsync(dst, src, bytes, kind, s), "hipMemcpyAsync");
    HIP_OK(hipStreamSynchronize(s), "hipStreamSynchronize");
    return kOk;
  }
};

}  // namespace

OptimDevice* optim_device() {
  static HipOptimDevice d;
  return &d;
}

}  // namespace ddpb
