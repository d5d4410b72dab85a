// optim.hip -- CDNA4 (gfx950) kernels of the operators that follow a
// synchronisation: the global gradient norm and the AdamW step, with 32-bit or
// 8-bit states, over many tensors in one launch each.
#include <hip/hip_runtime.h>

#include "optim.hpp"

namespace ddpb {
namespace {

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

// A table entry that nothing writes while the kernel runs: a scalar load.
template <typename T>
__device__ __forceinline__ T constant(const T* p) {
  T x;
  __builtin_memcpy(&x, (const __attribute__((address_space(4))) T*)p, sizeof(T));
  return x;
}

template <typename T>
__device__ __forceinline__ __attribute__((address_space(1))) T* G(uint64_t a) {
  return (__attribute__((address_space(1))) T*)a;
}

// Address of element i < 2^30 of the array at `a` (a 32-bit offset, which the
// memory instructions add for free).
template <int D>
__device__ __forceinline__ uint64_t element(uint64_t a, int i) {
  return a + static_cast<uint32_t>(i) * static_cast<uint32_t>(sizeof(typename Elem<D>::one));
}

// Elements i .. i+3 of the array at `a`, of which `left` (1..4, or more) exist;
// FULL: all four do. Every byte is touched once per call, so all accesses are
// non-temporal.
template <int D, bool FULL>
__device__ __forceinline__ typename Elem<D>::raw load4(uint64_t a, int i, int left) {
  typedef typename Elem<D>::one one;
  typedef typename Elem<D>::four four;
  if (FULL || left >= 4) return __builtin_nontemporal_load(G<const four>(element<D>(a, i)));
  typename Elem<D>::raw x = {};
  const auto* p = G<const one>(a) + i;
  if (left > 0) x.x = p[0];
  if (left > 1) x.y = p[1];
  if (left > 2) x.z = p[2];
  return x;
}

// Full vectors are stored through a buffer resource over the tile, which lets
// the store carry device scope beside the non-temporal hint (4 workgroups per
// CU: 1.62 against 1.65 ms for BERT-large in fp32, 0.245 against 0.264 ms for
// ResNet-50 with 8 replicas). Only addresses on a multiple of 4.
typedef unsigned int v2u __attribute__((ext_vector_type(2)));
constexpr int kPolicyDeviceNT = 2 | 16;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(uint64_t a) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>((static_cast<uint64_t>(hi) << 32) | lo), 0,
                                           kOptimTile * 4, 0x00020000);
}

template <typename R>
__device__ __forceinline__ v4f widen(R x) { return __builtin_convertvector(x, v4f); }

// Rounds to nearest even where D has 16 bits: the one rounding a stored
// parameter goes through (its fp32 master, if there is one, keeps the rest).
template <int D, bool FULL>
__device__ __forceinline__ void store4(uint64_t a, int i, int left, v4f x) {
  typedef typename Elem<D>::one one;
  typedef typename Elem<D>::four four;
  typedef typename Elem<D>::raw raw;
  const raw y = __builtin_convertvector(x, raw);
  if (FULL && (sizeof(one) == 4 || (a & 3) == 0)) {
    if constexpr (sizeof(one) == 4)
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u, y), rsrc(a), i * 4, 0, kPolicyDeviceNT);
    else
      __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(v2u, y), rsrc(a), i * 2, 0, kPolicyDeviceNT);
    return;
  }
  if (FULL || left >= 4) {
    __builtin_nontemporal_store(static_cast<four>(y), G<four>(element<D>(a, i)));
    return;
  }
  auto* p = G<one>(a) + i;
  if (left > 0) p[0] = y.x;
  if (left > 1) p[1] = y.y;
  if (left > 2) p[2] = y.z;
}

template <bool FULL>
__device__ __forceinline__ uint32_t load_codes(uint64_t a, int i, int left) {
  typedef uint32_t u1 __attribute__((aligned(1)));
  if (FULL || left >= 4) return __builtin_nontemporal_load(G<const u1>(a + static_cast<uint32_t>(i)));
  const auto* p = G<const uint8_t>(a) + i;
  uint32_t x = 0;
  if (left > 0) x = p[0];
  if (left > 1) x |= static_cast<uint32_t>(p[1]) << 8;
  if (left > 2) x |= static_cast<uint32_t>(p[2]) << 16;
  return x;
}

template <bool FULL>
__device__ __forceinline__ void store_codes(uint64_t a, int i, int left, uint32_t x) {
  typedef uint32_t u1 __attribute__((aligned(1)));
  if (FULL && (a & 3) == 0) {
    __builtin_amdgcn_raw_buffer_store_b32(x, rsrc(a), i, 0, kPolicyDeviceNT);
    return;
  }
  if (FULL || left >= 4) {
    __builtin_nontemporal_store(x, G<u1>(a + static_cast<uint32_t>(i)));
    return;
  }
  auto* p = G<uint8_t>(a) + i;
  if (left > 0) p[0] = static_cast<uint8_t>(x);
  if (left > 1) p[1] = static_cast<uint8_t>(x >> 8);
  if (left > 2) p[2] = static_cast<uint8_t>(x >> 16);
}

// ---------------------------------------------------------------------------
// Counts a workgroup as done; true for the last one. One counter took 12.4 ns
// for each workgroup (82,000 tiles: 1.02 ms, whatever else the kernel did), so
// workgroups count on 64 lines, and the last of each line on one more.
__device__ __forceinline__ bool last_to_arrive(uint32_t* counters) {
  const uint32_t slot = blockIdx.x % kArriveSlots;
  const uint32_t slots = min(gridDim.x, static_cast<uint32_t>(kArriveSlots));
  const uint32_t mine = (gridDim.x - slot + kArriveSlots - 1) / kArriveSlots;
  auto count = [&](uint32_t* c, uint32_t all) {
    if (__hip_atomic_fetch_add(c, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) != all - 1) return false;
    __hip_atomic_store(c, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return true;
  };
  return count(counters + slot * kArriveStride, mine) && count(counters + kArriveSlots * kArriveStride, slots);
}

// ---------------------------------------------------------------------------
// Global norm: n = grad_scale * sqrt(sum g^2), coef = max_norm / n if n >
// max_norm, else 1. Summed in fp64, in an order that only the sizes decide:
// each lane over its elements, each workgroup over its lanes, the workgroup
// that finishes last over all partial sums.
//
// Bound by HBM: 512 workgroups of 512 threads, 16 KiB of a tensor each at a
// time, two 16-byte loads in flight per lane, non-temporal: 186 us for
// BERT-large's 1.34 GB in fp32 (7.2 TB/s), 99 us in bf16 (6.8 TB/s). 256 x
// 1024 threads or 1024 x 256 of them took 191-198 us, one load in flight 284,
// four 198. What is left of a tensor after its whole tiles is summed element by
// element (ResNet-50's 161 tensors: 19.1 us in fp32, 5.4 TB/s, 13.3 us in bf16,
// 3.9 TB/s; 5000 tensors of 64 elements 7.2 us).
constexpr int kNormThreads = 512;
constexpr int kNormUnroll = 2;

__device__ __forceinline__ double block_sum(double x, double* lds) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  x = lds[0];
#pragma unroll
  for (int w = 1; w < kNormThreads / 64; ++w) x += lds[w];
  return x;
}

// 16 bytes of a gradient, or the elements of them that exist, as fp32 pairs.
template <int D>
struct Chunk {
  static constexpr int kElems = D == kF32 ? 4 : 8;
  typedef typename Elem<D>::one raw __attribute__((ext_vector_type(kElems)));
  typedef raw any __attribute__((aligned(sizeof(typename Elem<D>::one))));
};

template <int D>
__device__ __forceinline__ void add_squares(typename Chunk<D>::raw x, double (&acc)[4]) {
#pragma unroll
  for (int j = 0; j < Chunk<D>::kElems; ++j) {
    const double y = static_cast<double>(static_cast<float>(x[j]));
    acc[j & 3] = __builtin_fma(y, y, acc[j & 3]);
  }
}

template <int D>
__device__ __forceinline__ void tile_squares(const NormTile& t, double (&acc)[4]) {
  typedef Chunk<D> C;
  constexpr int kStep = C::kElems * kNormThreads, U = kNormUnroll;
  const int first = C::kElems * static_cast<int>(threadIdx.x);
  int at = 0;
  for (; at + kStep * U <= t.len; at += kStep * U) {
    typename C::raw x[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      x[u] = __builtin_nontemporal_load(G<const typename C::any>(element<D>(t.grad, at + kStep * u + first)));
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < U; ++u) add_squares<D>(x[u], acc);
  }
  for (int i = at + threadIdx.x; i < t.len; i += kNormThreads) {
    const double y = static_cast<double>(static_cast<float>(G<const typename Elem<D>::one>(t.grad)[i]));
    acc[0] = __builtin_fma(y, y, acc[0]);
  }
}

__global__ __launch_bounds__(kNormThreads) void norm_kernel(const NormTile* __restrict__ tiles, int32_t ntiles,
                                                            double* partials, uint32_t* arrived, NormResult* result,
                                                            double max_norm, double grad_scale,
                                                            int32_t skip_nonfinite) {
  __shared__ double lds[kNormThreads / 64];
  __shared__ bool last;
  double part[4] = {0.0, 0.0, 0.0, 0.0};
  for (int k = blockIdx.x; k < ntiles; k += gridDim.x) {
    const NormTile t = constant(tiles + k);
    if (t.dtype == kF32) tile_squares<kF32>(t, part);
    else if (t.dtype == kBF16) tile_squares<kBF16>(t, part);
    else tile_squares<kF16>(t, part);
  }
  double acc = block_sum((part[0] + part[1]) + (part[2] + part[3]), lds);
  if (threadIdx.x == 0) {
    // The exchange has happened where all XCDs see it once its old value is
    // back: no fence (whose L2 write-back cost 45 ns a workgroup, one after
    // the other) has to stand between it and the count.
    const uint64_t old = __hip_atomic_exchange(reinterpret_cast<uint64_t*>(partials + blockIdx.x),
                                               __builtin_bit_cast(uint64_t, acc), __ATOMIC_RELAXED,
                                               __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("" : : "v"(old) : "memory");
    last = last_to_arrive(arrived);
  }
  __syncthreads();
  if (!last) return;
  acc = 0.0;
  for (int k = threadIdx.x; k < static_cast<int>(gridDim.x); k += kNormThreads)
    acc += __hip_atomic_load(&partials[k], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  acc = block_sum(acc, lds);
  if (threadIdx.x == 0) {
    const double n = __builtin_sqrt(acc) * __builtin_fabs(grad_scale);
    const float norm = static_cast<float>(n);   // infinite above fp32's range
    result->norm = norm;
    result->coef = n > max_norm ? static_cast<float>(max_norm / n) : 1.0f;
    result->skip = skip_nonfinite && !__builtin_isfinite(norm);
  }
}

// ---------------------------------------------------------------------------
// AdamW.

// The random bits of a group of four elements.
__device__ __forceinline__ v4u random_bits(uint32_t h, uint32_t key1) {
  h = hash_mix(h, key1);
  v4u x;
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = hash_element(h, j);
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

constexpr uint32_t kInf = 0x7F800000u;

// Values of four codes under a scale, 2^(scale - 127).
__device__ __forceinline__ v4f decode4(uint32_t codes, uint32_t scale) {
  const float f = as_float(scale << 23);
  const auto lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(codes, f, false);
  const auto hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(codes, f, true);
  return v4f{lo[0], lo[1], hi[0], hi[1]};
}

// e4m3 codes of four elements and the scale of their block, the 64 elements of
// the lane's row, whose largest magnitude has the bits `top`. The scale is the
// smallest power of two with max|x| / scale <= 448; the hardware's stochastic
// conversion divides by it, adds the random bits below the 3 fraction bits (or
// below the step of 2^-9 under 2^-6) and cuts there. ROOT: r > 0 keeps at
// least the smallest code, since the step divides by it. x is 2^SHIFT times
// the value that is stored.
template <bool ROOT, int SHIFT>
__device__ __forceinline__ uint32_t encode4(v4f x, uint32_t top, v4u random, uint32_t* scale) {
  // top's exponent, one more if its fraction is over 3/4, less 8; as the bits of a float
  const uint32_t bits = max(top + 0x1FFFFFu, static_cast<uint32_t>(9 + SHIFT) << 23) - (8u << 23);
  *scale = (bits >> 23) - SHIFT;
  const float f = as_float(bits & kInf);
  // fmed3: with x = 0, 0 is the middle one; else x 2^127 is over `least` < 2^48
  // (for all x >= 2^-63, which did not underflow).
  const float least = f * 0x1p-9f;
  int codes = 0;
#define DDPB_SR(J)                                                                                     \
  {                                                                                                    \
    const float y = !ROOT ? x[J]                                                                       \
                    : SHIFT ? __builtin_amdgcn_fmed3f(x[J], least, x[J] * 0x1p127f)                    \
                            : __builtin_fmaxf(x[J], x[J] > 0.0f ? least : 0.0f);                       \
    const uint32_t u = ROOT ? random[J] << 16 : random[J] & 0xFFFF0000u;                               \
    codes = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(codes, y, u, f, J);                               \
  }
  DDPB_SR(0) DDPB_SR(1) DDPB_SR(2) DDPB_SR(3)
#undef DDPB_SR
  return static_cast<uint32_t>(codes);
}

__device__ __forceinline__ uint32_t magnitude(float x) { return as_bits(x) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t top4(v4f x) {
  return max(max(magnitude(x.x), magnitude(x.y)), max(magnitude(x.z), magnitude(x.w)));
}

// The same for values of any kind: those that are not finite become NaN and do
// not count for the scale.
template <bool ROOT>
__device__ __forceinline__ uint32_t encode4_any(v4f x, v4u random, uint32_t* scale) {
  uint32_t nan = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (magnitude(x[j]) >= kInf) {
      x[j] = 0.0f;
      nan |= 0x7Fu << (8 * j);
    }
  return encode4<ROOT, 0>(x, row_max(top4(x)), random, scale) | nan;
}

// Square root and quotient in 9 and 7 issue slots instead of 16 and 15: an
// estimate, its residual by fma, one correction. For normal arguments with
// normal results 16.8 M random ones each gave the bits of the IEEE sequences
// (samples, no proof). The 8-bit step is bound by instructions.
//
// v below 2^-126: the estimate is infinite there (0 and all numbers that are not
// normal), and its bound of 2^63 = 1 / sqrt(2^-126) takes the root on from 2^-63
// downwards without a jump: 2^-63 (1.5 c - c^2 / 2) for v = 2^-126 c, never above
// the true 2^-63 sqrt(c), and 0 for 0.
__device__ __forceinline__ float fast_sqrt(float v) {
  const float h = __builtin_fminf(__builtin_amdgcn_rsqf(v), 0x1p63f);
  const float r = v * h;
  return __builtin_fmaf(__builtin_fmaf(-r, r, v), 0.5f * h, r);
}
// Divisors whose reciprocal is a normal number, too (an estimate of one that is
// not would be 0 or infinite, and 0 / d then NaN).
constexpr float kLeastDivisor = 0x1p-126f, kMostDivisor = 0x1p126f;
__device__ __forceinline__ float fast_div(float x, float d) {
  const float c = __builtin_amdgcn_rcpf(d);
  const float q = x * c;
  return __builtin_fmaf(__builtin_fmaf(-d, q, x), c, q);
}

struct AdamwArgs {
  const AdamwTile* tiles;
  const AdamwVar* vars;
  const uint64_t* replicas;
  StepScalars* scalars;
  uint32_t* arrived;
  const NormResult* clip;
  const float* lr_device;
  double lr, beta1d, beta2d;
  uint64_t seed;
  float grad_scale, beta1, beta2, one_minus_beta1, one_minus_beta2, eps;
  int32_t whole, rests, R, P;
  // 8-bit states: waves with an m or r of at least these bits take no shortcuts.
  // (Between the floats it made the compiler keep five of them in LDS, 5 KiB a
  // workgroup: ResNet-50 68 -> 82 us.)
  uint32_t special;
};

// A tile with its addresses.
struct Tile {
  uint64_t src, out, grad, avg, second, avg_scale, root_scale;
  int64_t start;
  int32_t len, var;
};

// What a lane reads for four elements, as stored.
template <int SD, int GD, bool F8>
struct Quad {
  typename Elem<SD>::raw w;
  typename Elem<GD>::raw g;
  v4f m, v;                    // fp32 states
  uint32_t mc, rc, ms, rs;     // codes and scales
};

template <int SD, int GD, bool F8, bool FULL>
__device__ __forceinline__ void load_quad(Quad<SD, GD, F8>& q, const Tile& t, int i) {
  const int left = t.len - i;
  q.w = load4<SD, FULL>(t.src, i, left);
  q.g = load4<GD, FULL>(t.grad, i, left);
  if constexpr (F8) {
    q.mc = load_codes<FULL>(t.avg, i, left);
    q.rc = load_codes<FULL>(t.second, i, left);
    q.ms = q.rs = 0;
    if (FULL || left > 0) {
      const uint32_t block = static_cast<uint32_t>(i) / kStateBlock;
      q.ms = G<const uint8_t>(t.avg_scale)[block];
      q.rs = G<const uint8_t>(t.root_scale)[block];
    }
  } else {
    q.m = load4<kF32, FULL>(t.avg, i, left);
    q.v = load4<kF32, FULL>(t.second, i, left);
  }
}

struct StepValues {      // of the step, in registers
  float gs, inv_rbc2;
  uint32_t key1;
  float decay, rate;     // of the tile's variable
  uint32_t hash;         // of the lane's first group in the tile
  uint32_t tile;         // low word of the tile's first group
};

// The replicas' addresses are read between the stores, which may alias them as
// far as the compiler knows: each turn loads one and waits for it, and with it
// for the store before (vmcnt counts both). Likely what separates ResNet-50 with
// 8 replicas (5.9 TB/s in fp32, 5.4 with 8-bit states) from one (6.4 TB/s).
template <int PD, bool MASTER, bool FULL>
__device__ __forceinline__ void store_params(v4f w, const Tile& t, int i, const AdamwArgs& a) {
  const int left = t.len - i;
  store4<PD, FULL>(t.out, i, left, w);
  if constexpr (MASTER) store4<kF32, FULL>(t.src, i, left, w);
  for (int rep = 1; rep < a.R; ++rep)
    store4<PD, FULL>(a.replicas[static_cast<int64_t>(rep - 1) * a.P + t.var] +
                         static_cast<uint64_t>(t.start) * sizeof(typename Elem<PD>::one),
                     i, left, w);
}

template <int PD, int GD, bool MASTER, bool FULL>
__device__ __forceinline__ void update_quad(const Quad<MASTER ? kF32 : PD, GD, false>& q, const Tile& t, int at,
                                            int lane4, const AdamwArgs& a, const StepValues& s) {
  const int i = at + lane4, left = t.len - i;
  const v4f g = widen(q.g) * s.gs;
  const v4f m = q.m * a.beta1 + g * a.one_minus_beta1;
  const v4f v = q.v * a.beta2 + (g * g) * a.one_minus_beta2;
  v4f w = widen(q.w);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w[j] = w[j] * s.decay - (m[j] / (__builtin_sqrtf(v[j]) * s.inv_rbc2 + a.eps)) * s.rate;
  store_params<PD, MASTER, FULL>(w, t, i, a);
  store4<kF32, FULL>(t.avg, i, left, m);
  store4<kF32, FULL>(t.second, i, left, v);
}

// 8-bit states. m and v are rounded operation by operation, as in the 32-bit
// step (one rounding more or less would move a code here and there); in the
// parameter's update products are fused into the sums they feed. v and r are
// carried as 2^64 v and 2^32 r, which keeps v normal for roots down to 2^-95
// (below, fast_sqrt lets them underflow gradually). What then overflows (r >
// 4e9), or is not finite, takes the way without shortcuts, and with an eps
// outside fast_div's range everything does. A whole wave goes that way, in which
// the elements that need none of it keep what they have: none depends on what
// lies beside it.
template <int PD, int GD, bool MASTER, bool FULL>
__device__ __forceinline__ void update_quad(const Quad<MASTER ? kF32 : PD, GD, true>& q, const Tile& t, int at,
                                            int lane4, const AdamwArgs& a, const StepValues& s) {
  const int i = at + lane4, left = t.len - i;
  const v4f g = widen(q.g) * s.gs;
  const v4f m = decode4(q.mc, q.ms) * a.beta1 + g * a.one_minus_beta1;
  v4f v = decode4(q.rc, min(q.rs, 222u) + 32u), w = widen(q.w), r;
  v = (v * v) * a.beta2 + (g * g) * (a.one_minus_beta2 * 0x1p64f);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    r[j] = fast_sqrt(v[j]);
    w[j] = __builtin_fmaf(-fast_div(m[j], __builtin_fmaf(r[j], s.inv_rbc2 * 0x1p-32f, a.eps)), s.rate,
                          w[j] * s.decay);
  }
  const uint32_t mtop = as_bits(__builtin_elementwise_maximum(
      __builtin_elementwise_maximum(__builtin_fabsf(m.x), __builtin_fabsf(m.y)),
      __builtin_elementwise_maximum(__builtin_fabsf(m.z), __builtin_fabsf(m.w))));    // NaN stays
  const uint32_t rtop = max(max(as_bits(r.x), as_bits(r.y)), max(as_bits(r.z), as_bits(r.w)));
  const v4u random = random_bits(hash_at(s.hash, s.tile, threadIdx.x, static_cast<uint32_t>(at / 4)), s.key1);
  uint32_t ms, rs, mc, rc;
  if (__builtin_expect(__any(max(mtop, rtop) >= a.special), 0)) {
    v4f u = decode4(q.rc, q.rs);
    u = (u * u) * a.beta2 + (g * g) * a.one_minus_beta2;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool root = magnitude(r[j]) < kInf;
      r[j] = root ? r[j] * 0x1p-32f : __builtin_sqrtf(u[j]);
      const float d = r[j] * s.inv_rbc2 + a.eps;
      if (!root || magnitude(m[j]) >= kInf || !(d >= kLeastDivisor && d <= kMostDivisor))
        w[j] = static_cast<float>(q.w[j]) * s.decay - (m[j] / d) * s.rate;
    }
    mc = encode4_any<false>(m, random, &ms);
    rc = encode4_any<true>(r, random, &rs);
  } else {
    mc = encode4<false, 0>(m, row_max(mtop), random, &ms);
    rc = encode4<true, 32>(r, row_max(rtop), random, &rs);
  }
  store_params<PD, MASTER, FULL>(w, t, i, a);
  store_codes<FULL>(t.avg, i, left, mc);
  store_codes<FULL>(t.second, i, left, rc);
  if ((threadIdx.x & 15) == 0 && (FULL || left > 0)) {
    G<uint8_t>(t.avg_scale)[static_cast<uint32_t>(i) / kStateBlock] = static_cast<uint8_t>(ms);
    G<uint8_t>(t.root_scale)[static_cast<uint32_t>(i) / kStateBlock] = static_cast<uint8_t>(rs);
  }
}

// How a step is cut into workgroups; none of them loops over tiles.
//
// 32-bit states are bound by HBM (28 bytes and some 45 instructions an
// element). One wave and 256 elements per workgroup, 12 or 16 workgroups per
// CU (each reserves its share of the LDS, which the kernel does not use): the
// accesses of the whole GPU then move through every array in step. 12 where a
// workgroup reads and writes 28 bytes an element (BERT-large, fp32: 1.446 ms,
// 6.5 TB/s, against 1.455 with 16, 1.57 with 8 and 1.52 without the limit; two
// replicas 1.625 against 1.655), 16 where it reads less (bf16 without masters:
// 1.125 ms against 1.151) or mostly writes, from five replicas on. At the
// border, BERT-large in fp32, 12 against 16: R = 4 2.081 and 2.094 ms, R = 5
// 2.327 and 2.312, R = 8 3.105 and 2.996; ResNet-50 R = 4 167.0 and 167.3 us,
// R = 5 185.5 and 185.2, R = 8 246.6 and 243. (16-bit parameters with masters
// would take 16 at R = 4 already: ResNet-50 149.5 and 143.0 us.) Other cuts of
// BERT-large in fp32: workgroups of 256 threads at the same waves per CU 1.55,
// two groups per lane 1.61, all workgroups of a tile on one XCD 1.66,
// workgroups of 256 threads that loop over 4096 elements 1.68, and with plain
// loads and stores 1.79.
//
// 8-bit states are bound by instructions nearly as much as by HBM (16 bytes
// and 52 instructions an element with fp32 parameters, 10 bytes and 54 in
// bf16, the whole kernel's): the eight waves per SIMD that 64 registers allow,
// in workgroups of 256 threads, since each workgroup costs a start. Where the
// parameters are 16-bit and have no master, two groups per lane: BERT-large
// 0.547 ms (6.2 TB/s) against 0.592 with one and 0.566 with 7 waves; with
// fp32 parameters or masters one: 0.849 ms (6.3 TB/s) against 0.905 with two
// and 0.875 with 7 waves, bf16 with masters 0.860 against 0.905 with two. The
// scales in scalar loads, or the groups of several lanes per XCD, gained
// nothing.
template <int PD, bool MASTER, bool F8>
struct Shape {
  static constexpr int kThreads = adamw_threads(F8);
  static constexpr int kU = adamw_unroll(PD, MASTER, F8);
  static constexpr int kPart = adamw_part(PD, MASTER, F8);
  static constexpr int kParts = kOptimTile / kPart;
  // Of 160 KiB, in pieces of 1280 bytes: 8 of them for 16 workgroups a CU, 10 for 12.
  static int lds(int R) { return F8 ? 0 : 1280 * ((PD != kF32 && !MASTER) || R > 4 ? 8 : 10); }
  static constexpr int kWaves = F8 ? 8 : 1;                // per SIMD, at least
  static_assert(kParts * kPart == kOptimTile, "a tile is a whole number of parts");
};

template <int PD, int GD, bool MASTER, bool F8>
__global__ __launch_bounds__((Shape<PD, MASTER, F8>::kThreads), (Shape<PD, MASTER, F8>::kWaves))
void adamw_kernel(const AdamwArgs a) {
  constexpr int SD = MASTER ? kF32 : PD;
  typedef Shape<PD, MASTER, F8> S;
  constexpr int U = S::kU, kStep = 4 * S::kThreads;
  // One of the rests (which come first: at the end, nothing would run beside
  // them), or this workgroup's part of a whole tile.
  const int b = static_cast<int>(blockIdx.x) - a.rests;
  const bool rest = b < 0;
  const uint32_t k = rest ? a.whole + static_cast<int>(blockIdx.x) : b / S::kParts;
  const int at = rest ? 0 : b % S::kParts * S::kPart;
  // Two scalar round trips stand before the first data: these, which do not
  // wait for one another (there is always a norm result and a tile to read,
  // neutral ones if need be), and the variable's record. So a step that is to
  // be skipped is one of empty tiles, too: a branch would be a third.
  const AdamwTile e = constant(a.tiles + k);
  const NormResult clip = constant(a.clip);
  const StepScalars sc = constant(a.scalars);
  const AdamwVar x = constant(a.vars + e.var);
  constexpr uint64_t kS = sizeof(typename Elem<SD>::one), kP = sizeof(typename Elem<PD>::one),
                     kG = sizeof(typename Elem<GD>::one), kA = F8 ? 1 : 4;
  const uint64_t from = static_cast<uint64_t>(e.start);
  const Tile t = {x.src + from * kS,    x.out + from * kP,    x.grad + from * kG,
                  x.avg + from * kA,    x.second + from * kA, x.avg_scale + from / kStateBlock,
                  x.root_scale + from / kStateBlock, e.start, clip.skip ? 0 : e.len, e.var};
  const int i = 4 * static_cast<int>(threadIdx.x);
  auto step_values = [&] {
    StepValues s;
    s.gs = a.grad_scale * clip.coef;
    s.inv_rbc2 = sc.inv_rbc2;
    s.key1 = sc.key1;
    const double lr = a.lr_device != nullptr ? static_cast<double>(constant(a.lr_device)) : a.lr;
    s.decay = static_cast<float>(1.0 - lr * x.lr_scale * x.weight_decay);
    s.rate = static_cast<float>(lr * x.lr_scale * sc.inv_bc1);
    const uint64_t group = x.group0 + from / 4;
    s.hash = hash_start(group, threadIdx.x, sc.key0);
    s.tile = static_cast<uint32_t>(group);
    return s;
  };
  if (at + S::kPart <= t.len) {
    Quad<SD, GD, F8> q[U];
#pragma unroll
    for (int u = 0; u < U; ++u) load_quad<SD, GD, F8, true>(q[u], t, at + kStep * u + i);
    __builtin_amdgcn_sched_barrier(0);
    const StepValues s = step_values();
#pragma unroll
    for (int u = 0; u < U; ++u) update_quad<PD, GD, MASTER, true>(q[u], t, at + kStep * u, i, a, s);
  } else {
    // All lanes of a wave stay together (row_max), those beyond the end on zeros
    // that are not stored. As a loop, its constants were spilled.
    const StepValues s = step_values();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int o = at + kStep * u;
      if (o >= t.len) break;
      Quad<SD, GD, F8> q;
      load_quad<SD, GD, F8, false>(q, t, o + i);
      update_quad<PD, GD, MASTER, false>(q, t, o, i, a, s);
    }
  }
  // The workgroup that is done last has seen every other read the scalars: it
  // advances them for the next step.
  __syncthreads();
  if (threadIdx.x == 0 && last_to_arrive(a.arrived) && !clip.skip)
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
  typedef Shape<PD, MASTER, F8> S;
  const unsigned blocks = static_cast<unsigned>(a.whole) * S::kParts + static_cast<unsigned>(a.rests);
  hipLaunchKernelGGL((adamw_kernel<PD, GD, MASTER, F8>), dim3(blocks > 0 ? blocks : 1), dim3(S::kThreads),
                     S::lds(a.R), s, a);
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
    hipLaunchKernelGGL(norm_kernel, dim3(blocks), dim3(kNormThreads), 0, static_cast<hipStream_t>(l.stream), l.tiles,
                       l.ntiles, l.partials, l.arrived, l.result, l.max_norm, l.grad_scale, l.skip_nonfinite);
    HIP_OK(hipGetLastError(), "launch norm_kernel");
    return kOk;
  }

  int adamw(const AdamwLaunch& l, std::string* err) override {
    const OnDevice on(l.device);
    if (!on.ok()) return no_device(err);
    AdamwArgs a;
    a.tiles = l.tiles;
    a.vars = l.vars;
    a.replicas = l.replicas;
    a.scalars = l.scalars;
    a.arrived = l.arrived;
    a.clip = l.clip != nullptr ? l.clip : l.neutral;
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
    // With eps in range every divisor is: r / sqrt(1 - beta2^t) < 2^32 2^27.
    a.special = a.eps >= kLeastDivisor && a.eps <= kMostDivisor / 2 ? kInf : 0;
    a.whole = l.whole;
    a.rests = l.rests;
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
