// group8.hpp -- what the kernels of layer norm, dropout and the embedding share:
// groups of eight consecutive elements, and the dropout's random bits.
#pragma once

#include <hip/hip_runtime.h>

#include "layers.hpp"

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

constexpr int kPolicyDeviceNT = 2 | 16;   // of a buffer store

typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v8f __attribute__((ext_vector_type(8)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

inline uint64_t addr(const void* p) { return static_cast<uint64_t>(reinterpret_cast<uintptr_t>(p)); }

// f with an element type as a constant.
template <typename F>
void by_type(int32_t dtype, F f) {
  if (dtype == kF32) f(std::integral_constant<int, kF32>());
  else if (dtype == kBF16) f(std::integral_constant<int, kBF16>());
  else f(std::integral_constant<int, kF16>());
}

template <int D> struct Of;
template <> struct Of<kF32> { typedef float one; };
template <> struct Of<kBF16> { typedef __bf16 one; };
template <> struct Of<kF16> { typedef _Float16 one; };

template <typename T>
__device__ __forceinline__ __attribute__((address_space(1))) T* G(uint64_t a) {
  return (__attribute__((address_space(1))) T*)a;
}

// How rows end. Rows of a multiple of eight consist of whole groups. Where they
// do not, the last group begins eight elements before the end: its lane reads
// and writes whole vectors too, some of them a second time with the same values
// (one element at a time took up to three times as long). Rows of less than eight
// elements are one group that is read and written element by element.
enum Edge { kWhole = 0, kShifted = 1, kSmall = 2 };

struct Group {
  uint32_t c;      // first column
  int left;        // columns that exist, 0 where the lane has none
  int skip;        // of these, how many the lane before has too (kShifted)
};

template <int EDGE>
__device__ __forceinline__ Group group_at(uint32_t cols, uint32_t c) {
  if (c >= cols) return {0, 0, 0};
  if (EDGE == kSmall) return {c, static_cast<int>(min(cols - c, 8u)), 0};
  if (EDGE == kShifted && cols - c < 8) return {cols - 8, 8, static_cast<int>(c + 8 - cols)};
  return {c, 8, 0};
}

// Whether element j of a group is its lane's own.
template <int EDGE>
__device__ __forceinline__ bool own(const Group& g, int j) {
  return EDGE == kWhole || (EDGE == kShifted ? j >= g.skip : j < g.left);
}

// Eight elements at the address `a` as they lie there, or `left` of them (kSmall).
// Vectors are only assumed to be aligned like their element: gfx950's memory
// instructions take any such address, and odd row lengths and bucket views make
// them.
template <int D>
using Raw = typename Of<D>::one __attribute__((ext_vector_type(8)));

template <int D, int EDGE>
__device__ __forceinline__ Raw<D> load_raw(uint64_t a, int left) {
  typedef typename Of<D>::one one;
  typedef Raw<D> any __attribute__((aligned(sizeof(one))));
  if (EDGE != kSmall || left >= 8) return *G<const any>(a);
  Raw<D> x = {};
#pragma unroll
  for (int j = 0; j < 7; ++j)
    if (j < left) x[j] = G<const one>(a)[j];
  return x;
}

template <int D>
__device__ __forceinline__ v8f widen(Raw<D> x) { return __builtin_convertvector(x, v8f); }

// A group of an array whose type is known when the kernel runs, as fp32.
template <int EDGE>
__device__ __forceinline__ v8f load8(int dtype, uint64_t a, const Group& g) {
  if (dtype == kF32) return widen<kF32>(load_raw<kF32, EDGE>(a + g.c * 4u, g.left));
  if (dtype == kBF16) return widen<kBF16>(load_raw<kBF16, EDGE>(a + g.c * 2u, g.left));
  return widen<kF16>(load_raw<kF16, EDGE>(a + g.c * 2u, g.left));
}

// Rounds to nearest even where D has 16 bits: the one rounding that an output
// goes through. 16-bit vectors are stored non-temporally (BERT-large's norm:
// forward 23.5 us instead of 25.5, backward 28.5 instead of 32.8); fp32's are
// not, whose halves of 16 bytes would reach memory as parts of lines (a backward
// pass of 8192 x 8192: 209 us instead of 203).
template <int D, int EDGE>
__device__ __forceinline__ void store8(uint64_t a, int left, v8f x) {
  typedef typename Of<D>::one one;
  typedef one raw __attribute__((ext_vector_type(8)));
  typedef raw any __attribute__((aligned(sizeof(one))));
  const raw y = __builtin_convertvector(x, raw);
  if (EDGE != kSmall || left >= 8) {
    if constexpr (sizeof(one) == 2) __builtin_nontemporal_store(static_cast<any>(y), G<any>(a));
    else *G<any>(a) = y;
    return;
  }
#pragma unroll
  for (int j = 0; j < 7; ++j)
    if (j < left) G<one>(a)[j] = y[j];
}

// ---------------------------------------------------------------------------
// Dropout's random bits: Philox4x32 (Salmon, Moraes, Dror and Shaw, "Parallel
// random numbers: as easy as 1, 2, 3", 2011) with 7 rounds, the fewest that the
// paper reports to pass all of its test batteries. One call gives 128 bits, 16
// for each of eight elements: the counter is (index of the first / 8, offset),
// the key is the seed. p is thereby a multiple of 2^-16, and what is kept is
// scaled by just that p.
__device__ __forceinline__ v4u philox(uint64_t group, uint64_t offset, uint64_t seed) {
  uint32_t c0 = static_cast<uint32_t>(group), c1 = static_cast<uint32_t>(group >> 32);
  uint32_t c2 = static_cast<uint32_t>(offset), c3 = static_cast<uint32_t>(offset >> 32);
  uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
  for (int r = 0; r < 7; ++r) {
    const uint64_t a = static_cast<uint64_t>(c0) * 0xD2511F53u, b = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    const uint32_t n0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0, n2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
    c1 = static_cast<uint32_t>(b);
    c3 = static_cast<uint32_t>(a);
    c0 = n0;
    c2 = n2;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return v4u{c0, c1, c2, c3};
}

// The offset that a kernel's waves work with.
__device__ __forceinline__ uint64_t offset_of(const DropSpec& d) {
  return d.offset + (d.offset_device != nullptr ? *G<const uint64_t>(reinterpret_cast<uint64_t>(d.offset_device)) : 0);
}

// The 16-bit halves of elements first .. first+7.
__device__ __forceinline__ v4u random8(uint64_t first, uint64_t offset, uint64_t seed) {
  v4u w = philox(first >> 3, offset, seed);
  const uint32_t skip = static_cast<uint32_t>(first) & 7;
  if (skip != 0) {   // eight halves of two groups (rows whose length is no multiple of 8)
    const v4u n = philox((first >> 3) + 1, offset, seed);
    uint32_t x[8] = {w[0], w[1], w[2], w[3], n[0], n[1], n[2], n[3]};
    if (skip & 4) {
#pragma unroll
      for (int j = 0; j < 6; ++j) x[j] = x[j + 2];
    }
    if (skip & 2) {
#pragma unroll
      for (int j = 0; j < 5; ++j) x[j] = x[j + 1];
    }
    if (skip & 1) {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = (x[j] >> 16) | (x[j + 1] << 16);
    }
    w = v4u{x[0], x[1], x[2], x[3]};
  }
  return w;
}

// Drops and scales: what is dropped is 0, whatever stood there.
__device__ __forceinline__ v8f drop8(v8f x, uint64_t first, uint64_t offset, const DropSpec& d) {
  const v4u w = random8(first, offset, d.seed);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t u = j & 1 ? w[j >> 1] >> 16 : w[j >> 1] & 0xFFFFu;
    x[j] = u >= d.limit ? x[j] * d.scale : 0.0f;
  }
  return x;
}

}  // namespace
}  // namespace ddpb
