// layers.hip -- CDNA4 (gfx950) kernels of layer norm, forward and backward, and
// of dropout.
#include "group8.hpp"

namespace ddpb {
int enqueue_lookup(const LookupArgs& a, std::string* err);
int enqueue_lookup_backward(const LookupBackwardArgs& a, std::string* err);

namespace {

// ---------------------------------------------------------------------------
// Sums over the lanes of a row, in all of them and in an order that only LANES
// decides: rotations inside 16 lanes, then halves of the wave, then the waves
// of the workgroup through LDS.
template <int ROR>
__device__ __forceinline__ float rotated(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), 0x120 + ROR, 0xf, 0xf, true));
}

template <int LANES>
__device__ __forceinline__ float wave_sum(float x) {
  x += rotated<8>(x);
  x += rotated<4>(x);
  x += rotated<2>(x);
  x += rotated<1>(x);
  if constexpr (LANES >= 64) {
    // (an element of a vector has to be copied before a bit cast, which takes element 0 otherwise)
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    const auto rows = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const uint32_t r0 = rows[0], r1 = rows[1];
    x = __builtin_bit_cast(float, r0) + __builtin_bit_cast(float, r1);
    const uint32_t v = __builtin_bit_cast(uint32_t, x);
    const auto halves = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    const uint32_t h0 = halves[0], h1 = halves[1];
    x = __builtin_bit_cast(float, h0) + __builtin_bit_cast(float, h1);
  }
  return x;
}

// One or two sums at a time; `lds` holds 2 floats for each wave of a row, and
// alternates between two places from call to call, so that one barrier is
// enough.
template <int LANES, int N>
__device__ __forceinline__ void row_sum(float (&x)[N], float* lds) {
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = wave_sum<LANES>(x[i]);
  if constexpr (LANES > 64) {
    constexpr int W = LANES / 64;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) lds[(threadIdx.x >> 6) * 2 + i] = x[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = lds[i];
#pragma unroll
      for (int w = 1; w < W; ++w) s += lds[w * 2 + i];
      x[i] = s;
    }
  }
}

__device__ __forceinline__ float total(v8f x) { return ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7])); }
__device__ __forceinline__ v8f fma8(v8f a, v8f b, v8f c) { return __builtin_elementwise_fma(a, b, c); }

struct Forward {
  uint64_t x, residual, weight, bias, y, h, stats;
  int64_t x_stride, residual_stride;      // in elements
  uint32_t rows, cols;
  int32_t weight_dtype;
  float eps;
  DropSpec drop;
};

// z of elements c .. c+7 of a row: what the norm is taken of, in fp32.
template <int D, bool FUSED>
__device__ __forceinline__ v8f input8(const Forward& a, int64_t row, uint32_t c, uint64_t offset) {
  typedef typename Of<D>::one one;
  const int64_t left = static_cast<int64_t>(a.cols) - c;
  v8f z = load8<D>(a.x + (row * a.x_stride + c) * sizeof(one), left);
  if constexpr (FUSED) {
    if (a.drop.limit != 0) z = drop8(z, static_cast<uint64_t>(row) * a.cols + c, offset, a.drop);
    if (a.residual != 0) z = z + load8<D>(a.residual + (row * a.residual_stride + c) * sizeof(one), left);
  }
  return z;
}

// y = (z - mean) rstd w + b. The statistics are those of z in fp32 (the mean
// first, then the squares of what is left: no cancellation); h, z as the
// backward pass reads it, is rounded to the type of x for its store only.
template <int D, int LANES, int K, bool FUSED>
__global__ __launch_bounds__(LANES > 256 ? LANES : 256) void norm_forward_kernel(Forward a) {
  typedef typename Of<D>::one one;
  constexpr int THREADS = LANES > 256 ? LANES : 256, ROWS = THREADS / LANES;
  __shared__ float lds[2][LANES > 64 ? LANES / 64 * 2 : 1];
  const uint32_t lane = threadIdx.x % LANES;
  const uint64_t offset = FUSED ? offset_of(a.drop) : 0;
  const float inverse = 1.0f / static_cast<float>(a.cols);
  v8f w[K], b[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const uint32_t c = (lane + k * LANES) * 8;
    const int64_t left = static_cast<int64_t>(a.cols) - c;
    const uint32_t size = a.weight_dtype == kF32 ? 4 : 2;
    w[k] = 1.0f;
    b[k] = 0.0f;
    if (left > 0 && a.weight != 0) w[k] = load8(a.weight_dtype, a.weight + static_cast<uint64_t>(c) * size, left);
    if (left > 0 && a.bias != 0) b[k] = load8(a.weight_dtype, a.bias + static_cast<uint64_t>(c) * size, left);
  }
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / LANES; row < a.rows;
       row += static_cast<int64_t>(gridDim.x) * ROWS) {
    v8f z[K];
    float s[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const uint32_t c = (lane + k * LANES) * 8;
      z[k] = 0.0f;
      if (c < a.cols) z[k] = input8<D, FUSED>(a, row, c, offset);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) s[0] += total(z[k]);
    row_sum<LANES>(s, lds[0]);
    const float mean = s[0] * inverse;
    float q[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const uint32_t c = (lane + k * LANES) * 8;
      if (FUSED && a.h != 0 && c < a.cols)
        store8<D>(a.h + (row * a.cols + c) * sizeof(one), static_cast<int64_t>(a.cols) - c, z[k]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = z[k][j] - mean;
        q[0] = __builtin_fmaf(c + j < a.cols ? d : 0.0f, d, q[0]);
        z[k][j] = d;
      }
    }
    row_sum<LANES>(q, lds[1]);
    const float rstd = 1.0f / __builtin_sqrtf(q[0] * inverse + a.eps);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const uint32_t c = (lane + k * LANES) * 8;
      if (c < a.cols)
        store8<D>(a.y + (row * a.cols + c) * sizeof(one), static_cast<int64_t>(a.cols) - c,
                  fma8(z[k] * rstd, w[k], b[k]));
    }
    if (lane == 0) {
      G<float>(a.stats)[row * 2] = mean;
      G<float>(a.stats)[row * 2 + 1] = rstd;
    }
  }
}

constexpr int kLong = 1024;   // threads for a row that no shape holds in registers

template <int D, bool FUSED>
__global__ __launch_bounds__(kLong) void norm_forward_long_kernel(Forward a) {
  typedef typename Of<D>::one one;
  __shared__ float lds[2][kLong / 64 * 2];
  const uint64_t offset = FUSED ? offset_of(a.drop) : 0;
  const float inverse = 1.0f / static_cast<float>(a.cols);
  const uint32_t size = a.weight_dtype == kF32 ? 4 : 2;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    float s[1] = {0.0f}, q[1] = {0.0f};
    for (uint32_t c = threadIdx.x * 8; c < a.cols; c += kLong * 8) s[0] += total(input8<D, FUSED>(a, row, c, offset));
    row_sum<kLong>(s, lds[0]);
    const float mean = s[0] * inverse;
    for (uint32_t c = threadIdx.x * 8; c < a.cols; c += kLong * 8) {
      const v8f z = input8<D, FUSED>(a, row, c, offset);
      if (FUSED && a.h != 0)
        store8<D>(a.h + (row * a.cols + c) * sizeof(one), static_cast<int64_t>(a.cols) - c, z);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = c + j < a.cols ? z[j] - mean : 0.0f;
        q[0] = __builtin_fmaf(d, d, q[0]);
      }
    }
    row_sum<kLong>(q, lds[1]);
    const float rstd = 1.0f / __builtin_sqrtf(q[0] * inverse + a.eps);
    for (uint32_t c = threadIdx.x * 8; c < a.cols; c += kLong * 8) {
      const int64_t left = static_cast<int64_t>(a.cols) - c;
      v8f w = 1.0f, b = 0.0f;
      if (a.weight != 0) w = load8(a.weight_dtype, a.weight + static_cast<uint64_t>(c) * size, left);
      if (a.bias != 0) b = load8(a.weight_dtype, a.bias + static_cast<uint64_t>(c) * size, left);
      store8<D>(a.y + (row * a.cols + c) * sizeof(one), left,
                fma8((input8<D, FUSED>(a, row, c, offset) - mean) * rstd, w, b));
    }
    if (threadIdx.x == 0) {
      G<float>(a.stats)[row * 2] = mean;
      G<float>(a.stats)[row * 2 + 1] = rstd;
    }
  }
}

// ---------------------------------------------------------------------------
// Backward. With n = (h - mean) rstd and g = dy w:
//   dh = rstd (g - mean g - n mean(g n)) + grad_h,  dx = drop(dh),
//   dweight = sum over rows of dy n,  dbias = sum of dy.
// A workgroup goes over rows, keeps its lanes' parts of the weights' gradients
// in fp32 registers and leaves one partial sum, which norm_weights_kernel adds
// up: no atomics, so the same bits on every run.
struct Backward {
  uint64_t dy, h, stats, grad_h, weight, dh, dx;
  int64_t dy_stride, h_stride, grad_h_stride;   // in elements
  float* partials;                              // [workgroup][dweight, dbias][cols], or NULL
  uint32_t rows, cols;
  int32_t weight_dtype;
  DropSpec drop;
};

template <int D>
__device__ __forceinline__ void store_grads(const Backward& a, int64_t row, uint32_t c, int64_t left, v8f d,
                                            uint64_t offset) {
  typedef typename Of<D>::one one;
  if (a.grad_h != 0) d = d + load8<D>(a.grad_h + (row * a.grad_h_stride + c) * sizeof(one), left);
  const uint64_t at = (row * a.cols + c) * sizeof(one);
  store8<D>(a.dh + at, left, d);
  if (a.drop.limit != 0) store8<D>(a.dx + at, left, drop8(d, static_cast<uint64_t>(row) * a.cols + c, offset, a.drop));
}

template <int D, int LANES, int K>
__global__ __launch_bounds__(LANES == 1024 ? 1024 : LANES == 256 ? 256 : 512) void norm_backward_kernel(Backward a) {
  typedef typename Of<D>::one one;
  constexpr int THREADS = LANES == 1024 ? 1024 : LANES == 256 ? 256 : 512, ROWS = THREADS / LANES;
  __shared__ float lds[2][LANES > 64 ? LANES / 64 * 2 : 1];
  const uint32_t lane = threadIdx.x % LANES, mine = threadIdx.x / LANES;
  const uint64_t offset = offset_of(a.drop);
  const float inverse = 1.0f / static_cast<float>(a.cols);
  const uint32_t size = a.weight_dtype == kF32 ? 4 : 2;
  v8f w[K], dw[K], db[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const uint32_t c = (lane + k * LANES) * 8;
    w[k] = 1.0f;
    dw[k] = db[k] = 0.0f;
    if (c < a.cols && a.weight != 0)
      w[k] = load8(a.weight_dtype, a.weight + static_cast<uint64_t>(c) * size, static_cast<int64_t>(a.cols) - c);
  }
  int turn = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + mine; row < a.rows;
       row += static_cast<int64_t>(gridDim.x) * ROWS, turn ^= 1) {
    const float mean = G<const float>(a.stats)[row * 2], rstd = G<const float>(a.stats)[row * 2 + 1];
    v8f g[K], n[K];
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const uint32_t c = (lane + k * LANES) * 8;
      const int64_t left = static_cast<int64_t>(a.cols) - c;
      g[k] = n[k] = 0.0f;
      if (left > 0) {
        g[k] = load8<D>(a.dy + (row * a.dy_stride + c) * sizeof(one), left);
        n[k] = load8<D>(a.h + (row * a.h_stride + c) * sizeof(one), left);
      }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      n[k] = (n[k] - mean) * rstd;
      dw[k] = fma8(g[k], n[k], dw[k]);
      db[k] = db[k] + g[k];
      g[k] = g[k] * w[k];
      s[0] += total(g[k]);
      s[1] += total(g[k] * n[k]);
    }
    row_sum<LANES>(s, lds[turn]);
    s[0] *= inverse;
    s[1] *= inverse;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const uint32_t c = (lane + k * LANES) * 8;
      const int64_t left = static_cast<int64_t>(a.cols) - c;
      if (left > 0) store_grads<D>(a, row, c, left, (fma8(n[k], v8f(-s[1]), g[k]) - s[0]) * rstd, offset);
    }
  }
  if (a.partials == nullptr) return;
  float* to = a.partials + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
  if constexpr (ROWS == 1) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const uint32_t c = (lane + k * LANES) * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (c + j < a.cols) {
          to[c + j] = dw[k][j];
          to[a.cols + c + j] = db[k][j];
        }
      }
    }
  } else {
    // the rows of the workgroup side by side in LDS, a column to a thread
    constexpr int WIDTH = LANES * K * 8;
    __shared__ float part[ROWS * WIDTH];
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < K; ++k)
        *reinterpret_cast<v8f*>(part + mine * WIDTH + (lane + k * LANES) * 8) = which ? db[k] : dw[k];
      __syncthreads();
      for (uint32_t c = threadIdx.x; c < a.cols; c += THREADS) {
        float x = part[c];
#pragma unroll
        for (int r = 1; r < ROWS; ++r) x += part[r * WIDTH + c];
        to[which * a.cols + c] = x;
      }
    }
  }
}

template <int D>
__global__ __launch_bounds__(kLong) void norm_backward_long_kernel(Backward a) {
  typedef typename Of<D>::one one;
  __shared__ float lds[2][kLong / 64 * 2];
  const uint64_t offset = offset_of(a.drop);
  const float inverse = 1.0f / static_cast<float>(a.cols);
  const uint32_t size = a.weight_dtype == kF32 ? 4 : 2;
  float* to = a.partials == nullptr ? nullptr : a.partials + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
  bool first = true;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, first = false, turn ^= 1) {
    const float mean = G<const float>(a.stats)[row * 2], rstd = G<const float>(a.stats)[row * 2 + 1];
    float s[2] = {0.0f, 0.0f};
    for (int pass = 0; pass < 2; ++pass) {
      for (uint32_t c = threadIdx.x * 8; c < a.cols; c += kLong * 8) {
        const int64_t left = static_cast<int64_t>(a.cols) - c;
        const v8f dy = load8<D>(a.dy + (row * a.dy_stride + c) * sizeof(one), left);
        const v8f n = (load8<D>(a.h + (row * a.h_stride + c) * sizeof(one), left) - mean) * rstd;
        v8f g = dy;
        if (a.weight != 0) g = g * load8(a.weight_dtype, a.weight + static_cast<uint64_t>(c) * size, left);
        if (pass == 1) {
          store_grads<D>(a, row, c, left, (fma8(n, v8f(-s[1]), g) - s[0]) * rstd, offset);
          continue;
        }
        s[0] += total(g);
        s[1] += total(g * n);
        if (to != nullptr) {   // the workgroup's own sums, each element always by the same lane
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (j < left) {
              to[c + j] = __builtin_fmaf(dy[j], n[j], first ? 0.0f : to[c + j]);
              to[a.cols + c + j] = dy[j] + (first ? 0.0f : to[a.cols + c + j]);
            }
          }
        }
      }
      if (pass == 0) {
        row_sum<kLong>(s, lds[turn]);
        s[0] *= inverse;
        s[1] *= inverse;
      }
    }
  }
}

// Adds up the workgroups' sums, 64 columns to a workgroup: 16 waves each take
// every 16th of them.
constexpr int kWeightCols = 64, kWeightWaves = 16;
__global__ __launch_bounds__(kWeightCols * kWeightWaves) void norm_weights_kernel(const float* partials, int32_t count,
                                                                                  uint32_t cols, uint64_t dweight,
                                                                                  uint64_t dbias, int32_t dtype,
                                                                                  int32_t accumulate) {
  __shared__ float part[kWeightWaves][kWeightCols];
  const uint32_t c = blockIdx.x * kWeightCols + (threadIdx.x & 63), wave = threadIdx.x >> 6, which = blockIdx.y;
  const uint64_t out = which ? dbias : dweight;
  if (out == 0) return;
  float x = 0.0f;
  if (c < cols) {
    const float* p = partials + static_cast<int64_t>(which) * cols + c;
#pragma unroll 8
    for (int32_t k = wave; k < count; k += kWeightWaves) x += p[static_cast<int64_t>(k) * 2 * cols];
  }
  part[wave][threadIdx.x & 63] = x;
  __syncthreads();
  if (wave != 0 || c >= cols) return;
#pragma unroll
  for (int w = 1; w < kWeightWaves; ++w) x += part[w][threadIdx.x];
  const uint64_t at = out + static_cast<uint64_t>(c) * (dtype == kF32 ? 4 : 2);
  auto put = [&](auto one) {
    auto* p = G<decltype(one)>(at);
    if (accumulate) x += static_cast<float>(*p);
    *p = static_cast<decltype(one)>(x);
  };
  if (dtype == kF32) put(float());
  else if (dtype == kBF16) put(__bf16());
  else put(_Float16());
}

// ---------------------------------------------------------------------------
// Dropout, with or without a residual. A workgroup takes kDropTile groups of
// eight elements at a time, counted row by row.
struct Drop {
  uint64_t x, residual, y;
  int64_t x_stride, residual_stride;   // in elements
  int64_t groups;                      // rows * groups of a row
  int64_t cols;
  uint32_t row_groups;                 // groups of a row, if there is more than one row
  DropSpec drop;
};
constexpr int kDropThreads = 256, kDropUnroll = 4, kDropTile = kDropThreads * kDropUnroll;

template <int D, bool FLAT>
__global__ __launch_bounds__(kDropThreads) void dropout_kernel(Drop a) {
  typedef typename Of<D>::one one;
  const uint64_t offset = offset_of(a.drop);
  for (int64_t tile = static_cast<int64_t>(blockIdx.x) * kDropTile; tile < a.groups;
       tile += static_cast<int64_t>(gridDim.x) * kDropTile) {
    int64_t row[kDropUnroll], c[kDropUnroll];
    v8f x[kDropUnroll], r[kDropUnroll];
    const int64_t row0 = FLAT ? 0 : tile / a.row_groups;
    const uint32_t rest = FLAT ? 0 : static_cast<uint32_t>(tile - row0 * a.row_groups);
#pragma unroll
    for (int u = 0; u < kDropUnroll; ++u) {
      const uint32_t i = u * kDropThreads + threadIdx.x;
      if (FLAT) {
        row[u] = 0;
        c[u] = (tile + i) * 8;
      } else {
        const uint32_t q = (rest + i) / a.row_groups;
        row[u] = row0 + q;
        c[u] = static_cast<int64_t>(rest + i - q * a.row_groups) * 8;
      }
      x[u] = r[u] = 0.0f;
      if (tile + i < a.groups) {
        x[u] = load8<D>(a.x + (row[u] * a.x_stride + c[u]) * sizeof(one), a.cols - c[u]);
        if (a.residual != 0) r[u] = load8<D>(a.residual + (row[u] * a.residual_stride + c[u]) * sizeof(one), a.cols - c[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kDropUnroll; ++u) {
      if (tile + u * kDropThreads + threadIdx.x >= a.groups) continue;
      const int64_t first = row[u] * a.cols + c[u];
      v8f z = x[u];
      if (a.drop.limit != 0) z = drop8(z, static_cast<uint64_t>(first), offset, a.drop);
      if (a.residual != 0) z = z + r[u];
      store8<D>(a.y + first * sizeof(one), a.cols - c[u], z);
    }
  }
}

uint64_t addr(const void* p) { return static_cast<uint64_t>(reinterpret_cast<uintptr_t>(p)); }

unsigned grid_of(int64_t want, int64_t most) {
  return static_cast<unsigned>(want < 1 ? 1 : want < most ? want : most);
}

template <int D, bool FUSED>
void launch_forward(const Forward& a, hipStream_t s) {
  const NormShape shape = norm_shape(a.cols);
  auto go = [&](auto kernel, int threads, int rows) {
    hipLaunchKernelGGL(kernel, dim3(grid_of((int64_t(a.rows) + rows - 1) / rows, 2048)), dim3(threads), 0, s, a);
  };
  if (shape.lanes == 16) go(norm_forward_kernel<D, 16, 1, FUSED>, 256, 16);
  else if (shape.lanes == 64 && shape.groups == 1) go(norm_forward_kernel<D, 64, 1, FUSED>, 256, 4);
  else if (shape.lanes == 64) go(norm_forward_kernel<D, 64, 2, FUSED>, 256, 4);
  else if (shape.lanes == 256 && shape.groups == 1) go(norm_forward_kernel<D, 256, 1, FUSED>, 256, 1);
  else if (shape.lanes == 256) go(norm_forward_kernel<D, 256, 2, FUSED>, 256, 1);
  else if (shape.lanes == 1024 && shape.groups == 1) go(norm_forward_kernel<D, 1024, 1, FUSED>, 1024, 1);
  else if (shape.lanes == 1024) go(norm_forward_kernel<D, 1024, 2, FUSED>, 1024, 1);
  else go(norm_forward_long_kernel<D, FUSED>, kLong, 1);
}

template <int D>
void launch_backward(const Backward& a, unsigned blocks, hipStream_t s) {
  const NormShape shape = norm_shape(a.cols);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(blocks), dim3(norm_backward_threads(shape)), 0, s, a);
  };
  if (shape.lanes == 16) go(norm_backward_kernel<D, 16, 1>);
  else if (shape.lanes == 64 && shape.groups == 1) go(norm_backward_kernel<D, 64, 1>);
  else if (shape.lanes == 64) go(norm_backward_kernel<D, 64, 2>);
  else if (shape.lanes == 256 && shape.groups == 1) go(norm_backward_kernel<D, 256, 1>);
  else if (shape.lanes == 256) go(norm_backward_kernel<D, 256, 2>);
  else if (shape.lanes == 1024 && shape.groups == 1) go(norm_backward_kernel<D, 1024, 1>);
  else if (shape.lanes == 1024) go(norm_backward_kernel<D, 1024, 2>);
  else go(norm_backward_long_kernel<D>);
}

template <typename F>
void by_type(int32_t dtype, F f) {
  if (dtype == kF32) f(std::integral_constant<int, kF32>());
  else if (dtype == kBF16) f(std::integral_constant<int, kBF16>());
  else f(std::integral_constant<int, kF16>());
}

class HipLayersDevice final : public LayersDevice {
 public:
  int norm_forward(const NormForwardArgs& a, std::string* err) override {
    if (a.rows == 0) return kOk;
    const Forward f = {addr(a.x.data), addr(a.residual.data), addr(a.weight), addr(a.bias), addr(a.y), addr(a.h),
                       addr(a.stats), a.x.stride, a.residual.stride, static_cast<uint32_t>(a.rows),
                       static_cast<uint32_t>(a.cols), a.weight_dtype, static_cast<float>(a.eps), a.drop};
    hipStream_t s = static_cast<hipStream_t>(a.stream);
    by_type(a.dtype, [&](auto d) {
      if (a.residual.data != nullptr || a.drop.limit != 0) launch_forward<decltype(d)::value, true>(f, s);
      else launch_forward<decltype(d)::value, false>(f, s);
    });
    HIP_OK(hipGetLastError(), "launch norm_forward_kernel");
    return kOk;
  }

  int norm_backward(const NormBackwardArgs& a, std::string* err) override {
    const bool weights = a.dweight != nullptr || a.dbias != nullptr;
    hipStream_t s = static_cast<hipStream_t>(a.stream);
    const int32_t blocks = norm_backward_blocks(a.rows, a.cols);
    if (a.rows > 0) {
      const Backward b = {addr(a.dy.data), addr(a.h.data), addr(a.stats), addr(a.grad_h.data), addr(a.weight),
                          addr(a.dh), addr(a.dx), a.dy.stride, a.h.stride, a.grad_h.stride,
                          weights ? static_cast<float*>(a.workspace) : nullptr, static_cast<uint32_t>(a.rows),
                          static_cast<uint32_t>(a.cols), a.weight_dtype, a.drop};
      by_type(a.dtype, [&](auto d) { launch_backward<decltype(d)::value>(b, static_cast<unsigned>(blocks), s); });
      HIP_OK(hipGetLastError(), "launch norm_backward_kernel");
    }
    if (weights) {
      hipLaunchKernelGGL(norm_weights_kernel, dim3((a.cols + kWeightCols - 1) / kWeightCols, 2),
                         dim3(kWeightCols * kWeightWaves), 0, s, static_cast<const float*>(a.workspace),
                         a.rows > 0 ? blocks : 0, static_cast<uint32_t>(a.cols), addr(a.dweight), addr(a.dbias),
                         a.grad_dtype, a.accumulate ? 1 : 0);
      HIP_OK(hipGetLastError(), "launch norm_weights_kernel");
    }
    return kOk;
  }

  int dropout(const DropoutArgs& a, std::string* err) override {
    if (a.rows * a.cols == 0) return kOk;
    Drop d = {addr(a.x.data), addr(a.residual.data), addr(a.y), a.x.stride, a.residual.stride, 0, a.cols, 0, a.drop};
    const bool flat = a.rows == 1 || (a.x.stride == a.cols && (a.residual.data == nullptr || a.residual.stride == a.cols));
    if (flat) d.cols = a.rows * a.cols;
    const int64_t row_groups = (d.cols + kGroup - 1) / kGroup;
    d.groups = flat ? row_groups : row_groups * a.rows;
    d.row_groups = flat ? 1 : static_cast<uint32_t>(row_groups);
    const unsigned blocks = grid_of((d.groups + kDropTile - 1) / kDropTile, 1 << 20);
    hipStream_t s = static_cast<hipStream_t>(a.stream);
    by_type(a.dtype, [&](auto t) {
      if (flat) hipLaunchKernelGGL((dropout_kernel<decltype(t)::value, true>), dim3(blocks), dim3(kDropThreads), 0, s, d);
      else hipLaunchKernelGGL((dropout_kernel<decltype(t)::value, false>), dim3(blocks), dim3(kDropThreads), 0, s, d);
    });
    HIP_OK(hipGetLastError(), "launch dropout_kernel");
    return kOk;
  }

  int lookup(const LookupArgs& a, std::string* err) override { return enqueue_lookup(a, err); }
  int lookup_backward(const LookupBackwardArgs& a, std::string* err) override { return enqueue_lookup_backward(a, err); }
};

}  // namespace

LayersDevice* layers_device() {
  static HipLayersDevice d;
  return &d;
}

}  // namespace ddpb
