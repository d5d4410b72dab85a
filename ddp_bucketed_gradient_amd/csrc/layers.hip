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

__device__ __forceinline__ v8f fma8(v8f a, v8f b, v8f c) { return __builtin_elementwise_fma(a, b, c); }

// The statistics of a row: mean, 1 / deviation.
__device__ __forceinline__ void put_stats(uint64_t stats, uint32_t row, float mean, float rstd) {
  G<float>(stats)[static_cast<uint64_t>(row) * 2] = mean;
  G<float>(stats)[static_cast<uint64_t>(row) * 2 + 1] = rstd;
}
__device__ __forceinline__ float2 get_stats(uint64_t stats, uint32_t row) {
  const auto* p = G<const float>(stats) + static_cast<uint64_t>(row) * 2;
  return make_float2(p[0], p[1]);
}

struct Forward {
  uint64_t x, residual, weight, bias, y, h, stats;
  uint64_t x_row, residual_row;           // bytes from row to row
  uint32_t rows, cols;
  int32_t weight_dtype;
  float eps;
  DropSpec drop;
};

constexpr int norm_threads(int lanes) { return lanes > 256 ? lanes : 256; }
constexpr int norm_back_threads(int lanes) { return lanes > 512 ? lanes : lanes == 256 ? 256 : 512; }

// The row of a workgroup's rows that a lane belongs to: the same in a wave
// unless several share it, so that addresses of rows stay in scalar registers.
template <int LANES>
__device__ __forceinline__ uint32_t row_of_lane() {
  const uint32_t r = threadIdx.x / LANES;
  return LANES >= 64 ? __builtin_amdgcn_readfirstlane(r) : r;
}

// z of a group of a row: what the norm is taken of, in fp32.
template <int D, bool FUSED, int EDGE>
__device__ __forceinline__ v8f input8(const Forward& a, uint32_t row, const Group& g, uint64_t offset) {
  constexpr uint32_t size = sizeof(typename Of<D>::one);
  Raw<D> r = {};
  if (FUSED && a.residual != 0) r = load_raw<D, EDGE>(a.residual + row * a.residual_row + g.c * size, g.left);
  v8f z = widen<D>(load_raw<D, EDGE>(a.x + row * a.x_row + g.c * size, g.left));
  if constexpr (FUSED) {
    if (a.drop.limit != 0) z = drop8(z, static_cast<uint64_t>(row) * a.cols + g.c, offset, a.drop);
    if (a.residual != 0) z = z + widen<D>(r);
  }
  return z;
}

// The sum of a group's own elements.
template <int EDGE>
__device__ __forceinline__ float total(v8f x, const Group& g) {
  if (EDGE != kWhole) {   // (the last element of a shifted group is always its own)
#pragma unroll
    for (int j = 0; j < (EDGE == kShifted ? 7 : 8); ++j) x[j] = own<EDGE>(g, j) ? x[j] : 0.0f;
  }
  return ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
}

// y = (z - mean) rstd w + b. The statistics are those of z in fp32 (the mean
// first, then the squares of what is left: no cancellation); h, z as the
// backward pass reads it, is rounded to the type of x for its store only.
//
// Bound by HBM: 16384 x 1024 in bf16 with residual and dropout (two streams in,
// two out) 22.4 us, 6.0 TB/s. Rows up to 1024 elements stay in one wave, with no
// barrier; the weights stay in registers over the rows of a workgroup (2048
// workgroups at most).
template <int D, int LANES, int K, bool FUSED, int EDGE>
__global__ __launch_bounds__(norm_threads(LANES)) void norm_forward_kernel(Forward a) {
  constexpr uint32_t size = sizeof(typename Of<D>::one);
  constexpr uint32_t ROWS = norm_threads(LANES) / LANES;
  __shared__ float lds[2][LANES > 64 ? LANES / 64 * 2 : 1];
  const uint32_t lane = threadIdx.x % LANES;
  const uint64_t offset = FUSED ? offset_of(a.drop) : 0;
  const float inverse = 1.0f / static_cast<float>(a.cols);
  v8f w[K], b[K];
  Group g[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    g[k] = group_at<EDGE>(a.cols, (lane + k * LANES) * 8);
    w[k] = 1.0f;
    b[k] = 0.0f;
    if (g[k].left > 0 && a.weight != 0) w[k] = load8<EDGE>(a.weight_dtype, a.weight, g[k]);
    if (g[k].left > 0 && a.bias != 0) b[k] = load8<EDGE>(a.weight_dtype, a.bias, g[k]);
  }
  for (uint32_t row = blockIdx.x * ROWS + row_of_lane<LANES>(); row < a.rows; row += gridDim.x * ROWS) {
    v8f z[K];
    float s[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      z[k] = 0.0f;
      if (g[k].left > 0) z[k] = input8<D, FUSED, EDGE>(a, row, g[k], offset);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) s[0] += total<EDGE>(z[k], g[k]);
    row_sum<LANES>(s, lds[0]);
    const float mean = s[0] * inverse;
    float q[1] = {0.0f};
    const uint64_t at = static_cast<uint64_t>(row) * a.cols * size;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (g[k].left <= 0) continue;
      if (FUSED && a.h != 0) store8<D, EDGE>(a.h + at + g[k].c * size, g[k].left, z[k]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = z[k][j] - mean;
        q[0] = __builtin_fmaf(own<EDGE>(g[k], j) ? d : 0.0f, d, q[0]);
        z[k][j] = d;
      }
    }
    row_sum<LANES>(q, lds[1]);
    const float rstd = 1.0f / __builtin_sqrtf(q[0] * inverse + a.eps);
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (g[k].left > 0) store8<D, EDGE>(a.y + at + g[k].c * size, g[k].left, fma8(z[k] * rstd, w[k], b[k]));
    if (lane == 0) put_stats(a.stats, row, mean, rstd);
  }
}

constexpr int kLong = 1024;   // threads for a row that no shape holds in registers

template <int D, bool FUSED>
__global__ __launch_bounds__(kLong) void norm_forward_long_kernel(Forward a) {
  constexpr uint32_t size = sizeof(typename Of<D>::one);
  constexpr int EDGE = kShifted;
  __shared__ float lds[2][kLong / 64 * 2];
  const uint64_t offset = FUSED ? offset_of(a.drop) : 0;
  const float inverse = 1.0f / static_cast<float>(a.cols);
  for (uint32_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    float s[1] = {0.0f}, q[1] = {0.0f};
    const uint64_t at = static_cast<uint64_t>(row) * a.cols * size;
    for (uint32_t c = threadIdx.x * 8; c < a.cols; c += kLong * 8) {
      const Group g = group_at<EDGE>(a.cols, c);
      s[0] += total<EDGE>(input8<D, FUSED, EDGE>(a, row, g, offset), g);
    }
    row_sum<kLong>(s, lds[0]);
    const float mean = s[0] * inverse;
    for (uint32_t c = threadIdx.x * 8; c < a.cols; c += kLong * 8) {
      const Group g = group_at<EDGE>(a.cols, c);
      const v8f z = input8<D, FUSED, EDGE>(a, row, g, offset);
      if (FUSED && a.h != 0) store8<D, EDGE>(a.h + at + g.c * size, g.left, z);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = own<EDGE>(g, j) ? z[j] - mean : 0.0f;
        q[0] = __builtin_fmaf(d, d, q[0]);
      }
    }
    row_sum<kLong>(q, lds[1]);
    const float rstd = 1.0f / __builtin_sqrtf(q[0] * inverse + a.eps);
    for (uint32_t c = threadIdx.x * 8; c < a.cols; c += kLong * 8) {
      const Group g = group_at<EDGE>(a.cols, c);
      v8f w = 1.0f, b = 0.0f;
      if (a.weight != 0) w = load8<EDGE>(a.weight_dtype, a.weight, g);
      if (a.bias != 0) b = load8<EDGE>(a.weight_dtype, a.bias, g);
      const v8f z = input8<D, FUSED, EDGE>(a, row, g, offset);
      store8<D, EDGE>(a.y + at + g.c * size, g.left, fma8((z - mean) * rstd, w, b));
    }
    if (threadIdx.x == 0) put_stats(a.stats, row, mean, rstd);
  }
}

// ---------------------------------------------------------------------------
// Backward. With n = (h - mean) rstd and g = dy w:
//   dh = rstd (g - mean g - n mean(g n)) + grad_h,  dx = drop(dh),
//   dweight = sum over rows of dy n,  dbias = sum of dy.
// A workgroup goes over rows, keeps its lanes' parts of the weights' gradients
// in fp32 registers and leaves one partial sum, which norm_weights_kernel adds
// up: no atomics, so the same bits on every run.
//
// Bound by HBM: 16384 x 1024 in bf16 with dropout 24.1 us, 5.6 TB/s; 8192 x 8192 in
// fp32 with grad_h 196 us, 5.5 TB/s. One workgroup of 512 a CU: two a CU took 25.3
// and 207 us, four 27.6 and 221, and leave more partial sums.
struct Backward {
  uint64_t dy, h, stats, grad_h, weight, dh, dx;
  uint64_t dy_row, h_row, grad_h_row;           // bytes from row to row
  float* partials;                              // [workgroup][dweight, dbias][cols], or NULL
  uint64_t dweight, dbias;                      // one workgroup: written by it (else 0)
  uint32_t rows, cols;
  int32_t weight_dtype, grad_dtype, accumulate;
  DropSpec drop;
};

// Writes, or adds to, one element of a gradient.
__device__ __forceinline__ void put_grad(uint64_t to, int dtype, bool add, uint32_t c, float x) {
  auto put = [&](auto one) {
    auto* p = G<decltype(one)>(to + c * static_cast<uint32_t>(sizeof(one)));
    if (add) x += static_cast<float>(*p);
    *p = static_cast<decltype(one)>(x);
  };
  if (dtype == kF32) put(float());
  else if (dtype == kBF16) put(__bf16());
  else put(_Float16());
}

template <int D, int EDGE>
__device__ __forceinline__ void store_grads(const Backward& a, uint32_t row, const Group& g, v8f d, uint64_t offset) {
  constexpr uint32_t size = sizeof(typename Of<D>::one);
  const uint64_t at = static_cast<uint64_t>(row) * a.cols * size + g.c * size;
  if (a.grad_h != 0) d = d + widen<D>(load_raw<D, EDGE>(a.grad_h + row * a.grad_h_row + g.c * size, g.left));
  store8<D, EDGE>(a.dh + at, g.left, d);
  if (a.drop.limit != 0) {
    d = drop8(d, static_cast<uint64_t>(row) * a.cols + g.c, offset, a.drop);
    store8<D, EDGE>(a.dx + at, g.left, d);
  }
}

// The next row is loaded while this one is worked on (8192 x 8192 in fp32: 195 us,
// 199 without), except by 1024 lanes, whose 128 registers do not hold it, nor the
// weights.
template <int D, int LANES, int K, int EDGE>
__global__ __launch_bounds__(norm_back_threads(LANES)) void norm_backward_kernel(Backward a) {
  constexpr uint32_t size = sizeof(typename Of<D>::one);
  constexpr uint32_t THREADS = norm_back_threads(LANES), ROWS = THREADS / LANES;
  constexpr bool AHEAD = LANES < 1024;
  __shared__ float lds[2][LANES > 64 ? LANES / 64 * 2 : 1];
  const uint32_t lane = threadIdx.x % LANES, mine = row_of_lane<LANES>(), step = gridDim.x * ROWS;
  const uint64_t offset = offset_of(a.drop);
  const float inverse = 1.0f / static_cast<float>(a.cols);
  v8f w[K], dw[K], db[K];
  Group g[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    g[k] = group_at<EDGE>(a.cols, (lane + k * LANES) * 8);
    w[k] = 1.0f;
    dw[k] = db[k] = 0.0f;
    if (AHEAD && g[k].left > 0 && a.weight != 0) w[k] = load8<EDGE>(a.weight_dtype, a.weight, g[k]);
  }
  auto weigh = [&](int k, v8f x) __attribute__((always_inline)) {
    if constexpr (AHEAD) return x * w[k];
    if (g[k].left <= 0 || a.weight == 0) return x;
    return x * load8<EDGE>(a.weight_dtype, a.weight, g[k]);
  };
  Raw<D> dy_next[K], h_next[K];
  float2 stats_next = {};
  auto fetch = [&](uint32_t r) __attribute__((always_inline)) {
    stats_next = get_stats(a.stats, r);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      dy_next[k] = h_next[k] = Raw<D>{};
      if (g[k].left <= 0) continue;
      dy_next[k] = load_raw<D, EDGE>(a.dy + r * a.dy_row + g[k].c * size, g[k].left);
      h_next[k] = load_raw<D, EDGE>(a.h + r * a.h_row + g[k].c * size, g[k].left);
    }
  };
  uint32_t row = blockIdx.x * ROWS + mine;
  if (row < a.rows) fetch(row);
  for (int turn = 0; row < a.rows; row += step, turn ^= 1) {
    const float mean = stats_next.x, rstd = stats_next.y;
    Raw<D> dy[K], h[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      dy[k] = dy_next[k];
      h[k] = h_next[k];
    }
    if (AHEAD && row + step < a.rows) fetch(row + step);
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (!AHEAD) __builtin_amdgcn_sched_barrier(0);
      const v8f n = (widen<D>(h[k]) - mean) * rstd, d = widen<D>(dy[k]), x = weigh(k, d);
      dw[k] = fma8(d, n, dw[k]);
      db[k] = db[k] + d;
      s[0] += total<EDGE>(x, g[k]);
      // a lane without columns holds n = -mean rstd, which may be infinite, and x = 0
      s[1] += g[k].left > 0 ? total<EDGE>(x * n, g[k]) : 0.0f;
    }
    row_sum<LANES>(s, lds[turn]);
    s[0] *= inverse;
    s[1] *= inverse;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (!AHEAD) __builtin_amdgcn_sched_barrier(0);
      const v8f n = (widen<D>(h[k]) - mean) * rstd, x = weigh(k, widen<D>(dy[k]));
      if (g[k].left > 0) store_grads<D, EDGE>(a, row, g[k], (fma8(n, v8f(-s[1]), x) - s[0]) * rstd, offset);
    }
    if (!AHEAD && row + step < a.rows) fetch(row + step);
  }
  const bool alone = (a.dweight | a.dbias) != 0;
  if (a.partials == nullptr && !alone) return;
  float* to = a.partials + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
  auto put = [&](int which, uint32_t c, float x) __attribute__((always_inline)) {
    const uint64_t grad = which ? a.dbias : a.dweight;
    if (!alone) to[which * a.cols + c] = x;
    else if (grad != 0) put_grad(grad, a.grad_dtype, a.accumulate != 0, c, x);
  };
  if constexpr (ROWS == 1) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (g[k].left > 0 && own<EDGE>(g[k], j)) {
          put(0, g[k].c + j, dw[k][j]);
          put(1, g[k].c + j, db[k][j]);
        }
      }
    }
  } else {
    // the rows of the workgroup side by side in LDS, a column to a thread
    constexpr uint32_t WIDTH = LANES * K * 8;
    __shared__ float part[ROWS * WIDTH];
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < g[k].left) part[mine * WIDTH + g[k].c + j] = which ? db[k][j] : dw[k][j];
      }
      __syncthreads();
      for (uint32_t c = threadIdx.x; c < a.cols; c += THREADS) {
        float x = part[c];
#pragma unroll
        for (uint32_t r = 1; r < ROWS; ++r) x += part[r * WIDTH + c];
        put(which, c, x);
      }
    }
  }
}

template <int D>
__global__ __launch_bounds__(kLong) void norm_backward_long_kernel(Backward a) {
  constexpr uint32_t size = sizeof(typename Of<D>::one);
  constexpr int EDGE = kShifted;
  __shared__ float lds[2][kLong / 64 * 2];
  const uint64_t offset = offset_of(a.drop);
  const float inverse = 1.0f / static_cast<float>(a.cols);
  float* to = a.partials == nullptr ? nullptr : a.partials + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
  bool first = true;
  int turn = 0;
  for (uint32_t row = blockIdx.x; row < a.rows; row += gridDim.x, first = false, turn ^= 1) {
    const float2 stats = get_stats(a.stats, row);
    float s[2] = {0.0f, 0.0f};
    for (int pass = 0; pass < 2; ++pass) {
      for (uint32_t c = threadIdx.x * 8; c < a.cols; c += kLong * 8) {
        const Group g = group_at<EDGE>(a.cols, c);
        const v8f dy = widen<D>(load_raw<D, EDGE>(a.dy + row * a.dy_row + g.c * size, g.left));
        const v8f n = (widen<D>(load_raw<D, EDGE>(a.h + row * a.h_row + g.c * size, g.left)) - stats.x) * stats.y;
        v8f x = dy;
        if (a.weight != 0) x = x * load8<EDGE>(a.weight_dtype, a.weight, g);
        if (pass == 1) {
          store_grads<D, EDGE>(a, row, g, (fma8(n, v8f(-s[1]), x) - s[0]) * stats.y, offset);
          continue;
        }
        s[0] += total<EDGE>(x, g);
        s[1] += total<EDGE>(x * n, g);
        if (to != nullptr) {   // the workgroup's own sums, each element always by the same lane
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (!own<EDGE>(g, j)) continue;
            to[g.c + j] = __builtin_fmaf(dy[j], n[j], first ? 0.0f : to[g.c + j]);
            to[a.cols + g.c + j] = dy[j] + (first ? 0.0f : to[a.cols + g.c + j]);
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
// every 16th of them. 3.9 us for 256 sums of 1024 columns, most of it the launch.
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
  put_grad(out, dtype, accumulate != 0, c, x);
}

// ---------------------------------------------------------------------------
// Dropout, with or without a residual: a group of eight elements to a lane,
// counted row by row. Bound by HBM: 8192 x 8192 in bf16 45.4 us, 5.9 TB/s (with
// two or four groups to a lane, measured in turn, 46.2 and 48.4; 2048 x 1024: 2.96,
// 2.84 and 3.50).
struct Drop {
  uint64_t x, residual, y;
  int64_t x_stride, residual_stride;   // in elements
  int64_t groups;                      // rows * groups of a row
  int64_t cols;
  uint32_t row_groups;                 // groups of a row, if there is more than one row
  DropSpec drop;
};
constexpr int kDropThreads = 256;

template <int D, bool FLAT, int EDGE>
__global__ __launch_bounds__(kDropThreads) void dropout_kernel(Drop a) {
  typedef typename Of<D>::one one;
  const uint64_t offset = offset_of(a.drop);
  for (int64_t tile = static_cast<int64_t>(blockIdx.x) * kDropThreads; tile < a.groups;
       tile += static_cast<int64_t>(gridDim.x) * kDropThreads) {
    if (tile + threadIdx.x >= a.groups) return;
    int64_t row = 0, c = (tile + threadIdx.x) * 8;
    if (!FLAT) {
      const int64_t row0 = tile / a.row_groups;
      const uint32_t i = static_cast<uint32_t>(tile - row0 * a.row_groups) + threadIdx.x, q = i / a.row_groups;
      row = row0 + q;
      c = static_cast<int64_t>(i - q * a.row_groups) * 8;
    }
    const int left = static_cast<int>(min(a.cols - c, int64_t(8)));
    if (EDGE == kShifted && left < 8) c = a.cols - 8;
    v8f z = widen<D>(load_raw<D, EDGE>(a.x + (row * a.x_stride + c) * sizeof(one), left));
    Raw<D> r = {};
    if (a.residual != 0) r = load_raw<D, EDGE>(a.residual + (row * a.residual_stride + c) * sizeof(one), left);
    const int64_t first = row * a.cols + c;
    if (a.drop.limit != 0) z = drop8(z, static_cast<uint64_t>(first), offset, a.drop);
    if (a.residual != 0) z = z + widen<D>(r);
    store8<D, EDGE>(a.y + first * sizeof(one), left, z);
  }
}

uint64_t bytes(int64_t stride, int32_t dtype) { return static_cast<uint64_t>(stride * dtype_size(dtype)); }

unsigned grid_of(int64_t want, int64_t most) {
  return static_cast<unsigned>(want < 1 ? 1 : want < most ? want : most);
}

// f(lanes, groups) with the row's shape as constants; false if there is none.
template <typename F>
bool by_shape(int64_t cols, F f) {
  const NormShape s = norm_shape(cols);
  auto is = [&](auto lanes, auto groups) {
    if (s.lanes != lanes.value || s.groups != groups.value) return false;
    f(lanes, groups);
    return true;
  };
  constexpr std::integral_constant<int, 1> one;
  constexpr std::integral_constant<int, 2> two;
  return is(std::integral_constant<int, 16>(), one) || is(std::integral_constant<int, 64>(), one) ||
         is(std::integral_constant<int, 64>(), two) || is(std::integral_constant<int, 256>(), one) ||
         is(std::integral_constant<int, 256>(), two) || is(std::integral_constant<int, 512>(), two) ||
         is(std::integral_constant<int, 1024>(), two);
}

template <int D, bool FUSED>
void launch_forward(const Forward& a, hipStream_t s) {
  auto go = [&](auto kernel, int threads, int rows) {
    hipLaunchKernelGGL(kernel, dim3(grid_of((int64_t(a.rows) + rows - 1) / rows, 2048)), dim3(threads), 0, s, a);
  };
  const bool short_row = by_shape(a.cols, [&](auto lanes, auto groups) {
    constexpr int L = decltype(lanes)::value, K = decltype(groups)::value, T = norm_threads(L);
    if (a.cols % 8 == 0) return go(norm_forward_kernel<D, L, K, FUSED, kWhole>, T, T / L);
    if constexpr (L == 16)
      if (a.cols < 8) return go(norm_forward_kernel<D, L, K, FUSED, kSmall>, T, T / L);
    go(norm_forward_kernel<D, L, K, FUSED, kShifted>, T, T / L);
  });
  if (!short_row) go(norm_forward_long_kernel<D, FUSED>, kLong, 1);
}

template <int D>
void launch_backward(const Backward& a, unsigned blocks, hipStream_t s) {
  auto go = [&](auto kernel, int threads) { hipLaunchKernelGGL(kernel, dim3(blocks), dim3(threads), 0, s, a); };
  const bool short_row = by_shape(a.cols, [&](auto lanes, auto groups) {
    constexpr int L = decltype(lanes)::value, K = decltype(groups)::value, T = norm_back_threads(L);
    if (a.cols % 8 == 0) return go(norm_backward_kernel<D, L, K, kWhole>, T);
    if constexpr (L == 16)
      if (a.cols < 8) return go(norm_backward_kernel<D, L, K, kSmall>, T);
    go(norm_backward_kernel<D, L, K, kShifted>, T);
  });
  if (!short_row) go(norm_backward_long_kernel<D>, kLong);
}

class HipLayersDevice final : public LayersDevice {
 public:
  int norm_forward(const NormForwardArgs& a, std::string* err) override {
    if (a.rows == 0) return kOk;
    const Forward f = {addr(a.x.data), addr(a.residual.data), addr(a.weight), addr(a.bias), addr(a.y), addr(a.h),
                       addr(a.stats), bytes(a.x.stride, a.dtype), bytes(a.residual.stride, a.dtype), static_cast<uint32_t>(a.rows),
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
    const bool alone = norm_backward_alone(a.rows, a.cols);
    if (a.rows > 0) {
      const Backward b = {addr(a.dy.data), addr(a.h.data), addr(a.stats), addr(a.grad_h.data), addr(a.weight),
                          addr(a.dh), addr(a.dx), bytes(a.dy.stride, a.dtype), bytes(a.h.stride, a.dtype),
                          bytes(a.grad_h.stride, a.dtype),
                          weights && !alone ? static_cast<float*>(a.workspace) : nullptr,
                          alone ? addr(a.dweight) : 0, alone ? addr(a.dbias) : 0, static_cast<uint32_t>(a.rows),
                          static_cast<uint32_t>(a.cols), a.weight_dtype, a.grad_dtype, a.accumulate ? 1 : 0, a.drop};
      by_type(a.dtype, [&](auto d) { launch_backward<decltype(d)::value>(b, static_cast<unsigned>(blocks), s); });
      HIP_OK(hipGetLastError(), "launch norm_backward_kernel");
    }
    if (weights && !alone) {
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
    hipStream_t s = static_cast<hipStream_t>(a.stream);
    const unsigned blocks = grid_of((d.groups + kDropThreads - 1) / kDropThreads, 1 << 22);
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(blocks), dim3(kDropThreads), 0, s, d); };
    // Groups that are written twice must not be read after the first time: in
    // place (and in a flat array, of which it is one group) the last one is cut.
    const bool whole = d.cols % 8 == 0, cut = d.cols < 8 || a.y == a.x.data || a.y == a.residual.data;
    by_type(a.dtype, [&](auto t) {
      constexpr int D = decltype(t)::value;
      if (flat) whole ? go(dropout_kernel<D, true, kWhole>) : go(dropout_kernel<D, true, kSmall>);
      else if (whole) go(dropout_kernel<D, false, kWhole>);
      else cut ? go(dropout_kernel<D, false, kSmall>) : go(dropout_kernel<D, false, kShifted>);
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
