// embedding.hip -- CDNA4 (gfx950) kernels of the embedding: the lookup, and its
// gradient by sorted tokens.
#include "group8.hpp"

namespace ddpb {
namespace {

// A token of 4 or 8 bytes; what lies outside of the table becomes `vocab`.
__device__ __forceinline__ uint32_t token_at(uint64_t tokens, int32_t bytes, int64_t i, uint32_t vocab) {
  if (bytes == 4) {
    const uint32_t t = G<const uint32_t>(tokens)[i];
    return t < vocab ? t : vocab;
  }
  const uint64_t t = G<const uint64_t>(tokens)[i];
  return t < vocab ? static_cast<uint32_t>(t) : vocab;
}

// ---------------------------------------------------------------------------
// y_i = scale table[t_i] + residual_i, in fp32, rounded once. The groups of
// eight elements of all rows are counted through; a workgroup takes kTile of
// them at a time.
struct Lookup {
  uint64_t tokens, table, residual, y;
  int64_t groups, residual_stride;
  uint32_t row_groups, cols, vocab;
  int32_t token_bytes;
  float scale;
};
constexpr int kThreads = 256, kUnroll = 2, kTile = kThreads * kUnroll;

template <int TD, int D>
__global__ __launch_bounds__(kThreads) void lookup_kernel(Lookup a) {
  typedef typename Of<D>::one one;
  typedef typename Of<TD>::one table_one;
  for (int64_t tile = static_cast<int64_t>(blockIdx.x) * kTile; tile < a.groups;
       tile += static_cast<int64_t>(gridDim.x) * kTile) {
    const int64_t row0 = tile / a.row_groups;
    const uint32_t rest = static_cast<uint32_t>(tile - row0 * a.row_groups);
    uint32_t c[kUnroll], t[kUnroll];
    int64_t row[kUnroll];
    v8f x[kUnroll], r[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t i = u * kThreads + threadIdx.x, q = (rest + i) / a.row_groups;
      row[u] = row0 + q;
      c[u] = (rest + i - q * a.row_groups) * 8;
      t[u] = a.vocab;
      x[u] = r[u] = 0.0f;
      if (tile + i < a.groups) {
        t[u] = token_at(a.tokens, a.token_bytes, row[u], a.vocab);
        if (a.residual != 0) r[u] = load8<D>(a.residual + (row[u] * a.residual_stride + c[u]) * sizeof(one), static_cast<int64_t>(a.cols) - c[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (t[u] < a.vocab)
        x[u] = load8<TD>(a.table + (static_cast<uint64_t>(t[u]) * a.cols + c[u]) * sizeof(table_one), static_cast<int64_t>(a.cols) - c[u]) * a.scale;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (tile + u * kThreads + threadIdx.x < a.groups)
        store8<D>(a.y + (static_cast<uint64_t>(row[u]) * a.cols + c[u]) * sizeof(one), static_cast<int64_t>(a.cols) - c[u], x[u] + r[u]);
  }
}

// ---------------------------------------------------------------------------
// The gradient: dtable[v] = scale * sum of dy_i over the places i of token v, in
// order of i and without atomics on values, so the same bits on every run.
//
//  1. Sort the places by token: a stable radix sort, `digit` bits a pass. With
//     one tile of keys one workgroup does it in LDS; with more each pass is a
//     histogram of every tile and a scatter. Beside it, workgroups that would
//     be idle write the zeros of a gradient that is not added to.
//  2. Sum: the sorted places are cut into units of equal length, so that a
//     token that holds many places (padding, the commonest words) is shared
//     by many waves. A run of one token that covers no whole unit belongs to
//     the unit where it begins. One that does leaves a partial sum in each of
//     its units, and
//  3. a last kernel adds those up.
struct Zeros {
  uint64_t at;        // 16-byte aligned
  int64_t first, last;   // of the 16-byte pieces there, this launch's share
  uint64_t head, tail;   // odd bytes before and behind the pieces: addresses
  int32_t head_bytes, tail_bytes;   // 0 but in the first launch
};
constexpr int64_t kZeroPieces = kSortThreads * 8;   // of a workgroup

__device__ __forceinline__ void write_zeros(const Zeros& z, int64_t block) {
  const int64_t from = z.first + block * kZeroPieces;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int64_t i = from + u * kSortThreads + threadIdx.x;
    if (i < z.last) G<v4u>(z.at)[i] = v4u{0, 0, 0, 0};
  }
  if (block == 0) {   // element by element (of at least two bytes)
    if (static_cast<int>(threadIdx.x) * 2 < z.head_bytes) G<uint16_t>(z.head)[threadIdx.x] = 0;
    if (static_cast<int>(threadIdx.x) * 2 < z.tail_bytes) G<uint16_t>(z.tail)[threadIdx.x] = 0;
  }
}

struct Sort {
  uint64_t tokens;              // of the first pass; else NULL
  const uint32_t *keys_in, *order_in;
  uint32_t *keys, *order;       // sorted by this pass
  uint32_t* hist;               // [tile][digit]: counts, or what stands before the tile after the scan
  uint32_t* totals;             // [digit] (after the scan)
  uint32_t* joins;              // the count of the long runs, which the first launch clears
  int64_t n;
  uint32_t vocab, tiles;
  int32_t token_bytes, shift, digit, scanned;
  int32_t passes;               // of a sort by one workgroup
  Zeros zeros;
};

__device__ __forceinline__ void load_keys(const Sort& a, int64_t tile, uint32_t (&key)[kSortKeys], uint32_t (&place)[kSortKeys]) {
  // a wave's keys are consecutive: 64 at a time
  const int64_t at = tile * kSortTile + (threadIdx.x >> 6) * (64 * kSortKeys) + (threadIdx.x & 63);
#pragma unroll
  for (int e = 0; e < kSortKeys; ++e) {
    const int64_t i = at + e * 64;
    key[e] = place[e] = 0;
    if (i >= a.n) continue;
    if (a.tokens != 0) {
      key[e] = token_at(a.tokens, a.token_bytes, i, a.vocab);
      place[e] = static_cast<uint32_t>(i);
    } else {
      key[e] = a.keys_in[i];
      place[e] = a.order_in[i];
    }
  }
}

constexpr int kWaves = kSortThreads / 64, kBins = 1 << kMaxDigit;

// What lanes of a wave wrote to LDS is seen by its other lanes behind this.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Each key's place among the equal digits of its wave, and the waves' counts.
// Stable: the keys of a wave are taken 64 at a time in their order, and a key's
// rank is the count of equal digits in the lanes below it.
__device__ __forceinline__ void rank_keys(const uint32_t (&key)[kSortKeys], uint32_t (&rank)[kSortKeys], int64_t at,
                                          int64_t n, int shift, int digit, uint16_t (*count)[kBins]) {
  const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63, mask = (1u << digit) - 1;
  for (uint32_t d = lane; d <= mask; d += 64) count[wave][d] = 0;
  const uint64_t below = (uint64_t(1) << lane) - 1;
  wave_fence();
#pragma unroll
  for (int e = 0; e < kSortKeys; ++e) {
    const bool there = at + e * 64 < n;
    const uint32_t d = key[e] >> shift & mask;
    uint64_t same = __ballot(there);
    for (int b = 0; b < digit; ++b) {
      const bool one = d >> b & 1;
      const uint64_t ones = __ballot(one);
      same &= one ? ones : ~ones;
    }
    uint32_t before = 0;
    if (there) before = count[wave][d];
    rank[e] = before + __popcll(same & below);
    wave_fence();
    if (there && (same & below) == 0) count[wave][d] = static_cast<uint16_t>(before + __popcll(same));
    wave_fence();
  }
}

// Exclusive sum over the threads of a workgroup.
__device__ __forceinline__ uint32_t scan(uint32_t x, uint32_t* waves) {
  const uint32_t lane = threadIdx.x & 63;
  uint32_t sum = x;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t y = __shfl_up(sum, d, 64);
    if (lane >= static_cast<uint32_t>(d)) sum += y;
  }
  if (lane == 63) waves[threadIdx.x >> 6] = sum;
  __syncthreads();
  uint32_t before = 0;
  for (uint32_t w = 0; w < threadIdx.x >> 6; ++w) before += waves[w];
  __syncthreads();
  return before + sum - x;
}

// All passes for one tile of keys, in LDS.
__global__ __launch_bounds__(kSortThreads) void sort_tile_kernel(Sort a) {
  if (blockIdx.x != 0) {
    write_zeros(a.zeros, static_cast<int64_t>(blockIdx.x) - 1);
    return;
  }
  __shared__ uint16_t count[kWaves][kBins];
  __shared__ uint32_t keys[kSortTile], base[kBins], waves[kWaves];
  __shared__ uint16_t places[kSortTile];
  if (threadIdx.x == 0) *a.joins = 0;
  uint32_t key[kSortKeys], place[kSortKeys], rank[kSortKeys];
  load_keys(a, 0, key, place);
  const uint32_t at = (threadIdx.x >> 6) * (64 * kSortKeys) + (threadIdx.x & 63);
  for (int pass = 0, shift = 0; pass < a.passes; ++pass, shift += a.digit) {
    rank_keys(key, rank, at, a.n, shift, a.digit, count);
    __syncthreads();
    uint32_t all = 0;
    const uint32_t bins = 1u << a.digit;
    if (threadIdx.x < bins) {
      for (int w = 0; w < kWaves; ++w) {
        const uint32_t x = count[w][threadIdx.x];
        count[w][threadIdx.x] = static_cast<uint16_t>(all);
        all += x;
      }
    }
    const uint32_t before = scan(all, waves);
    if (threadIdx.x < bins) base[threadIdx.x] = before;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kSortKeys; ++e) {
      if (at + e * 64 >= a.n) continue;
      const uint32_t d = key[e] >> shift & (bins - 1), to = base[d] + count[threadIdx.x >> 6][d] + rank[e];
      if (pass == a.passes - 1) {
        a.keys[to] = key[e];
        a.order[to] = place[e];
      } else {
        keys[to] = key[e];
        places[to] = static_cast<uint16_t>(place[e]);
      }
    }
    __syncthreads();
    if (pass < a.passes - 1) {
#pragma unroll
      for (int e = 0; e < kSortKeys; ++e) {
        if (at + e * 64 >= a.n) continue;
        key[e] = keys[at + e * 64];
        place[e] = places[at + e * 64];
      }
    }
  }
}

__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(Sort a) {
  if (blockIdx.x >= a.tiles) {
    write_zeros(a.zeros, static_cast<int64_t>(blockIdx.x) - a.tiles);
    return;
  }
  __shared__ uint32_t count[kBins];
  const uint32_t bins = 1u << a.digit;
  if (threadIdx.x < bins) count[threadIdx.x] = 0;
  if (a.tokens != 0 && blockIdx.x == 0 && threadIdx.x == 0) *a.joins = 0;
  uint32_t key[kSortKeys], place[kSortKeys];
  load_keys(a, blockIdx.x, key, place);
  __syncthreads();
  const int64_t at = blockIdx.x * kSortTile + (threadIdx.x >> 6) * (64 * kSortKeys) + (threadIdx.x & 63);
#pragma unroll
  for (int e = 0; e < kSortKeys; ++e)
    if (at + e * 64 < a.n) atomicAdd(&count[key[e] >> a.shift & (bins - 1)], 1u);
  __syncthreads();
  if (threadIdx.x < bins) a.hist[static_cast<int64_t>(blockIdx.x) * bins + threadIdx.x] = count[threadIdx.x];
}

// Many tiles: what stands before each tile in its digit, 64 digits to a
// workgroup, a sixteenth of the tiles to a wave.
__global__ __launch_bounds__(kSortThreads) void sort_scan_kernel(Sort a) {
  __shared__ uint32_t part[kWaves][64];
  const uint32_t bins = 1u << a.digit, d = blockIdx.x * 64 + (threadIdx.x & 63), wave = threadIdx.x >> 6;
  const uint32_t each = (a.tiles + kWaves - 1) / kWaves, from = min(wave * each, a.tiles), to = min(from + each, a.tiles);
  uint32_t sum = 0;
  if (d < bins)
    for (uint32_t t = from; t < to; ++t) sum += a.hist[static_cast<int64_t>(t) * bins + d];
  part[wave][threadIdx.x & 63] = sum;
  __syncthreads();
  if (d >= bins) return;
  uint32_t before = 0, all = 0;
  for (uint32_t w = 0; w < static_cast<uint32_t>(kWaves); ++w) {
    if (w < wave) before += part[w][threadIdx.x & 63];
    all += part[w][threadIdx.x & 63];
  }
  if (wave == 0) a.totals[d] = all;
  for (uint32_t t = from; t < to; ++t) {
    const int64_t i = static_cast<int64_t>(t) * bins + d;
    const uint32_t x = a.hist[i];
    a.hist[i] = before;
    before += x;
  }
}

__global__ __launch_bounds__(kSortThreads) void sort_scatter_kernel(Sort a) {
  if (blockIdx.x >= a.tiles) {
    write_zeros(a.zeros, static_cast<int64_t>(blockIdx.x) - a.tiles);
    return;
  }
  __shared__ uint16_t count[kWaves][kBins];
  __shared__ uint32_t base[kBins], waves[kWaves];
  const uint32_t bins = 1u << a.digit;
  uint32_t key[kSortKeys], place[kSortKeys], rank[kSortKeys];
  load_keys(a, blockIdx.x, key, place);
  uint32_t all = 0, before = 0;   // keys of this thread's digit: in all tiles, in those before this one
  if (threadIdx.x < bins) {
    if (a.scanned) {
      all = a.totals[threadIdx.x];
      before = a.hist[static_cast<int64_t>(blockIdx.x) * bins + threadIdx.x];
    } else {
#pragma unroll 8
      for (uint32_t t = 0; t < a.tiles; ++t) {
        const uint32_t x = a.hist[static_cast<int64_t>(t) * bins + threadIdx.x];
        all += x;
        before += t < blockIdx.x ? x : 0;
      }
    }
  }
  const int64_t at = blockIdx.x * kSortTile + (threadIdx.x >> 6) * (64 * kSortKeys) + (threadIdx.x & 63);
  rank_keys(key, rank, at, a.n, a.shift, a.digit, count);
  before += scan(all, waves);     // its barriers also stand behind the counts
  if (threadIdx.x < bins) {
    base[threadIdx.x] = before;
    uint32_t sum = 0;
    for (int w = 0; w < kWaves; ++w) {
      const uint32_t x = count[w][threadIdx.x];
      count[w][threadIdx.x] = static_cast<uint16_t>(sum);
      sum += x;
    }
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < kSortKeys; ++e) {
    if (at + e * 64 >= a.n) continue;
    const uint32_t d = key[e] >> a.shift & (bins - 1), to = base[d] + count[threadIdx.x >> 6][d] + rank[e];
    a.keys[to] = key[e];
    a.order[to] = place[e];
  }
}

struct Sum {
  uint64_t dy, dtable;
  int64_t dy_stride, n, unit, units;
  const uint32_t *keys, *order;
  float* partials;              // [unit][run from the left, run to the right][cols]
  uint32_t *joins, *list;
  uint32_t cols, vocab;
  int32_t grad_dtype, accumulate;
  float scale;
};

__device__ __forceinline__ void write_row(const Sum& a, uint32_t token, uint32_t c, int64_t left, v8f x) {
  const uint64_t at = a.dtable + (static_cast<uint64_t>(token) * a.cols + c) * (a.grad_dtype == kF32 ? 4 : 2);
  x = x * a.scale;
  if (a.accumulate) x = x + load8(a.grad_dtype, at, left);
  store8(a.grad_dtype, at, left, x);
}

// A unit has LANES lanes, eight columns each.
constexpr int kAhead = 8;       // places whose rows are loaded together
template <int D>
__global__ __launch_bounds__(256) void sum_kernel(Sum a, int lanes) {
  typedef typename Of<D>::one one;
  const int64_t u = static_cast<int64_t>(blockIdx.x) * (256 / lanes) + threadIdx.x / lanes;
  if (u >= a.units) return;
  const uint32_t c = (blockIdx.y * lanes + threadIdx.x % lanes) * 8;
  const int64_t left = static_cast<int64_t>(a.cols) - c;
  if (left <= 0) return;
  const int64_t s = u * a.unit, e = min(s + a.unit, a.n);
  const uint32_t first = a.keys[s], last = a.keys[e - 1];
  if (first >= a.vocab) return;
  // the run that comes in from the left: another unit's, unless it covers a whole unit
  const bool from_left = s > 0 && a.keys[s - 1] == first;
  const bool mine = !from_left || last == first || a.keys[s - a.unit] == first;
  // the run that goes out to the right: ours to its end, unless it covers a whole unit
  const bool to_right = e < a.n && last < a.vocab && a.keys[e] == last;
  const int64_t e2 = min(e + a.unit, a.n);
  const bool long_right = to_right && (first == last || a.keys[e2 - 1] == last);
  const int64_t stop = to_right && !long_right ? e2 : e;
  float* const partial = a.partials + u * 2 * a.cols + c;
  auto put = [&](float* p, v8f x) { store8<kF32>(reinterpret_cast<uint64_t>(p), left, x); };

  uint32_t run = first;
  bool open_left = from_left;     // the run in `x` began in another unit
  v8f x = 0.0f;
  for (int64_t j = s; j < stop; j += kAhead) {
    uint32_t key[kAhead];
    v8f d[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      key[i] = j + i < stop ? a.keys[j + i] : a.vocab;
      if (j + i >= e && key[i] != last) key[i] = a.vocab;        // behind the run that we finish
      d[i] = 0.0f;
      if (key[i] < a.vocab && (mine || key[i] != first))
        d[i] = load8<D>(a.dy + (a.order[j + i] * a.dy_stride + c) * sizeof(one), left);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (key[i] != run) {
        if (run < a.vocab) {
          if (!open_left) write_row(a, run, c, left, x);
          else if (mine) put(partial, x);
        }
        run = key[i];
        open_left = false;
        x = 0.0f;
      }
      x = x + d[i];
    }
  }
  if (run >= a.vocab) return;
  if (open_left) {
    if (mine) put(partial, x);
  } else if (!long_right) {
    write_row(a, run, c, left, x);
  } else {
    put(partial + a.cols, x);
    if (c == 0) a.list[atomicAdd(a.joins, 1u)] = static_cast<uint32_t>(u);
  }
}

// The runs that cover whole units: 64 columns to a workgroup, in which 16 lanes
// side by side hold four columns each and 16 rows of lanes take every 16th unit.
constexpr int kJoinCols = 64;
__global__ __launch_bounds__(256) void join_kernel(Sum a) {
  __shared__ v4f part[16][16];
  __shared__ uint32_t found;
  const uint32_t slices = (a.cols + kJoinCols - 1) / kJoinCols;
  const uint64_t work = static_cast<uint64_t>(*a.joins) * slices;
  const uint32_t lane = threadIdx.x & 15, line = threadIdx.x >> 4;
  for (uint64_t k = blockIdx.x; k < work; k += gridDim.x) {
    const int64_t u = a.list[k / slices];
    const uint32_t c = static_cast<uint32_t>(k % slices) * kJoinCols + lane * 4;
    const uint32_t token = a.keys[(u + 1) * a.unit - 1];
    // units behind u that begin with the token
    int64_t count = 0;
    for (bool more = true; more; count += found, more = found == 256) {
      const int64_t next = u + 1 + count + threadIdx.x;
      __syncthreads();
      if (threadIdx.x == 0) found = 0;
      __syncthreads();
      const bool same = next < a.units && a.keys[next * a.unit] == token;
      const uint64_t votes = __ballot(same);
      if ((threadIdx.x & 63) == 0) atomicAdd(&found, static_cast<uint32_t>(__popcll(votes)));
      __syncthreads();
    }
    const uint32_t left = c < a.cols ? min(a.cols - c, 4u) : 0;
    v4f x = 0.0f;
    // part 0 is the beginning in unit u, part i the run in unit u + i
#pragma unroll 4
    for (int64_t i = line; i <= count; i += 16) {
      const float* p = a.partials + ((u + i) * 2 + (i == 0)) * a.cols + c;
      v4f y = 0.0f;
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j)
        if (j < left) y[j] = p[j];
      x = x + y;
    }
    part[line][lane] = x;
    __syncthreads();
    if (line == 0) {
      for (int l = 1; l < 16; ++l) x = x + part[l][lane];
      const int size = a.grad_dtype == kF32 ? 4 : 2;
      const uint64_t at = a.dtable + (static_cast<uint64_t>(token) * a.cols + c) * size;
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j) {
        if (j >= left) continue;
        auto put = [&](auto one) {
          auto* p = G<decltype(one)>(at) + j;
          const float old = a.accumulate ? static_cast<float>(*p) : 0.0f;
          *p = static_cast<decltype(one)>(x[j] * a.scale + old);
        };
        if (a.grad_dtype == kF32) put(float());
        else if (a.grad_dtype == kBF16) put(__bf16());
        else put(_Float16());
      }
    }
    __syncthreads();
  }
}

uint64_t addr(const void* p) { return static_cast<uint64_t>(reinterpret_cast<uintptr_t>(p)); }

template <typename F>
void by_type(int32_t dtype, F f) {
  if (dtype == kF32) f(std::integral_constant<int, kF32>());
  else if (dtype == kBF16) f(std::integral_constant<int, kBF16>());
  else f(std::integral_constant<int, kF16>());
}

// The share of the zeros that launch i of `launches` writes.
Zeros zeros_of(const LookupBackwardArgs& a, int i, int launches) {
  Zeros z = {};
  if (a.accumulate) return z;
  const uint64_t from = addr(a.dtable);
  const uint64_t to = from + static_cast<uint64_t>(a.vocab * a.cols * dtype_size(a.grad_dtype));
  const uint64_t lo = (from + 15) / 16 * 16, hi = to / 16 * 16;
  if (lo >= hi) {              // within two pieces: all of it is odd bytes
    z.head = from;
    z.head_bytes = i == 0 ? static_cast<int32_t>(to - from) : 0;
    return z;
  }
  const int64_t pieces = static_cast<int64_t>((hi - lo) / 16);
  z.at = lo;
  z.first = pieces * i / launches;
  z.last = pieces * (i + 1) / launches;
  z.head = from;
  z.tail = hi;
  if (i == 0) {
    z.head_bytes = static_cast<int32_t>(lo - from);
    z.tail_bytes = static_cast<int32_t>(to - hi);
  }
  return z;
}

// Workgroups for a share of the zeros; threads of a launch stay below 2^32.
int64_t zero_blocks(const Zeros& z) {
  const int64_t b = (z.last - z.first + kZeroPieces - 1) / kZeroPieces;
  return b == 0 && z.head_bytes + z.tail_bytes > 0 ? 1 : b;
}

}  // namespace

int enqueue_lookup(const LookupArgs& a, std::string* err) {
  if (a.n == 0) return kOk;
  const int64_t row_groups = (a.cols + kGroup - 1) / kGroup;
  const Lookup l = {addr(a.tokens), addr(a.table), addr(a.residual.data), addr(a.y), a.n * row_groups,
                    a.residual.stride, static_cast<uint32_t>(row_groups), static_cast<uint32_t>(a.cols),
                    static_cast<uint32_t>(a.vocab), a.token_bytes, a.scale};
  const int64_t want = (l.groups + kTile - 1) / kTile;
  const dim3 grid(static_cast<unsigned>(want < (1 << 20) ? want : 1 << 20));
  hipStream_t s = static_cast<hipStream_t>(a.stream);
  by_type(a.table_dtype, [&](auto t) {
    by_type(a.dtype, [&](auto d) {
      hipLaunchKernelGGL((lookup_kernel<decltype(t)::value, decltype(d)::value>), grid, dim3(kThreads), 0, s, l);
    });
  });
  HIP_OK(hipGetLastError(), "launch lookup_kernel");
  return kOk;
}

int enqueue_lookup_backward(const LookupBackwardArgs& a, std::string* err) {
  if (a.vocab == 0 || (a.n == 0 && a.accumulate)) return kOk;
  const LookupPlan p = lookup_plan(a.n, a.vocab, a.cols);
  hipStream_t s = static_cast<hipStream_t>(a.stream);
  char* ws = static_cast<char*>(a.workspace);
  auto words = [&](int64_t at) { return reinterpret_cast<uint32_t*>(ws + at); };
  Sort k = {};
  k.n = a.n;
  k.vocab = static_cast<uint32_t>(a.vocab);
  k.tiles = static_cast<uint32_t>(p.tiles);
  k.token_bytes = a.token_bytes;
  k.digit = p.digit;
  k.passes = p.passes;
  k.hist = words(p.hist);
  k.totals = words(p.totals);
  k.joins = words(p.joins);
  int sorted = 0;                                  // which of the two buffers holds the result
  if (p.tiles == 1) {
    k.tokens = addr(a.tokens);
    k.keys = words(p.keys[0]);
    k.order = words(p.order[0]);
    k.zeros = zeros_of(a, 0, 1);
    hipLaunchKernelGGL(sort_tile_kernel, dim3(static_cast<unsigned>(1 + zero_blocks(k.zeros))), dim3(kSortThreads), 0,
                       s, k);
    HIP_OK(hipGetLastError(), "launch sort_tile_kernel");
  } else {
    k.scanned = p.tiles > kScanTiles;
    for (int pass = 0; pass < p.passes; ++pass) {
      k.tokens = pass == 0 ? addr(a.tokens) : 0;
      k.keys_in = words(p.keys[sorted]);
      k.order_in = words(p.order[sorted]);
      sorted = pass == 0 ? 0 : 1 - sorted;
      k.keys = words(p.keys[sorted]);
      k.order = words(p.order[sorted]);
      k.shift = pass * p.digit;
      k.zeros = zeros_of(a, 2 * pass, 2 * p.passes);
      hipLaunchKernelGGL(sort_count_kernel, dim3(static_cast<unsigned>(p.tiles + zero_blocks(k.zeros))),
                         dim3(kSortThreads), 0, s, k);
      HIP_OK(hipGetLastError(), "launch sort_count_kernel");
      if (k.scanned) {
        hipLaunchKernelGGL(sort_scan_kernel, dim3(((1u << p.digit) + 63) / 64), dim3(kSortThreads), 0, s, k);
        HIP_OK(hipGetLastError(), "launch sort_scan_kernel");
      }
      k.zeros = zeros_of(a, 2 * pass + 1, 2 * p.passes);
      hipLaunchKernelGGL(sort_scatter_kernel, dim3(static_cast<unsigned>(p.tiles + zero_blocks(k.zeros))),
                         dim3(kSortThreads), 0, s, k);
      HIP_OK(hipGetLastError(), "launch sort_scatter_kernel");
    }
  }
  if (a.n == 0) return kOk;
  const Sum m = {addr(a.dy.data), addr(a.dtable), a.dy.stride, a.n, p.unit, p.units, words(p.keys[sorted]),
                 words(p.order[sorted]), reinterpret_cast<float*>(ws + p.partials), words(p.joins), words(p.list),
                 static_cast<uint32_t>(a.cols), static_cast<uint32_t>(a.vocab), a.grad_dtype, a.accumulate ? 1 : 0,
                 a.scale};
  const int64_t groups = (a.cols + kGroup - 1) / kGroup;
  int lanes = 8;
  while (lanes < 256 && lanes < groups) lanes *= 2;
  const int64_t each = 256 / lanes;
  const dim3 grid(static_cast<unsigned>((p.units + each - 1) / each), static_cast<unsigned>((groups + lanes - 1) / lanes));
  by_type(a.dtype, [&](auto d) { hipLaunchKernelGGL((sum_kernel<decltype(d)::value>), grid, dim3(256), 0, s, m, lanes); });
  HIP_OK(hipGetLastError(), "launch sum_kernel");
  if (p.units > 1) {
    hipLaunchKernelGGL(join_kernel, dim3(1024), dim3(256), 0, s, m);
    HIP_OK(hipGetLastError(), "launch join_kernel");
  }
  return kOk;
}

}  // namespace ddpb
