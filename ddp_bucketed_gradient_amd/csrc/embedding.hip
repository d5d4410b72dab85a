// embedding.hip -- CDNA4 (gfx950) kernels of the embedding: the lookup, and its
// gradient by sorted tokens.
#include "group8.hpp"

namespace ddpb {
namespace {

// A token of 4 or 8 bytes; what lies outside of the table becomes `vocab`. Without
// a branch, so that several can be loaded together: the upper half of a token of
// four bytes is read where the lower one is, and left out.
__device__ __forceinline__ uint32_t token_at(uint64_t tokens, uint32_t bytes, uint32_t i, uint32_t vocab) {
  const uint64_t at = tokens + static_cast<uint64_t>(i) * bytes;
  const uint32_t low = *G<const uint32_t>(at), high = *G<const uint32_t>(at + (bytes - 4));
  return (bytes == 4 || high == 0) && low < vocab ? low : vocab;
}

// ---------------------------------------------------------------------------
// y_i = scale table[t_i] + residual_i, in fp32, rounded once.
struct Lookup {
  uint64_t tokens, table, residual, y;
  uint64_t residual_row;        // bytes from row to row
  uint32_t n, cols, vocab, slice, shift;
  uint32_t token_bytes;
  float scale;
};

// A wave takes kRows rows of one slice, 64 groups of eight columns or less, so
// that tokens and row addresses are uniform. Rows of 32 groups and less share a
// wave, a power of two of lanes each (PACKED). BERT-large's words, fp32 to bf16:
// 11.9 us, 4.7 TB/s; the chain of token, row and store bounds it.
constexpr int kRows = 4;
template <int TD, int D, bool PACKED, int EDGE>
__global__ __launch_bounds__(256) void lookup_kernel(Lookup a) {
  constexpr uint32_t size = sizeof(typename Of<D>::one), table_size = sizeof(typename Of<TD>::one);
  const uint32_t lane = PACKED ? threadIdx.x & ((1u << a.shift) - 1) : threadIdx.x & 63;
  const uint32_t part = PACKED ? threadIdx.x >> a.shift : __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t parts = PACKED ? 256u >> a.shift : 4;
  const Group g = group_at<EDGE>(a.cols, (blockIdx.y * a.slice + lane) * 8);
  if (g.left <= 0 || lane >= a.slice) return;
  for (uint32_t first = (blockIdx.x * parts + part) * kRows; first < a.n; first += gridDim.x * parts * kRows) {
    uint32_t t[kRows];
    Raw<TD> x[kRows];
    Raw<D> r[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k)
      t[k] = token_at(a.tokens, a.token_bytes, min(first + k, a.n - 1), a.vocab);
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      x[k] = Raw<TD>{};
      r[k] = Raw<D>{};
      if (t[k] < a.vocab) x[k] = load_raw<TD, EDGE>(a.table + static_cast<uint64_t>(t[k]) * a.cols * table_size + g.c * table_size, g.left);
      if (a.residual != 0 && first + k < a.n) r[k] = load_raw<D, EDGE>(a.residual + (first + k) * a.residual_row + g.c * size, g.left);
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      if (first + k >= a.n) break;
      v8f y = 0.0f;
      if (t[k] < a.vocab) y = widen<TD>(x[k]) * a.scale;
      if (a.residual != 0) y = y + widen<D>(r[k]);
      store8<D, EDGE>(a.y + static_cast<uint64_t>(first + k) * a.cols * size + g.c * size, g.left, y);
    }
  }
}

// ---------------------------------------------------------------------------
// The gradient: dtable[v] = scale * sum of dy_i over the places i of token v, in
// order of i and without atomics on values, so the same bits on every run.
//
//  1. Sort the places by token, stably: a radix sort, `digit` bits a pass, each
//     a histogram of every tile of keys and a scatter; few tokens in one launch,
//     by ranges of them. Beside it, workgroups that would be idle write the zeros
//     of a gradient that is not added to.
//  2. Sum: the sorted places are cut into units of equal length, so that a
//     token that holds many places (padding, the commonest words) is shared
//     by many waves. A run of one token that covers no whole unit belongs to
//     the unit where it begins. One that does leaves a partial sum in each of
//     its units, and
//  3. a last kernel adds those up.
//
// BERT-large (16384 tokens, 30522 x 1024 in fp32 from bf16): 41 us, of which the
// zeros beside the sort take 22 (5.7 TB/s), the sum 14.5 and the join 5.2.
struct Zeros {
  uint64_t at;        // 16-byte aligned
  int64_t first, last;   // of the 16-byte pieces there, this launch's share
  uint64_t head, tail;   // odd bytes before and behind the pieces: addresses
  int32_t head_bytes, tail_bytes;   // 0 but in the first launch
};
constexpr int kZeroBlocks = 448;                    // workgroups that write them, at most
constexpr int64_t kZeroPieces = kSortThreads * 8;   // that one of them writes at a time

// Non-temporal stores of device scope: BERT-large's 125 MB of zeros beside the
// sort take 22.2 us instead of 31.9, and the sum that follows, whose reads would
// meet the caches full of them, 14.6 us instead of 22.8.
__device__ __forceinline__ void write_zeros(const Zeros& z, uint32_t block, uint32_t blocks) {
  for (int64_t from = z.first + block * kZeroPieces; from < z.last; from += blocks * kZeroPieces) {
    const uint64_t base = z.at + static_cast<uint64_t>(from) * 16;
    const int64_t rest = min((z.last - from) * 16, kZeroPieces * 16);
    const auto r = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(base), 0, static_cast<int>(rest), 0x00020000);
#pragma unroll
    for (int u = 0; u < 8; ++u)
      __builtin_amdgcn_raw_buffer_store_b128(v4u{0, 0, 0, 0}, r, (u * kSortThreads + threadIdx.x) * 16, 0, kPolicyDeviceNT);
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
  uint32_t token_bytes;
  int32_t shift, digit, scanned;
  int32_t passes;               // of a sort by one workgroup
  Zeros zeros;
};

__device__ __forceinline__ void load_keys(const Sort& a, int64_t tile, uint32_t (&key)[kSortKeys], uint32_t (&place)[kSortKeys]) {
  // a wave's keys are consecutive: 64 at a time
  const uint32_t n = static_cast<uint32_t>(a.n);
  const uint32_t at = static_cast<uint32_t>(tile * kSortTile) + (threadIdx.x >> 6) * (64 * kSortKeys) + (threadIdx.x & 63);
#pragma unroll
  for (int e = 0; e < kSortKeys; ++e) {
    const uint32_t i = min(at + e * 64, n - 1);            // (what is behind the end is not used)
    key[e] = a.tokens != 0 ? token_at(a.tokens, a.token_bytes, i, a.vocab) : a.keys_in[i];
    place[e] = a.tokens != 0 ? i : a.order_in[i];
  }
}

constexpr int kWaves = kSortThreads / 64, kBins = 1 << kMaxDigit;

// What lanes of a wave wrote to LDS is seen by its other lanes behind this.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The lanes that are there and hold the same digit.
template <int BITS>
__device__ __forceinline__ uint64_t equal_digits(uint32_t d, bool there) {
  uint64_t same = __ballot(there);
#pragma unroll
  for (int b = 0; b < BITS; ++b) {
    const bool one = d >> b & 1;
    const uint64_t ones = __ballot(one);
    same &= one ? ones : ~ones;
  }
  return same;
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

// All of the sort in one launch, for up to kRangeKeys tokens. Workgroup g of
// kRanges takes the tokens t with t % kRanges = g (so that neighbouring common
// ones do not meet in one), finds their places among all, and sorts those by t /
// kRanges in LDS, six bits a pass, one counter of a wave's digits to a thread.
// What it counts of the ranges before its own is where its places begin. The
// order is one of groups: t % kRanges, then t. Bound by latency: 8192 tokens take
// 10.5 us, where two passes of count and scatter took 24.
//
// 16384 tokens, because their LDS (132 KB) is the largest that holds a power of two
// of them. The whole added-to gradient of 64 columns, by ranges and by tiles, which
// sort in two passes (30522 rows) or in one (1000 rows):
//   tokens  30522 rows: ranges, tiles   1000 rows: ranges, tiles
//     1024        17.2, 23.5 us              15.2, 18.5 us
//     8192        23.0, 29.3                 20.9, 22.0
//    16384        32.8, 36.2                 28.5, 25.7
//    16385        39.1, 42.9                 33.0, 29.7
// and BERT-large's 30522 x 1024 written: 16384 tokens 39.4, 49.7, 16385 tokens 50.8,
// 56.7 (ranges of up to 18432 tokens built for this comparison).
constexpr int kRangeBits = 6, kDigits = 1 << kRangeBits;
struct RangeLds {
  uint32_t token[kRangeKeys];
  uint16_t place[2][kRangeKeys];
  uint32_t count[kDigits * kWaves];         // [digit][wave]
  uint32_t waves[kWaves];
  uint2 here[kWaves];                       // of each wave: tokens of the range, and of those before it
};

__global__ __launch_bounds__(kSortThreads) void sort_ranges_kernel(Sort a) {
  extern __shared__ char raw_lds[];
  if (blockIdx.x >= kRanges) {
    write_zeros(a.zeros, blockIdx.x - kRanges, gridDim.x - kRanges);
    return;
  }
  RangeLds& s = *reinterpret_cast<RangeLds*>(raw_lds);
  const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63, range = blockIdx.x, n = static_cast<uint32_t>(a.n);
  const uint64_t under = (uint64_t(1) << lane) - 1;
  if (range == 0 && threadIdx.x == 0) *a.joins = 0;
  // a wave's share of the tokens is consecutive
  const uint32_t each = (n + kSortThreads - 1) / kSortThreads * 64, from = wave * each, to = min(from + each, n);
  for (uint32_t i = from + lane; i < to; i += 64 * 4) {
    uint32_t t[4];
#pragma unroll
    for (uint32_t e = 0; e < 4; ++e) t[e] = token_at(a.tokens, a.token_bytes, min(i + e * 64, to - 1), a.vocab);
#pragma unroll
    for (uint32_t e = 0; e < 4; ++e)
      if (i + e * 64 < to) s.token[i + e * 64] = t[e];
  }
  uint32_t mine = 0, below = 0;
  for (uint32_t i = from; i < to; i += 64) {
    const uint32_t t = i + lane < to ? s.token[i + lane] : a.vocab;
    mine += __popcll(__ballot(t < a.vocab && t % kRanges == range));
    below += __popcll(__ballot(t < a.vocab && t % kRanges < range));
  }
  if (lane == 0) s.here[wave] = make_uint2(mine, below);
  __syncthreads();
  uint32_t at = 0, m = 0, first = 0;               // first: where the range's places begin; m: how many
  for (uint32_t w = 0; w < static_cast<uint32_t>(kWaves); ++w) {
    const uint2 h = s.here[w];
    at += w < wave ? h.x : 0;
    m += h.x;
    first += h.y;
  }
  for (uint32_t i = from; i < to; i += 64) {
    const uint32_t t = i + lane < to ? s.token[i + lane] : a.vocab;
    const uint64_t in = __ballot(t < a.vocab && t % kRanges == range);
    if (in >> lane & 1) s.place[0][at + __popcll(in & under)] = static_cast<uint16_t>(i + lane);
    at += __popcll(in);
  }
  // behind the last range: the tokens outside of the table
  if (range == kRanges - 1)
    for (uint32_t i = first + m + threadIdx.x; i < n; i += kSortThreads) a.keys[i] = a.vocab;

  const uint32_t share = (m + kSortThreads - 1) / kSortThreads * 64, begin = min(wave * share, m), end = min(begin + share, m);
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * kRangeBits;
    const uint16_t* in = s.place[pass & 1];
    uint16_t* out = s.place[~pass & 1];
    s.count[threadIdx.x] = 0;
    __syncthreads();
    for (uint32_t i = begin + lane; i < end; i += 64)
      atomicAdd(&s.count[(s.token[in[i]] / kRanges >> shift) % kDigits * kWaves + wave], 1u);
    __syncthreads();
    const uint32_t before = scan(s.count[threadIdx.x], s.waves);
    s.count[threadIdx.x] = before;
    __syncthreads();
    for (uint32_t i = begin; i < end; i += 64) {   // stable: 64 at a time, each behind the equal ones below it
      const bool there = i + lane < end;
      const uint32_t place = there ? in[i + lane] : 0, token = s.token[place];
      const uint32_t d = (token / kRanges >> shift) % kDigits;
      const uint64_t same = equal_digits<kRangeBits>(d, there), lower = same & under;
      const uint32_t base = s.count[d * kWaves + wave], to_place = base + __popcll(lower);
      wave_fence();
      if (there && lower == 0) s.count[d * kWaves + wave] = base + __popcll(same);
      wave_fence();
      if (!there) continue;
      if (pass < a.passes - 1) {
        out[to_place] = static_cast<uint16_t>(place);
      } else {
        a.keys[first + to_place] = token;
        a.order[first + to_place] = place;
      }
    }
    __syncthreads();
  }
}

__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(Sort a) {
  if (blockIdx.x >= a.tiles) {
    write_zeros(a.zeros, blockIdx.x - a.tiles, gridDim.x - a.tiles);
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
    write_zeros(a.zeros, blockIdx.x - a.tiles, gridDim.x - a.tiles);
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
#pragma unroll 16
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
  uint64_t dy, dtable, keys, order;
  uint64_t dy_row, table_row;   // bytes from row to row
  uint32_t n, unit, units;      // at most 2^30 places
  uint32_t cols, vocab;
  uint32_t slice;               // groups of eight columns that a wave takes: equal shares, at most 64
  float* partials;              // [unit][run from the left, run to the right][cols]
  uint32_t* joins;
  uint2* list;                  // of the long runs: the unit where it begins, its token
  float scale;
};

// Written before this kernel, by one that has ended: a scalar load.
__device__ __forceinline__ uint32_t key_at(const Sum& a, uint32_t i) {
  return *(const __attribute__((address_space(4))) uint32_t*)(a.keys + static_cast<uint64_t>(i * 4));
}

__device__ __forceinline__ uint32_t lane_of(uint32_t x, int i) {
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(x), i));
}

// A wave sums eight columns a lane of one unit. The keys and places of 64 sorted
// places lie in its lanes, so that the run ends are a mask and everything but
// the rows themselves is uniform. The rows of kAhead places are loaded together,
// with what stands in the table where the sums are added to that.
//
// BERT-large's 16384 places in bf16 into fp32: 14.5 us behind the zeros (3.4 TB/s of
// rows in and out; four waves a CU, of which each goes through the latencies of
// keys, rows and stores once). 131072 places of 768 columns, 40 % of them one
// token, added to: 77 us for 257 MB of scattered rows in and out, 3.3 TB/s (3.6 of
// the bytes that counters see; the rows of dy alone: 41 us, 4.4 TB/s). Twice or four times the waves took 69-78 us (and the
// join twice as long), finished rows collected in LDS and written eight at a
// time 84, old rows loaded only when a run ends 89.
template <int D, int GD, bool ADD, int EDGE>
__global__ __launch_bounds__(256) void sum_kernel(Sum a) {
  typedef typename Of<D>::one one;
  typedef typename Of<GD>::one grad_one;
  constexpr int kAhead = 8;
  const uint32_t u = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (u >= a.units) return;
  const uint32_t lane = threadIdx.x & 63;
  const Group g = group_at<EDGE>(a.cols, lane < a.slice ? (blockIdx.y * a.slice + lane) * 8 : a.cols);
  const uint32_t c = g.c;
  const int left = g.left;
  const uint32_t s = u * a.unit, e = min(s + a.unit, a.n), e2 = min(e + a.unit, a.n);
  const uint32_t first = key_at(a, s), last = key_at(a, e - 1);
  const uint32_t before = key_at(a, s > 0 ? s - 1 : 0), unit_before = key_at(a, s > 0 ? s - a.unit : 0);
  const uint32_t behind = key_at(a, e < a.n ? e : e - 1), unit_behind = key_at(a, e2 - 1);
  uint32_t key, next, place;       // of a lane's place among 64
  auto window = [&](uint32_t i) {
    key = next = a.vocab;
    place = 0;
    if (i < e2) {
      key = *G<const uint32_t>(a.keys + static_cast<uint64_t>(i * 4));
      place = *G<const uint32_t>(a.order + static_cast<uint64_t>(i * 4));
      if (i + 1 < a.n) next = *G<const uint32_t>(a.keys + static_cast<uint64_t>(i * 4 + 4));
    }
  };
  window(s + lane);
  if (first >= a.vocab) return;
  // the run that comes in from the left: another unit's, unless it covers a whole unit
  const bool from_left = s > 0 && before == first;
  const bool mine = !from_left || last == first || unit_before == first;
  // the run that goes out to the right: ours to its end, unless it covers a whole unit
  const bool to_right = e < a.n && last < a.vocab && behind == last;
  const bool long_right = to_right && (first == last || unit_behind == last);
  const uint32_t stop = to_right && !long_right ? e2 : e;
  const uint64_t partial = reinterpret_cast<uint64_t>(a.partials) + (static_cast<uint64_t>(u) * 2 * a.cols + c) * 4;

  v8f x = 0.0f;
  bool open_left = from_left && mine, pending = false;   // the run in x began in another unit; it has not ended
  for (uint32_t p = s; p < stop; p += 64) {
    const uint32_t i = p + lane;
    if (p > s) window(i);
    const bool ours = i < stop && key < a.vocab && (mine || key != first) && (i < e || key == last);
    const uint64_t todo = __ballot(ours), ends = __ballot(ours && key != next);
    if (todo == 0) continue;
    const int from = __builtin_ctzll(todo), to = 64 - __builtin_clzll(todo);    // they are consecutive
    for (int j = from; j < to; j += kAhead) {
      Raw<D> rows[kAhead];
      Raw<GD> old[ADD ? kAhead : 1];
      if (left > 0) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int at = min(j + k, to - 1);
          rows[k] = load_raw<D, EDGE>(a.dy + lane_of(place, at) * a.dy_row + c * static_cast<uint32_t>(sizeof(one)), left);
          if constexpr (ADD) {
            if (j + k < to && (ends >> at & 1))
              old[k] = load_raw<GD, EDGE>(a.dtable + lane_of(key, at) * a.table_row + c * static_cast<uint32_t>(sizeof(grad_one)), left);
          }
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          if (j + k >= to) break;
          x = x + widen<D>(rows[k]);
          if ((ends >> (j + k) & 1) == 0) continue;
          if (open_left) {
            store8<kF32, EDGE>(partial, left, x);
          } else {
            x = x * a.scale;
            if constexpr (ADD) x = x + widen<GD>(old[k]);
            store8<GD, EDGE>(a.dtable + lane_of(key, j + k) * a.table_row + c * static_cast<uint32_t>(sizeof(grad_one)), left, x);
          }
          open_left = false;
          x = 0.0f;
        }
      }
    }
    pending = (ends >> (to - 1) & 1) == 0;
    open_left = open_left && ends == 0;               // the same in lanes without columns
  }
  if (!pending) return;
  if (left > 0) store8<kF32, EDGE>(partial + (open_left ? 0 : static_cast<uint64_t>(a.cols) * 4), left, x);
  if (!open_left && blockIdx.y == 0 && lane == 0) a.list[atomicAdd(a.joins, 1u)] = make_uint2(u, last);
}

// The runs that cover whole units: 16 columns to a wave, four to a lane, and 16
// lanes for each of them, which take every 16th unit. Bound by latency: 5 us for
// some 30 runs, 13 us where one run has 410 parts.
constexpr int kJoinCols = 16, kJoinLanes = kJoinCols / 4, kJoinLines = 64 / kJoinLanes, kJoinAhead = 4;
template <int GD, bool ADD>
__global__ __launch_bounds__(256) void join_kernel(Sum a) {
  typedef typename Of<GD>::one one;
  typedef v4f any __attribute__((aligned(4)));
  const uint32_t lane = threadIdx.x % kJoinLanes, line = (threadIdx.x & 63) / kJoinLanes, joins = *a.joins;
  const uint32_t c = (blockIdx.y * 4 + (threadIdx.x >> 6)) * kJoinCols + lane * 4;
  const uint32_t left = c < a.cols ? min(a.cols - c, 4u) : 0;
  uint2 run = a.list[blockIdx.x];                 // read beside the count: there is room for every unit
  for (uint32_t k = blockIdx.x; k < joins; k += gridDim.x) {
    if (k != blockIdx.x) run = a.list[k];
    const uint32_t u = run.x, token = run.y;
    v4f x = 0.0f;
    // part 0 is the beginning in unit u, part i what unit u + i begins with, as long as that is the token
    bool more = left > 0;
    for (uint32_t i = line; __any(more); i += kJoinLines * kJoinAhead) {
      bool same[kJoinAhead];
      v4f y[kJoinAhead];
#pragma unroll
      for (int q = 0; q < kJoinAhead; ++q) {
        const uint32_t at = u + i + q * kJoinLines;
        same[q] = more && at < a.units && (at == u || *G<const uint32_t>(a.keys + static_cast<uint64_t>(at * a.unit * 4)) == token);
      }
#pragma unroll
      for (int q = 0; q < kJoinAhead; ++q) {
        const uint32_t at = u + i + q * kJoinLines;
        y[q] = 0.0f;
        if (!same[q]) continue;
        const float* p = a.partials + (static_cast<uint64_t>(at) * 2 + (at == u)) * a.cols + c;
        if (left == 4) {
          y[q] = *reinterpret_cast<const any*>(p);
        } else {
#pragma unroll
          for (uint32_t j = 0; j < 3; ++j)
            if (j < left) y[q][j] = p[j];
        }
      }
#pragma unroll
      for (int q = 0; q < kJoinAhead; ++q) x = x + y[q];
      more = same[kJoinAhead - 1];
    }
#pragma unroll
    for (int d = kJoinLanes; d < 64; d *= 2) {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] += __shfl_xor(x[j], d, 64);
    }
    if (line != 0) continue;
    auto* p = G<one>(a.dtable + token * a.table_row + c * static_cast<uint32_t>(sizeof(one)));
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j)
      if (j < left) p[j] = static_cast<one>(x[j] * a.scale + (ADD ? static_cast<float>(p[j]) : 0.0f));
  }
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

// Workgroups for a share of the zeros.
int64_t zero_blocks(const Zeros& z) {
  const int64_t b = (z.last - z.first + kZeroPieces - 1) / kZeroPieces;
  return b == 0 && z.head_bytes + z.tail_bytes > 0 ? 1 : b < kZeroBlocks ? b : kZeroBlocks;
}

}  // namespace

int enqueue_lookup(const LookupArgs& a, std::string* err) {
  if (a.n == 0) return kOk;
  const int64_t groups = (a.cols + kGroup - 1) / kGroup, slices = (groups + 63) / 64;
  uint32_t shift = 0;                              // lanes of a row
  while ((1 << shift) < groups && shift < 6) ++shift;
  const Lookup l = {addr(a.tokens), addr(a.table), addr(a.residual.data), addr(a.y),
                    static_cast<uint64_t>(a.residual.stride * dtype_size(a.dtype)), static_cast<uint32_t>(a.n),
                    static_cast<uint32_t>(a.cols), static_cast<uint32_t>(a.vocab),
                    static_cast<uint32_t>((groups + slices - 1) / slices), shift, static_cast<uint32_t>(a.token_bytes), a.scale};
  hipStream_t s = static_cast<hipStream_t>(a.stream);
  const int64_t rows = (256 >> shift) * kRows, want = (a.n + rows - 1) / rows;         // rows of a workgroup
  const dim3 grid(static_cast<unsigned>(want < (1 << 20) ? want : 1 << 20), static_cast<unsigned>(slices));
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, l); };
  by_type(a.table_dtype, [&](auto t) {
    by_type(a.dtype, [&](auto d) {
      constexpr int TD = decltype(t)::value, OD = decltype(d)::value;
      if (a.cols < 8) go(lookup_kernel<TD, OD, true, kSmall>);
      else if (a.cols % 8 == 0) shift < 6 ? go(lookup_kernel<TD, OD, true, kWhole>) : go(lookup_kernel<TD, OD, false, kWhole>);
      else shift < 6 ? go(lookup_kernel<TD, OD, true, kShifted>) : go(lookup_kernel<TD, OD, false, kShifted>);
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
  k.token_bytes = static_cast<uint32_t>(a.token_bytes);
  k.digit = p.digit;
  k.passes = p.passes;
  k.hist = words(p.hist);
  k.totals = words(p.totals);
  k.joins = words(p.joins);
  int sorted = 0;                                  // which of the two buffers holds the result
  if (p.tiles == 0) {
    k.tokens = addr(a.tokens);
    k.keys = words(p.keys[0]);
    k.order = words(p.order[0]);
    k.zeros = zeros_of(a, 0, 1);
    hipLaunchKernelGGL(sort_ranges_kernel, dim3(static_cast<unsigned>(kRanges + zero_blocks(k.zeros))),
                       dim3(kSortThreads), sizeof(RangeLds), s, k);
    HIP_OK(hipGetLastError(), "launch sort_ranges_kernel");
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
  // Slices of the columns, a wave each. A last group that is shifted has the lane
  // before it in its own wave, which reads what both add to before either writes it.
  const int64_t groups = (a.cols + kGroup - 1) / kGroup;
  int64_t sums = (groups + 63) / 64;
  auto slice = [&] { return (groups + sums - 1) / sums; };
  while (sums > 1 && groups % slice() == 1) ++sums;
  const Sum m = {addr(a.dy.data), addr(a.dtable), addr(words(p.keys[sorted])), addr(words(p.order[sorted])),
                 static_cast<uint64_t>(a.dy.stride * dtype_size(a.dtype)),
                 static_cast<uint64_t>(a.cols * dtype_size(a.grad_dtype)), static_cast<uint32_t>(a.n),
                 static_cast<uint32_t>(p.unit), static_cast<uint32_t>(p.units), static_cast<uint32_t>(a.cols),
                 static_cast<uint32_t>(a.vocab), static_cast<uint32_t>(slice()),
                 reinterpret_cast<float*>(ws + p.partials), words(p.joins),
                 reinterpret_cast<uint2*>(ws + p.list), a.scale};
  const dim3 grid(static_cast<unsigned>((p.units + 3) / 4), static_cast<unsigned>(sums));
  const int64_t slices = (a.cols + 4 * kJoinCols - 1) / (4 * kJoinCols), runs = slices < 32 ? 2048 / slices : 64;
  const dim3 join_grid(static_cast<unsigned>(runs < p.units ? runs : p.units), static_cast<unsigned>(slices));
  by_type(a.grad_dtype, [&](auto g) {
    constexpr int GD = decltype(g)::value;
    by_type(a.dtype, [&](auto d) {
      constexpr int TD = decltype(d)::value;
      auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, m); };
      auto pick = [&](auto add) {
        constexpr bool ADD = decltype(add)::value;
        if (a.cols < 8) go(sum_kernel<TD, GD, ADD, kSmall>);
        else a.cols % 8 == 0 ? go(sum_kernel<TD, GD, ADD, kWhole>) : go(sum_kernel<TD, GD, ADD, kShifted>);
      };
      if (a.accumulate) pick(std::true_type());
      else pick(std::false_type());
    });
    if (p.units <= 1) return;
    if (a.accumulate) hipLaunchKernelGGL((join_kernel<GD, true>), join_grid, dim3(256), 0, s, m);
    else hipLaunchKernelGGL((join_kernel<GD, false>), join_grid, dim3(256), 0, s, m);
  });
  HIP_OK(hipGetLastError(), "launch sum_kernel or join_kernel");
  return kOk;
}

}  // namespace ddpb
