// optim.hpp -- host side of the operators that follow a synchronisation: the
// global gradient norm and the AdamW step over many tensors, with their tile
// tables and workspace layouts. No HIP types appear here; device work goes
// through OptimDevice.
#pragma once

#include <cstdint>
#include <memory>
#include <string>
#include <vector>

#include "core.hpp"

#ifdef __HIP__
#define DDPB_HD __host__ __device__
#else
#define DDPB_HD
#endif

namespace ddpb {

enum DType : int32_t { kF32 = 0, kBF16 = 1, kF16 = 2 };
constexpr int64_t dtype_size(int32_t d) { return d == kF32 ? 4 : 2; }

// Elements that share the scale of an 8-bit state.
constexpr uint32_t kStateBlock = 64;
// Elements per tile of AdamW's table; tiles start on block boundaries. The
// workgroups of a whole tile share its entry. What is left of a variable has
// an entry for each workgroup: with entries of whole tiles there too, 5000
// variables of 64 elements took 49 us instead of 7, most of it workgroups
// without work.
constexpr int64_t kOptimTile = 4096;

// How a step is cut into workgroups (why so: optim.hip): threads, groups of
// four elements per lane, elements per workgroup.
constexpr int adamw_threads(bool f8) { return f8 ? 256 : 64; }
constexpr int adamw_unroll(int32_t param_dtype, bool master, bool f8) {
  return f8 && param_dtype != 0 && !master ? 2 : 1;
}
constexpr int64_t adamw_part(int32_t param_dtype, bool master, bool f8) {
  return 4 * adamw_threads(f8) * adamw_unroll(param_dtype, master, f8);
}
// A launch has fewer than 2^32 threads.
constexpr int64_t kMaxThreads = (int64_t(1) << 32) - 1;
// The norm's tiles, and its workgroups, each of which leaves one partial sum:
// constants, so that the order of the sum does not depend on the device.
constexpr int64_t kNormTileBytes = 16384;
constexpr int32_t kNormBlocks = 512;

// Counters of the workgroups that are done, kArriveSlots of them and one of
// the slots, each in a cache line of its own. All return to 0 with the last.
constexpr int kArriveSlots = 64;
constexpr int kArriveStride = 32;   // uint32 per counter
constexpr int64_t kArriveBytes = (kArriveSlots + 1) * kArriveStride * 4;

// Device-side work descriptors, read by the kernels.
struct NormTile {
  uint64_t grad;      // address of the tile's first element
  int32_t len;        // elements
  int32_t dtype;      // DType
};
static_assert(sizeof(NormTile) == 16, "tile layout is shared with the kernels");

// A tile names its variable, whose record holds the addresses: all tiles of a
// large variable share one record, which the scalar caches then hold.
struct AdamwTile {
  int32_t var;
  int32_t len;        // elements: kOptimTile, or at most a workgroup's
  int64_t start;      // first element inside the variable
};
static_assert(sizeof(AdamwTile) == 16, "tile layout is shared with the kernels");

struct AdamwVar {
  uint64_t src;       // fp32 master, or the parameter of replica 0
  uint64_t out;       // parameter of replica 0
  uint64_t grad;
  uint64_t avg;       // exp_avg: fp32, or e4m3 codes
  uint64_t second;    // exp_avg_sq: fp32, or e4m3 codes of its root
  uint64_t avg_scale; // e8m0 scales (8-bit states)
  uint64_t root_scale;
  uint64_t group0;    // index of the first group of four elements, for the random bits
  double weight_decay;
  double lr_scale;
};
static_assert(sizeof(AdamwVar) == 80, "record layout is shared with the kernels");

// What a norm leaves on the device (ddpb_norm_result).
struct NormResult {
  float norm;
  float coef;
  int32_t skip;
  uint32_t pad;
};
static_assert(sizeof(NormResult) == 16, "layout is shared with the header");

// The scalars of the coming step, advanced on the device by each step that is
// not skipped, so that a replayed graph counts its steps too.
struct StepScalars {
  int64_t done;       // steps done
  double inv_bc1;     // 1 / (1 - beta1^t), t = done + 1
  float inv_rbc2;     // 1 / sqrt(1 - beta2^t)
  uint32_t key0, key1;
  uint32_t pad;
};
static_assert(sizeof(StepScalars) == 32, "layout is shared with the kernels");

// x^e by squaring, the same operations on host and device.
DDPB_HD inline double int_power(double x, int64_t e) {
  double y = 1.0;
  for (; e > 0; e >>= 1, x *= x)
    if (e & 1) y *= x;
  return y;
}

DDPB_HD inline StepScalars step_scalars(int64_t done, double beta1, double beta2, uint64_t seed) {
  StepScalars s;
  const int64_t t = done + 1;
  s.done = done;
  s.inv_bc1 = 1.0 / (1.0 - int_power(beta1, t));
  s.inv_rbc2 = static_cast<float>(1.0 / __builtin_sqrt(1.0 - int_power(beta2, t)));
  // The key of the step's random bits: multiply and xor-shift mixing of seed and t.
  uint64_t k = seed + static_cast<uint64_t>(t) * 0xA3B1956C7E4D2F89ull;
  k ^= k >> 32;
  k *= 0xD6C7F2A94B1E8653ull;
  k ^= k >> 29;
  k *= 0x9E6B3F85C2D4A717ull;
  k ^= k >> 32;
  s.key0 = static_cast<uint32_t>(k);
  s.key1 = static_cast<uint32_t>(k >> 32);
  s.pad = 0;
  return s;
}

// The 16 + 16 random bits of an element (high half: m, low half: r),
// counter-based: multiply and xor-shift rounds over the 64-bit index of its
// group of four elements under the step's key, then a short round for each
// element. A lane starts from the hash of its first group in a tile and goes on
// by `groups`, which are few; the index's high word changes where the low one
// wraps, inside one tile in 4 G groups at most.
constexpr uint32_t kHashIndex = 0x9C8E5A6Du, kHashHigh = 0x7F4A3C15u;

// The hash of group `tile` + `lane`, but for a wrap between the two.
DDPB_HD inline uint32_t hash_start(uint64_t tile, uint32_t lane, uint32_t key0) {
  return (static_cast<uint32_t>(tile) + lane) * kHashIndex + static_cast<uint32_t>(tile >> 32) * kHashHigh + key0;
}
// The hash of group `tile` + `lane` + `groups` from that start; `tile_low` is
// the low word of the tile's first group.
DDPB_HD inline uint32_t hash_at(uint32_t start, uint32_t tile_low, uint32_t lane, uint32_t groups) {
  uint32_t h = start + groups * kHashIndex;
  if (__builtin_expect(tile_low > UINT32_MAX - static_cast<uint32_t>(kOptimTile / 4 - 1), 0))
    h += tile_low + lane + groups < tile_low ? kHashHigh : 0;
  return h;
}
DDPB_HD inline uint32_t hash_mix(uint32_t h, uint32_t key1) {
  h ^= h >> 15;
  h *= 0x85D3B2A7u;
  h ^= (h >> 13) ^ key1;
  h *= 0xC5A7E36Bu;
  return h ^ (h >> 16);
}
DDPB_HD inline uint32_t hash_element(uint32_t mixed, uint32_t j) {
  uint32_t y = mixed + j * 0x6D2B4E95u;
  y ^= y >> 16;
  y *= 0xB5297A4Du;
  return y ^ (y >> 15);
}

struct NormLaunch {
  void* stream;
  int device;
  const NormTile* tiles;
  int32_t ntiles;
  double* partials;
  uint32_t* arrived;          // kArriveBytes
  NormResult* result;
  double max_norm, grad_scale;
  int32_t skip_nonfinite;
};

struct AdamwLaunch {
  void* stream;
  int device;
  int32_t param_dtype, grad_dtype, f8, master;
  const AdamwTile* tiles;     // whole tiles, then the rests
  const AdamwVar* vars;
  int32_t whole, rests;
  const uint64_t* replicas;   // (R - 1) * P parameter addresses, replica-major
  int32_t R, P;
  StepScalars* scalars;
  uint32_t* arrived;          // kArriveBytes
  const NormResult* clip;     // or NULL
  const NormResult* neutral;  // norm 0, coef 1
  const float* lr_device;     // or NULL: lr
  double lr, grad_scale;
  double beta1, beta2, eps;
  uint64_t seed;
};

// Device work. The HIP implementation enqueues kernels; the test build's
// does nothing.
class OptimDevice {
 public:
  virtual ~OptimDevice() = default;
  virtual int current(int* device, std::string* err) = 0;
  // Refuses (kErrState) while `stream` is being captured; copies and waits.
  virtual int upload(int device, void* stream, void* dst, const void* src, size_t bytes, std::string* err) = 0;
  virtual int download(int device, void* stream, void* dst, const void* src, size_t bytes, std::string* err) = 0;
  virtual int norm(const NormLaunch& l, std::string* err) = 0;
  virtual int adamw(const AdamwLaunch& l, std::string* err) = 0;
};
OptimDevice* optim_device();

// A caller's binding to a reducer's gradients: which binding of the reducer
// they were taken from.
struct ReducerTie {
  int64_t bind_id = 0;
  // Checked by every call that reads the gradients: the reducer (may be NULL)
  // still has that binding, no iteration is open and none has failed.
  int check(const Reducer* red, const char* what, std::string* err) const;
};

class Norm {
 public:
  Norm(std::vector<int64_t> numel, std::vector<int32_t> dtypes)
      : numel_(std::move(numel)), dtypes_(std::move(dtypes)) {}
  int64_t workspace_bytes() const;
  int bind(void* const* grads, void* ws, int64_t ws_bytes, void* stream, const Reducer* red, std::string* err);
  int compute(const Reducer* red, double max_norm, double grad_scale, bool skip_nonfinite, std::string* err);

 private:
  int64_t ntiles() const;
  std::vector<int64_t> numel_;
  std::vector<int32_t> dtypes_;
  NormLaunch l_{};
  ReducerTie tie_;
  bool bound_ = false;
};

struct AdamwConfig {
  std::vector<int64_t> numel;
  int32_t R = 1;
  int32_t param_dtype = kF32, grad_dtype = kF32;
  bool f8 = false, master = false;
  double beta1 = 0.9, beta2 = 0.999, eps = 1e-8;
  std::vector<double> weight_decay, lr_scale;
  uint64_t seed = 0;
};

struct AdamwBuffers {
  void* const* params;        // R * P, replica-major
  void* const* grads;
  void* const* master;
  void* const* avg;
  void* const* second;
  void* const* avg_scale;
  void* const* root_scale;
};

class Adamw {
 public:
  explicit Adamw(AdamwConfig c) : c_(std::move(c)) {}
  int64_t workspace_bytes() const;
  int bind(const AdamwBuffers& b, int64_t done, void* ws, int64_t ws_bytes, void* stream, const Reducer* red,
           std::string* err);
  int step(const Reducer* red, double lr, const float* lr_device, double grad_scale, const void* clip,
           std::string* err);
  int set_step(int64_t done, std::string* err);
  int get_step(int64_t* done, std::string* err);
  const AdamwConfig& config() const { return c_; }

 private:
  int64_t whole() const;
  int64_t rests() const;
  int64_t vars_at() const;
  int64_t replicas_at() const;
  AdamwConfig c_;
  AdamwLaunch l_{};
  ReducerTie tie_;
  bool bound_ = false;
};

}  // namespace ddpb
