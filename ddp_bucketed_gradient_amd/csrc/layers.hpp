// layers.hpp -- host side of the operators beside a model's matrix products:
// layer norm, dropout and the embedding, each with its backward pass. Arguments,
// checks, workspace layouts and the rules that choose a kernel's shape. No HIP
// types appear here; device work goes through LayersDevice.
#pragma once

#include <cstdint>
#include <string>

#include "core.hpp"
#include "optim.hpp"

namespace ddpb {

// Elements a lane handles at a time, of any type: 16 bytes of a 16-bit type,
// and as many as one call of the generator has random bits for.
constexpr int64_t kGroup = 8;

// Rows of consecutive elements, `stride` elements from one to the next.
struct Matrix {
  const void* data = nullptr;
  int64_t stride = 0;
};

// What the kernels know of a dropout.
struct DropSpec {
  uint64_t seed = 0, offset = 0;
  const uint64_t* offset_device = nullptr;   // added to offset when the kernel runs
  uint32_t limit = 0;                        // of 65536: 16 random bits below it drop; 0: nothing is dropped
  float scale = 1.0f;                        // 65536 / (65536 - limit), or 0 where all is dropped
};

struct DropArgs {
  double p = 0.0;
  uint64_t seed = 0, offset = 0;
  const uint64_t* offset_device = nullptr;
};

struct NormForwardArgs {
  int64_t rows = 0, cols = 0;
  int32_t dtype = 0, weight_dtype = 0;
  Matrix x, residual;
  DropSpec drop;
  const void *weight = nullptr, *bias = nullptr;
  double eps = 0.0;
  void *y = nullptr, *h = nullptr;
  float* stats = nullptr;
  void* stream = nullptr;
};

struct NormBackwardArgs {
  int64_t rows = 0, cols = 0;
  int32_t dtype = 0, weight_dtype = 0, grad_dtype = 0;
  Matrix dy, h, grad_h;
  const float* stats = nullptr;
  DropSpec drop;
  const void* weight = nullptr;
  void *dh = nullptr, *dx = nullptr, *dweight = nullptr, *dbias = nullptr;
  bool accumulate = false;
  void* workspace = nullptr;
  int64_t ws_bytes = 0;
  void* stream = nullptr;
};

struct DropoutArgs {
  int64_t rows = 0, cols = 0;
  int32_t dtype = 0;
  Matrix x, residual;
  DropSpec drop;
  void* y = nullptr;
  void* stream = nullptr;
};

struct LookupArgs {
  int64_t n = 0, vocab = 0, cols = 0;
  const void* tokens = nullptr;
  int32_t token_bytes = 8;
  const void* table = nullptr;
  int32_t table_dtype = 0, dtype = 0;
  float scale = 1.0f;
  Matrix residual;
  void* y = nullptr;
  void* stream = nullptr;
};

struct LookupBackwardArgs {
  int64_t n = 0, vocab = 0, cols = 0;
  const void* tokens = nullptr;
  int32_t token_bytes = 8;
  Matrix dy;
  int32_t dtype = 0, grad_dtype = 0;
  float scale = 1.0f;
  void* dtable = nullptr;
  bool accumulate = false;
  void* workspace = nullptr;
  int64_t ws_bytes = 0;
  void* stream = nullptr;
};

// How a layer norm is cut: lanes of a row, groups of each lane. Rows up to 1024
// elements stay in one wave (no barrier), longer ones in a workgroup; a row that
// no shape holds in registers is read again for each of its passes (lanes = 0).
// The smallest shape that holds a row, against the next one, at and behind each
// border, in bf16 with 2^25 elements: the norm with a residual, its backward pass
// with the weights' gradients (us):
//     cols      taken              next
//      128   16 x 1   41,  37   64 x 1    75, 119
//      136   64 x 1   71, 115   64 x 2    91, 124
//      512   64 x 1   41,  41   64 x 2    43,  43
//      520   64 x 2   48,  50   256 x 1   61, 132
//     1024   64 x 2   42,  38   256 x 1   42,  73
//     1032   256 x 1  44,  74   256 x 2   56,  81
//     2048   256 x 1  41,  49   256 x 2   42,  53
//     2056   256 x 2  51,  58   512 x 2   60,  83
//     4096   256 x 2  42,  50   512 x 2   44,  55
//     4104   512 x 2  52,  58   1024 x 2  69,  85
//     8192   512 x 2  41,  53   1024 x 2  52,  69
//     8200   1024 x 2 54,  74   none      79, 473
//    16384   1024 x 2 42,  75   none      61, 257
// In fp32 (2^24 elements) the same are ahead, but for 1024 columns (forward 49, next
// 46), 2056 (52, 44) and 4096 (forward 47, 45; backward 45, 39).
struct NormShape {
  int lanes, groups;
};
NormShape norm_shape(int64_t cols);

// Workgroups of the backward pass, each of which leaves one partial sum of the
// weights' gradients: a function of the sizes only, so that the order of the
// sums does not depend on the device.
int32_t norm_backward_blocks(int64_t rows, int64_t cols);
// Few rows: one workgroup takes them and writes the gradients itself, without a
// workspace and a second launch (whose host time is more than its rows take).
bool norm_backward_alone(int64_t rows, int64_t cols);

// How the embedding's gradient is cut.
constexpr int kSortThreads = 1024;
constexpr int kSortKeys = 2;                                  // keys of a thread (131072 tokens, a pass: 12.2 us, 14.8 with 4)
constexpr int64_t kSortTile = kSortThreads * kSortKeys;       // keys of a workgroup
constexpr int64_t kRangeKeys = 16384;                         // most tokens of a sort in one launch
constexpr int kRanges = 32;                                   // workgroups of it
constexpr int kMaxDigit = 10;                                 // bits that one pass sorts by
constexpr int64_t kScanTiles = 64;                            // more tiles than this are scanned by a kernel of their own

struct LookupPlan {
  int passes, digit;        // passes of the sort, bits of each
  int64_t tiles;            // workgroups of the sort; 0: one launch by ranges of tokens
  int64_t unit, units;      // sorted places of a unit of the sum, units
  // byte offsets into the workspace
  int64_t keys[2], order[2], hist, totals, joins, list, partials, bytes;
};
LookupPlan lookup_plan(int64_t n, int64_t vocab, int64_t cols);

// Host checks; kOk, or an error with its reason.
int make_drop(const DropArgs* d, DropSpec* out, const char* what, std::string* err);
int check(const NormForwardArgs& a, std::string* err);
int check(const NormBackwardArgs& a, std::string* err);
int check(const DropoutArgs& a, std::string* err);
int check(const LookupArgs& a, std::string* err);
int check(const LookupBackwardArgs& a, std::string* err);
int64_t norm_backward_workspace(int64_t rows, int64_t cols);
bool norm_sizes_ok(int64_t rows, int64_t cols);
bool lookup_sizes_ok(int64_t n, int64_t vocab, int64_t cols);

// Enqueues checked calls on their stream, which belongs to the current device.
class LayersDevice {
 public:
  virtual ~LayersDevice() = default;
  virtual int norm_forward(const NormForwardArgs& a, std::string* err) = 0;
  virtual int norm_backward(const NormBackwardArgs& a, std::string* err) = 0;
  virtual int dropout(const DropoutArgs& a, std::string* err) = 0;
  virtual int lookup(const LookupArgs& a, std::string* err) = 0;
  virtual int lookup_backward(const LookupBackwardArgs& a, std::string* err) = 0;
};
LayersDevice* layers_device();

}  // namespace ddpb
