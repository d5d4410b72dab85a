// layers.cpp -- checks, shapes and workspace layouts of layer norm, dropout and
// the embedding.
#include "layers.hpp"

#include <algorithm>
#include <cmath>

namespace ddpb {
namespace {

constexpr int64_t kMaxElems = int64_t(1) << 40;
constexpr int64_t kMaxCols = int64_t(1) << 20;
constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxSplitCols = int64_t(1) << 33;   // their groups are counted in 32 bits
constexpr int64_t kMaxTokens = int64_t(1) << 30;

int64_t up256(int64_t x) { return (x + 255) / 256 * 256; }
uint64_t addr(const void* p) { return static_cast<uint64_t>(reinterpret_cast<uintptr_t>(p)); }
bool aligned(const void* p, int64_t a) { return addr(p) % static_cast<uint64_t>(a) == 0; }

int fail(std::string* err, const char* what, const char* why) {
  *err = std::string(what) + ": " + why;
  return kErrArg;
}

struct Span {
  uint64_t lo = 0, hi = 0;
};
Span span(const void* p, int64_t bytes) { return {addr(p), addr(p) + static_cast<uint64_t>(bytes)}; }
Span span(const Matrix& m, int64_t rows, int64_t cols, int64_t size) {
  return m.data == nullptr || rows == 0 ? Span{} : span(m.data, ((rows - 1) * m.stride + cols) * size);
}
bool meet(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }

// An input of rows: an address aligned to its type, a stride that stays in range.
bool matrix_ok(const Matrix& m, int64_t rows, int64_t size, bool needed) {
  if (m.data == nullptr) return !needed || rows == 0;
  return aligned(m.data, size) && (rows <= 1 || (m.stride >= 0 && m.stride <= kMaxElems / rows));
}

// An output or plain array: not NULL unless empty, aligned to its type.
bool array_ok(const void* p, int64_t elems, int64_t size) {
  return elems == 0 || (p != nullptr && aligned(p, size));
}

// No output may touch an input or another output.
template <size_t O, size_t I>
bool apart(const Span (&out)[O], const Span (&in)[I]) {
  for (size_t o = 0; o < O; ++o) {
    for (const Span& i : in)
      if (meet(out[o], i)) return false;
    for (size_t q = 0; q < o; ++q)
      if (meet(out[o], out[q])) return false;
  }
  return true;
}

}  // namespace

int make_drop(const DropArgs* d, DropSpec* out, const char* what, std::string* err) {
  *out = DropSpec();
  if (d == nullptr) return kOk;
  if (!(d->p >= 0.0 && d->p <= 1.0)) return fail(err, what, "p must be in [0, 1]");
  if (!aligned(d->offset_device, 8)) return fail(err, what, "the offset in device memory must be 8-byte aligned");
  out->limit = static_cast<uint32_t>(std::lround(d->p * 65536.0));
  out->scale = out->limit < 65536 ? static_cast<float>(65536.0 / (65536.0 - out->limit)) : 0.0f;
  out->seed = d->seed;
  out->offset = d->offset;
  out->offset_device = d->offset_device;
  return kOk;
}

NormShape norm_shape(int64_t cols) {
  if (cols <= 16 * kGroup) return {16, 1};
  if (cols <= 64 * kGroup) return {64, 1};
  if (cols <= 128 * kGroup) return {64, 2};
  if (cols <= 256 * kGroup) return {256, 1};
  if (cols <= 512 * kGroup) return {256, 2};
  if (cols <= 1024 * kGroup) return {512, 2};
  if (cols <= 2048 * kGroup) return {1024, 2};
  return {0, 0};
}

namespace {
// Rows that a workgroup of the backward pass takes at once.
int64_t rows_at_once(NormShape s) { return s.lanes == 0 || s.lanes > 64 ? 1 : 512 / s.lanes; }
}  // namespace

bool norm_backward_alone(int64_t rows, int64_t cols) {
  const NormShape s = norm_shape(cols);
  return s.lanes != 0 && rows > 0 && rows <= 4 * rows_at_once(s);
}

int32_t norm_backward_blocks(int64_t rows, int64_t cols) {
  if (norm_backward_alone(rows, cols)) return 1;
  const NormShape s = norm_shape(cols);
  // workgroups that leave a partial sum: eight waves a CU
  int64_t most = s.lanes == 256 ? 512 : 256;
  if (s.lanes == 0) most = std::max<int64_t>(32, std::min<int64_t>(256, (int64_t(64) << 20) / (8 * cols)));
  const int64_t need = (rows + rows_at_once(s) - 1) / rows_at_once(s);
  return static_cast<int32_t>(std::max<int64_t>(1, std::min(most, need)));
}

bool norm_sizes_ok(int64_t rows, int64_t cols) {
  return rows >= 0 && rows <= kMaxRows && cols >= 1 && cols <= kMaxCols && (rows == 0 || cols <= kMaxElems / rows);
}

int64_t norm_backward_workspace(int64_t rows, int64_t cols) {
  if (rows == 0 || norm_backward_alone(rows, cols)) return 0;
  return up256(static_cast<int64_t>(norm_backward_blocks(rows, cols)) * 2 * cols * 4);
}

int check(const NormForwardArgs& a, std::string* err) {
  const char* what = "layer_norm";
  const int64_t size = dtype_size(a.dtype);
  if (!norm_sizes_ok(a.rows, a.cols)) return fail(err, what, "rows must be in 0..2^31 - 1, cols in 1..2^20");
  const int64_t n = a.rows * a.cols;
  if (!(a.eps >= 0.0) || !std::isfinite(static_cast<float>(a.eps))) return fail(err, what, "eps must be finite and not negative");
  if (!matrix_ok(a.x, a.rows, size, true) || !matrix_ok(a.residual, a.rows, size, false))
    return fail(err, what, "NULL, misaligned or too widely spread input");
  const int64_t ws = dtype_size(a.weight_dtype);
  if (!aligned(a.weight, ws) || !aligned(a.bias, ws)) return fail(err, what, "misaligned weight or bias");
  const bool fused = a.residual.data != nullptr || a.drop.limit != 0;
  if (!array_ok(a.y, n, size) || !array_ok(a.stats, a.rows, 4) || (a.h != nullptr && !array_ok(a.h, n, size)))
    return fail(err, what, "NULL or misaligned output");
  if (a.h != nullptr && !fused) return fail(err, what, "h is x where there is neither a residual nor a dropout: pass NULL");
  const Span out[] = {span(a.y, n * size), a.h != nullptr ? span(a.h, n * size) : Span{}, span(a.stats, a.rows * 8)};
  const Span in[] = {span(a.x, a.rows, a.cols, size), span(a.residual, a.rows, a.cols, size),
                     a.weight != nullptr ? span(a.weight, a.cols * ws) : Span{},
                     a.bias != nullptr ? span(a.bias, a.cols * ws) : Span{}};
  if (n > 0 && !apart(out, in)) return fail(err, what, "an output overlaps an input or another output");
  return kOk;
}

int check(const NormBackwardArgs& a, std::string* err) {
  const char* what = "layer_norm_backward";
  const int64_t size = dtype_size(a.dtype), ws = dtype_size(a.weight_dtype), gs = dtype_size(a.grad_dtype);
  if (!norm_sizes_ok(a.rows, a.cols)) return fail(err, what, "rows must be in 0..2^31 - 1, cols in 1..2^20");
  if (!matrix_ok(a.dy, a.rows, size, true) || !matrix_ok(a.h, a.rows, size, true) ||
      !matrix_ok(a.grad_h, a.rows, size, false) || !array_ok(a.stats, a.rows, 4))
    return fail(err, what, "NULL, misaligned or too widely spread input");
  if (!aligned(a.weight, ws)) return fail(err, what, "misaligned weight");
  const int64_t n = a.rows * a.cols;
  if (!array_ok(a.dh, n, size) || (a.dx != nullptr && !array_ok(a.dx, n, size)) || !aligned(a.dweight, gs) ||
      !aligned(a.dbias, gs))
    return fail(err, what, "NULL or misaligned output");
  if ((a.dx != nullptr) != (a.drop.limit != 0) && n > 0)
    return fail(err, what, "dx goes with a dropout: without one dh is the gradient of x");
  const bool weights = a.dweight != nullptr || a.dbias != nullptr;
  const int64_t need = weights ? norm_backward_workspace(a.rows, a.cols) : 0;
  if (need > 0 && (a.workspace == nullptr || a.ws_bytes < need || !aligned(a.workspace, 256)))
    return fail(err, what, "workspace smaller than its workspace_bytes, or not 256-byte aligned");
  const Span out[] = {span(a.dh, n * size), a.dx != nullptr ? span(a.dx, n * size) : Span{},
                      a.dweight != nullptr ? span(a.dweight, a.cols * gs) : Span{},
                      a.dbias != nullptr ? span(a.dbias, a.cols * gs) : Span{},
                      need > 0 ? span(a.workspace, need) : Span{}};
  const Span in[] = {span(a.dy, a.rows, a.cols, size), span(a.h, a.rows, a.cols, size),
                     span(a.grad_h, a.rows, a.cols, size), a.rows > 0 ? span(a.stats, a.rows * 8) : Span{},
                     a.weight != nullptr ? span(a.weight, a.cols * ws) : Span{}};
  if (!apart(out, in)) return fail(err, what, "an output overlaps an input or another output");
  return kOk;
}

int check(const DropoutArgs& a, std::string* err) {
  const char* what = "dropout";
  const int64_t size = dtype_size(a.dtype);
  if (a.rows < 0 || a.cols < 0 || a.rows > kMaxElems || a.cols > kMaxElems ||
      (a.rows > 0 && a.cols > kMaxElems / a.rows))
    return fail(err, what, "rows and cols must not be negative, rows * cols at most 2^40");
  const int64_t n = a.rows * a.cols;
  if (n == 0) return kOk;
  if (!matrix_ok(a.x, a.rows, size, true) || !matrix_ok(a.residual, a.rows, size, false))
    return fail(err, what, "NULL, misaligned or too widely spread input");
  if (!array_ok(a.y, n, size)) return fail(err, what, "NULL or misaligned output");
  const bool flat = a.x.stride == a.cols && (a.residual.data == nullptr || a.residual.stride == a.cols);
  if (a.rows > 1 && !flat && a.cols > kMaxSplitCols) return fail(err, what, "rows of more than 2^33 elements must be contiguous");
  // In place is fine: an element is read by the lane that writes it, before.
  const Span y = span(a.y, n * size);
  for (const Matrix* m : {&a.x, &a.residual}) {
    const bool same = m->data == a.y && (m->stride == a.cols || a.rows == 1);
    if (m->data != nullptr && !same && meet(y, span(*m, a.rows, a.cols, size)))
      return fail(err, what, "y overlaps an input without being it");
  }
  return kOk;
}

bool lookup_sizes_ok(int64_t n, int64_t vocab, int64_t cols) {
  return n >= 0 && n <= kMaxTokens && vocab >= 0 && vocab <= kMaxRows - 1 && cols >= 1 && cols <= kMaxCols &&
         (n == 0 || cols <= kMaxElems / n) && (vocab == 0 || cols <= kMaxElems / vocab);
}

int check(const LookupArgs& a, std::string* err) {
  const char* what = "embedding";
  const int64_t size = dtype_size(a.dtype), ts = dtype_size(a.table_dtype);
  if (!lookup_sizes_ok(a.n, a.vocab, a.cols))
    return fail(err, what, "tokens must be 0..2^30, the table 0..2^31 - 2 rows of 1..2^20");
  if (!std::isfinite(a.scale)) return fail(err, what, "scale must be finite in fp32");
  if (!array_ok(a.tokens, a.n, a.token_bytes) || !array_ok(a.table, a.vocab, ts) ||
      !matrix_ok(a.residual, a.n, size, false))
    return fail(err, what, "NULL, misaligned or too widely spread input");
  if (!array_ok(a.y, a.n, size)) return fail(err, what, "NULL or misaligned output");
  const Span out[] = {span(a.y, a.n * a.cols * size)};
  const Span in[] = {span(a.tokens, a.n * a.token_bytes), span(a.table, a.vocab * a.cols * ts),
                     span(a.residual, a.n, a.cols, size)};
  if (a.n > 0 && !apart(out, in)) return fail(err, what, "y overlaps an input");
  return kOk;
}

LookupPlan lookup_plan(int64_t n, int64_t vocab, int64_t cols) {
  LookupPlan p{};
  int bits = 1;                                      // a token is 0..vocab, vocab standing for all others
  while ((int64_t(1) << bits) <= vocab) ++bits;
  if (n <= kRangeKeys) {                             // t / kRanges, six bits a pass
    p.passes = (std::max(bits - 5, 1) + 5) / 6;
    p.digit = 6;
  } else {
    p.passes = (bits + kMaxDigit - 1) / kMaxDigit;
    p.digit = (bits + p.passes - 1) / p.passes;
    p.tiles = (n + kSortTile - 1) / kSortTile;
  }
  // Units of 8 places or more, so that 1024 waves (four a CU) share the sum; at
  // most 65536 units, which bounds the partial sums.
  const int64_t waves = (cols + 64 * kGroup - 1) / (64 * kGroup);
  p.unit = 8;
  while (p.unit < 128 && n * waves > p.unit * 1024) p.unit *= 2;
  while (n > p.unit * 65536) p.unit *= 2;
  p.units = (n + p.unit - 1) / p.unit;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += up256(bytes);
    return here;
  };
  for (int i = 0; i < 2; ++i) {
    p.keys[i] = take(n * 4);
    p.order[i] = take(n * 4);
  }
  p.hist = take((p.tiles << p.digit) * 4);
  p.totals = take(int64_t(4) << p.digit);
  p.joins = take(4);
  p.list = take(p.units * 8);
  p.partials = take(p.units > 1 ? p.units * 2 * cols * 4 : 0);
  p.bytes = at;
  return p;
}

int check(const LookupBackwardArgs& a, std::string* err) {
  const char* what = "embedding_backward";
  const int64_t size = dtype_size(a.dtype), gs = dtype_size(a.grad_dtype);
  if (!lookup_sizes_ok(a.n, a.vocab, a.cols))
    return fail(err, what, "tokens must be 0..2^30, the table 0..2^31 - 2 rows of 1..2^20");
  if (!std::isfinite(a.scale)) return fail(err, what, "scale must be finite in fp32");
  if (!array_ok(a.tokens, a.n, a.token_bytes) || !matrix_ok(a.dy, a.n, size, true))
    return fail(err, what, "NULL, misaligned or too widely spread input");
  if (!array_ok(a.dtable, a.vocab, gs)) return fail(err, what, "NULL or misaligned output");
  const int64_t need = lookup_plan(a.n, a.vocab, a.cols).bytes;
  if (a.workspace == nullptr || a.ws_bytes < need || !aligned(a.workspace, 256))
    return fail(err, what, "workspace smaller than its workspace_bytes, or not 256-byte aligned");
  const Span out[] = {span(a.dtable, a.vocab * a.cols * gs), span(a.workspace, need)};
  const Span in[] = {span(a.tokens, a.n * a.token_bytes), span(a.dy, a.n, a.cols, size)};
  if (!apart(out, in)) return fail(err, what, "an output overlaps an input or another output");
  return kOk;
}

}  // namespace ddpb
