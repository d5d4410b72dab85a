// optim.cpp -- tile tables, checks and workspace layouts of the gradient norm
// and the AdamW step.
#include "optim.hpp"

#include <algorithm>
#include <cmath>
#include <cstring>
#include <utility>

namespace ddpb {
namespace {

int64_t up256(int64_t x) { return (x + 255) / 256 * 256; }


bool aligned(const void* p, int64_t a) { return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(a) == 0; }

uint64_t addr(const void* p) { return static_cast<uint64_t>(reinterpret_cast<uintptr_t>(p)); }

int check_workspace(void* ws, int64_t have, int64_t need, const char* what, std::string* err) {
  if (ws == nullptr || have < need) {
    *err = std::string(what) + ": workspace smaller than its workspace_bytes";
    return kErrArg;
  }
  if (!aligned(ws, 256)) {
    *err = std::string(what) + ": workspace must be 256-byte aligned";
    return kErrArg;
  }
  return kOk;
}

struct Range {
  uint64_t lo, hi;
  bool written;
};

// No memory that a step writes may be named twice: two tiles would update it
// in an unknown order (a tied parameter listed twice, a state shared by two
// parameters). Gradients are only read and may coincide with one another.
int check_overlap(std::vector<Range>* rs, std::string* err) {
  std::sort(rs->begin(), rs->end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
  uint64_t end = 0, written_end = 0;
  for (const Range& r : *rs) {
    if (r.lo < written_end || (r.written && r.lo < end)) {
      *err = "adamw bind: buffers overlap (each parameter, master, state and scale needs memory of its own)";
      return kErrArg;
    }
    end = std::max(end, r.hi);
    if (r.written) written_end = std::max(written_end, r.hi);
  }
  return kOk;
}

}  // namespace

int ReducerTie::check(const Reducer* red, const char* what, std::string* err) const {
  if (red == nullptr) return kOk;
  if (red->bind_id() != bind_id) {
    *err = std::string(what) + ": the reducer was bound again after this handle took its gradients; bind it again";
    return kErrState;
  }
  return red->check_idle(what, err);
}

namespace {

int tie_to(const Reducer* red, const char* what, ReducerTie* tie, std::string* err) {
  tie->bind_id = red != nullptr ? red->bind_id() : 0;
  if (red != nullptr && tie->bind_id == 0) {
    *err = std::string(what) + ": the reducer is not bound";
    return kErrState;
  }
  return kOk;
}

}  // namespace

// ---------------------------------------------------------------------------
// norm: [result, 256 bytes][counters][partial sums][tiles]

namespace {
constexpr int64_t kPartialsAt = 256 + (kArriveBytes + 255) / 256 * 256;
constexpr int64_t kNormTilesAt = kPartialsAt + (kNormBlocks * 8 + 255) / 256 * 256;
}

int64_t Norm::ntiles() const {
  int64_t n = 0;
  for (size_t v = 0; v < numel_.size(); ++v) {
    const int64_t tile = kNormTileBytes / dtype_size(dtypes_[v]);
    n += (numel_[v] + tile - 1) / tile;
  }
  return n;
}

int64_t Norm::workspace_bytes() const {
  return kNormTilesAt + up256(ntiles() * static_cast<int64_t>(sizeof(NormTile)));
}

int Norm::bind(void* const* grads, void* ws, int64_t ws_bytes, void* stream, const Reducer* red, std::string* err) {
  if (const int rc = check_workspace(ws, ws_bytes, workspace_bytes(), "norm bind", err); rc != kOk) return rc;
  if (ntiles() > INT32_MAX) {
    *err = "norm bind: too many elements";
    return kErrArg;
  }
  std::vector<char> h(static_cast<size_t>(workspace_bytes()), 0);
  NormTile* t = reinterpret_cast<NormTile*>(h.data() + kNormTilesAt);
  for (size_t v = 0; v < numel_.size(); ++v) {
    if (numel_[v] == 0) continue;
    if (grads[v] == nullptr || !aligned(grads[v], dtype_size(dtypes_[v]))) {
      *err = "norm bind: NULL or misaligned gradient pointer";
      return kErrArg;
    }
    const int64_t tile = kNormTileBytes / dtype_size(dtypes_[v]);
    for (int64_t s = 0; s < numel_[v]; s += tile)
      *t++ = NormTile{addr(grads[v]) + static_cast<uint64_t>(s * dtype_size(dtypes_[v])),
                      static_cast<int32_t>(std::min(tile, numel_[v] - s)), dtypes_[v]};
  }
  NormLaunch l{};
  l.stream = stream;
  if (const int rc = optim_device()->current(&l.device, err); rc != kOk) return rc;
  char* base = static_cast<char*>(ws);
  l.result = reinterpret_cast<NormResult*>(base);
  l.arrived = reinterpret_cast<uint32_t*>(base + 256);
  l.partials = reinterpret_cast<double*>(base + kPartialsAt);
  l.tiles = reinterpret_cast<const NormTile*>(base + kNormTilesAt);
  l.ntiles = static_cast<int32_t>(ntiles());
  reinterpret_cast<NormResult*>(h.data())->coef = 1.0f;
  ReducerTie tie;
  if (const int rc = tie_to(red, "norm bind", &tie, err); rc != kOk) return rc;
  bound_ = false;
  if (const int rc = optim_device()->upload(l.device, stream, ws, h.data(), h.size(), err); rc != kOk) return rc;
  l_ = l;
  tie_ = tie;
  bound_ = true;
  return kOk;
}

int Norm::compute(const Reducer* red, double max_norm, double grad_scale, bool skip_nonfinite, std::string* err) {
  if (!bound_) {
    *err = "norm compute: not bound";
    return kErrState;
  }
  if (!(max_norm > 0) || !std::isfinite(grad_scale)) {
    *err = "norm compute: max_norm must be positive and grad_scale finite";
    return kErrArg;
  }
  if (const int rc = tie_.check(red, "norm compute", err); rc != kOk) return rc;
  NormLaunch l = l_;
  l.max_norm = max_norm;
  l.grad_scale = grad_scale;
  l.skip_nonfinite = skip_nonfinite ? 1 : 0;
  return optim_device()->norm(l, err);
}

// ---------------------------------------------------------------------------
// AdamW: [scalars, neutral norm result, 256 bytes][counters][tiles][variables][replica pointers]
// There is always a tile and a variable: empty ones for a step of nothing.

namespace {
constexpr int64_t kNeutralAt = 64;

// Counts of steps that leave room to count on.
bool step_ok(int64_t done) { return done >= 0 && done <= (int64_t(1) << 53); }
constexpr int64_t kTilesAt = 256 + (kArriveBytes + 255) / 256 * 256;
}

int64_t Adamw::whole() const {
  int64_t n = 0;
  for (int64_t k : c_.numel) n += k / kOptimTile;
  return n;
}

int64_t Adamw::rests() const {
  const int64_t part = adamw_part(c_.param_dtype, c_.master, c_.f8);
  int64_t n = 0;
  for (int64_t k : c_.numel) n += (k % kOptimTile + part - 1) / part;
  return n;
}

int64_t Adamw::vars_at() const {
  return kTilesAt + up256(std::max<int64_t>(whole() + rests(), 1) * static_cast<int64_t>(sizeof(AdamwTile)));
}

int64_t Adamw::replicas_at() const {
  return vars_at() + up256(static_cast<int64_t>(std::max<size_t>(c_.numel.size(), 1) * sizeof(AdamwVar)));
}

int64_t Adamw::workspace_bytes() const {
  return replicas_at() + up256(static_cast<int64_t>(c_.R - 1) * static_cast<int64_t>(c_.numel.size()) * 8);
}

int Adamw::bind(const AdamwBuffers& b, int64_t done, void* ws, int64_t ws_bytes, void* stream, const Reducer* red,
                std::string* err) {
  const int64_t part = adamw_part(c_.param_dtype, c_.master, c_.f8);
  const int64_t groups = whole() * (kOptimTile / part) + rests();
  if (groups > kMaxThreads / adamw_threads(c_.f8)) {
    *err = "adamw bind: one launch takes " + std::to_string(kMaxThreads / adamw_threads(c_.f8)) + " workgroups of " +
           std::to_string(part) + " elements, this needs " + std::to_string(groups) +
           "; split the variables over several handles";
    return kErrArg;
  }
  if (const int rc = check_workspace(ws, ws_bytes, workspace_bytes(), "adamw bind", err); rc != kOk) return rc;
  if (!step_ok(done)) {
    *err = "adamw bind: step out of range";
    return kErrArg;
  }
  const size_t P = c_.numel.size();
  const int64_t ps = dtype_size(c_.param_dtype), gs = dtype_size(c_.grad_dtype), ss = c_.f8 ? 1 : 4;
  std::vector<char> h(static_cast<size_t>(workspace_bytes()), 0);
  AdamwTile* t = reinterpret_cast<AdamwTile*>(h.data() + kTilesAt);
  AdamwTile* rest = t + whole();
  AdamwVar* vars = reinterpret_cast<AdamwVar*>(h.data() + vars_at());
  uint64_t* rep = reinterpret_cast<uint64_t*>(h.data() + replicas_at());
  std::vector<Range> ranges;
  ranges.reserve(P * static_cast<size_t>(c_.R + 7) + 1);
  ranges.push_back(Range{addr(ws), addr(ws) + static_cast<uint64_t>(workspace_bytes()), true});
  uint64_t base = 0;                     // of the random bits: every variable starts a new block
  for (size_t v = 0; v < P; ++v) {
    const int64_t n = c_.numel[v];
    if (n == 0) continue;
    const int64_t blocks = (n + int64_t(kStateBlock) - 1) / int64_t(kStateBlock);
    bool ok = true;
    auto take = [&](const void* p, int64_t size, int64_t bytes, bool written) {
      ok = ok && p != nullptr && aligned(p, size);
      ranges.push_back(Range{addr(p), addr(p) + static_cast<uint64_t>(bytes), written});
    };
    for (int32_t r = 0; r < c_.R; ++r) {
      void* p = b.params[static_cast<size_t>(r) * P + v];
      take(p, ps, n * ps, true);
      if (r > 0) rep[static_cast<size_t>(r - 1) * P + v] = addr(p);
    }
    take(b.grads[v], gs, n * gs, false);
    if (c_.master) take(b.master[v], 4, n * 4, true);
    take(b.avg[v], ss, n * ss, true);
    take(b.second[v], ss, n * ss, true);
    if (c_.f8) {
      take(b.avg_scale[v], 1, blocks, true);
      take(b.root_scale[v], 1, blocks, true);
    }
    if (!ok) {
      *err = "adamw bind: NULL or misaligned pointer";
      return kErrArg;
    }
    AdamwVar& x = vars[v];
    x.out = addr(b.params[v]);
    x.src = c_.master ? addr(b.master[v]) : x.out;
    x.grad = addr(b.grads[v]);
    x.avg = addr(b.avg[v]);
    x.second = addr(b.second[v]);
    if (c_.f8) {
      x.avg_scale = addr(b.avg_scale[v]);
      x.root_scale = addr(b.root_scale[v]);
    }
    x.group0 = base / 4;
    x.weight_decay = c_.weight_decay.empty() ? 0.0 : c_.weight_decay[v];
    x.lr_scale = c_.lr_scale.empty() ? 1.0 : c_.lr_scale[v];
    int64_t s = 0;
    for (; s + kOptimTile <= n; s += kOptimTile)
      *t++ = AdamwTile{static_cast<int32_t>(v), static_cast<int32_t>(kOptimTile), s};
    for (; s < n; s += part)
      *rest++ = AdamwTile{static_cast<int32_t>(v), static_cast<int32_t>(std::min(part, n - s)), s};
    base += static_cast<uint64_t>(blocks * kStateBlock);
  }
  if (const int rc = check_overlap(&ranges, err); rc != kOk) return rc;
  AdamwLaunch l{};
  l.stream = stream;
  if (const int rc = optim_device()->current(&l.device, err); rc != kOk) return rc;
  const StepScalars sc = step_scalars(done, c_.beta1, c_.beta2, c_.seed);
  std::memcpy(h.data(), &sc, sizeof(sc));
  reinterpret_cast<NormResult*>(h.data() + kNeutralAt)->coef = 1.0f;
  char* dev = static_cast<char*>(ws);
  l.param_dtype = c_.param_dtype;
  l.grad_dtype = c_.grad_dtype;
  l.f8 = c_.f8 ? 1 : 0;
  l.master = c_.master ? 1 : 0;
  l.scalars = reinterpret_cast<StepScalars*>(dev);
  l.neutral = reinterpret_cast<const NormResult*>(dev + kNeutralAt);
  l.arrived = reinterpret_cast<uint32_t*>(dev + 256);
  l.tiles = reinterpret_cast<const AdamwTile*>(dev + kTilesAt);
  l.vars = reinterpret_cast<const AdamwVar*>(dev + vars_at());
  l.whole = static_cast<int32_t>(whole());
  l.rests = static_cast<int32_t>(rests());
  l.replicas = reinterpret_cast<const uint64_t*>(dev + replicas_at());
  l.R = c_.R;
  l.P = static_cast<int32_t>(P);
  l.beta1 = c_.beta1;
  l.beta2 = c_.beta2;
  l.eps = c_.eps;
  l.seed = c_.seed;
  ReducerTie tie;
  if (const int rc = tie_to(red, "adamw bind", &tie, err); rc != kOk) return rc;
  bound_ = false;
  if (const int rc = optim_device()->upload(l.device, stream, ws, h.data(), h.size(), err); rc != kOk) return rc;
  l_ = l;
  tie_ = tie;
  bound_ = true;
  return kOk;
}

int Adamw::step(const Reducer* red, double lr, const float* lr_device, double grad_scale, const void* clip,
                std::string* err) {
  if (!bound_) {
    *err = "adamw step: not bound";
    return kErrState;
  }
  if (!std::isfinite(lr) || lr < 0 || !std::isfinite(static_cast<float>(grad_scale))) {
    *err = "adamw step: lr must be finite and not negative, grad_scale finite in fp32";
    return kErrArg;
  }
  if (!aligned(lr_device, 4) || !aligned(clip, 4)) {
    *err = "adamw step: misaligned lr or norm result";
    return kErrArg;
  }
  if (const int rc = tie_.check(red, "adamw step", err); rc != kOk) return rc;
  AdamwLaunch l = l_;
  l.lr = lr;
  l.lr_device = lr_device;
  l.grad_scale = grad_scale;
  l.clip = static_cast<const NormResult*>(clip);
  return optim_device()->adamw(l, err);
}

int Adamw::set_step(int64_t done, std::string* err) {
  if (!bound_) {
    *err = "adamw set_step: not bound";
    return kErrState;
  }
  if (!step_ok(done)) {
    *err = "adamw set_step: step out of range";
    return kErrArg;
  }
  const StepScalars sc = step_scalars(done, c_.beta1, c_.beta2, c_.seed);
  return optim_device()->upload(l_.device, l_.stream, l_.scalars, &sc, sizeof(sc), err);
}

int Adamw::get_step(int64_t* done, std::string* err) {
  if (!bound_) {
    *err = "adamw get_step: not bound";
    return kErrState;
  }
  StepScalars sc{};
  if (const int rc = optim_device()->download(l_.device, l_.stream, &sc, l_.scalars, sizeof(sc), err); rc != kOk)
    return rc;
  *done = sc.done;
  return kOk;
}

}  // namespace ddpb
