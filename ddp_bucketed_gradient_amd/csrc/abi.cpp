// abi.cpp -- the extern "C" surface declared in include/ddpb.h. Argument
// checking and marshalling only; the work happens in plan.cpp, core.cpp and the
// launcher.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <string>
#include <vector>

#include "../../include/ddpb.h"
#include "core.hpp"
#include "layers.hpp"
#include "optim.hpp"

struct ddpb_reducer {
  explicit ddpb_reducer(ddpb::Plan p) : red(std::move(p)) {}
  ddpb::Reducer red;
};

struct ddpb_norm {
  ddpb_norm(std::vector<int64_t> numel, std::vector<int32_t> dtypes) : norm(std::move(numel), std::move(dtypes)) {}
  ddpb::Norm norm;
  int32_t P = 0;
};

struct ddpb_adamw {
  explicit ddpb_adamw(ddpb::AdamwConfig c) : opt(std::move(c)) {}
  ddpb::Adamw opt;
};

namespace {
thread_local std::string g_err;

int fail(int code, const std::string& msg) {
  g_err = msg;
  return code;
}

int pass(int code, const std::string& msg) {
  if (code != 0) g_err = msg;
  return code;
}

bool is_dtype(int32_t d) { return d == DDPB_F32 || d == DDPB_BF16 || d == DDPB_F16; }

const ddpb::Reducer* reducer_of(ddpb_t h) { return h != nullptr ? &h->red : nullptr; }

// Element counts whose tables and addresses stay in range.
bool numels_ok(const int64_t* numel, int32_t P) {
  int64_t total = 0;
  for (int32_t v = 0; v < P; ++v) {
    if (numel[v] < 0 || numel[v] > (int64_t(1) << 40) || (total += numel[v]) > (int64_t(1) << 40)) return false;
  }
  return true;
}

// A call that may allocate host memory: no C++ exception crosses the ABI.
template <typename F>
int guarded(const char* what, F f) {
  try {
    std::string err;
    const int rc = f(&err);
    return rc == DDPB_OK ? rc : fail(rc, err);
  } catch (const std::exception&) {
    return fail(DDPB_E_NOMEM, std::string(what) + ": out of host memory");
  }
}

// Builds the kernels' arguments, checks them and enqueues the call (if there is one).
template <typename Args, typename Fill>
int enqueue(const char* what, int (ddpb::LayersDevice::*call)(const Args&, std::string*), Fill fill) {
  return guarded(what, [&](std::string* err) {
    Args a;
    int rc = fill(&a, err);
    if (rc == DDPB_OK) rc = ddpb::check(a, err);
    return rc == DDPB_OK && call != nullptr ? (ddpb::layers_device()->*call)(a, err) : rc;
  });
}

int drop_of(const ddpb_drop* d, ddpb::DropSpec* out, const char* what, std::string* err) {
  if (d == nullptr) return DDPB_OK;
  const ddpb::DropArgs a{d->p, d->seed, d->offset, d->offset_device};
  return ddpb::make_drop(&a, out, what, err);
}

typedef int (ddpb::LayersDevice::*NormBackwardCall)(const ddpb::NormBackwardArgs&, std::string*);
typedef int (ddpb::LayersDevice::*LookupBackwardCall)(const ddpb::LookupBackwardArgs&, std::string*);

int norm_backward(NormBackwardCall call, int64_t rows, int64_t cols, int32_t dtype, ddpb::Matrix dy, ddpb::Matrix h,
                  const float* stats, ddpb::Matrix grad_h, const ddpb_drop* drop, const void* weight,
                  int32_t weight_dtype, void* dh, void* dx, void* dweight, void* dbias, int32_t grad_dtype,
                  int32_t accumulate, void* workspace, int64_t ws_bytes, void* stream) {
  if (!is_dtype(dtype) || !is_dtype(weight_dtype) || !is_dtype(grad_dtype))
    return fail(DDPB_E_ARG, "layer_norm_backward: bad dtype");
  return enqueue("layer_norm_backward", call, [&](ddpb::NormBackwardArgs* a, std::string* err) {
    a->rows = rows;
    a->cols = cols;
    a->dtype = dtype;
    a->weight_dtype = weight_dtype;
    a->grad_dtype = grad_dtype;
    a->dy = dy;
    a->h = h;
    a->grad_h = grad_h;
    a->stats = stats;
    a->weight = weight;
    a->dh = dh;
    a->dx = dx;
    a->dweight = dweight;
    a->dbias = dbias;
    a->accumulate = accumulate != 0;
    a->workspace = workspace;
    a->ws_bytes = ws_bytes;
    a->stream = stream;
    return drop_of(drop, &a->drop, "layer_norm_backward", err);
  });
}

int embedding_backward(LookupBackwardCall call, int64_t n, const void* tokens, int32_t token_bytes, int64_t vocab,
                       int64_t cols, ddpb::Matrix dy, int32_t dtype, double scale, void* dtable, int32_t grad_dtype,
                       int32_t accumulate, void* workspace, int64_t ws_bytes, void* stream) {
  if (!is_dtype(dtype) || !is_dtype(grad_dtype) || (token_bytes != 4 && token_bytes != 8))
    return fail(DDPB_E_ARG, "embedding_backward: bad dtype or token_bytes");
  return enqueue("embedding_backward", call, [&](ddpb::LookupBackwardArgs* a, std::string*) {
    a->n = n;
    a->vocab = vocab;
    a->cols = cols;
    a->tokens = tokens;
    a->token_bytes = token_bytes;
    a->dy = dy;
    a->dtype = dtype;
    a->grad_dtype = grad_dtype;
    a->scale = static_cast<float>(scale);
    a->dtable = dtable;
    a->accumulate = accumulate != 0;
    a->workspace = workspace;
    a->ws_bytes = ws_bytes;
    a->stream = stream;
    return DDPB_OK;
  });
}
}  // namespace

extern "C" {

const char* ddpb_last_error(void) { return g_err.c_str(); }

int ddpb_reducer_create(const int64_t* shapes, const int32_t* ndims, int32_t P, int32_t dtype,
                        int64_t bucket_cap_bytes, int32_t R, ddpb_t* out) {
  if (out == nullptr) return fail(DDPB_E_ARG, "create: out is NULL");
  *out = nullptr;
  if (P < 0 || (P > 0 && ndims == nullptr)) return fail(DDPB_E_ARG, "create: bad P or ndims");
  if (dtype != DDPB_F32) return fail(DDPB_E_ARG, "create: only fp32 gradients are supported");
  if (bucket_cap_bytes < 0) return fail(DDPB_E_ARG, "create: negative bucket cap");
  if (R < 1 || R > ddpb::kMaxReplicas) return fail(DDPB_E_ARG, "create: R must be in 1..64");
  std::vector<int64_t> numel(P);
  int64_t k = 0;
  for (int32_t v = 0; v < P; ++v) {
    if (ndims[v] < 0 || ndims[v] > 16) return fail(DDPB_E_ARG, "create: bad ndims");
    if (ndims[v] > 0 && shapes == nullptr) return fail(DDPB_E_ARG, "create: shapes is NULL");
    int64_t n = 1;
    for (int32_t d = 0; d < ndims[v]; ++d) {
      const int64_t s = shapes[k++];
      if (s < 0) return fail(DDPB_E_ARG, "create: negative dimension");
      if (s != 0 && n > (int64_t(1) << 50) / s) return fail(DDPB_E_ARG, "create: tensor too large");
      n *= s;
    }
    numel[v] = n;
  }
  try {
    *out = new ddpb_reducer(ddpb::make_plan(numel, 4, bucket_cap_bytes, R));
  } catch (const std::bad_alloc&) {
    return fail(DDPB_E_NOMEM, "create: out of host memory");
  }
  return DDPB_OK;
}

void ddpb_destroy(ddpb_t h) { delete h; }

int ddpb_num_buckets(ddpb_t h, int32_t* B) {
  if (!h || !B) return fail(DDPB_E_ARG, "num_buckets: NULL argument");
  *B = h->red.plan().B();
  return DDPB_OK;
}

int ddpb_get_locator(ddpb_t h, int32_t v, int32_t* bucket, int32_t* intra, int64_t* offset,
                     int64_t* length) {
  if (!h) return fail(DDPB_E_ARG, "get_locator: NULL handle");
  const ddpb::Plan& p = h->red.plan();
  if (v < 0 || v >= p.P) return fail(DDPB_E_INDEX, "get_locator: variable index out of range");
  const ddpb::Locator& L = p.loc[v];
  if (bucket) *bucket = L.bucket;
  if (intra) *intra = L.intra;
  if (offset) *offset = L.offset;
  if (length) *length = L.length;
  return DDPB_OK;
}

int ddpb_get_bucket(ddpb_t h, int32_t b, int32_t* nvars, int64_t* bytes, int32_t* vars) {
  if (!h) return fail(DDPB_E_ARG, "get_bucket: NULL handle");
  const ddpb::Plan& p = h->red.plan();
  if (b < 0 || b >= p.B()) return fail(DDPB_E_INDEX, "get_bucket: bucket index out of range");
  if (nvars) *nvars = static_cast<int32_t>(p.members[b].size());
  if (bytes) *bytes = p.bucket_elems[b] * p.elem_size;
  if (vars) std::memcpy(vars, p.members[b].data(), p.members[b].size() * sizeof(int32_t));
  return DDPB_OK;
}

int ddpb_num_segments(ddpb_t h, int32_t* n, int64_t* seg_elems) {
  if (!h) return fail(DDPB_E_ARG, "num_segments: NULL handle");
  if (n) *n = static_cast<int32_t>(h->red.plan().segs.size());
  if (seg_elems) *seg_elems = ddpb::kSegElems;
  return DDPB_OK;
}

int ddpb_get_bucket_segments(ddpb_t h, int32_t b, int32_t* first, int32_t* count) {
  if (!h) return fail(DDPB_E_ARG, "get_bucket_segments: NULL handle");
  const ddpb::Plan& p = h->red.plan();
  if (b < 0 || b >= p.B()) return fail(DDPB_E_INDEX, "get_bucket_segments: bucket index out of range");
  if (first) *first = p.seg_first[b];
  if (count) *count = p.seg_first[b + 1] - p.seg_first[b];
  return DDPB_OK;
}

int ddpb_get_segment(ddpb_t h, int32_t s, int32_t* var, int32_t* bucket, int64_t* start,
                     int64_t* length, int64_t* bucket_offset) {
  if (!h) return fail(DDPB_E_ARG, "get_segment: NULL handle");
  const ddpb::Plan& p = h->red.plan();
  if (s < 0 || s >= static_cast<int32_t>(p.segs.size()))
    return fail(DDPB_E_INDEX, "get_segment: segment index out of range");
  const ddpb::Segment& g = p.segs[s];
  if (var) *var = g.var;
  if (bucket) *bucket = p.seg_bucket[s];
  if (start) *start = g.start;
  if (length) *length = g.len;
  if (bucket_offset) *bucket_offset = g.boff;
  return DDPB_OK;
}

int ddpb_workspace_bytes(ddpb_t h, int32_t mode, int64_t* bytes) {
  if (!h || !bytes) return fail(DDPB_E_ARG, "workspace_bytes: NULL argument");
  if (mode != DDPB_MODE_FUSED && mode != DDPB_MODE_STAGED) return fail(DDPB_E_ARG, "workspace_bytes: bad mode");
  *bytes = ddpb::workspace_bytes(h->red.plan(), mode);
  return DDPB_OK;
}

int ddpb_bind(ddpb_t h, void* const* grad_ptrs, void* workspace, int64_t ws_bytes, void* compute_stream,
              void* const* side_streams, int32_t n_side, int32_t mode, int32_t flags) {
  if (!h) return fail(DDPB_E_ARG, "bind: NULL handle");
  const ddpb::Plan& p = h->red.plan();
  if (mode != DDPB_MODE_FUSED && mode != DDPB_MODE_STAGED) return fail(DDPB_E_ARG, "bind: bad mode");
  if (flags & ~(DDPB_BIND_DEVICE_TIMESTAMPS | DDPB_BIND_TIME_LAUNCHES | DDPB_BIND_ROCTX | DDPB_BIND_OVERLAP)) return fail(DDPB_E_ARG, "bind: bad flags");
  if (n_side < 1 || n_side > 16 || side_streams == nullptr) return fail(DDPB_E_ARG, "bind: need 1..16 side streams");
  const int64_t need = ddpb::workspace_bytes(p, mode);
  if (ws_bytes < need || (need > 0 && workspace == nullptr))
    return fail(DDPB_E_ARG, "bind: workspace smaller than ddpb_workspace_bytes");
  const size_t n = static_cast<size_t>(p.R) * p.P;
  if (n > 0 && grad_ptrs == nullptr) return fail(DDPB_E_ARG, "bind: grad_ptrs is NULL");
  ddpb::BindArgs a;
  a.grad_ptrs.assign(grad_ptrs, grad_ptrs + n);
  for (size_t i = 0; i < n; ++i)
    if (a.grad_ptrs[i] == nullptr && p.numel[i % p.P] > 0) return fail(DDPB_E_ARG, "bind: NULL gradient pointer");
  a.workspace = workspace;
  a.ws_bytes = ws_bytes;
  a.compute_stream = compute_stream;
  a.side_streams.assign(side_streams, side_streams + n_side);
  a.mode = mode;
  a.flags = flags;
  std::string err;
  return pass(h->red.bind(a, &err), err);
}

int ddpb_bind_static(ddpb_t h, void* const* grad_ptrs, void* compute_stream, int32_t mode) {
  if (!h) return fail(DDPB_E_ARG, "bind_static: NULL handle");
  const ddpb::Plan& p = h->red.plan();
  if (mode != DDPB_MODE_FUSED && mode != DDPB_MODE_STAGED) return fail(DDPB_E_ARG, "bind_static: bad mode");
  const size_t n = static_cast<size_t>(p.R) * p.P;
  if (n > 0 && grad_ptrs == nullptr) return fail(DDPB_E_ARG, "bind_static: grad_ptrs is NULL");
  ddpb::BindArgs a;
  a.grad_ptrs.assign(grad_ptrs, grad_ptrs + n);
  for (size_t i = 0; i < n; ++i)
    if (a.grad_ptrs[i] == nullptr && p.numel[i % p.P] > 0) return fail(DDPB_E_ARG, "bind_static: NULL gradient pointer");
  a.compute_stream = compute_stream;
  a.side_streams.assign(1, compute_stream);
  a.mode = mode;
  a.no_alloc = true;
  std::string err;
  return pass(h->red.bind(a, &err), err);
}

int ddpb_rebuild_buckets(ddpb_t h, int64_t bucket_cap_bytes) {
  if (!h) return fail(DDPB_E_ARG, "rebuild_buckets: NULL handle");
  std::string err;
  return pass(h->red.rebuild_buckets(bucket_cap_bytes, &err), err);
}

int ddpb_get_ready_order(ddpb_t h, int32_t* order, int32_t cap, int32_t* n) {
  if (!h || !n || cap < 0 || (cap > 0 && !order)) return fail(DDPB_E_ARG, "get_ready_order: bad argument");
  const auto& o = h->red.last_ready_order();
  *n = static_cast<int32_t>(o.size());
  for (int32_t i = 0; i < std::min<int32_t>(cap, *n); ++i) order[i] = o[i];
  return DDPB_OK;
}

int ddpb_view_storage_elems(ddpb_t h, int64_t* elems) {
  if (!h || !elems) return fail(DDPB_E_ARG, "view_storage_elems: NULL argument");
  *elems = h->red.plan().flat_elems;
  return DDPB_OK;
}

int ddpb_get_view_offset(ddpb_t h, int32_t v, int64_t* offset) {
  if (!h || !offset) return fail(DDPB_E_ARG, "get_view_offset: NULL argument");
  const ddpb::Plan& p = h->red.plan();
  if (v < 0 || v >= p.P) return fail(DDPB_E_INDEX, "get_view_offset: variable index out of range");
  *offset = p.view_offset(v);
  return DDPB_OK;
}

int ddpb_bind_bucket_views(ddpb_t h, void* const* replica_storage, int64_t storage_elems, void* compute_stream,
                           void* const* side_streams, int32_t n_side, int32_t flags) {
  if (!h) return fail(DDPB_E_ARG, "bind_bucket_views: NULL handle");
  const ddpb::Plan& p = h->red.plan();
  if (flags & ~(DDPB_BIND_DEVICE_TIMESTAMPS | DDPB_BIND_TIME_LAUNCHES | DDPB_BIND_ROCTX | DDPB_BIND_OVERLAP))
    return fail(DDPB_E_ARG, "bind_bucket_views: bad flags");
  if (n_side < 1 || n_side > 16 || side_streams == nullptr)
    return fail(DDPB_E_ARG, "bind_bucket_views: need 1..16 side streams");
  if (storage_elems < p.flat_elems) return fail(DDPB_E_ARG, "bind_bucket_views: storage smaller than needed");
  if (replica_storage == nullptr) return fail(DDPB_E_ARG, "bind_bucket_views: replica_storage is NULL");
  ddpb::BindArgs a;
  a.view_bases.assign(replica_storage, replica_storage + p.R);
  for (void* s : a.view_bases)
    if (s == nullptr && p.flat_elems > 0) return fail(DDPB_E_ARG, "bind_bucket_views: NULL storage");
  a.compute_stream = compute_stream;
  a.side_streams.assign(side_streams, side_streams + n_side);
  a.mode = ddpb::kModeBucketView;
  a.flags = flags;
  std::string err;
  return pass(h->red.bind(a, &err), err);
}

int ddpb_ensure_prior_reduction_finished(ddpb_t h) {
  if (!h) return fail(DDPB_E_ARG, "NULL handle");
  std::string err;
  return pass(h->red.ensure_prior_reduction_finished(&err), err);
}

int ddpb_mark_ready(ddpb_t h, int32_t v) {
  if (!h) return fail(DDPB_E_ARG, "NULL handle");
  std::string err;
  const int rc = h->red.mark_ready(v, &err);
  if (rc != DDPB_OK) g_err = err;
  return rc;
}

int ddpb_mark_ready_many(ddpb_t h, const int32_t* vs, int32_t n) {
  if (!h || (n > 0 && vs == nullptr) || n < 0) return fail(DDPB_E_ARG, "mark_ready_many: bad argument");
  std::string err;
  for (int32_t i = 0; i < n; ++i) {
    const int rc = h->red.mark_ready(vs[i], &err);
    if (rc != DDPB_OK) return fail(rc, err);
  }
  return DDPB_OK;
}

int ddpb_finalize(ddpb_t h) {
  if (!h) return fail(DDPB_E_ARG, "NULL handle");
  std::string err;
  return pass(h->red.finalize(&err), err);
}

int ddpb_set_sync(ddpb_t h, int32_t enabled) {
  if (!h) return fail(DDPB_E_ARG, "NULL handle");
  std::string err;
  return pass(h->red.set_sync(enabled != 0, &err), err);
}

int ddpb_no_sync_accumulate(ddpb_t h, void* const* step_ptrs, int32_t step_dtype, int32_t first_step) {
  if (!h) return fail(DDPB_E_ARG, "NULL handle");
  std::string err;
  return pass(h->red.accumulate(step_ptrs, step_dtype, first_step != 0, &err), err);
}

int ddpb_reset(ddpb_t h) {
  if (!h) return fail(DDPB_E_ARG, "NULL handle");
  std::string err;
  return pass(h->red.reset(&err), err);
}

int ddpb_get_launch_log(ddpb_t h, int32_t* buckets, int32_t* trigger_call, int64_t* dev_t0,
                        int64_t* dev_t1, int32_t cap, int32_t* n) {
  if (!h || !n || cap < 0) return fail(DDPB_E_ARG, "get_launch_log: bad argument");
  const auto& log = h->red.log();
  *n = static_cast<int32_t>(log.size());
  const int32_t m = std::min<int32_t>(cap, *n);
  for (int32_t i = 0; i < m; ++i) {
    if (buckets) buckets[i] = log[i].bucket;
    if (trigger_call) trigger_call[i] = log[i].trigger_call;
  }
  if ((dev_t0 || dev_t1) && m > 0) {
    std::vector<ddpb::LaunchRecord> part(log.begin(), log.begin() + m);
    std::vector<int64_t> t0, t1;
    std::string err;
    const int rc = h->red.launcher()->read_stamps(part, &t0, &t1, &err);
    if (rc != DDPB_OK) return fail(rc, err);
    for (int32_t i = 0; i < m; ++i) {
      if (dev_t0) dev_t0[i] = t0[i];
      if (dev_t1) dev_t1[i] = t1[i];
    }
  }
  return DDPB_OK;
}

int ddpb_get_launch_times(ddpb_t h, int32_t iterations_ago, float* start_ms, float* ms, int32_t cap,
                          int32_t* n) {
  if (!h || !n || cap < 0 || (cap > 0 && !ms)) return fail(DDPB_E_ARG, "get_launch_times: bad argument");
  const int64_t fin = h->red.finalized();
  if (iterations_ago < 0 || iterations_ago >= ddpb::kTimeRing || iterations_ago >= fin)
    return fail(DDPB_E_INDEX, "get_launch_times: no such finalized iteration");
  const int64_t it = fin - 1 - iterations_ago;
  if (it < h->red.timed_from())
    return fail(DDPB_E_INDEX, "get_launch_times: that iteration ran before the current binding");
  const auto& log = h->red.log_of(it);
  *n = static_cast<int32_t>(log.size());
  const int32_t m = std::min<int32_t>(cap, *n);
  if (m == 0) return DDPB_OK;
  std::vector<ddpb::LaunchRecord> part(log.begin(), log.begin() + m);
  std::vector<float> st, t;
  std::string err;
  const int rc = h->red.launcher()->read_times(it, part, &st, &t, &err);
  if (rc != DDPB_OK) return fail(rc, err);
  for (int32_t i = 0; i < m; ++i) {
    ms[i] = t[i];
    if (start_ms) start_ms[i] = st[i];
  }
  return DDPB_OK;
}

int ddpb_set_local_used(ddpb_t h, const uint8_t* used) {
  if (!h) return fail(DDPB_E_ARG, "NULL handle");
  std::string err;
  return pass(h->red.set_local_used(used, &err), err);
}

int ddpb_set_launch_blocks(ddpb_t h, int32_t max_blocks) {
  if (!h || max_blocks < 0) return fail(DDPB_E_ARG, "set_launch_blocks: bad argument");
  h->red.launcher()->set_max_blocks(max_blocks);
  return DDPB_OK;
}

int ddpb_set_sync_step(ddpb_t h, void* const* step_ptrs, int32_t step_dtype, int32_t first_step) {
  if (!h) return fail(DDPB_E_ARG, "set_sync_step: NULL handle");
  std::string err;
  return pass(h->red.set_sync_step(step_ptrs, step_dtype, first_step != 0, &err), err);
}

int ddpb_set_workgroups_per_cu(ddpb_t h, int32_t n) {
  if (!h || n < 0 || n > 2) return fail(DDPB_E_ARG, "set_workgroups_per_cu: n must be 0, 1 or 2");
  std::string err;
  return pass(h->red.launcher()->set_workgroups_per_cu(n, &err), err);
}

int ddpb_device_clock_hz(ddpb_t h, int64_t* hz) {
  if (!h || !hz) return fail(DDPB_E_ARG, "device_clock_hz: NULL argument");
  std::string err;
  return pass(h->red.launcher()->clock_hz(hz, &err), err);
}

int ddpb_norm_create(const int64_t* numel, const int32_t* dtypes, int32_t P, ddpb_norm_t* out) {
  if (out == nullptr) return fail(DDPB_E_ARG, "norm create: out is NULL");
  *out = nullptr;
  if (P < 0 || (P > 0 && (numel == nullptr || dtypes == nullptr)))
    return fail(DDPB_E_ARG, "norm create: bad P, numel or dtypes");
  if (!numels_ok(numel, P)) return fail(DDPB_E_ARG, "norm create: bad numel");
  for (int32_t v = 0; v < P; ++v)
    if (!is_dtype(dtypes[v])) return fail(DDPB_E_ARG, "norm create: bad dtype");
  return guarded("norm create", [&](std::string*) {
    *out = new ddpb_norm(std::vector<int64_t>(numel, numel + P), std::vector<int32_t>(dtypes, dtypes + P));
    (*out)->P = P;
    return DDPB_OK;
  });
}

void ddpb_norm_destroy(ddpb_norm_t n) { delete n; }

int ddpb_norm_workspace_bytes(ddpb_norm_t n, int64_t* bytes) {
  if (!n || !bytes) return fail(DDPB_E_ARG, "norm workspace_bytes: NULL argument");
  *bytes = n->norm.workspace_bytes();
  return DDPB_OK;
}

int ddpb_norm_bind(ddpb_norm_t n, void* const* grads, void* workspace, int64_t ws_bytes, void* stream, ddpb_t h) {
  if (!n) return fail(DDPB_E_ARG, "norm bind: NULL handle");
  if (n->P > 0 && grads == nullptr) return fail(DDPB_E_ARG, "norm bind: grads is NULL");
  return guarded("norm bind", [&](std::string* err) {
    return n->norm.bind(grads, workspace, ws_bytes, stream, reducer_of(h), err);
  });
}

int ddpb_norm_compute(ddpb_norm_t n, ddpb_t h, double max_norm, double grad_scale, int32_t flags) {
  if (!n) return fail(DDPB_E_ARG, "norm compute: NULL handle");
  if (flags & ~DDPB_NORM_SKIP_NONFINITE) return fail(DDPB_E_ARG, "norm compute: bad flags");
  return guarded("norm compute", [&](std::string* err) {
    return n->norm.compute(reducer_of(h), max_norm, grad_scale, (flags & DDPB_NORM_SKIP_NONFINITE) != 0, err);
  });
}

int ddpb_adamw_create(const int64_t* numel, int32_t P, int32_t R, int32_t param_dtype, int32_t grad_dtype,
                      int32_t state, int32_t flags, double beta1, double beta2, double eps,
                      const double* weight_decay, const double* lr_scale, uint64_t seed, ddpb_adamw_t* out) {
  if (out == nullptr) return fail(DDPB_E_ARG, "adamw create: out is NULL");
  *out = nullptr;
  if (P < 0 || (P > 0 && numel == nullptr) || !numels_ok(numel, P))
    return fail(DDPB_E_ARG, "adamw create: bad P or numel");
  if (R < 1 || R > ddpb::kMaxReplicas) return fail(DDPB_E_ARG, "adamw create: R must be in 1..64");
  if (!is_dtype(param_dtype) || !is_dtype(grad_dtype)) return fail(DDPB_E_ARG, "adamw create: bad dtype");
  if (state != DDPB_STATE_F32 && state != DDPB_STATE_F8) return fail(DDPB_E_ARG, "adamw create: bad state type");
  if (flags & ~DDPB_ADAMW_MASTER) return fail(DDPB_E_ARG, "adamw create: bad flags");
  if ((flags & DDPB_ADAMW_MASTER) && param_dtype == DDPB_F32)
    return fail(DDPB_E_ARG, "adamw create: fp32 parameters take no master copy");
  if (!(beta1 >= 0 && beta1 < 1) || !(beta2 >= 0 && beta2 < 1) || !(eps >= 0) || !std::isfinite(eps))
    return fail(DDPB_E_ARG, "adamw create: betas must be in [0, 1), eps finite and not negative");
  for (int32_t v = 0; v < P; ++v) {
    if (weight_decay != nullptr && !(weight_decay[v] >= 0 && std::isfinite(weight_decay[v])))
      return fail(DDPB_E_ARG, "adamw create: weight_decay must be finite and not negative");
    if (lr_scale != nullptr && !(lr_scale[v] >= 0 && std::isfinite(lr_scale[v])))
      return fail(DDPB_E_ARG, "adamw create: lr_scale must be finite and not negative");
  }
  return guarded("adamw create", [&](std::string*) {
    ddpb::AdamwConfig c;
    c.numel.assign(numel, numel + P);
    c.R = R;
    c.param_dtype = param_dtype;
    c.grad_dtype = grad_dtype;
    c.f8 = state == DDPB_STATE_F8;
    c.master = (flags & DDPB_ADAMW_MASTER) != 0;
    c.beta1 = beta1;
    c.beta2 = beta2;
    c.eps = eps;
    if (weight_decay != nullptr) c.weight_decay.assign(weight_decay, weight_decay + P);
    if (lr_scale != nullptr) c.lr_scale.assign(lr_scale, lr_scale + P);
    c.seed = seed;
    *out = new ddpb_adamw(std::move(c));
    return DDPB_OK;
  });
}

void ddpb_adamw_destroy(ddpb_adamw_t a) { delete a; }

int ddpb_adamw_workspace_bytes(ddpb_adamw_t a, int64_t* bytes) {
  if (!a || !bytes) return fail(DDPB_E_ARG, "adamw workspace_bytes: NULL argument");
  *bytes = a->opt.workspace_bytes();
  return DDPB_OK;
}

int ddpb_adamw_bind(ddpb_adamw_t a, void* const* params, void* const* grads, void* const* master,
                    void* const* exp_avg, void* const* second, void* const* avg_scale, void* const* root_scale,
                    int64_t step, void* workspace, int64_t ws_bytes, void* stream, ddpb_t h) {
  if (!a) return fail(DDPB_E_ARG, "adamw bind: NULL handle");
  const ddpb::AdamwConfig& c = a->opt.config();
  if (!c.numel.empty()) {
    if (!params || !grads || !exp_avg || !second) return fail(DDPB_E_ARG, "adamw bind: NULL pointer array");
    if (c.master && !master) return fail(DDPB_E_ARG, "adamw bind: master is NULL");
    if (c.f8 && (!avg_scale || !root_scale)) return fail(DDPB_E_ARG, "adamw bind: 8-bit states need their scales");
  }
  const ddpb::AdamwBuffers b{params, grads, master, exp_avg, second, avg_scale, root_scale};
  return guarded("adamw bind", [&](std::string* err) {
    return a->opt.bind(b, step, workspace, ws_bytes, stream, reducer_of(h), err);
  });
}

int ddpb_adamw_step(ddpb_adamw_t a, ddpb_t h, double lr, const float* lr_device, double grad_scale,
                    const void* clip) {
  if (!a) return fail(DDPB_E_ARG, "adamw step: NULL handle");
  return guarded("adamw step", [&](std::string* err) {
    return a->opt.step(reducer_of(h), lr, lr_device, grad_scale, clip, err);
  });
}

int ddpb_adamw_set_step(ddpb_adamw_t a, int64_t step) {
  if (!a) return fail(DDPB_E_ARG, "adamw set_step: NULL handle");
  return guarded("adamw set_step", [&](std::string* err) { return a->opt.set_step(step, err); });
}

int ddpb_adamw_get_step(ddpb_adamw_t a, int64_t* step) {
  if (!a || !step) return fail(DDPB_E_ARG, "adamw get_step: NULL argument");
  return guarded("adamw get_step", [&](std::string* err) { return a->opt.get_step(step, err); });
}

int ddpb_check_writable(ddpb_t h, int32_t v) {
  if (!h) return fail(DDPB_E_ARG, "check_writable: NULL handle");
  std::string err;
  return pass(h->red.check_writable(v, &err), err);
}

int ddpb_begin_writes(ddpb_t h, const int32_t* vs, int32_t n) {
  if (!h || n < 0 || (n > 0 && !vs)) return fail(DDPB_E_ARG, "begin_writes: bad argument");
  std::string err;
  return pass(h->red.begin_writes(vs, n, &err), err);
}

int ddpb_layer_norm(int64_t rows, int64_t cols, int32_t dtype, const void* x, int64_t x_stride, const void* residual,
                    int64_t residual_stride, const ddpb_drop* drop, const void* weight, const void* bias,
                    int32_t weight_dtype, double eps, void* y, void* h, float* stats, void* stream) {
  if (!is_dtype(dtype) || !is_dtype(weight_dtype)) return fail(DDPB_E_ARG, "layer_norm: bad dtype");
  return enqueue("layer_norm", &ddpb::LayersDevice::norm_forward, [&](ddpb::NormForwardArgs* a, std::string* err) {
    a->rows = rows;
    a->cols = cols;
    a->dtype = dtype;
    a->weight_dtype = weight_dtype;
    a->x = {x, x_stride};
    a->residual = {residual, residual_stride};
    a->weight = weight;
    a->bias = bias;
    a->eps = eps;
    a->y = y;
    a->h = h;
    a->stats = stats;
    a->stream = stream;
    return drop_of(drop, &a->drop, "layer_norm", err);
  });
}

int ddpb_layer_norm_backward_workspace_bytes(int64_t rows, int64_t cols, int64_t* bytes) {
  if (bytes == nullptr || !ddpb::norm_sizes_ok(rows, cols))
    return fail(DDPB_E_ARG, "layer_norm_backward workspace_bytes: bad argument");
  *bytes = ddpb::norm_backward_workspace(rows, cols);
  return DDPB_OK;
}

int ddpb_layer_norm_backward(int64_t rows, int64_t cols, int32_t dtype, const void* dy, int64_t dy_stride,
                             const void* h, int64_t h_stride, const float* stats, const void* grad_h,
                             int64_t grad_h_stride, const ddpb_drop* drop, const void* weight, int32_t weight_dtype,
                             void* dh, void* dx, void* dweight, void* dbias, int32_t grad_dtype, int32_t accumulate,
                             void* workspace, int64_t ws_bytes, void* stream) {
  return norm_backward(&ddpb::LayersDevice::norm_backward, rows, cols, dtype, {dy, dy_stride}, {h, h_stride}, stats,
                       {grad_h, grad_h_stride}, drop, weight, weight_dtype, dh, dx, dweight, dbias, grad_dtype,
                       accumulate, workspace, ws_bytes, stream);
}

int ddpb_layer_norm_backward_check(int64_t rows, int64_t cols, int32_t dtype, const void* dy, int64_t dy_stride,
                                   const void* h, int64_t h_stride, const float* stats, const void* grad_h,
                                   int64_t grad_h_stride, const ddpb_drop* drop, const void* weight,
                                   int32_t weight_dtype, void* dh, void* dx, void* dweight, void* dbias,
                                   int32_t grad_dtype, int32_t accumulate, void* workspace, int64_t ws_bytes) {
  return norm_backward(nullptr, rows, cols, dtype, {dy, dy_stride}, {h, h_stride}, stats, {grad_h, grad_h_stride}, drop,
                       weight, weight_dtype, dh, dx, dweight, dbias, grad_dtype, accumulate, workspace, ws_bytes,
                       nullptr);
}

int ddpb_dropout(int64_t rows, int64_t cols, int32_t dtype, const void* x, int64_t x_stride, const void* residual,
                 int64_t residual_stride, const ddpb_drop* drop, void* y, void* stream) {
  if (!is_dtype(dtype)) return fail(DDPB_E_ARG, "dropout: bad dtype");
  if (drop == nullptr) return fail(DDPB_E_ARG, "dropout: drop is NULL");
  return enqueue("dropout", &ddpb::LayersDevice::dropout, [&](ddpb::DropoutArgs* a, std::string* err) {
    a->rows = rows;
    a->cols = cols;
    a->dtype = dtype;
    a->x = {x, x_stride};
    a->residual = {residual, residual_stride};
    a->y = y;
    a->stream = stream;
    return drop_of(drop, &a->drop, "dropout", err);
  });
}

int ddpb_embedding(int64_t n, const void* tokens, int32_t token_bytes, int64_t vocab, int64_t cols, const void* table,
                   int32_t table_dtype, double scale, const void* residual, int64_t residual_stride, void* y,
                   int32_t dtype, void* stream) {
  if (!is_dtype(dtype) || !is_dtype(table_dtype) || (token_bytes != 4 && token_bytes != 8))
    return fail(DDPB_E_ARG, "embedding: bad dtype or token_bytes");
  return enqueue("embedding", &ddpb::LayersDevice::lookup, [&](ddpb::LookupArgs* a, std::string*) {
    a->n = n;
    a->vocab = vocab;
    a->cols = cols;
    a->tokens = tokens;
    a->token_bytes = token_bytes;
    a->table = table;
    a->table_dtype = table_dtype;
    a->scale = static_cast<float>(scale);
    a->residual = {residual, residual_stride};
    a->y = y;
    a->dtype = dtype;
    a->stream = stream;
    return DDPB_OK;
  });
}

int ddpb_embedding_backward_workspace_bytes(int64_t n, int64_t vocab, int64_t cols, int64_t* bytes) {
  if (bytes == nullptr || !ddpb::lookup_sizes_ok(n, vocab, cols))
    return fail(DDPB_E_ARG, "embedding_backward workspace_bytes: bad argument");
  *bytes = ddpb::lookup_plan(n, vocab, cols).bytes;
  return DDPB_OK;
}

int ddpb_embedding_backward(int64_t n, const void* tokens, int32_t token_bytes, int64_t vocab, int64_t cols,
                            const void* dy, int64_t dy_stride, int32_t dtype, double scale, void* dtable,
                            int32_t grad_dtype, int32_t accumulate, void* workspace, int64_t ws_bytes, void* stream) {
  return embedding_backward(&ddpb::LayersDevice::lookup_backward, n, tokens, token_bytes, vocab, cols, {dy, dy_stride},
                            dtype, scale, dtable, grad_dtype, accumulate, workspace, ws_bytes, stream);
}

int ddpb_embedding_backward_check(int64_t n, const void* tokens, int32_t token_bytes, int64_t vocab, int64_t cols,
                                  const void* dy, int64_t dy_stride, int32_t dtype, double scale, void* dtable,
                                  int32_t grad_dtype, int32_t accumulate, void* workspace, int64_t ws_bytes) {
  return embedding_backward(nullptr, n, tokens, token_bytes, vocab, cols, {dy, dy_stride}, dtype, scale, dtable,
                            grad_dtype, accumulate, workspace, ws_bytes, nullptr);
}

}  // extern "C"
