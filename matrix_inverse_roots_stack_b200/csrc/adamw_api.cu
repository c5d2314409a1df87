// Entry points of AdamW over a list of tensors (declared in
// include/dash_b200.h): argument checks, the table, and the launches of
// adamw.cu's kernels.
#include <cmath>
#include <new>

#include "adamw.cuh"
#include "gemm.cuh"
#include "profile.cuh"

using dash::AdamwHeader;
using dash::AdamwTable;
using dash::AdamwTensorDev;

struct shampoo_adamw {
  shampoo_adamw_hparams hp{};
  std::vector<int> first_tile;           // of each tensor
  std::vector<AdamwTensorDev> tensors;
  AdamwHeader start{};         // header that bind uploads
  int bits = 32;               // of every tensor's moments, or 0
  int stage_bytes = 0;         // of a tile in shared memory, at most
  bool stages = false;         // there are tiles that a step can fetch into shared memory
  int64_t blocks = 0, tiles = 0;
  size_t off_tensors = 0, total = 0;  // workspace
  const void* bound_ws = nullptr;
  dash::ListMemory all, written, moments;  // the list's arrays, those that steps write, and the moments with their scales
  dash::AdamwLaunch launch{};
};

namespace {

constexpr size_t kHeaderBytes = 256;
constexpr float kMinEps = 1e-30f;  // keeps eps (1 - beta1^t) in fp32's normal range for every beta1 < 1
constexpr int64_t kMaxBlocks = 0x7fffffff - 0xffff;  // a block's number plus a grid's warps stays an int
static_assert(sizeof(AdamwHeader) <= kHeaderBytes, "header fits");

bool tensor_ok(const shampoo_adamw_tensor& q) {
  if (q.n < 0 || q.n > SHAMPOO_MAX_TENSOR || (q.state_bits != 32 && q.state_bits != 8)) return false;
  if (q.param_dtype != SHAMPOO_DTYPE_F32 && q.param_dtype != SHAMPOO_DTYPE_BF16) return false;
  if (!dash::valid_dtype(q.grad_dtype)) return false;
  if (!std::isfinite(q.lr_scale) || q.lr_scale < 0.0f || !std::isfinite(q.weight_decay) || q.weight_decay < 0.0f)
    return false;
  if (q.copy && (q.param_dtype != SHAMPOO_DTYPE_F32 ||
                 (q.copy_dtype != SHAMPOO_DTYPE_BF16 && q.copy_dtype != SHAMPOO_DTYPE_F16)))
    return false;
  if (q.n == 0) return true;
  if (!q.param || !q.grad || !q.m || !q.v || (q.state_bits == 8 && (!q.m_scale || !q.v_scale))) return false;
  const size_t ms = q.state_bits == 32 ? 4 : 1;
  return dash::aligned_to(q.param, dash::dtype_bytes(q.param_dtype)) &&
         dash::aligned_to(q.grad, dash::dtype_bytes(q.grad_dtype)) && dash::aligned_to(q.copy, 2) &&
         dash::aligned_to(q.m, ms) && dash::aligned_to(q.v, ms);
}

// Whether every array but the scales lies on a 16-byte boundary, so that bulk
// copies and accesses of eight elements reach it.
bool vector_ok(const shampoo_adamw_tensor& q) {
  bool ok = true;
  for (const void* p : {static_cast<const void*>(q.param), q.grad, static_cast<const void*>(q.copy),
                        static_cast<const void*>(q.m), static_cast<const void*>(q.v)})
    ok = ok && dash::aligned_to(p, 16);
  return ok;
}

// And whether eight fp32 elements can be written in one access, and scales
// fetched four at a time.
bool wide_ok(const shampoo_adamw_tensor& q) {
  if (!vector_ok(q) || (q.param_dtype == SHAMPOO_DTYPE_F32 && !dash::aligned_to(q.param, 32))) return false;
  return q.state_bits == 32 ? dash::aligned_to(q.m, 32) && dash::aligned_to(q.v, 32)
                            : dash::aligned_to(q.m_scale, 4) && dash::aligned_to(q.v_scale, 4);
}

size_t blocks_of(const shampoo_adamw_tensor& q) {
  return (static_cast<size_t>(q.n) + dash::kQBlock - 1) / dash::kQBlock;
}

void add_moments(std::vector<dash::ByteRange>& r, const shampoo_adamw_tensor& q) {
  const size_t bytes = static_cast<size_t>(q.n) * (q.state_bits == 32 ? 4 : 1);
  dash::add_range(r, q.m, bytes, true);
  dash::add_range(r, q.v, bytes, true);
  if (q.state_bits == 8) {
    dash::add_range(r, q.m_scale, blocks_of(q), true);
    dash::add_range(r, q.v_scale, blocks_of(q), true);
  }
}

void add_tensor(shampoo_adamw* c, const shampoo_adamw_tensor& q, int index) {
  const bool eight = q.state_bits == 8;
  AdamwTensorDev r{};
  r.param = q.param;
  r.grad = q.grad;
  r.copy = q.copy;
  r.m = q.m;
  r.v = q.v;
  r.m_scale = eight ? q.m_scale : nullptr;
  r.v_scale = eight ? q.v_scale : nullptr;
  r.n = q.n;
  r.first = static_cast<int>(c->blocks);
  r.first_tile = static_cast<int>(c->tiles);
  r.flags = (q.param_dtype << dash::kParamShift) | (q.grad_dtype << dash::kGradShift) |
            ((q.copy ? q.copy_dtype : 0) << dash::kCopyShift) | (eight ? dash::kFlagEight : 0) |
            (vector_ok(q) ? dash::kFlagVec : 0) | (wide_ok(q) ? dash::kFlagWide : 0);
  r.index = index;
  r.lr_scale = q.lr_scale;
  r.decay = q.weight_decay;
  c->stages = c->stages || ((r.flags & dash::kFlagWide) && q.n >= dash::kTile);
  c->bits = c->tensors.empty() || c->bits == q.state_bits ? q.state_bits : 0;
  c->first_tile.push_back(r.first_tile);
  c->tensors.push_back(r);
  c->blocks += static_cast<int64_t>(blocks_of(q));
  c->tiles += (q.n + dash::kTile - 1) / dash::kTile;
  c->stage_bytes = std::max(c->stage_bytes, dash::adamw_stage_bytes(eight, q.param_dtype, q.grad_dtype));
}

// Step t's constants, in double from the fp32 hyper-parameters.
struct StepConstants {
  double pow1, pow2;  // beta^t
  float d1, d0;
};
StepConstants step_constants(const shampoo_adamw_hparams& hp, double t) {
  StepConstants s;
  s.pow1 = std::pow(static_cast<double>(hp.beta1), t);
  s.pow2 = std::pow(static_cast<double>(hp.beta2), t);
  s.d1 = static_cast<float>((1.0 - s.pow1) / std::sqrt(1.0 - s.pow2));
  s.d0 = static_cast<float>(hp.adam_eps * (1.0 - s.pow1));
  return s;
}

int check_bound(const shampoo_adamw* c, const void* ws, size_t ws_bytes) {
  if (!c) return SHAMPOO_EINVAL;
  if (!ws || ws_bytes < c->total) return SHAMPOO_EWORKSPACE;
  return ws == c->bound_ws ? SHAMPOO_OK : SHAMPOO_EINVAL;
}

// Flat moments, and whether their memory is their own; a list without
// elements has none.
bool flat_ok(const shampoo_adamw* c, const void* p) { return c->blocks == 0 || (p && dash::aligned_to(p, 16)); }
size_t flat_bytes(const shampoo_adamw* c, int dtype) {
  return static_cast<size_t>(c->blocks) * dash::kQBlock * dash::dtype_bytes(dtype);
}
bool apart(const shampoo_adamw* c, const dash::ListMemory& from, const void* p, size_t bytes, const void* ws) {
  return !from.meets(p, bytes) && !dash::share(p, bytes, ws, c->total);
}
// A rate or coefficient on the device.
bool scalar_ok(const shampoo_adamw* c, const float* p, const void* ws) {
  return !p || (dash::aligned_to(p, 4) && apart(c, c->written, p, sizeof(float), ws));
}

AdamwTable table(const shampoo_adamw* c, const void* ws) {
  const char* w = static_cast<const char*>(ws);
  return {reinterpret_cast<const int*>(w + kHeaderBytes), reinterpret_cast<const AdamwTensorDev*>(w + c->off_tensors),
          static_cast<int>(c->tensors.size()), static_cast<int>(c->tiles)};
}

}  // namespace

extern "C" {

int shampoo_adamw_init(shampoo_adamw** out, const shampoo_adamw_tensor* tensors, int n_tensors,
                       const shampoo_adamw_hparams* hp, size_t* workspace_bytes, int64_t* moment_elems) {
  if (!out || !tensors || n_tensors < 1 || !hp || !workspace_bytes) return SHAMPOO_EINVAL;
  *out = nullptr;
  if (!(hp->beta1 >= 0.0f && hp->beta1 < 1.0f) || !(hp->beta2 >= 0.0f && hp->beta2 < 1.0f) ||
      !(hp->adam_eps >= kMinEps) || !std::isfinite(hp->adam_eps))
    return SHAMPOO_EINVAL;
  shampoo_adamw* c = nullptr;
  try {
    c = new shampoo_adamw();
    c->hp = *hp;
    std::vector<dash::ByteRange> ranges;
    int64_t blocks_total = 0;
    bool ok = true;
    for (int i = 0; i < n_tensors && ok; ++i) {
      const shampoo_adamw_tensor& q = tensors[i];
      ok = tensor_ok(q);
      if (!ok || q.n == 0) continue;
      const size_t n = static_cast<size_t>(q.n);
      blocks_total += static_cast<int64_t>(blocks_of(q));
      dash::add_range(ranges, q.param, n * dash::dtype_bytes(q.param_dtype), true);
      dash::add_range(ranges, q.grad, n * dash::dtype_bytes(q.grad_dtype), false);
      if (q.copy) dash::add_range(ranges, q.copy, 2 * n, true);
      add_moments(ranges, q);
    }
    if (!ok || blocks_total > kMaxBlocks || dash::ranges_clash(ranges)) {
      delete c;
      return SHAMPOO_EINVAL;
    }
    c->all = dash::ListMemory(ranges, false);
    c->written = dash::ListMemory(ranges, true);
    std::vector<dash::ByteRange> moments;
    for (int i = 0; i < n_tensors; ++i) add_moments(moments, tensors[i]);
    std::sort(moments.begin(), moments.end(), [](const auto& a, const auto& b) { return a.lo < b.lo; });
    c->moments = dash::ListMemory(moments, true);
    for (int i = 0; i < n_tensors; ++i)
      if (tensors[i].n > 0) add_tensor(c, tensors[i], i);
    if (c->tensors.empty()) c->stage_bytes = dash::adamw_stage_bytes(false, SHAMPOO_DTYPE_F32, SHAMPOO_DTYPE_F32);
  } catch (...) {
    delete c;
    return SHAMPOO_EINVAL;
  }
  c->off_tensors = (kHeaderBytes + c->first_tile.size() * sizeof(int) + 255) / 256 * 256;
  c->total = c->off_tensors + c->tensors.size() * sizeof(AdamwTensorDev);
  *workspace_bytes = c->total;
  if (moment_elems) *moment_elems = c->blocks * dash::kQBlock;
  *out = c;
  return SHAMPOO_OK;
}

int shampoo_adamw_bind(shampoo_adamw* c, int steps_taken, void* ws, size_t ws_bytes, void* stream) {
  if (!c || steps_taken < 0) return SHAMPOO_EINVAL;
  if (!ws || !dash::aligned_to(ws, 256) || ws_bytes < c->total) return SHAMPOO_EWORKSPACE;
  if (c->all.meets(ws, c->total)) return SHAMPOO_EINVAL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(st, &cap) != cudaSuccess) return SHAMPOO_ECUDA;
  if (cap != cudaStreamCaptureStatusNone) return SHAMPOO_EINVAL;
  c->bound_ws = nullptr;
  const int rc = dash::adamw_prepare(c->bits, c->stage_bytes, &c->launch);
  if (rc) return rc;
  const StepConstants next = step_constants(c->hp, steps_taken + 1.0);
  const StepConstants last = step_constants(c->hp, steps_taken);
  c->start = AdamwHeader{};
  c->start.t = steps_taken;
  c->start.pow1 = last.pow1;
  c->start.pow2 = last.pow2;
  c->start.d1 = next.d1;
  c->start.d0 = next.d0;
  char* w = static_cast<char*>(ws);
  if (cudaMemcpyAsync(w, &c->start, sizeof(c->start), cudaMemcpyHostToDevice, st) != cudaSuccess)
    return SHAMPOO_ECUDA;
  if (!c->tensors.empty() &&
      (cudaMemcpyAsync(w + kHeaderBytes, c->first_tile.data(), c->first_tile.size() * sizeof(int),
                       cudaMemcpyHostToDevice, st) != cudaSuccess ||
       cudaMemcpyAsync(w + c->off_tensors, c->tensors.data(), c->tensors.size() * sizeof(AdamwTensorDev),
                       cudaMemcpyHostToDevice, st) != cudaSuccess))
    return SHAMPOO_ECUDA;
  c->bound_ws = ws;
  return SHAMPOO_OK;
}

int shampoo_adamw_step(shampoo_adamw* c, int step, float lr, const float* lr_device, const float* coef, void* ws,
                       size_t ws_bytes, void* stream) {
  const int rc = check_bound(c, ws, ws_bytes);
  if (rc) return rc;
  if (step < 0 || (!lr_device && !std::isfinite(lr)) || !scalar_ok(c, lr_device, ws) || !scalar_ok(c, coef, ws))
    return SHAMPOO_EINVAL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  dash::AdamwArgs a{};
  a.beta1 = make_float2(c->hp.beta1, c->hp.beta1);
  a.beta2 = make_float2(c->hp.beta2, c->hp.beta2);
  a.om1 = make_float2(1.0f - c->hp.beta1, 1.0f - c->hp.beta1);
  a.om2 = make_float2(1.0f - c->hp.beta2, 1.0f - c->hp.beta2);
  a.one = make_float2(1.0f, 1.0f);
  a.eps = c->hp.adam_eps;
  a.seed_lo = static_cast<unsigned>(c->hp.seed);
  a.seed_hi = static_cast<unsigned>(c->hp.seed >> 32);
  // only a step that has loads to withhold takes the fault
  a.withhold = c->stages && c->tiles > c->launch.direct && dash::take_load_fault() ? 1 : 0;
  a.step = step;
  if (step > 0) {
    const StepConstants s = step_constants(c->hp, step);
    a.pow1 = s.pow1;
    a.pow2 = s.pow2;
    a.d1 = s.d1;
    a.d0 = s.d0;
  }
  a.lr = lr;
  a.lr_device = lr_device;
  a.coef = coef;
  const int slot = dash::prof_begin(dash::kProfAdam, st);
  const int grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(c->tiles, c->launch.step)));
  dash::launch_adamw(table(c, ws), c->launch, grid, static_cast<AdamwHeader*>(ws), a, st);
  const cudaError_t e = cudaGetLastError();
  dash::prof_end(slot, st);
  return e == cudaSuccess ? SHAMPOO_OK : SHAMPOO_ECUDA;
}

int shampoo_adamw_load_moments(shampoo_adamw* c, const float* m, const float* v, void* ws, size_t ws_bytes,
                               void* stream) {
  const int rc = check_bound(c, ws, ws_bytes);
  if (rc) return rc;
  const size_t bytes = flat_bytes(c, SHAMPOO_DTYPE_F32);
  if (!flat_ok(c, m) || !flat_ok(c, v) || !apart(c, c->moments, m, bytes, ws) ||
      !apart(c, c->moments, v, bytes, ws))
    return SHAMPOO_EINVAL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(ws, 0, sizeof(unsigned), st) != cudaSuccess) return SHAMPOO_ECUDA;
  if (c->blocks == 0) return SHAMPOO_OK;
  dash::launch_load_moments(table(c, ws), static_cast<AdamwHeader*>(ws), m, v, st);
  return cudaGetLastError() == cudaSuccess ? SHAMPOO_OK : SHAMPOO_ECUDA;
}

int shampoo_adamw_read_moments(shampoo_adamw* c, void* m, void* v, int dtype, void* ws, size_t ws_bytes,
                               void* stream) {
  const int rc = check_bound(c, ws, ws_bytes);
  if (rc) return rc;
  if ((dtype != SHAMPOO_DTYPE_F32 && dtype != SHAMPOO_DTYPE_BF16) || !flat_ok(c, m) || !flat_ok(c, v))
    return SHAMPOO_EINVAL;
  const size_t bytes = flat_bytes(c, dtype);
  if (dash::share(m, bytes, v, bytes) || !apart(c, c->moments, m, bytes, ws) || !apart(c, c->moments, v, bytes, ws))
    return SHAMPOO_EINVAL;
  if (c->blocks == 0) return SHAMPOO_OK;
  dash::launch_read_moments(table(c, ws), m, v, dtype, static_cast<cudaStream_t>(stream));
  return cudaGetLastError() == cudaSuccess ? SHAMPOO_OK : SHAMPOO_ECUDA;
}

int shampoo_adamw_steps_taken(const shampoo_adamw* c, const void* ws, size_t ws_bytes, void* stream,
                              int* steps_taken) {
  const int rc = check_bound(c, ws, ws_bytes);
  if (rc) return rc;
  if (!steps_taken) return SHAMPOO_EINVAL;
  AdamwHeader h;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaStreamSynchronize(st) != cudaSuccess ||
      cudaMemcpy(&h, ws, sizeof(h), cudaMemcpyDeviceToHost) != cudaSuccess)
    return SHAMPOO_ECUDA;
  *steps_taken = h.t;
  return SHAMPOO_OK;
}

void shampoo_adamw_destroy(shampoo_adamw* c) { delete c; }

}  // extern "C"
