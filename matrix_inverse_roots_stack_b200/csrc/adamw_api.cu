// Entry points of AdamW over a list of tensors (declared in
// include/dash_b200.h): argument checks, the chunk table, and the launches of
// adamw.cu's kernels.
#include <cfloat>
#include <cmath>
#include <new>

#include "adamw.cuh"
#include "profile.cuh"

using dash::AdamwChunk;
using dash::AdamwHeader;

struct shampoo_adamw {
  shampoo_adamw_hparams hp{};
  std::vector<AdamwChunk> chunks;
  AdamwHeader start{};         // header that bind uploads
  int which = 0;               // 0: 32-bit moments only, 1: 8-bit only, 2: both
  int64_t moment_elems = 0;    // of the flat moments
  size_t total = 0;            // workspace bytes
  const void* bound_ws = nullptr;
  int step_blocks = 0, load_blocks = 0, read_blocks = 0;
};

namespace {

constexpr size_t kHeaderBytes = 256;
static_assert(sizeof(AdamwHeader) <= kHeaderBytes, "header fits");

// Elements of a chunk: one step of a block's warps, or four where that still
// leaves the device many chunks for each block.
int chunk_elems(int64_t total) {
  const int one = dash::kListWarps * dash::kQBlock;
  return total > (1ll << 28) ? 4 * one : one;
}

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

// Whether every pointer lets a lane take eight elements in one access.
bool vector_ok(const shampoo_adamw_tensor& q) {
  const size_t ms = q.state_bits == 32 ? 32 : 8;
  return dash::aligned_to(q.param, 8 * dash::dtype_bytes(q.param_dtype)) &&
         dash::aligned_to(q.grad, 8 * dash::dtype_bytes(q.grad_dtype)) && dash::aligned_to(q.copy, 16) &&
         dash::aligned_to(q.m, ms) && dash::aligned_to(q.v, ms);
}

void add_tensor(shampoo_adamw* c, const shampoo_adamw_tensor& q, int index, int chunk) {
  const size_t ps = dash::dtype_bytes(q.param_dtype), gs = dash::dtype_bytes(q.grad_dtype);
  const bool eight = q.state_bits == 8;
  const size_t ms = eight ? 1 : 4;
  int flags = (q.param_dtype << dash::kParamShift) | (q.grad_dtype << dash::kGradShift) |
              ((q.copy ? q.copy_dtype : 0) << dash::kCopyShift);
  if (eight) flags |= dash::kFlagEight;
  if (vector_ok(q)) flags |= dash::kFlagVec;
  for (int64_t at = 0; at < q.n; at += chunk) {
    AdamwChunk r{};
    r.param = static_cast<char*>(q.param) + ps * at;
    r.grad = static_cast<const char*>(q.grad) + gs * at;
    r.copy = q.copy ? static_cast<char*>(q.copy) + 2 * at : nullptr;
    r.m = static_cast<char*>(q.m) + ms * at;
    r.v = static_cast<char*>(q.v) + ms * at;
    r.m_scale = eight ? q.m_scale + at / dash::kQBlock : nullptr;
    r.v_scale = eight ? q.v_scale + at / dash::kQBlock : nullptr;
    r.elem = at;
    r.flat = c->moment_elems + at;
    r.count = static_cast<int>(std::min<int64_t>(chunk, q.n - at));
    r.flags = flags;
    r.tensor = index;
    r.lr_scale = q.lr_scale;
    r.decay = q.weight_decay;
    c->chunks.push_back(r);
  }
  c->moment_elems += (q.n + dash::kQBlock - 1) / dash::kQBlock * dash::kQBlock;
}

// beta^t and the corrections of step t, in double, from the fp32 betas.
double pow_beta(float beta, int t) { return std::pow(static_cast<double>(beta), t); }
float correction1(double p1) { return static_cast<float>(1.0 / (1.0 - p1)); }
float correction2(double p2) { return static_cast<float>(std::sqrt(1.0 / (1.0 - p2))); }

int check_bound(const shampoo_adamw* c, const void* ws, size_t ws_bytes) {
  if (!c) return SHAMPOO_EINVAL;
  if (!ws || ws_bytes < c->total) return SHAMPOO_EWORKSPACE;
  return ws == c->bound_ws ? SHAMPOO_OK : SHAMPOO_EINVAL;
}

const AdamwChunk* table(const void* ws) {
  return reinterpret_cast<const AdamwChunk*>(static_cast<const char*>(ws) + kHeaderBytes);
}

}  // namespace

extern "C" {

int shampoo_adamw_init(shampoo_adamw** out, const shampoo_adamw_tensor* tensors, int n_tensors,
                       const shampoo_adamw_hparams* hp, size_t* workspace_bytes, int64_t* moment_elems) {
  if (!out || !tensors || n_tensors < 1 || !hp || !workspace_bytes) return SHAMPOO_EINVAL;
  *out = nullptr;
  if (!(hp->beta1 >= 0.0f && hp->beta1 < 1.0f) || !(hp->beta2 >= 0.0f && hp->beta2 < 1.0f) ||
      !(hp->adam_eps >= FLT_MIN) || !std::isfinite(hp->adam_eps))
    return SHAMPOO_EINVAL;
  shampoo_adamw* c = nullptr;
  try {
    c = new shampoo_adamw();
    c->hp = *hp;
    std::vector<dash::ByteRange> ranges;
    int64_t total = 0;
    bool has32 = false, has8 = false, ok = true;
    for (int i = 0; i < n_tensors && ok; ++i) {
      const shampoo_adamw_tensor& q = tensors[i];
      ok = tensor_ok(q);
      if (!ok || q.n == 0) continue;
      const size_t n = static_cast<size_t>(q.n), ms = q.state_bits == 32 ? 4 : 1;
      const size_t blocks = (n + dash::kQBlock - 1) / dash::kQBlock;
      (q.state_bits == 32 ? has32 : has8) = true;
      total += q.n;
      dash::add_range(ranges, q.param, n * dash::dtype_bytes(q.param_dtype), true);
      dash::add_range(ranges, q.grad, n * dash::dtype_bytes(q.grad_dtype), false);
      if (q.copy) dash::add_range(ranges, q.copy, 2 * n, true);
      dash::add_range(ranges, q.m, n * ms, true);
      dash::add_range(ranges, q.v, n * ms, true);
      if (q.state_bits == 8) {
        dash::add_range(ranges, q.m_scale, blocks, true);
        dash::add_range(ranges, q.v_scale, blocks, true);
      }
    }
    const int chunk = chunk_elems(total);
    if (!ok || dash::ranges_clash(ranges) || total / chunk + n_tensors > 0x7ffffff) {
      delete c;
      return SHAMPOO_EINVAL;
    }
    for (int i = 0; i < n_tensors; ++i) add_tensor(c, tensors[i], i, chunk);
    c->which = has32 && has8 ? 2 : has8 ? 1 : 0;
  } catch (...) {
    delete c;
    return SHAMPOO_EINVAL;
  }
  c->total = kHeaderBytes + c->chunks.size() * sizeof(AdamwChunk);
  *workspace_bytes = c->total;
  if (moment_elems) *moment_elems = c->moment_elems;
  *out = c;
  return SHAMPOO_OK;
}

int shampoo_adamw_bind(shampoo_adamw* c, int steps_taken, void* ws, size_t ws_bytes, void* stream) {
  if (!c || steps_taken < 0) return SHAMPOO_EINVAL;
  if (!ws || !dash::aligned_to(ws, 256) || ws_bytes < c->total) return SHAMPOO_EWORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(st, &cap) != cudaSuccess) return SHAMPOO_ECUDA;
  if (cap != cudaStreamCaptureStatusNone) return SHAMPOO_EINVAL;
  c->bound_ws = nullptr;
  c->step_blocks = dash::adamw_blocks(c->which);
  c->load_blocks = dash::adamw_blocks(3);
  c->read_blocks = dash::adamw_blocks(4);
  if (c->step_blocks < 0 || c->load_blocks < 0 || c->read_blocks < 0) return SHAMPOO_ECUDA;
  const double p1 = pow_beta(c->hp.beta1, steps_taken), p2 = pow_beta(c->hp.beta2, steps_taken);
  c->start = AdamwHeader{};
  c->start.t = steps_taken;
  c->start.pow1 = p1;
  c->start.pow2 = p2;
  c->start.c1 = correction1(p1 * c->hp.beta1);
  c->start.c2 = correction2(p2 * c->hp.beta2);
  if (cudaMemcpyAsync(ws, &c->start, sizeof(c->start), cudaMemcpyHostToDevice, st) != cudaSuccess)
    return SHAMPOO_ECUDA;
  if (!c->chunks.empty() &&
      cudaMemcpyAsync(static_cast<char*>(ws) + kHeaderBytes, c->chunks.data(),
                      c->chunks.size() * sizeof(AdamwChunk), cudaMemcpyHostToDevice, st) != cudaSuccess)
    return SHAMPOO_ECUDA;
  c->bound_ws = ws;
  return SHAMPOO_OK;
}

int shampoo_adamw_step(shampoo_adamw* c, int step, float lr, const float* lr_device, const float* coef, void* ws,
                       size_t ws_bytes, void* stream) {
  const int rc = check_bound(c, ws, ws_bytes);
  if (rc) return rc;
  if (step < 0 || (!lr_device && !std::isfinite(lr))) return SHAMPOO_EINVAL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  dash::AdamwArgs a{};
  a.beta1 = c->hp.beta1;
  a.beta2 = c->hp.beta2;
  a.eps = c->hp.adam_eps;
  a.seed_lo = static_cast<unsigned>(c->hp.seed);
  a.seed_hi = static_cast<unsigned>(c->hp.seed >> 32);
  a.step = step;
  if (step > 0) {
    a.pow1 = pow_beta(a.beta1, step);
    a.pow2 = pow_beta(a.beta2, step);
    a.c1 = correction1(a.pow1);
    a.c2 = correction2(a.pow2);
  }
  a.lr = lr;
  a.lr_device = lr_device;
  a.coef = coef;
  const int n = static_cast<int>(c->chunks.size());
  const int slot = dash::prof_begin(dash::kProfAdam, st);
  dash::launch_adamw(table(ws), n, c->which, std::max(1, std::min(n, c->step_blocks)),
                     static_cast<AdamwHeader*>(ws), a, st);
  const cudaError_t e = cudaGetLastError();
  dash::prof_end(slot, st);
  return e == cudaSuccess ? SHAMPOO_OK : SHAMPOO_ECUDA;
}

int shampoo_adamw_load_moments(shampoo_adamw* c, const float* m, const float* v, void* ws, size_t ws_bytes,
                               void* stream) {
  const int rc = check_bound(c, ws, ws_bytes);
  if (rc) return rc;
  if (!m || !v || !dash::aligned_to(m, 32) || !dash::aligned_to(v, 32)) return SHAMPOO_EINVAL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(ws, 0, sizeof(unsigned), st) != cudaSuccess) return SHAMPOO_ECUDA;
  const int n = static_cast<int>(c->chunks.size());
  if (n == 0) return SHAMPOO_OK;
  dash::launch_load_moments(table(ws), n, std::min(n, c->load_blocks), static_cast<AdamwHeader*>(ws), m, v, st);
  return cudaGetLastError() == cudaSuccess ? SHAMPOO_OK : SHAMPOO_ECUDA;
}

int shampoo_adamw_read_moments(shampoo_adamw* c, void* m, void* v, int dtype, void* ws, size_t ws_bytes,
                               void* stream) {
  const int rc = check_bound(c, ws, ws_bytes);
  if (rc) return rc;
  if (!m || !v || (dtype != SHAMPOO_DTYPE_F32 && dtype != SHAMPOO_DTYPE_BF16) || !dash::aligned_to(m, 32) ||
      !dash::aligned_to(v, 32))
    return SHAMPOO_EINVAL;
  const int n = static_cast<int>(c->chunks.size());
  if (n == 0) return SHAMPOO_OK;
  dash::launch_read_moments(table(ws), n, std::min(n, c->read_blocks), m, v, dtype, static_cast<cudaStream_t>(stream));
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
