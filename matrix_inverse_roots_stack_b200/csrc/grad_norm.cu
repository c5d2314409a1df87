// Global norm and clipping of a list of gradients (shampoo_grad_norm,
// shampoo_grad_clip in include/dash_b200.h).
//
// norm = inv_scale sqrt(sum g^2) over every element of every tensor, and
// coef = inv_scale min(1, max_norm / norm), the factor that unscales and
// clips a gradient; clipping writes g <- coef g in place.  Both are bound by
// HBM: one read of the gradients for the norm, one more read and a write for
// clipping.
#include <cmath>
#include <new>

#include "profile.cuh"
#include "tensor_list.cuh"

namespace dash {
namespace {

struct GradChunk {
  void* grad;
  int count;   // elements, at most chunk_elems
  int flags;   // element type, and kVec when the start is on a 16-byte boundary
};
constexpr int kVec = 16;
constexpr int kTypeMask = 15;

// Start of the workspace.
struct NormHeader {
  unsigned status;  // first word: the status word
  unsigned ticket;
  unsigned next;    // shares taken in the running call, beyond the first of each block
};
constexpr size_t kHeaderBytes = 256;
// A chunk is 32 KB: 8192 fp32 or 16384 16-bit elements, 128 bytes for each
// thread, all of them in flight at once (32 registers).  With chunks half as
// long the norm of 1.36G bf16 elements takes 389 instead of 378 us, in a long
// run 408 instead of 387.
constexpr int kChunkBytes = 32768;
__host__ __device__ constexpr int chunk_elems(int dtype) { return kChunkBytes / (dtype == SHAMPOO_DTYPE_F32 ? 4 : 2); }
constexpr int kLoads = kChunkBytes / (kListThreads * 16);  // 16-byte pieces of a thread
// Shares for each resident block in a long list, or up to twice that.  With 2, 4, 8, 16 and 32 of them 129 chunks a
// block take 345, 343, 341, 345 and 346 us (fp32) and 16 chunks a block 51.4, 53, 52, 56 and 58 us (bf16).
constexpr int kTurns = 8;

__device__ __forceinline__ void add_squares(const float* x, double* acc) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const double d = x[j];
    acc[j & 1] = fma(d, d, acc[j & 1]);
  }
}

// The same for eight bf16 elements as they lie in memory.  An SM converts 16
// fp32 numbers a clock to fp64, and at two bytes an element that is two thirds
// of the time; so every other one is made of its bits instead.  bf16's exponent and
// mantissa, put where fp64 has its own, are |x| 2^-896, subnormals and 0 included.  An
// exponent of infinity or NaN would pass as a number: 'special' becomes NaN
// then (the word as an fp32 number has that exponent too).  1.36G elements with
// every element converted: 394 instead of 378 us, in a long run 404 instead of 388.
__device__ __forceinline__ void add_squares_bf16(const unsigned* w, double* acc, float& special) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const double lo = __uint_as_float(w[j] << 16);
    const double hi = __hiloint2double(static_cast<int>((w[j] >> 3) & 0x0fffe000u), 0) * 0x1p896;
    acc[0] = fma(lo, lo, acc[0]);
    acc[1] = fma(hi, hi, acc[1]);
    special = fmaf(__uint_as_float(w[j]), 0.0f, special);
  }
}

// Sum of a block's values, in a fixed order; valid in thread 0.
__device__ __forceinline__ double block_sum(double x) {
  __shared__ double part[kListWarps];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
  __syncthreads();
  double s = 0.0;
  if (threadIdx.x == 0)
    for (int w = 0; w < kListWarps; ++w) s += part[w];
  __syncthreads();
  return s;
}

// The squares are formed and added in fp64: the square of any finite fp32
// value is exact and in range there, so neither small nor large gradients
// are lost, and the result is not finite exactly when an element is not.
//
// A share is 'rounds' chunks, a grid's width apart, so that blocks that run
// side by side read side by side.  A block adds up a share in a fixed order,
// wherever it runs, and the last block to finish adds the shares' sums: the
// result is the same on every call, while the blocks take shares as they come
// (SMs differ in how far from memory they are).  Chunks are counted from the
// end, because what the L2 cache still holds afterwards is then the front of
// the list, where the pass that follows starts.
__global__ void __launch_bounds__(kListThreads) grad_norm_kernel(const GradChunk* __restrict__ chunks, int n_chunks,
                                                                 int shares, int rounds, NormHeader* hdr, double* partial,
                                                                 double max_norm, double inv_scale, float* out) {
  __shared__ int taken;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int p = blockIdx.x; p < shares;) {
    unsigned next = 0;  // looked at behind the share
    if (threadIdx.x == 0) next = atomicAdd(&hdr->next, 1u);
    double acc[2] = {0.0, 0.0};
    float special = 0.0f;
    const int width = gridDim.x, first = p / width * (width * rounds) + p % width;
    for (int j = 0, k = n_chunks - 1 - first; j < rounds && k >= 0; ++j, k -= width) {
      const GradChunk c = chunks[k];
      const int type = c.flags & kTypeMask;
      const bool whole = (c.flags & kVec) && c.count == chunk_elems(type);
      if (whole && type == SHAMPOO_DTYPE_F32) {
        Raw8 r[kLoads / 2];
#pragma unroll
        for (int s = 0; s < kLoads / 2; ++s)
          load32B(static_cast<const float*>(c.grad) + 8 * (s * kListThreads + threadIdx.x), r[s].w);
#pragma unroll
        for (int s = 0; s < kLoads / 2; ++s) {
          float x[8];
          widen8(r[s], SHAMPOO_DTYPE_F32, x);
          add_squares(x, acc);
        }
      } else if (whole) {
        Raw8 r[kLoads];
        const uint4* from = static_cast<const uint4*>(c.grad) + threadIdx.x;
#pragma unroll
        for (int s = 0; s < kLoads; ++s) {
          const uint4 q = from[s * kListThreads];
          r[s].w[0] = q.x, r[s].w[1] = q.y, r[s].w[2] = q.z, r[s].w[3] = q.w;
        }
        if (type == SHAMPOO_DTYPE_BF16) {
#pragma unroll
          for (int s = 0; s < kLoads; ++s) add_squares_bf16(r[s].w, acc, special);
        } else {
#pragma unroll
          for (int s = 0; s < kLoads; ++s) {
            float x[8];
            widen8(r[s], SHAMPOO_DTYPE_F16, x);
            add_squares(x, acc);
          }
        }
      } else {
        for (int b = warp * kQBlock; b < c.count; b += kListWarps * kQBlock) {
          float x[8];
          load8_strided(c.grad, b + lane, c.count, type, x);
          add_squares(x, acc);
        }
      }
    }
    if (threadIdx.x == 0) taken = static_cast<int>(gridDim.x + next);
    const double sum = block_sum(acc[0] + acc[1] + special);  // with barriers: 'taken' is there
    if (threadIdx.x == 0) partial[p] = sum;
    p = taken;
    __syncthreads();
  }
  if (!last_block(&hdr->ticket)) return;
  double t = 0.0;
  for (int i = threadIdx.x; i < shares; i += kListThreads) t += __ldcg(partial + i);
  t = block_sum(t);
  if (threadIdx.x == 0) {
    const double norm = sqrt(t) * inv_scale;
    const bool ok = isfinite(t);
    out[0] = static_cast<float>(norm);
    out[1] = ok ? static_cast<float>((norm > max_norm ? max_norm / norm : 1.0) * inv_scale) : __int_as_float(0x7fffffff);
    hdr->status = ok ? 0u : kStatusNonFinite;
    hdr->next = 0;
  }
}

// g <- coef g; a coefficient of 1 leaves the gradients unread, one that is
// not finite sets them to zero.  Two blocks of threads to a chunk.
constexpr int kClipParts = 2;
__global__ void __launch_bounds__(kListThreads) grad_clip_kernel(const GradChunk* __restrict__ chunks,
                                                                 const float* __restrict__ out) {
  const GradChunk c = chunks[blockIdx.x / kClipParts];
  const float coef = out[1];
  if (coef == 1.0f) return;
  const bool zero = not_finite(coef);
  const int part = blockIdx.x % kClipParts, warp = part * kListWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int type = c.flags & kTypeMask;
  constexpr int kStep = kClipParts * kListWarps;  // blocks of 256 from a warp's to its next
  if ((c.flags & kVec) && c.count == chunk_elems(type)) {
    uint4* at = static_cast<uint4*>(c.grad) + part * (kLoads / kClipParts * kListThreads) + threadIdx.x;
    uint4 q[kLoads / kClipParts];
#pragma unroll
    for (int s = 0; s < kLoads / kClipParts; ++s) q[s] = at[s * kListThreads];
#pragma unroll
    for (int s = 0; s < kLoads / kClipParts; ++s) {
      unsigned* w = reinterpret_cast<unsigned*>(&q[s]);
      if (type == SHAMPOO_DTYPE_F32) {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = zero ? 0u : __float_as_uint(__uint_as_float(w[j]) * coef);
      } else {
        Raw8 r;
        float x[8];
        r.w[0] = w[0], r.w[1] = w[1], r.w[2] = w[2], r.w[3] = w[3];
        widen8(r, type, x);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = zero ? 0u : narrow2(x[2 * j] * coef, x[2 * j + 1] * coef, type);
      }
      at[s * kListThreads] = q[s];
    }
  } else {
    for (int b = warp * kQBlock; b < c.count; b += kStep * kQBlock) {
      float x[8];
      load8_strided(c.grad, b + lane, c.count, type, x);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (b + lane + 32 * j < c.count) store1(c.grad, b + lane + 32 * j, type, zero ? 0.0f : x[j] * coef);
    }
  }
}

}  // namespace
}  // namespace dash

struct shampoo_grads {
  std::vector<dash::GradChunk> chunks;
  size_t off_partial = 0, total = 0;
  dash::ListMemory memory;
  const void* bound_ws = nullptr;
  int shares = 0, rounds = 1, grid = 1;
};

namespace {

constexpr int kMaxShares = 1 << 15;  // partial sums kept in the workspace

int norm_pass(shampoo_grads* c, float max_norm, float inv_scale, float* out, void* ws, size_t ws_bytes, void* stream,
              bool clip) {
  if (!c || !out || !dash::aligned_to(out, 4) || !(max_norm > 0.0f) || !(inv_scale > 0.0f) || !std::isfinite(inv_scale))
    return SHAMPOO_EINVAL;
  if (!ws || ws_bytes < c->total) return SHAMPOO_EWORKSPACE;
  if (ws != c->bound_ws) return SHAMPOO_EINVAL;
  if ((clip && c->memory.meets(out, 2 * sizeof(float))) || dash::share(out, 2 * sizeof(float), ws, c->total))
    return SHAMPOO_EINVAL;
  char* w = static_cast<char*>(ws);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const auto* table = reinterpret_cast<const dash::GradChunk*>(w + dash::kHeaderBytes);
  const int n = static_cast<int>(c->chunks.size());
  dash::grad_norm_kernel<<<c->grid, dash::kListThreads, 0, st>>>(
      table, n, c->shares, c->rounds, reinterpret_cast<dash::NormHeader*>(w),
      reinterpret_cast<double*>(w + c->off_partial), max_norm, inv_scale, out);
  dash::prof_count_launch();
  if (cudaGetLastError() != cudaSuccess) return SHAMPOO_ECUDA;
  if (clip && n > 0) {
    dash::grad_clip_kernel<<<n * dash::kClipParts, dash::kListThreads, 0, st>>>(table, out);
    dash::prof_count_launch();
    if (cudaGetLastError() != cudaSuccess) return SHAMPOO_ECUDA;
  }
  return SHAMPOO_OK;
}

}  // namespace

extern "C" {

int shampoo_grads_init(shampoo_grads** out, const shampoo_grad* grads, int n_grads, size_t* workspace_bytes) {
  if (!out || !grads || n_grads < 1 || !workspace_bytes) return SHAMPOO_EINVAL;
  *out = nullptr;
  shampoo_grads* c = nullptr;
  try {
    c = new shampoo_grads();
    std::vector<dash::ByteRange> ranges;
    for (int i = 0; i < n_grads; ++i) {
      const shampoo_grad& g = grads[i];
      const bool ok = g.n >= 0 && g.n <= SHAMPOO_MAX_TENSOR && dash::valid_dtype(g.dtype) &&
                      (g.n == 0 || (g.grad && dash::aligned_to(g.grad, dash::dtype_bytes(g.dtype))));
      if (!ok) {
        delete c;
        return SHAMPOO_EINVAL;
      }
      const size_t size = dash::dtype_bytes(g.dtype);
      dash::add_range(ranges, g.grad, size * static_cast<size_t>(g.n), true);
      const int flags = g.dtype | (dash::aligned_to(g.grad, 16) ? dash::kVec : 0);
      const int chunk = dash::chunk_elems(g.dtype);
      for (int64_t at = 0; at < g.n; at += chunk)
        c->chunks.push_back({static_cast<char*>(g.grad) + size * static_cast<size_t>(at),
                             static_cast<int>(std::min<int64_t>(chunk, g.n - at)), flags});
    }
    if (dash::ranges_clash(ranges) || c->chunks.size() > 0x7ffffff) {
      delete c;
      return SHAMPOO_EINVAL;
    }
    c->memory = dash::ListMemory(ranges, false);
  } catch (...) {
    delete c;
    return SHAMPOO_EINVAL;
  }
  const size_t table = (c->chunks.size() * sizeof(dash::GradChunk) + 255) / 256 * 256;
  c->off_partial = dash::kHeaderBytes + table;
  c->total = c->off_partial + kMaxShares * sizeof(double);
  *workspace_bytes = c->total;
  *out = c;
  return SHAMPOO_OK;
}

int shampoo_grads_bind(shampoo_grads* c, void* ws, size_t ws_bytes, void* stream) {
  if (!c) return SHAMPOO_EINVAL;
  if (!ws || !dash::aligned_to(ws, 256) || ws_bytes < c->total) return SHAMPOO_EWORKSPACE;
  if (c->memory.meets(ws, c->total)) return SHAMPOO_EINVAL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(st, &cap) != cudaSuccess) return SHAMPOO_ECUDA;
  if (cap != cudaStreamCaptureStatusNone) return SHAMPOO_EINVAL;
  c->bound_ws = nullptr;
  const int blocks = dash::resident_blocks(dash::grad_norm_kernel);
  if (blocks < 0) return SHAMPOO_ECUDA;
  const int n = static_cast<int>(c->chunks.size());
  c->grid = std::max(1, std::min({n, blocks, kMaxShares / (2 * dash::kTurns)}));
  // A list of under four chunks a block is one share a block, a longer one shares from the counter.  The two in us, in
  // a graph, by chunks a block: 2.6: 12.8 and 13.9; 4.25: 17.5 and 19.4; 8.1: 27.3 and 29.6; 16: 48.5 and 50.2; 32:
  // 90.0 and 91.6; 129: 343.6 and 341 (all fp32; in fp16 395 and 364).  So one
  // share is ahead up to some 30 chunks a block already, by 2 to 10%.
  c->rounds = n < 4 * c->grid ? (n + c->grid - 1) / c->grid : std::max(1, n / (dash::kTurns * c->grid));
  // whole groups of grid x rounds chunks, the last one short
  const int group = c->grid * std::max(1, c->rounds);
  c->shares = (n + group - 1) / group * c->grid;
  if (cudaMemsetAsync(ws, 0, dash::kHeaderBytes, st) != cudaSuccess) return SHAMPOO_ECUDA;
  if (!c->chunks.empty() &&
      cudaMemcpyAsync(static_cast<char*>(ws) + dash::kHeaderBytes, c->chunks.data(),
                      c->chunks.size() * sizeof(dash::GradChunk), cudaMemcpyHostToDevice, st) != cudaSuccess)
    return SHAMPOO_ECUDA;
  c->bound_ws = ws;
  return SHAMPOO_OK;
}

int shampoo_grad_norm(shampoo_grads* c, float max_norm, float inv_scale, float* out, void* ws, size_t ws_bytes,
                      void* stream) {
  return norm_pass(c, max_norm, inv_scale, out, ws, ws_bytes, stream, false);
}

int shampoo_grad_clip(shampoo_grads* c, float max_norm, float inv_scale, float* out, void* ws, size_t ws_bytes,
                      void* stream) {
  return norm_pass(c, max_norm, inv_scale, out, ws, ws_bytes, stream, true);
}

void shampoo_grads_destroy(shampoo_grads* c) { delete c; }

}  // extern "C"
