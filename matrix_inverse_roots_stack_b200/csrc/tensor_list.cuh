// Shared pieces of the kernels that work on a list of tensors in one launch
// (adamw.cu, grad_norm.cu): element types, 8-element vector accesses, and the
// host checks of a list's memory.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <utility>
#include <vector>

#include "dash_b200.h"
#include "ptx.cuh"

namespace dash {

// One warp step: 256 consecutive elements of a tensor, 8 to a lane.  It is
// also the block that shares a scale in the 8-bit moments.
constexpr int kQBlock = SHAMPOO_QBLOCK;
constexpr int kListThreads = 256;
constexpr int kListWarps = kListThreads / 32;

inline bool valid_dtype(int d) {
  return d == SHAMPOO_DTYPE_F32 || d == SHAMPOO_DTYPE_BF16 || d == SHAMPOO_DTYPE_F16;
}
inline size_t dtype_bytes(int d) { return d == SHAMPOO_DTYPE_F32 ? 4 : 2; }
inline bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Byte ranges of a list's buffers: true when a written range meets any other.
struct ByteRange {
  uintptr_t lo, hi;
  bool written;
};
inline bool ranges_clash(std::vector<ByteRange>& r) {
  std::sort(r.begin(), r.end(), [](const ByteRange& a, const ByteRange& b) { return a.lo < b.lo; });
  uintptr_t hi_any = 0, hi_written = 0;  // furthest ends seen so far
  for (const ByteRange& x : r) {
    if (x.lo < hi_written || (x.written && x.lo < hi_any)) return true;
    hi_any = std::max(hi_any, x.hi);
    if (x.written) hi_written = std::max(hi_written, x.hi);
  }
  return false;
}
inline void add_range(std::vector<ByteRange>& r, const void* p, size_t bytes, bool written) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  if (bytes) r.push_back({lo, lo + bytes, written});
}
inline bool share(const void* p, size_t p_bytes, const void* q, size_t q_bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return p_bytes && q_bytes && a < b + q_bytes && b < a + p_bytes;
}

// A list's memory, kept for the buffers that later calls pass: disjoint
// ranges in order, made of those that ranges_clash has sorted.
class ListMemory {
 public:
  ListMemory() = default;
  ListMemory(const std::vector<ByteRange>& sorted, bool written_only) {
    for (const ByteRange& x : sorted) {
      if (written_only && !x.written) continue;
      if (ends_.empty() || x.lo > ends_.back().second) ends_.emplace_back(x.lo, x.hi);
      else ends_.back().second = std::max(ends_.back().second, x.hi);
    }
  }
  bool meets(const void* p, size_t bytes) const {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    const auto behind = std::lower_bound(ends_.begin(), ends_.end(), lo + bytes,
                                         [](const auto& x, uintptr_t at) { return x.first < at; });
    return bytes && behind != ends_.begin() && (behind - 1)->second > lo;
  }

 private:
  std::vector<std::pair<uintptr_t, uintptr_t>> ends_;
};

// ------------------------------------------------------------ device side

// Eight elements as they lie in memory: 32 bytes of fp32, or 16 bytes of a
// 16-bit type in w[0..3].
struct Raw8 {
  unsigned w[8];
};

// A lane's eight fp32 elements, from a 16-byte boundary.  On a 32-byte one
// they are one 256-bit access (sm_100), and a warp covers 1 KB without a
// strided second access.
__device__ __forceinline__ bool half_sector(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 16u) != 0; }
__device__ __forceinline__ void load32B(const void* p, unsigned* w) {
  if (half_sector(p)) {
    const uint4 a = static_cast<const uint4*>(p)[0], b = static_cast<const uint4*>(p)[1];
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    return;
  }
  asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void store32B_wide(void* p, const unsigned* w) {  // from a 32-byte boundary
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ void store32B(void* p, const unsigned* w) {
  if (half_sector(p)) {
    static_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  } else {
    store32B_wide(p, w);
  }
}

__device__ __forceinline__ float widen(unsigned short b, int dtype) {
  return dtype == SHAMPOO_DTYPE_BF16 ? __uint_as_float(static_cast<unsigned>(b) << 16)
                                     : __half2float(__ushort_as_half(b));
}
__device__ __forceinline__ unsigned short narrow(float x, int dtype) {
  return dtype == SHAMPOO_DTYPE_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x))
                                     : __half_as_ushort(__float2half_rn(x));
}
__device__ __forceinline__ unsigned narrow2(float lo, float hi, int dtype) {
  if (dtype == SHAMPOO_DTYPE_BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const unsigned*>(&h);
  }
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const unsigned*>(&h);
}

// Vector path: elements 8 i .. 8 i + 7 of a buffer that starts on a 16-byte
// boundary.
__device__ __forceinline__ void load8(const void* base, int i, int dtype, Raw8& r) {
  if (dtype == SHAMPOO_DTYPE_F32) {
    load32B(static_cast<const float*>(base) + 8ll * i, r.w);
  } else {
    const uint4 q = *(static_cast<const uint4*>(base) + i);
    r.w[0] = q.x, r.w[1] = q.y, r.w[2] = q.z, r.w[3] = q.w;
  }
}
__device__ __forceinline__ void widen8(const Raw8& r, int dtype, float* x) {
  if (dtype == SHAMPOO_DTYPE_F32) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(r.w[j]);
  } else if (dtype == SHAMPOO_DTYPE_BF16) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = __uint_as_float(r.w[j] << 16);
      x[2 * j + 1] = __uint_as_float(r.w[j] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r.w[j]));
      x[2 * j] = f.x;
      x[2 * j + 1] = f.y;
    }
  }
}
template <bool kWide = false>  // fp32 from a 32-byte boundary
__device__ __forceinline__ void store8(void* base, int i, int dtype, const float* x) {
  if (dtype == SHAMPOO_DTYPE_F32) {
    unsigned w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(x[j]);
    if (kWide) store32B_wide(static_cast<float*>(base) + 8ll * i, w);
    else store32B(static_cast<float*>(base) + 8ll * i, w);
  } else {
    *(static_cast<uint4*>(base) + i) = make_uint4(narrow2(x[0], x[1], dtype), narrow2(x[2], x[3], dtype),
                                                  narrow2(x[4], x[5], dtype), narrow2(x[6], x[7], dtype));
  }
}

// Eight elements i, i + 32, ..., those below n, of a buffer with no more than
// its type's alignment; the others are 0.  The loads leave together: nothing
// is converted between them.
__device__ __forceinline__ void load8_strided(const void* base, int i, int n, int dtype, float* x) {
  unsigned w[8];
  if (dtype == SHAMPOO_DTYPE_F32) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = i + 32 * j < n ? static_cast<const unsigned*>(base)[i + 32 * j] : 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(w[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = i + 32 * j < n ? static_cast<const unsigned short*>(base)[i + 32 * j] : 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = widen(static_cast<unsigned short>(w[j]), dtype);
  }
}

// Element i of a buffer with no more than its type's alignment.
__device__ __forceinline__ void store1(void* base, int i, int dtype, float x) {
  if (dtype == SHAMPOO_DTYPE_F32) static_cast<float*>(base)[i] = x;
  else static_cast<unsigned short*>(base)[i] = narrow(x, dtype);
}

// Not finite: exponent bits all set.
__device__ __forceinline__ bool not_finite(float x) { return (__float_as_uint(x) & 0x7fffffffu) >= 0x7f800000u; }

// True in every thread of the last block of the grid to get here; what the
// other blocks wrote before is then visible.  'ticket' is 0 between launches.
__device__ __forceinline__ bool last_block(unsigned* ticket) {
  __shared__ bool last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(ticket, 1u) == gridDim.x - 1;
    if (last) {
      *ticket = 0;
      __threadfence();
    }
  }
  __syncthreads();
  return last;
}

// Blocks of 'kernel' that fill the device, or a negative SHAMPOO_E* code.
template <typename Kernel>
int resident_blocks(Kernel kernel, int threads = kListThreads, size_t smem = 0) {
  int dev = 0, sms = 0, per = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, smem) != cudaSuccess || per < 1)
    return SHAMPOO_ECUDA;
  return sms * per;
}

}  // namespace dash
