// AdamW over a list of tensors in one launch, with moments in 32 or 8 bits,
// and the 8-bit moments' way in and out (include/dash_b200.h has the
// formulas and the formats).
//
// All of it streams through HBM once.  Each warp takes 256 consecutive
// elements at a time, eight to a lane, so that every access of an aligned
// tensor is 8 to 32 bytes a lane and a block of 8-bit moments belongs to one
// warp: its maximum is two warp reductions and never leaves registers.
//
// The moments are computed with every product and sum rounded on its own (no
// contraction), so that their 8-bit codes do not depend on how a compiler
// fuses them.
#include "adamw.cuh"
#include "profile.cuh"

namespace dash {
namespace {

// ---------------------------------------------------------------- rounding draws
//
// The rounding of an element draws from a hash of (seed, step, tensor,
// element): two rounds of xor-shift and odd multiplication behind a Weyl
// sequence.  The multipliers are the leading 32 bits of the golden ratio's
// and of the square roots of 2, 3 and 5's fractional parts, made odd.
constexpr unsigned kWeyl = 0x9E3779B9u, kMulA = 0x6A09E667u, kMulB = 0xBB67AE85u, kMulC = 0x3C6EF373u;

__device__ __forceinline__ unsigned key_word(unsigned x, unsigned w) {
  x ^= w;
  x ^= x >> 16;
  x *= kMulA;
  x ^= x >> 16;
  x *= kMulB;
  x ^= x >> 15;
  return x + kWeyl;
}
// key: of the seed, step, tensor and the high half of the element's index.
__device__ __forceinline__ unsigned draw_bits(unsigned key, unsigned elem) {
  unsigned x = elem * kWeyl + key;
  x ^= x >> 16;
  x *= kMulA;
  x ^= x >> 15;
  x *= kMulB;
  return x ^ (x >> 16);
}

// ---------------------------------------------------------------- 8-bit formats
//
// m: sign and e4m3.  r = sqrt(v): e4m4, unsigned.  Magnitudes y (already
// divided by the block's scale) are written as the fp32 number y 2^-120
// (e4m3: smallest normal 2^-6) or y 2^-126 (e4m4: smallest normal 1): there
// fp32's gradual underflow is the format's, and the code is the top of the
// bit pattern, rounded by what is added below it.
constexpr float kM8Down = 0x1p-120f, kV8Down = 0x1p-126f;

__device__ __forceinline__ float power_of_two(int i) { return __int_as_float(i << 23); }  // 2^(i-127), 1 <= i <= 254

// Scale byte i of a block, standing for 2^(i - 127): the smallest that brings
// the block's maximum within the format (448 = 1.75 2^8, 31744 = 1.9375
// 2^14).  255: the maximum is not finite, and the block reads back so.
__device__ __forceinline__ int m8_scale(unsigned amax) {
  return amax >= 0x7f800000u ? 255 : max(1, static_cast<int>((amax + 0x1fffffu) >> 23) - 8);
}
__device__ __forceinline__ int v8_scale(unsigned amax) {
  return amax >= 0x7f800000u ? 255 : max(1, static_cast<int>((amax + 0x07ffffu) >> 23) - 14);
}
// What to multiply an element of the block by: 1 / scale (0 for a scale that
// is not finite, whose codes do not matter).
__device__ __forceinline__ float inverse_scale(int i) { return i == 255 ? 0.0f : power_of_two(254 - i); }

// Code of a magnitude that 'unit' = inverse_scale brings into range; u: 16
// random bits (rounded up where the dropped part and they reach a whole).
__device__ __forceinline__ unsigned m8_code(float y, float unit, unsigned u) {
  const float x = __fmul_rn(__fmul_rn(fabsf(y), unit), kM8Down);
  return ((__float_as_uint(x) + (u << 4)) >> 20) | ((__float_as_uint(y) >> 24) & 0x80u);
}
// r > 0 is never stored as 0: beside a nonzero first moment a vanished
// second one would make the next update explode.
__device__ __forceinline__ unsigned v8_code(float r, float unit, unsigned u) {
  const float x = __fmul_rn(__fmul_rn(r, unit), kV8Down);
  return max((__float_as_uint(x) + (u << 3)) >> 19, r > 0.0f ? 1u : 0u);
}
__device__ __forceinline__ unsigned nearest_even(unsigned b, int low) {
  return (b + ((1u << (low - 1)) - 1u) + ((b >> low) & 1u)) >> low;
}
__device__ __forceinline__ unsigned m8_nearest(float y, float unit) {
  const float x = __fmul_rn(__fmul_rn(fabsf(y), unit), kM8Down);
  return nearest_even(__float_as_uint(x), 20) | ((__float_as_uint(y) >> 24) & 0x80u);
}
__device__ __forceinline__ unsigned v8_nearest(float r, float unit) {
  const float x = __fmul_rn(__fmul_rn(r, unit), kV8Down);
  return max(nearest_even(__float_as_uint(x), 19), r > 0.0f ? 1u : 0u);
}

// Two codes at a time are the bits of fp16 numbers: e4m3 and e4m4 lie inside
// e5m10 up to the exponent's bias, 2^8 and 2^14, which goes into the
// block's factor.
__device__ __forceinline__ float m8_factor(int i) {
  return i == 0 ? 0.0f : i == 255 ? __int_as_float(0x7f800000) : power_of_two(i + 8);
}
__device__ __forceinline__ float v8_factor(int i) {
  return i == 0 ? 0.0f : i == 255 ? __int_as_float(0x7f800000) : power_of_two(i + 14);
}
__device__ __forceinline__ void m8_values4(unsigned codes, float factor, float* m) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    unsigned w = __byte_perm(codes, 0, h ? 0x3424 : 0x1404);  // codes in the high bytes of the halves
    w = (w & 0x80008000u) | ((w & 0x7f007f00u) >> 1);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    m[2 * h] = __fmul_rn(f.x, factor);
    m[2 * h + 1] = __fmul_rn(f.y, factor);
  }
}
__device__ __forceinline__ void v8_values4(unsigned codes, float factor, float* r) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const unsigned w = __byte_perm(codes, 0, h ? 0x4342 : 0x4140) << 6;
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    r[2 * h] = __fmul_rn(f.x, factor);
    r[2 * h + 1] = __fmul_rn(f.y, factor);
  }
}
__device__ __forceinline__ unsigned pack4(const unsigned* c) {
  return c[0] | (c[1] << 8) | (c[2] << 16) | (c[3] << 24);
}

// bf16 pattern of a parameter, rounded by 16 random bits: where parameters
// have no fp32 master, rounding to nearest would drop every update below half
// a bf16 step (2^-9 of the value).
__device__ __forceinline__ unsigned bf16_bits(float p, unsigned draw) {
  const unsigned b = __float_as_uint(p);
  if (not_finite(p)) return (b >> 16) | ((b & 0x7fffffu) ? 0x40u : 0u);
  return (b + ((draw * kMulC) >> 16)) >> 16;
}

struct Coefs {
  float beta1, beta2, om1, om2, eps, c1, c2, lr, decay, coef;
};

// One element: moments, then the parameter.  Returns what the caller flags
// as not finite, as bits of magnitudes.
__device__ __forceinline__ void moments(const Coefs& k, float grad, float& m, float& v) {
  const float g = __fmul_rn(grad, k.coef);
  m = __fadd_rn(__fmul_rn(m, k.beta1), __fmul_rn(g, k.om1));
  v = __fadd_rn(__fmul_rn(v, k.beta2), __fmul_rn(__fmul_rn(g, k.om2), g));
}
__device__ __forceinline__ float updated(const Coefs& k, float p, float m, float r) {
  return p - k.lr * (__fdividef(m * k.c1, fmaf(r, k.c2, k.eps)) + k.decay * p);
}
__device__ __forceinline__ unsigned magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// ---------------------------------------------------------------- 32-bit moments

__device__ __forceinline__ unsigned step32(const AdamwChunk& c, const Coefs& k, unsigned key) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pt = (c.flags >> kParamShift) & 15, gt = (c.flags >> kGradShift) & 15, ct = (c.flags >> kCopyShift) & 15;
  const unsigned elem = static_cast<unsigned>(c.elem);
  unsigned worst = 0;
  for (int b = warp * kQBlock; b < c.count; b += kListWarps * kQBlock) {
    if ((c.flags & kFlagVec) && b + kQBlock <= c.count) {
      const int i = (b >> 3) + lane;
      Raw8 rp, rg, rm, rv;
      load8(c.grad, i, gt, rg);
      load32B(static_cast<const float*>(c.m) + 8 * i, rm.w);
      load32B(static_cast<const float*>(c.v) + 8 * i, rv.w);
      load8(c.param, i, pt, rp);
      float p[8], g[8], m[8], v[8];
      widen8(rg, gt, g);
      widen8(rp, pt, p);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        m[j] = __uint_as_float(rm.w[j]);
        v[j] = __uint_as_float(rv.w[j]);
        moments(k, g[j], m[j], v[j]);
        p[j] = updated(k, p[j], m[j], __fsqrt_rn(v[j]));
        worst = max(worst, max(magnitude(m[j]), max(magnitude(v[j]), magnitude(p[j]))));
      }
      store8(c.m, i, SHAMPOO_DTYPE_F32, m);
      store8(c.v, i, SHAMPOO_DTYPE_F32, v);
      if (pt == SHAMPOO_DTYPE_F32) {
        store8(c.param, i, SHAMPOO_DTYPE_F32, p);
        if (c.copy) store8(c.copy, i, ct, p);
      } else {
        unsigned w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[j] = bf16_bits(p[2 * j], draw_bits(key, elem + 8 * i + 2 * j)) |
                 (bf16_bits(p[2 * j + 1], draw_bits(key, elem + 8 * i + 2 * j + 1)) << 16);
        *(static_cast<uint4*>(c.param) + i) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    } else {
      for (int i = b + lane; i < min(b + kQBlock, c.count); i += 32) {
        float m = static_cast<const float*>(c.m)[i], v = static_cast<const float*>(c.v)[i];
        moments(k, load1(c.grad, i, gt), m, v);
        const float p = updated(k, load1(c.param, i, pt), m, __fsqrt_rn(v));
        worst = max(worst, max(magnitude(m), max(magnitude(v), magnitude(p))));
        static_cast<float*>(c.m)[i] = m;
        static_cast<float*>(c.v)[i] = v;
        if (pt == SHAMPOO_DTYPE_F32) {
          static_cast<float*>(c.param)[i] = p;
          if (c.copy) store1(c.copy, i, ct, p);
        } else {
          static_cast<unsigned short*>(c.param)[i] = bf16_bits(p, draw_bits(key, elem + i));
        }
      }
    }
  }
  return worst;
}

// ---------------------------------------------------------------- 8-bit moments

__device__ __forceinline__ unsigned step8(const AdamwChunk& c, const Coefs& k, unsigned key) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pt = (c.flags >> kParamShift) & 15, gt = (c.flags >> kGradShift) & 15, ct = (c.flags >> kCopyShift) & 15;
  const unsigned elem = static_cast<unsigned>(c.elem);
  unsigned worst = 0;
  for (int b = warp * kQBlock; b < c.count; b += kListWarps * kQBlock) {
    const bool vec = (c.flags & kFlagVec) && b + kQBlock <= c.count;
    uint8_t* ms = c.m_scale + (b >> 8);
    uint8_t* vs = c.v_scale + (b >> 8);
    const int i0 = vec ? b + 8 * lane : b + lane;  // this lane's elements: i0 + j, or i0 + 32 j
    const int stride = vec ? 1 : 32;
    float p[8], m[8], r[8];
    unsigned mmax = 0, rmax = 0;
    {
      float g[8];
      unsigned cm[2], cv[2];
      const float mf = m8_factor(*ms), vf = v8_factor(*vs);
      if (vec) {
        Raw8 rp, rg;
        load8(c.grad, i0 >> 3, gt, rg);
        load8(c.param, i0 >> 3, pt, rp);
        const uint2 qm = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(c.m) + i0);
        const uint2 qv = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(c.v) + i0);
        cm[0] = qm.x, cm[1] = qm.y, cv[0] = qv.x, cv[1] = qv.y;
        widen8(rg, gt, g);
        widen8(rp, pt, p);
      } else {
        cm[0] = cm[1] = cv[0] = cv[1] = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i = i0 + 32 * j;
          const bool in = i < c.count;
          g[j] = in ? load1(c.grad, i, gt) : 0.0f;
          p[j] = in ? load1(c.param, i, pt) : 0.0f;
          if (in) {
            cm[j >> 2] |= static_cast<unsigned>(static_cast<const uint8_t*>(c.m)[i]) << (8 * (j & 3));
            cv[j >> 2] |= static_cast<unsigned>(static_cast<const uint8_t*>(c.v)[i]) << (8 * (j & 3));
          }
        }
      }
      m8_values4(cm[0], mf, m);
      m8_values4(cm[1], mf, m + 4);
      v8_values4(cv[0], vf, r);
      v8_values4(cv[1], vf, r + 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float v = __fmul_rn(r[j], r[j]);
        moments(k, g[j], m[j], v);
        r[j] = __fsqrt_rn(v);
        p[j] = updated(k, p[j], m[j], r[j]);
        if (!vec && i0 + 32 * j >= c.count) m[j] = r[j] = p[j] = 0.0f;
        mmax = max(mmax, magnitude(m[j]));
        rmax = max(rmax, magnitude(r[j]));
        worst = max(worst, magnitude(p[j]));
      }
    }
    worst = max(worst, max(mmax, rmax));
    mmax = __reduce_max_sync(0xffffffffu, mmax);
    rmax = __reduce_max_sync(0xffffffffu, rmax);
    const int mi = m8_scale(mmax), vi = v8_scale(rmax);
    const float mu = inverse_scale(mi), vu = inverse_scale(vi);
    unsigned cm[8], cv[8], h[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      h[j] = draw_bits(key, elem + i0 + stride * j);
      cm[j] = m8_code(m[j], mu, h[j] >> 16);
      cv[j] = v8_code(r[j], vu, h[j] & 0xffffu);
    }
    if (lane == 0) {
      *ms = static_cast<uint8_t>(mi);
      *vs = static_cast<uint8_t>(vi);
    }
    if (vec) {
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(c.m) + i0) = make_uint2(pack4(cm), pack4(cm + 4));
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(c.v) + i0) = make_uint2(pack4(cv), pack4(cv + 4));
      if (pt == SHAMPOO_DTYPE_F32) {
        store8(c.param, i0 >> 3, SHAMPOO_DTYPE_F32, p);
        if (c.copy) store8(c.copy, i0 >> 3, ct, p);
      } else {
        unsigned w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = bf16_bits(p[2 * j], h[2 * j]) | (bf16_bits(p[2 * j + 1], h[2 * j + 1]) << 16);
        *(static_cast<uint4*>(c.param) + (i0 >> 3)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = i0 + 32 * j;
        if (i >= c.count) continue;
        static_cast<uint8_t*>(c.m)[i] = static_cast<uint8_t>(cm[j]);
        static_cast<uint8_t*>(c.v)[i] = static_cast<uint8_t>(cv[j]);
        if (pt == SHAMPOO_DTYPE_F32) {
          static_cast<float*>(c.param)[i] = p[j];
          if (c.copy) store1(c.copy, i, ct, p[j]);
        } else {
          static_cast<unsigned short*>(c.param)[i] = bf16_bits(p[j], h[j]);
        }
      }
    }
  }
  return worst;
}

// ---------------------------------------------------------------- the step

// Which: 0 every tensor has 32-bit moments, 1 every tensor has 8-bit ones, 2
// both occur.
template <int Which>
__global__ void __launch_bounds__(kListThreads) adamw_step_kernel(const AdamwChunk* __restrict__ chunks, int n_chunks,
                                                                  AdamwHeader* hdr, const AdamwArgs a) {
  Coefs k;
  k.coef = a.coef ? *a.coef : 1.0f;
  k.beta1 = a.beta1;
  k.beta2 = a.beta2;
  k.om1 = 1.0f - a.beta1;
  k.om2 = 1.0f - a.beta2;
  k.eps = a.eps;
  k.c1 = a.step ? a.c1 : hdr->c1;
  k.c2 = a.step ? a.c2 : hdr->c2;
  const int t = a.step ? a.step : hdr->t + 1;
  const float lr = a.lr_device ? *a.lr_device : a.lr;
  const bool skip = not_finite(k.coef);  // non-finite gradients: the step is not taken
  const unsigned base = key_word(key_word(key_word(0u, a.seed_lo), a.seed_hi), static_cast<unsigned>(t));
  unsigned worst = 0;
  if (!skip) {
    for (int i = blockIdx.x; i < n_chunks; i += gridDim.x) {
      const AdamwChunk c = chunks[i];
      k.lr = lr * c.lr_scale;
      k.decay = c.decay;
      const unsigned key =
          key_word(key_word(base, static_cast<unsigned>(c.tensor)), static_cast<unsigned>(c.elem >> 32));
      const bool eight = Which == 1 || (Which == 2 && (c.flags & kFlagEight));
      worst = max(worst, eight ? step8(c, k, key) : step32(c, k, key));
    }
  }
  if (worst >= 0x7f800000u) atomicOr(&hdr->bad, 1u);
  if (!last_block(&hdr->ticket) || threadIdx.x != 0) return;
  const unsigned bad = atomicExch(&hdr->bad, 0u);
  hdr->status = (bad || skip) ? kStatusNonFinite : 0u;
  if (skip) return;
  const double p1 = a.step ? a.pow1 : hdr->pow1 * static_cast<double>(a.beta1);
  const double p2 = a.step ? a.pow2 : hdr->pow2 * static_cast<double>(a.beta2);
  hdr->t = t;
  hdr->pow1 = p1;
  hdr->pow2 = p2;
  hdr->c1 = static_cast<float>(1.0 / (1.0 - p1 * static_cast<double>(a.beta1)));
  hdr->c2 = static_cast<float>(sqrt(1.0 / (1.0 - p2 * static_cast<double>(a.beta2))));
}

// ---------------------------------------------------------------- moments in and out

// From flat fp32 moments into the list's own: 8-bit tensors are rounded to
// nearest, 32-bit ones copied.
__global__ void __launch_bounds__(kListThreads) load_moments_kernel(const AdamwChunk* __restrict__ chunks,
                                                                    int n_chunks, AdamwHeader* hdr,
                                                                    const float* __restrict__ m_in,
                                                                    const float* __restrict__ v_in) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  unsigned worst = 0;
  for (int n = blockIdx.x; n < n_chunks; n += gridDim.x) {
    const AdamwChunk c = chunks[n];
    const float* fm = m_in + c.flat;
    const float* fv = v_in + c.flat;
    for (int b = warp * kQBlock; b < c.count; b += kListWarps * kQBlock) {
      const bool vec = (c.flags & kFlagVec) && b + kQBlock <= c.count;
      const int i0 = vec ? b + 8 * lane : b + lane, stride = vec ? 1 : 32;
      float m[8], v[8];
      if (vec) {
        Raw8 rm, rv;
        load32B(fm + i0, rm.w);
        load32B(fv + i0, rv.w);
#pragma unroll
        for (int j = 0; j < 8; ++j) m[j] = __uint_as_float(rm.w[j]), v[j] = __uint_as_float(rv.w[j]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const bool in = i0 + 32 * j < c.count;
          m[j] = in ? fm[i0 + 32 * j] : 0.0f;
          v[j] = in ? fv[i0 + 32 * j] : 0.0f;
        }
      }
      unsigned mmax = 0, rmax = 0;
      float r[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        r[j] = __fsqrt_rn(v[j]);
        mmax = max(mmax, magnitude(m[j]));
        rmax = max(rmax, magnitude(r[j]));
      }
      worst = max(worst, max(mmax, rmax));
      if (!(c.flags & kFlagEight)) {
        if (vec) {
          store8(c.m, i0 >> 3, SHAMPOO_DTYPE_F32, m);
          store8(c.v, i0 >> 3, SHAMPOO_DTYPE_F32, v);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (i0 + 32 * j < c.count) {
              static_cast<float*>(c.m)[i0 + 32 * j] = m[j];
              static_cast<float*>(c.v)[i0 + 32 * j] = v[j];
            }
        }
        continue;
      }
      const int mi = m8_scale(__reduce_max_sync(0xffffffffu, mmax));
      const int vi = v8_scale(__reduce_max_sync(0xffffffffu, rmax));
      const float mu = inverse_scale(mi), vu = inverse_scale(vi);
      unsigned cm[8], cv[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        cm[j] = m8_nearest(m[j], mu);
        cv[j] = v8_nearest(r[j], vu);
      }
      if (lane == 0) {
        c.m_scale[b >> 8] = static_cast<uint8_t>(mi);
        c.v_scale[b >> 8] = static_cast<uint8_t>(vi);
      }
      if (vec) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(c.m) + i0) = make_uint2(pack4(cm), pack4(cm + 4));
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(c.v) + i0) = make_uint2(pack4(cv), pack4(cv + 4));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (i0 + stride * j < c.count) {
            static_cast<uint8_t*>(c.m)[i0 + stride * j] = static_cast<uint8_t>(cm[j]);
            static_cast<uint8_t*>(c.v)[i0 + stride * j] = static_cast<uint8_t>(cv[j]);
          }
      }
    }
  }
  if (worst >= 0x7f800000u) atomicOr(&hdr->status, kStatusNonFinite);
}

// The list's moments as flat fp32 or bf16 values; what lies behind a tensor's
// end, up to the next multiple of kQBlock, is written as zeros.
__global__ void __launch_bounds__(kListThreads) read_moments_kernel(const AdamwChunk* __restrict__ chunks,
                                                                    int n_chunks, void* m_out, void* v_out,
                                                                    int dtype) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t size = dtype == SHAMPOO_DTYPE_F32 ? 4 : 2;
  for (int n = blockIdx.x; n < n_chunks; n += gridDim.x) {
    const AdamwChunk c = chunks[n];
    void* om = static_cast<char*>(m_out) + size * c.flat;
    void* ov = static_cast<char*>(v_out) + size * c.flat;
    for (int b = warp * kQBlock; b < c.count; b += kListWarps * kQBlock) {
      const int i0 = b + 8 * lane;
      const bool vec = (c.flags & kFlagVec) && b + kQBlock <= c.count;
      float m[8], v[8];
      if (c.flags & kFlagEight) {
        unsigned cm[2] = {0, 0}, cv[2] = {0, 0};
        if (vec) {
          const uint2 qm = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(c.m) + i0);
          const uint2 qv = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(c.v) + i0);
          cm[0] = qm.x, cm[1] = qm.y, cv[0] = qv.x, cv[1] = qv.y;
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (i0 + j < c.count) {
              cm[j >> 2] |= static_cast<unsigned>(static_cast<const uint8_t*>(c.m)[i0 + j]) << (8 * (j & 3));
              cv[j >> 2] |= static_cast<unsigned>(static_cast<const uint8_t*>(c.v)[i0 + j]) << (8 * (j & 3));
            }
        }
        const float mf = m8_factor(c.m_scale[b >> 8]), vf = v8_factor(c.v_scale[b >> 8]);
        m8_values4(cm[0], mf, m);
        m8_values4(cm[1], mf, m + 4);
        v8_values4(cv[0], vf, v);
        v8_values4(cv[1], vf, v + 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(v[j], v[j]);
      } else if (vec) {
        Raw8 rm, rv;
        load32B(static_cast<const float*>(c.m) + i0, rm.w);
        load32B(static_cast<const float*>(c.v) + i0, rv.w);
#pragma unroll
        for (int j = 0; j < 8; ++j) m[j] = __uint_as_float(rm.w[j]), v[j] = __uint_as_float(rv.w[j]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          m[j] = i0 + j < c.count ? static_cast<const float*>(c.m)[i0 + j] : 0.0f;
          v[j] = i0 + j < c.count ? static_cast<const float*>(c.v)[i0 + j] : 0.0f;
        }
      }
      if (!vec) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (i0 + j >= c.count) m[j] = v[j] = 0.0f;
      }
      store8(om, i0 >> 3, dtype, m);
      store8(ov, i0 >> 3, dtype, v);
    }
  }
}

}  // namespace

int adamw_blocks(int which) {
  switch (which) {
    case 0: return resident_blocks(adamw_step_kernel<0>);
    case 1: return resident_blocks(adamw_step_kernel<1>);
    case 2: return resident_blocks(adamw_step_kernel<2>);
    case 3: return resident_blocks(load_moments_kernel);
    default: return resident_blocks(read_moments_kernel);
  }
}

void launch_adamw(const AdamwChunk* chunks, int n, int which, int grid, AdamwHeader* hdr, const AdamwArgs& a,
                  cudaStream_t st) {
  if (which == 0) adamw_step_kernel<0><<<grid, kListThreads, 0, st>>>(chunks, n, hdr, a);
  else if (which == 1) adamw_step_kernel<1><<<grid, kListThreads, 0, st>>>(chunks, n, hdr, a);
  else adamw_step_kernel<2><<<grid, kListThreads, 0, st>>>(chunks, n, hdr, a);
  prof_count_launch();
}

void launch_load_moments(const AdamwChunk* chunks, int n, int grid, AdamwHeader* hdr, const float* m, const float* v,
                         cudaStream_t st) {
  load_moments_kernel<<<grid, kListThreads, 0, st>>>(chunks, n, hdr, m, v);
  prof_count_launch();
}

void launch_read_moments(const AdamwChunk* chunks, int n, int grid, void* m, void* v, int dtype, cudaStream_t st) {
  read_moments_kernel<<<grid, kListThreads, 0, st>>>(chunks, n, m, v, dtype);
  prof_count_launch();
}

}  // namespace dash
