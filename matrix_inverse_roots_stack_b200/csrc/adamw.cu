// AdamW over a list of tensors in one launch, with moments in 32 or 8 bits,
// and the 8-bit moments' way in and out (include/dash_b200.h has the
// formulas and the formats).
//
// All of it streams through HBM once.  A warp takes a block of 256
// consecutive elements at a time, eight to a lane, so that a block of 8-bit
// moments belongs to one warp: its maximum is one warp reduction and never
// leaves registers.  HBM is the bound with 32-bit moments (28 bytes an
// element); with 8-bit ones (10 to 16 bytes) the instructions count as much:
// at the copy rate an SM has about 55 issue slots for an element of 10 bytes.
// Hence products and sums two at a time (f32x2), codes that are cut out of
// fp32 bit patterns instead of converted, three-operand maxima, and loads
// that are taken off the warps that compute (adamw_step).
//
// The moments' products and sums are rounded one by one (no contraction), so
// that their 8-bit codes do not depend on how a compiler fuses them.  Packed
// products and sums are fused by the assembler even where each asks for its
// own rounding, so the sums are written as a b + c with a 1 that it does not
// know to be one (AdamwArgs::one).
#include <atomic>

#include "adamw.cuh"
#include "launch_util.cuh"
#include "profile.cuh"

namespace dash {
namespace {

// ---------------------------------------------------------------- two fp32 numbers at a time

typedef unsigned long long f32x2;

__device__ __forceinline__ f32x2 pack2(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ f32x2 both(float a) { return pack2(a, a); }
__device__ __forceinline__ float low(f32x2 a) { return __uint_as_float(static_cast<unsigned>(a)); }
__device__ __forceinline__ float high(f32x2 a) { return __uint_as_float(static_cast<unsigned>(a >> 32)); }
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// Square roots of v >= 0, and a reciprocal within 2^-23 whose operand is
// normal, as the smallest adam_eps sees to.
//
// root: within 2^-23; below fp32's normal range v counts as 0.
// root2: rounded to nearest, but for about one number in a million, by
// Markstein's correction of an approximation (P. Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990): with y
// near 1 / sqrt(v) and s = v y, the remainder v - s^2 is exact in a fused
// product, and s + (v - s^2) y / 2 is off by the product of two errors before
// it is rounded.  8-bit moments take this one: their codes then are those of
// the correctly rounded root.  (The operand's floor keeps v = 0 at 0; below
// the normal range the root comes out smaller, and an infinite v's is NaN,
// which the step sees to.)
__device__ __forceinline__ float root(float v) {
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float inverse_root(float v) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaxf(v, 0x1p-126f)));
  return r;
}
__device__ __forceinline__ f32x2 root2(f32x2 v) {
  const f32x2 y = pack2(inverse_root(low(v)), inverse_root(high(v)));
  const f32x2 s = mul2(v, y);
  return fma2(fma2(s ^ 0x8000000080000000ull, s, v), mul2(y, both(0.5f)), s);
}
__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// max(a, |b|, |c|), NaN when one of them is.
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.abs.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

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
// x: the element's index (low half) times kWeyl, plus a key of the seed, the
// step, the tensor and the index's high half.  The upper 16 bits round m, the
// lower 16 v.
__device__ __forceinline__ unsigned draw_bits(unsigned x) {
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
constexpr int kM8Shift = 4, kV8Shift = 5;  // bring the code into the pattern's top byte

// Scale byte i of a block, standing for 2^(i - 127): the smallest that brings
// the block's maximum within the format (448 = 1.75 2^8, 31744 = 1.9375
// 2^14).  255: the maximum is not finite, and the block reads back so,
// whatever its codes.  What is kept of the scale is the exponent field of a
// float: (i + 8) << 23 or (i + 14) << 23.
__device__ __forceinline__ unsigned bits_of(float x) { return __float_as_uint(x); }
__device__ __forceinline__ float float_of(unsigned b) { return __uint_as_float(b); }
template <int kTop, unsigned kSlack>
struct BlockScale {
  unsigned e;
  __device__ __forceinline__ explicit BlockScale(float amax)
      : e(max((bits_of(amax) + kSlack) & 0xff800000u, (kTop + 1u) << 23)) {}
  // 1 / scale (of no use where the maximum is not finite)
  __device__ __forceinline__ float inverse() const { return float_of(((254u + kTop) << 23) - e); }
  __device__ __forceinline__ uint8_t byte(float amax) const {
    return static_cast<uint8_t>(not_finite(amax) ? 255u : (e >> 23) - kTop);
  }
};
typedef BlockScale<8, 0x1fffffu> M8Scale;
typedef BlockScale<14, 0x07ffffu> V8Scale;

// Code in the top byte.  x: bits of the scaled magnitude (or signed number),
// as above; y: the number itself; u: 16 random bits in bytes 1 and 2, so that
// x is rounded up where the dropped part and they reach a whole.
__device__ __forceinline__ unsigned m8_code(unsigned x, float y, unsigned u) {
  const unsigned c = (x << kM8Shift) + u;  // the sign is shifted out
  return (c & 0x7fffffffu) | (__float_as_uint(y) & 0x80000000u);
}
__device__ __forceinline__ unsigned v8_code(unsigned x, unsigned u) { return (x << kV8Shift) + u; }
// r > 0 is never stored as 0: beside a nonzero first moment a vanished
// second one would make the next update explode.  Four codes in one word:
// whether one is 0, and the codes with 1 in its place where r > 0, or
// everywhere ('all': a block that is not finite reads back as infinite).
__device__ __forceinline__ unsigned zero_bytes(unsigned w) { return (w - 0x01010101u) & ~w & 0x80808080u; }
__device__ __forceinline__ unsigned v8_floor(unsigned w, const f32x2* r, bool all) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float x = j & 1 ? high(r[j / 2]) : low(r[j / 2]);
    if ((all || x > 0.0f) && !(w & (0xffu << (8 * j)))) w |= 1u << (8 * j);
  }
  return w;
}
__device__ __forceinline__ unsigned top_bytes(unsigned a, unsigned b, unsigned c, unsigned d) {
  return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
}
// To nearest, ties to even: what to add for that.
__device__ __forceinline__ unsigned nearest_even(unsigned x, int shift) {
  return 0x7fffffu + ((x >> (24 - shift)) & 1u);
}

// Decoding goes through fp16, two codes at a time: there is an instruction
// for e4m3, and e4m4 lies inside e5m10 up to the exponent's bias, 2^14, which
// goes into the block's factor.  (A block of zeros that no kernel has written
// has scale 0 and codes 0.)
__device__ __forceinline__ float m8_factor(int i) { return __int_as_float(i << 23); }  // infinite for 255
__device__ __forceinline__ float v8_factor(int i) { return __int_as_float(i << 23) * 0x1p14f; }
__device__ __forceinline__ f32x2 from_half2(unsigned w) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return pack2(f.x, f.y);
}
__device__ __forceinline__ void m8_values4(unsigned codes, f32x2 factor, f32x2* m) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    unsigned w;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(w) : "h"(static_cast<unsigned short>(codes >> (16 * h))));
    m[h] = mul2(from_half2(w), factor);
  }
}
__device__ __forceinline__ void v8_values4(unsigned codes, f32x2 factor, f32x2* r) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
    r[h] = mul2(from_half2(__byte_perm(codes, 0, h ? 0x4342 : 0x4140) << 6), factor);
}

// ---------------------------------------------------------------- the list's blocks

// The tensor that unit 'b' (a block or tile) belongs to, at or behind tensor
// 'at': 'first' holds the n tensors' first units.  Whole warp, 32 tensors at
// a time.
__device__ __forceinline__ int find_tensor(const int* first, int n, int b, int at) {
  const int lane = threadIdx.x & 31;
  for (;;) {
    const int k = at + 1 + lane;
    const int c = __popc(__ballot_sync(0xffffffffu, k < n && __ldg(first + k) <= b));
    at += c;
    if (c < 32) return at;
  }
}

// The same from anywhere in the list: the search narrows 32 ways at a time.
__device__ __forceinline__ int first_tensor(const int* first, int n, int b) {
  const int lane = threadIdx.x & 31;
  int at = 0, span = n;
  while (span > 32) {
    const int step = (span + 31) / 32, k = at + lane * step;
    const int c = __popc(__ballot_sync(0xffffffffu, lane * step < span && __ldg(first + k) <= b));
    at += max(c - 1, 0) * step;
    span = min(step, n - at);
  }
  return find_tensor(first, n, b, at);
}

// ---------------------------------------------------------------- the step

// Scalars of a step that are not launch arguments.
struct Coefs {
  float coef, d1, d0, lr;
};
__device__ __forceinline__ f32x2 pair(float2 a) { return pack2(a.x, a.y); }

// bf16 pattern of a parameter, rounded by 16 random bits: where parameters
// have no fp32 master, rounding to nearest would drop every update below half
// a bf16 step (2^-9 of the value).
__device__ __forceinline__ unsigned bf16_up(float p, unsigned draw) {
  return __float_as_uint(p) + ((draw * kMulC) >> 16);  // its upper half
}
__device__ __forceinline__ unsigned bf16_not_finite(float p) {  // the upper half, a NaN kept one
  const unsigned b = __float_as_uint(p);
  return (b & 0x7fffffffu) > 0x7f800000u ? b | 0x400000u : b;
}

// Where a tile of a tensor lies: every pointer at its first element.
struct TileDesc {
  char* param;
  const char* grad;
  char* m;
  char* v;
  uint8_t* m_scale;
  uint8_t* v_scale;
  char* copy;
  int left;       // elements from there to the tensor's end, at most kTile; negative: no more tiles
  int flags;      // of the tensor
  unsigned key;   // of the rounding draws
  unsigned elem;  // index of the first element, low half
  float neg_lr, decay;
  int staged;     // the tile's data are in the ring
  int pad;
};
constexpr int kDescWords = sizeof(TileDesc) / 8;
static_assert(kDescWords == 11, "written as 8-byte words, one by each lane");

// A tile in shared memory: parameters, gradients, moments and, in 8 bits,
// scales, one behind the other.
__host__ __device__ constexpr int type_bytes(int dtype) { return dtype == SHAMPOO_DTYPE_F32 ? 4 : 2; }
__host__ __device__ constexpr int bulk_bytes(bool eight, int pt, int gt) {
  return kTile * (type_bytes(pt) + type_bytes(gt) + (eight ? 2 : 8));
}
__host__ __device__ constexpr int staged_bytes(bool eight, int pt, int gt) {
  return bulk_bytes(eight, pt, gt) + (eight ? 2 * kTileBlocks : 0);
}
template <bool kEight>
struct StagedAt {
  int grad, m, v, m_scale, v_scale;  // offsets; the parameters are at 0
  __device__ __forceinline__ StagedAt(int pt, int gt)
      : grad(kTile * type_bytes(pt)), m(grad + kTile * type_bytes(gt)), v(m + kTile * (kEight ? 1 : 4)),
        m_scale(v + kTile), v_scale(m_scale + kTileBlocks) {}  // the scales: 8 bits only
};

__device__ __forceinline__ void load8_shared(const unsigned char* base, int i, int dtype, Raw8& r) {
  if (dtype == SHAMPOO_DTYPE_F32) {
    const uint4 a = *reinterpret_cast<const uint4*>(base + 32 * i), b = *reinterpret_cast<const uint4*>(base + 32 * i + 16);
    r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w, r.w[4] = b.x, r.w[5] = b.y, r.w[6] = b.z, r.w[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(base + 16 * i);
    r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w;
  }
}

// How a block is read: from the ring's stage, from global memory eight
// elements to an access, or element by element (a short block, or a tensor
// without the alignment).
enum Access { kStaged, kVector, kScalar };

// One block of a tile, 'at' elements into it.  stage: the tile in shared
// memory, most: where its new maxima go, of which the fetching warp makes the
// scales (kStaged).  Returns whether a value in this lane is not finite.
// pt, gt: the tensor's types, constants where the caller has branched on them.
template <bool kEight, Access kAccess>
__device__ __forceinline__ bool step_block(const TileDesc& t, int pt, int gt, int at, const AdamwArgs& args,
                                           const Coefs& k, const unsigned char* stage, float2* most) {
  constexpr bool vec = kAccess != kScalar;
  const int lane = threadIdx.x & 31;
  const int ct = (t.flags >> kCopyShift) & 15;
  const int left = vec ? kQBlock : min(kQBlock, t.left - at);
  // this lane's elements: 8 lane + j of the block, or lane + 32 j
  constexpr int stride = vec ? 1 : 32;
  const int i0 = vec ? 8 * lane : lane;

  // where the block lies (of no use to kStaged, which reads shared memory)
  const char* grad = t.grad + at * (gt == SHAMPOO_DTYPE_F32 ? 4 : 2);
  const char* from = t.param + at * (pt == SHAMPOO_DTYPE_F32 ? 4 : 2);
  const char* m_from = t.m + at * (kEight ? 1 : 4);
  const char* v_from = t.v + at * (kEight ? 1 : 4);

  Raw8 rp, rg, rm, rv;
  f32x2 m[4], v[4], g[4], p[4], r[4];
  int ms = 0, vs = 0;
  if (kAccess == kStaged) {
    const int i = (at >> 3) + lane;
    const StagedAt<kEight> off(pt, gt);
    load8_shared(stage + off.grad, i, gt, rg);
    load8_shared(stage, i, pt, rp);
    if (kEight) {
      const uint2 qm = reinterpret_cast<const uint2*>(stage + off.m)[i], qv = reinterpret_cast<const uint2*>(stage + off.v)[i];
      rm.w[0] = qm.x, rm.w[1] = qm.y, rv.w[0] = qv.x, rv.w[1] = qv.y;
      ms = stage[off.m_scale + (at >> 8)];
      vs = stage[off.v_scale + (at >> 8)];
    } else {
      load8_shared(stage + off.m, i, SHAMPOO_DTYPE_F32, rm);
      load8_shared(stage + off.v, i, SHAMPOO_DTYPE_F32, rv);
    }
  } else if (kAccess == kVector) {
    load8(grad, lane, gt, rg);
    if (kEight) {
      const uint2 qm = *(reinterpret_cast<const uint2*>(m_from) + lane), qv = *(reinterpret_cast<const uint2*>(v_from) + lane);
      rm.w[0] = qm.x, rm.w[1] = qm.y, rv.w[0] = qv.x, rv.w[1] = qv.y;
      ms = t.m_scale[at >> 8];
      vs = t.v_scale[at >> 8];
    } else {
      load8(m_from, lane, SHAMPOO_DTYPE_F32, rm);
      load8(v_from, lane, SHAMPOO_DTYPE_F32, rv);
    }
    load8(from, lane, pt, rp);
  } else {
    if (kEight) {
      ms = t.m_scale[at >> 8];
      vs = t.v_scale[at >> 8];
      rm.w[0] = rm.w[1] = rv.w[0] = rv.w[1] = 0;
    }
    float x[8], y[8];
    load8_strided(grad, i0, left, gt, x);
    load8_strided(from, i0, left, pt, y);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      rg.w[j] = __float_as_uint(x[j]);
      rp.w[j] = __float_as_uint(y[j]);
    }
    unsigned char bm[8], bv[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = i0 + 32 * j;
      const bool in = i < left;
      if (kEight) {
        bm[j] = in ? static_cast<unsigned char>(m_from[i]) : 0;
        bv[j] = in ? static_cast<unsigned char>(v_from[i]) : 0;
      } else {
        rm.w[j] = in ? reinterpret_cast<const unsigned*>(m_from)[i] : 0u;
        rv.w[j] = in ? reinterpret_cast<const unsigned*>(v_from)[i] : 0u;
      }
    }
    if (kEight) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        rm.w[j >> 2] |= static_cast<unsigned>(bm[j]) << (8 * (j & 3));
        rv.w[j >> 2] |= static_cast<unsigned>(bv[j]) << (8 * (j & 3));
      }
    }
  }
  {
    float x[8], y[8];
    widen8(rg, vec ? gt : SHAMPOO_DTYPE_F32, x);
    widen8(rp, vec ? pt : SHAMPOO_DTYPE_F32, y);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      g[j] = pack2(x[2 * j], x[2 * j + 1]);
      p[j] = pack2(y[2 * j], y[2 * j + 1]);
    }
  }
  if (kEight) {
    const f32x2 mf = both(m8_factor(ms)), vf = both(v8_factor(vs));
    m8_values4(rm.w[0], mf, m);
    m8_values4(rm.w[1], mf, m + 2);
    v8_values4(rv.w[0], vf, r);
    v8_values4(rv.w[1], vf, r + 2);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = mul2(r[j], r[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      m[j] = pack2(__uint_as_float(rm.w[2 * j]), __uint_as_float(rm.w[2 * j + 1]));
      v[j] = pack2(__uint_as_float(rv.w[2 * j]), __uint_as_float(rv.w[2 * j + 1]));
    }
  }

  float mmax = 0.0f, rmax = 0.0f;
  f32x2 zero = 0ull;  // the sum of 0 p: NaN where a parameter is not finite
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const f32x2 gs2 = mul2(g[j], both(k.coef));
    m[j] = fma2(mul2(m[j], pair(args.beta1)), pair(args.one), mul2(gs2, pair(args.om1)));
    v[j] = fma2(mul2(v[j], pair(args.beta2)), pair(args.one), mul2(mul2(gs2, pair(args.om2)), gs2));
    r[j] = kEight ? root2(v[j]) : pack2(root(low(v[j])), root(high(v[j])));
    const f32x2 den = fma2(r[j], both(k.d1), both(k.d0));
    const f32x2 ratio = mul2(m[j], pack2(reciprocal(low(den)), reciprocal(high(den))));
    p[j] = fma2(both(t.neg_lr), fma2(both(t.decay), p[j], ratio), p[j]);
  }
  if (!vec) {  // nothing behind the tensor's end counts
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (i0 + 64 * j >= left) m[j] = v[j] = r[j] = p[j] = 0ull;
      if (i0 + 64 * j + 32 >= left) {
        m[j] &= 0xffffffffull, v[j] &= 0xffffffffull, r[j] &= 0xffffffffull, p[j] &= 0xffffffffull;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    mmax = max_abs3(mmax, low(m[j]), high(m[j]));
    rmax = kEight ? max_abs3(rmax, low(r[j]), high(r[j])) : max_abs3(rmax, low(v[j]), high(v[j]));
    zero = fma2(p[j], 0ull, zero);
  }
  if (kEight && not_finite(rmax)) {
    // v has overflowed, now or before: sqrt(v) is infinite, m / sqrt(v) is 0 and the update only the decay.  Rare, so
    // the parameters are read again here; a select in root2, for every element, made the step of GPT-2's tables 111.2
    // us instead of 110.1.
    float y[8];
    if (kAccess == kScalar) {
      load8_strided(from, i0, left, pt, y);
    } else {
      if (kAccess == kStaged) load8_shared(stage, (at >> 3) + lane, pt, rp);
      else load8(from, lane, pt, rp);
      widen8(rp, pt, y);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = j & 1 ? high(r[j / 2]) : low(r[j / 2]), mj = j & 1 ? high(m[j / 2]) : low(m[j / 2]);
      const float old = j & 1 ? high(p[j / 2]) : low(p[j / 2]);
      y[j] = x != x && !not_finite(mj) ? fmaf(t.neg_lr, t.decay * y[j], y[j]) : old;
    }
    zero = 0ull;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      p[j] = pack2(y[2 * j], y[2 * j + 1]);
      zero = fma2(p[j], 0ull, zero);
    }
  }
  const bool p_bad = low(zero) + high(zero) != 0.0f;
  const bool bad = p_bad || not_finite(max_abs3(0.0f, mmax, rmax));

  unsigned h[8];
  if (kEight || pt == SHAMPOO_DTYPE_BF16) {
    const unsigned x0 = (t.elem + at + i0) * kWeyl + t.key;
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = draw_bits(x0 + static_cast<unsigned>(stride * j) * kWeyl);
  }

  // the parameter leaves first: its registers are free for the codes
  float y[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) y[2 * j] = low(p[j]), y[2 * j + 1] = high(p[j]);
  char* param = t.param + at * (pt == SHAMPOO_DTYPE_F32 ? 4 : 2);
  if (pt == SHAMPOO_DTYPE_F32) {
    char* copy = t.copy ? t.copy + 2 * at : nullptr;
    if (vec) {
      store8<kAccess == kStaged>(param, lane, SHAMPOO_DTYPE_F32, y);
      if (copy) store8(copy, lane, ct, y);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i0 + 32 * j < left) {
          reinterpret_cast<float*>(param)[i0 + 32 * j] = y[j];
          if (copy) store1(copy, i0 + 32 * j, ct, y[j]);
        }
    }
  } else {
    unsigned w[8];
    if (__any_sync(0xffffffffu, p_bad)) {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = not_finite(y[j]) ? bf16_not_finite(y[j]) : bf16_up(y[j], h[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = bf16_up(y[j], h[j]);
    }
    if (vec) {
      *(reinterpret_cast<uint4*>(param) + lane) =
          make_uint4(__byte_perm(w[0], w[1], 0x7632), __byte_perm(w[2], w[3], 0x7632),
                     __byte_perm(w[4], w[5], 0x7632), __byte_perm(w[6], w[7], 0x7632));
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i0 + 32 * j < left) reinterpret_cast<unsigned short*>(param)[i0 + 32 * j] = static_cast<unsigned short>(w[j] >> 16);
    }
  }

  char* cm = t.m + at * (kEight ? 1 : 4);
  char* cv = t.v + at * (kEight ? 1 : 4);
  if (kEight) {
    mmax = warp_max(mmax);
    rmax = warp_max(rmax);
    const M8Scale mi(mmax);
    const V8Scale vi(rmax);
    const f32x2 mu = both(mi.inverse()), vu = both(vi.inverse());
    unsigned a[8], b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const f32x2 x = mul2(mul2(m[j / 2], mu), both(kM8Down)), y = mul2(mul2(r[j / 2], vu), both(kV8Down));
      const float xm = j & 1 ? high(x) : low(x), xr = j & 1 ? high(y) : low(y);
      const float mj = j & 1 ? high(m[j / 2]) : low(m[j / 2]);
      a[j] = m8_code(__float_as_uint(xm), mj, __byte_perm(h[j], 0, 0x4324));
      b[j] = v8_code(__float_as_uint(xr), __byte_perm(h[j], 0, 0x4104));
    }
    const uint2 am = make_uint2(top_bytes(a[0], a[1], a[2], a[3]), top_bytes(a[4], a[5], a[6], a[7]));
    uint2 bv = make_uint2(top_bytes(b[0], b[1], b[2], b[3]), top_bytes(b[4], b[5], b[6], b[7]));
    if (zero_bytes(bv.x) | zero_bytes(bv.y)) {
      bv.x = v8_floor(bv.x, r, not_finite(rmax));
      bv.y = v8_floor(bv.y, r + 2, not_finite(rmax));
    }
    if (kAccess == kStaged) {
      if (lane == 0) most[at >> 8] = make_float2(mmax, rmax);
    } else if (lane == 0) {
      t.m_scale[at >> 8] = mi.byte(mmax);
      t.v_scale[at >> 8] = vi.byte(rmax);
    }
    if (vec) {
      *(reinterpret_cast<uint2*>(cm) + lane) = am;
      *(reinterpret_cast<uint2*>(cv) + lane) = bv;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i0 + 32 * j < left) {
          cm[i0 + 32 * j] = static_cast<char>((j < 4 ? am.x : am.y) >> (8 * (j & 3)));
          cv[i0 + 32 * j] = static_cast<char>((j < 4 ? bv.x : bv.y) >> (8 * (j & 3)));
        }
    }
  } else if (vec) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      rm.w[2 * j] = __float_as_uint(low(m[j])), rm.w[2 * j + 1] = __float_as_uint(high(m[j]));
      rv.w[2 * j] = __float_as_uint(low(v[j])), rv.w[2 * j + 1] = __float_as_uint(high(v[j]));
    }
    if (kAccess == kStaged) {
      store32B_wide(reinterpret_cast<float*>(cm) + 8 * lane, rm.w);
      store32B_wide(reinterpret_cast<float*>(cv) + 8 * lane, rv.w);
    } else {
      store32B(reinterpret_cast<float*>(cm) + 8 * lane, rm.w);
      store32B(reinterpret_cast<float*>(cv) + 8 * lane, rv.w);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i0 + 32 * j < left) {
        reinterpret_cast<float*>(cm)[i0 + 32 * j] = j & 1 ? high(m[j / 2]) : low(m[j / 2]);
        reinterpret_cast<float*>(cv)[i0 + 32 * j] = j & 1 ? high(v[j / 2]) : low(v[j / 2]);
      }
  }

  return bad;
}

__device__ __forceinline__ Coefs step_coefs(const AdamwArgs& a, const AdamwHeader* hdr) {
  Coefs k;
  k.coef = a.coef ? *a.coef : 1.0f;
  k.lr = a.lr_device ? *a.lr_device : a.lr;
  k.d1 = a.step ? a.d1 : hdr->d1;
  k.d0 = a.step ? a.d0 : hdr->d0;
  return k;
}
__device__ __forceinline__ unsigned step_key(const AdamwArgs& a, int t) {
  return key_word(key_word(key_word(0u, a.seed_lo), a.seed_hi), static_cast<unsigned>(t));
}

// The last block of the grid writes the status word and, unless the step was
// skipped, moves the counter on.
__device__ __forceinline__ void finish_step(const AdamwArgs& a, AdamwHeader* hdr, int t, bool skip) {
  if (!last_block(&hdr->ticket) || threadIdx.x != 0) return;
  hdr->status = atomicExch(&hdr->bad, 0u) | (skip ? kStatusNonFinite : 0u);
  hdr->next = 0;
  if (skip) return;
  const double b1 = a.beta1.x, b2 = a.beta2.x;
  const double p1 = a.step ? a.pow1 : hdr->pow1 * b1, p2 = a.step ? a.pow2 : hdr->pow2 * b2;
  const double n1 = 1.0 - p1 * b1, n2 = 1.0 - p2 * b2;
  hdr->t = t;
  hdr->pow1 = p1;
  hdr->pow2 = p2;
  hdr->d1 = static_cast<float>(n1 / sqrt(n2));
  hdr->d0 = static_cast<float>(a.eps * n1);
}

__device__ __forceinline__ int param_type(const TileDesc& t) { return (t.flags >> kParamShift) & 15; }
__device__ __forceinline__ int grad_type(const TileDesc& t) { return (t.flags >> kGradShift) & 15; }
__device__ __forceinline__ bool vector_block(const TileDesc& t, int at) {
  return (t.flags & kFlagVec) && t.left - at >= kQBlock;
}

// A block of a staged tile, with its types as constants.
template <bool kEight>
__device__ __forceinline__ bool step_staged(const TileDesc& t, int at, const AdamwArgs& args, const Coefs& k,
                                            const unsigned char* stage, float2* most) {
  constexpr int f32 = SHAMPOO_DTYPE_F32, b16 = SHAMPOO_DTYPE_BF16, f16 = SHAMPOO_DTYPE_F16;
  const int gt = grad_type(t);
  if (param_type(t) == f32) {
    if (gt == f32) return step_block<kEight, kStaged>(t, f32, f32, at, args, k, stage, most);
    if (gt == b16) return step_block<kEight, kStaged>(t, f32, b16, at, args, k, stage, most);
    return step_block<kEight, kStaged>(t, f32, f16, at, args, k, stage, most);
  }
  if (gt == f32) return step_block<kEight, kStaged>(t, b16, f32, at, args, k, stage, most);
  if (gt == b16) return step_block<kEight, kStaged>(t, b16, b16, at, args, k, stage, most);
  return step_block<kEight, kStaged>(t, b16, f16, at, args, k, stage, most);
}

// Blocks that are not in shared memory, kept out of line.
template <int kBits>
__device__ __noinline__ bool step_direct(const TileDesc& t, int at, const AdamwArgs& args, const Coefs& k) {
  const int pt = param_type(t), gt = grad_type(t);
  if (kBits == 8 || (kBits == 0 && (t.flags & kFlagEight)))
    return vector_block(t, at) ? step_block<true, kVector>(t, pt, gt, at, args, k, nullptr, nullptr)
                               : step_block<true, kScalar>(t, pt, gt, at, args, k, nullptr, nullptr);
  return vector_block(t, at) ? step_block<false, kVector>(t, pt, gt, at, args, k, nullptr, nullptr)
                             : step_block<false, kScalar>(t, pt, gt, at, args, k, nullptr, nullptr);
}

// One block of threads an SM.  One of its warps fetches tiles of 16 blocks
// with bulk copies into a ring of stages in shared memory, ahead of the 19
// that compute.  It also forms and writes a finished tile's new scales: a byte
// for every block, written by its own warp, cost 7 to 10% of the step.  A tile
// that bulk copies cannot fetch (a tensor's short end, or other alignment) is
// only described in the ring, and read from global memory by the warps
// themselves.
//
// Long lists are dealt out from a counter, since SMs differ in how far from
// memory they are: with equal parts 32-bit steps took 10% longer.  See Deal.
// Equal parts and parts from the counter, fp32 with 32-bit moments, us in a
// graph: 8.3 tiles a block 28.9 and 28.4, 15.3 48.3 and 45.7, 17.3 53.7 and
// 50.6, 33.3 99.0 and 90.2, 512 1397 and 1263; with 8-bit moments the two are
// within 5% up to 15 tiles and within 2% beyond.  So a counter is ahead from
// 8 tiles on already, by 2 to 6% up to the border below.
//
// Tiles of one share, at 512 tiles a block, us: 1: 793 (8-bit, bf16), 937
// (8-bit, fp32) and 1252 (32-bit); 2: 753, 910, 1256; 4: 733, 884, 1263; 8:
// 734, 890, 1272.
constexpr int kRingWarps = 19;  // and the fetching one: 5 to a scheduler, 96 registers a thread
constexpr int kRingThreads = (kRingWarps + 1) * 32;
constexpr int kMaxStages = 4;
constexpr int kScaleLanes = 2 * kTileBlocks / 4;  // lanes of the fetching warp that fetch scales
constexpr int kLongList = 16;  // tiles a block, from which on they are dealt out
constexpr int kDeal = 4;       // tiles of one share
constexpr int kSmemLimit = 226 * 1024;  // of an SM's 227 KB; a little is static
struct Ring {
  TileDesc tile[kMaxStages];  // left < 0: no more tiles
  float2 most[kMaxStages][kTileBlocks];
  uint64_t full[kMaxStages];   // a tile is there
  uint64_t empty[kMaxStages];  // every warp is done with it
  int abort;
};
constexpr int kRingHead = (sizeof(Ring) + 127) / 128 * 128;

__device__ __forceinline__ void give_up(Ring& ring, AdamwHeader* hdr) {
  *const_cast<volatile int*>(&ring.abort) = 1;
  atomicOr(&hdr->bad, kStatusTimeout);
}

// The new scales of a staged tile: lanes 0 to 15 have a block's of m, the
// others of v.  old_scale: where this lane's goes, or null; 'most': the
// block's maxima.
__device__ __forceinline__ uint8_t* old_scale(const TileDesc& t) {
  const int lane = threadIdx.x & 31;
  uint8_t* to = lane < kTileBlocks ? t.m_scale + lane : t.v_scale + (lane - kTileBlocks);
  return t.staged && (t.flags & kFlagEight) ? to : nullptr;
}
__device__ __forceinline__ void write_scale(uint8_t* to, float2 most) {
  *to = (threadIdx.x & 31) < kTileBlocks ? M8Scale(most.x).byte(most.x) : V8Scale(most.y).byte(most.y);
}

// A long list's tiles, dealt to the grid's blocks: share p < 'whole' is kDeal
// tiles, a grid's width apart, so that blocks that run side by side read side
// by side (kDeal tiles in a row, all blocks a multiple of that apart, cost
// 8%); the last four to eight grids' width of tiles are shares of one tile.
struct Deal {
  int grid, whole, tile, left;  // tile: the current one; left: tiles behind it in its share
  __device__ __forceinline__ Deal(int n_tiles, int grid) : grid(grid), whole((n_tiles / (kDeal * grid) - 1) * grid) {}
  __device__ __forceinline__ void take(int p) {
    const bool single = p >= whole;
    tile = single ? kDeal * whole + (p - whole) : p / grid * (kDeal * grid) + p % grid;
    left = single ? 0 : kDeal - 1;
  }
};

// One tensor's arrays as the lanes of the fetching warp see them: lanes 0 to 6
// have one pointer each, in the order of AdamwTensorDev and TileDesc.
struct Arrays {
  char* at;            // lane's array
  unsigned rate;       // its bytes for 256 elements
  unsigned to, bytes;  // where a tile of it goes in a stage, and its size; 0: not copied in bulk
  long long n;
  int first_tile, flags;
  unsigned tensor_key, key;
  int high;            // of the element's index, for which 'key' is
  float neg_lr, decay;
};
__device__ __forceinline__ Arrays arrays_of(const AdamwTensorDev& t, float lr, unsigned base) {
  const int lane = threadIdx.x & 31;
  Arrays a;
  a.n = t.n;
  a.first_tile = t.first_tile;
  a.flags = t.flags;
  a.tensor_key = key_word(base, static_cast<unsigned>(t.index));
  a.key = key_word(a.tensor_key, 0u);
  a.high = 0;
  a.neg_lr = -(lr * t.lr_scale);
  a.decay = t.decay;
  const bool eight = t.flags & kFlagEight;
  const unsigned p = 256u * type_bytes((t.flags >> kParamShift) & 15), g = 256u * type_bytes((t.flags >> kGradShift) & 15);
  const unsigned m = eight ? 256u : 1024u;
  a.at = lane < 7 ? reinterpret_cast<char* const*>(&t)[lane] : nullptr;
  a.rate = lane == 0 ? p : lane == 1 ? g : lane < 4 ? m : lane < 6 ? 1u : 512u;
  const unsigned before = (lane > 0 ? p : 0u) + (lane > 1 ? g : 0u) + (lane > 2 ? m : 0u) + (lane > 3 ? m : 0u) + (lane > 4 ? 1u : 0u);
  a.to = before * (kTile / 256);
  a.bytes = lane < 4 ? a.rate * (kTile / 256) : 0u;
  return a;
}

// One warp: tiles from the list to the ring, and their scales back.  Stage s
// gets its i-th tile when the warps have emptied it of the one before.  What
// is issued here is done in few, wide steps: among 19 busy warps an
// instruction of this one takes a dozen cycles, and a tile has under 3000.
__device__ __forceinline__ void fetch_tiles(const AdamwTable& table, Ring& ring, unsigned char* stages, int n_stages,
                                            int stride, float lr, unsigned base, bool withhold, AdamwHeader* hdr) {
  const int lane = threadIdx.x & 31, grid = gridDim.x;
  const bool dealt = table.n_tiles / kLongList >= grid;
  Deal deal(table.n_tiles, grid);
  deal.take(blockIdx.x);
  int tile = dealt ? deal.tile : blockIdx.x, next = 0;
  bool ask = true;  // at the first tile of a share, or of all
  int at = -1, s = 0;
  unsigned i = 0;  // the ring's turn
  bool ok = true, more = true;
  Arrays a;
  while (more) {
    more = tile < table.n_tiles;
    unsigned long long word = lane == 7 ? 0xffffffffull : 0ull;  // this lane's of the description; left: -1
    bool staged = false;
    char* from = nullptr;
    if (more) {
      // the next share, looked at when this one is through: asked for and awaited tile by tile it cost 10%
      if (dealt && ask && lane == 0) next = static_cast<int>(atomicAdd(&hdr->next, 1u));
      if (at < 0 || tile < a.first_tile || static_cast<long long>(tile - a.first_tile) * kTile >= a.n) {
        // another tensor; a new share may begin before the end of the last
        at = ask ? first_tensor(table.first_tile, table.n_tensors, tile)
                 : find_tensor(table.first_tile, table.n_tensors, tile, at);
        a = arrays_of(table.tensors[at], lr, base);
      }
      ask = false;
      const long long e0 = static_cast<long long>(tile - a.first_tile) * kTile;
      const int left = static_cast<int>(min(static_cast<long long>(kTile), a.n - e0)), high = static_cast<int>(e0 >> 32);
      if (high != a.high) {
        a.high = high;
        a.key = key_word(a.tensor_key, static_cast<unsigned>(high));
      }
      staged = (a.flags & kFlagWide) && left == kTile;
      from = a.at ? a.at + ((static_cast<unsigned long long>(e0) * a.rate) >> 8) : nullptr;
      const unsigned lo = lane == 7 ? left : lane == 8 ? a.key : lane == 9 ? __float_as_uint(a.neg_lr) : staged;
      const unsigned hi = lane == 7 ? a.flags : lane == 8 ? static_cast<unsigned>(e0) : lane == 9 ? __float_as_uint(a.decay) : 0u;
      word = lane < 7 ? reinterpret_cast<unsigned long long>(from) : lo | (static_cast<unsigned long long>(hi) << 32);
    }
    uint8_t* scale = nullptr;  // of the stage's old tile
    float2 most;
    if (i > 0) {
      ok = __all_sync(0xffffffffu, mbar_wait_sleep(&ring.empty[s], (i - 1) & 1, &ring.abort));
      if (!ok) break;
      scale = old_scale(ring.tile[s]);
      most = ring.most[s][lane & (kTileBlocks - 1)];
      __syncwarp();
    }
    if (lane < kDescWords) reinterpret_cast<unsigned long long*>(&ring.tile[s])[lane] = word;
    __syncwarp();
    uint64_t* bar = &ring.full[s];
    unsigned char* to = stages + s * stride;
    if (lane == 0) {
      if (staged) mbar_arrive_expect_tx(bar, bulk_bytes(a.flags & kFlagEight, (a.flags >> kParamShift) & 15, (a.flags >> kGradShift) & 15));
      else mbar_arrive(bar);
    }
    __syncwarp();
    if (staged && a.bytes && !withhold) bulk_load(to + a.to, from, a.bytes, bar);
    // the scales, 16 bytes of m's and 16 of v's, four to a lane: a scale array need not be aligned for bulk copies
    const unsigned long long at_m = __shfl_sync(0xffffffffu, word, 4), at_v = __shfl_sync(0xffffffffu, word, 5);
    const unsigned at_scales = __shfl_sync(0xffffffffu, a.to, 4);
    if (lane < kScaleLanes) {
      if (staged && (a.flags & kFlagEight))
        copy4_async(to + at_scales + 4 * lane, reinterpret_cast<const char*>(lane < 4 ? at_m : at_v) + 4 * (lane & 3));
      arrive_behind_copies(bar);
    }
    if (scale) write_scale(scale, most);
    __syncwarp();
    if (!dealt || deal.left-- > 0) {
      tile += grid;
    } else {
      deal.take(grid + __shfl_sync(0xffffffffu, next, 0));
      tile = deal.tile;
      ask = true;
    }
    if (++s == n_stages) s = 0, ++i;
  }
  // the stages behind the last tile's, in turn: what is still in them is finished
  for (int j = 1; ok && j < n_stages; ++j) {
    if (i > 0) {
      ok = __all_sync(0xffffffffu, mbar_wait_sleep(&ring.empty[s], (i - 1) & 1, &ring.abort));
      uint8_t* scale = ok ? old_scale(ring.tile[s]) : nullptr;
      if (scale) write_scale(scale, ring.most[s][lane & (kTileBlocks - 1)]);
    }
    if (++s == n_stages) s = 0, ++i;
  }
  if (!ok) {
    give_up(ring, hdr);
    // copies in flight land before the block ends: each stage's last tile, of this turn or the one before
    int never = 0;
    for (int j = 0; j < n_stages && !withhold; ++j) {
      const int turn = static_cast<int>(i) - (j < s ? 0 : 1);
      if (turn >= 0 && !mbar_wait(&ring.full[j], turn & 1, &never)) break;
    }
  }
}

// kBits: 32 or 8, where all of the list's moments have them, or 0 for both.
template <int kBits>
__device__ __forceinline__ void adamw_step(const AdamwTable& table, AdamwHeader* hdr, const AdamwArgs& a,
                                           int n_stages, int stride) {
  extern __shared__ unsigned char raw[];
  Ring& ring = *reinterpret_cast<Ring*>((reinterpret_cast<uintptr_t>(raw) + 127) & ~static_cast<uintptr_t>(127));
  unsigned char* stages = reinterpret_cast<unsigned char*>(&ring) + kRingHead;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Coefs k = step_coefs(a, hdr);
  const int t = a.step ? a.step : hdr->t + 1;
  const bool skip = not_finite(k.coef);  // non-finite gradients: the step is not taken
  if (threadIdx.x == 0) {
    for (int s = 0; s < n_stages; ++s) {
      mbar_init(&ring.full[s], 1 + kScaleLanes);
      mbar_init(&ring.empty[s], kRingWarps);
    }
    ring.abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  if (!skip && warp == kRingWarps) {
    fetch_tiles(table, ring, stages, n_stages, stride, k.lr, step_key(a, t), a.withhold, hdr);
  } else if (!skip) {
    // the tiles' blocks are dealt to the warps one after another; every warp waits for every tile and arrives when
    // done with it, also where it has no block, so that a stage's phases cannot run ahead of a warp
    bool bad = false;
    unsigned parity = 0;
    for (int s = 0, i = warp;;) {
      const bool ok = mbar_wait(&ring.full[s], parity, &ring.abort);
      if (!__all_sync(0xffffffffu, ok)) {
        give_up(ring, hdr);
        break;
      }
      const TileDesc& d = ring.tile[s];
      if (d.left < 0) break;
      for (; i < kTileBlocks; i += kRingWarps) {
        const int at = i * kQBlock;
        const bool eight = kBits == 8 || (kBits == 0 && (d.flags & kFlagEight));
        if (d.staged) {
          bad |= eight ? step_staged<true>(d, at, a, k, stages + s * stride, ring.most[s])
                       : step_staged<false>(d, at, a, k, stages + s * stride, nullptr);
        } else if (at < d.left) {
          bad |= step_direct<kBits>(d, at, a, k);
        }
      }
      i -= kTileBlocks;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ring.empty[s]);
      if (++s == n_stages) s = 0, parity ^= 1;
    }
    if (bad) atomicOr(&hdr->bad, kStatusNonFinite);
  }
  finish_step(a, hdr, t, skip);
}

__global__ void __launch_bounds__(kRingThreads, 1) adamw32_kernel(const __grid_constant__ AdamwTable table,
                                                                  AdamwHeader* hdr,
                                                                  const __grid_constant__ AdamwArgs a, int n_stages,
                                                                  int stride) {
  adamw_step<32>(table, hdr, a, n_stages, stride);
}
__global__ void __launch_bounds__(kRingThreads, 1) adamw8_kernel(const __grid_constant__ AdamwTable table,
                                                                 AdamwHeader* hdr,
                                                                 const __grid_constant__ AdamwArgs a, int n_stages,
                                                                 int stride) {
  adamw_step<8>(table, hdr, a, n_stages, stride);
}
__global__ void __launch_bounds__(kRingThreads, 1) adamw_mixed_kernel(const __grid_constant__ AdamwTable table,
                                                                      AdamwHeader* hdr,
                                                                      const __grid_constant__ AdamwArgs a,
                                                                      int n_stages, int stride) {
  adamw_step<0>(table, hdr, a, n_stages, stride);
}

// Lists of no more tiles than the device has SMs: a block of threads to a
// tile, a warp to a block of elements, straight from global memory.  There is
// nothing to fetch ahead, and the ring would only be in the way: 49 vectors
// of 2048 take 5.3 instead of 6.9 us (in a graph), 148 tiles 6.2 instead of
// 7.2; from two tiles an SM on the ring is faster (296 tiles: 8.3 against 9.9
// us, 1184: 16.7 against 31.8).
constexpr int kDirectThreads = kTileBlocks * 32;

__global__ void __launch_bounds__(kDirectThreads) adamw_direct_kernel(const AdamwTable table, AdamwHeader* hdr,
                                                                      const __grid_constant__ AdamwArgs a) {
  const Coefs k = step_coefs(a, hdr);
  const int t = a.step ? a.step : hdr->t + 1;
  const bool skip = not_finite(k.coef);
  const int tile = blockIdx.x, at = (threadIdx.x >> 5) * kQBlock;
  if (!skip && tile < table.n_tiles) {
    const AdamwTensorDev& here = table.tensors[first_tensor(table.first_tile, table.n_tensors, tile)];
    const long long e0 = static_cast<long long>(tile - here.first_tile) * kTile;
    if (e0 + at < here.n) {
      const int flags = here.flags, pt = (flags >> kParamShift) & 15, gt = (flags >> kGradShift) & 15;
      const bool eight = flags & kFlagEight;
      TileDesc d;
      d.param = static_cast<char*>(here.param) + e0 * type_bytes(pt);
      d.grad = static_cast<const char*>(here.grad) + e0 * type_bytes(gt);
      d.m = static_cast<char*>(here.m) + e0 * (eight ? 1 : 4);
      d.v = static_cast<char*>(here.v) + e0 * (eight ? 1 : 4);
      d.m_scale = here.m_scale + (e0 >> 8);
      d.v_scale = here.v_scale + (e0 >> 8);
      d.copy = here.copy ? static_cast<char*>(here.copy) + 2 * e0 : nullptr;
      d.left = static_cast<int>(min(static_cast<long long>(kTile), here.n - e0));
      d.flags = flags;
      d.key = key_word(key_word(step_key(a, t), static_cast<unsigned>(here.index)), static_cast<unsigned>(e0 >> 32));
      d.elem = static_cast<unsigned>(e0);
      d.neg_lr = -(k.lr * here.lr_scale);
      d.decay = here.decay;
      bool bad;
      if (vector_block(d, at)) bad = eight ? step_block<true, kVector>(d, pt, gt, at, a, k, nullptr, nullptr) : step_block<false, kVector>(d, pt, gt, at, a, k, nullptr, nullptr);
      else bad = eight ? step_block<true, kScalar>(d, pt, gt, at, a, k, nullptr, nullptr) : step_block<false, kScalar>(d, pt, gt, at, a, k, nullptr, nullptr);
      if (bad) atomicOr(&hdr->bad, kStatusNonFinite);
    }
  }
  finish_step(a, hdr, t, skip);
}

// ---------------------------------------------------------------- moments in and out

// From flat fp32 moments into the list's own: 8-bit tensors are rounded to
// nearest, 32-bit ones copied.  One block of threads to a tile, here and
// below; a warp has two blocks and asks for both before it uses either.
constexpr int kLoadBlocks = kTileBlocks / kListWarps;

__global__ void __launch_bounds__(kListThreads) load_moments_kernel(const AdamwTable table, AdamwHeader* hdr,
                                                                    const float* __restrict__ m_in,
                                                                    const float* __restrict__ v_in) {
  const int lane = threadIdx.x & 31;
  const AdamwTensorDev& t = table.tensors[first_tensor(table.first_tile, table.n_tensors, static_cast<int>(blockIdx.x))];
  const long long first = static_cast<long long>(static_cast<int>(blockIdx.x) - t.first_tile) * kTile +
                          (threadIdx.x >> 5) * kQBlock;
  const long long flat = static_cast<long long>(t.first) * kQBlock;
  const bool vec = t.flags & kFlagVec, eight = t.flags & kFlagEight;
  float m[kLoadBlocks][8], v[kLoadBlocks][8];
#pragma unroll
  for (int w = 0; w < kLoadBlocks; ++w) {
    const long long e0 = first + w * (kListWarps * kQBlock);
    const float* fm = m_in + flat + e0;
    const float* fv = v_in + flat + e0;
    if (vec && e0 + kQBlock <= t.n) {
      Raw8 rm, rv;
      load32B(fm + 8 * lane, rm.w);
      load32B(fv + 8 * lane, rv.w);
#pragma unroll
      for (int j = 0; j < 8; ++j) m[w][j] = __uint_as_float(rm.w[j]), v[w][j] = __uint_as_float(rv.w[j]);
    } else {
      const int left = static_cast<int>(min(static_cast<long long>(kQBlock), max(t.n - e0, 0ll)));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool in = lane + 32 * j < left;
        m[w][j] = in ? fm[lane + 32 * j] : 0.0f;
        v[w][j] = in ? fv[lane + 32 * j] : 0.0f;
      }
    }
  }
  bool bad = false;
#pragma unroll
  for (int w = 0; w < kLoadBlocks; ++w) {
    const long long e0 = first + w * (kListWarps * kQBlock);
    if (e0 >= t.n) break;
    const bool whole = vec && e0 + kQBlock <= t.n;
    const int left = static_cast<int>(min(static_cast<long long>(kQBlock), t.n - e0));
    float mmax = 0.0f, rmax = 0.0f, r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = __fsqrt_rn(v[w][j]);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      mmax = max_abs3(mmax, m[w][j], m[w][j + 1]);
      rmax = max_abs3(rmax, r[j], r[j + 1]);
    }
    bad |= not_finite(max_abs3(mmax, rmax, 0.0f));
    if (eight) {
      uint8_t* cm = static_cast<uint8_t*>(t.m) + e0;
      uint8_t* cv = static_cast<uint8_t*>(t.v) + e0;
      mmax = warp_max(mmax);
      rmax = warp_max(rmax);
      const M8Scale mi(mmax);
      const V8Scale vi(rmax);
      const float mu = mi.inverse(), vu = vi.inverse();
      unsigned ca[8], cb[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const unsigned x = __float_as_uint(__fmul_rn(__fmul_rn(m[w][j], mu), kM8Down));
        const unsigned y = __float_as_uint(__fmul_rn(__fmul_rn(r[j], vu), kV8Down));
        ca[j] = m8_code(x, m[w][j], nearest_even(x, kM8Shift));
        cb[j] = v8_code(y, nearest_even(y, kV8Shift));
      }
      const uint2 am = make_uint2(top_bytes(ca[0], ca[1], ca[2], ca[3]), top_bytes(ca[4], ca[5], ca[6], ca[7]));
      uint2 bv = make_uint2(top_bytes(cb[0], cb[1], cb[2], cb[3]), top_bytes(cb[4], cb[5], cb[6], cb[7]));
      if (zero_bytes(bv.x) | zero_bytes(bv.y)) {
        const f32x2 r2[4] = {pack2(r[0], r[1]), pack2(r[2], r[3]), pack2(r[4], r[5]), pack2(r[6], r[7])};
        bv.x = v8_floor(bv.x, r2, not_finite(rmax));
        bv.y = v8_floor(bv.y, r2 + 2, not_finite(rmax));
      }
      if (lane == 0) {
        t.m_scale[e0 >> 8] = mi.byte(mmax);
        t.v_scale[e0 >> 8] = vi.byte(rmax);
      }
      if (whole) {
        *(reinterpret_cast<uint2*>(cm) + lane) = am;
        *(reinterpret_cast<uint2*>(cv) + lane) = bv;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (lane + 32 * j < left) {
            cm[lane + 32 * j] = static_cast<uint8_t>((j < 4 ? am.x : am.y) >> (8 * (j & 3)));
            cv[lane + 32 * j] = static_cast<uint8_t>((j < 4 ? bv.x : bv.y) >> (8 * (j & 3)));
          }
      }
    } else {
      float* om = static_cast<float*>(t.m) + e0;
      float* ov = static_cast<float*>(t.v) + e0;
      if (whole) {
        store8(om, lane, SHAMPOO_DTYPE_F32, m[w]);
        store8(ov, lane, SHAMPOO_DTYPE_F32, v[w]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (lane + 32 * j < left) {
            om[lane + 32 * j] = m[w][j];
            ov[lane + 32 * j] = v[w][j];
          }
      }
    }
  }
  if (bad) atomicOr(&hdr->status, kStatusNonFinite);
}

// The list's moments as flat fp32 or bf16 values; what lies behind a tensor's
// end, up to the next multiple of kQBlock, is written as zeros.  A warp has
// four blocks of the tile, and asks for all of their codes and scales before
// it uses any: 6 or 10 bytes an element are little to hide HBM's latency with.
constexpr int kReadBlocks = 4;
constexpr int kReadThreads = kTileBlocks / kReadBlocks * 32;

__device__ __forceinline__ void write_moments(const AdamwTensorDev& t, long long e0, f32x2* m, f32x2* v, bool squared,
                                              void* m_out, void* v_out, int dtype) {
  const int lane = threadIdx.x & 31, left = static_cast<int>(min(static_cast<long long>(kQBlock), t.n - e0));
  const size_t at = (dtype == SHAMPOO_DTYPE_F32 ? 4 : 2) * static_cast<size_t>(static_cast<long long>(t.first) * kQBlock + e0);
  float x[8], y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const bool in = 8 * lane + j < left;
    if (!squared && !(j & 1)) v[j / 2] = mul2(v[j / 2], v[j / 2]);
    x[j] = !in ? 0.0f : j & 1 ? high(m[j / 2]) : low(m[j / 2]);
    y[j] = !in ? 0.0f : j & 1 ? high(v[j / 2]) : low(v[j / 2]);
  }
  store8(static_cast<char*>(m_out) + at, lane, dtype, x);
  store8(static_cast<char*>(v_out) + at, lane, dtype, y);
}

__global__ void __launch_bounds__(kReadThreads) read_moments_kernel(const AdamwTable table, void* m_out, void* v_out,
                                                                    int dtype) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const AdamwTensorDev& t = table.tensors[first_tensor(table.first_tile, table.n_tensors, static_cast<int>(blockIdx.x))];
  const long long tile0 = static_cast<long long>(static_cast<int>(blockIdx.x) - t.first_tile) * kTile;
  const long long first = tile0 + warp * kQBlock;
  constexpr int kNext = kReadThreads / 32 * kQBlock;  // from a warp's block to its next
  f32x2 m[4], v[4];
  if ((t.flags & kFlagEight) && (t.flags & kFlagVec) && tile0 + kTile <= t.n) {
    uint2 qm[kReadBlocks], qv[kReadBlocks];
    int ms[kReadBlocks], vs[kReadBlocks];
#pragma unroll
    for (int w = 0; w < kReadBlocks; ++w) {
      const long long e0 = first + w * kNext;
      qm[w] = *(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.m) + e0) + lane);
      qv[w] = *(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.v) + e0) + lane);
      ms[w] = t.m_scale[e0 >> 8];
      vs[w] = t.v_scale[e0 >> 8];
    }
#pragma unroll
    for (int w = 0; w < kReadBlocks; ++w) {
      const f32x2 mf = both(m8_factor(ms[w])), vf = both(v8_factor(vs[w]));
      m8_values4(qm[w].x, mf, m);
      m8_values4(qm[w].y, mf, m + 2);
      v8_values4(qv[w].x, vf, v);
      v8_values4(qv[w].y, vf, v + 2);
      write_moments(t, first + w * kNext, m, v, false, m_out, v_out, dtype);
    }
    return;
  }
  for (int w = 0; w < kReadBlocks; ++w) {
    const long long e0 = first + w * kNext;
    if (e0 >= t.n) break;
    const int left = static_cast<int>(min(static_cast<long long>(kQBlock), t.n - e0)), i0 = 8 * lane;
    if (t.flags & kFlagEight) {
      const uint8_t* cm = static_cast<const uint8_t*>(t.m) + e0;
      const uint8_t* cv = static_cast<const uint8_t*>(t.v) + e0;
      unsigned am[2] = {0, 0}, av[2] = {0, 0};
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i0 + j < left) {
          am[j >> 2] |= static_cast<unsigned>(cm[i0 + j]) << (8 * (j & 3));
          av[j >> 2] |= static_cast<unsigned>(cv[i0 + j]) << (8 * (j & 3));
        }
      const f32x2 mf = both(m8_factor(t.m_scale[e0 >> 8])), vf = both(v8_factor(t.v_scale[e0 >> 8]));
      m8_values4(am[0], mf, m);
      m8_values4(am[1], mf, m + 2);
      v8_values4(av[0], vf, v);
      v8_values4(av[1], vf, v + 2);
    } else {
      const float* fm = static_cast<const float*>(t.m) + e0;
      const float* fv = static_cast<const float*>(t.v) + e0;
      Raw8 rm, rv;
      if ((t.flags & kFlagVec) && left == kQBlock) {
        load32B(fm + i0, rm.w);
        load32B(fv + i0, rv.w);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          rm.w[j] = i0 + j < left ? __float_as_uint(fm[i0 + j]) : 0u;
          rv.w[j] = i0 + j < left ? __float_as_uint(fv[i0 + j]) : 0u;
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        m[j] = pack2(__uint_as_float(rm.w[2 * j]), __uint_as_float(rm.w[2 * j + 1]));
        v[j] = pack2(__uint_as_float(rv.w[2 * j]), __uint_as_float(rv.w[2 * j + 1]));
      }
    }
    write_moments(t, e0, m, v, !(t.flags & kFlagEight), m_out, v_out, dtype);
  }
}

}  // namespace

int adamw_stage_bytes(bool eight, int param_dtype, int grad_dtype) {
  return (staged_bytes(eight, param_dtype, grad_dtype) + 127) / 128 * 128;
}

template <typename Kernel>
int prepare(Kernel kernel, std::atomic<unsigned long long>& done, AdamwLaunch* out) {
  if (smem_limit_once(kernel, kSmemLimit, done) != cudaSuccess) return SHAMPOO_ECUDA;
  out->step = resident_blocks(kernel, kRingThreads, out->smem);
  return SHAMPOO_OK;
}

int adamw_prepare(int bits, int stage_bytes, AdamwLaunch* out) {
  constexpr int kHead = kRingHead + 128;  // the kernel aligns to 128
  out->bits = bits;
  out->stages = std::min(kMaxStages, (kSmemLimit - kHead) / stage_bytes);
  out->stride = stage_bytes;
  out->smem = kHead + out->stages * stage_bytes;
  static std::atomic<unsigned long long> done[3];
  const int rc = bits == 32  ? prepare(adamw32_kernel, done[0], out)
                 : bits == 8 ? prepare(adamw8_kernel, done[1], out)
                             : prepare(adamw_mixed_kernel, done[2], out);
  if (rc) return rc;
  out->direct = out->step;
  return out->step < 0 ? SHAMPOO_ECUDA : SHAMPOO_OK;
}

void launch_adamw(const AdamwTable& t, const AdamwLaunch& l, int grid, AdamwHeader* hdr, const AdamwArgs& a,
                  cudaStream_t st) {
  if (t.n_tiles <= l.direct) adamw_direct_kernel<<<grid, kDirectThreads, 0, st>>>(t, hdr, a);
  else if (l.bits == 32) adamw32_kernel<<<grid, kRingThreads, l.smem, st>>>(t, hdr, a, l.stages, l.stride);
  else if (l.bits == 8) adamw8_kernel<<<grid, kRingThreads, l.smem, st>>>(t, hdr, a, l.stages, l.stride);
  else adamw_mixed_kernel<<<grid, kRingThreads, l.smem, st>>>(t, hdr, a, l.stages, l.stride);
  prof_count_launch();
}

void launch_load_moments(const AdamwTable& t, AdamwHeader* hdr, const float* m, const float* v, cudaStream_t st) {
  load_moments_kernel<<<t.n_tiles, kListThreads, 0, st>>>(t, hdr, m, v);
  prof_count_launch();
}

void launch_read_moments(const AdamwTable& t, void* m, void* v, int dtype, cudaStream_t st) {
  read_moments_kernel<<<t.n_tiles, kReadThreads, 0, st>>>(t, m, v, dtype);
  prof_count_launch();
}

}  // namespace dash
