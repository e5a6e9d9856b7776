// pvl_grad_norm, pvl_adamw_step: the norm of all gradients and the AdamW update
// of many tensors at once, with moments in 32 or in 8 bits, for sm_103a.
//
// With c = min(1, max_norm / norm) where a norm is given,
//   g' = c g,  m' = b1 m + (1 - b1) g',  v' = b2 v + (1 - b2) g'^2,
//   p' = p (1 - lr decay) - lr / (1 - b1^t) m' / (sqrt(v' / (1 - b2^t)) + eps).
// 1 - lr decay is the sum of two fp32 numbers, so that p is rounded once: one
// number would be 1, no decay, for lr decay below 2^-25, and 19 % off at 1e-7.
// The moments of all tensors lie in one buffer, each tensor from a whole block
// of 256 elements on (zeros after its end); so do fp32 masters of bf16
// parameters.  Parameters and gradients are wherever their tensors are.
//
// States in 8 bits: a block holds m and sqrt(v) as e4m3 values times one scale
// each, the block's largest magnitude / 448.  The root halves the range that
// v needs (e4m3 spans 2^-9 to 448), and is what the update divides by.
//   Both are rounded stochastically.  A step moves sqrt(v) by 0.05 % of itself
// (b2 = 0.999) and half a code is 3 to 6 %: rounding to nearest would never
// move a code.  A code of sqrt(v) that is not zero stays at least 2^-9, so that
// an element far below its block's largest keeps a denominator (a larger one
// than its own: a smaller step).  The update itself uses the moments before
// they are rounded.
//   The 16 random bits of a value come from its place, the tensor's step and
// the seed: the vector of eight elements hashes (Wellons' lowbias32), and its
// elements take members of a linear congruential sequence (Numerical Recipes'
// multiplier and increment) from there, each by one multiply-add.
//
// Bound by HBM: 16 bytes a parameter and step at least (bf16 parameter and
// gradient, fp32 master, 8-bit moments), 28 with 32-bit moments.  A warp takes
// a block at a time, eight elements a lane, all its loads issued before the
// first is used, and arithmetic in packed pairs; the tables of tensors come as
// kernel parameters, so a step copies nothing to the device and can be
// captured.  A tensor's step count is on the device and counted up by the last
// block of the grid to finish, when all have read it.
//
// Measured (one GB300, of the 6793 GB/s of its copy): 680 M parameters, bf16 over
// fp32 masters, bf16 gradients: 32-bit moments 2947-3024 us = 6.46-6.30 TB/s
// (95-93 %, by box), 8-bit 1814-1821 us = 6.02 TB/s (88 %); 28 M parameters in
// fp32 131 us = 6.13 TB/s; the norm of 680 M bf16 gradients 204-214 us = 6.67-6.37
// TB/s (98-94 %).  With 8-bit moments half the bytes go in pieces of 256 and less a
// warp and stream (five streams to read, five to write), and issue slots are 65 %
// full.  At 1811 us (63 %), before small decay and what is not finite were seen to,
// chunks of four blocks a warp (1861 us), the next block's loads ahead of this
// one's arithmetic (1866 us) and no random bits at all (1888 us beside 1861) moved
// it less than what is left.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>

#include "pvl_device.cuh"

namespace pvl {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBlock = 256;        // elements that share a scale
// Tensors of a launch.  The table of 512 is 22 KB of kernel parameters; handing it
// over for a few tensors costs the caller 4 us a step (36 beside 32).
constexpr int kFew = 32, kMany = 512;
constexpr float kTop = 448.0f;     // largest e4m3 value
constexpr int kNormUnit = 1024;    // elements a warp takes at a time for the norm
constexpr int kMaxNormCtas = 4096;

// Tensors of a launch.
template <int kT>
struct Tensors {
  uint32_t start[kT + 1];  // running count of blocks
  int32_t slot[kT];        // place in the step counts
  float decay[kT];
  int32_t n;
  void* param[kT];
  const void* grad[kT];
  long long size[kT];
  long long block[kT];     // first block in the states
};

struct StepParams {
  float lr, b1, c1, b2, c2, log_b1, log_b2, eps, max_norm;  // c = 1 - b
  uint32_t seed;
  const float* lr_dev;
  const float* norm;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  float* master;
  int32_t* steps;
  unsigned int* done;
};

// Loads that pass through once.
__device__ __forceinline__ uint4 ld16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

__device__ __forceinline__ uint2 ld8(const void* p) {
  uint2 v;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
  return v;
}

// Eight elements: 32 bytes of fp32, 16 of bf16.  32 bytes on their boundary move
// in one instruction, a whole sector a lane; two of 16 with half a sector each
// reached 79 % of the copy rate where this reaches more.
struct Eight {
  uint32_t w[8];
};

__device__ __forceinline__ Eight ld32(const void* p) {
  Eight e;
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(e.w[0]), "=r"(e.w[1]), "=r"(e.w[2]), "=r"(e.w[3]), "=r"(e.w[4]), "=r"(e.w[5]), "=r"(e.w[6]),
                 "=r"(e.w[7])
               : "l"(p)
               : "memory");
  return e;
}

__device__ __forceinline__ void st32(void* p, const float (&f)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(f[0]), "f"(f[1]), "f"(f[2]),
               "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
               : "memory");
}

// kBy: what the address is a multiple of, for fp32 (16 or 32).
template <typename T, int kBy>
__device__ __forceinline__ Eight load8(const T* p) {
  if constexpr (sizeof(T) == 4 && kBy == 32) {
    return ld32(p);
  } else {
    Eight e;
    const uint4 a = ld16(p);
    e.w[0] = a.x, e.w[1] = a.y, e.w[2] = a.z, e.w[3] = a.w;
    if constexpr (sizeof(T) == 4) {
      const uint4 b = ld16(p + 4);
      e.w[4] = b.x, e.w[5] = b.y, e.w[6] = b.z, e.w[7] = b.w;
    }
    return e;
  }
}

template <typename T>
__device__ __forceinline__ void open8(const Eight& e, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (sizeof(T) == 4) {
      f[i] = __uint_as_float(e.w[i]);
    } else {
      f[i] = __uint_as_float(i % 2 ? e.w[i / 2] & 0xFFFF0000u : e.w[i / 2] << 16);
    }
  }
}

template <typename T, int kBy>
__device__ __forceinline__ void store8(T* p, const float (&f)[8]) {
  if constexpr (sizeof(T) == 4 && kBy == 32) {
    st32(p, f);
  } else if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    *(reinterpret_cast<float4*>(p) + 1) = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                              pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  }
}

__device__ __forceinline__ float wide(float f) { return f; }
__device__ __forceinline__ float wide(__nv_bfloat16 f) { return __bfloat162float(f); }
__device__ __forceinline__ void narrow(float* p, float f) { *p = f; }
__device__ __forceinline__ void narrow(__nv_bfloat16* p, float f) { *p = __float2bfloat16_rn(f); }

// Elements of a tensor that does not start on a 16-byte boundary, or its end.
template <typename T>
__device__ __forceinline__ void load_some(const T* p, int n, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = i < n ? wide(p[i]) : 0.0f;
}

// Not flushed to 0 below the normal numbers: an eps of 1e-15 and less does not cover those roots.
__device__ __forceinline__ float root_of(float x) {
  float y;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float inverse(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ------------------------------------------------------------- 8 bits
__device__ __forceinline__ uint32_t mix(uint32_t z) {
  z ^= z >> 16;
  z *= 0x7FEB352Du;
  z ^= z >> 15;
  z *= 0x846CA68Bu;
  return z ^ (z >> 16);
}

// Member k of the congruential sequence from h is lcg_mul(k) h + lcg_add(k).
constexpr uint32_t lcg_mul(int k) { return k ? lcg_mul(k - 1) * 1664525u : 1u; }
constexpr uint32_t lcg_add(int k) { return k ? lcg_add(k - 1) * 1664525u + 1013904223u : 0u; }

template <int kK>
__device__ __forceinline__ uint32_t chance(uint32_t h) {
  constexpr uint32_t mul = lcg_mul(kK), add = lcg_add(kK);
  return (((h * mul + add) >> 16) << 4) | 8u;  // 20 bits, of which the upper 16 are random
}

// x, of magnitude 2^-6 to 448, to three fraction bits towards 0 after `r` of 2^20
// parts of a step are added to its magnitude.
__device__ __forceinline__ float round_normal(float x, uint32_t r) {
  return __uint_as_float((__float_as_uint(x) + r) & 0xFFF00000u);
}

// The same for magnitudes of 0 to 448 and NaN: below 2^-6 steps are 2^-9
// throughout, as those of [2^-6, 2^-5).
__device__ __forceinline__ float round_any(float x, uint32_t r) {
  const float shift = fabsf(x) < 0.015625f ? 0.015625f : 0.0f;
  return x == x ? copysignf(round_normal(fabsf(x) + shift, r) - shift, x) : x;
}

__device__ __forceinline__ float smallest(const float (&f)[8]) {
  float low = fabsf(f[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) low = fminf(low, fabsf(f[i]));
  return low;
}

__device__ __forceinline__ void open_e4m3(uint2 q, float scale, float (&f)[8]) {
  const uint32_t w[2] = {q.x, q.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i / 2] >> (16 * (i % 2))), __NV_E4M3);
    const float2 g = fmul2(__half22float2(__half2(h)), make_float2(scale, scale));
    f[2 * i] = g.x;
    f[2 * i + 1] = g.y;
  }
}

__device__ __forceinline__ uint2 close_e4m3(const float (&f)[8]) {
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t q = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * i], f[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    w[i / 2] |= q << (16 * (i % 2));
  }
  return make_uint2(w[0], w[1]);
}

// The largest of three magnitudes, NaN if one of them is.
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float y;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// Largest magnitude of a block; NaN, whose bits are above those of infinity, if it holds one.
__device__ __forceinline__ float block_top(const float (&f)[8]) {
  const float top = max_nan(max_nan(max_nan(f[0], f[1], f[2]), f[3], f[4]), max_nan(f[5], f[6], f[7]), 0.0f);
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
}

// A block that holds what is not finite: such an element takes the NaN code, and the scales are those of the others.
// An infinite or NaN gradient leaves NaN in both moments.  Where the square of a finite gradient alone left fp32, v is
// infinite for good: a NaN code of v beside a finite m stands for that, and the update is 0, as with 32-bit moments.
__device__ __forceinline__ void set_apart(float (&m)[8], float (&root)[8], float& top_m, float& top_root) {
  const float nan = __int_as_float(0x7FFFFFFF);
  float a[8], b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool in = fabsf(m[i]) < INFINITY;
    if (!in || !(root[i] < INFINITY)) {
      m[i] = in ? 0.0f : nan;
      root[i] = nan;
    }
    a[i] = in ? m[i] : 0.0f;
    b[i] = root[i] == root[i] ? root[i] : 0.0f;
  }
  top_m = block_top(a);
  top_root = block_top(b);
}

// a + b, which the compiler may not make a multiply-add of the product that a
// or b is (it does so with packed additions, rounding by name or not).
__device__ __forceinline__ float2 sum_of(float2 a, float2 b) {
  return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y));
}

// Quotients of a block's values by its scale, rounded to nearest: a product with
// the reciprocal (itself rounded to nearest), corrected by its remainder, which a
// multiply-add gives exactly (Markstein's theorem).  0 for a block below 2^-100.
struct Divisor {
  float scale, inverse;
  __device__ __forceinline__ explicit Divisor(float top) {
    scale = top < 0x1p-100f ? 0.0f : top * (1.0f / kTop);
    inverse = top < 0x1p-100f ? 0.0f : __frcp_rn(scale);
  }
  __device__ __forceinline__ float2 quotient(float2 a) const {
    const float2 y = make_float2(inverse, inverse), q = fmul2(a, y);
    return ffma2(ffma2(q, make_float2(-scale, -scale), a), y, q);
  }
};

// ---------------------------------------------------------------- step
// 1 - x as hi + lo: exact up to a rounding of lo, at most 2^-23 of hi.  Both have one sign and lo is not 0 unless
// 1 - x is, so that an infinite parameter stays what it is.
struct Keep {
  float hi, lo;
};

__device__ __forceinline__ Keep keep_of(float x) {
  float hi = __fsub_rn(1.0f, x);
  const float t = __fsub_rn(hi, 1.0f);
  float lo = __fsub_rn(__fsub_rn(1.0f, __fsub_rn(hi, t)), __fadd_rn(x, t));  // Knuth's two-sum
  if (lo != 0.0f && (lo < 0.0f) != (hi < 0.0f)) {
    const float down = __int_as_float(__float_as_int(hi) - 1);  // the next towards 0
    lo = __fadd_rn(lo, __fsub_rn(hi, down));
    hi = down;
  }
  if (lo == 0.0f) lo = hi * 0x1p-100f;
  return {hi, lo};
}

// What a block's elements share.
struct Shared {
  float clip, rate, second;
  Keep keep;
  uint32_t key;
};

// One block: this lane's eight elements, n of which are the tensor's.  kBy: what
// fp32 addresses of the tensors are multiples of, or 0 where the block is not
// whole or not aligned and elements go one by one.
template <typename P, typename G, bool k8, int kBy>
__device__ __forceinline__ void step_block(const StepParams& p, const Shared& c, P* param, const G* grad, long long sb,
                                           int n) {
  constexpr bool kMaster = sizeof(P) == 2;
  const int lane = threadIdx.x % 32;
  const long long st = sb * kBlock + lane * 8;
  Eight qg, qp, qm, qv;
  uint2 cm, cv;
  float sm = 0.0f, sv = 0.0f;
  if constexpr (kBy != 0) qg = load8<G, kBy>(grad);
  if constexpr (kMaster) qp = ld32(p.master + st);
  else if constexpr (kBy != 0) qp = load8<P, kBy>(param);
  if constexpr (k8) {
    cm = ld8(static_cast<const uint8_t*>(p.m) + st);
    cv = ld8(static_cast<const uint8_t*>(p.v) + st);
    sm = p.m_scale[sb];
    sv = p.v_scale[sb];
  } else {
    qm = ld32(static_cast<const float*>(p.m) + st);
    qv = ld32(static_cast<const float*>(p.v) + st);
  }
  float g[8], w[8], m[8], v[8], root[8];
  if constexpr (kBy != 0) open8<G>(qg, g);
  else load_some(grad, n, g);
  if constexpr (kMaster) open8<float>(qp, w);
  else if constexpr (kBy != 0) open8<P>(qp, w);
  else load_some(param, n, w);
  if constexpr (k8) {
    open_e4m3(cm, sm, m);
    open_e4m3(cv, sv, v);
  } else {
    open8<float>(qm, m);
    open8<float>(qv, v);
  }
  const float2 b1 = make_float2(p.b1, p.b1), c1 = make_float2(p.c1, p.c1), b2 = make_float2(p.b2, p.b2),
               c2 = make_float2(p.c2, p.c2), clip = make_float2(c.clip, c.clip), second = make_float2(c.second, c.second),
               eps = make_float2(p.eps, p.eps), rate = make_float2(-c.rate, -c.rate), keep = make_float2(c.keep.hi, c.keep.hi),
               keep_lo = make_float2(c.keep.lo, c.keep.lo);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 gc = fmul2(make_float2(g[i], g[i + 1]), clip);
    float2 mm = make_float2(m[i], m[i + 1]), vv = make_float2(v[i], v[i + 1]), r;
    if constexpr (k8) {
      // Each operation rounded by itself, and the root to nearest: moments whose codes are chosen by their last
      // bits are then what plain fp32 arithmetic gives anywhere.
      mm = sum_of(fmul2(mm, b1), fmul2(gc, c1));
      vv = sum_of(fmul2(fmul2(vv, vv), b2), fmul2(fmul2(gc, gc), c2));
      r = make_float2(__fsqrt_rn(vv.x), __fsqrt_rn(vv.y));
    } else {
      mm = ffma2(b1, mm, fmul2(c1, gc));
      vv = ffma2(fmul2(c2, gc), gc, fmul2(b2, vv));
      r = make_float2(root_of(vv.x), root_of(vv.y));
    }
    m[i] = mm.x, m[i + 1] = mm.y;
    v[i] = vv.x, v[i + 1] = vv.y;
    root[i] = r.x, root[i + 1] = r.y;
  }
  float tm = 0.0f, tv = 0.0f;
  bool odd = false;  // whether the block holds what is not finite: the same for the whole warp
  if constexpr (k8) {
    tm = block_top(m);
    tv = block_top(root);
    odd = !(tm < INFINITY && tv < INFINITY);
    if (odd) {
#pragma unroll
      for (int i = 0; i < 8; ++i)  // an infinite v, held as NaN
        if (fabsf(m[i]) < INFINITY && !(root[i] < INFINITY)) root[i] = INFINITY;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 d = ffma2(make_float2(root[i], root[i + 1]), second, eps);
    const float2 q = fmul2(make_float2(m[i], m[i + 1]), make_float2(inverse(d.x), inverse(d.y)));
    const float2 was = make_float2(w[i], w[i + 1]);
    const float2 ww = ffma2(was, keep, ffma2(was, keep_lo, fmul2(rate, q)));
    w[i] = ww.x, w[i + 1] = ww.y;
  }
  if constexpr (kMaster) st32(p.master + st, w);
  if constexpr (kBy != 0) {
    store8<P, kBy>(param, w);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) narrow(param + i, w[i]);
  }
  if constexpr (k8) {
    if (odd) set_apart(m, root, tm, tv);
    // a block below 2^-100 becomes zeros: its scale would not be a normal number
    const Divisor by_m(tm), by_v(tv);
    const uint32_t h = mix((static_cast<uint32_t>(sb) * 32u + lane) ^ c.key);
    const uint32_t rm[8] = {chance<1>(h), chance<2>(h), chance<3>(h), chance<4>(h),
                            chance<5>(h), chance<6>(h), chance<7>(h), chance<8>(h)};
    const uint32_t rv[8] = {chance<9>(h), chance<10>(h), chance<11>(h), chance<12>(h),
                            chance<13>(h), chance<14>(h), chance<15>(h), chance<16>(h)};
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float2 a = by_m.quotient(make_float2(m[i], m[i + 1]));
      const float2 b = by_v.quotient(make_float2(root[i], root[i + 1]));
      m[i] = a.x, m[i + 1] = a.y;
      v[i] = b.x, v[i + 1] = b.y;
    }
    // few blocks hold a value below 3e-5 of their largest: a third of the work less for the others
    if (!odd && smallest(m) >= 0.015625f) {
#pragma unroll
      for (int i = 0; i < 8; ++i) m[i] = round_normal(m[i], rm[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) m[i] = round_any(m[i], rm[i]);
    }
    if (!odd && smallest(v) >= 0.015625f) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = round_normal(v[i], rv[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = v[i] > 0.0f ? fmaxf(round_any(v[i], rv[i]), 0.001953125f) : v[i];
    }
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.m) + st) = close_e4m3(m);
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.v) + st) = close_e4m3(v);
    if (lane == 0) {
      p.m_scale[sb] = by_m.scale;
      p.v_scale[sb] = by_v.scale;
    }
  } else {
    st32(static_cast<float*>(p.m) + st, m);
    st32(static_cast<float*>(p.v) + st, v);
  }
}

template <typename P, typename G, bool k8, int kT>
__global__ void __launch_bounds__(kThreads, k8 ? 4 : 2) adamw_kernel(const __grid_constant__ Tensors<kT> tab,
                                                         const __grid_constant__ StepParams p) {
  const int lane = threadIdx.x % 32;
  Shared c;
  c.clip = 1.0f;
  if (p.norm) {
    const float norm = __ldg(p.norm);
    if (!(norm < INFINITY)) return;  // NaN or infinite gradients: no step, the same for the whole grid
    c.clip = norm > p.max_norm ? p.max_norm / norm : 1.0f;
  }
  const float lr = p.lr_dev ? __ldg(p.lr_dev) : p.lr;
  const uint32_t total = tab.start[tab.n];
  uint32_t u = blockIdx.x * kWarps + threadIdx.x / 32;
  int t = 0;
  {
    int hi = tab.n - 1;  // last tensor that starts at or before u
    while (t < hi) {
      const int mid = (t + hi + 1) / 2;
      if (tab.start[mid] <= u) t = mid; else hi = mid - 1;
    }
  }
  int32_t step = -1;
  for (; u < total; u += gridDim.x * kWarps) {
    while (u >= tab.start[t + 1]) ++t;
    const uint32_t b = u - tab.start[t];       // block of the tensor
    const long long sb = tab.block[t] + b;     // block of the states
    const long long at = static_cast<long long>(b) * kBlock + lane * 8;
    P* param = static_cast<P*>(tab.param[t]) + at;
    const G* grad = static_cast<const G*>(tab.grad[t]) + at;
    const long long left = tab.size[t] - at;   // of this lane
    const int32_t now = p.steps[tab.slot[t]] + 1;
    if (now != step) {
      step = now;
      const float s = static_cast<float>(now);
      c.rate = lr / -expm1f(s * p.log_b1);
      c.second = rsqrtf(-expm1f(s * p.log_b2));
      c.key = mix(p.seed + static_cast<uint32_t>(now) * 0x9E3779B9u);
    }
    c.keep = keep_of(lr * tab.decay[t]);
    // The same for the whole warp, which takes one way through the block: by the tensors' addresses, not a lane's (a
    // lane's eight bf16 elements start at every 16 bytes).
    const bool whole = tab.size[t] - static_cast<long long>(b) * kBlock >= kBlock;
    const uintptr_t at_p = reinterpret_cast<uintptr_t>(tab.param[t]), at_g = reinterpret_cast<uintptr_t>(tab.grad[t]);
    if (whole && at_p % (8 * sizeof(P)) == 0 && at_g % (8 * sizeof(G)) == 0)
      step_block<P, G, k8, 32>(p, c, param, grad, sb, 8);
    else if ((sizeof(P) == 4 || sizeof(G) == 4) && whole && (at_p | at_g) % 16 == 0)
      step_block<P, G, k8, 16>(p, c, param, grad, sb, 8);
    else
      step_block<P, G, k8, 0>(p, c, param, grad, sb, left >= 8 ? 8 : left > 0 ? static_cast<int>(left) : 0);
  }
  // every block has read the step counts once it has counted itself
  __shared__ bool last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(p.done, 1u) == gridDim.x - 1;
    __threadfence();
  }
  __syncthreads();
  if (!last) return;
  for (int i = threadIdx.x; i < tab.n; i += kThreads) p.steps[tab.slot[i]] += 1;
  if (threadIdx.x == 0) *p.done = 0;  // for the next step
}

// ---------------------------------------------------------------- norm
template <int kT>
struct Grads {
  uint32_t start[kT + 1];  // running count of units
  int32_t n;
  const void* grad[kT];
  long long size[kT];
};

struct NormParams {
  double* part;        // one a block of every launch
  unsigned int* done;  // cleared before the first launch
  int first, total;    // this launch's first part; parts of all launches, or 0 before the last
  float* norm;
};

// A lane's 32 elements of a unit: four vectors of eight, a warp's vectors side
// by side.  Squares are added in fp32, even and odd elements apart; a sum that
// overflows, or that is so small that squares may have been lost below the
// normal numbers, is taken again in 64 bits.
template <typename G>
__device__ __noinline__ double unit_again(const G* grad, int n) {
  double d = 0.0;
  for (int i = threadIdx.x % 32; i < n; i += 32) {
    const float f = wide(grad[i]);
    if (f != 0.0f) d = fma(static_cast<double>(f), static_cast<double>(f), d);  // zeros cost nothing
  }
  return d;
}

template <typename G>
__device__ __forceinline__ double unit_squares(const G* grad, long long left) {
  const int lane = threadIdx.x % 32;
  float2 s = make_float2(0.0f, 0.0f);
  if (left >= kNormUnit && reinterpret_cast<uintptr_t>(grad) % (8 * sizeof(G)) == 0) {
    Eight q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = load8<G, 32>(grad + (i * 32 + lane) * 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float f[8];
      open8<G>(q[i], f);
#pragma unroll
      for (int j = 0; j < 8; j += 2) s = ffma2(make_float2(f[j], f[j + 1]), make_float2(f[j], f[j + 1]), s);
    }
  } else if (left >= kNormUnit) {  // off a boundary: element by element, sixteen on their way at once
#pragma unroll
    for (int i = 0; i < kNormUnit; i += 512) {
      float f[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) f[j] = wide(grad[i + j * 32 + lane]);
#pragma unroll
      for (int j = 0; j < 16; ++j) s.x = fmaf(f[j], f[j], s.x);
    }
  } else {
    for (int i = lane; i < left; i += 32) {
      const float f = wide(grad[i]);
      s.x = fmaf(f, f, s.x);
    }
  }
  const float sum = s.x + s.y;
  // the warp's lanes take other elements in unit_again than here: all or none
  if (__all_sync(0xffffffffu, sum > 0x1p-60f && sum < INFINITY)) return static_cast<double>(sum);
  return unit_again(grad, left < kNormUnit ? static_cast<int>(left) : kNormUnit);
}

__device__ double block_sum(double v) {
  __shared__ double part[kWarps];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) v += part[i];
  return v;
}

template <typename G, int kT>
__global__ void __launch_bounds__(kThreads) norm_kernel(const __grid_constant__ Grads<kT> tab,
                                                        const __grid_constant__ NormParams p) {
  const uint32_t total = tab.start[tab.n];
  uint32_t u = blockIdx.x * kWarps + threadIdx.x / 32;
  int t = 0;
  {
    int hi = tab.n - 1;
    while (t < hi) {
      const int mid = (t + hi + 1) / 2;
      if (tab.start[mid] <= u) t = mid; else hi = mid - 1;
    }
  }
  double d = 0.0;
  for (; u < total; u += gridDim.x * kWarps) {
    while (u >= tab.start[t + 1]) ++t;
    const long long at = static_cast<long long>(u - tab.start[t]) * kNormUnit;
    d += unit_squares(static_cast<const G*>(tab.grad[t]) + at, tab.size[t] - at);
  }
  d = block_sum(d);
  __shared__ bool last;
  if (threadIdx.x == 0) {
    p.part[p.first + blockIdx.x] = d;
    __threadfence();
    last = p.total && atomicAdd(p.done, 1u) == gridDim.x - 1;
    __threadfence();
  }
  __syncthreads();
  if (!last) return;
  d = 0.0;
  for (int i = threadIdx.x; i < p.total; i += kThreads) d += __ldcg(p.part + i);
  d = block_sum(d);
  if (threadIdx.x == 0) *p.norm = static_cast<float>(sqrt(d));
}

// ---------------------------------------------------------------- host
long long blocks_of(long long n) { return (n + kBlock - 1) / kBlock; }

template <typename P, typename G, bool k8, int kT>
pvl_status launch_step(const Tensors<kT>& tab, const StepParams& p, int sms, cudaStream_t s) {
  const void* fn = reinterpret_cast<const void*>(adamw_kernel<P, G, k8, kT>);
  const int fit = blocks_per_sm(fn, kThreads, 0);
  if (fit < 1) return fail(PVL_ERR_CUDA, "pvl_adamw_step: the kernel does not fit on an SM");
  const long long need = (static_cast<long long>(tab.start[tab.n]) + kWarps - 1) / kWarps;
  const long long most = static_cast<long long>(fit) * sms;
  adamw_kernel<P, G, k8, kT><<<static_cast<unsigned>(need < most ? need : most), kThreads, 0, s>>>(tab, p);
  return check_cuda(cudaGetLastError(), "pvl_adamw_step launch");
}

template <typename P, typename G, int kT>
pvl_status step_bits(int bits, const Tensors<kT>& tab, const StepParams& p, int sms, cudaStream_t s) {
  return bits == 8 ? launch_step<P, G, true, kT>(tab, p, sms, s) : launch_step<P, G, false, kT>(tab, p, sms, s);
}

template <int kT>
pvl_status step_types(const pvl_adamw* h, const Tensors<kT>& tab, const StepParams& p, int sms, cudaStream_t s) {
  if (h->param_dtype == 0)
    return h->grad_dtype == 0 ? step_bits<__nv_bfloat16, __nv_bfloat16, kT>(h->bits, tab, p, sms, s)
                              : step_bits<__nv_bfloat16, float, kT>(h->bits, tab, p, sms, s);
  return h->grad_dtype == 0 ? step_bits<float, __nv_bfloat16, kT>(h->bits, tab, p, sms, s)
                            : step_bits<float, float, kT>(h->bits, tab, p, sms, s);
}

// Tensors first.. of the list, as many as a launch takes: kT of them, and fewer
// than 2^31 blocks.  Returns how many.
template <int kT>
int fill(const pvl_adamw_tensor* list, int first, int count, Tensors<kT>* tab) {
  int n = 0;
  long long blocks = 0;
  for (; n < kT && first + n < count; ++n) {
    const pvl_adamw_tensor& q = list[first + n];
    if (blocks + blocks_of(q.size) >= (1ll << 31)) break;
    tab->start[n] = static_cast<uint32_t>(blocks);
    blocks += blocks_of(q.size);
    tab->param[n] = q.param;
    tab->grad[n] = q.grad;
    tab->size[n] = q.size;
    tab->block[n] = q.block;
    tab->slot[n] = q.slot;
    tab->decay[n] = q.decay;
  }
  tab->start[n] = static_cast<uint32_t>(blocks);
  tab->n = n;
  return n;
}

template <typename G, int kT>
pvl_status launch_norm(const Grads<kT>& tab, const NormParams& p, int grid, cudaStream_t s) {
  norm_kernel<G, kT><<<grid, kThreads, 0, s>>>(tab, p);
  return check_cuda(cudaGetLastError(), "pvl_grad_norm launch");
}

template <int kT>
pvl_status norm_all(const void* const* grads, const int64_t* sizes, int count, int dtype, NormParams p, int sms,
                    cudaStream_t s) {
  Grads<kT> tab;
  const void* fn = dtype ? reinterpret_cast<const void*>(norm_kernel<float, kT>)
                         : reinterpret_cast<const void*>(norm_kernel<__nv_bfloat16, kT>);
  const int most = blocks_per_sm(fn, kThreads, 0) * sms;
  if (most < 1) return fail(PVL_ERR_CUDA, "pvl_grad_norm: the kernel does not fit on an SM");
  const int launches = (count + kT - 1) / kT;
  const int cap = kMaxNormCtas / launches < most ? kMaxNormCtas / launches : most;
  int parts = 0;
  for (int i = 0; i < launches; ++i) {
    long long units = 0;
    int n = 0;
    for (; n < kT && i * kT + n < count; ++n) {
      tab.start[n] = static_cast<uint32_t>(units);
      tab.grad[n] = grads[i * kT + n];
      tab.size[n] = sizes[i * kT + n];
      units += (tab.size[n] + kNormUnit - 1) / kNormUnit;
    }
    tab.start[n] = static_cast<uint32_t>(units);
    tab.n = n;
    const long long need = (units + kWarps - 1) / kWarps;
    const int grid = static_cast<int>(need < cap ? need : cap);
    p.first = parts;
    parts += grid;
    p.total = i == launches - 1 ? parts : 0;
    const pvl_status st = dtype ? launch_norm<float, kT>(tab, p, grid, s) : launch_norm<__nv_bfloat16, kT>(tab, p, grid, s);
    if (st != PVL_OK) return st;
  }
  return PVL_OK;
}

constexpr size_t kNormWsBytes = 256 + 8 * kMaxNormCtas;

}  // namespace
}  // namespace pvl

using namespace pvl;

extern "C" pvl_status pvl_adamw_step(const pvl_adamw* h, const pvl_adamw_tensor* list, int count, pvl_stream_t stream) {
  const char* who = "pvl_adamw_step";
  if (!h || !list || !h->m || !h->v || !h->steps || !h->done) return fail(PVL_ERR_INVALID_ARG, "%s: null pointer", who);
  if (count < 1) return fail(PVL_ERR_INVALID_ARG, "%s: needs a tensor", who);
  if ((h->param_dtype & ~1) || (h->grad_dtype & ~1))
    return fail(PVL_ERR_INVALID_ARG, "%s: dtypes are 0 (bf16) or 1 (fp32)", who);
  if (h->bits != 8 && h->bits != 32) return fail(PVL_ERR_INVALID_ARG, "%s: bits %d (8 or 32)", who, h->bits);
  if (h->bits == 8 && (!h->m_scale || !h->v_scale)) return fail(PVL_ERR_INVALID_ARG, "%s: 8 bits need the scales", who);
  if ((h->param_dtype == 0) != (h->master != nullptr))
    return fail(PVL_ERR_INVALID_ARG, "%s: bf16 parameters, and only they, need fp32 masters", who);
  if (!h->lr_dev && !(fabsf(h->lr) < 1e30f)) return fail(PVL_ERR_INVALID_ARG, "%s: lr must be finite", who);
  if (!(h->beta1 >= 0.0 && h->beta1 < 1.0 && h->beta2 >= 0.0 && h->beta2 < 1.0))
    return fail(PVL_ERR_INVALID_ARG, "%s: betas lie in [0, 1)", who);
  if (!(h->eps >= 1e-30f && h->eps < 1e30f))
    return fail(PVL_ERR_INVALID_ARG, "%s: eps must be at least 1e-30 and finite", who);
  if (h->norm && !(h->max_norm > 0.0f)) return fail(PVL_ERR_INVALID_ARG, "%s: max_norm must be positive", who);
  const uintptr_t wide32 = reinterpret_cast<uintptr_t>(h->m) | reinterpret_cast<uintptr_t>(h->v) |
                           reinterpret_cast<uintptr_t>(h->master);
  const uintptr_t wide4 = reinterpret_cast<uintptr_t>(h->m_scale) | reinterpret_cast<uintptr_t>(h->v_scale) |
                          reinterpret_cast<uintptr_t>(h->steps) | reinterpret_cast<uintptr_t>(h->done) |
                          reinterpret_cast<uintptr_t>(h->lr_dev) | reinterpret_cast<uintptr_t>(h->norm);
  if (wide32 % 32 || wide4 % 4) return fail(PVL_ERR_UNSUPPORTED, "%s: m, v and master must be 32-byte aligned", who);
  for (int i = 0; i < count; ++i) {
    const pvl_adamw_tensor& q = list[i];
    if (!q.param || !q.grad) return fail(PVL_ERR_INVALID_ARG, "%s: tensor %d has a null pointer", who, i);
    if (q.size < 1 || q.block < 0 || q.slot < 0 || !(fabsf(q.decay) < 1e30f))
      return fail(PVL_ERR_INVALID_ARG, "%s: tensor %d: size must be >= 1, block and slot not negative, decay finite", who, i);
    if (q.size >= (1ll << 38) || q.block >= (1ll << 40))
      return fail(PVL_ERR_UNSUPPORTED, "%s: tensor %d is too large", who, i);
    if (reinterpret_cast<uintptr_t>(q.param) % (h->param_dtype ? 4 : 2) ||
        reinterpret_cast<uintptr_t>(q.grad) % (h->grad_dtype ? 4 : 2))
      return fail(PVL_ERR_UNSUPPORTED, "%s: tensor %d is not aligned to its elements", who, i);
  }
  const int sms = sm_count();
  if (sms <= 0) return fail(PVL_ERR_CUDA, "%s: no usable CUDA device", who);
  StepParams p{};
  p.lr = h->lr;
  p.b1 = static_cast<float>(h->beta1);
  p.c1 = static_cast<float>(1.0 - h->beta1);
  p.b2 = static_cast<float>(h->beta2);
  p.c2 = static_cast<float>(1.0 - h->beta2);
  p.log_b1 = static_cast<float>(std::log(h->beta1));
  p.log_b2 = static_cast<float>(std::log(h->beta2));
  p.eps = h->eps;
  p.max_norm = h->max_norm;
  p.seed = h->seed;
  p.lr_dev = h->lr_dev;
  p.norm = h->norm;
  p.m = h->m;
  p.v = h->v;
  p.m_scale = h->m_scale;
  p.v_scale = h->v_scale;
  p.master = h->master;
  p.steps = h->steps;
  p.done = h->done;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  pvl_status st = PVL_OK;
  for (int first = 0; first < count && st == PVL_OK;) {
    if (count - first <= kFew) {
      Tensors<kFew> tab;
      first += fill(list, first, count, &tab);
      st = step_types(h, tab, p, sms, s);
    } else {
      Tensors<kMany> tab;
      first += fill(list, first, count, &tab);
      st = step_types(h, tab, p, sms, s);
    }
  }
  return st;
}

extern "C" size_t pvl_grad_norm_ws_bytes(void) { return kNormWsBytes; }

extern "C" pvl_status pvl_grad_norm(const void* const* grads, const int64_t* sizes, int count, int dtype, float* norm,
                                    void* ws, size_t ws_bytes, pvl_stream_t stream) {
  const char* who = "pvl_grad_norm";
  if (!grads || !sizes || !norm || !ws) return fail(PVL_ERR_INVALID_ARG, "%s: null pointer", who);
  if (count < 1) return fail(PVL_ERR_INVALID_ARG, "%s: needs a tensor", who);
  if (dtype & ~1) return fail(PVL_ERR_INVALID_ARG, "%s: dtype %d (0: bf16, 1: fp32)", who, dtype);
  if (ws_bytes < kNormWsBytes)
    return fail(PVL_ERR_INVALID_ARG, "%s: workspace %zu bytes < %zu needed", who, ws_bytes, kNormWsBytes);
  if (reinterpret_cast<uintptr_t>(ws) % 16 || reinterpret_cast<uintptr_t>(norm) % 4)
    return fail(PVL_ERR_UNSUPPORTED, "%s: ws must be 16-byte and norm 4-byte aligned", who);
  if (count > kMany * 256) return fail(PVL_ERR_UNSUPPORTED, "%s: %d tensors (at most %d)", who, count, kMany * 256);
  long long units = 0;
  for (int i = 0; i < count; ++i) {
    if (!grads[i] || sizes[i] < 1) return fail(PVL_ERR_INVALID_ARG, "%s: tensor %d is null or empty", who, i);
    if (sizes[i] >= (1ll << 41)) return fail(PVL_ERR_UNSUPPORTED, "%s: tensor %d is too large", who, i);
    if (reinterpret_cast<uintptr_t>(grads[i]) % (dtype ? 4 : 2))
      return fail(PVL_ERR_UNSUPPORTED, "%s: tensor %d is not aligned to its elements", who, i);
    units += (sizes[i] + kNormUnit - 1) / kNormUnit;
  }
  if (units >= (1ll << 31)) return fail(PVL_ERR_UNSUPPORTED, "%s: too many elements", who);
  const int sms = sm_count();
  if (sms <= 0) return fail(PVL_ERR_CUDA, "%s: no usable CUDA device", who);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  NormParams p{};
  p.done = static_cast<unsigned int*>(ws);
  p.part = reinterpret_cast<double*>(static_cast<uint8_t*>(ws) + 256);
  p.norm = norm;
  const pvl_status st = check_cuda(cudaMemsetAsync(ws, 0, 256, s), who);
  if (st != PVL_OK) return st;
  return count <= kFew ? norm_all<kFew>(grads, sizes, count, dtype, p, sms, s)
                       : norm_all<kMany>(grads, sizes, count, dtype, p, sms, s);
}
