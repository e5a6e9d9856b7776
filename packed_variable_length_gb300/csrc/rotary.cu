// pack_rotary_fwd / pack_rotary_bwd: rotary positions of queries and keys,
// with the RMS norm before them and its weight gradients, for sm_103a.
//
// What it computes, per head vector x [D]: z = x r w (no norm: z = x), then
// for each pair (a, b) of the first R features, with t = position x frequency,
//   (a, b) -> gain (a cos t - b sin t, a sin t + b cos t).
// Backward, with g the upstream gradient turned by -t (times gain):
//   no norm: dx = g (the forward with the sine negated);  else, n the features
//   the norm runs over,
//   dx = r (g w - xh mean_n(g w xh)),  xh = x r,   dw = sum g xh.
//
// Angles.  A frequency is given in turns per position as a fraction F of
// 2^64, so the angle in turns is position x F mod 2^64: one wrapping integer
// product, whose top 32 bits are the angle as a signed fraction of a turn,
// exact for any position.  sin.approx / cos.approx on [-pi, pi] are then off
// by about 2^-21, far below the 2^-9 of the bf16 result.
//
// Layout of the work.  HBM bound: 4 bytes an element forward, 6 backward with
// a norm.  Measured (of 6770 GB/s, the card's copy rate), 65,536 tokens of 12 +
// 12 heads of 128 out of a fused projection: forward 126 us without a norm
// (95 %), 131 with the norm per head (91 %), 136 over the token (88 %); backward
// 209 us per head (85 %), 227 over the token (79 %: the chain of sum, norm and
// product of a token at twelve warps an SM, not the bytes).
//   - A unit is two V-wide vectors of a head, R / (2 V) vectors apart, so that
//     neighbouring threads read neighbouring 16 bytes in both layouts: in the
//     half layout the vectors hold the two sides of V pairs, in the
//     interleaved one V / 2 pairs each.  Its 2 V values are kept as packed
//     fp32 pairs A (first sides) and B (second sides), two pairs to a float2.
//   - A team of threads takes one token: a thread owns one unit column of the
//     head and every hpi-th head, kM of them at a time; queries and keys are
//     one run of heads.  The kM heads' vectors are all loaded before the
//     first is used.  Teams are whole warps, or a power of two below 32.
//   - A warp (or smaller team) computes its token's R / 2 angles once, one or
//     two a lane, into shared memory, from where each thread takes its V.
//   - The norm over the token holds all of a token's heads at once; its
//     weights stand in shared memory in the order in which the threads read
//     them.  Its sums cross warps only where a team has several: one barrier.
#include <cuda_runtime.h>

#include <algorithm>

#include "pvl_device.cuh"

namespace pvl {
namespace {

constexpr int kMaxBlock = 384;  // 168 registers a thread, the most that a kernel here takes
constexpr int kMaxD = 256;
constexpr int kPart = 2;        // beside pvl_rotary_layout: interleaved, R < D
constexpr size_t kMaxSmem = 227 * 1024;  // of a block
constexpr int kMaxPartials = 1216;  // rows of partial weight gradients at most
constexpr float kRadians = 1.4629180792671596e-9f;  // 2 pi / 2^32

// A tensor's address and strides in bytes.
struct View {
  char* data;
  int64_t b, l;
  int64_t step;  // of a block's next token
  int32_t h;
};

struct RotaryParams {
  View x[2];    // q, k: what is rotated (backward of a norm: the forward's input)
  View g[2];    // backward of a norm: gradients of the outputs
  View out[2];  // rotated, or dq, dk
  const uint64_t* turns;
  const int32_t* positions;
  const float* w[2];
  float* part;       // backward: [rows][width] partial weight gradients, null: none
  int L, rows;       // tokens of a row; rows (one where the strides let all tokens be one row)
  int H, Ht, D, R;
  int axes, section_1, section_2;
  int units;         // units of a head, D / (2 V)
  int turned;        // units of a head that are rotated: all, or in the half layout R / (2 V)
  int hpi, chunks;   // heads a team takes at once; rounds of kM hpi heads
  int team, teams;   // threads of a team, teams of a block
  int width;         // columns of part
  float gain, sign;  // sign: of the sine
  float eps;
};

template <int V>
struct Vec;
template <>
struct Vec<8> {
  using T = uint4;
};
template <>
struct Vec<4> {
  using T = uint2;
};
template <>
struct Vec<2> {
  using T = uint32_t;
};
template <>
struct Vec<1> {
  using T = uint16_t;
};

__device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// A unit's values: kP packed pairs of first and of second sides (one plain
// pair where V is 1), and the arithmetic on either kind.
template <int V>
struct Unit {
  using F = float2;
  static constexpr int kP = V / 2;
  F a[kP], b[kP];
};
template <>
struct Unit<1> {
  using F = float;
  static constexpr int kP = 1;
  F a[1], b[1];
};
using pvl::ffma2;
using pvl::fmul2;
__device__ __forceinline__ float fmul2(float a, float b) { return a * b; }
__device__ __forceinline__ float ffma2(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float both_of(float2 v) { return v.x + v.y; }
__device__ __forceinline__ float both_of(float v) { return v; }
template <typename F>
__device__ __forceinline__ F splat(float v) {
  if constexpr (sizeof(F) == 8) return make_float2(v, v);
  else return v;
}
// first and second sides of a pair's (a.x, a.y, b.x, b.y)
template <typename F>
__device__ __forceinline__ F side_a(const float4& t) {
  if constexpr (sizeof(F) == 8) return make_float2(t.x, t.y);
  else return t.x;
}
template <typename F>
__device__ __forceinline__ F side_b(const float4& t) {
  if constexpr (sizeof(F) == 8) return make_float2(t.z, t.w);
  else return t.z;
}
__device__ __forceinline__ float2 minus(float2 v) { return make_float2(-v.x, -v.y); }
__device__ __forceinline__ float minus(float v) { return -v; }
// v into `to`, but where a bit of `not_these` is set
__device__ __forceinline__ void take_unless(uint32_t not_these, float2 v, float2& to) {
  if (!(not_these & 1)) to.x = v.x;
  if (!(not_these & 2)) to.y = v.y;
}
__device__ __forceinline__ void take_unless(uint32_t not_these, float v, float& to) {
  if (!(not_these & 1)) to = v;
}

template <int V, bool kHalf>
__device__ __forceinline__ void unpack(const typename Vec<V>::T& u0, const typename Vec<V>::T& u1, Unit<V>& z) {
  if constexpr (V == 1) {
    z.a[0] = __uint_as_float(static_cast<uint32_t>(u0) << 16);
    z.b[0] = __uint_as_float(static_cast<uint32_t>(u1) << 16);
  } else {
    const uint32_t* w0 = reinterpret_cast<const uint32_t*>(&u0);
    const uint32_t* w1 = reinterpret_cast<const uint32_t*>(&u1);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      if (kHalf) {
        z.a[i] = make_float2(lo(w0[i]), hi(w0[i]));
        z.b[i] = make_float2(lo(w1[i]), hi(w1[i]));
      } else {
        const uint32_t v0 = V == 2 ? w0[0] : i < V / 4 ? w0[2 * i] : w1[2 * i - V / 2];
        const uint32_t v1 = V == 2 ? w1[0] : i < V / 4 ? w0[2 * i + 1] : w1[2 * i + 1 - V / 2];
        z.a[i] = make_float2(lo(v0), lo(v1));
        z.b[i] = make_float2(hi(v0), hi(v1));
      }
    }
  }
}
template <int V, bool kHalf>
__device__ __forceinline__ void pack(const Unit<V>& z, typename Vec<V>::T& u0, typename Vec<V>::T& u1) {
  if constexpr (V == 1) {
    u0 = __bfloat16_as_ushort(__float2bfloat16_rn(z.a[0]));
    u1 = __bfloat16_as_ushort(__float2bfloat16_rn(z.b[0]));
  } else {
    uint32_t* w0 = reinterpret_cast<uint32_t*>(&u0);
    uint32_t* w1 = reinterpret_cast<uint32_t*>(&u1);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      if (kHalf) {
        w0[i] = pack_bf16x2(z.a[i].x, z.a[i].y);
        w1[i] = pack_bf16x2(z.b[i].x, z.b[i].y);
      } else {
        (V == 2 ? w0[0] : i < V / 4 ? w0[2 * i] : w1[2 * i - V / 2]) = pack_bf16x2(z.a[i].x, z.b[i].x);
        (V == 2 ? w1[0] : i < V / 4 ? w0[2 * i + 1] : w1[2 * i + 1 - V / 2]) = pack_bf16x2(z.a[i].y, z.b[i].y);
      }
    }
  }
}

// Feature of value k of a unit (k < kP * 2: first sides, then second sides),
// from the offsets of its vectors.
template <int V, bool kHalf>
__device__ __forceinline__ int feature(int k, int e0, int e1) {
  const int e = k % (V > 1 ? V : 1), side = k / (V > 1 ? V : 1);
  if (kHalf || V == 1) return (side ? e1 : e0) + e;
  return e < V / 2 ? e0 + 2 * e + side : e1 + 2 * e - V + side;
}

// Offsets of the two vectors of unit u.  Interleaved pairs lie inside a
// vector, so all units are the same: R may end anywhere (pairs_past).  In the
// half layout the units past the rotated part are their own.
template <int V, bool kHalf>
__device__ __forceinline__ void vectors_of(const RotaryParams& p, int u, int* e0, int* e1) {
  if (!kHalf) {
    *e0 = V > 1 ? u * V : 2 * u;
    *e1 = V > 1 ? u * V + p.D / 2 : 2 * u + 1;
  } else if (u < p.turned) {
    *e0 = u * V;
    *e1 = u * V + p.R / 2;
  } else {
    *e0 = p.R + (u - p.turned) * V;
    *e1 = *e0 + (p.D - p.R) / 2;
  }
}

// The pairs of an interleaved unit that lie past R, one bit each.  They are not
// turned by an angle of 0, which would make a NaN of an infinity beside them.
// Kernels of their own (kPart) have the test: in those of a whole head it cost
// 3 % (64k pack, norm over the token: forward 138 us, 136 without, backward 233,
// 226).
template <int V>
__device__ __forceinline__ uint32_t pairs_past(const RotaryParams& p, int u) {
  uint32_t past = 0;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const int pair = V == 1 ? u : e < V / 2 ? u * (V / 2) + e : p.D / 4 + u * (V / 2) + e - V / 2;
    past |= (pair >= p.R / 2 ? 1u : 0u) << e;
  }
  return past;
}

// Head (of those a team takes at once) and unit of thread t of a team; false
// for a thread without one.  With the norm per head, heads do not straddle
// warps where a warp holds at least one, so that their sums are shuffles.
__host__ __device__ inline bool place(bool per_head, int units, int hpi, int team, int t, int* hl, int* u) {
  if (per_head && team > 32 && units <= 32) {
    const int per = 32 / units, i = t % 32;
    *hl = t / 32 * per + i / units;
    *u = i % units;
    return i < per * units && *hl < hpi;
  }
  *hl = t / units;
  *u = t % units;
  return *hl < hpi;
}

// Sum over the `n` threads of an aligned power-of-two lane group.
__device__ __forceinline__ float lane_sum(float v, int n) {
  for (int o = 1; o < n; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Sum over a head's lanes u = 0 .. units - 1 (neighbours in a warp), in all of them.
__device__ __forceinline__ float head_sum(float v, int u, int units) {
  for (int o = 1; o < units; o <<= 1) {
    const float w = __shfl_down_sync(0xffffffffu, v, o);
    v += u + o < units ? w : 0.0f;
  }
  return __shfl_sync(0xffffffffu, v, (threadIdx.x & 31) - u);
}

// 16, 8 or 4 bytes into shared memory without passing registers; past L1
// where kPast and the width allow it.
template <bool kPast, typename T>
__device__ __forceinline__ void copy_async(T* dst, const char* src) {
  if constexpr (kPast && sizeof(T) == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(dst)), "l"(src), "n"(sizeof(T)) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Stages of a thread's ring of vectors.
constexpr int kRing = 2;

// Shared memory, in floats: the angles' cosines and sines of each warp or
// smaller team, the norm's weights, the sums that cross threads, the threads'
// rings of vectors (at the end their place holds the weight gradients of the
// norm per head).
struct SmemPlan {
  int weights, sums, ring, total;  // offsets; the angles are first
};
__host__ __device__ inline SmemPlan smem_plan(int V, int kM, int norm, bool bwd, int Ht, int D, int units, int hpi, int team,
                                              int teams, int threads) {
  SmemPlan s{};
  const int group = team < 32 ? team : 32;
  const int unit = 2 * (V > 1 ? V : 2), column = kMaxD / (2 * V);  // floats of a unit (V = 1: half unused); units kept
  s.weights = threads / group * column * unit;
  const int weights = norm == PVL_NORM_TOKEN ? (team + 31) / 32 * 32 * kM * unit
                      : norm == PVL_NORM_HEAD ? 2 * column * unit
                                              : 0;
  s.sums = s.weights + weights;
  int sums = 0;
  if (norm == PVL_NORM_TOKEN) sums = 2 * (threads / 32) * 4;
  if (norm == PVL_NORM_HEAD && units > 32) sums = (threads * kM * (bwd ? 2 : 1) + 3) / 4 * 4;
  s.ring = s.sums + sums;
  s.total = s.ring + (V > 1 && norm != PVL_NORM_NONE ? kRing * kM * (bwd ? 4 : 2) * threads * V / 2 : 0);
  const int gradients = !bwd ? 0 : norm == PVL_NORM_HEAD ? teams * hpi * D : teams > 1 ? teams * Ht * D : 0;
  if (s.ring + gradients > s.total) s.total = s.ring + gradients;
  return s;
}

// kNorm: PVL_NORM_NONE, _HEAD or _TOKEN; kBwd only with a norm.  Forward takes
// 96 registers: left to itself the compiler stays at 64 for the sake of warps
// that the shared memory leaves no room for (norm per head, 64k pack: 154 us
// at 64, 132 at 96).
template <int V, int kM, int kNorm, bool kBwd, int kLayout>
__global__ void __maxnreg__(!kBwd ? 96 : V == 8 || V == 1 ? 168 : 128) rotary_kernel(const __grid_constant__ RotaryParams p) {
  using T = typename Vec<V>::T;
  using F = typename Unit<V>::F;
  constexpr bool kHalf = kLayout == PVL_ROTARY_HALF;
  constexpr int kP = Unit<V>::kP, kColumn = kMaxD / (2 * V);
  constexpr bool kHead = kNorm == PVL_NORM_HEAD, kToken = kNorm == PVL_NORM_TOKEN, kAny = kHead || kToken;
  constexpr int kSums = kBwd ? 2 : 1;  // sum x^2, and backward sum g w x
  extern __shared__ __align__(16) float smem[];
  const SmemPlan plan = smem_plan(V, kM, kNorm, kBwd, p.Ht, p.D, p.units, p.hpi, p.team, p.teams, blockDim.x);
  const int tid = threadIdx.x, lane32 = tid & 31;
  const int slot = tid / p.team, lane = tid - slot * p.team;
  int hl, u;
  const bool on = place(kHead, p.units, p.hpi, p.team, lane, &hl, &u) && slot < p.teams;
  const bool turned = u < p.turned;
  int e0, e1;  // features of the unit's two vectors
  vectors_of<V, kHalf>(p, u, &e0, &e1);
  const uint32_t past = kLayout == kPart ? pairs_past<V>(p, u) : 0u;
  const int group = p.team < 32 ? p.team : 32, in_group = tid & (group - 1);
  float4* const angles = reinterpret_cast<float4*>(smem) + tid / group * kP * kColumn;  // [kP][kColumn]
  float4* const weights = reinterpret_cast<float4*>(smem + plan.weights);
  float* const sums_s = smem + plan.sums;

  // the norm's weights, (a.x, a.y, b.x, b.y) of each pair of a unit: for the
  // norm per token [warp of the team][kM][kP][lane], per head [queries,
  // keys][kP][unit]
  if (kAny) {
    const int n = kToken ? kM * p.team : 2 * p.units;
    for (int i = tid; i < n; i += blockDim.x) {
      const int m = kToken ? i / p.team : i / p.units;
      const int t = kToken ? i - m * p.team : i - m * p.units;
      int h = 0, ul = t;
      bool real = true;
      if (kToken) {
        real = place(kHead, p.units, p.hpi, p.team, t, &h, &ul);
        h += m * p.hpi;
        real = real && h < p.Ht;
      }
      const bool key = kToken ? h >= p.H : m == 1;
      const float* w = key ? p.w[1] : p.w[0];
      if (kToken && w) w += (key ? h - p.H : h) * p.D;
      int f0, f1;
      vectors_of<V, kHalf>(p, ul, &f0, &f1);
      for (int q = 0; q < kP; ++q) {
        float v[4];
        for (int c = 0; c < 4; ++c) {
          const int e = 2 * q + (c & 1);  // pair of the unit
          v[c] = w && real && (V > 1 || !(c & 1)) ? __ldg(w + feature<V, kHalf>((c >> 1) * (V > 1 ? V : 1) + e, f0, f1)) : 1.0f;
        }
        weights[kToken ? ((t / 32 * kM + m) * kP + q) * 32 + t % 32 : (m * kP + q) * kColumn + t] =
            make_float4(v[0], v[1], v[2], v[3]);
      }
    }
    __syncthreads();
  }
  const float4* const my_weights = kToken ? weights + lane / 32 * kM * kP * 32 + lane % 32 : weights + u;
  // weights of the unit's pairs q in round m of a head
  auto weight = [&](int m, bool key, int q) {
    return kToken ? my_weights[(m * kP + q) * 32] : my_weights[(key ? kP * kColumn : 0) + q * kColumn];
  };

  constexpr int kAcc = kBwd ? (kToken ? kM : 2) : 1;
  Unit<V> acc[kAcc];
  if (kBwd) {
#pragma unroll
    for (int i = 0; i < kAcc; ++i)
#pragma unroll
      for (int q = 0; q < kP; ++q) acc[i].a[q] = acc[i].b[q] = splat<F>(0.0f);
  }
  const float inv_nq = 1.0f / static_cast<float>(kHead ? p.D : p.D * p.H);
  const float inv_nk = 1.0f / static_cast<float>(kHead ? p.D : p.D * max(p.Ht - p.H, 1));
  const int step = gridDim.x * p.teams;
  const int chunks = kToken ? 1 : p.chunks;
  const int apart = 2 * (e1 - e0);
  // The unit's first vector in head 0 (keys: head -H) of token l of a row.
  auto start_at = [&](const View (&v)[2], int row, int l, char* (&to)[2]) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
      to[k] = v[k].data + row * v[k].b + l * v[k].l + 2 * e0 - (k ? static_cast<int64_t>(p.H) * v[1].h : 0);
  };
  auto step_on = [&](const View (&v)[2], char* (&to)[2]) {
    to[0] += v[0].step;
    to[1] += v[1].step;
  };
  auto head_at = [&](const View (&v)[2], char* const (&to)[2], int h) {
    const bool key = h >= p.H;
    return (key ? to[1] : to[0]) + static_cast<int64_t>(h) * (key ? v[1].h : v[0].h);
  };
  // A thread's vectors of kM heads (x0, x1, and backward g0, g1 of each).
  // With a norm they are copied one item (a token's kM heads a thread) ahead
  // into the thread's own part of a ring: no other thread reads it, so waiting
  // for the copies is all the synchronisation.  Without a norm a thread works
  // so little on them that direct loads and more threads are faster (64k pack,
  // blocks of four warps: 138 us against 146).
  constexpr bool kAsync = V > 1 && kAny;
  constexpr int kVecs = kBwd ? 4 : 2;
  T* const ring = reinterpret_cast<T*>(smem + plan.ring) + (tid >> 5) * kRing * kM * kVecs * 32 + lane32;
  int turn = 0;
  for (int row = blockIdx.y; row < p.rows; row += gridDim.y) {
    const int base0 = blockIdx.x * p.teams;
    int l = base0 + slot, lf = l, cf = 0, held = 0, to = 0;  // token; token and heads of the next copies; ring stages
    char *xp[2], *gp[2], *op[2];
    start_at(p.x, row, l, xp);
    if (kBwd) start_at(p.g, row, l, gp);
    start_at(p.out, row, l, op);
    auto fetch = [&]() {
      T* dst = ring + to * kM * kVecs * 32;
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        const int h = hl + (cf * kM + m) * p.hpi;
        if (on && lf < p.L && h < p.Ht) {
          const char* q = head_at(p.x, xp, h);
          copy_async<kBwd>(dst + (m * kVecs) * 32, q);
          copy_async<kBwd>(dst + (m * kVecs + 1) * 32, q + apart);
          if (kBwd) {
            q = head_at(p.g, gp, h);
            copy_async<kBwd>(dst + (m * kVecs + 2) * 32, q);
            copy_async<kBwd>(dst + (m * kVecs + 3) * 32, q + apart);
          }
        }
      }
      copy_commit();
      to = to + 1 == kRing ? 0 : to + 1;
      if (++cf == chunks) {
        cf = 0;
        lf += step;
        step_on(p.x, xp);
        if (kBwd) step_on(p.g, gp);
      }
    };
    if constexpr (kAsync) {
#pragma unroll
      for (int s = 0; s < kRing - 1; ++s) fetch();
    }
    const int32_t* pp = p.positions + (static_cast<size_t>(row) * p.L + l) * p.axes;
    int32_t pos[3] = {0, 0, 0};
    auto positions = [&](bool some) {
#pragma unroll
      for (int a = 0; a < 3; ++a)
        if (some && a < p.axes) pos[a] = __ldg(pp + a);
      pp += static_cast<size_t>(step) * p.axes;
    };
    positions(l < p.L);
    for (int base = base0; base < p.L; base += step, l += step) {
      const bool live = on && l < p.L;
      for (int chunk = 0; chunk < chunks; ++chunk) {
        const int h0 = hl + chunk * kM * p.hpi;
        T vx[kAsync ? 1 : kM][kVecs];
        if (kAsync) vx[0][0] = vx[0][1] = T{};  // not used
        if constexpr (kAsync) {
          fetch();
          copy_wait<kRing - 1>();
        } else {
#pragma unroll
          for (int m = 0; m < kM; ++m) {
            const int h = min(h0 + m * p.hpi, p.Ht - 1);
            const char *q = head_at(p.x, xp, h), *d = kBwd ? head_at(p.g, gp, h) : nullptr;
            if (live) {
              vx[kAsync ? 0 : m][0] = *reinterpret_cast<const T*>(q);
              vx[kAsync ? 0 : m][1] = *reinterpret_cast<const T*>(q + apart);
              if (kBwd) {
                vx[kAsync ? 0 : m][kVecs - 2] = *reinterpret_cast<const T*>(d);
                vx[kAsync ? 0 : m][kVecs - 1] = *reinterpret_cast<const T*>(d + apart);
              }
            }
          }
        }
        const T* const mine = ring + held * kM * kVecs * 32;
        auto vec = [&](int m, int j) { return kAsync ? mine[(m * kVecs + j) * 32] : vx[kAsync ? 0 : m][j]; };
        if (chunk == 0) {
          // the token's angles
          __syncwarp();
          for (int i = in_group; i < p.turned * V; i += group) {
            int unit, e;
            if constexpr (kHalf || V == 1) {
              unit = i / V;
              e = i % V;
            } else {
              const int side = i >= p.D / 4, j = i - side * (p.D / 4);
              unit = j / (V / 2);
              e = j % (V / 2) + side * (V / 2);
            }
            float* q = reinterpret_cast<float*>(angles + (e / 2) * kColumn + unit) + (e & 1);
            if (kHalf || i < p.R / 2) {
              const int32_t n = i < p.section_1 ? pos[0] : i < p.section_2 ? pos[1] : pos[2];
              // the product mod 2^64, its upper half: n times the lower word
              // carries, a negative n borrows
              const uint64_t f = __ldg(p.turns + i);
              const uint32_t flo = static_cast<uint32_t>(f), fhi = static_cast<uint32_t>(f >> 32);
              const uint32_t un = static_cast<uint32_t>(n);
              const uint32_t frac = __umulhi(flo, un) + fhi * un - (n < 0 ? flo : 0u);
              const float t = static_cast<float>(static_cast<int32_t>(frac)) * kRadians;
              q[0] = __cosf(t) * p.gain;
              q[2] = __sinf(t) * p.sign;
            } else {
              q[0] = 1.0f;
              q[2] = 0.0f;
            }
          }
          __syncwarp();
          positions(l + step < p.L);  // the next token's
        }
        auto rotate = [&](Unit<V>& z) {
          auto turn_pair = [&](int q, F& a, F& b) {
            const float4 t = angles[q * kColumn + u];
            const F c = side_a<F>(t), s = side_b<F>(t), a0 = a;
            a = ffma2(a0, c, fmul2(b, minus(s)));
            b = ffma2(a0, s, fmul2(b, c));
          };
#pragma unroll
          for (int q = 0; q < kP; ++q) {
            F a = z.a[q], b = z.b[q];
            turn_pair(q, a, b);
            if (kLayout == kPart) {
              take_unless(past >> 2 * q, a, z.a[q]);
              take_unless(past >> 2 * q, b, z.b[q]);
            } else {
              z.a[q] = a;
              z.b[q] = b;
            }
          }
        };
        // the norms' sums; backward the gradient is turned back on the way
        float r[kM], mean[kM];  // 1 / rms; backward -mean(g w xh) / rms
        Unit<V> g[kBwd ? kM : 1];
        if (kAny) {
          float part[kM][kSums];
#pragma unroll
          for (int m = 0; m < kM; ++m) {
            const int h = h0 + m * p.hpi;
            const bool real = live && h < p.Ht;
            Unit<V> x;
            unpack<V, kHalf>(vec(m, 0), vec(m, 1), x);
            F s = splat<F>(0.0f);
#pragma unroll
            for (int q = 0; q < kP; ++q) s = ffma2(x.a[q], x.a[q], ffma2(x.b[q], x.b[q], s));
            part[m][0] = real ? both_of(s) : 0.0f;
            if (kBwd) {
              Unit<V>& z = g[kBwd ? m : 0];
              unpack<V, kHalf>(vec(m, kVecs - 2), vec(m, kVecs - 1), z);
              if (turned) rotate(z);
              s = splat<F>(0.0f);
#pragma unroll
              for (int q = 0; q < kP; ++q) {
                const float4 w = weight(m, h >= p.H, q);
                s = ffma2(fmul2(z.a[q], side_a<F>(w)), x.a[q], s);
                s = ffma2(fmul2(z.b[q], side_b<F>(w)), x.b[q], s);
              }
              part[m][kSums - 1] = real ? both_of(s) : 0.0f;
            }
          }
          if (kHead) {
            if (p.units == 8) {
#pragma unroll
              for (int m = 0; m < kM; ++m)
#pragma unroll
                for (int k = 0; k < kSums; ++k)
#pragma unroll
                  for (int o = 1; o < 8; o <<= 1) part[m][k] += __shfl_xor_sync(0xffffffffu, part[m][k], o);
            } else if (p.units <= 32) {
#pragma unroll
              for (int m = 0; m < kM; ++m)
#pragma unroll
                for (int k = 0; k < kSums; ++k) part[m][k] = head_sum(part[m][k], u, p.units);
            } else {
              const int n = blockDim.x;
              __syncthreads();
#pragma unroll
              for (int m = 0; m < kM; ++m)
#pragma unroll
                for (int k = 0; k < kSums; ++k) sums_s[(m * kSums + k) * n + tid] = part[m][k];
              __syncthreads();
#pragma unroll
              for (int m = 0; m < kM; ++m)
#pragma unroll
                for (int k = 0; k < kSums; ++k) {
                  const float* q = sums_s + (m * kSums + k) * n + tid - u;
                  float t = 0.0f;
                  if (on)
                    for (int i = 0; i < p.units; ++i) t += q[i];
                  part[m][k] = t;
                }
            }
#pragma unroll
            for (int m = 0; m < kM; ++m) {
              r[m] = rsqrtf(fmaf(part[m][0], inv_nq, p.eps));
              mean[m] = kBwd ? -r[m] * r[m] * (part[m][kSums - 1] * inv_nq) : 0.0f;
            }
          } else {
            // queries and keys apart: sums of x^2 of both, then of g w x
            float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int m = 0; m < kM; ++m) {
              const bool key = h0 + m * p.hpi >= p.H;
#pragma unroll
              for (int k = 0; k < kSums; ++k) {
                sum[2 * k] += key ? 0.0f : part[m][k];
                sum[2 * k + 1] += key ? part[m][k] : 0.0f;
              }
            }
            if (p.team >= 32) {
              // halves of the values are exchanged until a lane holds one
              int o = 16;
#pragma unroll
              for (int n = 2 * kSums; n > 1; n >>= 1, o >>= 1) {
                const bool up = lane32 & o;
#pragma unroll
                for (int j = 0; j < n / 2; ++j) {
                  const float keep = up ? sum[j + n / 2] : sum[j], send = up ? sum[j] : sum[j + n / 2];
                  sum[j] = keep + __shfl_xor_sync(0xffffffffu, send, o);
                }
              }
#pragma unroll
              for (int q = 16 / (2 * kSums); q >= 1; q >>= 1) sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], q);
              constexpr int kLanes = 32 / (2 * kSums);  // that hold one value
              if (p.team == 32) {
                const float t = sum[0];
#pragma unroll
                for (int k = 0; k < 2 * kSums; ++k) sum[k] = __shfl_sync(0xffffffffu, t, k * kLanes);
              } else {
                // a warp's values side by side, in two tables by turns: one
                // barrier a token
                float* q = sums_s + turn * (blockDim.x / 32) * 4;
                if ((lane32 & (kLanes - 1)) == 0) q[(tid >> 5) * 4 + lane32 / kLanes] = sum[0];
                __syncthreads();
                const float4* t = reinterpret_cast<const float4*>(q) + slot * (p.team / 32);
                float4 v = t[0];
                for (int w = 1; w < p.team / 32; ++w) {
                  const float4 x = t[w];
                  v.x += x.x;
                  v.y += x.y;
                  v.z += x.z;
                  v.w += x.w;
                }
                sum[0] = v.x;
                sum[1] = v.y;
                sum[2] = v.z;
                sum[3] = v.w;
                turn ^= 1;
              }
            } else {
#pragma unroll
              for (int k = 0; k < 2 * kSums; ++k) sum[k] = lane_sum(sum[k], group);
            }
            const float rq = rsqrtf(fmaf(sum[0], inv_nq, p.eps)), rk = rsqrtf(fmaf(sum[1], inv_nk, p.eps));
            const float mq = kBwd ? -rq * rq * (sum[2] * inv_nq) : 0.0f, mk = kBwd ? -rk * rk * (sum[3] * inv_nk) : 0.0f;
#pragma unroll
            for (int m = 0; m < kM; ++m) {
              const bool key = h0 + m * p.hpi >= p.H;
              r[m] = key ? rk : rq;
              mean[m] = key ? mk : mq;
            }
          }
        }
#pragma unroll
        for (int m = 0; m < kM; ++m) {
          const int h = h0 + m * p.hpi;
          if (live && h < p.Ht) {
            const bool key = h >= p.H;
            Unit<V> z;
            unpack<V, kHalf>(vec(m, 0), vec(m, 1), z);
            if (kBwd) {
              const Unit<V>& d = g[kBwd ? m : 0];
              const F rr = splat<F>(r[m]), mm = splat<F>(mean[m]);
#pragma unroll
              for (int q = 0; q < kP; ++q) {
                const float4 w = weight(m, key, q);
                z.a[q] = fmul2(z.a[q], rr);  // xh
                z.b[q] = fmul2(z.b[q], rr);
                if (kToken) {
                  Unit<V>& s = acc[kAcc > 1 ? m : 0];
                  s.a[q] = ffma2(z.a[q], d.a[q], s.a[q]);
                  s.b[q] = ffma2(z.b[q], d.b[q], s.b[q]);
                } else if (key) {
                  acc[kAcc - 1].a[q] = ffma2(z.a[q], d.a[q], acc[kAcc - 1].a[q]);
                  acc[kAcc - 1].b[q] = ffma2(z.b[q], d.b[q], acc[kAcc - 1].b[q]);
                } else {
                  acc[0].a[q] = ffma2(z.a[q], d.a[q], acc[0].a[q]);
                  acc[0].b[q] = ffma2(z.b[q], d.b[q], acc[0].b[q]);
                }
                z.a[q] = ffma2(fmul2(d.a[q], side_a<F>(w)), rr, fmul2(z.a[q], mm));
                z.b[q] = ffma2(fmul2(d.b[q], side_b<F>(w)), rr, fmul2(z.b[q], mm));
              }
            } else {
              if (kAny) {
                const F rr = splat<F>(r[m]);
#pragma unroll
                for (int q = 0; q < kP; ++q) {
                  const float4 w = weight(m, key, q);
                  z.a[q] = fmul2(fmul2(z.a[q], rr), side_a<F>(w));
                  z.b[q] = fmul2(fmul2(z.b[q], rr), side_b<F>(w));
                }
              }
              if (turned) rotate(z);
            }
            T o0, o1;
            pack<V, kHalf>(z, o0, o1);
            char* q = head_at(p.out, op, h);
            *reinterpret_cast<T*>(q) = o0;
            *reinterpret_cast<T*>(q + apart) = o1;
          }
        }
        held = held + 1 == kRing ? 0 : held + 1;
      }
      step_on(p.out, op);
      if constexpr (!kAsync) {
        step_on(p.x, xp);
        if (kBwd) step_on(p.g, gp);
      }
    }
    if constexpr (kAsync) copy_wait<0>();
  }
  if (kBwd) {
    if (p.part == nullptr) return;
    constexpr int kValues = V > 1 ? 2 * V : 2;
    // value k of a unit's sums
    auto value = [](const Unit<V>& s, int k) {
      const int e = k % (V > 1 ? V : 1), side = k / (V > 1 ? V : 1);
      const F t = side ? s.b[e / 2] : s.a[e / 2];
      if constexpr (V > 1) return e & 1 ? t.y : t.x;
      else return t;
    };
    // the block's sums, in the ring's place (it is done with): of its teams,
    // and with the norm per head of all heads, queries and keys in turn
    float* out = p.part + static_cast<size_t>(blockIdx.y * gridDim.x + blockIdx.x) * p.width;
    float* const table = smem + plan.ring;
    if (kToken) {
      // teams are not in step behind their last barrier (of one warp or less
      // they never are): every ring is done with before a table overwrites it
      if (p.teams > 1) __syncthreads();
      if (on) {
#pragma unroll
        for (int m = 0; m < kM; ++m) {
          const int h = hl + m * p.hpi;
          if (h < p.Ht) {
#pragma unroll
            for (int k = 0; k < kValues; ++k)
              (p.teams == 1 ? out : table + slot * p.width)[h * p.D + feature<V, kHalf>(k, e0, e1)] =
                  value(acc[kAcc > 1 ? m : 0], k);
          }
        }
      }
      if (p.teams == 1) return;
      __syncthreads();
      for (int d = tid; d < p.width; d += blockDim.x) {
        float t = 0.0f;
        for (int j = 0; j < p.teams; ++j) t += table[j * p.width + d];
        out[d] = t;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        __syncthreads();
        if (on) {
#pragma unroll
          for (int k = 0; k < kValues; ++k)
            table[(slot * p.hpi + hl) * p.D + feature<V, kHalf>(k, e0, e1)] = value(acc[i ? kAcc - 1 : 0], k);
        }
        __syncthreads();
        for (int d = tid; d < p.D; d += blockDim.x) {
          float t = 0.0f;
          for (int j = 0; j < p.teams * p.hpi; ++j) t += table[j * p.D + d];
          out[i * p.D + d] = t;
        }
      }
    }
  }
}

// Column sums of the [rows][width] partials, added in a fixed order: a CTA
// takes 32 columns, warp w the rows w, w + 32, ...
__global__ void __launch_bounds__(1024) rotary_weights_kernel(const float* __restrict__ part, int rows, int width,
                                                              int q_width, float* __restrict__ dwq,
                                                              float* __restrict__ dwk) {
  __shared__ float acc[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  float t = 0.0f;
  if (col < width) {
#pragma unroll 8
    for (int i = w; i < rows; i += 32) t += __ldg(part + static_cast<size_t>(i) * width + col);
  }
  acc[w][lane] = t;
  __syncthreads();
  if (w == 0 && col < width) {
    t = 0.0f;
    for (int i = 0; i < 32; ++i) t += acc[i][lane];
    if (col < q_width) {
      if (dwq) dwq[col] = t;
    } else if (dwk) {
      dwk[col - q_width] = t;
    }
  }
}

struct Shape {
  int V, kM, units, hpi, team, teams, threads;
};

int round32(int n) { return (n + 31) / 32 * 32; }

// The team of a token for vectors V wide and kM heads a thread: a power of
// two below 32 threads, or whole warps.  False where one pass over a token's
// heads does not fit a block and the norm per token needs it: by its threads,
// or backward, with 384 of them on 8-wide vectors (from 16,800 features on),
// by its shared memory.
bool team_of(int V, int kM, int Ht, int D, int norm, bool bwd, Shape* s) {
  s->V = V;
  s->kM = kM;
  s->units = D / (2 * V);
  const int want = (Ht + kM - 1) / kM;  // heads at once
  if (s->units * want <= 32) {
    s->team = 1;
    while (s->team < s->units * want) s->team <<= 1;
    s->hpi = std::min(Ht, s->team / s->units);
  } else {
    const int per = norm == PVL_NORM_HEAD ? 32 / s->units : 0;  // heads of a warp, where they keep to one
    const int most = per ? per * (kMaxBlock / 32) : kMaxBlock / s->units;
    if (want > most && norm == PVL_NORM_TOKEN) return false;
    s->hpi = std::min(want, most);
    s->team = per ? (s->hpi + per - 1) / per * 32 : round32(s->units * s->hpi);
    // heads that the rounding leaves room for
    s->hpi = std::min(Ht, per ? s->team / 32 * per : s->team / s->units);
  }
  // Without a norm teams share nothing but the block, and 8-wide vectors want
  // eight warps of them (64k pack, 12 + 12 heads of 128: 126 us; four warps 138,
  // twelve 137; heads of 64: 67, 72, 75); 4-wide ones four (129; eight 132), and
  // teams of part of a warp two (2 + 1 heads: 28; eight 31).  Few tokens (one
  // head a thread) want many blocks.
  const int threads = norm == PVL_NORM_NONE && V == 8 && kM > 1 && s->team >= 32 ? 256 : s->team < 32 ? 64 : 128;
  s->teams = s->team >= threads ? 1 : threads / s->team;
  s->threads = s->team * s->teams;
  const SmemPlan plan = smem_plan(V, kM, norm, bwd, Ht, D, s->units, s->hpi, s->team, s->teams, s->threads);
  return sizeof(float) * plan.total <= kMaxSmem;
}

template <int V, int kM, int kNorm, bool kBwd>
const void* kernel_of(int layout) {
  if (layout == PVL_ROTARY_HALF)
    return reinterpret_cast<const void*>(&rotary_kernel<V, kM, kNorm, kBwd, PVL_ROTARY_HALF>);
  if (layout == kPart) return reinterpret_cast<const void*>(&rotary_kernel<V, kM, kNorm, kBwd, kPart>);
  return reinterpret_cast<const void*>(&rotary_kernel<V, kM, kNorm, kBwd, PVL_ROTARY_INTERLEAVED>);
}

// The kernels that exist (shape_of picks among the same).
const void* find_kernel(const Shape& s, int norm, bool bwd, int layout) {
#define PVL_ROTARY_KERNEL(VV, MM, NN, BB) \
  if (s.V == VV && s.kM == MM && norm == NN && bwd == BB) return kernel_of<VV, MM, NN, BB>(layout)
  PVL_ROTARY_KERNEL(8, 1, PVL_NORM_NONE, false);
  PVL_ROTARY_KERNEL(8, 3, PVL_NORM_NONE, false);
  PVL_ROTARY_KERNEL(4, 4, PVL_NORM_NONE, false);
  PVL_ROTARY_KERNEL(2, 8, PVL_NORM_NONE, false);
  PVL_ROTARY_KERNEL(1, 8, PVL_NORM_NONE, false);
  PVL_ROTARY_KERNEL(8, 1, PVL_NORM_HEAD, false);
  PVL_ROTARY_KERNEL(8, 3, PVL_NORM_HEAD, false);
  PVL_ROTARY_KERNEL(4, 4, PVL_NORM_HEAD, false);
  PVL_ROTARY_KERNEL(2, 8, PVL_NORM_HEAD, false);
  PVL_ROTARY_KERNEL(1, 8, PVL_NORM_HEAD, false);
  PVL_ROTARY_KERNEL(8, 1, PVL_NORM_HEAD, true);
  PVL_ROTARY_KERNEL(8, 2, PVL_NORM_HEAD, true);
  PVL_ROTARY_KERNEL(4, 4, PVL_NORM_HEAD, true);
  PVL_ROTARY_KERNEL(2, 8, PVL_NORM_HEAD, true);
  PVL_ROTARY_KERNEL(1, 8, PVL_NORM_HEAD, true);
  PVL_ROTARY_KERNEL(8, 1, PVL_NORM_TOKEN, false);
  PVL_ROTARY_KERNEL(8, 3, PVL_NORM_TOKEN, false);
  PVL_ROTARY_KERNEL(8, 6, PVL_NORM_TOKEN, false);
  PVL_ROTARY_KERNEL(4, 4, PVL_NORM_TOKEN, false);
  PVL_ROTARY_KERNEL(2, 8, PVL_NORM_TOKEN, false);
  PVL_ROTARY_KERNEL(1, 8, PVL_NORM_TOKEN, false);
  PVL_ROTARY_KERNEL(1, 16, PVL_NORM_TOKEN, false);
  PVL_ROTARY_KERNEL(8, 1, PVL_NORM_TOKEN, true);
  PVL_ROTARY_KERNEL(8, 3, PVL_NORM_TOKEN, true);
  PVL_ROTARY_KERNEL(4, 4, PVL_NORM_TOKEN, true);
  PVL_ROTARY_KERNEL(2, 8, PVL_NORM_TOKEN, true);
  PVL_ROTARY_KERNEL(1, 8, PVL_NORM_TOKEN, true);
  PVL_ROTARY_KERNEL(1, 16, PVL_NORM_TOKEN, true);
#undef PVL_ROTARY_KERNEL
  return nullptr;
}

pvl_status launch(const RotaryParams& p, const Shape& sh, int norm, bool bwd, int layout, int grid_limit, int* grid_out,
                  cudaStream_t s, const char* who) {
  const void* fn = find_kernel(sh, norm, bwd, layout == PVL_ROTARY_INTERLEAVED && p.R < p.D ? kPart : layout);
  if (!fn) return fail(PVL_ERR_UNSUPPORTED, "%s: no kernel for this shape", who);
  const size_t smem =
      sizeof(float) * smem_plan(sh.V, sh.kM, norm, bwd, p.Ht, p.D, sh.units, sh.hpi, sh.team, sh.teams, sh.threads).total;
  const int occ = blocks_per_sm(fn, sh.threads, smem), sms = sm_count();
  if (sms <= 0 || occ <= 0) return fail(PVL_ERR_CUDA, "%s: no usable CUDA device", who);
  long long grid = static_cast<long long>(occ) * sms;
  if (grid > grid_limit) grid = grid_limit;
  const long long gy = std::min<long long>({p.rows, grid, 65535});
  const long long gx = std::min<long long>(grid / gy, (static_cast<long long>(p.L) + p.teams - 1) / p.teams);
  *grid_out = static_cast<int>(gx * gy);
  RotaryParams q = p;
  for (View* v : {q.x, q.g, q.out})
    for (int i = 0; i < 2; ++i) v[i].step = gx * p.teams * v[i].l;
  void* args[] = {&q};
  return check_cuda(cudaLaunchKernel(fn, dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy)), dim3(sh.threads),
                                     args, smem, s),
                    who);
}

// Widest vector that divides the head, its rotated part (half layout), every
// stride and every address.
int widest(const pvl_rotary* a, const pvl_heads* const* views, int n) {
  for (int V : {8, 4, 2}) {
    bool ok = a->D % (2 * V) == 0 && (a->layout != PVL_ROTARY_HALF || a->R % (2 * V) == 0);
    for (int i = 0; i < n && ok; ++i)
      if (views[i])
        ok = reinterpret_cast<uintptr_t>(views[i]->data) % (2 * V) == 0 && views[i]->stride_b % V == 0 &&
             views[i]->stride_l % V == 0 && views[i]->stride_h % V == 0;
    if (ok) return V;
  }
  return 1;
}

// Heads a thread at a time.  One up to two tokens an SM, where latency counts
// (most threads, fewest dependent steps; 12 + 12 heads of 128, 304 tokens and,
// past the border, 305, in a graph: forward without a norm 2.65 and 2.68 us, per
// head 3.26 and 3.41, over the token 3.58 and 4.15; backward per head 3.70 and
// 3.99, over the token 3.98 and 4.57); else the largest count that a kernel
// exists for whose registers hold it.
bool shape_of(const pvl_rotary* a, int V, bool bwd, Shape* s) {
  const int Ht = a->H + a->Hk;
  const bool whole = a->norm == PVL_NORM_TOKEN;
  if (V != 8 && team_of(V, V == 4 ? 4 : 8, Ht, a->D, a->norm, bwd, s)) return true;
  if (V != 8) return V == 1 && team_of(V, 16, Ht, a->D, a->norm, bwd, s);
  const long long tokens = static_cast<long long>(a->B) * a->L;
  if (tokens <= 2ll * sm_count() && team_of(8, 1, Ht, a->D, a->norm, bwd, s)) return true;
  if (!whole) return team_of(8, bwd ? 2 : 3, Ht, a->D, a->norm, bwd, s);
  // six while a token stays within two warps, else more warps count for more
  // (10,240 features a token: 215 us at six, 178 at three; 6,144: 165, 177)
  if (!bwd && Ht * a->D <= 6144 && team_of(8, 6, Ht, a->D, a->norm, bwd, s)) return true;
  return team_of(8, 3, Ht, a->D, a->norm, bwd, s);
}

pvl_status check_views(const char* who, const pvl_rotary* a, const pvl_heads* v, int which, const char* name,
                       bool written = false) {
  const int heads = which ? a->Hk : a->H;
  if (heads == 0) return PVL_OK;
  if (!v || !v->data) return fail(PVL_ERR_INVALID_ARG, "%s: %s is null", who, name);
  if (reinterpret_cast<uintptr_t>(v->data) % 2 != 0)
    return fail(PVL_ERR_UNSUPPORTED, "%s: %s is not 2-byte aligned", who, name);
  // several threads would write one place
  if (written && ((a->B > 1 && v->stride_b == 0) || (a->L > 1 && v->stride_l == 0) || (heads > 1 && v->stride_h == 0)))
    return fail(PVL_ERR_INVALID_ARG, "%s: %s is broadcast (a stride of 0)", who, name);
  return PVL_OK;
}

pvl_status common(const char* who, const pvl_rotary* a, RotaryParams& p) {
  if (!a) return fail(PVL_ERR_INVALID_ARG, "%s: null description", who);
  if (a->B < 1 || a->L < 1 || a->H < 1 || a->Hk < 0 || a->D < 1 || a->R < 0)
    return fail(PVL_ERR_INVALID_ARG, "%s: B, L, H, D must be >= 1, Hk and R >= 0", who);
  if (a->layout != PVL_ROTARY_HALF && a->layout != PVL_ROTARY_INTERLEAVED)
    return fail(PVL_ERR_INVALID_ARG, "%s: layout %d", who, a->layout);
  if (a->norm != PVL_NORM_NONE && a->norm != PVL_NORM_HEAD && a->norm != PVL_NORM_TOKEN)
    return fail(PVL_ERR_INVALID_ARG, "%s: norm %d", who, a->norm);
  if (a->axes < 1 || a->axes > 3) return fail(PVL_ERR_INVALID_ARG, "%s: axes = %d (1 to 3)", who, a->axes);
  if (a->D % 2 != 0 || a->R % 2 != 0 || a->D > kMaxD)
    return fail(PVL_ERR_UNSUPPORTED, "%s: D = %d, R = %d (supported: even, D up to %d)", who, a->D, a->R, kMaxD);
  if (a->R > a->D) return fail(PVL_ERR_INVALID_ARG, "%s: R = %d exceeds D = %d", who, a->R, a->D);
  if (a->section_1 < 0 || a->section_2 < a->section_1 || a->section_2 > a->R / 2 ||
      (a->axes < 2 && a->section_1 != a->R / 2) || (a->axes < 3 && a->section_2 != a->R / 2))
    return fail(PVL_ERR_INVALID_ARG, "%s: sections %d, %d of %d pairs with %d axes", who, a->section_1, a->section_2,
                a->R / 2, a->axes);
  if (!a->positions || (a->R > 0 && !a->turns)) return fail(PVL_ERR_INVALID_ARG, "%s: null pointer", who);
  if (reinterpret_cast<uintptr_t>(a->positions) % 4 != 0 || reinterpret_cast<uintptr_t>(a->turns) % 8 != 0 ||
      reinterpret_cast<uintptr_t>(a->q_weight) % 4 != 0 || reinterpret_cast<uintptr_t>(a->k_weight) % 4 != 0)
    return fail(PVL_ERR_UNSUPPORTED, "%s: a table is not aligned to its type", who);
  if (!(a->gain > -1e30f && a->gain < 1e30f)) return fail(PVL_ERR_INVALID_ARG, "%s: gain must be finite", who);
  if (!(a->eps >= 0.0f) || !(a->eps < 1e30f)) return fail(PVL_ERR_INVALID_ARG, "%s: eps must be >= 0 and finite", who);
  if (a->norm == PVL_NORM_NONE && (a->q_weight || a->k_weight))
    return fail(PVL_ERR_INVALID_ARG, "%s: a weight without a norm", who);
  if (a->Hk == 0 && a->k_weight) return fail(PVL_ERR_INVALID_ARG, "%s: k_weight without keys", who);
  if (static_cast<long long>(a->H) + a->Hk > PVL_MAX_ROTARY_HEADS)
    return fail(PVL_ERR_UNSUPPORTED, "%s: %d + %d heads", who, a->H, a->Hk);
  if (static_cast<long long>(a->B) * a->L >= (1ll << 30))
    return fail(PVL_ERR_UNSUPPORTED, "%s: too many tokens", who);
  p.turns = a->turns;
  p.positions = a->positions;
  p.w[0] = a->q_weight;
  p.w[1] = a->k_weight;
  p.L = a->L;
  p.rows = a->B;
  p.H = a->H;
  p.Ht = a->H + a->Hk;
  p.D = a->D;
  p.R = a->R;
  p.axes = a->axes;
  p.section_1 = a->section_1;
  p.section_2 = a->section_2;
  p.gain = p.sign = a->gain;
  p.eps = a->eps;
  return PVL_OK;
}

// A view in bytes; an absent tensor's stays zero.
bool view(const pvl_heads* h, View* v) {
  if (!h) return true;
  if (h->stride_h >= 1 << 30 || h->stride_h <= -(1 << 30)) return false;
  *v = View{static_cast<char*>(h->data), 2 * h->stride_b, 2 * h->stride_l, 0, static_cast<int32_t>(2 * h->stride_h)};
  return true;
}

// All tokens as one row where every tensor's batch stride continues its tokens.
void flatten(RotaryParams& p, bool grads) {
  const View* all[] = {&p.x[0], &p.x[1], &p.out[0], &p.out[1], grads ? &p.g[0] : nullptr, grads ? &p.g[1] : nullptr};
  for (const View* v : all)
    if (v && v->data && v->b != v->l * p.L && p.rows > 1) {
      if (p.L > 1) return;
    }
  if (p.L == 1)
    for (const View* v : all)
      if (v && v->data) const_cast<View*>(v)->l = v->b;
  p.L *= p.rows;
  p.rows = 1;
}

void fill(RotaryParams& p, const pvl_rotary* a, const Shape& s) {
  p.units = s.units;
  p.turned = a->layout == PVL_ROTARY_HALF ? a->R / (2 * s.V) : s.units;
  p.hpi = s.hpi;
  p.chunks = (p.Ht + s.kM * s.hpi - 1) / (s.kM * s.hpi);
  p.team = s.team;
  p.teams = s.teams;
  p.width = a->norm == PVL_NORM_TOKEN ? (a->H + a->Hk) * a->D : 2 * a->D;
}

}  // namespace
}  // namespace pvl

using namespace pvl;

extern "C" pvl_status pack_rotary_fwd(const pvl_rotary* a, const pvl_heads* q, const pvl_heads* k,
                                      const pvl_heads* q_out, const pvl_heads* k_out, pvl_stream_t stream) {
  const char* who = "pack_rotary_fwd";
  RotaryParams p{};
  pvl_status st = common(who, a, p);
  if (st == PVL_OK) st = check_views(who, a, q, 0, "q");
  if (st == PVL_OK) st = check_views(who, a, k, 1, "k");
  if (st == PVL_OK) st = check_views(who, a, q_out, 0, "q_out", true);
  if (st == PVL_OK) st = check_views(who, a, k_out, 1, "k_out", true);
  if (st != PVL_OK) return st;
  if (!a->Hk) k = k_out = nullptr;
  const pvl_heads* views[] = {q, k, q_out, k_out};
  Shape s{};
  if (!shape_of(a, widest(a, views, 4), false, &s))
    return fail(PVL_ERR_UNSUPPORTED, "%s: a token of %d heads of %d features does not fit a block", who, p.Ht, p.D);
  fill(p, a, s);
  if (!view(q, &p.x[0]) || !view(k, &p.x[1]) || !view(q_out, &p.out[0]) || !view(k_out, &p.out[1]))
    return fail(PVL_ERR_UNSUPPORTED, "%s: a head stride of 2^30 elements or more", who);
  flatten(p, false);
  int grid = 0;
  return launch(p, s, a->norm, false, a->layout, 1 << 30, &grid,
                reinterpret_cast<cudaStream_t>(stream), who);
}

extern "C" size_t pack_rotary_bwd_ws_bytes(const pvl_rotary* a) {
  if (!a || a->norm == PVL_NORM_NONE || (!a->q_weight && !a->k_weight)) return 0;
  if (a->B < 1 || a->L < 1 || a->H < 1 || a->Hk < 0 || a->D < 1) return 0;
  const size_t width = a->norm == PVL_NORM_TOKEN ? static_cast<size_t>(a->H + a->Hk) * a->D : 2 * a->D;
  const long long tokens = static_cast<long long>(a->B) * a->L;
  return static_cast<size_t>(tokens < kMaxPartials ? tokens : kMaxPartials) * width * sizeof(float);
}

extern "C" pvl_status pack_rotary_bwd(const pvl_rotary* a, const pvl_heads* dq_out, const pvl_heads* dk_out,
                                      const pvl_heads* q, const pvl_heads* k, const pvl_heads* dq,
                                      const pvl_heads* dk, float* dq_weight, float* dk_weight, void* ws,
                                      size_t ws_bytes, pvl_stream_t stream) {
  const char* who = "pack_rotary_bwd";
  RotaryParams p{};
  pvl_status st = common(who, a, p);
  if (st == PVL_OK) st = check_views(who, a, dq_out, 0, "dq_out");
  if (st == PVL_OK) st = check_views(who, a, dk_out, 1, "dk_out");
  if (st == PVL_OK) st = check_views(who, a, dq, 0, "dq", true);
  if (st == PVL_OK) st = check_views(who, a, dk, 1, "dk", true);
  const bool norm = st == PVL_OK && a->norm != PVL_NORM_NONE;
  if (norm) st = check_views(who, a, q, 0, "q");
  if (norm && st == PVL_OK) st = check_views(who, a, k, 1, "k");
  if (st != PVL_OK) return st;
  if ((!!dq_weight != !!a->q_weight) || (!!dk_weight != !!a->k_weight))
    return fail(PVL_ERR_INVALID_ARG, "%s: one gradient for each weight, and no others", who);
  if (reinterpret_cast<uintptr_t>(dq_weight) % 4 != 0 || reinterpret_cast<uintptr_t>(dk_weight) % 4 != 0)
    return fail(PVL_ERR_UNSUPPORTED, "%s: a weight gradient is not 4-byte aligned", who);
  const bool weights = a->q_weight || a->k_weight;
  const size_t need = pack_rotary_bwd_ws_bytes(a);
  if (weights && (!ws || ws_bytes < need))
    return fail(PVL_ERR_INVALID_ARG, "%s: workspace %zu bytes < %zu needed", who, ws ? ws_bytes : 0, need);
  if (reinterpret_cast<uintptr_t>(ws) % 16 != 0)
    return fail(PVL_ERR_UNSUPPORTED, "%s: the workspace is not 16-byte aligned", who);
  if (!a->Hk) dk_out = dk = k = nullptr;
  if (!norm) q = k = nullptr;
  const pvl_heads* views[] = {dq_out, dk_out, dq, dk, q, k};
  Shape s{};
  if (!shape_of(a, widest(a, views, 6), norm, &s))
    return fail(PVL_ERR_UNSUPPORTED, "%s: a token of %d heads of %d features does not fit a block", who, p.Ht, p.D);
  fill(p, a, s);
  p.sign = -a->gain;  // turned back
  // without a norm the gradient is rotated in the input's place
  View* up = norm ? p.g : p.x;
  if (!view(dq_out, &up[0]) || !view(dk_out, &up[1]) || !view(dq, &p.out[0]) || !view(dk, &p.out[1]) ||
      (norm && (!view(q, &p.x[0]) || !view(k, &p.x[1]))))
    return fail(PVL_ERR_UNSUPPORTED, "%s: a head stride of 2^30 elements or more", who);
  flatten(p, norm);
  p.part = weights ? static_cast<float*>(ws) : nullptr;
  // a row of partial sums for each block
  const long long tokens = static_cast<long long>(a->B) * a->L;
  const int limit = weights ? static_cast<int>(std::min<long long>(tokens, kMaxPartials)) : 1 << 30;
  int grid = 0;
  cudaStream_t stm = reinterpret_cast<cudaStream_t>(stream);
  st = launch(p, s, a->norm, norm, a->layout, limit, &grid, stm, who);
  if (st != PVL_OK || !weights) return st;
  const int q_width = a->norm == PVL_NORM_TOKEN ? a->H * a->D : a->D;
  rotary_weights_kernel<<<(p.width + 31) / 32, 1024, 0, stm>>>(p.part, grid, p.width, q_width, dq_weight, dk_weight);
  return check_cuda(cudaGetLastError(), who);
}
