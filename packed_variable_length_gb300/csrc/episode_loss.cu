// pack_preference_*, pack_policy_*: losses of a packed policy over whole
// episodes, for sm_103a.
//
// Every token t of the pack carries an episode id e = seq_id[t] (negative:
// padding or prompt, not trained on) and its log-probability.
//
// Preference.  D_e = sum over the episode's tokens of logp - ref (divided by
// their number with `mean`); for a pair (c, r), h = D_c - D_r - margin, and
//   sigmoid  l = -(1 - s) log sigmoid(beta h) - s log sigmoid(-beta h)
//   squared  l = (h - 1 / (2 beta))^2
//   hinge    l = max(0, 1 - beta h)
// averaged over the pairs.  dl/dlogp_t = coef[e]: the forward leaves a table of
// one factor an episode, the backward spreads it over the tokens.
//
// Policy.  With d = logp - old and r = exp d (d averaged over the episode
// first where the ratio is the episode's), A the advantage,
//   l = -min(r A, clip(r, 1 - low, 1 + high) A) + kl_weight (exp f - f - 1),
// f = ref - logp, averaged over the valid tokens, or over the episodes' means.
// The gradient of the first term is -r A, or 0 where the clipped ratio is the
// smaller; of the second kl_weight (1 - exp f).
//
// Both are bound by latency: a 64k pack is 1.6 MB.  One kernel reads the
// tokens, four a thread; blocks whose tokens belong to one episode add one sum,
// others one per warp, or one per episode and warp and one per run of a thread
// whose tokens belong to several.  The last block to finish turns the episodes'
// sums into the loss and the table.
//
// Measured (one GB300; a captured forward and backward together, with the clear
// of the sums): the 64k pack's policy loss 17.4 us, 262,144 tokens of 512 episodes
// 18.8 us, preferences of four episodes of 10,944 tokens 12.7 us, of 512 episodes
// in 2048 pairs 18.9 us, of 4096 in 2048 pairs 47.0 us; what they move takes 0.1
// to 0.8 us.  (16.5, 17.7, 12.4, 18.6 and 46.9 us without units of 2^-80 and means
// of large terms.)  One cluster of eight blocks of 1024 threads instead, which
// needs no clear, took 24 us for the 64k pack: a token costs a hundred
// instructions, and eight SMs issue them.  Sums in 64-bit floating point took
// twice the time.
//
// Sums are integers, so that they are the same whatever order blocks finish in,
// and exact.  A token's value in units of 2^-40, with what is left in units of
// 2^-80 where that could be 2^-24 of a sum (each rounded once; differences are
// taken as exact pairs of fp32 values first), is added in 64 bits within the
// block, so that small advantages and divergences count as large ones do; an
// episode holds digits in base 2^40, from 2^-80 to 2^160, to which a block, warp
// or run adds by integer atomics.  Values of 2^11 and more go to the digits one by
// one, infinities and NaN to flags.  With at most 2^23 tokens a digit's sum stays
// below 2^63.  64-bit floating point, of which this GPU does little, is left to
// values that are large or below 2^-19.
#include <cuda_runtime.h>

#include <cmath>
#include <initializer_list>

#include "pvl_device.cuh"

namespace pvl {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kTokens = 4 * kThreads;  // of a block
constexpr int kBwdThreads = 256;
constexpr uint32_t kSiteEpisode = 71, kSitePair = 72;
constexpr long long kMaxTokens = 1ll << 23;
constexpr int kMaxEpisodes = 1 << 16;
constexpr int kMaxPairs = 1 << 20;
constexpr unsigned kAll = 0xffffffffu;

// ------------------------------------------------- pairs of fp32 values
// hi + lo with |lo| at most half a step of hi; lo = 0 where hi is not finite.
struct Pair {
  float hi, lo;
};

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < INFINITY; }

// The exact sum of two fp32 values (Knuth's two-sum).
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  const float e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
  return {s, finite(s) ? e : 0.0f};
}

// hi + lo for a small lo (Dekker's fast two-sum).
__device__ __forceinline__ Pair renormal(float hi, float lo) {
  const float s = __fadd_rn(hi, lo);
  return {s, finite(s) ? __fsub_rn(lo, __fsub_rn(s, hi)) : 0.0f};
}

__device__ __forceinline__ Pair add(Pair a, Pair b) {
  const Pair s = two_sum(a.hi, b.hi);
  return renormal(s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)));
}

__device__ __forceinline__ Pair times(float a, float b) {
  const float p = __fmul_rn(a, b);
  return {p, finite(p) ? fmaf(a, b, -p) : 0.0f};
}

__device__ __forceinline__ Pair over(Pair a, float n) {
  const float q = __fdiv_rn(a.hi, n);
  return finite(q) ? renormal(q, __fdiv_rn(__fadd_rn(fmaf(-q, n, a.hi), a.lo), n)) : Pair{q, 0.0f};
}

// ------------------------------------------------------------ exact sums
constexpr double kUp = 1099511627776.0;     // 2^40
constexpr float kFine = 1099511627776.0f;   // units of 2^-40
constexpr long long kMask = (1ll << 40) - 1;

struct Sum {
  long long digit[6];  // of weight 2^120, 2^80, 2^40, 1, 2^-40, 2^-80
};

__device__ __forceinline__ void add_digit(long long* d, long long v) {
  if (v) atomicAdd(reinterpret_cast<unsigned long long*>(d), static_cast<unsigned long long>(v));
}

// Adds v units of 2^-40.
__device__ __forceinline__ void add_units(Sum* s, long long v) {
  const unsigned long long m = v < 0 ? 0ull - static_cast<unsigned long long>(v) : static_cast<unsigned long long>(v);
  const long long whole = static_cast<long long>(m >> 40), part = static_cast<long long>(m) & kMask;
  add_digit(&s->digit[3], v < 0 ? -whole : whole);
  add_digit(&s->digit[4], v < 0 ? -part : part);
}

// Adds any x; what is not finite goes into three bits of *flags at `shift`.
__device__ __noinline__ void add_any(Sum* s, unsigned int* flags, int shift, double x) {
  if (!(fabs(x) < 1e300)) {
    atomicOr(flags, (x != x ? 1u : x > 0.0 ? 2u : 4u) << shift);
    return;
  }
  double weight = kUp * kUp * kUp;
#pragma unroll 1
  for (int i = 0; i < 6; ++i, weight *= 1.0 / kUp) {
    const double v = i < 5 ? trunc(x * (1.0 / weight)) : rint(x * (1.0 / weight));
    add_digit(&s->digit[i], __double2ll_rn(v));
    x -= v * weight;  // exact: a multiple of x's last bit, and no longer than x
  }
}

// The digits with carries taken upwards and one sign: magnitude in d, returns
// whether the sum is negative.
__device__ __forceinline__ bool carry(long long (&d)[6]) {
  bool negative = false;
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
#pragma unroll
    for (int i = 5; i > 0; --i) {
      d[i - 1] += d[i] >> 40;
      d[i] &= kMask;
    }
    if (pass || d[0] >= 0) break;
    negative = true;
#pragma unroll
    for (int i = 0; i < 6; ++i) d[i] = -d[i];
  }
  return negative;
}

__device__ __noinline__ double large_value(const long long (&digit)[6], unsigned int flags) {
  if (flags) return flags == 2u ? __longlong_as_double(0x7FF0000000000000ll)
                  : flags == 4u ? __longlong_as_double(0xFFF0000000000000ll)
                                : __longlong_as_double(0x7FF8000000000000ll);
  long long d[6];
#pragma unroll
  for (int i = 0; i < 6; ++i) d[i] = digit[i];
  const bool negative = carry(d);
  double v = 0.0, weight = 1.0 / (kUp * kUp);
#pragma unroll
  for (int i = 5; i >= 0; --i, weight *= kUp) v += static_cast<double>(d[i]) * weight;
  return negative ? -v : v;
}

// The digits as they are, so that those of several sums can be on their way at
// once.
struct Digits {
  long long d[6];
};

__device__ __forceinline__ Digits digits(const Sum* s) {
  Digits v;
#pragma unroll
  for (int i = 0; i < 6; ++i) v.d[i] = __ldcg(&s->digit[i]);
  return v;
}

// A sum's value: a pair, and in 64 bits in *far or times kSmall in *small
// wherever its magnitude is kNear and more (also for others, which nothing
// reads).
constexpr float kNear = 1e6f;
constexpr float kSmall = 1.0f / 4294967296.0f;

__device__ __forceinline__ Pair split_of(double v) {
  const float hi = static_cast<float>(v);
  return {hi, finite(hi) ? static_cast<float>(v - hi) : 0.0f};
}

__device__ __forceinline__ Pair value(const Digits& s, unsigned int flags, int shift, double* far = nullptr,
                                      Pair* small = nullptr) {
  flags = (flags >> shift) & 7u;
  const long long(&d)[6] = s.d;
  const long long next = d[4] + (d[5] >> 40), top = d[3] + (next >> 40);
  const long long last = d[5] & kMask;  // units of 2^-80
  const long long whole = static_cast<long long>(static_cast<unsigned long long>(top) << 40) + (next & kMask);  // 2^-40
  // below 2^-19 what is left of units of 2^-40 counts, and not to 24 bits
  const bool fast = !(whole < (1ll << 21) && whole >= -(1ll << 21)) || (whole | last) == 0;
  if (!(flags | d[0] | d[1] | d[2]) && top < (1ll << 19) && top >= -(1ll << 19) && fast) {
    const float rest = __ll2float_rn(last) * (1.0f / kFine);
    const float hi = __ll2float_rn(whole);
    const Pair u = renormal(hi, __ll2float_rn(whole - __float2ll_rn(hi)) + rest);
    return {u.hi * (1.0f / kFine), u.lo * (1.0f / kFine)};
  }
  const double v = large_value(d, flags);
  if (far) *far = v;
  if (small) *small = split_of(v * kSmall);
  return split_of(v);
}

// What is summed of an episode: two values, valid tokens, clipped tokens.
struct Episode {
  Sum a, b;
  unsigned int n, cut, flags, unused;
};
static_assert(sizeof(Episode) == 112, "workspace layout");

// A thread's, warp's or block's part of it: sums in units of 2^-40, what is left
// of their terms in units of 2^-80.
struct Part {
  long long a, b, fine_a, fine_b;
  unsigned int n, cut;
};

__device__ __forceinline__ void add_part(Episode* e, const Part& p) {
  add_units(&e->a, p.a);
  add_units(&e->b, p.b);
  add_digit(&e->a.digit[5], p.fine_a);
  add_digit(&e->b.digit[5], p.fine_b);
  if (p.n) atomicAdd(&e->n, p.n);
  if (p.cut) atomicAdd(&e->cut, p.cut);
}

__device__ __forceinline__ Part operator+(const Part& x, const Part& y) {
  return {x.a + y.a, x.b + y.b, x.fine_a + y.fine_a, x.fine_b + y.fine_b, x.n + y.n, x.cut + y.cut};
}

// The sum of v over the lanes of `mask`, which all call this: in pieces of 22
// bits, whose sums fit in 32.
__device__ __forceinline__ long long group_sum(unsigned mask, long long v) {
  constexpr unsigned kPiece = (1u << 22) - 1;
  const unsigned lo = __reduce_add_sync(mask, static_cast<unsigned>(v) & kPiece);
  const unsigned mid = __reduce_add_sync(mask, static_cast<unsigned>(v >> 22) & kPiece);
  const int hi = __reduce_add_sync(mask, static_cast<int>(v >> 44));
  return (static_cast<long long>(hi) << 44) + (static_cast<long long>(mid) << 22) + lo;
}

// The same where it is seldom needed: out of the way of the code that always runs.
__device__ __noinline__ long long rare_sum(unsigned mask, long long v) { return group_sum(mask, v); }

__device__ __forceinline__ Part warp_sum(Part p, bool two) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) p.a += __shfl_xor_sync(kAll, p.a, o);
  if (two) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) p.b += __shfl_xor_sync(kAll, p.b, o);
  }
  if (__any_sync(kAll, (p.fine_a | p.fine_b) != 0)) {
    p.fine_a = rare_sum(kAll, p.fine_a);
    p.fine_b = rare_sum(kAll, p.fine_b);
  }
  p.n = __reduce_add_sync(kAll, p.n);
  p.cut = __reduce_add_sync(kAll, p.cut);
  return p;
}

// Sums over the block in a fixed order; every thread gets them.
__device__ Pair block_sum(Pair v) {
  __shared__ Pair part[kWarps];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = add(v, Pair{__shfl_xor_sync(kAll, v.hi, o), __shfl_xor_sync(kAll, v.lo, o)});
  __syncthreads();
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
  __syncthreads();
  v = part[threadIdx.x % kWarps];
#pragma unroll
  for (int o = kWarps / 2; o > 0; o >>= 1)
    v = add(v, Pair{__shfl_xor_sync(kAll, v.hi, o), __shfl_xor_sync(kAll, v.lo, o)});
  return v;
}

__device__ unsigned int block_count(unsigned int n) {
  __shared__ unsigned int part[kWarps];
  n = __reduce_add_sync(kAll, n);
  __syncthreads();
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = n;
  __syncthreads();
  return __reduce_add_sync(kAll, threadIdx.x % 32 < kWarps ? part[threadIdx.x % 32] : 0u);
}

// A sum of losses.  What is kNear and more is added times kSmall, where no sum
// of fp32 values overflows before it is divided by their number.
struct Total {
  Pair near, far;
  bool any;  // whether there is a far part

  // small(): v kSmall, which few calls need
  template <typename Small>
  __device__ __forceinline__ void put(Pair v, Small small) {
    if (fabsf(v.hi) < kNear) {
      near = add(near, v);
    } else {
      far = add(far, small());
      any = true;
    }
  }
};

// Counts with a flag: which warps have a far part.
constexpr unsigned int kFarFlag = 1u << 24;

__device__ __forceinline__ unsigned int far_flag(bool any) {
  return __any_sync(kAll, any) && threadIdx.x % 32 == 0 ? kFarFlag : 0u;
}

// The mean of n values whose sum the block's threads hold; every thread gets it.
__device__ __forceinline__ Pair mean_of(const Total& t, float n, bool any) {
  Pair mean = over(block_sum(t.near), n);
  if (any) {
    const Pair far = over(block_sum(t.far), n);
    mean = add(mean, Pair{far.hi * (1.0f / kSmall), far.lo * (1.0f / kSmall)});
  }
  return mean;
}

// ------------------------------------------------------------- parameters
struct LossParams {
  const float* logp;
  const float* old;
  const float* ref;
  const float* adv;
  const int32_t* seq_id;
  long long N;
  int E;
  // policy
  bool by_token, adv_by_token, ratio_episode, mean_episode;
  float bound_low, bound_high;  // 1 - low, 1 + high
  Pair log_low, log_high;       // their logarithms
  float kl_weight;
  // preference
  const int32_t* pairs;
  int P, kind;
  bool mean;
  float beta, smoothing;
  double beta_d, margin_d;
  Pair margin, target;  // target: 1 / (2 beta)
  float* rewards;
  // results
  float* loss;
  float* stats;
  float* coef;
  const float* dloss;
  float* dlogp;
  // workspace
  unsigned int* done;
  Episode* episodes;
  Sum* factors;  // preference: sums of the pairs' derivatives, one an episode
  unsigned int* factor_flags;
  Pair* sums;    // D_e
  double* far;   // D_e in 64 bits where it is kNear and more
  DeviceError* err;
};

__device__ __forceinline__ void report(DeviceError* err, uint32_t where) {
  if (atomicCAS(&err->code, 0u, kDevErrEpisode) == 0u) {
    err->where = where;
    err->block = blockIdx.x;
    err->thread = threadIdx.x;
  }
}

// Four tokens from `first` on; those at or past N get `other`.
template <typename T>
__device__ __forceinline__ void load4(const T* p, long long first, long long N, T other, T (&v)[4]) {
  if (first + 4 <= N && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
    const uint4 q = __ldg(reinterpret_cast<const uint4*>(p + first));
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const T*>(&w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = first + i < N ? p[first + i] : other;
  }
}

// exp f - f - 1 without cancellation: its series up to 0.5 (the next term is
// below 2^-24 of the sum), else the formula.
__device__ __forceinline__ float kl_term(float f) {
  if (fabsf(f) < 0.5f) {
    float s = 1.0f / 362880.0f;
    s = fmaf(s, f, 1.0f / 40320.0f);
    s = fmaf(s, f, 1.0f / 5040.0f);
    s = fmaf(s, f, 1.0f / 720.0f);
    s = fmaf(s, f, 1.0f / 120.0f);
    s = fmaf(s, f, 1.0f / 24.0f);
    s = fmaf(s, f, 1.0f / 6.0f);
    s = fmaf(s, f, 0.5f);
    return s * f * f;
  }
  // far above, f + 1 is nothing beside exp f, and infinity less infinity is not taken
  return f > 64.0f ? expf(f) : expf(f) - 1.0f - f;
}

// a > b, for pairs: the lower parts decide where the upper are equal.
__device__ __forceinline__ bool above(Pair a, Pair b) { return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo); }

// Whether the clipped ratio is the one that counts.
__device__ __forceinline__ bool clipped(const LossParams& p, Pair d, float adv) {
  return adv > 0.0f ? above(d, p.log_high) : adv < 0.0f && above(p.log_low, d);
}

// -min(r A, clip(r) A).  An advantage of 0 gives 0 whatever the ratio.
__device__ __forceinline__ float policy_term(const LossParams& p, float d, float adv, bool cut) {
  if (adv == 0.0f) return 0.0f;
  return -(cut ? (adv > 0.0f ? p.bound_high : p.bound_low) : expf(d)) * adv;
}

// ------------------------------------------------------------- forward
// A value that units of 2^-40 hold, else 0: it went to the episode at once.
__device__ __forceinline__ Pair ordinary(Pair v, Sum* s, unsigned int* flags, int shift) {
  if (fabsf(v.hi) < 2048.0f) return v;
  add_any(s, flags, shift, static_cast<double>(v.hi) + static_cast<double>(v.lo));
  return {0.0f, 0.0f};
}

__device__ __forceinline__ long long units(Pair v) {
  return __float2ll_rn(v.hi * kFine) + __float2ll_rn(v.lo * kFine);
}

// Whether units of 2^-40 leave anything of hi.
__device__ __forceinline__ bool leaves(float hi) { return hi != 0.0f && fabsf(hi) < 0x1p-16f; }

// Whether the b of a part's terms are 2^-17 on average.
__device__ __forceinline__ bool enough(const Part& p) { return p.b >= static_cast<long long>(p.n) << 23; }

// What they leave, in units of 2^-80.
__device__ __noinline__ long long rest_units(Pair v) {
  const float x = v.hi * kFine, y = v.lo * kFine;
  return __float2ll_rn((x - rintf(x)) * kFine) + __float2ll_rn((y - rintf(y)) * kFine);
}

// Sums of this block's tokens into the episodes'.
template <bool kPolicy>
__device__ void sum_tokens(const LossParams& p) {
  __shared__ int warp_lo[kWarps], warp_hi[kWarps];
  __shared__ Part warp_part[kWarps];
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
  const long long first = static_cast<long long>(blockIdx.x) * kTokens + threadIdx.x * 4;
  int id[4];
  float logp[4], old[4], ref[4], adv[4];
  load4(p.seq_id, first, p.N, -1, id);
  load4(p.logp, first, p.N, 0.0f, logp);
  if (p.ref) load4(p.ref, first, p.N, 0.0f, ref);
  if (kPolicy && p.old) load4(p.old, first, p.N, 0.0f, old);
  if (kPolicy && p.adv_by_token) load4(p.adv, first, p.N, 0.0f, adv);
  const bool two = kPolicy && p.ref;
  Part t[4];
  Pair va[4], vb[4];
  bool small_a = false, small_b = false, large_a = false;
  int lo = INT32_MAX, hi = -1;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    t[i] = Part{};
    va[i] = vb[i] = Pair{0.0f, 0.0f};
    if (id[i] >= p.E) {
      report(p.err, kSiteEpisode);
      id[i] = -1;
    }
    if (id[i] < 0) continue;
    t[i].n = 1;
    Pair a, b{0.0f, 0.0f};
    int to = id[i];
    if constexpr (kPolicy) {
      a = p.old ? two_sum(logp[i], -old[i]) : Pair{0.0f, 0.0f};
      if (p.ref) b = Pair{kl_term(__fsub_rn(ref[i], logp[i])), 0.0f};
      if (!p.ratio_episode) {
        const float v = p.adv_by_token ? adv[i] : __ldg(p.adv + id[i]);
        const bool cut = clipped(p, a, v);
        a = Pair{policy_term(p, a.hi, v, cut), 0.0f};
        t[i].cut = cut;
      }
      if (p.by_token) to = 0;  // one sum over all tokens
      id[i] = to;
    } else {
      a = p.ref ? two_sum(logp[i], -ref[i]) : Pair{logp[i], 0.0f};
    }
    Episode* e = p.episodes + to;
    va[i] = ordinary(a, &e->a, &e->flags, 0);
    t[i].a = units(va[i]);
    if (two) {
      vb[i] = ordinary(b, &e->b, &e->flags, 3);
      t[i].b = units(vb[i]);
    }
    small_a = small_a || leaves(va[i].hi);
    small_b = small_b || leaves(vb[i].hi);
    large_a = large_a || !(fabsf(a.hi) < 0x1p-10f);
    lo = min(lo, to);
    hi = max(hi, to);
  }
  lo = __reduce_min_sync(kAll, lo);
  hi = __reduce_max_sync(kAll, hi);
  if (lane == 0) {
    warp_lo[w] = lo;
    warp_hi[w] = hi;
  }
  const Part own = t[0] + t[1] + t[2] + t[3];
  Part sum = warp_sum(own, two);
  // What units of 2^-40 leave, where it may count: beside a term of 2^-10, or terms of 2^-17 on average that are none
  // negative, the 4 or 128 tokens of a thread's or warp's sum lose less than 2^-24 of them.
  const bool one = lo == hi, alike = id[0] == id[1] && id[1] == id[2] && id[2] == id[3];
  const bool any_large = __any_sync(kAll, large_a);
  const bool more_a = small_a && !(alike && large_a) && !(one && any_large);
  const bool more_b = small_b && !(alike && enough(own)) && !(one && enough(sum));
  if (__any_sync(kAll, more_a)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i].fine_a = rest_units(va[i]);
    sum.fine_a = rare_sum(kAll, t[0].fine_a + t[1].fine_a + t[2].fine_a + t[3].fine_a);
  }
  if (__any_sync(kAll, more_b)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i].fine_b = rest_units(vb[i]);
    sum.fine_b = rare_sum(kAll, t[0].fine_b + t[1].fine_b + t[2].fine_b + t[3].fine_b);
  }
  if (lane == 0) warp_part[w] = sum;
  __syncthreads();
  const int block_lo = __reduce_min_sync(kAll, warp_lo[lane % kWarps]);
  const int block_hi = __reduce_max_sync(kAll, warp_hi[lane % kWarps]);
  if (block_hi < 0) return;
  if (block_lo == block_hi) {
    if (w == 0) {
      sum = lane < kWarps ? warp_part[lane] : Part{};
      sum = warp_sum(sum, two);
      if (lane == 0) add_part(p.episodes + block_lo, sum);
    }
  } else if (lo == hi) {
    if (lane == 0) add_part(p.episodes + lo, sum);
  } else if (alike) {
    // lanes of one episode each: those of the same one add together
    const unsigned mask = __match_any_sync(__activemask(), id[0]);
    if (id[0] < 0) return;
    sum = t[0] + t[1] + t[2] + t[3];
    sum.a = group_sum(mask, sum.a);
    if (two) sum.b = group_sum(mask, sum.b);
    if (__any_sync(mask, (sum.fine_a | sum.fine_b) != 0)) {
      sum.fine_a = rare_sum(mask, sum.fine_a);
      sum.fine_b = rare_sum(mask, sum.fine_b);
    }
    sum.n = __reduce_add_sync(mask, sum.n);
    sum.cut = __reduce_add_sync(mask, sum.cut);
    if (lane == __ffs(mask) - 1) add_part(p.episodes + id[0], sum);
  } else {
    Part run = t[0];
    int at = id[0];
#pragma unroll
    for (int i = 1; i < 4; ++i) {
      if (id[i] != at) {
        if (at >= 0) add_part(p.episodes + at, run);
        run = t[i];
        at = id[i];
      } else {
        run = run + t[i];
      }
    }
    if (at >= 0) add_part(p.episodes + at, run);
  }
}

// D_e in 64 bits.
__device__ __forceinline__ double wide(const LossParams& p, int e, Pair v) {
  return fabsf(v.hi) < kNear ? static_cast<double>(v.hi) + static_cast<double>(v.lo) : p.far[e];
}

// Whether this block is the last of the grid to get here; it then sees what
// all others wrote.
__device__ bool last_block(const LossParams& p) {
  __shared__ bool last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(p.done, 1u) == gridDim.x - 1;
    __threadfence();
  }
  __syncthreads();
  return last;
}

__global__ void __launch_bounds__(kThreads) preference_kernel(const LossParams p) {
  sum_tokens<false>(p);
  if (!last_block(p)) return;
  // two episodes a thread and turn, whose digits are on their way together
  for (int first = threadIdx.x; first < p.E; first += 2 * kThreads) {
    Digits s[2];
    unsigned int n[2], flags[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const Episode* q = p.episodes + min(first + i * kThreads, p.E - 1);
      s[i] = digits(&q->a);
      n[i] = __ldcg(&q->n);
      flags[i] = __ldcg(&q->flags);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = first + i * kThreads;
      if (e >= p.E) continue;
      Pair v = value(s[i], flags[i], 0, p.far + e);
      if (p.mean && n[i]) {
        if (!(fabsf(v.hi) < kNear)) p.far[e] /= n[i];
        v = over(v, static_cast<float>(n[i]));
      }
      p.sums[e] = v;
    }
  }
  __syncthreads();
  Total loss{};
  unsigned int count = 0;
  for (int i = threadIdx.x; i < p.P; i += kThreads) {
    const int c = p.pairs[2 * i], r = p.pairs[2 * i + 1];
    if (c >= p.E || r >= p.E) report(p.err, kSitePair);
    if (c < 0 || r < 0 || c >= p.E || r >= p.E) {
      p.rewards[2 * i] = p.rewards[2 * i + 1] = 0.0f;
      continue;
    }
    ++count;
    const Pair vc = p.sums[c], vr = p.sums[r];
    Pair h;   // D_c - D_r - margin, to 2^-46 of its terms
    float x;  // beta h
    float rc = p.beta * vc.hi, rr = p.beta * vr.hi;
    bool short_of;  // beta h < 1
    if (fabsf(vc.hi) < kNear && fabsf(vr.hi) < kNear) {
      h = add(add(vc, Pair{-vr.hi, -vr.lo}), Pair{-p.margin.hi, -p.margin.lo});
      x = p.beta * h.hi;
      short_of = above(Pair{2.0f * p.target.hi, 2.0f * p.target.lo}, h);
    } else {
      const double dc = wide(p, c, vc), dr = wide(p, r, vr), d = dc - dr - p.margin_d;
      h = split_of(d);
      x = static_cast<float>(p.beta_d * d);
      short_of = p.beta_d * d < 1.0;
      rc = static_cast<float>(p.beta_d * dc);
      rr = static_cast<float>(p.beta_d * dr);
    }
    p.rewards[2 * i] = rc;
    p.rewards[2 * i + 1] = rr;
    float l, up;  // up: the derivative to h, over beta but for the squared loss
    if (p.kind == PVL_PREFERENCE_SIGMOID) {
      const float e = expf(-fabsf(x)), soft = log1pf(e);
      const float s = p.smoothing;
      l = (1.0f - s) * (soft + fmaxf(-x, 0.0f));
      if (s > 0.0f) l = fmaf(s, soft + fmaxf(x, 0.0f), l);  // not 0 times infinity
      const float other = x >= 0.0f ? e / (1.0f + e) : 1.0f / (1.0f + e);  // sigmoid(-x)
      up = s - other;
    } else if (p.kind == PVL_PREFERENCE_SQUARED) {
      const Pair miss = add(h, Pair{-p.target.hi, -p.target.lo});
      l = miss.hi * miss.hi;
      up = 2.0f * miss.hi;
    } else {
      l = short_of ? 1.0f - x : 0.0f;
      up = short_of ? -1.0f : 0.0f;
    }
    if (x != x) l = up = x;
    loss.put(Pair{l, 0.0f}, [&] { return Pair{l * kSmall, 0.0f}; });
    if (c != r) {  // an episode against itself has no gradient
      if (fabsf(up) < 2048.0f) {
        const float fine = up * kFine;
        const long long v = __float2ll_rn(fine), rest = __float2ll_rn((fine - __ll2float_rn(v)) * kFine);
        add_units(p.factors + c, v);
        add_units(p.factors + r, -v);
        add_digit(&p.factors[c].digit[5], rest);
        add_digit(&p.factors[r].digit[5], -rest);
      } else {
        add_any(p.factors + c, p.factor_flags + c, 0, up);
        add_any(p.factors + r, p.factor_flags + r, 0, -up);
      }
    }
  }
  count = block_count(count + far_flag(loss.any));
  const bool any = count >= kFarFlag;
  count %= kFarFlag;
  const float share = count ? static_cast<float>(count) : 1.0f;
  const Pair mean = mean_of(loss, share, any);
  if (threadIdx.x == 0) p.loss[0] = mean.hi;
  __threadfence();
  __syncthreads();
  const float slope = p.kind == PVL_PREFERENCE_SQUARED ? 1.0f : p.beta;
  for (int e = threadIdx.x; e < p.E; e += kThreads) {
    const unsigned int n = __ldcg(&p.episodes[e].n);
    const float f = slope * over(value(digits(p.factors + e), __ldcg(p.factor_flags + e), 0), share).hi;
    p.coef[e] = p.mean && n ? f / static_cast<float>(n) : f;
  }
}

__global__ void __launch_bounds__(kThreads) policy_kernel(const LossParams p) {
  sum_tokens<true>(p);
  if (!last_block(p)) return;
  const int E = p.by_token ? 1 : p.E;
  unsigned int tokens = 0, some = 0;
  for (int e = threadIdx.x; e < E; e += kThreads) {
    const unsigned int n = __ldcg(&p.episodes[e].n);
    tokens += n;
    some += n ? 1u : 0u;
  }
  tokens = block_count(tokens);
  some = block_count(some);
  // what sums are divided by at the end
  const float whole = static_cast<float>(max(1u, p.mean_episode ? some : tokens));
  Total losses{}, divergences{};
  unsigned int cut = 0;
  for (int e = threadIdx.x; e < E; e += kThreads) {
    const Episode* q = p.episodes + e;
    const unsigned int n = __ldcg(&q->n), flags = __ldcg(&q->flags);
    float slope = 0.0f, weight = 0.0f;
    if (n) {
      const float fn = static_cast<float>(n);
      Pair small{0.0f, 0.0f};
      const Pair a = value(digits(&q->a), flags, 0, nullptr, &small);
      weight = p.mean_episode ? 1.0f / (whole * fn) : 1.0f / whole;
      if (p.ratio_episode) {
        const Pair d = over(a, fn);
        const float adv = p.adv[e];
        const bool clip = clipped(p, d, adv);
        const float term = policy_term(p, d.hi, adv, clip);
        losses.put(p.mean_episode ? Pair{term, 0.0f} : times(term, fn),
                   [&] { return p.mean_episode ? Pair{term * kSmall, 0.0f} : times(term * kSmall, fn); });
        slope = clip ? 0.0f : weight * term;
        cut += clip;
      } else {
        losses.put(p.mean_episode ? over(a, fn) : a, [&] { return p.mean_episode ? over(small, fn) : small; });
        cut += __ldcg(&q->cut);
      }
      if (p.ref) {
        const Pair b = value(digits(&q->b), flags, 3, nullptr, &small);
        divergences.put(p.mean_episode ? over(b, fn) : b, [&] { return p.mean_episode ? over(small, fn) : small; });
      }
    }
    if (!p.by_token) *reinterpret_cast<float2*>(p.coef + 2 * e) = make_float2(slope, weight);
  }
  cut = block_count(cut + far_flag(losses.any || divergences.any));
  const bool any = cut >= kFarFlag;
  cut %= kFarFlag;
  Pair loss = mean_of(losses, whole, any);
  const Pair kl = mean_of(divergences, whole, any);
  if (threadIdx.x == 0) {
    // 0 times an infinite divergence is no part of the loss
    if (p.kl_weight != 0.0f) {
      Pair k = times(p.kl_weight, kl.hi);
      k.lo = finite(k.hi) ? fmaf(p.kl_weight, kl.lo, k.lo) : 0.0f;
      loss = add(loss, k);
    }
    p.loss[0] = loss.hi;
    p.stats[0] = kl.hi;
    p.stats[1] = static_cast<float>(cut) / static_cast<float>(max(1u, p.ratio_episode ? some : tokens));
  }
  if (p.by_token)
    for (int e = threadIdx.x; e < p.E; e += kThreads)
      *reinterpret_cast<float2*>(p.coef + 2 * e) = make_float2(0.0f, tokens ? 1.0f / whole : 0.0f);
}

// ------------------------------------------------------------- backward
template <bool kPolicy>
__global__ void __launch_bounds__(kBwdThreads) token_grad_kernel(const LossParams p) {
  const long long first = (static_cast<long long>(blockIdx.x) * kBwdThreads + threadIdx.x) * 4;
  if (first >= p.N) return;
  int id[4];
  float logp[4], old[4], ref[4], adv[4], g[4];
  load4(p.seq_id, first, p.N, -1, id);
  const bool kl = kPolicy && p.ref && p.kl_weight != 0.0f;
  if constexpr (kPolicy) {
    load4(p.logp, first, p.N, 0.0f, logp);
    if (p.old && !p.ratio_episode) load4(p.old, first, p.N, 0.0f, old);
    if (kl) load4(p.ref, first, p.N, 0.0f, ref);
    if (p.adv_by_token) load4(p.adv, first, p.N, 0.0f, adv);
  }
  const float up = p.dloss ? __ldg(p.dloss) : 1.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    g[i] = 0.0f;
    if (id[i] < 0 || id[i] >= p.E) continue;
    if constexpr (kPolicy) {
      const float2 c = __ldg(reinterpret_cast<const float2*>(p.coef) + id[i]);
      float slope = c.x;
      if (!p.ratio_episode) {
        const Pair d = p.old ? two_sum(logp[i], -old[i]) : Pair{0.0f, 0.0f};
        const float a = p.adv_by_token ? adv[i] : __ldg(p.adv + id[i]);
        const bool cut = clipped(p, d, a);
        slope = cut ? 0.0f : c.y * policy_term(p, d.hi, a, false);
      }
      if (kl) slope = fmaf(-c.y * p.kl_weight, expm1f(__fsub_rn(ref[i], logp[i])), slope);
      g[i] = up * slope;
    } else {
      g[i] = up * __ldg(p.coef + id[i]);
    }
  }
  if (first + 4 <= p.N && reinterpret_cast<uintptr_t>(p.dlogp) % 16 == 0) {
    *reinterpret_cast<float4*>(p.dlogp + first) = make_float4(g[0], g[1], g[2], g[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (first + i < p.N) p.dlogp[first + i] = g[i];
  }
}

// ------------------------------------------------------------------ host
// Workspace: counter (cleared), episodes (cleared), factors and their flags
// (cleared, preference), D_e (preference).
struct Layout {
  size_t episodes, factors, flags, clear, sums, far, total;
};

Layout layout(int E, bool preference) {
  Layout l{};
  l.episodes = 256;
  l.factors = l.episodes + align256(static_cast<size_t>(E) * sizeof(Episode));
  l.flags = l.factors + (preference ? align256(static_cast<size_t>(E) * sizeof(Sum)) : 0);
  l.clear = l.flags + (preference ? align256(static_cast<size_t>(E) * 4) : 0);
  l.sums = l.clear;
  l.far = l.sums + (preference ? align256(static_cast<size_t>(E) * sizeof(Pair)) : 0);
  l.total = l.far + (preference ? align256(static_cast<size_t>(E) * 8) : 0);
  return l;
}

bool misaligned(std::initializer_list<const void*> ptrs, uintptr_t to) {
  for (const void* q : ptrs)
    if (reinterpret_cast<uintptr_t>(q) % to) return true;
  return false;
}

Pair split(double v) {
  const float hi = static_cast<float>(v);
  return {hi, static_cast<float>(v - hi)};
}

pvl_status sizes(const char* who, int64_t N, int E) {
  if (N < 1 || E < 1) return fail(PVL_ERR_INVALID_ARG, "%s: tokens and episodes must be >= 1", who);
  if (N > kMaxTokens || E > kMaxEpisodes)
    return fail(PVL_ERR_UNSUPPORTED, "%s: %lld tokens of %d episodes (at most %lld, %d)", who, static_cast<long long>(N),
                E, kMaxTokens, kMaxEpisodes);
  return PVL_OK;
}

// The workspace into p, its counters and sums cleared on the stream.
pvl_status workspace(const char* who, LossParams& p, void* ws, size_t ws_bytes, bool preference, cudaStream_t s) {
  const Layout l = layout(p.E, preference);
  if (!ws) return fail(PVL_ERR_INVALID_ARG, "%s: null workspace", who);
  if (ws_bytes < l.total) return fail(PVL_ERR_INVALID_ARG, "%s: workspace %zu bytes < %zu needed", who, ws_bytes, l.total);
  if (misaligned({ws}, 16)) return fail(PVL_ERR_UNSUPPORTED, "%s: the workspace is not 16-byte aligned", who);
  p.err = device_error_record();
  if (!p.err) return fail(PVL_ERR_CUDA, "%s: no usable CUDA device", who);
  uint8_t* b = static_cast<uint8_t*>(ws);
  p.done = reinterpret_cast<unsigned int*>(b);
  p.episodes = reinterpret_cast<Episode*>(b + l.episodes);
  p.factors = reinterpret_cast<Sum*>(b + l.factors);
  p.factor_flags = reinterpret_cast<unsigned int*>(b + l.flags);
  p.sums = reinterpret_cast<Pair*>(b + l.sums);
  p.far = reinterpret_cast<double*>(b + l.far);
  return check_cuda(cudaMemsetAsync(ws, 0, l.clear, s), who);
}

pvl_status policy_params(const char* who, const pvl_policy* h, LossParams* p) {
  if (!h || !h->logp || !h->advantages || !h->seq_id) return fail(PVL_ERR_INVALID_ARG, "%s: null pointer", who);
  const pvl_status st = sizes(who, h->tokens, h->episodes);
  if (st != PVL_OK) return st;
  if ((h->ratio | h->mean | h->token_advantages) & ~1)
    return fail(PVL_ERR_INVALID_ARG, "%s: ratio, mean and token_advantages are 0 or 1", who);
  if (h->ratio == 1 && h->token_advantages)
    return fail(PVL_ERR_INVALID_ARG, "%s: ratios of episodes need advantages of episodes", who);
  if (!(h->clip_low >= 0.0 && h->clip_low < 1.0) || !(h->clip_high >= 0.0 && h->clip_high < 1e30))
    return fail(PVL_ERR_INVALID_ARG, "%s: needs 0 <= clip_low < 1 and 0 <= clip_high", who);
  if (!(h->kl_weight >= 0.0f) || !(h->kl_weight < 1e30f) || (h->kl_weight > 0.0f && !h->ref_logp))
    return fail(PVL_ERR_INVALID_ARG, "%s: kl_weight must be finite, not negative, and needs ref_logp above 0", who);
  if (misaligned({h->logp, h->old_logp, h->ref_logp, h->advantages, h->seq_id}, 4))
    return fail(PVL_ERR_UNSUPPORTED, "%s: a pointer is not aligned to its elements", who);
  p->logp = h->logp;
  p->old = h->old_logp;
  p->ref = h->ref_logp;
  p->adv = h->advantages;
  p->seq_id = h->seq_id;
  p->N = h->tokens;
  p->E = h->episodes;
  p->ratio_episode = h->ratio == 1;
  p->mean_episode = h->mean == 1;
  p->by_token = !p->ratio_episode && !p->mean_episode;
  p->adv_by_token = h->token_advantages != 0;
  p->bound_low = static_cast<float>(1.0 - h->clip_low);
  p->bound_high = static_cast<float>(1.0 + h->clip_high);
  p->log_low = split(std::log1p(-h->clip_low));
  p->log_high = split(std::log1p(h->clip_high));
  p->kl_weight = h->kl_weight;
  return PVL_OK;
}

unsigned blocks_of(long long n, int per) { return static_cast<unsigned>((n + per - 1) / per); }

}  // namespace
}  // namespace pvl

using namespace pvl;

extern "C" size_t pack_preference_ws_bytes(int episodes) {
  return episodes < 1 || episodes > kMaxEpisodes ? 0 : layout(episodes, true).total;
}

extern "C" size_t pack_policy_ws_bytes(int episodes) {
  return episodes < 1 || episodes > kMaxEpisodes ? 0 : layout(episodes, false).total;
}

extern "C" pvl_status pack_preference_fwd(const pvl_preference* h, float* loss, float* rewards, float* coef, void* ws,
                                          size_t ws_bytes, pvl_stream_t stream) {
  const char* who = "pack_preference_fwd";
  if (!h || !h->logp || !h->seq_id || !h->pairs || !loss || !rewards || !coef)
    return fail(PVL_ERR_INVALID_ARG, "%s: null pointer", who);
  pvl_status st = sizes(who, h->tokens, h->episodes);
  if (st != PVL_OK) return st;
  if (h->n_pairs < 1) return fail(PVL_ERR_INVALID_ARG, "%s: needs a pair", who);
  if (h->n_pairs > kMaxPairs) return fail(PVL_ERR_UNSUPPORTED, "%s: %d pairs (at most %d)", who, h->n_pairs, kMaxPairs);
  if (h->kind < 0 || h->kind > 2) return fail(PVL_ERR_INVALID_ARG, "%s: kind %d (0 to 2)", who, h->kind);
  if (h->mean & ~1) return fail(PVL_ERR_INVALID_ARG, "%s: mean is 0 or 1", who);
  if (!(h->beta > 1e-30) || !(h->beta < 1e30) || !(std::fabs(h->margin) < 1e30))
    return fail(PVL_ERR_INVALID_ARG, "%s: beta must be positive, beta and margin finite", who);
  if (!(h->smoothing >= 0.0 && h->smoothing <= 0.5) || (h->smoothing > 0.0 && h->kind != PVL_PREFERENCE_SIGMOID))
    return fail(PVL_ERR_INVALID_ARG, "%s: smoothing lies in [0, 0.5] and belongs to the sigmoid loss", who);
  if (misaligned({h->logp, h->ref_logp, h->seq_id, h->pairs, loss, rewards, coef}, 4))
    return fail(PVL_ERR_UNSUPPORTED, "%s: a pointer is not aligned to its elements", who);
  LossParams p{};
  p.logp = h->logp;
  p.ref = h->ref_logp;
  p.seq_id = h->seq_id;
  p.N = h->tokens;
  p.E = h->episodes;
  p.pairs = h->pairs;
  p.P = h->n_pairs;
  p.kind = h->kind;
  p.mean = h->mean != 0;
  p.beta = static_cast<float>(h->beta);
  p.beta_d = h->beta;
  p.smoothing = static_cast<float>(h->smoothing);
  p.margin = split(h->margin);
  p.margin_d = h->margin;
  p.target = split(0.5 / h->beta);
  p.loss = loss;
  p.rewards = rewards;
  p.coef = coef;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  st = workspace(who, p, ws, ws_bytes, true, s);
  if (st != PVL_OK) return st;
  preference_kernel<<<blocks_of(p.N, kTokens), kThreads, 0, s>>>(p);
  return check_cuda(cudaGetLastError(), "pack_preference_fwd launch");
}

extern "C" pvl_status pack_preference_bwd(const float* dloss, const float* coef, const int32_t* seq_id, int64_t tokens,
                                          int episodes, float* dlogp, pvl_stream_t stream) {
  const char* who = "pack_preference_bwd";
  if (!coef || !seq_id || !dlogp) return fail(PVL_ERR_INVALID_ARG, "%s: null pointer", who);
  const pvl_status st = sizes(who, tokens, episodes);
  if (st != PVL_OK) return st;
  if (misaligned({dloss, coef, seq_id, dlogp}, 4))
    return fail(PVL_ERR_UNSUPPORTED, "%s: a pointer is not aligned to its elements", who);
  LossParams p{};
  p.dloss = dloss;
  p.coef = const_cast<float*>(coef);
  p.seq_id = seq_id;
  p.N = tokens;
  p.E = episodes;
  p.dlogp = dlogp;
  token_grad_kernel<false><<<blocks_of(p.N, 4 * kBwdThreads), kBwdThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return check_cuda(cudaGetLastError(), "pack_preference_bwd launch");
}

extern "C" pvl_status pack_policy_fwd(const pvl_policy* h, float* loss, float* stats, float* coef, void* ws,
                                      size_t ws_bytes, pvl_stream_t stream) {
  const char* who = "pack_policy_fwd";
  LossParams p{};
  pvl_status st = policy_params(who, h, &p);
  if (st != PVL_OK) return st;
  if (!loss || !stats || !coef) return fail(PVL_ERR_INVALID_ARG, "%s: null pointer", who);
  if (misaligned({loss, stats}, 4) || misaligned({coef}, 8))
    return fail(PVL_ERR_UNSUPPORTED, "%s: loss and stats must be 4-byte and coef 8-byte aligned", who);
  p.loss = loss;
  p.stats = stats;
  p.coef = coef;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  st = workspace(who, p, ws, ws_bytes, false, s);
  if (st != PVL_OK) return st;
  policy_kernel<<<blocks_of(p.N, kTokens), kThreads, 0, s>>>(p);
  return check_cuda(cudaGetLastError(), "pack_policy_fwd launch");
}

extern "C" pvl_status pack_policy_bwd(const pvl_policy* h, const float* dloss, const float* coef, float* dlogp,
                                      pvl_stream_t stream) {
  const char* who = "pack_policy_bwd";
  LossParams p{};
  const pvl_status st = policy_params(who, h, &p);
  if (st != PVL_OK) return st;
  if (!coef || !dlogp) return fail(PVL_ERR_INVALID_ARG, "%s: null pointer", who);
  if (misaligned({dloss, dlogp}, 4) || misaligned({coef}, 8))
    return fail(PVL_ERR_UNSUPPORTED, "%s: dloss and dlogp must be 4-byte and coef 8-byte aligned", who);
  p.dloss = dloss;
  p.coef = const_cast<float*>(coef);
  p.dlogp = dlogp;
  token_grad_kernel<true><<<blocks_of(p.N, 4 * kBwdThreads), kBwdThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return check_cuda(cudaGetLastError(), "pack_policy_bwd launch");
}
