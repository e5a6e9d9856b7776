// pack_logprob_fwd / pack_logprob_bwd: log-probabilities of given tokens under
// rows of logits, with the entropy of each row, and the gradient to the
// logits, for sm_103a.
//
// With z = x / temperature over the V logits of a token,
//   lse = log sum_i exp z_i,  logp = z_target - lse,  H = lse - sum_i p_i z_i,
//   dx_i = (dlogp (1[i = target] - p_i) - dH p_i (z_i - lse + H)) / temperature,
// with p_i = exp(z_i - lse).  Tokens whose seq_id is negative or whose target
// lies outside [0, V) read nothing, give zeros and have zero gradients.
//
// Forward: one pass.  Every thread keeps a running maximum m (raw logits) and
// the sums s = sum exp2(k (x - m)) and w = sum k (x - m) exp2(k (x - m)),
// k = log2(e) / temperature; states join as sums do after each is scaled to
// the common maximum.  Differences are taken before they are scaled, so that
// large common offsets of the logits cost nothing.  m starts at the lowest
// finite value: a logit of -inf then adds 0, and -inf - (-inf) never arises;
// w clamps the exponent, so that a banned logit adds 0 and not 0 times -inf.
//   Bound by HBM (V elements read once, 16-byte loads, four in flight a
// thread).  A row goes to 8 threads, to a warp, to a block or to a cluster of
// eight blocks that join their states through shared memory: as few threads as
// still fill the device (launch rules below).
//
// Backward: elementwise, given lse and H: V elements read, V written.  A block
// takes up to 4096 vectors of a row, so that what it looks up of the row is
// shared by sixteen vectors a thread, the next four read while four are worked
// on; shorter rows go to a warp or 8 threads.
//
// Measured (one GB300, of the 6793 GB/s of its copy): 65,536 rows of 32,768 bf16
// logits forward 619 us = 6.94 TB/s (102 %), backward 1227 us = 7.00 TB/s (103 %).
//
// Rows need no alignment: the elements up to the first 16-byte boundary and
// those after the last whole vector go one by one.
#include <cuda_runtime.h>

#include <cfloat>

#include "pvl_device.cuh"

namespace pvl {
namespace {

constexpr int kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kFar = -1e30f;  // stands for -inf where it is multiplied by 0
// The same in the gradient, whose probabilities are 0 from -88 on: no further than that, so that its product with a
// large gradient of the entropy stays finite.
constexpr float kGone = -128.0f;
constexpr int kCluster = 8;
constexpr int kSegVec = 16 * kThreads;  // vectors of a row that a backward block takes: sixteen a thread

struct LogprobParams {
  const void* x;
  int64_t sb, sl;  // strides of batch row and token, elements
  const void* target;
  const int32_t* seq_id;
  int32_t L, V;
  int64_t N;
  bool wide;
  float inv_t;
  // forward
  float* logp;
  float* lse;
  float* ent;
  // backward
  const float* dlogp;
  const float* lse_in;
  const float* ent_in;
  const float* dent;
  void* dx;
  int64_t db, dl;
};

// Not through the read-only path: the gradient may be written over the logits.
__device__ __forceinline__ uint4 ld_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// 16 bytes of logits as floats, and back.
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int n = 8;
  static constexpr uint32_t low = 0xFF80FF80u;  // two elements of -inf
  static __device__ __forceinline__ void open(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 close(const float* f) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
  static __device__ __forceinline__ float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  static __device__ __forceinline__ __nv_bfloat16 put(float f) { return __float2bfloat16_rn(f); }
};
template <>
struct Vec<float> {
  static constexpr int n = 4;
  static constexpr uint32_t low = 0xFF800000u;
  static __device__ __forceinline__ void open(const uint4& v, float* f) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 close(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
  static __device__ __forceinline__ float put(float f) { return f; }
};

// Running statistics of a row.
struct Stat {
  float m, s, w;
};

template <bool kEnt, int kN>
__device__ __forceinline__ void take(Stat& a, const float (&x)[kN], float k) {
  float top = x[0];
#pragma unroll
  for (int i = 1; i < kN; ++i) top = fmaxf(top, x[i]);
  const float m = fmaxf(a.m, top);
  const float back = (a.m - m) * k;
  const float c = ex2(back);
  float s = a.s * c, w = 0.0f;
  if (kEnt) w = c * fmaf(a.s, fmaxf(back, kFar), a.w);
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const float t = (x[i] - m) * k;
    const float e = ex2(t);
    s += e;
    if (kEnt) w = fmaf(e, fmaxf(t, kFar), w);
  }
  a.m = m;
  a.s = s;
  a.w = w;
}

template <bool kEnt>
__device__ __forceinline__ void join(Stat& a, const Stat& b, float k) {
  const float m = fmaxf(a.m, b.m);
  const float ta = (a.m - m) * k, tb = (b.m - m) * k;
  const float ca = ex2(ta), cb = ex2(tb);
  if (kEnt) a.w = fmaf(ca, fmaf(a.s, fmaxf(ta, kFar), a.w), cb * fmaf(b.s, fmaxf(tb, kFar), b.w));
  a.s = fmaf(a.s, ca, b.s * cb);
  a.m = m;
}

__device__ __forceinline__ int64_t target_of(const LogprobParams& p, int64_t row) {
  return p.wide ? static_cast<const int64_t*>(p.target)[row] : static_cast<const int32_t*>(p.target)[row];
}

__device__ __forceinline__ bool row_valid(const LogprobParams& p, int64_t row, int64_t target) {
  return target >= 0 && target < p.V && (!p.seq_id || p.seq_id[row] >= 0);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// kG threads a row (8, 32, or the block), or a cluster of blocks.
template <typename T, int kG, bool kEnt, bool kClu>
__global__ void __launch_bounds__(kThreads, 4) logprob_fwd_kernel(const LogprobParams p) {
  constexpr int kN = Vec<T>::n;
  __shared__ Stat warp_stat[kThreads / 32];
  __shared__ Stat block_stat[kCluster];
  const int lane = threadIdx.x % kG;
  const uint32_t rank = kClu ? cluster_rank() : 0;
  if constexpr (kClu) cluster_arrive();  // seen below: every block of the cluster runs before its memory is written
  const int64_t row = kClu ? blockIdx.x / kCluster
                           : static_cast<int64_t>(blockIdx.x) * (kThreads / kG) + threadIdx.x / kG;
  const bool inside = row < p.N;
  const int64_t target = inside ? target_of(p, row) : -1;
  const bool live = inside && row_valid(p, row, target);
  const float k = p.inv_t * kLog2e;
  Stat a{-FLT_MAX, 0.0f, 0.0f};
  float x_target = 0.0f;
  if (live) {
    const T* x = static_cast<const T*>(p.x) + (row / p.L) * p.sb + (row % p.L) * p.sl;
    if (lane == 0) x_target = Vec<T>::one(x + target);
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(x) % 16 / sizeof(T));
    const int head = off ? min(kN - off, p.V) : 0;
    const int nvec = (p.V - head) / kN;
    const int rest = p.V - nvec * kN;  // head and tail elements
    const uint4* v = reinterpret_cast<const uint4*>(x + head);
    constexpr int kStep = kG * (kClu ? kCluster : 1);
    const int first = lane + (kClu ? static_cast<int>(rank) * kG : 0);
    for (int i = first; i < nvec; i += 4 * kStep) {
      uint4 q[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        q[u] = i + u * kStep < nvec ? ld_once(v + i + u * kStep)
                                    : make_uint4(Vec<T>::low, Vec<T>::low, Vec<T>::low, Vec<T>::low);
#pragma unroll
      for (int u = 0; u < 4; u += 2) {
        float f[2 * kN];
        Vec<T>::open(q[u], f);
        Vec<T>::open(q[u + 1], f + kN);
        take<kEnt>(a, f, k);
      }
    }
    if (rest && rank == 0) {
      for (int j = lane; j < rest; j += kG) {
        const float f[1] = {Vec<T>::one(x + (j < head ? j : nvec * kN + j))};
        take<kEnt>(a, f, k);
      }
    }
  }
#pragma unroll
  for (int o = (kG < 32 ? kG : 32) / 2; o > 0; o >>= 1) {
    Stat b;
    b.m = __shfl_xor_sync(0xffffffffu, a.m, o);
    b.s = __shfl_xor_sync(0xffffffffu, a.s, o);
    b.w = kEnt ? __shfl_xor_sync(0xffffffffu, a.w, o) : 0.0f;
    join<kEnt>(a, b, k);
  }
  if constexpr (kG > 32) {
    const int w = threadIdx.x / 32;
    if (threadIdx.x % 32 == 0) warp_stat[w] = a;
    __syncthreads();
    if (w == 0) {
      a = warp_stat[threadIdx.x % (kG / 32)];
#pragma unroll
      for (int o = kG / 64; o > 0; o >>= 1) {
        Stat b;
        b.m = __shfl_xor_sync(0xffffffffu, a.m, o);
        b.s = __shfl_xor_sync(0xffffffffu, a.s, o);
        b.w = kEnt ? __shfl_xor_sync(0xffffffffu, a.w, o) : 0.0f;
        join<kEnt>(a, b, k);
      }
    }
  }
  if constexpr (kClu) {
    cluster_wait();
    if (threadIdx.x == 0) {  // into the slot of this block in the first block's shared memory
      uint32_t to;
      asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(to) : "r"(smem_u32(&block_stat[rank])));
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(a.m) : "memory");
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 4), "f"(a.s) : "memory");
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 8), "f"(a.w) : "memory");
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    if (rank != 0) return;
    if (threadIdx.x == 0) {
#pragma unroll
      for (int i = 1; i < kCluster; ++i) join<kEnt>(a, block_stat[i], k);
    }
  }
  if (lane == 0 && inside) {
    const float log_s = logf(a.s);
    p.logp[row] = live ? fmaf(x_target - a.m, p.inv_t, -log_s) : 0.0f;
    p.lse[row] = live ? fmaf(a.m, p.inv_t, log_s) : 0.0f;
    if (kEnt) p.ent[row] = live ? log_s - kLn2 * a.w / a.s : 0.0f;
  }
}

// What a row's gradient depends on.
struct RowGrad {
  int32_t target;  // -1: the row is zero
  float up;        // dlogp / temperature
  float lse;
  float dent;      // dH / temperature
  float ent;
};

template <bool kEnt>
__device__ __forceinline__ RowGrad row_grad(const LogprobParams& p, int64_t row) {
  const int64_t target = target_of(p, row);
  RowGrad g{-1, 0.0f, 0.0f, 0.0f, 0.0f};
  if (row_valid(p, row, target)) {
    g.target = static_cast<int32_t>(target);
    g.up = p.dlogp ? p.dlogp[row] * p.inv_t : 0.0f;
    g.lse = p.lse_in[row];
    if (kEnt) {
      g.dent = p.dent[row] * p.inv_t;
      g.ent = p.ent_in[row];
    }
  }
  return g;
}

template <bool kEnt>
__device__ __forceinline__ float grad_of(float x, float inv_t, const RowGrad& g) {
  const float z = fmaf(x, inv_t, -g.lse);
  const float pr = ex2(z * kLog2e);
  float up = g.up;
  if (kEnt) up = fmaf(g.dent, fmaxf(z, kGone) + g.ent, up);
  return -pr * up;
}

// Four vectors i, i + step, ... of a row: their logits.
template <typename T, bool kSame>
__device__ __forceinline__ void load_vectors(const T* x, int i, int step, int end, uint4 (&q)[4]) {
  constexpr int kN = Vec<T>::n;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    if (i + u * step >= end) continue;
    const T* at = x + static_cast<int64_t>(i + u * step) * kN;
    if (kSame) {
      q[u] = ld_once(at);
    } else {  // the rows lie differently to the 16-byte boundaries: vectors of dx, elements of x
      float f[kN];
#pragma unroll
      for (int e = 0; e < kN; ++e) f[e] = Vec<T>::one(at + e);
      q[u] = Vec<T>::close(f);
    }
  }
}

// Vectors first, first + step, ... below end of a row (x, dx: its first whole
// vector of dx), the next four read while these are worked on.
template <typename T, bool kEnt, bool kSame>
__device__ __forceinline__ void grad_vectors(const RowGrad& g, float inv_t, const T* x, T* dx, int target, int first,
                                             int step, int end) {
  constexpr int kN = Vec<T>::n;
  uint4 q[4], next[4];
  load_vectors<T, kSame>(x, first, step, end, q);
  for (int i = first; i < end; i += 4 * step) {
    load_vectors<T, kSame>(x, i + 4 * step, step, end, next);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int at = i + u * step;
      if (at >= end) continue;
      float f[kN];
      Vec<T>::open(q[u], f);
#pragma unroll
      for (int e = 0; e < kN; ++e) f[e] = grad_of<kEnt>(f[e], inv_t, g);
      const int here = target - at * kN;
      if (here >= 0 && here < kN) {
#pragma unroll
        for (int e = 0; e < kN; ++e) f[e] += e == here ? g.up : 0.0f;
      }
      *reinterpret_cast<uint4*>(dx + static_cast<int64_t>(at) * kN) = Vec<T>::close(f);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) q[u] = next[u];
  }
}

// kG threads a row (8, 32), or per_row blocks of kSegVec vectors each.
template <typename T, bool kEnt, int kG>
__global__ void __launch_bounds__(kThreads, 3) logprob_bwd_kernel(const LogprobParams p, uint32_t per_row) {
  constexpr int kN = Vec<T>::n;
  constexpr bool kBlock = kG == kThreads;
  const int lane = threadIdx.x % kG;
  const int64_t row = kBlock ? blockIdx.x / per_row
                             : static_cast<int64_t>(blockIdx.x) * (kThreads / kG) + threadIdx.x / kG;
  if (row >= p.N) return;
  const int seg = kBlock ? static_cast<int>(blockIdx.x % per_row) : 0;
  const int64_t b = row / p.L, l = row - b * p.L;
  const T* x = static_cast<const T*>(p.x) + b * p.sb + l * p.sl;
  T* dx = static_cast<T*>(p.dx) + b * p.db + l * p.dl;
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(dx) % 16 / sizeof(T));
  const bool same = (reinterpret_cast<uintptr_t>(x) - reinterpret_cast<uintptr_t>(dx)) % 16 == 0;
  const int head = off ? min(kN - off, p.V) : 0;
  const int nvec = (p.V - head) / kN;
  const int first = seg * kSegVec + lane;
  const int end = kBlock ? min(nvec, (seg + 1) * kSegVec) : nvec;
  const RowGrad g = row_grad<kEnt>(p, row);
  if (g.target < 0) {
    for (int i = first; i < end; i += kG)
      *reinterpret_cast<uint4*>(dx + head + static_cast<int64_t>(i) * kN) = make_uint4(0u, 0u, 0u, 0u);
  } else if (same) {
    grad_vectors<T, kEnt, true>(g, p.inv_t, x + head, dx + head, g.target - head, first, kG, end);
  } else {
    grad_vectors<T, kEnt, false>(g, p.inv_t, x + head, dx + head, g.target - head, first, kG, end);
  }
  const int rest = seg == 0 ? p.V - nvec * kN : 0;
  for (int r = lane; r < rest; r += kG) {
    const int j = r < head ? r : nvec * kN + r;
    float f = 0.0f;
    if (g.target >= 0) {
      f = grad_of<kEnt>(Vec<T>::one(x + j), p.inv_t, g);
      if (j == g.target) f += g.up;
    }
    dx[j] = Vec<T>::put(f);
  }
}

pvl_status validate(const char* who, const pvl_logprob* h, LogprobParams* p) {
  if (!h || !h->logits || !h->targets) return fail(PVL_ERR_INVALID_ARG, "%s: null pointer", who);
  if (h->B < 1 || h->L < 1 || h->V < 1) return fail(PVL_ERR_INVALID_ARG, "%s: B, L and V must be >= 1", who);
  if (h->dtype != 0 && h->dtype != 1) return fail(PVL_ERR_INVALID_ARG, "%s: dtype %d (0: bf16, 1: fp32)", who, h->dtype);
  if (h->wide_targets != 0 && h->wide_targets != 1)
    return fail(PVL_ERR_INVALID_ARG, "%s: wide_targets %d (0: int32, 1: int64)", who, h->wide_targets);
  if (!(h->temperature > 1e-30f) || !(h->temperature < 1e30f))
    return fail(PVL_ERR_INVALID_ARG, "%s: temperature must be positive and finite", who);
  const int64_t N = static_cast<int64_t>(h->B) * h->L;
  if (h->V > (1 << 28) || N >= (1ll << 27) || N * h->V >= (1ll << 42))
    return fail(PVL_ERR_UNSUPPORTED, "%s: %lld rows of %d logits are too many", who, static_cast<long long>(N), h->V);
  if (h->batch_stride < 0 || h->token_stride < 0 || h->batch_stride >= (1ll << 46) || h->token_stride >= (1ll << 46))
    return fail(PVL_ERR_INVALID_ARG, "%s: strides must not be negative", who);
  const uintptr_t es = h->dtype ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(h->logits) % es || reinterpret_cast<uintptr_t>(h->targets) % (h->wide_targets ? 8 : 4) ||
      reinterpret_cast<uintptr_t>(h->seq_id) % 4)
    return fail(PVL_ERR_UNSUPPORTED, "%s: a pointer is not aligned to its elements", who);
  p->x = h->logits;
  p->sb = h->batch_stride;
  p->sl = h->token_stride;
  p->target = h->targets;
  p->seq_id = h->seq_id;
  p->L = h->L;
  p->V = h->V;
  p->N = N;
  p->wide = h->wide_targets != 0;
  p->inv_t = 1.0f / h->temperature;
  return PVL_OK;
}

template <typename T, int kG, bool kClu>
pvl_status launch_fwd(const LogprobParams& p, cudaStream_t s) {
  const int64_t blocks = kClu ? p.N * kCluster : (p.N + kThreads / kG - 1) / (kThreads / kG);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = kCluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = kClu ? 1 : 0;
  const cudaError_t e = p.ent ? cudaLaunchKernelEx(&cfg, logprob_fwd_kernel<T, kG, true, kClu>, p)
                              : cudaLaunchKernelEx(&cfg, logprob_fwd_kernel<T, kG, false, kClu>, p);
  return check_cuda(e, "pack_logprob_fwd launch");
}

// How many threads take a row, measured in microseconds (bf16, N rows of V, 8
// logits a vector; a row's other choice beside it).
//   8 threads, for up to 256 vectors, once rows are many enough that 8 threads
// each fill the SMs, the more the longer they are: 20,000 x 256 3.9 (a warp
// 10.1), x 1024 8.6 (10.4), x 2048 14.6 (15.8); 4864 x 256 2.5 (3.7), x 1024 3.7
// (3.7), x 2048 5.6 (4.8: a warp); 1216 x 512 2.7 (2.3: a warp).
//   A warp, for up to 2048 vectors, with eight rows an SM and more: 20,000 x 8192
// 51 (a block 75), x 16,384 102 (113), x 32,768 195 (193: a block); 1216 x 8192
// 5.3 (6.0); 300 x 8192 5.2 (2.9: a block).  With fewer rows up to 128 vectors:
// 64 x 512 2.3 (2.3), 300 x 2048 2.9 (2.9).
//   A cluster for few long rows, whose eight blocks must be worth their barrier:
// 8 x 32,768 2.9 (a block 3.7), 64 x 128,000 5.6 (8.6), 152 x 128,000 10.9
// (14.2); 8 x 16,384 3.1 (2.9: a block), 64 x 32,768 4.7 (3.9: a block).
template <typename T>
pvl_status fwd(const LogprobParams& p, cudaStream_t s) {
  const int64_t vectors = p.V / Vec<T>::n;
  const int64_t sms = sm_count();
  if (sms <= 0) return fail(PVL_ERR_CUDA, "pack_logprob_fwd: no usable CUDA device");
  if (vectors <= 256 && 4 * p.N >= sms * vectors) return launch_fwd<T, 8, false>(p, s);
  if (vectors <= 128 || (vectors <= 2048 && p.N >= 8 * sms)) return launch_fwd<T, 32, false>(p, s);
  if (vectors >= 4096 && 80 * p.N <= vectors) return launch_fwd<T, kThreads, true>(p, s);
  return launch_fwd<T, kThreads, false>(p, s);
}

// 8 threads, a warp or a block a row (microseconds as above).  8 threads: 20,000 x
// 256 4.3 (a warp 7.8), x 512 6.4 (9.3), x 1024 12.5 (12.2: a warp), 4864 x 512 3.1
// (3.2).  A warp: 20,000 x 2048 26 (a block 67), x 8192 100 (118), x 16,384 207
// (196: a block), 1216 x 8192 5.6 (6.2); with fewer rows than eight an SM up to 64
// vectors: 300 x 512 2.3 (2.5), x 2048 3.1 (2.6: a block).
template <typename T, bool kEnt>
pvl_status launch_bwd(const LogprobParams& p, cudaStream_t s) {
  const int64_t vectors = p.V / Vec<T>::n;
  const int64_t sms = sm_count();
  if (sms <= 0) return fail(PVL_ERR_CUDA, "pack_logprob_bwd: no usable CUDA device");
  if (vectors <= 64 && 4 * p.N >= sms * vectors) {
    constexpr int kRows = kThreads / 8;
    logprob_bwd_kernel<T, kEnt, 8><<<static_cast<unsigned>((p.N + kRows - 1) / kRows), kThreads, 0, s>>>(p, 1);
  } else if (vectors > 1024 || (vectors > 64 && p.N < 8 * sms)) {
    const int64_t per_row = (vectors + kSegVec - 1) / kSegVec;
    if (p.N * per_row >= (1ll << 31)) return fail(PVL_ERR_UNSUPPORTED, "pack_logprob_bwd: too many rows");
    logprob_bwd_kernel<T, kEnt, kThreads><<<static_cast<unsigned>(p.N * per_row), kThreads, 0, s>>>(
        p, static_cast<uint32_t>(per_row));
  } else {
    constexpr int kRows = kThreads / 32;
    logprob_bwd_kernel<T, kEnt, 32><<<static_cast<unsigned>((p.N + kRows - 1) / kRows), kThreads, 0, s>>>(p, 1);
  }
  return check_cuda(cudaGetLastError(), "pack_logprob_bwd launch");
}

template <typename T>
pvl_status bwd(const LogprobParams& p, cudaStream_t s) {
  return p.dent ? launch_bwd<T, true>(p, s) : launch_bwd<T, false>(p, s);
}

}  // namespace
}  // namespace pvl

using namespace pvl;

extern "C" pvl_status pack_logprob_fwd(const pvl_logprob* how, float* logp, float* lse, float* entropy,
                                       pvl_stream_t stream) {
  LogprobParams p{};
  const pvl_status st = validate("pack_logprob_fwd", how, &p);
  if (st != PVL_OK) return st;
  if (!logp || !lse) return fail(PVL_ERR_INVALID_ARG, "pack_logprob_fwd: null pointer");
  if (reinterpret_cast<uintptr_t>(logp) % 4 || reinterpret_cast<uintptr_t>(lse) % 4 ||
      reinterpret_cast<uintptr_t>(entropy) % 4)
    return fail(PVL_ERR_UNSUPPORTED, "pack_logprob_fwd: a pointer is not aligned to its elements");
  p.logp = logp;
  p.lse = lse;
  p.ent = entropy;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return how->dtype ? fwd<float>(p, s) : fwd<__nv_bfloat16>(p, s);
}

extern "C" pvl_status pack_logprob_bwd(const pvl_logprob* how, const float* lse, const float* entropy,
                                       const float* dlogp, const float* dentropy, void* dlogits, int64_t batch_stride,
                                       int64_t token_stride, pvl_stream_t stream) {
  LogprobParams p{};
  const pvl_status st = validate("pack_logprob_bwd", how, &p);
  if (st != PVL_OK) return st;
  if (!lse || !dlogits || (!dlogp && !dentropy)) return fail(PVL_ERR_INVALID_ARG, "pack_logprob_bwd: null pointer");
  if (dentropy && !entropy)
    return fail(PVL_ERR_INVALID_ARG, "pack_logprob_bwd: the gradient of the entropy needs the entropy");
  const uintptr_t es = how->dtype ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(lse) % 4 || reinterpret_cast<uintptr_t>(entropy) % 4 ||
      reinterpret_cast<uintptr_t>(dlogp) % 4 || reinterpret_cast<uintptr_t>(dentropy) % 4 ||
      reinterpret_cast<uintptr_t>(dlogits) % es)
    return fail(PVL_ERR_UNSUPPORTED, "pack_logprob_bwd: a pointer is not aligned to its elements");
  // rows laid token by token inside batch rows, or batch row by batch row inside tokens
  const int64_t B = how->B, L = how->L, V = how->V;
  const bool tokens_inside = (L == 1 || token_stride >= V) && (B == 1 || batch_stride >= (L - 1) * token_stride + V);
  const bool batch_inside = (B == 1 || batch_stride >= V) && (L == 1 || token_stride >= (B - 1) * batch_stride + V);
  if (batch_stride < 0 || token_stride < 0 || batch_stride >= (1ll << 46) || token_stride >= (1ll << 46) ||
      !(tokens_inside || batch_inside))
    return fail(PVL_ERR_INVALID_ARG, "pack_logprob_bwd: rows of dlogits overlap");
  const uintptr_t from = reinterpret_cast<uintptr_t>(how->logits), to = reinterpret_cast<uintptr_t>(dlogits);
  const uintptr_t reads = ((B - 1) * how->batch_stride + (L - 1) * how->token_stride + V) * es;
  const uintptr_t writes = ((B - 1) * batch_stride + (L - 1) * token_stride + V) * es;
  const bool same = from == to && (B == 1 || batch_stride == how->batch_stride) && (L == 1 || token_stride == how->token_stride);
  if (!same && from < to + writes && to < from + reads)
    return fail(PVL_ERR_INVALID_ARG, "pack_logprob_bwd: dlogits reaches into the logits without being them");
  p.lse_in = lse;
  p.ent_in = entropy;
  p.dlogp = dlogp;
  p.dent = dentropy;
  p.dx = dlogits;
  p.db = batch_stride;
  p.dl = token_stride;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return how->dtype ? bwd<float>(p, s) : bwd<__nv_bfloat16>(p, s);
}
