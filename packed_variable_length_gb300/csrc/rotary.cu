// pack_rotary_fwd / pack_rotary_bwd: rotary positions of queries and keys,
// with the RMS norm before them and its weight gradients, for sm_103a.
//
// What it computes, per head vector x [D]: z = x r w (no norm: z = x), then
// for each pair (a, b) of the first R features, with t = position x frequency,
//   (a, b) -> gain (a cos t - b sin t, a sin t + b cos t).
// Backward, with g the upstream gradient turned by -t (times gain):
//   no norm: dx = g;  else, n the features the norm runs over,
//   dx = r (g w - xh mean_n(g w xh)),  xh = x r,   dw = sum g xh.
//
// Angles.  A frequency is given in turns per position as a fraction F of
// 2^64, so the angle in turns is position x F mod 2^64: one wrapping integer
// product, whose top 32 bits are the angle as a signed fraction of a turn,
// exact for any position.  sin.approx / cos.approx on [-pi, pi] are then off
// by about 2^-21, far below the 2^-9 of the bf16 result.
//
// Layout of the work.  HBM bound: 4 bytes an element forward, 6 backward with
// a norm.  A unit is the 2 V features of V pairs: two V-wide vectors, R / 2
// apart in the half layout, adjacent in the interleaved one.  A team of
// threads takes one token: a thread owns one unit column of the head (so its
// angles, computed once a token, serve all its heads) and every hpi-th head,
// kM of them at a time; queries and keys are one run of heads.  The kM heads'
// vectors are all loaded before the first is used; the norm over the token
// holds all of its heads at once.  Teams are whole warps, or a
// power of two below 32 for tokens of few units.
#include <cuda_runtime.h>

#include "pvl_device.cuh"

namespace pvl {
namespace {

constexpr int kMaxBlock = 512;
constexpr int kMaxD = 256;
constexpr int kMaxPartials = 1216;  // blocks of a backward that sums weight gradients

struct RotaryParams {
  pvl_heads x[2];    // q, k: the forward's input (backward: with a norm)
  pvl_heads g[2];    // backward: gradients of the outputs
  pvl_heads out[2];  // forward: rotated; backward: dq, dk
  const uint64_t* turns;
  const int32_t* positions;
  const float* w[2];
  float* part;       // backward: [blocks][width] partial weight gradients, null: none
  int L, H, Ht, D, R;
  int half, axes, section_1, section_2;
  int units;         // units of a head, D / (2 V)
  int turned;        // units of a head that are rotated, R / (2 V)
  int hpi;           // heads a team takes at once
  int team, teams;   // threads of a team, teams of a block
  uint32_t tokens;   // B * L
  int width;         // columns of part
  float gain, eps;
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
struct Vec<1> {
  using T = uint16_t;
};

template <int V>
__device__ __forceinline__ void unpack(const typename Vec<V>::T& u, float* f) {
  if constexpr (V == 1) {
    f[0] = __uint_as_float(static_cast<uint32_t>(u) << 16);
  } else {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&u);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}
template <int V>
__device__ __forceinline__ typename Vec<V>::T pack(const float* f) {
  typename Vec<V>::T u;
  if constexpr (V == 1) {
    u = __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
  } else {
    uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
  }
  return u;
}

constexpr float kRadians = 1.4629180792671596e-9f;  // 2 pi / 2^32

// Rotates one unit (z[0..V) the first vector, z[V..2V) the second).
template <int V>
__device__ __forceinline__ void rotate(float* z, const float* c, const float* s, bool half) {
  if (half) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float a = z[e], b = z[V + e];
      z[e] = fmaf(a, c[e], -(b * s[e]));
      z[V + e] = fmaf(a, s[e], b * c[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float a = z[2 * e], b = z[2 * e + 1];
      z[2 * e] = fmaf(a, c[e], -(b * s[e]));
      z[2 * e + 1] = fmaf(a, s[e], b * c[e]);
    }
  }
}

// Sum over the `n` threads of an aligned power-of-two lane group.
__device__ __forceinline__ float lane_sum(float v, int n) {
  for (int o = 1; o < n; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// kNorm: PVL_NORM_NONE, _HEAD or _TOKEN.
template <int V, int kM, int kNorm, bool kBwd>
__global__ void __launch_bounds__(kMaxBlock) rotary_kernel(const RotaryParams p) {
  using T = typename Vec<V>::T;
  constexpr bool kHead = kNorm == PVL_NORM_HEAD, kToken = kNorm == PVL_NORM_TOKEN, kAny = kHead || kToken;
  constexpr int kSums = kBwd ? 2 : 1;      // sum x^2, and backward sum g w x
  extern __shared__ float table[];         // reductions, and at the end the head norm's weight gradients
  const int tid = threadIdx.x;
  const int slot = tid / p.team, lane = tid % p.team;
  const int u = lane % p.units, hl = lane / p.units;
  const bool on = slot < p.teams && hl < p.hpi;
  const bool turned = u < p.turned;
  // features of the unit's two vectors
  const int e0 = turned && p.half ? u * V : 2 * u * V;
  const int e1 = turned && p.half ? u * V + p.R / 2 : e0 + V;
  uint64_t turns[V];
  uint32_t axis = 0;  // 2 bits a pair
  if (turned) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int pair = u * V + e;
      turns[e] = __ldg(p.turns + pair);
      axis |= (pair < p.section_1 ? 0u : pair < p.section_2 ? 1u : 2u) << (2 * e);
    }
  }
  float acc[kBwd && kAny ? (kToken ? kM : 2) : 1][2 * V];
  if (kBwd && kAny) {
#pragma unroll
    for (int i = 0; i < (kToken ? kM : 2); ++i)
#pragma unroll
      for (int e = 0; e < 2 * V; ++e) acc[kBwd && kAny ? i : 0][e] = 0.0f;
  }
  // a head of the run of queries and keys: address of its vectors in a view
  auto at = [&](const pvl_heads (&v)[2], int h, uint32_t b, uint32_t l) {
    const bool key = h >= p.H;
    const int64_t off = b * (key ? v[1].stride_b : v[0].stride_b) + l * (key ? v[1].stride_l : v[0].stride_l) +
                        (key ? (h - p.H) * v[1].stride_h : h * v[0].stride_h);
    return static_cast<__nv_bfloat16*>(key ? v[1].data : v[0].data) + off;
  };
  // the norm weight of the unit's feature e of head h
  auto weight = [&](int h, int e) {
    const bool key = h >= p.H;
    const float* w = key ? p.w[1] : p.w[0];
    if (w == nullptr) return 1.0f;
    return __ldg(w + (kToken ? (key ? h - p.H : h) * p.D : 0) + (e < V ? e0 + e : e1 + e - V));
  };
  const uint32_t step = gridDim.x * p.teams;
  for (uint32_t base = blockIdx.x * p.teams; base < p.tokens; base += step) {
    const uint32_t token = base + slot;
    const bool live = on && token < p.tokens;
    const uint32_t b = token / p.L, l = token - b * p.L;
    float c[V], s[V];
    if (turned && live) {
      int32_t pos[3] = {0, 0, 0};
#pragma unroll
      for (int a = 0; a < 3; ++a)
        if (a < p.axes) pos[a] = __ldg(p.positions + static_cast<size_t>(token) * p.axes + a);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const uint32_t a = (axis >> (2 * e)) & 3u;
        const int32_t n = a == 0 ? pos[0] : a == 1 ? pos[1] : pos[2];
        const uint64_t frac = turns[e] * static_cast<uint64_t>(static_cast<int64_t>(n));  // mod 1 turn
        const float angle = static_cast<float>(static_cast<int32_t>(frac >> 32)) * kRadians;
        c[e] = __cosf(angle) * p.gain;
        s[e] = __sinf(angle) * (kBwd ? -p.gain : p.gain);
      }
    }
    for (int h0 = hl; h0 - hl < p.Ht; h0 += kM * p.hpi) {
    // the heads' loads first
    T xa[kM], xb[kM], ga[kM], gb[kM];
#pragma unroll
    for (int m = 0; m < kM; ++m) {
      const int h = h0 + m * p.hpi;
      if (live && h < p.Ht) {
        if (!kBwd || kAny) {
          const __nv_bfloat16* row = at(p.x, h, b, l);
          xa[m] = *reinterpret_cast<const T*>(row + e0);
          xb[m] = *reinterpret_cast<const T*>(row + e1);
        }
        if (kBwd) {
          const __nv_bfloat16* row = at(p.g, h, b, l);
          ga[m] = *reinterpret_cast<const T*>(row + e0);
          gb[m] = *reinterpret_cast<const T*>(row + e1);
        }
      }
    }
    // the norms' sums
    float r[kM], mean[kM];  // 1 / rms; backward r^3 mean(g w x)
    if (kAny) {
      float part[kM][kSums];
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        const int h = h0 + m * p.hpi;
        part[m][0] = 0.0f;
        if (kBwd) part[m][kSums - 1] = 0.0f;
        if (live && h < p.Ht) {
          float x[2 * V];
          unpack<V>(xa[m], x);
          unpack<V>(xb[m], x + V);
          float q = 0.0f;
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) q = fmaf(x[e], x[e], q);
          part[m][0] = q;
          if (kBwd) {
            float g[2 * V];
            unpack<V>(ga[m], g);
            unpack<V>(gb[m], g + V);
            if (turned) rotate<V>(g, c, s, p.half);
            q = 0.0f;
#pragma unroll
            for (int e = 0; e < 2 * V; ++e) q = fmaf(g[e] * weight(h, e), x[e], q);
            part[m][kSums - 1] = q;
          }
        }
      }
      const bool pow2 = (p.units & (p.units - 1)) == 0 && p.units <= 32;
      if (kHead) {
        if (pow2) {
#pragma unroll
          for (int m = 0; m < kM; ++m)
#pragma unroll
            for (int k = 0; k < kSums; ++k) part[m][k] = lane_sum(part[m][k], p.units);
        } else {
          const int n = blockDim.x;
          __syncthreads();
#pragma unroll
          for (int m = 0; m < kM; ++m)
#pragma unroll
            for (int k = 0; k < kSums; ++k) table[(m * kSums + k) * n + tid] = part[m][k];
          __syncthreads();
#pragma unroll
          for (int m = 0; m < kM; ++m)
#pragma unroll
            for (int k = 0; k < kSums; ++k) {
              const float* q = table + (m * kSums + k) * n + tid - u;
              float t = 0.0f;
              if (on)
                for (int i = 0; i < p.units; ++i) t += q[i];
              part[m][k] = t;
            }
        }
      } else {
        // queries and keys apart
        float sum[2][kSums];
#pragma unroll
        for (int k = 0; k < kSums; ++k) sum[0][k] = sum[1][k] = 0.0f;
#pragma unroll
        for (int m = 0; m < kM; ++m) {
          const bool key = h0 + m * p.hpi >= p.H;
#pragma unroll
          for (int k = 0; k < kSums; ++k) {
            sum[0][k] += key ? 0.0f : part[m][k];
            sum[1][k] += key ? part[m][k] : 0.0f;
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int k = 0; k < kSums; ++k) sum[i][k] = lane_sum(sum[i][k], p.team < 32 ? p.team : 32);
        if (p.team > 32) {
          const int warps = p.team / 32, first_warp = slot * warps;
          __syncthreads();
          if ((tid & 31) == 0) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int k = 0; k < kSums; ++k) table[(tid >> 5) * 2 * kSums + i * kSums + k] = sum[i][k];
          }
          __syncthreads();
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < kSums; ++k) sum[i][k] = 0.0f;
          for (int w = 0; w < warps; ++w) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int k = 0; k < kSums; ++k) sum[i][k] += table[(first_warp + w) * 2 * kSums + i * kSums + k];
          }
        }
#pragma unroll
        for (int m = 0; m < kM; ++m) {
          const bool key = h0 + m * p.hpi >= p.H;
#pragma unroll
          for (int k = 0; k < kSums; ++k) part[m][k] = key ? sum[1][k] : sum[0][k];
        }
      }
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        const bool key = h0 + m * p.hpi >= p.H;
        const float n = static_cast<float>(kHead ? p.D : p.D * (key ? p.Ht - p.H : p.H));
        r[m] = rsqrtf(part[m][0] / n + p.eps);
        mean[m] = kBwd ? r[m] * r[m] * r[m] * (part[m][kSums - 1] / n) : 0.0f;
      }
    }
#pragma unroll
    for (int m = 0; m < kM; ++m) {
      const int h = h0 + m * p.hpi;
      if (live && h < p.Ht) {
        float z[2 * V];
        if (!kBwd) {
          unpack<V>(xa[m], z);
          unpack<V>(xb[m], z + V);
          if (kAny) {
#pragma unroll
            for (int e = 0; e < 2 * V; ++e) z[e] = z[e] * r[m] * weight(h, e);
          }
          if (turned) rotate<V>(z, c, s, p.half);
        } else {
          unpack<V>(ga[m], z);
          unpack<V>(gb[m], z + V);
          if (turned) rotate<V>(z, c, s, p.half);
          if (kAny) {
            float x[2 * V];
            unpack<V>(xa[m], x);
            unpack<V>(xb[m], x + V);
#pragma unroll
            for (int e = 0; e < 2 * V; ++e) {
              const float d = z[e] * x[e] * r[m];  // g xh
              if (kToken) {
                acc[m][e] += d;
              } else {
                acc[0][e] += h >= p.H ? 0.0f : d;
                acc[1][e] += h >= p.H ? d : 0.0f;
              }
              z[e] = fmaf(z[e] * weight(h, e), r[m], -x[e] * mean[m]);
            }
          }
        }
        __nv_bfloat16* row = at(p.out, h, b, l);
        *reinterpret_cast<T*>(row + e0) = pack<V>(z);
        *reinterpret_cast<T*>(row + e1) = pack<V>(z + V);
      }
    }
    }
  }
  if (kBwd && kAny) {
    if (p.part == nullptr) return;
    if (kToken) {
      // one row of partial sums for each team
      if (on) {
        float* row = p.part + (static_cast<size_t>(blockIdx.x) * p.teams + slot) * p.width;
#pragma unroll
        for (int m = 0; m < kM; ++m) {
          const int h = hl + m * p.hpi;
          if (h < p.Ht) {
#pragma unroll
            for (int e = 0; e < 2 * V; ++e)
              row[static_cast<size_t>(h) * p.D + (e < V ? e0 + e : e1 + e - V)] = acc[kBwd && kAny ? m : 0][e];
          }
        }
      }
    } else {
      // the block's teams and heads added feature by feature, queries then keys
      float* row = p.part + static_cast<size_t>(blockIdx.x) * p.width;
      const int per = p.hpi;  // threads of a team that own one feature
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        __syncthreads();
        if (on) {
#pragma unroll
          for (int e = 0; e < 2 * V; ++e)
            table[(slot * per + hl) * p.D + (e < V ? e0 + e : e1 + e - V)] = acc[kBwd && kAny ? k : 0][e];
        }
        __syncthreads();
        for (int d = tid; d < p.D; d += blockDim.x) {
          float t = 0.0f;
          for (int i = 0; i < p.teams * per; ++i) t += table[i * p.D + d];
          row[k * p.D + d] = t;
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
// heads does not fit a block and `whole` asks for it.
bool team_of(int V, int kM, int Ht, int D, bool whole, Shape* s) {
  s->V = V;
  s->kM = kM;
  s->units = D / (2 * V);
  s->hpi = (Ht + kM - 1) / kM;
  if (s->units * s->hpi > kMaxBlock) {
    if (whole) return false;
    s->hpi = kMaxBlock / s->units;  // units <= 128
  }
  const int n = s->units * s->hpi;
  if (n >= 17) {
    s->team = round32(n);
    // heads that the rounding leaves room for
    const int fit = s->team / s->units;
    s->hpi = fit < Ht ? fit : Ht;
  } else {
    s->team = 1;
    while (s->team < n) s->team <<= 1;
  }
  s->teams = s->team >= 128 ? 1 : 128 / s->team;
  s->threads = s->team * s->teams;
  return true;
}

template <int V, int kM, bool kBwd>
pvl_status launch_norm(const RotaryParams& p, int norm, int threads, size_t smem, int grid_limit, int* grid_out,
                       cudaStream_t s, const char* who) {
  const void* fn = norm == PVL_NORM_NONE ? reinterpret_cast<const void*>(&rotary_kernel<V, kM, PVL_NORM_NONE, kBwd>)
                                         : reinterpret_cast<const void*>(&rotary_kernel<V, kM, PVL_NORM_HEAD, kBwd>);
  if constexpr (V < 8 || kM <= 2)
    if (norm == PVL_NORM_TOKEN) fn = reinterpret_cast<const void*>(&rotary_kernel<V, kM, PVL_NORM_TOKEN, kBwd>);
  pvl_status st = PVL_OK;
  if (smem > 48 * 1024) {
    st = check_cuda(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)), who);
    if (st != PVL_OK) return st;
  }
  int occ = 0;
  st = check_cuda(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, fn, threads, smem), who);
  if (st != PVL_OK) return st;
  const int sms = sm_count();
  if (sms <= 0 || occ <= 0) return fail(PVL_ERR_CUDA, "%s: no usable CUDA device", who);
  long long grid = static_cast<long long>(occ) * sms;
  if (grid > grid_limit) grid = grid_limit;
  const long long need = (static_cast<long long>(p.tokens) + p.teams - 1) / p.teams;
  if (grid > need) grid = need;
  *grid_out = static_cast<int>(grid);
  RotaryParams q = p;
  void* args[] = {&q};
  st = check_cuda(cudaLaunchKernel(fn, dim3(static_cast<unsigned>(grid)), dim3(threads), args, smem, s), who);
  return st;
}

template <bool kBwd>
pvl_status launch(const RotaryParams& p, const Shape& sh, int norm, int grid_limit, int* grid_out, cudaStream_t s,
                  const char* who) {
  // reductions: a float for each thread, head and sum; the weight gradients of
  // the norm per head: one row of D for each thread group that shares a unit
  size_t smem = 0;
  if (norm == PVL_NORM_TOKEN) smem = 32 * 4 * sizeof(float);
  if (norm == PVL_NORM_HEAD) {
    smem = static_cast<size_t>(sh.threads) * sh.kM * (kBwd ? 2 : 1) * sizeof(float);
    const size_t rows = static_cast<size_t>(sh.teams) * sh.hpi * p.D * sizeof(float);
    if (kBwd && rows > smem) smem = rows;
  }
#define PVL_ROTARY_CASE(VV, MM) \
  if (sh.V == VV && sh.kM == MM) return launch_norm<VV, MM, kBwd>(p, norm, sh.threads, smem, grid_limit, grid_out, s, who)
  PVL_ROTARY_CASE(8, 1);
  PVL_ROTARY_CASE(8, 2);
  PVL_ROTARY_CASE(8, 3);
  PVL_ROTARY_CASE(8, 4);
  PVL_ROTARY_CASE(4, 4);
  PVL_ROTARY_CASE(1, 16);
#undef PVL_ROTARY_CASE
  return fail(PVL_ERR_UNSUPPORTED, "%s: no kernel for this shape", who);
}

// Widest vector that divides the head, its rotated part, every stride and
// every address.
int widest(const pvl_rotary* a, const pvl_heads* const* views, int n) {
  for (int V : {8, 4}) {
    bool ok = a->D % (2 * V) == 0 && a->R % (2 * V) == 0;
    for (int i = 0; i < n && ok; ++i)
      if (views[i])
        ok = reinterpret_cast<uintptr_t>(views[i]->data) % (2 * V) == 0 && views[i]->stride_b % V == 0 &&
             views[i]->stride_l % V == 0 && views[i]->stride_h % V == 0;
    if (ok) return V;
  }
  return 1;
}

// Heads a thread at a time.  One while the tokens leave SMs without a block
// (latency counts: most threads, fewest dependent steps); else the count that
// leaves the fewest threads without a head, the larger one where equal.
bool shape_of(const pvl_rotary* a, int V, Shape* s) {
  const int Ht = a->H + a->Hk;
  const bool whole = a->norm == PVL_NORM_TOKEN;
  if (V != 8) return team_of(V, V == 4 ? 4 : 16, Ht, a->D, whole, s);
  const long long tokens = static_cast<long long>(a->B) * a->L;
  if (tokens <= 2 * 152 && team_of(8, 1, Ht, a->D, whole, s)) return true;
  bool found = false;
  double best = 0.0;
  for (int m = whole ? 2 : 4; m >= 1; --m) {
    Shape t{};
    if (!team_of(8, m, Ht, a->D, whole, &t)) continue;
    const int rounds = (Ht + t.hpi * m - 1) / (t.hpi * m);
    const double used = static_cast<double>(Ht) * t.units / (static_cast<double>(t.team) * m * rounds);
    if (!found || used > best + 1e-9) {
      best = used;
      *s = t;
    }
    found = true;
  }
  return found;
}

pvl_status check_views(const char* who, const pvl_rotary* a, const pvl_heads* v, int which, const char* name) {
  const int heads = which ? a->Hk : a->H;
  if (heads == 0) return PVL_OK;
  if (!v || !v->data) return fail(PVL_ERR_INVALID_ARG, "%s: %s is null", who, name);
  if (reinterpret_cast<uintptr_t>(v->data) % 2 != 0)
    return fail(PVL_ERR_UNSUPPORTED, "%s: %s is not 2-byte aligned", who, name);
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
  if (static_cast<long long>(a->B) * a->L >= (1ll << 31))
    return fail(PVL_ERR_UNSUPPORTED, "%s: too many tokens", who);
  p.turns = a->turns;
  p.positions = a->positions;
  p.w[0] = a->q_weight;
  p.w[1] = a->k_weight;
  p.L = a->L;
  p.H = a->H;
  p.Ht = a->H + a->Hk;
  p.D = a->D;
  p.R = a->R;
  p.half = a->layout == PVL_ROTARY_HALF;
  p.axes = a->axes;
  p.section_1 = a->section_1;
  p.section_2 = a->section_2;
  p.tokens = static_cast<uint32_t>(static_cast<long long>(a->B) * a->L);
  p.gain = a->gain;
  p.eps = a->eps;
  return PVL_OK;
}

void fill(RotaryParams& p, const pvl_rotary* a, const Shape& s) {
  p.units = s.units;
  p.turned = a->R / (2 * s.V);
  p.hpi = s.hpi;
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
  if (st == PVL_OK) st = check_views(who, a, q_out, 0, "q_out");
  if (st == PVL_OK) st = check_views(who, a, k_out, 1, "k_out");
  if (st != PVL_OK) return st;
  const pvl_heads* views[] = {q, a->Hk ? k : nullptr, q_out, a->Hk ? k_out : nullptr};
  Shape s{};
  if (!shape_of(a, widest(a, views, 4), &s))
    return fail(PVL_ERR_UNSUPPORTED, "%s: a token of %d heads of %d features does not fit a block", who, p.Ht, p.D);
  fill(p, a, s);
  p.x[0] = *q;
  p.out[0] = *q_out;
  if (a->Hk) {
    p.x[1] = *k;
    p.out[1] = *k_out;
  }
  int grid = 0;
  return launch<false>(p, s, a->norm, 1 << 30, &grid, reinterpret_cast<cudaStream_t>(stream), who);
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
  if (st == PVL_OK) st = check_views(who, a, dq, 0, "dq");
  if (st == PVL_OK) st = check_views(who, a, dk, 1, "dk");
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
  const pvl_heads* views[] = {dq_out, a->Hk ? dk_out : nullptr, dq, a->Hk ? dk : nullptr, norm ? q : nullptr,
                              norm && a->Hk ? k : nullptr};
  Shape s{};
  if (!shape_of(a, widest(a, views, 6), &s))
    return fail(PVL_ERR_UNSUPPORTED, "%s: a token of %d heads of %d features does not fit a block", who, p.Ht, p.D);
  fill(p, a, s);
  p.g[0] = *dq_out;
  p.out[0] = *dq;
  if (a->Hk) {
    p.g[1] = *dk_out;
    p.out[1] = *dk;
  }
  if (norm) {
    p.x[0] = *q;
    if (a->Hk) p.x[1] = *k;
  }
  p.part = weights ? static_cast<float*>(ws) : nullptr;
  // a partial row for each team (norm per token) or block (norm per head)
  const int rows_per_block = a->norm == PVL_NORM_TOKEN ? s.teams : 1;
  const long long tokens = p.tokens;
  const long long rows_max = tokens < kMaxPartials ? tokens : kMaxPartials;
  int limit = weights ? static_cast<int>(rows_max / rows_per_block) : 1 << 30;
  if (limit < 1) limit = 1;
  if (weights && static_cast<long long>(rows_per_block) > rows_max) {
    // fewer tokens than teams: one block, and only the teams that the workspace has rows for
    p.teams = static_cast<int>(rows_max);
  }
  int grid = 0;
  cudaStream_t stm = reinterpret_cast<cudaStream_t>(stream);
  st = launch<true>(p, s, a->norm, limit, &grid, stm, who);
  if (st != PVL_OK || !weights) return st;
  const int q_width = a->norm == PVL_NORM_TOKEN ? a->H * a->D : a->D;
  const int rows = grid * (a->norm == PVL_NORM_TOKEN ? p.teams : 1);
  rotary_weights_kernel<<<(p.width + 31) / 32, 1024, 0, stm>>>(p.part, rows, p.width, q_width, dq_weight, dk_weight);
  return check_cuda(cudaGetLastError(), who);
}
