// adaln_residual_fwd / adaln_residual_bwd: the gated residual of a block and
// the norms on both sides of it, fused, for sm_103a.
//
// What it computes, per token n with modulation row s:
//   u = h, or post(h) w2          (post: RMS or layer norm of the block's output)
//   t = alpha x + gate_s u        (the residual stream after the block: x_out)
//   y = (xh w + b)(1 + scale_s) + shift_s,  xh = norm(t)   (the next block's input)
// and backward, from dt0 = d x_out, dy, x_out and h, with g = dy w (1 + scale_s):
//   t' = dt0 + r (g - [mean g] - xh mean(g xh)),  dx = alpha t',
//   dz = t' gate_s w2,  dh = dz, or rh (dz - [mean dz] - hh mean(dz hh)),
//   A_s = sum dy xh,  B_s = sum dy,  C_s = sum t' hh  over the tokens of row s:
//   dscale = w A + b B, dshift = B, dgate = w2 C,
//   dw = sum_s (1 + scale_s) A_s, db = sum_s (1 + scale_s) B_s, dw2 = sum_s gate_s C_s
// ([.] only for the layer norm; a token with id -1 is padding: x_out = x,
// y = 0, dx = d x_out, dh = 0).
//
// Design.  HBM bound: 8 bytes an element forward and 12 backward with a bf16
// stream, each touched once.
//   - Persistent CTAs walk contiguous row ranges.  One lane streams the rows of
//     every input into a ring of shared-memory stages with bulk copies; each
//     thread owns the same 8-wide feature groups of every row.  Padding rows
//     skip the copies of what they do not use (their ids are read one row
//     ahead, so that the test costs no latency).
//   - What bounds a row's time is its chain of waits and reductions, not its
//     arithmetic, so two schemes take the reductions off it: the forward
//     without a post norm overlaps the phases of neighbouring rows
//     (residual_fwd_kernel), the others have warps of their own for the
//     statistics (the warp roles below).
//   - Forward, the three tables of the current modulation row (gate w2,
//     w (1 + scale), b (1 + scale) + shift) stay in registers and are loaded
//     again where the id changes.  Backward the registers hold the sums A, B
//     and C of the current modulation row and two tables, which a small kernel
//     has prepared so that the statistics' warps can have them copied into
//     shared memory.
//   - A row's statistics are one-pass sums shifted by K, the median of the
//     row's first three elements; the RMS norm takes K = 0.  The variance's rounding
//     grows with (mean - K)^2 over the variance: a common offset of the row
//     cancels in it, and one outlier channel, as residual streams have them,
//     cannot be the median (taken for K itself it would make that ratio D - 1:
//     1 / deviation off by 2^-10 at 5120 features, 2^-20 without).
//   - The sums of a CTA's run of equal ids go to slot (CTA + id): with ids
//     that do not decrease along the rows no two runs share a slot, so the
//     partial sums need n_cta + S rows and no atomics on values; a small
//     kernel adds the slots of each id in CTA order (deterministic).  A slot
//     claimed twice (ids out of order) is detected, recorded as an error and
//     turns every table gradient into NaN.
// Roundings to fewer than 32 bits: x_out and dx to the stream's type, y and dh
// to bf16, each once and last.
//
// Measured (of 6770 GB/s, the card's copy rate): 64,000 x 5120, bf16, seven
// episodes: forward 400 us = 97 %, backward 587 us = 99 %; with an RMS post norm
// 410 and 898 us (94 %, 65 %: there the statistics' two passes over a row hold
// one of its four stages too long).  Four padded rows of 10,944 x 1536, fp32
// stream, RMS norms on both sides, 1152 modulation rows: 138 and 228 us (86 %,
// 74 %, of which 31 us are the tables and the sums of the modulation rows).
// Every wait is bounded, as in the other kernels.
#include <cuda_runtime.h>

#include <algorithm>

#include "pvl_device.cuh"

namespace pvl {
namespace {

constexpr int kMaxStages = 8;
constexpr int kMaxWarps = 32;
constexpr int kMaxCtas = 1216;  // CTAs per launch at most (bounds the partial-sum slots)
constexpr int kMaxD = 8192;

enum ResidualSite : uint32_t { kSiteResRowFull = 51, kSiteModId = 52, kSiteModOrder = 53, kSiteResReady = 54, kSiteResEmpty = 55,
                                kSiteResTable = 56 };

// What the block adds: nothing (h absent), h, or post(h).
enum Branch : int { kNoBranch = 0, kPlain = 1, kPost = 2 };

struct ResidualParams {
  const void* x;                // forward x, backward x_out (TX)
  const __nv_bfloat16* h;       // null: not read
  const float *gate, *shift, *scale;  // [S, D] or null
  const float *w, *b, *w2;            // [D] or null
  const int32_t* ids;           // null: row / N
  void* x_out;                  // forward (TX)
  __nv_bfloat16* y;             // forward
  const void* dxo;              // backward (TX), null: zeros
  const __nv_bfloat16* dy;      // backward
  void* dx;                     // backward (TX)
  __nv_bfloat16* dh;            // backward
  float* part;                  // backward: [3][n_slots][D], null: no table or vector gradients
  unsigned int* lo;             // backward: first CTA of each id [S]
  int* hi;                      // backward: last CTA of each id [S]
  int* tag;                     // backward: id whose sums a slot holds [n_slots]
  int* ordered;                 // backward: -1 until ids are found out of order
  DeviceError* err;
  int N, D, S;
  bool one_row;                 // no [S, D] table: every valid id stands for row 0
  bool rms, post_rms;
  long long rows, rows_per_cta;
  int n_slots;
  int stages;
  const int* valid;             // backward: valid rows of each of kSegments row segments, null: rows split evenly
  int seg_rows, pad_weight;     // rows of a segment; cost of a padding row in sixteenths of a valid one
  int stats_warps, tables;      // backward: warps for the rows' statistics, table slots in shared memory
  const float *factors, *gates; // backward: w (1 + scale) and gate w2 as [S, D]
  float alpha, eps;
  uint64_t timeout_ns;
};

__device__ __forceinline__ void note_error(DeviceError* e, uint32_t code, uint32_t where) {
  if (atomicCAS(&e->code, 0u, code) == 0u) {
    e->where = where;
    e->block = blockIdx.x;
    e->thread = threadIdx.x;
  }
}

// CTA-wide sums of kN values in two halves around a barrier that the caller
// has anyway.  warp_part: in a warp the values are reduce-scattered (each
// halving step sends half of what remains), lane group lane / (32 / kN) ends
// with one value, and one lane of each stores it in red.  all_parts, after the
// barrier: every warp adds the table, the same bits in every thread.  red
// holds kMaxWarps * kN floats.
template <int kN>
__device__ __forceinline__ void warp_part(float (&a)[kN], float* red) {
  const int lane = threadIdx.x & 31;
  int o = 16;
#pragma unroll
  for (int n = kN; n > 1; n >>= 1, o >>= 1) {
    const bool hi = lane & o;
#pragma unroll
    for (int j = 0; j < n / 2; ++j) {
      const float keep = hi ? a[j + n / 2] : a[j];
      const float send = hi ? a[j] : a[j + n / 2];
      a[j] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
#pragma unroll
  for (int q = 16 / kN; q >= 1; q >>= 1) a[0] += __shfl_xor_sync(0xffffffffu, a[0], q);
  constexpr int kGroup = 32 / kN;
  if ((lane & (kGroup - 1)) == 0) red[(threadIdx.x >> 5) * kN + lane / kGroup] = a[0];
}
template <int kN>
__device__ __forceinline__ void all_parts(float (&a)[kN], const float* red, int nwarps) {
  const int lane = threadIdx.x & 31;
  float t = 0.0f;
  for (int i = lane; i < nwarps * kN; i += 32) t += red[i];
#pragma unroll
  for (int q = kN; q < 32; q <<= 1) t += __shfl_xor_sync(0xffffffffu, t, q);
#pragma unroll
  for (int q = 0; q < kN; ++q) a[q] = __shfl_sync(0xffffffffu, t, q);
}

__device__ __forceinline__ void unpack8(const uint4 u, float2 (&f)[4]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}

// A thread's unit of work is a group of 8 features, v of nvec.  kSplit says
// which: with a bf16 stream features 8 v .. 8 v + 7, one 16-byte vector; with
// an fp32 stream the quads v and nvec + v of the row, so that every fp32
// access of a warp covers 512 contiguous bytes (8 adjacent floats a lane
// would be two accesses at a stride of 32 bytes, each a two-way bank conflict
// in shared memory).
template <bool kSplit>
__device__ __forceinline__ void row8(const __nv_bfloat16* row, int v, int nvec, float2 (&f)[4]) {
  if (kSplit) {
    const uint2 a = reinterpret_cast<const uint2*>(row)[v], c = reinterpret_cast<const uint2*>(row)[nvec + v];
    unpack8(make_uint4(a.x, a.y, c.x, c.y), f);
  } else {
    unpack8(reinterpret_cast<const uint4*>(row)[v], f);
  }
}
template <bool kSplit>
__device__ __forceinline__ void row8(const float* row, int v, int nvec, float2 (&f)[4]) {
  const float4 a = reinterpret_cast<const float4*>(row)[kSplit ? v : 2 * v];
  const float4 c = reinterpret_cast<const float4*>(row)[kSplit ? nvec + v : 2 * v + 1];
  f[0] = make_float2(a.x, a.y);
  f[1] = make_float2(a.z, a.w);
  f[2] = make_float2(c.x, c.y);
  f[3] = make_float2(c.z, c.w);
}
template <bool kSplit>
__device__ __forceinline__ void store8(__nv_bfloat16* row, int v, int nvec, const float2 (&f)[4]) {
  const uint4 u = make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y), pack_bf16x2(f[2].x, f[2].y),
                             pack_bf16x2(f[3].x, f[3].y));
  if (kSplit) {
    reinterpret_cast<uint2*>(row)[v] = make_uint2(u.x, u.y);
    reinterpret_cast<uint2*>(row)[nvec + v] = make_uint2(u.z, u.w);
  } else {
    reinterpret_cast<uint4*>(row)[v] = u;
  }
}
template <bool kSplit>
__device__ __forceinline__ void store8(float* row, int v, int nvec, const float2 (&f)[4]) {
  reinterpret_cast<float4*>(row)[kSplit ? v : 2 * v] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
  reinterpret_cast<float4*>(row)[kSplit ? nvec + v : 2 * v + 1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
}
// a group of a table's row or of a vector in global memory, or `fill` where it is absent
template <bool kSplit>
__device__ __forceinline__ void table8(const float* row, int v, int nvec, float fill, float2 (&f)[4]) {
  if (row == nullptr) {
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = make_float2(fill, fill);
    return;
  }
  const float4 a = __ldg(reinterpret_cast<const float4*>(row) + (kSplit ? v : 2 * v));
  const float4 c = __ldg(reinterpret_cast<const float4*>(row) + (kSplit ? nvec + v : 2 * v + 1));
  f[0] = make_float2(a.x, a.y);
  f[1] = make_float2(a.z, a.w);
  f[2] = make_float2(c.x, c.y);
  f[3] = make_float2(c.z, c.w);
}
__device__ __forceinline__ const float* at_row(const float* table, int id, int D) {
  return table ? table + static_cast<size_t>(id) * D : nullptr;
}
// The elements that a row's shift K is taken from, its first three (one load),
// and their median.
struct Sample {
  float v[3];
};
__device__ __forceinline__ Sample sample(const __nv_bfloat16* row) {
  const uint2 u = *reinterpret_cast<const uint2*>(row);
  return Sample{{__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16)}};
}
__device__ __forceinline__ Sample sample(const float* row) {
  const float4 u = *reinterpret_cast<const float4*>(row);
  return Sample{{u.x, u.y, u.z}};
}
__device__ __forceinline__ float median(const Sample& s) {
  return fmaxf(fminf(s.v[0], s.v[1]), fminf(fmaxf(s.v[0], s.v[1]), s.v[2]));
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
// 1 / deviation; a variance that rounding has left below zero is zero, a NaN
// of the row's (fmaxf would drop it) makes the row NaN
__device__ __forceinline__ float inv_deviation(float var, float eps) { return rsqrtf((var < 0.0f ? 0.0f : var) + eps); }

// gate w2 of a modulation row: the factor of the (normalised) block output
template <bool kSplit>
__device__ __forceinline__ void gate8(const ResidualParams& p, int id, int v, int nvec, float2 (&f)[4]) {
  float2 q[4];
  table8<kSplit>(at_row(p.gate, id, p.D), v, nvec, 1.0f, f);
  if (p.w2) {
    table8<kSplit>(p.w2, v, nvec, 1.0f, q);
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = fmul2(f[e], q[e]);
  }
}
// w (1 + scale) of a modulation row: the factor of xh
template <bool kSplit>
__device__ __forceinline__ void factor8(const ResidualParams& p, int id, int v, int nvec, float2 (&f)[4]) {
  float2 q[4];
  table8<kSplit>(at_row(p.scale, id, p.D), v, nvec, 0.0f, f);
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] = fadd2(f[e], both(1.0f));
  if (p.w) {
    table8<kSplit>(p.w, v, nvec, 1.0f, q);
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = fmul2(f[e], q[e]);
  }
}

// The forward's tables of a modulation row: gate w2, w (1 + scale) and
// b (1 + scale) + shift.
template <bool kSplit>
__device__ __forceinline__ void load_tables(const ResidualParams& p, int id, int v, int nvec, float2 (&gt)[4],
                                            float2 (&fa)[4], float2 (&ad)[4]) {
  gate8<kSplit>(p, id, v, nvec, gt);
  factor8<kSplit>(p, id, v, nvec, fa);
  table8<kSplit>(at_row(p.shift, id, p.D), v, nvec, 0.0f, ad);
  if (p.b) {
    float2 q[4], sc[4];
    table8<kSplit>(p.b, v, nvec, 0.0f, q);
    table8<kSplit>(at_row(p.scale, id, p.D), v, nvec, 0.0f, sc);
#pragma unroll
    for (int e = 0; e < 4; ++e) ad[e] = fadd2(ad[e], ffma2(q[e], sc[e], q[e]));
  }
}

__host__ __device__ constexpr size_t align128(size_t n) { return (n + 127) / 128 * 128; }

// Stage layout: x (TX), h, and backward dy, dxo (TX); each part 128-byte aligned.
template <typename TX, bool kBwd>
struct Stage {
  size_t x_bytes, h_bytes;
  __host__ __device__ explicit Stage(int D) : x_bytes(align128(sizeof(TX) * D)), h_bytes(align128(2 * D)) {}
  __host__ __device__ size_t h() const { return x_bytes; }
  __host__ __device__ size_t dy() const { return x_bytes + h_bytes; }
  __host__ __device__ size_t dxo() const { return x_bytes + 2 * h_bytes; }
  __host__ __device__ size_t bytes() const { return kBwd ? 2 * x_bytes + 2 * h_bytes : x_bytes + h_bytes; }
};

// mbar_wait behind some tests without suspension: a suspended thread takes
// longer to wake than the waits of a well-fed pipeline last (64,000 x 5120:
// forward 419 -> 401 us, backward 595 -> 587).  Not for the kernels with a post
// norm, whose statistics warps need the issue slots (900 us, 927 with tests).
__device__ __forceinline__ bool test_wait(uint64_t* bar, uint32_t parity, const KernelCtl& ctl, uint32_t where) {
#pragma unroll 1
  for (int i = 0; i < 30; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
  }
  return mbar_wait(bar, parity, ctl, where);
}

// Thread 0's view of the CTA's row stream: which row to copy next, the id of
// that row (read one row ahead), and what has been issued.
template <typename TX, bool kBwd>
struct Producer {
  const ResidualParams& p;
  uint8_t* smem;
  uint64_t* full;
  int* ids_s;
  long long next, end;
  int32_t next_id;
  uint32_t issued;
  int st;

  __device__ Producer(const ResidualParams& q, uint8_t* sm, uint64_t* f, int* is, long long begin, long long e)
      : p(q), smem(sm), full(f), ids_s(is), next(begin), end(e), next_id(0), issued(0), st(0) {
    if (next < end) next_id = id_of(next);
  }
  __device__ int32_t id_of(long long r) const { return p.ids ? __ldg(p.ids + r) : static_cast<int32_t>(r / p.N); }
  // modulation row of the next row to issue, -1 for padding
  __device__ int32_t peek() const {
    if (next_id < 0) return -1;
    if (p.one_row) return 0;
    if (next_id < p.S) return next_id;
    note_error(p.err, kDevErrModId, kSiteModId);
    return -1;
  }
  __device__ void issue() {
    if (next >= end) return;
    const Stage<TX, kBwd> lay(p.D);
    const long long r = next++;
    const int32_t id = peek();
    if (next < end) next_id = id_of(next);
    ids_s[st] = id;
    uint8_t* dst = smem + st * lay.bytes();
    const uint32_t xb = sizeof(TX) * p.D, hb = 2 * p.D;
    const bool live = id >= 0;
    uint32_t bytes = 0;
    const bool want_x = !kBwd || live, want_h = p.h && live, want_dy = kBwd && live, want_dxo = kBwd && p.dxo;
    bytes += (want_x ? xb : 0) + (want_h ? hb : 0) + (want_dy ? hb : 0) + (want_dxo ? xb : 0);
    mbar_arrive_expect_tx(&full[st], bytes);
    if (want_x) bulk_load(dst, static_cast<const TX*>(p.x) + r * p.D, xb, &full[st]);
    if (want_h) bulk_load(dst + lay.h(), p.h + r * p.D, hb, &full[st]);
    if (want_dy) bulk_load(dst + lay.dy(), p.dy + r * p.D, hb, &full[st]);
    if (want_dxo) bulk_load(dst + lay.dxo(), static_cast<const TX*>(p.dxo) + r * p.D, xb, &full[st]);
    ++issued;
    if (++st == p.stages) st = 0;
  }
};

// Shared state of the forward below.
struct Shared {
  uint64_t full[kMaxStages];
  int ids[kMaxStages];
  float red[2][kMaxWarps * 2];
  int abort;
};

// A row between its two phases: which, its stage, its id, and the mean and
// 1 / deviation of x_out.
struct Flight {
  bool on;
  int row, st, id;
  float m, r;
};

// Forward without a post norm.  Every row has two phases: the first writes
// x_out and sums what the statistics need, the second writes y.  One iteration
// of the loop runs the second phase of a row and the first of the next and has
// one barrier, which makes the sums visible and frees the finished row's
// stage: no phase waits for a reduction of its own row (496 us at 64,000 x
// 5120 with a row at a time, 405 so).
template <typename TX, int kV, int kRegs, int kBranch>
__global__ void __maxnreg__(kRegs) residual_fwd_kernel(const ResidualParams p) {
  constexpr bool kSplit = sizeof(TX) == 4;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Shared sh;
  const Stage<TX, false> lay(p.D);
  const int D = p.D, nvec = D / 8, t = threadIdx.x, nthr = blockDim.x, nwarps = nthr / 32;
  const float inv_d = 1.0f / static_cast<float>(D);
  const KernelCtl ctl{p.err, &sh.abort, p.timeout_ns};
  const int r_begin = static_cast<int>(blockIdx.x * p.rows_per_cta);
  const int r_end = static_cast<int>(min(blockIdx.x * p.rows_per_cta + p.rows_per_cta, p.rows));
  if (t < kMaxStages) sh.ids[t] = -1;
  if (t == 0) {
    sh.abort = 0;
    for (int s = 0; s < p.stages; ++s) mbar_init(&sh.full[s], 1);
    fence_barrier_init();
  }
  __syncthreads();
  Producer<TX, false> prod(p, smem, sh.full, sh.ids, r_begin, t == 0 ? r_end : r_begin);
  if (t == 0)
    for (int s = 0; s < p.stages; ++s) prod.issue();

  float2 gt[kV][4], fa[kV][4], ad[kV][4];  // gate, w (1 + scale), b (1 + scale) + shift of row cur
  Sample g0{};                             // gate of the features that K is taken from
  int cur = -1;
  // the residual's 8 features of group v, from the stage
  auto residual8 = [&](const uint8_t* src, int i, int v, float2 (&f)[4]) {
    row8<kSplit>(reinterpret_cast<const TX*>(src), v, nvec, f);
    if (kBranch != kNoBranch) {
      float2 q[4];
      row8<kSplit>(reinterpret_cast<const __nv_bfloat16*>(src + lay.h()), v, nvec, q);
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = ffma2(q[e], gt[i][e], fmul2(f[e], both(p.alpha)));
    }
  };
  // what the row's sums are shifted by
  auto shift_of = [&](const uint8_t* src) {
    if (p.rms) return 0.0f;
    Sample x = sample(reinterpret_cast<const TX*>(src));
    if (kBranch != kNoBranch) {
      const Sample h = sample(reinterpret_cast<const __nv_bfloat16*>(src + lay.h()));
#pragma unroll
      for (int j = 0; j < 3; ++j) x.v[j] = fmaf(h.v[j], g0.v[j], p.alpha * x.v[j]);
    }
    return median(x);
  };

  Flight b{};
  int next = r_begin, st = 0, turn = 0;
  uint32_t ph = 0, freed = 0;
  while (next < r_end || b.on) {
    if (b.on) {  // y
      const uint8_t* src = smem + b.st * lay.bytes();
      __nv_bfloat16* out = p.y + static_cast<size_t>(b.row) * D;
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        const int v = t + i * nthr;
        if (v < nvec) {
          float2 f[4];
          if (b.id < 0) {
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = both(0.0f);
          } else {
            residual8(src, i, v, f);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = ffma2(fmul2(fadd2(f[e], both(-b.m)), both(b.r)), fa[i][e], ad[i][e]);
          }
          store8<kSplit>(out, v, nvec, f);
        }
      }
    }
    float2 s1 = both(0.0f), s2 = both(0.0f);
    Flight a{};
    float K = 0.0f;
    bool ok = true;
    if (next < r_end) {
      ok = test_wait(&sh.full[st], ph, ctl, kSiteResRowFull);
      const int id = sh.ids[st];
      a = Flight{true, next, st, id, 0.0f, 0.0f};
      if (id >= 0 && id != cur) {  // the row before is done with its tables
        cur = id;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
          const int v = t + i * nthr;
          if (v < nvec) load_tables<kSplit>(p, id, v, nvec, gt[i], fa[i], ad[i]);
        }
        if (kBranch != kNoBranch) g0 = p.gate ? sample(p.gate + static_cast<size_t>(id) * D) : Sample{{1.0f, 1.0f, 1.0f}};
      }
      const uint8_t* src = smem + st * lay.bytes();
      TX* out = static_cast<TX*>(p.x_out) + static_cast<size_t>(next) * D;
      if (id >= 0) K = shift_of(src);
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        const int v = t + i * nthr;
        if (v < nvec) {
          float2 q[4];
          if (id < 0) {
            if (kBranch != kNoBranch) {
              row8<kSplit>(reinterpret_cast<const TX*>(src), v, nvec, q);
              store8<kSplit>(out, v, nvec, q);
            }
          } else {
            residual8(src, i, v, q);
            if (kBranch != kNoBranch) store8<kSplit>(out, v, nvec, q);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              q[e] = fadd2(q[e], both(-K));
              s1 = fadd2(s1, q[e]);
              s2 = ffma2(q[e], q[e], s2);
            }
          }
        }
      }
    }
    float sums[2] = {s1.x + s1.y, s2.x + s2.y};
    warp_part<2>(sums, sh.red[turn]);
    if (!__syncthreads_and(ok)) break;
    all_parts<2>(sums, sh.red[turn], nwarps);
    turn ^= 1;
    if (b.on) {
      ++freed;
      if (t == 0) prod.issue();
    }
    const float m1 = p.rms ? 0.0f : sums[0] * inv_d;
    a.m = K + m1;
    a.r = inv_deviation(fmaf(-m1, m1, sums[1] * inv_d), p.eps);
    b = a;
    if (a.on) {
      ++next;
      if (++st == p.stages) {
        st = 0;
        ph ^= 1u;
      }
    }
  }
  // copies still in flight land before the CTA leaves
  __syncthreads();
  if (t == 0)
    for (uint32_t n = freed; n < prod.issued; ++n) mbar_drain(&sh.full[n % p.stages], (n / p.stages) & 1, 100000000ull);
  __syncthreads();
}

// ------------------------------------------------------------- warp roles
// The backward, and the forward with a post norm.  One warp's lane streams
// the rows (and, where the modulation row changes, the tables that statistics
// need) into shared memory.  p.stats_warps warps take whole rows in turn: a
// row's statistics are sums of one warp, so they need shuffles but no barrier,
// and sums that need earlier ones (a post norm's) simply follow them.  The
// other warps own feature groups: they wait for a row's statistics and write
// its results.  Nothing is CTA-wide; the roles meet at the stages' mbarriers
// only (full: copies landed; ready: statistics written; empty: every group
// warp done).
struct RowStats {
  float m, r;    // mean and 1 / deviation of x_out
  float c0, c1;  // backward: mean g, mean g xh
  float hm, hr;  // mean and 1 / deviation of the branch
  float z0, z1;  // backward: dh's means, -rh mean dz and -rh^3 mean dz (h - hm)
};

constexpr int kMaxTables = 2;
constexpr int kSegments = 512;  // a multiple of 128: a lane reads its part as int4

struct RoleShared {
  uint64_t full[kMaxStages], ready[kMaxStages], empty[kMaxStages], table[kMaxTables], w2;
  RowStats stats[kMaxStages];
  int ids[kMaxStages];
  int slot[kMaxStages];  // of the row's tables: slot, and the parity of its load in bit 8
  int range[2];
  int abort;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float total(float2 v) { return warp_sum(v.x + v.y); }
// A wait of a whole warp: the same answer in every lane.
template <bool kTest>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const KernelCtl& ctl, uint32_t where) {
  return __all_sync(0xffffffffu, kTest ? test_wait(bar, parity, ctl, where) : mbar_wait(bar, parity, ctl, where));
}

__device__ __forceinline__ void init_roles(const ResidualParams& p, RoleShared& sh, int group_warps) {
  sh.abort = 0;
  for (int s = 0; s < p.stages; ++s) {
    mbar_init(&sh.full[s], 1);
    mbar_init(&sh.ready[s], 1);
    mbar_init(&sh.empty[s], group_warps);
  }
  for (int s = 0; s < p.tables; ++s) mbar_init(&sh.table[s], 1);
  mbar_init(&sh.w2, 1);
  fence_barrier_init();
}

// The copying lane: rows [r_begin, r_begin + rows) into the ring, the rows of
// the tables t0 and t1 (null: none) of each new modulation row into the next
// table slot.
template <typename TX, bool kBwd>
__device__ __forceinline__ void stream_rows(const ResidualParams& p, RoleShared& sh, uint8_t* tables,
                                            uint32_t table_bytes, uint8_t* ring, const float* t0, const float* t1,
                                            int r_begin, int rows, const KernelCtl& ctl) {
  const int D = p.D, S = p.stages;
  Producer<TX, kBwd> prod(p, ring, sh.full, sh.ids, r_begin, r_begin + rows);
  int st = 0, slot = p.tables - 1, held = -1;  // held: the id whose tables the slot has
  uint32_t ph = 1;                             // parity of the stage's last empty phase, from the second round on
  uint32_t loads = 0;                          // table loads so far
  int last[kMaxTables];                        // the last row that uses each slot
#pragma unroll
  for (int i = 0; i < kMaxTables; ++i) last[i] = -1;
  for (int n = 0; n < rows; ++n) {
    if (n >= S && !mbar_wait(&sh.empty[st], ph, ctl, kSiteResEmpty)) break;
    const int id = prod.peek();
    if (p.tables && id >= 0 && id != held) {
      held = id;
      slot = slot + 1 == p.tables ? 0 : slot + 1;
      // every row that used the slot must have its statistics: those of
      // the last S - 1 rows are waited for one by one (different warps
      // take them, in no order), older ones have left their stages
      const int end = slot == 0 ? last[0] : last[1];
      bool free = true;
      for (int row = max(0, n - S + 1); row <= end && free; ++row)
        free = mbar_wait(&sh.ready[row % S], (row / S) & 1, ctl, kSiteResTable);
      if (!free) break;
      uint8_t* dst = tables + slot * table_bytes;
      mbar_arrive_expect_tx(&sh.table[slot], 4 * D * ((t0 ? 1 : 0) + (t1 ? 1 : 0)));
      if (t0) bulk_load(dst, t0 + static_cast<size_t>(id) * D, 4 * D, &sh.table[slot]);
      if (t1) bulk_load(dst + (t0 ? align128(4 * static_cast<size_t>(D)) : 0), t1 + static_cast<size_t>(id) * D, 4 * D,
                        &sh.table[slot]);
      ++loads;
    }
    if (id >= 0) (slot == 0 ? last[0] : last[1]) = n;
    sh.slot[st] = slot | (p.tables ? static_cast<int>(((loads - 1) / p.tables) & 1) << 8 : 0);
    prod.issue();
    if (++st == S) {
      st = 0;
      ph ^= 1u;
    }
  }
  // copies still in flight land before the CTA leaves
  for (int n = max(0, static_cast<int>(prod.issued) - S); n < static_cast<int>(prod.issued); ++n)
    mbar_drain(&sh.full[n % S], (n / S) & 1, 100000000ull);
  for (uint32_t n = loads > static_cast<uint32_t>(p.tables) ? loads - p.tables : 0; n < loads; ++n)
    mbar_drain(&sh.table[n % p.tables], (n / p.tables) & 1, 100000000ull);
}

// The forward with a post norm: statistics of the branch, then of the
// residual, need the row twice in order, which the phases of the kernel above
// would spread over three iterations (64,000 x 5120: 719 us there).
template <typename TX, int kV, int kRegs>
__global__ void __maxnreg__(kRegs) residual_post_fwd_kernel(const ResidualParams p) {
  constexpr bool kSplit = sizeof(TX) == 4;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ RoleShared sh;
  const Stage<TX, false> lay(p.D);
  const int D = p.D, nvec = D / 8, S = p.stages;
  // shared memory: w2 (if there is one), the gate's slots, the rows' stages
  const uint32_t table_bytes = align128(4 * static_cast<size_t>(D));
  uint8_t* const slots = smem + (p.w2 ? table_bytes : 0);
  uint8_t* const ring = slots + p.tables * table_bytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group_warps = blockDim.x / 32 - 1 - p.stats_warps;
  const float inv_d = 1.0f / static_cast<float>(D);
  const KernelCtl ctl{p.err, &sh.abort, p.timeout_ns};
  const int r_begin = static_cast<int>(blockIdx.x * p.rows_per_cta);
  const int rows = static_cast<int>(min(p.rows_per_cta, p.rows - blockIdx.x * p.rows_per_cta));
  if (threadIdx.x == 0) init_roles(p, sh, group_warps);
  __syncthreads();

  if (warp < group_warps) {
    const int t = threadIdx.x, nthr = group_warps * 32;
    float2 gt[kV][4], fa[kV][4], ad[kV][4];  // gate w2, w (1 + scale), b (1 + scale) + shift of row cur
    int cur = -1, st = 0;
    uint32_t ph = 0;
    for (int n = 0; n < rows; ++n) {
      if (!warp_wait<false>(&sh.ready[st], ph, ctl, kSiteResReady)) break;
      if (!warp_wait<false>(&sh.full[st], ph, ctl, kSiteResRowFull)) break;
      const uint8_t* src = ring + st * lay.bytes();
      const TX* xs = reinterpret_cast<const TX*>(src);
      const __nv_bfloat16* hs = reinterpret_cast<const __nv_bfloat16*>(src + lay.h());
      TX* xo = static_cast<TX*>(p.x_out) + static_cast<size_t>(r_begin + n) * D;
      __nv_bfloat16* yo = p.y + static_cast<size_t>(r_begin + n) * D;
      const int id = sh.ids[st];
      if (id < 0) {
#pragma unroll
        for (int i = 0; i < kV; ++i) {
          const int v = t + i * nthr;
          if (v < nvec) {
            float2 f[4];
            row8<kSplit>(xs, v, nvec, f);
            store8<kSplit>(xo, v, nvec, f);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = both(0.0f);
            store8<kSplit>(yo, v, nvec, f);
          }
        }
      } else {
        if (id != cur) {
          cur = id;
#pragma unroll
          for (int i = 0; i < kV; ++i) {
            const int v = t + i * nthr;
            if (v < nvec) load_tables<kSplit>(p, id, v, nvec, gt[i], fa[i], ad[i]);
          }
        }
        const RowStats q = sh.stats[st];
        const float2 hr = both(q.hr), hsub = both(-q.hm), rs = both(q.r), sub = both(-q.m), al = both(p.alpha);
#pragma unroll
        for (int i = 0; i < kV; ++i) {
          const int v = t + i * nthr;
          if (v < nvec) {
            float2 f[4], g[4];
            row8<kSplit>(xs, v, nvec, f);
            row8<kSplit>(hs, v, nvec, g);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = ffma2(fmul2(fadd2(g[e], hsub), hr), gt[i][e], fmul2(f[e], al));
            store8<kSplit>(xo, v, nvec, f);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = ffma2(fmul2(fadd2(f[e], sub), rs), fa[i][e], ad[i][e]);
            store8<kSplit>(yo, v, nvec, f);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.empty[st]);
      if (++st == S) {
        st = 0;
        ph ^= 1u;
      }
    }
  } else if (warp < group_warps + p.stats_warps) {
    // a warp keeps to its stages, so that it sees every phase of their barriers
    int st = 0;
    uint32_t ph = 0;
    auto step = [&]() {
      if (++st == S) {
        st = 0;
        ph ^= 1u;
      }
    };
    bool alive = !p.w2 || warp_wait<false>(&sh.w2, 0, ctl, kSiteResTable);
    const float* w2 = reinterpret_cast<const float*>(smem);
    for (int n = 0; n < rows && alive; ++n, step()) {
      if (st % p.stats_warps != warp - group_warps) continue;
      if (!warp_wait<false>(&sh.full[st], ph, ctl, kSiteResRowFull)) break;
      const uint8_t* src = ring + st * lay.bytes();
      const TX* xs = reinterpret_cast<const TX*>(src);
      const __nv_bfloat16* hs = reinterpret_cast<const __nv_bfloat16*>(src + lay.h());
      if (sh.ids[st] >= 0) {
        const int slot = sh.slot[st];
        if (p.tables && !warp_wait<false>(&sh.table[slot & 255], slot >> 8, ctl, kSiteResTable)) break;
        const float* gate = reinterpret_cast<const float*>(slots + (slot & 255) * table_bytes);
        RowStats q{};
        const float Kh = p.post_rms ? 0.0f : median(sample(hs));
        float2 s1 = both(0.0f), s2 = both(0.0f);
#pragma unroll 3
        for (int v = lane; v < nvec; v += 32) {
          float2 f[4];
          row8<true>(hs, v, nvec, f);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            f[e] = fadd2(f[e], both(-Kh));
            s1 = fadd2(s1, f[e]);
            s2 = ffma2(f[e], f[e], s2);
          }
        }
        const float hm1 = p.post_rms ? 0.0f : total(s1) * inv_d;
        q.hr = inv_deviation(fmaf(-hm1, hm1, total(s2) * inv_d), p.eps);
        q.hm = Kh + hm1;
        // the residual's difference from its K
        float K = 0.0f;
        if (!p.rms) {
          Sample x = sample(xs);
          const Sample h = sample(hs), one{{1.0f, 1.0f, 1.0f}};
          const Sample g = p.tables ? sample(gate) : one, w = p.w2 ? sample(w2) : one;
#pragma unroll
          for (int j = 0; j < 3; ++j) x.v[j] = fmaf((h.v[j] - q.hm) * q.hr, g.v[j] * w.v[j], p.alpha * x.v[j]);
          K = median(x);
        }
        const float2 hr = both(q.hr), hsub = both(-q.hm), al = both(p.alpha);
        s1 = s2 = both(0.0f);
#pragma unroll 3
        for (int v = lane; v < nvec; v += 32) {
          float2 f[4], g[4], m[4];
          row8<true>(xs, v, nvec, f);
          row8<true>(hs, v, nvec, g);
#pragma unroll
          for (int e = 0; e < 4; ++e) g[e] = fmul2(fadd2(g[e], hsub), hr);
          if (p.w2) {
            row8<true>(w2, v, nvec, m);
#pragma unroll
            for (int e = 0; e < 4; ++e) g[e] = fmul2(g[e], m[e]);
          }
          if (p.tables) {
            row8<true>(gate, v, nvec, m);
#pragma unroll
            for (int e = 0; e < 4; ++e) g[e] = fmul2(g[e], m[e]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            f[e] = fadd2(ffma2(f[e], al, g[e]), both(-K));
            s1 = fadd2(s1, f[e]);
            s2 = ffma2(f[e], f[e], s2);
          }
        }
        const float m1 = p.rms ? 0.0f : total(s1) * inv_d;
        q.r = inv_deviation(fmaf(-m1, m1, total(s2) * inv_d), p.eps);
        q.m = K + m1;
        if (lane == 0) sh.stats[st] = q;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.ready[st]);
    }
  } else if (lane == 0) {
    if (p.w2) {
      mbar_arrive_expect_tx(&sh.w2, 4 * D);
      bulk_load(smem, p.w2, 4 * D, &sh.w2);
    }
    stream_rows<TX, false>(p, sh, slots, table_bytes, ring, p.gate, nullptr, r_begin, rows, ctl);
    if (p.w2) mbar_drain(&sh.w2, 0, 100000000ull);
  }
  __syncthreads();
}

// --------------------------------------------------------------- backward
// Rows of a CTA where padding is cheaper than valid rows: with segment s's
// cost w_s = pad rows + (16 - pad) valid rows and P_s the cost before it, the
// k-th boundary is the row at cost k T / n_cta of the total T, taken as evenly
// spread within a segment.  One warp; every CTA computes the same boundaries.
// (In four padded episodes with a fifth of the rows padding at half the cost,
// the CTAs of valid rows would end 10 % after the mean.)
__device__ void split_rows(const ResidualParams& p, int lane, int* range) {
  constexpr int kPer = kSegments / 32;
  int w[kPer];
  long long sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; i += 4) {
    const int4 v = __ldg(reinterpret_cast<const int4*>(p.valid + lane * kPer + i));
    w[i] = v.x;
    w[i + 1] = v.y;
    w[i + 2] = v.z;
    w[i + 3] = v.w;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const long long first = static_cast<long long>(lane * kPer + i) * p.seg_rows;
    const long long len = max(0ll, min(static_cast<long long>(p.seg_rows), p.rows - first));
    w[i] = static_cast<int>(len) * p.pad_weight + w[i] * (16 - p.pad_weight);
    sum += w[i];
  }
  long long before = sum;  // inclusive, then exclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += v;
  }
  const long long all = __shfl_sync(0xffffffffu, before, 31);
  before -= sum;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const long long want = (static_cast<long long>(blockIdx.x) + k) * all / gridDim.x;
    if (want >= all) {
      if (lane == 0) range[k] = static_cast<int>(p.rows);
    } else if (want >= before && want < before + sum) {
      long long at = before;
      bool found = false;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (!found && want < at + w[i]) {
          const long long first = static_cast<long long>(lane * kPer + i) * p.seg_rows;
          const long long len = min(static_cast<long long>(p.seg_rows), p.rows - first);
          range[k] = static_cast<int>(first + (want - at) * len / w[i]);
          found = true;
        }
        at += w[i];
      }
    }
  }
}

template <typename TX, int kV, int kRegs, int kBranch>
__global__ void __maxnreg__(kRegs) residual_bwd_kernel(const ResidualParams p) {
  constexpr bool kSplit = sizeof(TX) == 4;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ RoleShared sh;
  const Stage<TX, true> lay(p.D);
  const int D = p.D, nvec = D / 8, S = p.stages;
  const uint32_t table_bytes = align128(4 * static_cast<size_t>(D)) * (kBranch == kPost ? 2 : 1);
  uint8_t* const ring = smem + p.tables * table_bytes;  // the rows' stages, behind the tables
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group_warps = blockDim.x / 32 - 1 - p.stats_warps;
  const float inv_d = 1.0f / static_cast<float>(D);
  const KernelCtl ctl{p.err, &sh.abort, p.timeout_ns};
  if (p.valid && warp == 1) split_rows(p, lane, sh.range);
  if (threadIdx.x == 0) {
    init_roles(p, sh, group_warps);
    if (!p.valid) {
      sh.range[0] = static_cast<int>(blockIdx.x * p.rows_per_cta);
      sh.range[1] = static_cast<int>(min(blockIdx.x * p.rows_per_cta + p.rows_per_cta, p.rows));
    }
  }
  __syncthreads();
  const int r_begin = sh.range[0], rows = sh.range[1] - r_begin;

  if (warp < group_warps) {
    const int t = threadIdx.x, nthr = group_warps * 32;
    float2 gt[kV][4], fa[kV][4];             // gate w2 and w (1 + scale) of modulation row cur
    float2 aa[kV][4], ab[kV][4], ac[kV][4];  // its sums A, B and C
    int cur = -1;
    // the run's sums go to slot (CTA + id)
    auto flush = [&]() {
      if (cur < 0 || p.part == nullptr) return;
      const int slot = static_cast<int>(blockIdx.x) + cur;
      if (t == 0) {
        if (atomicExch(&p.tag[slot], cur) != -1) {
          *p.ordered = 0;
          note_error(p.err, kDevErrModOrder, kSiteModOrder);
        }
        atomicMin(&p.lo[cur], blockIdx.x);
        atomicMax(&p.hi[cur], static_cast<int>(blockIdx.x));
      }
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        const int v = t + i * nthr;
        if (v < nvec) {
          float* q = p.part + static_cast<size_t>(slot) * D;
          const size_t next = static_cast<size_t>(p.n_slots) * D;
          store8<kSplit>(q, v, nvec, aa[i]);
          store8<kSplit>(q + next, v, nvec, ab[i]);
          if (kBranch != kNoBranch) store8<kSplit>(q + 2 * next, v, nvec, ac[i]);
        }
      }
    };
    int st = 0;
    uint32_t ph = 0;
    for (int n = 0; n < rows; ++n) {
      if (!warp_wait<kBranch != kPost>(&sh.ready[st], ph, ctl, kSiteResReady)) break;
      if (!warp_wait<kBranch != kPost>(&sh.full[st], ph, ctl, kSiteResRowFull)) break;
      const uint8_t* src = ring + st * lay.bytes();
      const TX* xs = reinterpret_cast<const TX*>(src);
      const __nv_bfloat16* hs = reinterpret_cast<const __nv_bfloat16*>(src + lay.h());
      const __nv_bfloat16* ys = reinterpret_cast<const __nv_bfloat16*>(src + lay.dy());
      const TX* us = reinterpret_cast<const TX*>(src + lay.dxo());
      TX* dxo = static_cast<TX*>(p.dx) + static_cast<size_t>(r_begin + n) * D;
      __nv_bfloat16* dho = kBranch == kNoBranch ? nullptr : p.dh + static_cast<size_t>(r_begin + n) * D;
      const int id = sh.ids[st];
      if (id < 0) {
#pragma unroll
        for (int i = 0; i < kV; ++i) {
          const int v = t + i * nthr;
          if (v < nvec) {
            float2 f[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = both(0.0f);
            if (kBranch != kNoBranch) store8<kSplit>(dho, v, nvec, f);
            if (p.dxo) row8<kSplit>(us, v, nvec, f);
            store8<kSplit>(dxo, v, nvec, f);
          }
        }
      } else {
        if (id != cur) {
          flush();
          cur = id;
#pragma unroll
          for (int i = 0; i < kV; ++i) {
            const int v = t + i * nthr;
            if (v < nvec) {
              if (kBranch != kNoBranch) table8<true>(at_row(p.gates, id, D), v, nvec, 1.0f, gt[i]);
              table8<true>(at_row(p.factors, id, D), v, nvec, 1.0f, fa[i]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) aa[i][e] = ab[i][e] = ac[i][e] = both(0.0f);
          }
        }
        const RowStats q = sh.stats[st];
        const float2 ca = both(-q.r * q.c1), cc = both(-q.r * q.c0), rs = both(q.r), sub = both(-q.m);
#pragma unroll
        for (int i = 0; i < kV; ++i) {
          const int v = t + i * nthr;
          if (v < nvec) {
            float2 f[4], g[4];
            row8<kSplit>(xs, v, nvec, f);
            row8<kSplit>(ys, v, nvec, g);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              f[e] = fmul2(fadd2(f[e], sub), rs);  // xh
              aa[i][e] = ffma2(g[e], f[e], aa[i][e]);
              ab[i][e] = fadd2(ab[i][e], g[e]);
              f[e] = ffma2(fmul2(g[e], fa[i][e]), rs, ffma2(f[e], ca, cc));
            }
            if (p.dxo) {
              row8<kSplit>(us, v, nvec, g);
#pragma unroll
              for (int e = 0; e < 4; ++e) f[e] = fadd2(f[e], g[e]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) g[e] = fmul2(f[e], both(p.alpha));
            store8<kSplit>(dxo, v, nvec, g);
            if (kBranch == kPost) {
              row8<kSplit>(hs, v, nvec, g);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                g[e] = fadd2(g[e], both(-q.hm));
                ac[i][e] = ffma2(f[e], fmul2(g[e], both(q.hr)), ac[i][e]);
                f[e] = ffma2(fmul2(f[e], gt[i][e]), both(q.hr), ffma2(g[e], both(q.z1), both(q.z0)));
              }
              store8<kSplit>(dho, v, nvec, f);
            } else if (kBranch == kPlain) {
              if (p.h) {
                row8<kSplit>(hs, v, nvec, g);
#pragma unroll
                for (int e = 0; e < 4; ++e) ac[i][e] = ffma2(f[e], g[e], ac[i][e]);
              }
#pragma unroll
              for (int e = 0; e < 4; ++e) f[e] = fmul2(f[e], gt[i][e]);
              store8<kSplit>(dho, v, nvec, f);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.empty[st]);
      if (++st == S) {
        st = 0;
        ph ^= 1u;
      }
    }
    flush();
  } else if (warp < group_warps + p.stats_warps) {
    // a warp keeps to its stages, so that it sees every phase of their barriers
    int st = 0;
    uint32_t ph = 0;
    auto step = [&]() {
      if (++st == S) {
        st = 0;
        ph ^= 1u;
      }
    };
    for (int n = 0; n < rows; ++n, step()) {
      if (st % p.stats_warps != warp - group_warps) continue;
      if (!warp_wait<kBranch != kPost>(&sh.full[st], ph, ctl, kSiteResRowFull)) break;
      const uint8_t* src = ring + st * lay.bytes();
      const TX* xs = reinterpret_cast<const TX*>(src);
      const __nv_bfloat16* hs = reinterpret_cast<const __nv_bfloat16*>(src + lay.h());
      const __nv_bfloat16* ys = reinterpret_cast<const __nv_bfloat16*>(src + lay.dy());
      const TX* us = reinterpret_cast<const TX*>(src + lay.dxo());
      const int id = sh.ids[st];
      if (id >= 0) {
        // sums of d = x_out - K, d^2, g = dy w (1 + scale) and g d; with a
        // post norm also those of the branch
        RowStats q{};
        q.hr = 1.0f;
        const float K = p.rms ? 0.0f : median(sample(xs));
        const float Kh = kBranch == kPost && !p.post_rms ? median(sample(hs)) : 0.0f;
        const int slot = sh.slot[st];
        if (p.tables && !warp_wait<kBranch != kPost>(&sh.table[slot & 255], slot >> 8, ctl, kSiteResTable)) break;
        const float* fac = reinterpret_cast<const float*>(smem + (slot & 255) * table_bytes);
        const float* gat = fac + align128(4 * static_cast<size_t>(D)) / 4;
        if (kRegs == 96 && p.tables == 0) {  // rows so wide that no table fits beside them: from L2
          fac = p.factors + static_cast<size_t>(id) * D;
          gat = p.gates + static_cast<size_t>(id) * D;
        }
        float2 s1 = both(0.0f), s2 = both(0.0f), sg = both(0.0f), sgd = both(0.0f), h1 = both(0.0f), h2 = both(0.0f);
#pragma unroll 2
        for (int v = lane; v < nvec; v += 32) {
          float2 f[4], g[4], m[4];
          row8<true>(fac, v, nvec, m);
          row8<kSplit>(xs, v, nvec, f);
          row8<kSplit>(ys, v, nvec, g);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            f[e] = fadd2(f[e], both(-K));
            g[e] = fmul2(g[e], m[e]);
            s1 = fadd2(s1, f[e]);
            s2 = ffma2(f[e], f[e], s2);
            sg = fadd2(sg, g[e]);
            sgd = ffma2(g[e], f[e], sgd);
          }
          if (kBranch == kPost) {
            row8<kSplit>(hs, v, nvec, f);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              f[e] = fadd2(f[e], both(-Kh));
              h1 = fadd2(h1, f[e]);
              h2 = ffma2(f[e], f[e], h2);
            }
          }
        }
        const float m1 = p.rms ? 0.0f : total(s1) * inv_d;
        q.r = inv_deviation(fmaf(-m1, m1, total(s2) * inv_d), p.eps);
        q.m = K + m1;
        const float sum_g = total(sg);
        q.c0 = p.rms ? 0.0f : sum_g * inv_d;
        q.c1 = q.r * fmaf(-m1, sum_g, total(sgd)) * inv_d;
        if (kBranch == kPost) {
          const float hm1 = p.post_rms ? 0.0f : total(h1) * inv_d;
          q.hr = inv_deviation(fmaf(-hm1, hm1, total(h2) * inv_d), p.eps);
          q.hm = Kh + hm1;
          // dz = t' gate w2: its sum, and that of dz (h - hm)
          const float2 ca = both(-q.r * q.c1), cc = both(-q.r * q.c0), rs = both(q.r), sub = both(-q.m);
          float2 z1 = both(0.0f), z2 = both(0.0f);
#pragma unroll 2
          for (int v = lane; v < nvec; v += 32) {
            float2 f[4], g[4], m[4];
            row8<true>(fac, v, nvec, m);
            row8<kSplit>(xs, v, nvec, f);
            row8<kSplit>(ys, v, nvec, g);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              f[e] = ffma2(fmul2(g[e], m[e]), rs, ffma2(fmul2(fadd2(f[e], sub), rs), ca, cc));
            if (p.dxo) {
              row8<kSplit>(us, v, nvec, g);
#pragma unroll
              for (int e = 0; e < 4; ++e) f[e] = fadd2(f[e], g[e]);
            }
            row8<true>(gat, v, nvec, m);
            row8<kSplit>(hs, v, nvec, g);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              f[e] = fmul2(f[e], m[e]);
              z1 = fadd2(z1, f[e]);
              z2 = ffma2(f[e], fadd2(g[e], both(-q.hm)), z2);
            }
          }
          q.z0 = p.post_rms ? 0.0f : -q.hr * total(z1) * inv_d;
          q.z1 = -q.hr * q.hr * q.hr * total(z2) * inv_d;
        }
        if (lane == 0) sh.stats[st] = q;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.ready[st]);
    }
  } else if (lane == 0) {
    stream_rows<TX, true>(p, sh, smem, table_bytes, ring, p.factors, kBranch == kPost ? p.gates : nullptr, r_begin, rows,
                          ctl);
  }
  __syncthreads();
}

// The backward's tables w (1 + scale) and gate w2 as [S, D], and its control
// words (all ones).  A row's quads stand in the order in which the kernel
// reads them: the first quads of all groups, then the second ones.
template <bool kSplit>
__global__ void __launch_bounds__(256) residual_tables_kernel(const ResidualParams p, float* factors, float* gates,
                                                              int* ints, size_t n_ints, int* valid,
                                                              int count_blocks) {
  if (blockIdx.x < count_blocks) {
    // valid rows of one segment
    __shared__ int part[8];
    const long long first = static_cast<long long>(blockIdx.x) * p.seg_rows;
    const long long end = min(first + p.seg_rows, p.rows);
    int n = 0;
    for (long long r = first + threadIdx.x; r < end; r += 256) {
      const int id = __ldg(p.ids + r);
      n += id >= 0 && (p.one_row || id < p.S);
    }
    n = __reduce_add_sync(0xffffffffu, n);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = n;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 1; i < 8; ++i) n += part[i];
      valid[blockIdx.x] = n;
    }
    return;
  }
  const size_t i = static_cast<size_t>(blockIdx.x - count_blocks) * 256 + threadIdx.x;
  if (i < n_ints) ints[i] = -1;
  const int per = p.D / 8;
  if (i >= static_cast<size_t>(p.S) * per) return;
  const int id = static_cast<int>(i / per), v = static_cast<int>(i - static_cast<size_t>(id) * per);
  float2 f[4];
  factor8<kSplit>(p, id, v, per, f);
  store8<true>(factors + static_cast<size_t>(id) * p.D, v, per, f);
  if (gates) {
    gate8<kSplit>(p, id, v, per, f);
    store8<true>(gates + static_cast<size_t>(id) * p.D, v, per, f);
  }
}

// Sums A, B and C of each modulation row from the slots of the CTAs lo..hi
// that met it.  A CTA takes one id and 4 kLanes features: lane l the float4 at
// feature 4 l, thread row g of G the CTAs lo + g, lo + g + G, ...; the thread
// rows' sums are then added in order.  Many ids with a CTA or two each take 32
// lanes and as many thread rows as an id has CTAs; few ids with hundreds each
// take 8 lanes and 32 thread rows (one id, 900 CTAs: one warp a 128 features
// took 60 us).  Writes the table gradients, and the plain sums to `tot`
// ([3][S][D]) where vector gradients follow.
struct FinalParams {
  const float* part;
  const unsigned int* lo;
  const int* hi;
  const int* tag;
  const int* ordered;
  const float *gate, *scale, *w, *b, *w2;
  float *dgate, *dshift, *dscale, *dw, *db, *dw2;
  float* tot;
  int D, S, n_slots;
  bool branch;
};
constexpr int kFinRows = 32;

__device__ __forceinline__ float4 add4(float4 a, float4 b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}
__device__ __forceinline__ float4 fma4(float4 a, float4 b, float4 c) {
  return make_float4(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y), fmaf(a.z, b.z, c.z), fmaf(a.w, b.w, c.w));
}
__device__ __forceinline__ float4 vec4(const float* p, int d, float fill) {
  return p ? __ldg(reinterpret_cast<const float4*>(p + d)) : make_float4(fill, fill, fill, fill);
}

template <int kLanes>
__global__ void __launch_bounds__(256) residual_rows_kernel(const FinalParams p) {
  __shared__ float4 acc[256 / kLanes][3][kLanes];
  const int lane = threadIdx.x, g = threadIdx.y, G = blockDim.y;
  const int s = blockIdx.x;
  const int d = (blockIdx.y * kLanes + lane) * 4;
  const int c0 = static_cast<int>(__ldg(p.lo + s)), c1 = __ldg(p.hi + s);  // none: lo = 0xffffffff, hi = -1
  const int ordered = __ldg(p.ordered);
  const int sums = p.branch ? 3 : 2;
  float4 a[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) a[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (d < p.D && c1 >= 0) {
#pragma unroll 4
    for (int c = c0 + g; c <= c1; c += G) {
      const int slot = c + s, tag = __ldg(p.tag + slot);
      float4 v[3];
#pragma unroll
      for (int k = 0; k < 3; ++k)
        if (k < sums)
          v[k] = __ldg(reinterpret_cast<const float4*>(p.part + (static_cast<size_t>(k) * p.n_slots + slot) * p.D + d));
      // a slot that is not this id's: a CTA of padding between two that met it
#pragma unroll
      for (int k = 0; k < 3; ++k)
        if (k < sums && tag == s) a[k] = add4(a[k], v[k]);
    }
  }
  if (G > 1) {
#pragma unroll
    for (int k = 0; k < 3; ++k) acc[g][k][lane] = a[k];
    __syncthreads();
    if (g > 0) return;
    for (int i = 1; i < G; ++i)
#pragma unroll
      for (int k = 0; k < 3; ++k) a[k] = add4(a[k], acc[i][k][lane]);
  }
  if (d >= p.D) return;
  if (ordered != -1) {
    const float nan = __int_as_float(0x7fffffff);
#pragma unroll
    for (int k = 0; k < 3; ++k) a[k] = make_float4(nan, nan, nan, nan);
  }
  const size_t at = static_cast<size_t>(s) * p.D + d;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  const float* vectors[3] = {p.w, p.b, p.w2};
#pragma unroll
  for (int k = 0; k < 3; ++k)
    if (vectors[k]) *reinterpret_cast<float4*>(p.tot + static_cast<size_t>(k) * p.S * p.D + at) = a[k];
  if (p.dshift) *reinterpret_cast<float4*>(p.dshift + at) = a[1];
  if (p.dscale) {
    float4 o = fma4(a[0], vec4(p.w, d, 1.0f), zero);
    if (p.b) o = fma4(a[1], vec4(p.b, d, 0.0f), o);
    *reinterpret_cast<float4*>(p.dscale + at) = o;
  }
  if (p.dgate) *reinterpret_cast<float4*>(p.dgate + at) = fma4(a[2], vec4(p.w2, d, 1.0f), zero);
}

// dw, db, dw2 = sums over the modulation rows of factor times A, B, C.  A CTA
// takes 16 features of one vector (blockIdx.y): lane group of 4 the float4s of
// one row, 64 rows at a time; then the 64 sums in a fixed tree.
__global__ void __launch_bounds__(256) residual_vectors_kernel(const FinalParams p) {
  __shared__ float4 acc[64][4];
  const int k = blockIdx.y;
  float* out = k == 0 ? p.dw : k == 1 ? p.db : p.dw2;
  if (!out) return;
  const float* table = k == 2 ? p.gate : p.scale;
  const float one = k == 2 && p.gate ? 0.0f : 1.0f;  // 1 + scale, gate, or 1
  const int lane = threadIdx.x & 3, g = threadIdx.x >> 2;
  const int d = blockIdx.x * 16 + lane * 4;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (d < p.D) {
    const float* tot = p.tot + static_cast<size_t>(k) * p.S * p.D + d;
#pragma unroll 8
    for (int s = g; s < p.S; s += 64) {
      const size_t at = static_cast<size_t>(s) * p.D;
      const float4 f = table ? __ldg(reinterpret_cast<const float4*>(table + at + d)) : make_float4(0.f, 0.f, 0.f, 0.f);
      a = fma4(add4(f, make_float4(one, one, one, one)), __ldg(reinterpret_cast<const float4*>(tot + at)), a);
    }
  }
  acc[g][lane] = a;
#pragma unroll
  for (int n = 32; n; n >>= 1) {
    __syncthreads();
    if (g < n) acc[g][lane] = add4(acc[g][lane], acc[g + n][lane]);
  }
  if (g == 0 && d < p.D) *reinterpret_cast<float4*>(out + d) = acc[0][lane];
}

// Launch shape: threads cover the row's 8-wide groups, kV each, in whole
// warps; as many CTAs per SM as registers and two stages each allow.  kRoles:
// the kernels with warp roles have their statistics and copying warps besides.
template <typename TX, int kV, int kRegs, int kBranch, bool kBwd>
pvl_status launch_rows(ResidualParams p, cudaStream_t s, const char* who) {
  constexpr bool kRoles = kBwd || kBranch == kPost;
  void (*fn)(ResidualParams);
  if constexpr (kBwd) fn = &residual_bwd_kernel<TX, kV, kRegs, kBranch>;
  else if constexpr (kRoles) fn = &residual_post_fwd_kernel<TX, kV, kRegs>;
  else fn = &residual_fwd_kernel<TX, kV, kRegs, kBranch>;
  int threads = ((p.D / 8 + kV - 1) / kV + 31) / 32 * 32;
  if (kRoles) {
    // registers are a quarter of the SM's per scheduler, warps whole
    constexpr int kMostWarps = 4 * (512 / kRegs);
    // four statistics warps where a row needs two passes of theirs; two where
    // one does, or where two more would cost a CTA of few warps its neighbour;
    // half as many for short rows, where the group warps are what a CTA lacks:
    // forward by the bytes that a row has them read (64,000 rows, bf16 stream:
    // 1024 features 137 us, four warps 152; 1536 157, 169; fp32 stream, four rows
    // of 10,944: 1024 96, 108; 1280 125, 119; 1536 152, 138)
    const bool narrow = kBwd ? kBranch != kPost && threads <= 64
                             : (sizeof(TX) + 2) * static_cast<size_t>(p.D) <= 6144;
    int stats = kBranch == kPost && (!kBwd || threads >= 160) ? 4 : 2;
    if (narrow) stats /= 2;
    p.stats_warps = std::min(stats, kMostWarps - threads / 32 - 1);
    threads += 32 * (p.stats_warps + 1);
  }
  const int stage_bytes = static_cast<int>(Stage<TX, kBwd>(p.D).bytes());
  const int sms = sm_count(), smem_sm = smem_per_sm();
  int occ = blocks_per_sm(reinterpret_cast<const void*>(fn), threads, 0);
  if (sms <= 0 || smem_sm <= 0 || occ <= 0) return fail(PVL_ERR_CUDA, "%s: no usable CUDA device", who);
  // per CTA: the system's share, the static shared memory, and what is kept of the tables
  const int row_bytes = static_cast<int>(align128(4 * p.D));
  const int reserve = 1024 + static_cast<int>(align128(kRoles ? sizeof(RoleShared) : sizeof(Shared)));
  const int fixed = kRoles && !kBwd && p.w2 ? row_bytes : 0;
  const int table_bytes = row_bytes * (kBwd && kBranch == kPost ? 2 : 1);
  const bool tables = kBwd || (kRoles && p.gate);
  int stages = 0;
  for (; occ >= 1; --occ) {
    const int room = smem_sm / occ - reserve - fixed;
    // two table slots where they leave five stages, else one
    p.tables = tables ? 2 : 0;
    stages = (room - p.tables * table_bytes) / stage_bytes;
    if (tables && stages < 5) {
      p.tables = 1;
      stages = (room - table_bytes) / stage_bytes;
    }
    if (kBwd && kRegs == 96 && stages < 2 && occ == 1) {
      p.tables = 0;
      stages = room / stage_bytes;
    }
    if (stages >= 2) break;
  }
  if (occ < 1) return fail(PVL_ERR_UNSUPPORTED, "%s: D = %d does not fit in shared memory", who, p.D);
  p.stages = stages < kMaxStages ? stages : kMaxStages;
  long long grid = static_cast<long long>(occ) * sms;
  if (kBwd && grid > kMaxCtas) grid = kMaxCtas;
  if (grid > p.rows) grid = p.rows;
  p.rows_per_cta = (p.rows + grid - 1) / grid;
  grid = (p.rows + p.rows_per_cta - 1) / p.rows_per_cta;
  if (p.stages > p.rows_per_cta) p.stages = p.rows_per_cta < 2 ? 2 : static_cast<int>(p.rows_per_cta);
  // each statistics warp has stages of its own; one too many works on groups
  if (p.stats_warps > p.stages) p.stats_warps = p.stages;
  const int smem = p.stages * stage_bytes + p.tables * table_bytes + fixed;
  // the exact size, so that the kernel is allowed it
  if (blocks_per_sm(reinterpret_cast<const void*>(fn), threads, smem) <= 0)
    return fail(PVL_ERR_CUDA, "%s: no usable CUDA device", who);
  fn<<<static_cast<unsigned>(grid), threads, smem, s>>>(p);
  return check_cuda(cudaGetLastError(), who);
}

// Groups a thread and registers.  Three groups a thread need the fewest
// warps, whose work on a row beyond its features (waits, statistics) is then
// paid least often; short rows take one (64k x 1024 backward: 247 us against
// 297), rows past 6912 features, whose nine warps of three groups leave no room for
// the others, two backward.
template <typename TX, int kBranch, bool kBwd>
pvl_status pick_width(const ResidualParams& p, cudaStream_t s, const char* who) {
  if constexpr (!kBwd) {
    if (p.D < 512) return launch_rows<TX, 1, 80, kBranch, kBwd>(p, s, who);
    return launch_rows<TX, 3, 128, kBranch, kBwd>(p, s, who);
  } else {
    if (p.D > 6912) return launch_rows<TX, 2, 96, kBranch, kBwd>(p, s, who);
    if (p.D >= 1536) return launch_rows<TX, 3, 168, kBranch, kBwd>(p, s, who);
    return launch_rows<TX, 1, 80, kBranch, kBwd>(p, s, who);
  }
}

template <bool kBwd>
pvl_status dispatch(const ResidualParams& p, bool fp32, int branch, cudaStream_t s, const char* who) {
  if (fp32) {
    if (branch == kPost) return pick_width<float, kPost, kBwd>(p, s, who);
    if (branch == kPlain) return pick_width<float, kPlain, kBwd>(p, s, who);
    return pick_width<float, kNoBranch, kBwd>(p, s, who);
  }
  if (branch == kPost) return pick_width<__nv_bfloat16, kPost, kBwd>(p, s, who);
  if (branch == kPlain) return pick_width<__nv_bfloat16, kPlain, kBwd>(p, s, who);
  return pick_width<__nv_bfloat16, kNoBranch, kBwd>(p, s, who);
}

// The checks both directions share; fills the parameters they have in common.
pvl_status common(const char* who, const pvl_residual* a, ResidualParams& p, int* branch) {
  if (!a) return fail(PVL_ERR_INVALID_ARG, "%s: null description", who);
  if (a->B < 1 || a->N < 1 || a->D < 1) return fail(PVL_ERR_INVALID_ARG, "%s: B, N and D must be >= 1", who);
  if (!(a->eps >= 0.0f) || !(a->eps < 1e30f))
    return fail(PVL_ERR_INVALID_ARG, "%s: eps must be >= 0 and finite", who);
  if (!(a->alpha > -1e30f && a->alpha < 1e30f)) return fail(PVL_ERR_INVALID_ARG, "%s: alpha must be finite", who);
  if (a->stream_dtype != PVL_BF16 && a->stream_dtype != PVL_F32)
    return fail(PVL_ERR_INVALID_ARG, "%s: stream_dtype %d", who, a->stream_dtype);
  if (a->norm != PVL_NORM_LAYER && a->norm != PVL_NORM_RMS)
    return fail(PVL_ERR_INVALID_ARG, "%s: norm %d (layer or RMS)", who, a->norm);
  if (a->post_norm != PVL_NORM_NONE && a->post_norm != PVL_NORM_LAYER && a->post_norm != PVL_NORM_RMS)
    return fail(PVL_ERR_INVALID_ARG, "%s: post_norm %d", who, a->post_norm);
  if (a->post_weight && a->post_norm == PVL_NORM_NONE)
    return fail(PVL_ERR_INVALID_ARG, "%s: post_weight without a post norm", who);
  if (a->D % 8 != 0 || a->D > kMaxD)
    return fail(PVL_ERR_UNSUPPORTED, "%s: D = %d (supported: multiples of 8 up to %d)", who, a->D, kMaxD);
  const long long rows = static_cast<long long>(a->B) * a->N;
  if (rows >= (1ll << 31) || rows * a->D >= (1ll << 40)) return fail(PVL_ERR_UNSUPPORTED, "%s: tensor too large", who);
  const bool tables = a->gate || a->shift || a->scale;
  if (tables && (a->S < 1 || a->S > PVL_MAX_MOD_ROWS))
    return fail(a->S < 1 ? PVL_ERR_INVALID_ARG : PVL_ERR_UNSUPPORTED, "%s: %d modulation rows (1 to %d)", who, a->S,
                PVL_MAX_MOD_ROWS);
  if (tables && !a->mod_id && a->S != a->B)
    return fail(PVL_ERR_INVALID_ARG, "%s: without mod_id the tables need B = %d rows, not %d", who, a->B, a->S);
  const void* ptrs[] = {a->gate, a->shift, a->scale, a->weight, a->bias, a->post_weight};
  for (const void* q : ptrs)
    if (reinterpret_cast<uintptr_t>(q) % 16 != 0)
      return fail(PVL_ERR_UNSUPPORTED, "%s: a table or vector is not 16-byte aligned", who);
  if (reinterpret_cast<uintptr_t>(a->mod_id) % 4 != 0)
    return fail(PVL_ERR_UNSUPPORTED, "%s: mod_id is not 4-byte aligned", who);
  p.gate = a->gate;
  p.shift = a->shift;
  p.scale = a->scale;
  p.w = a->weight;
  p.b = a->bias;
  p.w2 = a->post_weight;
  p.ids = a->mod_id;
  p.N = a->N;
  p.D = a->D;
  p.one_row = !tables;
  p.S = tables ? a->S : 1;
  p.rms = a->norm == PVL_NORM_RMS;
  p.post_rms = a->post_norm == PVL_NORM_RMS;
  p.rows = rows;
  p.alpha = a->alpha;
  p.eps = a->eps;
  p.timeout_ns = kDefaultTimeoutNs;
  *branch = a->post_norm != PVL_NORM_NONE ? kPost : kPlain;
  return PVL_OK;
}

pvl_status aligned(const char* who, const void* const* ptrs, int n) {
  for (int i = 0; i < n; ++i)
    if (reinterpret_cast<uintptr_t>(ptrs[i]) % 16 != 0)
      return fail(PVL_ERR_UNSUPPORTED, "%s: pointer argument %d is not 16-byte aligned", who, i);
  return PVL_OK;
}

// Workspace of the backward: the slots' sums [3][n_slots][D], the totals
// [3][S][D], the tables [2][S][D], the segments' valid rows, then the integers lo [S], hi [S], tag
// [n_slots], ordered.
struct WsLayout {
  size_t tot, tables, valid, ints, total;
  int n_slots;
  size_t n_ints;
};
WsLayout ws_layout(long long rows, int S, int D) {
  WsLayout w{};
  w.n_slots = static_cast<int>(rows < kMaxCtas ? rows : kMaxCtas) + S - 1;
  w.tot = align256(3ull * w.n_slots * D * sizeof(float));
  w.tables = w.tot + align256(3ull * S * D * sizeof(float));
  w.valid = w.tables + align256(2ull * S * D * sizeof(float));
  w.ints = w.valid + kSegments * sizeof(int);
  w.n_ints = 2ull * S + w.n_slots + 1;
  w.total = w.ints + align256(w.n_ints * sizeof(int));
  return w;
}

}  // namespace
}  // namespace pvl

using namespace pvl;

extern "C" pvl_status adaln_residual_fwd(const pvl_residual* a, const void* x, const pvl_bf16* h, void* x_out,
                                         pvl_bf16* y, pvl_stream_t stream) {
  const char* who = "adaln_residual_fwd";
  ResidualParams p{};
  int branch = 0;
  pvl_status st = common(who, a, p, &branch);
  if (st != PVL_OK) return st;
  if (!x || !y) return fail(PVL_ERR_INVALID_ARG, "%s: null pointer", who);
  if (!h) {
    if (a->gate || a->post_norm != PVL_NORM_NONE || a->alpha != 1.0f)
      return fail(PVL_ERR_INVALID_ARG, "%s: gate, post norm and alpha need a branch h", who);
    branch = kNoBranch;
  } else if (!x_out) {
    return fail(PVL_ERR_INVALID_ARG, "%s: null x_out", who);
  }
  const void* ptrs[] = {x, h, x_out, y};
  st = aligned(who, ptrs, 4);
  if (st != PVL_OK) return st;
  p.err = device_error_record();
  if (!p.err) return fail(PVL_ERR_CUDA, "%s: no usable CUDA device", who);
  p.x = x;
  p.h = reinterpret_cast<const __nv_bfloat16*>(h);
  p.x_out = x_out;
  p.y = reinterpret_cast<__nv_bfloat16*>(y);
  return dispatch<false>(p, a->stream_dtype == PVL_F32, branch, reinterpret_cast<cudaStream_t>(stream), who);
}

extern "C" size_t adaln_residual_bwd_ws_bytes(int B, int N, int D, int S) {
  if (B < 1 || N < 1 || D < 1 || S < 1) return 0;
  return ws_layout(static_cast<long long>(B) * N, S, D).total;
}

extern "C" pvl_status adaln_residual_bwd(const pvl_residual* a, const void* dx_out, const pvl_bf16* dy,
                                         const void* x_out, const pvl_bf16* h, int has_branch, void* dx, pvl_bf16* dh,
                                         const pvl_residual_grads* g, void* ws, size_t ws_bytes, pvl_stream_t stream) {
  const char* who = "adaln_residual_bwd";
  ResidualParams p{};
  int branch = 0;
  pvl_status st = common(who, a, p, &branch);
  if (st != PVL_OK) return st;
  if (!dy || !x_out || !dx || !g) return fail(PVL_ERR_INVALID_ARG, "%s: null pointer", who);
  if (!has_branch) {
    if (a->gate || a->post_norm != PVL_NORM_NONE || a->alpha != 1.0f)
      return fail(PVL_ERR_INVALID_ARG, "%s: gate, post norm and alpha need a branch h", who);
    branch = kNoBranch;
  } else if (!dh) {
    return fail(PVL_ERR_INVALID_ARG, "%s: null dh", who);
  }
  if (has_branch && !h && (a->gate || a->post_norm != PVL_NORM_NONE))
    return fail(PVL_ERR_INVALID_ARG, "%s: h is needed with a gate or a post norm", who);
  if ((!!g->dgate != !!a->gate) || (!!g->dshift != !!a->shift) || (!!g->dscale != !!a->scale) ||
      (!!g->dweight != !!a->weight) || (!!g->dbias != !!a->bias) || (!!g->dpost_weight != !!a->post_weight))
    return fail(PVL_ERR_INVALID_ARG, "%s: one gradient for each table and vector, and no others", who);
  const bool vectors = a->weight || a->bias || a->post_weight;
  const bool sums = a->gate || a->shift || a->scale || vectors;
  const void* ptrs[] = {dx_out, dy, x_out, h, dx, dh, g->dgate, g->dshift, g->dscale, g->dweight, g->dbias,
                        g->dpost_weight, ws};
  st = aligned(who, ptrs, 13);
  if (st != PVL_OK) return st;
  const WsLayout lay = ws_layout(p.rows, p.S, p.D);
  if (!ws || ws_bytes < lay.total)
    return fail(PVL_ERR_INVALID_ARG, "%s: workspace %zu bytes < %zu needed", who, ws ? ws_bytes : 0, lay.total);
  p.err = device_error_record();
  if (!p.err) return fail(PVL_ERR_CUDA, "%s: no usable CUDA device", who);
  p.x = x_out;
  // without a gate or a post norm nothing depends on h
  p.h = branch == kPost || a->gate ? reinterpret_cast<const __nv_bfloat16*>(h) : nullptr;
  p.dxo = dx_out;
  p.dy = reinterpret_cast<const __nv_bfloat16*>(dy);
  p.dx = dx;
  p.dh = reinterpret_cast<__nv_bfloat16*>(dh);
  p.n_slots = lay.n_slots;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  char* base = static_cast<char*>(ws);
  p.lo = reinterpret_cast<unsigned int*>(base + lay.ints);
  p.hi = reinterpret_cast<int*>(p.lo) + p.S;
  p.tag = p.hi + p.S;
  p.ordered = p.tag + lay.n_slots;
  p.part = sums ? static_cast<float*>(ws) : nullptr;
  float* tables = reinterpret_cast<float*>(base + lay.tables);
  p.factors = tables;
  p.gates = tables + static_cast<size_t>(p.S) * p.D;
  // padding is worth the splitting kernel's microsecond from some ten rows a CTA on
  const bool split = a->mod_id && p.rows >= 16 * kSegments;
  const int count_blocks = split ? kSegments : 0;
  int* valid = reinterpret_cast<int*>(base + lay.valid);
  p.valid = split ? valid : nullptr;
  p.seg_rows = static_cast<int>((p.rows + kSegments - 1) / kSegments);
  const int xb = a->stream_dtype == PVL_F32 ? 4 : 2;
  p.pad_weight = 16 * ((dx_out ? xb : 0) + xb + 2) / ((dx_out ? 3 : 2) * xb + (p.h ? 6 : 4));
  const size_t items = std::max(lay.n_ints, static_cast<size_t>(p.S) * (p.D / 8));
  (a->stream_dtype == PVL_F32 ? residual_tables_kernel<true> : residual_tables_kernel<false>)<<<
      static_cast<unsigned>(count_blocks + (items + 255) / 256), 256, 0, s>>>(
      p, tables, branch == kNoBranch ? nullptr : tables + static_cast<size_t>(p.S) * p.D,
      reinterpret_cast<int*>(p.lo), lay.n_ints, valid, count_blocks);
  st = check_cuda(cudaGetLastError(), who);
  if (st != PVL_OK) return st;
  st = dispatch<true>(p, a->stream_dtype == PVL_F32, branch, s, who);
  if (st != PVL_OK || !sums) return st;
  FinalParams f{};
  f.part = p.part;
  f.lo = p.lo;
  f.hi = p.hi;
  f.tag = p.tag;
  f.ordered = p.ordered;
  f.gate = a->gate;
  f.scale = a->scale;
  f.w = a->weight;
  f.b = a->bias;
  f.w2 = a->post_weight;
  f.dgate = g->dgate;
  f.dshift = g->dshift;
  f.dscale = g->dscale;
  f.dw = g->dweight;
  f.db = g->dbias;
  f.dw2 = g->dpost_weight;
  f.tot = vectors ? reinterpret_cast<float*>(base + lay.tot) : nullptr;
  f.D = p.D;
  f.S = p.S;
  f.n_slots = lay.n_slots;
  f.branch = branch != kNoBranch;
  // CTAs that an id meets on average
  const int per_id = 1 + (lay.n_slots - p.S) / p.S;
  if (per_id > 8)
    residual_rows_kernel<8><<<dim3(p.S, (p.D + 31) / 32), dim3(8, kFinRows), 0, s>>>(f);
  else
    residual_rows_kernel<32><<<dim3(p.S, (p.D + 127) / 128), dim3(32, per_id >= 4 ? 4 : per_id >= 2 ? 2 : 1), 0, s>>>(f);
  st = check_cuda(cudaGetLastError(), who);
  if (st != PVL_OK || !vectors) return st;
  residual_vectors_kernel<<<dim3((p.D + 15) / 16, 3), 256, 0, s>>>(f);
  return check_cuda(cudaGetLastError(), who);
}
