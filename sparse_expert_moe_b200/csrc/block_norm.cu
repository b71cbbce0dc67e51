// block_norm.cu -- the norms around a block, fused with its gate and residual scale, and
// their gradients (moe_block_norm, moe_block_norm_backward).
//
//   u = y i_y (w_post + o),  i_y = (mean y^2 + eps)^-1/2        (u = y without w_post)
//   r' = a r + b g u
//   h = r' i_r (w_pre + o),  i_r = (mean r'^2 + eps)^-1/2
// and backwards, with z = dh (w_pre + o) and G the whole gradient of r':
//   G  = dr' + i_r (z - r' i_r (i_r mean(z r')))    dr = a G       dw_pre  = sum_t dh r' i_r
//   q  = b g G (w_post + o)                                        dw_post = sum_t b g G y i_y
//   dy = i_y (q - y i_y (i_y mean(q y)))                           dgate   = sum b G u
// All arithmetic is fp32; each output is rounded once.  The backward pass recomputes both
// statistics from the rows it reads anyway, so the forward pass stores none.
//
// HBM-bound: every element of r and y is read once and of r' and h written once, held in
// registers between the (at most two) sums over a row.
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cmath>

#include "internal.h"
#include "ptx.cuh"

namespace moe {
namespace {

struct NormArgs {
  const void *r, *y, *w_post, *gate, *w_pre;
  void *r_out, *h;
  float* h_scale;
  int T, d, nvec;                 // nvec = d / 8
  int tpr, rows;                  // threads per row (a multiple of 32), rows per CTA
  int gate_kind;
  bool w_f32;
  int out;                        // moe_dtype of h
  float inv_d, eps, res_scale, branch_scale, w_offset;
};

// Eight consecutive elements as four pairs.
struct Vec8 {
  f32x2 p[4];
};
__device__ __forceinline__ Vec8 constant8(float v) {
  return Vec8{{both2(v), both2(v), both2(v), both2(v)}};
}
__device__ __forceinline__ Vec8 unpack_bf16(const uint4& a) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
  Vec8 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) f.p[i] = pack2(w[i] << 16, w[i] & 0xFFFF0000u);
  return f;
}
__device__ __forceinline__ Vec8 unpack_f32(const uint4& a, const uint4& b) {
  return Vec8{{pack2(a.x, a.y), pack2(a.z, a.w), pack2(b.x, b.y), pack2(b.z, b.w)}};
}
// Vector `v` (elements 8 v .. 8 v + 7) of a bf16 or fp32 array.
__device__ __forceinline__ Vec8 load8(const void* base, size_t v, bool f32) {
  const uint4* q = static_cast<const uint4*>(base);
  return f32 ? unpack_f32(q[2 * v], q[2 * v + 1]) : unpack_bf16(q[v]);
}
__device__ __forceinline__ void store8(void* base, size_t v, bool f32, const Vec8& f) {
  const float2 a = unpack2(f.p[0]), b = unpack2(f.p[1]), c = unpack2(f.p[2]), d = unpack2(f.p[3]);
  if (f32) {
    float4* o = static_cast<float4*>(base) + 2 * v;
    o[0] = make_float4(a.x, a.y, b.x, b.y);
    o[1] = make_float4(c.x, c.y, d.x, d.y);
  } else {
    uint4 q;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&q);
    h[0] = __floats2bfloat162_rn(a.x, a.y);
    h[1] = __floats2bfloat162_rn(b.x, b.y);
    h[2] = __floats2bfloat162_rn(c.x, c.y);
    h[3] = __floats2bfloat162_rn(d.x, d.y);
    static_cast<uint4*>(base)[v] = q;
  }
}

__device__ __forceinline__ float load1(const void* base, size_t i, bool f32) {
  return f32 ? static_cast<const float*>(base)[i]
             : __bfloat162float(static_cast<const __nv_bfloat16*>(base)[i]);
}

// load1 in two halves: the bits, wanted a turn later, and their value.
__device__ __forceinline__ uint32_t load1_bits(const void* base, size_t i, bool f32) {
  return f32 ? __ldg(static_cast<const uint32_t*>(base) + i) : __ldg(static_cast<const unsigned short*>(base) + i);
}
__device__ __forceinline__ float value1(uint32_t bits, bool f32) { return __uint_as_float(f32 ? bits : bits << 16); }

// Sums of N values over the threads of a row, the same in every thread of it and in the same
// order every time.  `part`: shared memory, 32 N floats, not touched since
// the __syncthreads before the call before last.  All threads of the CTA call this.
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* part, int tpr) {
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[j] += __shfl_xor_sync(0xffffffffu, v[j], o);
  const int warps = tpr >> 5;
  if (warps == 1) return;                      // (uniform over the CTA)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int first = warp / warps * warps;
  if (lane == 0)
#pragma unroll
    for (int j = 0; j < N; ++j) part[j * 32 + warp] = v[j];
  __syncthreads();
  if (warps <= 16) {                           // two values at a time, 16 lanes each
#pragma unroll
    for (int j = 0; j < N; j += 2) {
      const int at = j + (lane >> 4), w = lane & 15;
      float x = w < warps && at < N ? part[at * 32 + first + w] : 0.f;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      v[j] = __shfl_sync(0xffffffffu, x, 0);
      if (j + 1 < N) v[j + 1] = __shfl_sync(0xffffffffu, x, 16);
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      v[j] = lane < warps ? part[j * 32 + first + lane] : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v[j] += __shfl_xor_sync(0xffffffffu, v[j], o);
    }
  }
}

// Rows on their way in: each thread copies the vectors that it alone will read into its own
// places of shared memory with cp.async, kStages - 1 rows ahead of the one it finishes, so a CTA
// keeps rows in flight without holding them in registers and without a barrier (a thread waits for its own
// copies).  kStages = 0: rows are read from global memory directly (few rows per CTA).
template <int kStages>
__device__ __forceinline__ void rows_wait() {   // all but the newest kStages - 2 rows
  if (kStages) asm volatile("cp.async.wait_group %0;" ::"n"(kStages ? kStages - 2 : 0) : "memory");
}
__device__ __forceinline__ void rows_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Threads of a CTA whose rows are staged: with one CTA per SM they have 128 registers each, which
// hold two vectors per thread and array without spills (100 of them are used).
constexpr int kRowThreads = 512;

// One array's vectors of a thread in one stage: 16 or 32 bytes each, thread-interleaved, kPitch
// threads apart (a constant, so that the places are immediate offsets).
template <bool F32, int kPitch>
__device__ __forceinline__ void stage_in(uint4* st, int slot, const void* base, size_t v) {
  const uint4* g = static_cast<const uint4*>(base);
  if (F32) {
    cp_async_16_cg(st + (2 * slot) * kPitch, g + 2 * v);
    cp_async_16_cg(st + (2 * slot + 1) * kPitch, g + 2 * v + 1);
  } else {
    cp_async_16_cg(st + slot * kPitch, g + v);
  }
}
// Vector `slot` of this thread: from its stage, or (kPitch 0) straight from the array.
template <bool F32, int kPitch>
__device__ __forceinline__ Vec8 row8(const uint4* st, int slot, const void* base, size_t v) {
  if (!kPitch) return load8(base, v, F32);
  if (F32) return unpack_f32(st[2 * slot * kPitch], st[(2 * slot + 1) * kPitch]);
  return unpack_bf16(st[slot * kPitch]);
}

// Thread i of a row holds vectors i, i + tpr, ...; a CTA walks rows blockIdx.x * rows + row,
// + gridDim.x * rows, ...  What multiplies a channel in every row is fetched and combined once,
// into registers: c = branch_scale (w_post + o) (channel gate), and w_pre + o.
//
// Bound by HBM where rows are many.  Measured at T = 8192, d = 7168, bf16, post-norm, token gate
// and pre-norm (470 MB): 72 us alone, 78 in a run of cases back to back, 6.1-6.5 TB/s, 0.93-1.0 of the
// measured copy bandwidth; 21 instructions per element, issued in 48% of the cycles.  On the way there:
// one row per CTA, weights fetched per row 172 us (a row's loads and its two sums took turns); rows
// staged 134 us; packed arithmetic, the weights in registers, one barrier per row 96 us; no tests per
// vector, one CTA per SM without spills and the token gate's bits fetched a row ahead 74 us.  Launches
// that overlap: one token 4.0 -> 3.8 us.
//
// kAll (staged): a branch with its norm, no full gate, both outputs and no vectors past the row's
// end -- what a block normally has -- without the tests for it per vector.
template <bool RES32, bool ACT32, int VPT, int kStages, bool kAll = false>
__global__ void __launch_bounds__(kStages == 0 && VPT <= 2 ? 1024 : kRowThreads, 1)
    block_norm_kernel(const NormArgs p) {
  __shared__ float part[2][64];
  extern __shared__ uint4 ring[];
  constexpr bool kStaged = kStages > 0;
  constexpr int kRing = kStaged ? kStages : 1, kPitch = kStaged ? kRowThreads : 0;
  constexpr int kAtY = VPT * (RES32 ? 2 : 1), kAtGate = kAtY + VPT * (ACT32 ? 2 : 1);
  const int row = threadIdx.x / p.tpr, i0 = threadIdx.x - row * p.tpr;
  const int step = gridDim.x * p.rows;
  const bool full_gate = !kAll && p.gate_kind == MOE_GATE_FULL;
  const bool branch = kAll || p.y, post = kAll || p.w_post, pre = kAll || p.w_pre;
  const int stage_vecs = (branch ? kAtGate + (full_gate ? VPT * (ACT32 ? 2 : 1) : 0) : kAtY) * kPitch;
  auto fetch = [&](int t, int s) {
    if (t < p.T) {
      uint4* st = ring + s * stage_vecs + threadIdx.x;
      const size_t base = static_cast<size_t>(t) * p.nvec;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int v = i0 + j * p.tpr;
        if (!kAll && v >= p.nvec) break;
        stage_in<RES32, kPitch>(st, j, p.r, base + v);
        if (branch) stage_in<ACT32, kPitch>(st + kAtY * kPitch, j, p.y, base + v);
        if (full_gate) stage_in<ACT32, kPitch>(st + kAtGate * kPitch, j, p.gate, base + v);
      }
    }
    rows_commit();
  };
  launch_wait();
  launch_begin_next();
  if (kStaged)
    for (int s = 0; s + 1 < kStages; ++s) fetch(blockIdx.x * p.rows + row + s * step, s);

  Vec8 c[VPT], w[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = i0 + j * p.tpr;
    c[j] = constant8(p.branch_scale);
    w[j] = constant8(0.f);
    if (!kAll && v >= p.nvec) continue;
    if (post) {
      const Vec8 a = load8(p.w_post, v, p.w_f32);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        c[j].p[e] = mul2(c[j].p[e], add2(a.p[e], both2(p.w_offset)));
    }
    if (p.gate_kind == MOE_GATE_CHANNEL) {
      const Vec8 a = load8(p.gate, v, p.w_f32);
#pragma unroll
      for (int e = 0; e < 4; ++e) c[j].p[e] = mul2(c[j].p[e], a.p[e]);
    }
    if (pre) {
      w[j] = load8(p.w_pre, v, p.w_f32);
#pragma unroll
      for (int e = 0; e < 4; ++e) w[j].p[e] = add2(w[j].p[e], both2(p.w_offset));
    }
  }

  Vec8 r[VPT];
  // A: this thread's part of the sum of y^2 of row t
  auto branch_square = [&](int t, const uint4* st) {
    f32x2 s2 = both2(0.f);
    const size_t base = static_cast<size_t>(t) * p.nvec;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = i0 + j * p.tpr;
      if (t >= p.T || (!kAll && v >= p.nvec)) continue;
      const Vec8 y = row8<ACT32, kPitch>(st + kAtY * kPitch, j, p.y, base + v);
#pragma unroll
      for (int e = 0; e < 4; ++e) s2 = fma2(y.p[e], y.p[e], s2);
    }
    return sum2(s2);
  };
  // B: r' of row t into r and out, and this thread's part of the sum of its squares
  auto residual = [&](int t, const uint4* st, float tok) {       // tok = i_y (token gate)
    f32x2 s2 = both2(0.f);
    if (t >= p.T) return 0.f;
    const size_t base = static_cast<size_t>(t) * p.nvec;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = i0 + j * p.tpr;
      if (!kAll && v >= p.nvec) continue;
      if (kStaged) r[j] = row8<RES32, kPitch>(st, j, p.r, base + v);
      if (p.res_scale != 1.f) {
#pragma unroll
        for (int e = 0; e < 4; ++e) r[j].p[e] = mul2(both2(p.res_scale), r[j].p[e]);
      }
      if (branch) {
        Vec8 y = row8<ACT32, kPitch>(st + kAtY * kPitch, j, p.y, base + v);
        if (full_gate) {
          const Vec8 g = row8<ACT32, kPitch>(st + kAtGate * kPitch, j, p.gate, base + v);
#pragma unroll
          for (int e = 0; e < 4; ++e) y.p[e] = mul2(y.p[e], g.p[e]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) r[j].p[e] = fma2(mul2(both2(tok), y.p[e]), c[j].p[e], r[j].p[e]);
      }
      if (kAll || p.r_out) store8(p.r_out, base + v, RES32, r[j]);
#pragma unroll
      for (int e = 0; e < 4; ++e) s2 = fma2(r[j].p[e], r[j].p[e], s2);
    }
    return sum2(s2);
  };
  // C: h of row t from r
  auto normalised = [&](int t, float ss) {
    if (t >= p.T) return;
    const size_t base = static_cast<size_t>(t) * p.nvec;
    const f32x2 i_r = both2(rsqrtf(fmaf(ss, p.inv_d, p.eps)));
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = i0 + j * p.tpr;
      if (!kAll && v >= p.nvec) continue;               // for e4m3: whole half-warps at a time
      Vec8 h;
#pragma unroll
      for (int e = 0; e < 4; ++e) h.p[e] = mul2(mul2(r[j].p[e], i_r), w[j].p[e]);
      if (p.out != MOE_E4M3) {
        store8(p.h, base + v, p.out == MOE_F32, h);
      } else {
        // 16 consecutive threads (a half-warp: tpr is a multiple of 32) hold a 128-value block
        uint32_t amax = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = unpack2(h.p[e]);
          amax = max(amax, max(__float_as_uint(fabsf(f.x)), __float_as_uint(fabsf(f.y))));
        }
        amax = __reduce_max_sync((threadIdx.x & 16) ? 0xFFFF0000u : 0x0000FFFFu, amax);
        const int ex = e4m3_scale_exponent(amax);
        uint2 q;
        uint16_t* qh = reinterpret_cast<uint16_t*>(&q);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = unpack2(h.p[e]);
          qh[e] = __nv_cvt_float2_to_fp8x2(make_float2(scalbnf(f.x, -ex), scalbnf(f.y, -ex)), __NV_SATFINITE,
                                           __NV_E4M3);
        }
        static_cast<uint2*>(p.h)[base + v] = q;
        if ((v & 15) == 0) p.h_scale[(base + v) >> 4] = ldexpf(1.0f, ex);
      }
    }
  };
  auto i_of = [&](float ss) { return post ? rsqrtf(fmaf(ss, p.inv_d, p.eps)) : 1.f; };
  const bool tokens = p.gate_kind == MOE_GATE_TOKEN;
  auto token_bits = [&](int t) { return tokens && t < p.T ? load1_bits(p.gate, t, p.w_f32) : 0u; };
  auto gated = [&](float i_y, uint32_t bits) { return tokens ? i_y * value1(bits, p.w_f32) : i_y; };

  if (!kStaged) {                              // one row per row slot
    const int t = blockIdx.x * p.rows + row;
    if (t < p.T) {                             // the loads of r before the sum over y
#pragma unroll
      for (int j = 0; j < VPT; ++j)
        if (i0 + j * p.tpr < p.nvec) r[j] = load8(p.r, static_cast<size_t>(t) * p.nvec + i0 + j * p.tpr, RES32);
    }
    const uint32_t g = token_bits(t);
    float sy[1] = {0.f};
    if (post) {
      sy[0] = branch_square(t, nullptr);
      row_sums(sy, part[0], p.tpr);
    }
    float sr[1] = {residual(t, nullptr, gated(i_of(sy[0]), g))};
    if (!pre) return;
    row_sums(sr, part[1], p.tpr);
    normalised(t, sr[0]);
    return;
  }
  // Staged: B of row t and A of the next row share one pass to the row's sums, so a turn meets
  // one barrier and has the work of two rows around it.  Every thread of the CTA makes the same
  // number of turns.
  int t = blockIdx.x * p.rows + row;
  rows_wait<kStages>();                        // the first row (kStages - 1 are under way)
  float sums[2] = {0.f, post ? branch_square(t, ring + threadIdx.x) : 0.f};
  if (post) row_sums(sums, part[1], p.tpr);
  int turn = 0;
  uint32_t g = token_bits(t);
  for (int t0 = blockIdx.x * p.rows; t0 < p.T; t0 += step, t += step, ++turn) {
    const uint32_t g_next = token_bits(t + step);
    fetch(t + (kStages - 1) * step, (turn + kStages - 1) % kRing);
    rows_wait<kStages>();                      // row t + step
    const uint4* st = ring + turn % kRing * stage_vecs + threadIdx.x;
    const uint4* next = ring + (turn + 1) % kRing * stage_vecs + threadIdx.x;
    sums[0] = residual(t, st, gated(i_of(sums[1]), g));
    g = g_next;
    if (post) {
      sums[1] = branch_square(t + step, next);
      row_sums(sums, part[turn & 1], p.tpr);
    } else if (pre) {
      float one[1] = {sums[0]};
      row_sums(one, part[turn & 1], p.tpr);
      sums[0] = one[0];
    }
    if (pre) normalised(t, sums[0]);
  }
}

// ---------------------------------------------------------------- backward
struct NormGradArgs {
  const void *rp, *y, *w_post, *gate, *w_pre, *dh, *dr_out;
  void *dr, *dy, *dgate;
  float* parts;                   // [2][n_parts][d]: sums for dw_pre, and for dw_post / channel dgate
  int n_parts;
  bool want_pre, want_branch, want_gate;
  int T, d, nvec, tpr, rows;
  int gate_kind;
  bool w_f32;
  float inv_d, eps, res_scale, branch_scale, w_offset;
};

// Rows as in the forward kernel, read again from the stage (or from L1 / L2) in each of the
// three passes over a row, so that between its sums only one value per element lives in
// registers.  Two sums over tokens per channel are enough for all three channel gradients:
//   A = sum_t dh r' i_r                 dw_pre
//   B = sum_t b g_t G y i_y             dw_post = B (channel gate),  dgate = B (w_post + o)
// (g_t the token or full gate, 1 with a channel gate, which is constant over tokens).  A thread
// keeps those of its own vectors in registers (VPT <= 2) or in its own places of shared memory,
// and writes them at the end as one partial per row slot.
//
// Measured at T = 4095, d = 7168, bf16, both norms, channel gate, all gradients (352 MB): 72 us
// with the sum of the partials, 4.9 TB/s, 0.75 of the measured copy bandwidth; bound by
// instructions (41 per element with a token gate, issued in 50% of the cycles) and the shared-memory
// reads of the three passes.
template <bool RES32, bool ACT32, int VPT, int kStages, bool kAll = false>
__global__ void __launch_bounds__(kRowThreads) block_norm_backward_kernel(const NormGradArgs p) {
  constexpr bool kSmem = VPT > 2, kStaged = kStages > 0;
  static_assert(!(kSmem && kStaged), "shared memory holds the column sums or the stages");
  constexpr int kRing = kStaged ? kStages : 1, kPitch = kStaged ? kRowThreads : 0;
  constexpr int kR = RES32 ? 2 : 1, kY = ACT32 ? 2 : 1;
  __shared__ float part[2][32 * 5];
  extern __shared__ uint4 ring[];              // kSmem: fp32 column sums [2][d]
  float4* sums = reinterpret_cast<float4*>(ring);
  const int threads = blockDim.x;
  const int row = threadIdx.x / p.tpr, i0 = threadIdx.x - row * p.tpr;
  const int step = gridDim.x * p.rows;
  launch_wait();
  launch_begin_next();
  Vec8 A[kSmem ? 1 : VPT], B[kSmem ? 1 : VPT];
  if (kSmem) {
    for (int i = threadIdx.x; i < p.d / 2; i += threads) sums[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    __syncthreads();
  } else {
#pragma unroll
    for (int j = 0; j < VPT; ++j) A[kSmem ? 0 : j] = B[kSmem ? 0 : j] = constant8(0.f);
  }
  auto smem_add = [&](int which, int v, const Vec8& x) {
    float4* s = sums + which * (p.d / 4) + 2 * v;
    const float4 a = s[0], b = s[1];
    const float2 x0 = unpack2(x.p[0]), x1 = unpack2(x.p[1]), x2 = unpack2(x.p[2]), x3 = unpack2(x.p[3]);
    s[0] = make_float4(a.x + x0.x, a.y + x0.y, a.z + x1.x, a.w + x1.y);
    s[1] = make_float4(b.x + x2.x, b.y + x2.y, b.z + x3.x, b.w + x3.y);
  };
  // stage: r' and dh (with the pre-norm), dr_out, y, full gate -- in fixed places
  constexpr int kAtDh = VPT * kR, kAtDr = kAtDh + VPT * kY, kAtY = kAtDr + VPT * kR, kAtGate = kAtY + VPT * kY;
  const bool full_gate = !kAll && p.gate_kind == MOE_GATE_FULL;
  const bool branch = kAll || p.y, post = kAll || p.w_post, pre = kAll || p.w_pre, upper = kAll || p.dr_out;
  const int stage_vecs = (kAtGate + (full_gate ? VPT * kY : 0)) * kPitch;
  auto fetch = [&](int t, int s) {
    if (t < p.T) {
      uint4* st = ring + s * stage_vecs + threadIdx.x;
      const size_t base = static_cast<size_t>(t) * p.nvec;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int v = i0 + j * p.tpr;
        if (!kAll && v >= p.nvec) break;
        if (pre) {
          stage_in<RES32, kPitch>(st, j, p.rp, base + v);
          stage_in<ACT32, kPitch>(st + kAtDh * kPitch, j, p.dh, base + v);
        }
        if (upper) stage_in<RES32, kPitch>(st + kAtDr * kPitch, j, p.dr_out, base + v);
        if (branch) stage_in<ACT32, kPitch>(st + kAtY * kPitch, j, p.y, base + v);
        if (full_gate) stage_in<ACT32, kPitch>(st + kAtGate * kPitch, j, p.gate, base + v);
      }
    }
    rows_commit();
  };
  if (kStaged)
    for (int s = 0; s + 1 < kStages; ++s) fetch(blockIdx.x * p.rows + row + s * step, s);

  // w_pre + o, and c = (w_post + o) (channel gate): in registers unless a thread has too many
  auto pre_weight = [&](int v) {
    Vec8 a = load8(p.w_pre, v, p.w_f32);
#pragma unroll
    for (int e = 0; e < 4; ++e) a.p[e] = add2(a.p[e], both2(p.w_offset));
    return a;
  };
  auto branch_weight = [&](int v) {
    Vec8 a = constant8(1.f);
    if (post) {
      a = load8(p.w_post, v, p.w_f32);
#pragma unroll
      for (int e = 0; e < 4; ++e) a.p[e] = add2(a.p[e], both2(p.w_offset));
    }
    if (p.gate_kind == MOE_GATE_CHANNEL) {
      const Vec8 g = load8(p.gate, v, p.w_f32);
#pragma unroll
      for (int e = 0; e < 4; ++e) a.p[e] = mul2(a.p[e], g.p[e]);
    }
    return a;
  };
  Vec8 w[kSmem ? 1 : VPT], c[kSmem ? 1 : VPT];
  if (!kSmem) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = i0 + j * p.tpr;
      w[kSmem ? 0 : j] = c[kSmem ? 0 : j] = constant8(0.f);
      if (!kAll && v >= p.nvec) continue;
      if (pre) w[kSmem ? 0 : j] = pre_weight(v);
      c[kSmem ? 0 : j] = branch_weight(v);
    }
  }

  Vec8 q[VPT];
  // 1: this thread's parts of the sums of r'^2, z r' and y^2 of row t
  auto squares = [&](int t, const uint4* st, float* s) {
    f32x2 s0 = both2(0.f), s1 = both2(0.f), s2 = both2(0.f);
    const size_t base = static_cast<size_t>(t) * p.nvec;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = i0 + j * p.tpr;
      if (t >= p.T || (!kAll && v >= p.nvec)) continue;
      if (pre) {
        const Vec8 x = row8<RES32, kPitch>(st, j, p.rp, base + v);
        const Vec8 z = row8<ACT32, kPitch>(st + kAtDh * kPitch, j, p.dh, base + v);
        const Vec8 wj = kSmem ? pre_weight(v) : w[kSmem ? 0 : j];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s0 = fma2(x.p[e], x.p[e], s0);
          s1 = fma2(mul2(z.p[e], wj.p[e]), x.p[e], s1);
        }
      }
      if (post) {
        const Vec8 y = row8<ACT32, kPitch>(st + kAtY * kPitch, j, p.y, base + v);
#pragma unroll
        for (int e = 0; e < 4; ++e) s2 = fma2(y.p[e], y.p[e], s2);
      }
    }
    s[0] = sum2(s0);
    s[1] = sum2(s1);
    s[2] = sum2(s2);
  };
  // 2: G of row t (dr, the channel sums), q kept, and the parts of the sums of q y and G u
  auto gradients = [&](int t, const uint4* st, float tok, float i_r, float zr, float i_y, float* m) {
    m[0] = m[1] = 0.f;
    if (t >= p.T) return;
    const size_t base = static_cast<size_t>(t) * p.nvec;
    // x^ = r' i_r stands for r' throughout: i_r^3 by itself leaves the range of fp32 (rows of zeros
    // with an eps below 1e-25, rows past 1e12)
    const f32x2 k_r = both2(-i_r * (zr * p.inv_d));
    f32x2 m0 = both2(0.f), m1 = both2(0.f);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = i0 + j * p.tpr;
      if (!kAll && v >= p.nvec) continue;
      Vec8 G = constant8(0.f);
      if (upper) G = row8<RES32, kPitch>(st + kAtDr * kPitch, j, p.dr_out, base + v);
      if (pre) {
        const Vec8 x = row8<RES32, kPitch>(st, j, p.rp, base + v);
        const Vec8 z = row8<ACT32, kPitch>(st + kAtDh * kPitch, j, p.dh, base + v);
        const Vec8 wj = kSmem ? pre_weight(v) : w[kSmem ? 0 : j];
        Vec8 zx;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const f32x2 n = mul2(x.p[e], both2(i_r));
          if (!kSmem) A[kSmem ? 0 : j].p[e] = fma2(z.p[e], n, A[kSmem ? 0 : j].p[e]);
          else zx.p[e] = mul2(z.p[e], n);
          G.p[e] = fma2(both2(i_r), fma2(z.p[e], wj.p[e], mul2(k_r, n)), G.p[e]);
        }
        if (kSmem && p.want_pre) smem_add(0, v, zx);
      }
      Vec8 y = constant8(0.f), g = constant8(1.f);
      if (branch) y = row8<ACT32, kPitch>(st + kAtY * kPitch, j, p.y, base + v);
      if (full_gate) g = row8<ACT32, kPitch>(st + kAtGate * kPitch, j, p.gate, base + v);
      if (p.res_scale != 1.f) {
        Vec8 o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o.p[e] = mul2(both2(p.res_scale), G.p[e]);
        store8(p.dr, base + v, RES32, o);
      } else {
        store8(p.dr, base + v, RES32, G);
      }
      if (!branch) continue;
      const Vec8 cj = kSmem ? branch_weight(v) : c[kSmem ? 0 : j];
      Vec8 b;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const f32x2 n = mul2(y.p[e], both2(i_y));                // normalised branch
        f32x2 dn = mul2(both2(tok), G.p[e]);
        if (full_gate) dn = mul2(dn, g.p[e]);
        q[j].p[e] = mul2(dn, cj.p[e]);                           // q (dy itself without w_post)
        m0 = fma2(q[j].p[e], y.p[e], m0);
        if (!kSmem) B[kSmem ? 0 : j].p[e] = fma2(dn, n, B[kSmem ? 0 : j].p[e]);
        else b.p[e] = mul2(dn, n);
      }
      if (kSmem && p.want_branch) smem_add(1, v, b);
      if (p.want_gate && p.gate_kind != MOE_GATE_CHANNEL) {
        Vec8 dg;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const f32x2 u = mul2(mul2(both2(p.branch_scale), cj.p[e]), mul2(y.p[e], both2(i_y)));
          dg.p[e] = mul2(G.p[e], u);
          m1 = fma2(G.p[e], u, m1);
        }
        if (full_gate) store8(p.dgate, base + v, ACT32, dg);
      }
    }
    m[0] = sum2(m0);
    m[1] = sum2(m1);
  };
  // 3: dy of row t
  auto branch_gradient = [&](int t, const uint4* st, float i_y, float qy, float gu) {
    if (t >= p.T || !branch) return;
    const size_t base = static_cast<size_t>(t) * p.nvec;
    const f32x2 k_y = both2(-i_y * (qy * p.inv_d));
    if (i0 == 0 && p.want_gate && p.gate_kind == MOE_GATE_TOKEN) static_cast<float*>(p.dgate)[t] = gu;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = i0 + j * p.tpr;
      if (!kAll && v >= p.nvec) continue;
      if (post) {
        const Vec8 y = row8<ACT32, kPitch>(st + kAtY * kPitch, j, p.y, base + v);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          q[j].p[e] = mul2(both2(i_y), fma2(k_y, mul2(y.p[e], both2(i_y)), q[j].p[e]));
      }
      store8(p.dy, base + v, ACT32, q[j]);
    }
  };
  auto i_of = [&](float ss) { return rsqrtf(fmaf(ss, p.inv_d, p.eps)); };
  const bool tokens = p.gate_kind == MOE_GATE_TOKEN;
  auto token_bits = [&](int t) { return tokens && t < p.T ? load1_bits(p.gate, t, p.w_f32) : 0u; };
  auto scale_of = [&](uint32_t bits) {         // branch_scale (token gate)
    return tokens ? p.branch_scale * value1(bits, p.w_f32) : p.branch_scale;
  };

  int t = blockIdx.x * p.rows + row;
  if (!kStaged) {
    // every thread of the CTA makes the same number of turns (row_sums synchronises it)
    for (int t0 = blockIdx.x * p.rows; t0 < p.T; t0 += step, t += step) {
      float s[3], m[2];
      squares(t, nullptr, s);
      row_sums(s, part[0], p.tpr);
      const float i_y = post ? i_of(s[2]) : 1.f;
      gradients(t, nullptr, scale_of(token_bits(t)), i_of(s[0]), s[1], i_y, m);
      row_sums(m, part[1], p.tpr);
      branch_gradient(t, nullptr, i_y, m[0], m[1]);
    }
  } else {
    // 2 of row t and 1 of the next row share one pass to the row's sums (see the forward kernel)
    rows_wait<kStages>();
    float s[5];                                // row t + step: 0..2; row t: 3, 4
    {
      float f[3];
      squares(t, ring + threadIdx.x, f);
      row_sums(f, part[1], p.tpr);
      s[0] = f[0];
      s[1] = f[1];
      s[2] = f[2];
    }
    int turn = 0;
    for (int t0 = blockIdx.x * p.rows; t0 < p.T; t0 += step, t += step, ++turn) {
      const uint32_t tok = token_bits(t);      // (under way while the rows are waited for)
      fetch(t + (kStages - 1) * step, (turn + kStages - 1) % kRing);
      rows_wait<kStages>();                    // row t + step
      const uint4* st = ring + turn % kRing * stage_vecs + threadIdx.x;
      const float i_y = post ? i_of(s[2]) : 1.f;
      gradients(t, st, scale_of(tok), i_of(s[0]), s[1], i_y, s + 3);
      squares(t + step, ring + (turn + 1) % kRing * stage_vecs + threadIdx.x, s);
      row_sums(s, part[turn & 1], p.tpr);
      branch_gradient(t, st, i_y, s[3], s[4]);
    }
  }
  const size_t slot = static_cast<size_t>(blockIdx.x) * p.rows + row;
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    if (!(a == 0 ? p.want_pre : p.want_branch)) continue;
    float* out = p.parts + (static_cast<size_t>(a) * p.n_parts + slot) * p.d;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = i0 + j * p.tpr;
      if (!kAll && v >= p.nvec) continue;
      Vec8 f;
      if (kSmem) f = load8(sums + a * (p.d / 4), v, true);
      else f = a == 0 ? A[kSmem ? 0 : j] : B[kSmem ? 0 : j];
      store8(out, v, true, f);
    }
  }
}

// Sums of the partials: a CTA takes 32 channels of A (blockIdx.y = 0) or B (1), its 8 warps
// every 8th partial, joined in a fixed order; B gives dw_post and the channel gate's gradient.
__global__ void __launch_bounds__(256) sum_parts_kernel(const NormGradArgs p, float* dw_pre, float* dw_post,
                                                        float* dgate) {
  __shared__ float s[8][33];
  launch_wait();
  launch_begin_next();
  const bool branch = blockIdx.y != 0;
  if (branch ? !p.want_branch : !p.want_pre) return;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  const float* src = p.parts + static_cast<size_t>(blockIdx.y) * p.n_parts * p.d;
  float v = 0.f;
  if (col < p.d)
#pragma unroll 8
    for (int i = w; i < p.n_parts; i += 8) v += src[static_cast<size_t>(i) * p.d + col];
  s[w][lane] = v;
  __syncthreads();
  if (w == 0 && col < p.d) {
    for (int i = 1; i < 8; ++i) v += s[i][lane];
    if (!branch) {
      dw_pre[col] = v;
    } else {
      const bool channel = p.gate_kind == MOE_GATE_CHANNEL;
      if (dw_post) dw_post[col] = channel ? v * load1(p.gate, col, p.w_f32) : v;
      if (dgate) dgate[col] = p.w_post ? v * (load1(p.w_post, col, p.w_f32) + p.w_offset) : v;
    }
  }
}

constexpr size_t kNormHeader = 256;
constexpr int kBackwardCtas = 148;             // partial sums per row slot: one CTA per SM

struct BackwardShape {
  int vpt, tpr, rows;
};
// Threads hold two vectors of 8 (one up to 32 of them, four above 1024); short rows share a CTA.
BackwardShape backward_shape(int d) {
  const int nvec = d / 8;
  BackwardShape s;
  s.vpt = nvec <= 32 ? 1 : (nvec <= 1024 ? 2 : 4);
  s.tpr = ((nvec + s.vpt - 1) / s.vpt + 31) / 32 * 32;
  s.rows = kRowThreads / s.tpr;
  return s;
}

bool float_type(moe_dtype t) { return t == MOE_BF16 || t == MOE_F32; }

moe_status check_norm(const moe_norm_config* c) {
  if (!c || c->T < 0 || c->d_model <= 0) return MOE_ERR_INVALID_ARG;
  if (c->gate < MOE_GATE_NONE || c->gate > MOE_GATE_FULL) return MOE_ERR_INVALID_ARG;
  if (!(c->eps > 0.f) || !std::isfinite(c->eps) || !std::isfinite(c->res_scale) ||
      !std::isfinite(c->branch_scale) || !std::isfinite(c->w_offset))
    return MOE_ERR_INVALID_ARG;
  if (c->d_model % 8 || c->d_model > 16384 || c->T > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  if (!float_type(c->res) || !float_type(c->act) || !float_type(c->weight)) return MOE_ERR_UNSUPPORTED;
  if (!float_type(c->out) && !(c->out == MOE_E4M3 && c->d_model % 128 == 0)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

size_t backward_workspace(const moe_norm_config& c) {
  const BackwardShape s = backward_shape(c.d_model);
  return kNormHeader + sizeof(float) * 2 * static_cast<size_t>(kBackwardCtas) * s.rows * c.d_model;
}

// A token gate is read by the element.
size_t gate_alignment(const moe_norm_config& c) {
  return c.gate != MOE_GATE_TOKEN ? 16 : (c.weight == MOE_F32 ? 4 : 2);
}

moe_status ok_or_cuda(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

constexpr int kSms = 148;
constexpr size_t kSmemPerSm = 216 * 1024;

template <bool RES32, bool ACT32, int VPT>
cudaError_t launch_forward_typed(const NormArgs& a, cudaStream_t s) {
  if constexpr (VPT > 1) {
    // staged: one CTA per SM with as many rows as its threads hold vectors for, kStages - 1 turns
    // in flight, if every CTA gets at least that many.  (Two CTAs per SM leave 72 registers per
    // thread, which spill: 94 us against 83 at T = 8192, d = 7168 without a gate.)
    constexpr int kStages = VPT == 2 ? 4 : 3, kR = RES32 ? 2 : 1, kY = ACT32 ? 2 : 1;
    constexpr size_t kUnit = static_cast<size_t>(kStages) * VPT * kRowThreads * 16;
    const size_t smem = kUnit * (kR + ((a.y != nullptr) + (a.gate_kind == MOE_GATE_FULL)) * kY);
    NormArgs q = a;
    q.rows = kRowThreads / a.tpr;                // fill the CTA
    const int threads = q.tpr * q.rows;
    if (smem <= kSmemPerSm && q.rows >= 1 && a.T >= static_cast<int64_t>(kStages) * kSms * q.rows) {
      auto kernel = block_norm_kernel<RES32, ACT32, VPT, kStages, false>;
      if constexpr (kUnit * (kR + kY) <= kSmemPerSm)              // (a branch without a full gate fits)
        if (a.y && a.w_post && a.w_pre && a.r_out && a.gate_kind != MOE_GATE_FULL && a.nvec == VPT * a.tpr)
          kernel = block_norm_kernel<RES32, ACT32, VPT, kStages, true>;
      const cudaError_t e =
          cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
      if (e != cudaSuccess) return e;
      return launch_overlapped(kernel, dim3(kSms), threads, smem, s, q);
    }
  }
  const int64_t turns = (static_cast<int64_t>(a.T) + a.rows - 1) / a.rows;
  const int threads = a.tpr * a.rows;
  return launch_overlapped(block_norm_kernel<RES32, ACT32, VPT, 0>, dim3(static_cast<unsigned>(turns)), threads, 0, s, a);
}
template <int VPT>
cudaError_t launch_forward(const NormArgs& a, bool res32, bool act32, cudaStream_t s) {
  if (res32 && act32) return launch_forward_typed<true, true, VPT>(a, s);
  if (res32) return launch_forward_typed<true, false, VPT>(a, s);
  if (act32) return launch_forward_typed<false, true, VPT>(a, s);
  return launch_forward_typed<false, false, VPT>(a, s);
}

template <bool RES32, bool ACT32, int VPT>
cudaError_t launch_backward_typed(const NormGradArgs& a, unsigned grid, cudaStream_t s) {
  const int threads = a.tpr * a.rows;
  constexpr int kStages = 3, kR = RES32 ? 2 : 1, kY = ACT32 ? 2 : 1;
  constexpr size_t kUnit = static_cast<size_t>(kStages) * VPT * kRowThreads * 16;
  if constexpr (VPT <= 2 && kUnit * (2 * kR + 2 * kY) <= kSmemPerSm) {            // (without a full gate it fits)
    const size_t smem = kUnit * (2 * kR + (2 + (a.gate_kind == MOE_GATE_FULL)) * kY);
    if (smem <= kSmemPerSm && a.T > 2 * static_cast<int64_t>(grid) * a.rows) {
      const bool all = a.y && a.w_post && a.w_pre && a.dr_out && a.gate_kind != MOE_GATE_FULL && a.nvec == VPT * a.tpr;
      auto kernel = all ? block_norm_backward_kernel<RES32, ACT32, VPT, kStages, true>
                        : block_norm_backward_kernel<RES32, ACT32, VPT, kStages, false>;
      const cudaError_t e =
          cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
      if (e != cudaSuccess) return e;
      return launch_overlapped(kernel, dim3(grid), threads, smem, s, a);
    }
  }
  const size_t smem = VPT > 2 ? sizeof(float) * 2 * a.d : 0;
  if (smem) {
    const cudaError_t e = cudaFuncSetAttribute(block_norm_backward_kernel<RES32, ACT32, VPT, 0>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  return launch_overlapped(block_norm_backward_kernel<RES32, ACT32, VPT, 0>, dim3(grid), threads, smem, s, a);
}
template <int VPT>
cudaError_t launch_backward(const NormGradArgs& a, bool res32, bool act32, unsigned grid, cudaStream_t s) {
  if (res32 && act32) return launch_backward_typed<true, true, VPT>(a, grid, s);
  if (res32) return launch_backward_typed<true, false, VPT>(a, grid, s);
  if (act32) return launch_backward_typed<false, true, VPT>(a, grid, s);
  return launch_backward_typed<false, false, VPT>(a, grid, s);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_norm_workspace_size(const moe_norm_config* cfg, size_t* bytes) {
  if (!bytes) return MOE_ERR_INVALID_ARG;
  const moe_status st = check_norm(cfg);
  if (st != MOE_OK) return st;
  *bytes = backward_workspace(*cfg);
  return MOE_OK;
}

moe_status moe_block_norm(const moe_norm_config* cfg, const void* r, const void* y, const void* w_post,
                          const void* gate, const void* w_pre, void* r_out, void* h, float* h_scale,
                          cudaStream_t stream) {
  const moe_status st = check_norm(cfg);
  if (st != MOE_OK) return st;
  if (cfg->T == 0) return MOE_OK;                // (tensors of no rows have no address to check)
  if ((cfg->gate != MOE_GATE_NONE) != (gate != nullptr) || (!y && (w_post || gate)) || !w_pre != !h ||
      (h && (cfg->out == MOE_E4M3) != (h_scale != nullptr)) || (!h && h_scale) || (!r_out && !h) || !r)
    return MOE_ERR_INVALID_ARG;
  if (misaligned(r) || misaligned(y) || misaligned(w_post) || misaligned(w_pre) || misaligned(r_out) ||
      misaligned(h) || misaligned(gate, gate_alignment(*cfg)) || misaligned(h_scale, sizeof(float)))
    return MOE_ERR_INVALID_ARG;
  NormArgs a{r, y, w_post, gate, w_pre, r_out, h, h_scale};
  a.T = cfg->T;
  a.d = cfg->d_model;
  a.nvec = cfg->d_model / 8;
  a.gate_kind = cfg->gate;
  a.w_f32 = cfg->weight == MOE_F32;
  a.out = cfg->out;
  a.inv_d = 1.0f / cfg->d_model;
  a.eps = cfg->eps;
  a.res_scale = cfg->res_scale;
  a.branch_scale = cfg->branch_scale;
  a.w_offset = cfg->w_offset;
  // few tokens (two rows per SM): as many threads per row as it has vectors, for the shortest chain
  // (d = 4096: 128 rows 3.0 us so, 3.9 with two vectors per thread; 1000 rows 10.5 against 9.6);
  // many: two vectors per thread, rows staged (d = 8192, 8192 rows, fp32 residual: 156 us, 232 with
  // four vectors, whose stages do not fit), and four where kRowThreads threads need them
  const int vpt = cfg->T <= 2 * kSms ? (a.nvec <= 1024 ? 1 : 2)
                                     : (a.nvec <= 64 ? 1 : (a.nvec <= 2 * kRowThreads ? 2 : 4));
  a.tpr = ((a.nvec + vpt - 1) / vpt + 31) / 32 * 32;
  a.rows = a.tpr >= 128 ? 1 : 128 / a.tpr;
  const bool res32 = cfg->res == MOE_F32, act32 = cfg->act == MOE_F32;
  return ok_or_cuda(vpt == 1 ? launch_forward<1>(a, res32, act32, stream)
                             : (vpt == 2 ? launch_forward<2>(a, res32, act32, stream)
                                         : launch_forward<4>(a, res32, act32, stream)));
}

moe_status moe_block_norm_backward(const moe_norm_config* cfg, const void* r_out, const void* y,
                                   const void* w_post, const void* gate, const void* w_pre,
                                   const void* dh, const void* dr_out, void* dr, void* dy, void* dgate,
                                   float* dw_post, float* dw_pre, void* ws, size_t ws_bytes,
                                   cudaStream_t stream) {
  const moe_status st = check_norm(cfg);
  if (st != MOE_OK) return st;
  if (!ws || (dgate && cfg->gate == MOE_GATE_NONE) || (dw_post && !w_post) || (dw_pre && !w_pre) ||
      (cfg->gate == MOE_GATE_CHANNEL && !gate))
    return MOE_ERR_INVALID_ARG;
  if (cfg->T > 0 &&                              // (tensors of no rows have no address to check)
      ((cfg->gate != MOE_GATE_NONE) != (gate != nullptr) || (!y && (w_post || gate)) || !w_pre != !dh || !y != !dy ||
       !dr || (w_pre && !r_out) || (!dh && !dr_out)))
    return MOE_ERR_INVALID_ARG;
  if (misaligned(r_out) || misaligned(y) || misaligned(w_post) || misaligned(w_pre) || misaligned(dh) ||
      misaligned(dr_out) || misaligned(dr) || misaligned(dy) || misaligned(ws) || misaligned(dw_post) ||
      misaligned(dw_pre) || misaligned(gate, gate_alignment(*cfg)) ||
      misaligned(dgate, cfg->gate == MOE_GATE_TOKEN ? sizeof(float) : 16))
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < backward_workspace(*cfg)) return MOE_ERR_WORKSPACE;
  if (cfg->T == 0) {                             // empty sums, whatever gate and weights hold
    const size_t bytes = sizeof(float) * cfg->d_model;
    for (void* sum : {static_cast<void*>(dw_pre), static_cast<void*>(dw_post),
                      cfg->gate == MOE_GATE_CHANNEL ? dgate : nullptr})
      if (sum && cudaMemsetAsync(sum, 0, bytes, stream) != cudaSuccess) return MOE_ERR_CUDA;
    return MOE_OK;
  }
  const BackwardShape sh = backward_shape(cfg->d_model);
  const int64_t turns = (static_cast<int64_t>(cfg->T) + sh.rows - 1) / sh.rows;
  const unsigned grid = static_cast<unsigned>(turns < kBackwardCtas ? turns : kBackwardCtas);
  NormGradArgs a{r_out, y, w_post, gate, w_pre, dh, dr_out, dr, dy, dgate};
  a.parts = reinterpret_cast<float*>(static_cast<char*>(ws) + kNormHeader);
  a.n_parts = static_cast<int>(grid) * sh.rows;
  a.want_pre = dw_pre != nullptr;
  a.want_gate = dgate != nullptr;
  a.want_branch = dw_post || (dgate && cfg->gate == MOE_GATE_CHANNEL);
  a.T = cfg->T;
  a.d = cfg->d_model;
  a.nvec = cfg->d_model / 8;
  a.tpr = sh.tpr;
  a.rows = sh.rows;
  a.gate_kind = cfg->gate;
  a.w_f32 = cfg->weight == MOE_F32;
  a.inv_d = 1.0f / cfg->d_model;
  a.eps = cfg->eps;
  a.res_scale = cfg->res_scale;
  a.branch_scale = cfg->branch_scale;
  a.w_offset = cfg->w_offset;
  const bool res32 = cfg->res == MOE_F32, act32 = cfg->act == MOE_F32;
  const cudaError_t e = sh.vpt == 1 ? launch_backward<1>(a, res32, act32, grid, stream)
                                    : (sh.vpt == 2 ? launch_backward<2>(a, res32, act32, grid, stream)
                                                   : launch_backward<4>(a, res32, act32, grid, stream));
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  float* dgc = cfg->gate == MOE_GATE_CHANNEL ? static_cast<float*>(dgate) : nullptr;
  if (a.want_pre || a.want_branch)
    return ok_or_cuda(launch_overlapped(sum_parts_kernel, dim3((a.d + 31) / 32, 2), 256, 0, stream, a, dw_pre, dw_post, dgc));
  return MOE_OK;
}

}  // extern "C"
