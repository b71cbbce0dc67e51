// block_norm.cu -- the norms around a block, fused with its gate and residual scale, and
// their gradients (moe_block_norm, moe_block_norm_backward).
//
//   u = y i_y (w_post + o),  i_y = (mean y^2 + eps)^-1/2        (u = y without w_post)
//   r' = a r + b g u
//   h = r' i_r (w_pre + o),  i_r = (mean r'^2 + eps)^-1/2
// and backwards, with z = dh (w_pre + o) and G the whole gradient of r':
//   G  = dr' + i_r z - r' i_r^3 mean(z r')          dr = a G       dw_pre  = sum_t dh r' i_r
//   q  = b g G (w_post + o)                                        dw_post = sum_t b g G y i_y
//   dy = i_y q - y i_y^3 mean(q y)                                 dgate   = sum b G u
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

constexpr int kMaxThreads = 1024;

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

// Eight consecutive elements (vector `v`) of a bf16 or fp32 array.
template <bool F32>
__device__ __forceinline__ void load8(const void* base, size_t v, float (&f)[8]) {
  if (F32) {
    const float4* p = static_cast<const float4*>(base) + 2 * v;
    const float4 a = p[0], b = p[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  } else {
    const uint4 q = static_cast<const uint4*>(base)[v];
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}
__device__ __forceinline__ void load8(const void* base, size_t v, bool f32, float (&f)[8]) {
  if (f32) load8<true>(base, v, f);
  else load8<false>(base, v, f);
}

template <bool F32>
__device__ __forceinline__ void store8(void* base, size_t v, const float (&f)[8]) {
  if (F32) {
    float4* p = static_cast<float4*>(base) + 2 * v;
    p[0] = make_float4(f[0], f[1], f[2], f[3]);
    p[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    uint4 q;
    __nv_bfloat162* b = reinterpret_cast<__nv_bfloat162*>(&q);
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    static_cast<uint4*>(base)[v] = q;
  }
}

__device__ __forceinline__ float load1(const void* base, size_t i, bool f32) {
  return f32 ? static_cast<const float*>(base)[i]
             : __bfloat162float(static_cast<const __nv_bfloat16*>(base)[i]);
}

// Sums of N values over the threads of a row, the same in every thread of it and in the same
// order every time.  `part`: shared memory, N floats per warp of the CTA, not touched since
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
    for (int j = 0; j < N; ++j) part[warp * N + j] = v[j];
  __syncthreads();
#pragma unroll
  for (int j = 0; j < N; ++j) {
    v[j] = lane < warps ? part[(first + lane) * N + j] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[j] += __shfl_xor_sync(0xffffffffu, v[j], o);
  }
}

// Rows on their way in: each thread copies the vectors that it alone will read into its own
// places of shared memory with cp.async, kStages - 1 rows ahead, so a CTA keeps that many rows
// in flight without holding them in registers and without a barrier (a thread waits for its own
// copies).  kStages = 0: rows are read from global memory directly (few rows per CTA).
template <int kStages>
__device__ __forceinline__ void rows_wait() {
  if (kStages) asm volatile("cp.async.wait_group %0;" ::"n"(kStages ? kStages - 1 : 0) : "memory");
}
__device__ __forceinline__ void rows_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// One array's vectors of a thread in one stage: VPT x (16 or 32 bytes), thread-interleaved.
template <bool F32>
__device__ __forceinline__ void stage_in(uint4* st, int slot, int threads, const void* base, size_t v) {
  const uint4* g = static_cast<const uint4*>(base);
  if (F32) {
    cp_async_16_cg(st + (2 * slot) * threads, g + 2 * v);
    cp_async_16_cg(st + (2 * slot + 1) * threads, g + 2 * v + 1);
  } else {
    cp_async_16_cg(st + slot * threads, g + v);
  }
}
template <bool F32>
__device__ __forceinline__ void unpack8(const uint4& a, const uint4& b, float (&f)[8]) {
  if (F32) {
    f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y);
    f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
    f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y);
    f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
  } else {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}
// Vector `slot` of this thread: from its stage, or straight from the array.
template <bool F32, bool STAGED>
__device__ __forceinline__ void row8(const uint4* st, int slot, int threads, const void* base, size_t v,
                                     float (&f)[8]) {
  if (STAGED) {
    const uint4 a = st[(F32 ? 2 * slot : slot) * threads];
    unpack8<F32>(a, F32 ? st[(2 * slot + 1) * threads] : a, f);
  } else {
    load8<F32>(base, v, f);
  }
}

// Thread i of a row holds vectors i, i + tpr, ...; a CTA walks rows blockIdx.x * rows + row,
// + gridDim.x * rows, ...  Measured at T = 8192, d = 7168, bf16, post-norm, token gate and
// pre-norm (470 MB): one row per CTA without staging 172 us (2.7 TB/s: the loads of a row and
// its two sums take turns).
template <bool RES32, bool ACT32, int VPT, int kStages>
__global__ void __launch_bounds__(VPT == 4 ? 512 : kMaxThreads) block_norm_kernel(const NormArgs p) {
  __shared__ float part[2][32];
  extern __shared__ uint4 ring[];
  constexpr bool kStaged = kStages > 0;
  constexpr int kR = RES32 ? 2 : 1, kY = ACT32 ? 2 : 1;
  const int threads = blockDim.x;
  const int row = threadIdx.x / p.tpr, i0 = threadIdx.x - row * p.tpr;
  const int step = gridDim.x * p.rows;
  const bool full_gate = p.gate_kind == MOE_GATE_FULL;
  const int stage_vecs = VPT * (kR + (p.y ? kY : 0) + (full_gate ? kY : 0)) * threads;
  auto fetch = [&](int t, int s) {
    if (t < p.T) {
      uint4* st = ring + s * stage_vecs + threadIdx.x;
      const size_t base = static_cast<size_t>(t) * p.nvec;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int v = i0 + j * p.tpr;
        if (v >= p.nvec) break;
        stage_in<RES32>(st, j, threads, p.r, base + v);
        if (p.y) stage_in<ACT32>(st + VPT * kR * threads, j, threads, p.y, base + v);
        if (full_gate) stage_in<ACT32>(st + VPT * (kR + kY) * threads, j, threads, p.gate, base + v);
      }
    }
    rows_commit();
  };
  if (kStaged)
    for (int s = 0; s + 1 < kStages; ++s) fetch(blockIdx.x * p.rows + row + s * step, s);

  int turn = 0;
  // every thread of the CTA makes the same number of turns (row_sums synchronises it)
  for (int t0 = blockIdx.x * p.rows; t0 < p.T; t0 += step, ++turn) {
    const int t = t0 + row;
    const bool live = t < p.T;
    const size_t base = static_cast<size_t>(live ? t : 0) * p.nvec;
    const uint4* st = nullptr;
    if (kStaged) {
      fetch(t + (kStages - 1) * step, (turn + kStages - 1) % (kStaged ? kStages : 1));
      rows_wait<kStages>();
      st = ring + turn % (kStaged ? kStages : 1) * stage_vecs + threadIdx.x;
    }
    float r[VPT][8], u[VPT][8];
    float ss[1] = {0.f};
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = i0 + j * p.tpr;
      if (live && v < p.nvec) {
        row8<RES32, kStaged>(st, j, threads, p.r, base + v, r[j]);
        if (p.y) row8<ACT32, kStaged>(st + VPT * kR * threads, j, threads, p.y, base + v, u[j]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) r[j][e] = u[j][e] = 0.f;
      }
    }
    if (p.w_post) {
#pragma unroll
      for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) ss[0] = fmaf(u[j][e], u[j][e], ss[0]);
      row_sums(ss, part[0], p.tpr);
    }
    const float i_y = rsqrtf(fmaf(ss[0], p.inv_d, p.eps));
    float tok = p.branch_scale;
    if (p.gate_kind == MOE_GATE_TOKEN && live) tok *= load1(p.gate, t, p.w_f32);
    ss[0] = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = i0 + j * p.tpr;
      if (!live || v >= p.nvec) continue;
      float c[8];
      if (p.y) {
        if (p.w_post) {
          load8(p.w_post, v, p.w_f32, c);
#pragma unroll
          for (int e = 0; e < 8; ++e) u[j][e] *= i_y * (c[e] + p.w_offset);
        }
        if (p.gate_kind == MOE_GATE_CHANNEL || full_gate) {
          if (full_gate) row8<ACT32, kStaged>(st + VPT * (kR + kY) * threads, j, threads, p.gate, base + v, c);
          else load8(p.gate, v, p.w_f32, c);
#pragma unroll
          for (int e = 0; e < 8; ++e) u[j][e] *= c[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) r[j][e] = fmaf(tok, u[j][e], p.res_scale * r[j][e]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) r[j][e] *= p.res_scale;
      }
      if (p.r_out) store8<RES32>(p.r_out, base + v, r[j]);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss[0] = fmaf(r[j][e], r[j][e], ss[0]);
    }
    if (!p.w_pre) {                            // (uniform over the grid)
      __syncthreads();                         // part[0] is free for the next row
      continue;
    }
    row_sums(ss, part[1], p.tpr);
    const float i_r = rsqrtf(fmaf(ss[0], p.inv_d, p.eps));
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = i0 + j * p.tpr;
      if (!live || v >= p.nvec) continue;      // for e4m3: whole half-warps at a time
      float c[8];
      load8(p.w_pre, v, p.w_f32, c);
#pragma unroll
      for (int e = 0; e < 8; ++e) c[e] = r[j][e] * i_r * (c[e] + p.w_offset);
      if (p.out == MOE_BF16) {
        store8<false>(p.h, base + v, c);
      } else if (p.out == MOE_F32) {
        store8<true>(p.h, base + v, c);
      } else {
        // 16 consecutive threads (a half-warp: tpr is a multiple of 32) hold a 128-value block
        uint32_t amax = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = max(amax, __float_as_uint(fabsf(c[e])));
        amax = __reduce_max_sync((threadIdx.x & 16) ? 0xFFFF0000u : 0x0000FFFFu, amax);
        const int ex = e4m3_scale_exponent(amax);
        uint2 q;
        uint16_t* qh = reinterpret_cast<uint16_t*>(&q);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          qh[e] = __nv_cvt_float2_to_fp8x2(make_float2(scalbnf(c[2 * e], -ex), scalbnf(c[2 * e + 1], -ex)),
                                           __NV_SATFINITE, __NV_E4M3);
        static_cast<uint2*>(p.h)[base + v] = q;
        if ((v & 15) == 0) p.h_scale[(base + v) >> 4] = ldexpf(1.0f, ex);
      }
    }
  }
}

// ---------------------------------------------------------------- backward
struct NormGradArgs {
  const void *rp, *y, *w_post, *gate, *w_pre, *dh, *dr_out;
  void *dr, *dy, *dgate;
  float* parts;                   // [3][n_parts][d]: dw_pre, dw_post, channel dgate
  int n_parts;
  bool want_pre, want_post, want_gate;
  int T, d, nvec, tpr, rows;
  int gate_kind;
  bool w_f32;
  float inv_d, eps, res_scale, branch_scale, w_offset;
};

// Rows as in the forward kernel, read again from the stage (or from L1 / L2) in each of the
// three passes over a row, so that between its two sums only one value per element lives in
// registers.  A thread keeps the column sums of its own vectors over its rows in registers
// (VPT <= 2) or in its own places of shared memory, and writes them at the end as one partial
// per row slot.
template <bool RES32, bool ACT32, int VPT, int kStages>
__global__ void __launch_bounds__(512) block_norm_backward_kernel(const NormGradArgs p) {
  constexpr bool kSmem = VPT > 2, kStaged = kStages > 0;
  static_assert(!(kSmem && kStaged), "shared memory holds the column sums or the stages");
  constexpr int kR = RES32 ? 2 : 1, kY = ACT32 ? 2 : 1;
  __shared__ float part[2][16 * 3];
  extern __shared__ uint4 ring[];              // kSmem: fp32 column sums [3][d]
  float* acc_smem = reinterpret_cast<float*>(ring);
  const int threads = blockDim.x;
  const int row = threadIdx.x / p.tpr, i0 = threadIdx.x - row * p.tpr;
  const int step = gridDim.x * p.rows;
  float acc[kSmem ? 1 : 3][kSmem ? 1 : VPT][8];
  if (kSmem) {
    for (int i = threadIdx.x; i < 3 * p.d; i += threads) acc_smem[i] = 0.f;
    __syncthreads();
  } else {
#pragma unroll
    for (int a = 0; a < 3; ++a)
#pragma unroll
      for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[kSmem ? 0 : a][kSmem ? 0 : j][e] = 0.f;
  }
  auto add = [&](int a, int j, int v, int e, float x) {
    if (kSmem) acc_smem[a * p.d + v * 8 + e] += x;
    else acc[kSmem ? 0 : a][kSmem ? 0 : j][e] += x;
  };
  // stage: r' and dh (with the pre-norm), dr_out, y, full gate -- in fixed places
  constexpr int kAtDh = VPT * kR, kAtDr = kAtDh + VPT * kY, kAtY = kAtDr + VPT * kR, kAtGate = kAtY + VPT * kY;
  const bool full_gate = p.gate_kind == MOE_GATE_FULL;
  const int stage_vecs = (kAtGate + (full_gate ? VPT * kY : 0)) * threads;
  auto fetch = [&](int t, int s) {
    if (t < p.T) {
      uint4* st = ring + s * stage_vecs + threadIdx.x;
      const size_t base = static_cast<size_t>(t) * p.nvec;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int v = i0 + j * p.tpr;
        if (v >= p.nvec) break;
        if (p.w_pre) {
          stage_in<RES32>(st, j, threads, p.rp, base + v);
          stage_in<ACT32>(st + kAtDh * threads, j, threads, p.dh, base + v);
        }
        if (p.dr_out) stage_in<RES32>(st + kAtDr * threads, j, threads, p.dr_out, base + v);
        if (p.y) stage_in<ACT32>(st + kAtY * threads, j, threads, p.y, base + v);
        if (full_gate) stage_in<ACT32>(st + kAtGate * threads, j, threads, p.gate, base + v);
      }
    }
    rows_commit();
  };
  if (kStaged)
    for (int s = 0; s + 1 < kStages; ++s) fetch(blockIdx.x * p.rows + row + s * step, s);

  int turn = 0;
  // every thread of the CTA makes the same number of turns (row_sums synchronises it)
  for (int t0 = blockIdx.x * p.rows; t0 < p.T; t0 += step, ++turn) {
    const int t = t0 + row;
    const bool live = t < p.T;
    const size_t base = static_cast<size_t>(live ? t : 0) * p.nvec;
    const uint4* st = nullptr;
    if (kStaged) {
      fetch(t + (kStages - 1) * step, (turn + kStages - 1) % (kStaged ? kStages : 1));
      rows_wait<kStages>();
      st = ring + turn % (kStaged ? kStages : 1) * stage_vecs + threadIdx.x;
    }
    float x[8], y[8], z[8], c[8];
    float s[3] = {0.f, 0.f, 0.f};              // r'^2, z r', y^2
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = i0 + j * p.tpr;
      if (!live || v >= p.nvec) continue;
      if (p.w_pre) {
        row8<RES32, kStaged>(st, j, threads, p.rp, base + v, x);
        row8<ACT32, kStaged>(st + kAtDh * threads, j, threads, p.dh, base + v, z);
        load8(p.w_pre, v, p.w_f32, c);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          s[0] = fmaf(x[e], x[e], s[0]);
          s[1] = fmaf(z[e] * (c[e] + p.w_offset), x[e], s[1]);
        }
      }
      if (p.w_post) {
        row8<ACT32, kStaged>(st + kAtY * threads, j, threads, p.y, base + v, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[2] = fmaf(y[e], y[e], s[2]);
      }
    }
    row_sums(s, part[0], p.tpr);
    const float i_r = rsqrtf(fmaf(s[0], p.inv_d, p.eps));
    const float k_r = i_r * i_r * i_r * (s[1] * p.inv_d);
    const float i_y = p.w_post ? rsqrtf(fmaf(s[2], p.inv_d, p.eps)) : 1.f;
    float tok = p.branch_scale;
    if (p.gate_kind == MOE_GATE_TOKEN && live) tok *= load1(p.gate, t, p.w_f32);
    float m[2] = {0.f, 0.f};                   // q y, G u
    float q[VPT][8];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = i0 + j * p.tpr;
#pragma unroll
      for (int e = 0; e < 8; ++e) q[j][e] = 0.f;
      if (!live || v >= p.nvec) continue;
      float G[8];
      if (p.dr_out) {
        row8<RES32, kStaged>(st + kAtDr * threads, j, threads, p.dr_out, base + v, G);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) G[e] = 0.f;
      }
      if (p.w_pre) {
        row8<RES32, kStaged>(st, j, threads, p.rp, base + v, x);
        row8<ACT32, kStaged>(st + kAtDh * threads, j, threads, p.dh, base + v, z);
        load8(p.w_pre, v, p.w_f32, c);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          G[e] += i_r * z[e] * (c[e] + p.w_offset) - k_r * x[e];
          if (p.want_pre) add(0, j, v, e, z[e] * (x[e] * i_r));
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = p.res_scale * G[e];
      if (!p.y) {
        store8<RES32>(p.dr, base + v, x);
        continue;
      }
      row8<ACT32, kStaged>(st + kAtY * threads, j, threads, p.y, base + v, y);
      if (full_gate) row8<ACT32, kStaged>(st + kAtGate * threads, j, threads, p.gate, base + v, z);
      store8<RES32>(p.dr, base + v, x);
      if (p.gate_kind == MOE_GATE_CHANNEL) load8(p.gate, v, p.w_f32, z);
      if (p.w_post) load8(p.w_post, v, p.w_f32, c);
      float dg[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float w = p.w_post ? c[e] + p.w_offset : 1.f;
        const float n = y[e] * i_y;                               // normalised branch
        const float bg = p.gate_kind == MOE_GATE_CHANNEL || full_gate ? tok * z[e] : tok;
        const float dn = bg * G[e];                               // gradient of norm(y; w_post)
        dg[e] = p.branch_scale * G[e] * (n * w);
        m[1] += dg[e];
        if (p.want_post) add(1, j, v, e, dn * n);
        if (p.want_gate && p.gate_kind == MOE_GATE_CHANNEL) add(2, j, v, e, dg[e]);
        q[j][e] = dn * w;                                         // dy itself without w_post
        m[0] = fmaf(q[j][e], y[e], m[0]);
      }
      if (p.want_gate && full_gate) store8<ACT32>(p.dgate, base + v, dg);
    }
    if (!p.y) {                                // (uniform over the grid)
      __syncthreads();                         // part[0] is free for the next row
      continue;
    }
    row_sums(m, part[1], p.tpr);
    const float k_y = i_y * i_y * i_y * (m[0] * p.inv_d);
    if (live && i0 == 0 && p.want_gate && p.gate_kind == MOE_GATE_TOKEN)
      static_cast<float*>(p.dgate)[t] = m[1];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = i0 + j * p.tpr;
      if (!live || v >= p.nvec) continue;
      if (p.w_post) {
        row8<ACT32, kStaged>(st + kAtY * threads, j, threads, p.y, base + v, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) q[j][e] = i_y * q[j][e] - k_y * y[e];
      }
      store8<ACT32>(p.dy, base + v, q[j]);
    }
  }
  const size_t slot = static_cast<size_t>(blockIdx.x) * p.rows + row;
#pragma unroll
  for (int a = 0; a < 3; ++a) {
    if (!(a == 0 ? p.want_pre : (a == 1 ? p.want_post : p.want_gate && p.gate_kind == MOE_GATE_CHANNEL)))
      continue;
    float* out = p.parts + (static_cast<size_t>(a) * p.n_parts + slot) * p.d;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = i0 + j * p.tpr;
      if (v >= p.nvec) continue;
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        f[e] = kSmem ? acc_smem[a * p.d + v * 8 + e] : acc[kSmem ? 0 : a][kSmem ? 0 : j][e];
      store8<true>(out, v, f);
    }
  }
}

// Column sums of up to three [n_parts][d] arrays: a CTA takes 32 columns of one of them, its
// 8 warps every 8th partial, joined in a fixed order.
__global__ void __launch_bounds__(256) sum_parts_kernel(const float* __restrict__ parts, int n_parts,
                                                        int d, float* o0, float* o1, float* o2) {
  __shared__ float s[8][33];
  float* out = blockIdx.y == 0 ? o0 : (blockIdx.y == 1 ? o1 : o2);
  if (!out) return;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  const float* src = parts + static_cast<size_t>(blockIdx.y) * n_parts * d;
  float v = 0.f;
  if (col < d)
    for (int i = w; i < n_parts; i += 8) v += src[static_cast<size_t>(i) * d + col];
  s[w][lane] = v;
  __syncthreads();
  if (w == 0 && col < d) {
    for (int i = 1; i < 8; ++i) v += s[i][lane];
    out[col] = v;
  }
}

constexpr size_t kNormHeader = 256;
constexpr int kBackwardCtas = 148;             // partial sums per row slot: one CTA per SM

struct BackwardShape {
  int vpt, tpr, rows;
};
// Threads hold one vector of 8 (two above 512 threads, four above 1024); short rows share a CTA.
BackwardShape backward_shape(int d) {
  const int nvec = d / 8;
  BackwardShape s;
  s.vpt = nvec <= 512 ? 1 : (nvec <= 1024 ? 2 : 4);
  s.tpr = ((nvec + s.vpt - 1) / s.vpt + 31) / 32 * 32;
  s.rows = s.tpr >= 256 ? 1 : 256 / s.tpr;
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
  return kNormHeader + sizeof(float) * 3 * static_cast<size_t>(kBackwardCtas) * s.rows * c.d_model;
}

bool unaligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

moe_status ok_or_cuda(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

constexpr int kSms = 148;
constexpr size_t kSmemPerSm = 216 * 1024;

template <bool RES32, bool ACT32, int VPT>
cudaError_t launch_forward_typed(const NormArgs& a, cudaStream_t s) {
  const int64_t turns = (static_cast<int64_t>(a.T) + a.rows - 1) / a.rows;
  const int threads = a.tpr * a.rows;
  if constexpr (VPT == 4) {
    // staged: three rows in flight per CTA, as many CTAs per SM as their stages leave room for
    // (at most four), if every CTA then gets at least three rows
    constexpr int kStages = 3;
    const size_t smem = static_cast<size_t>(kStages) * VPT * threads * 16 *
                        ((RES32 ? 2 : 1) + ((a.y != nullptr) + (a.gate_kind == MOE_GATE_FULL)) * (ACT32 ? 2 : 1));
    int ctas = static_cast<int>(kSmemPerSm / (smem + 1024));
    if (ctas > 4) ctas = 4;
    if (ctas >= 1 && turns >= 3 * kSms * ctas) {
      const cudaError_t e = cudaFuncSetAttribute(block_norm_kernel<RES32, ACT32, VPT, kStages>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 static_cast<int>(smem));
      if (e != cudaSuccess) return e;
      block_norm_kernel<RES32, ACT32, VPT, kStages><<<kSms * ctas, threads, smem, s>>>(a);
      return cudaGetLastError();
    }
  }
  block_norm_kernel<RES32, ACT32, VPT, 0><<<static_cast<unsigned>(turns), threads, 0, s>>>(a);
  return cudaGetLastError();
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
  if constexpr (VPT <= 2) {
    constexpr int kStages = 3;
    const size_t smem = static_cast<size_t>(kStages) * VPT * threads * 16 *
                        (2 * (RES32 ? 2 : 1) + (2 + (a.gate_kind == MOE_GATE_FULL)) * (ACT32 ? 2 : 1));
    if (smem <= kSmemPerSm && a.T > 2 * static_cast<int64_t>(grid) * a.rows) {
      const cudaError_t e = cudaFuncSetAttribute(block_norm_backward_kernel<RES32, ACT32, VPT, kStages>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 static_cast<int>(smem));
      if (e != cudaSuccess) return e;
      block_norm_backward_kernel<RES32, ACT32, VPT, kStages><<<grid, threads, smem, s>>>(a);
      return cudaGetLastError();
    }
  }
  const size_t smem = VPT > 2 ? sizeof(float) * 3 * a.d : 0;
  if (smem) {
    const cudaError_t e = cudaFuncSetAttribute(block_norm_backward_kernel<RES32, ACT32, VPT, 0>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  block_norm_backward_kernel<RES32, ACT32, VPT, 0><<<grid, threads, smem, s>>>(a);
  return cudaGetLastError();
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
  if ((cfg->gate != MOE_GATE_NONE) != (gate != nullptr) || (!y && (w_post || gate)) || !w_pre != !h ||
      (h && (cfg->out == MOE_E4M3) != (h_scale != nullptr)) || (!h && h_scale) || (!r_out && !h))
    return MOE_ERR_INVALID_ARG;
  if (cfg->T == 0) return MOE_OK;
  if (!r) return MOE_ERR_INVALID_ARG;
  if (unaligned16(r) || unaligned16(y) || unaligned16(w_post) || unaligned16(w_pre) || unaligned16(r_out) ||
      unaligned16(h) || (cfg->gate != MOE_GATE_TOKEN && unaligned16(gate)))
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
  // few tokens: as many threads per row as it has vectors, for the shortest chain; many: four
  // vectors per thread, which keeps more loads in flight per thread and more CTAs on an SM
  const int vpt = a.nvec > 2048 ? 4 : (cfg->T <= 296 ? (a.nvec <= 1024 ? 1 : 2) : (a.nvec <= 64 ? 1 : 4));
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
  if ((cfg->gate != MOE_GATE_NONE) != (gate != nullptr) || (!y && (w_post || gate)) || !w_pre != !dh ||
      !y != !dy || (dgate && !gate) || (dw_post && !w_post) || (dw_pre && !w_pre) || !ws || !dr ||
      (w_pre && !r_out) || (!dh && !dr_out))
    return MOE_ERR_INVALID_ARG;
  if (unaligned16(r_out) || unaligned16(y) || unaligned16(w_post) || unaligned16(w_pre) || unaligned16(dh) ||
      unaligned16(dr_out) || unaligned16(dr) || unaligned16(dy) || unaligned16(ws) || unaligned16(dw_post) ||
      unaligned16(dw_pre) || (cfg->gate != MOE_GATE_TOKEN && (unaligned16(gate) || unaligned16(dgate))))
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < backward_workspace(*cfg)) return MOE_ERR_WORKSPACE;
  const BackwardShape sh = backward_shape(cfg->d_model);
  const int64_t turns = (static_cast<int64_t>(cfg->T) + sh.rows - 1) / sh.rows;
  const unsigned grid = static_cast<unsigned>(turns < kBackwardCtas ? turns : kBackwardCtas);
  NormGradArgs a{r_out, y, w_post, gate, w_pre, dh, dr_out, dr, dy, dgate};
  a.parts = reinterpret_cast<float*>(static_cast<char*>(ws) + kNormHeader);
  a.n_parts = static_cast<int>(grid) * sh.rows;
  a.want_pre = dw_pre != nullptr;
  a.want_post = dw_post != nullptr;
  a.want_gate = dgate != nullptr;
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
  if (grid) {
    const cudaError_t e = sh.vpt == 1 ? launch_backward<1>(a, res32, act32, grid, stream)
                                      : (sh.vpt == 2 ? launch_backward<2>(a, res32, act32, grid, stream)
                                                     : launch_backward<4>(a, res32, act32, grid, stream));
    if (e != cudaSuccess) return MOE_ERR_CUDA;
  }
  float* dgc = cfg->gate == MOE_GATE_CHANNEL ? static_cast<float*>(dgate) : nullptr;
  if (dw_pre || dw_post || dgc) {
    sum_parts_kernel<<<dim3((a.d + 31) / 32, 3), 256, 0, stream>>>(a.parts, a.n_parts, a.d, dw_pre, dw_post,
                                                                    dgc);
    return ok_or_cuda(cudaGetLastError());
  }
  return MOE_OK;
}

}  // extern "C"
