// grouped_product.cu -- products grouped by expert, one at a time, on the 5th-generation
// tensor cores (moe_grouped_gemm, _dgrad, _wgrad): for the rows r of group g
//   NT  y[r]  = a[r] W_g^T           inner index k
//   NN  da[r] = dy[r] W_g            inner index n
//   TN  dW_g  = sum_r dy[r]^T a[r]   inner index r: the rows of the group
// bf16 operands, or (NT) e4m3 operands with one fp32 scale per 128 inner elements of a row and
// per 128 x 128 block of a weight,
//   y[r, j] = sum_b s_a[r, b] s_w[j / 128, b] (sum over block b of a[r, i] w[j, i]),
// the inner sums on the tensor cores, the outer one in fp32 registers.
//
// Three kernels.  Each tile is one accumulator in TMEM, whose M side is its 128 lanes per CTA.
//
//   stream_kernel  NT (either type), NN on groups of few rows
//   pair_kernel    NT, NN in bf16 on larger groups; every TN
//   fold_kernel    NT in e4m3 on larger groups
//
// A tile whose K blocks fell to several CTAs is joined without waiting: each writes its fp32
// sums to the workspace, and the one that arrives last (a counter in the workspace header)
// adds all of them in K order, so that results do not depend on who was last.
//
// Launches may overlap the kernel before them in the stream: barriers, TMEM and descriptors are set
// up under its last CTAs, and launch_wait() stands before the first access to global memory (one
// bf16 token of 128 x 128: 5.2 -> 4.3 us; one token in eight of 64 groups, 4096 x 7168: 80.3 -> 77.7 us).
//
// Warp roles: 0 TMA producer, 1 MMA issuer (and TMEM owner), 2 scales (e4m3; in the fold
// kernel 2 and 3) or the zeroing of rows behind a group's last (TN), then the epilogue warps.  Producer and issuer
// keep the whole warp in their loops and let one elected lane issue: TMA and MMA instructions take
// their operands from uniform registers, and a branch on the lane number costs a transfer for
// each of them (pair kernel, TN, 8192 x 4096 x 7168: 1274 TFLOP/s so, 1460 uniform).
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include <atomic>
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"

namespace moe {
namespace {

enum Op { kNT = 0, kNN = 1, kTN = 2 };

constexpr int kMaxProductGroups = 1024;
constexpr uint32_t kBox = 64 * 128;             // one 64-row box of 128-byte rows
constexpr uint32_t kTileA = 2 * kBox;           // 128 x 128 bytes
constexpr int kCounterWord0 = 16;               // header words 16..63: four 8-bit counters each
constexpr int kMaxCounters = 192;
// bf16 operands: K blocks that the tensor cores sum before the sum is added to fp32 registers.  They
// cut each addend at 2^-23 of the largest, which leaves a sum about 1.1e-9 of its value short per
// element (7.9e-6 at 7168, which moves one bf16 rounding in 500); sums of 512 elements are short by
// 6e-7.  Adding m of them one after another in fp32 would round m times, the same way each time where
// the addends are alike: 2.4e-4 of a weight gradient over 2^23 rows.  kFoldSums of them are therefore
// added to one, and those to one another, at most (kFoldSums + m / kFoldSums) / 2^24 of the magnitudes.
// (TN, whose inner index are rows; the other products add 128 sums at most.)
constexpr int kFoldBlocks = 8, kFoldSums = 64;
constexpr int kLevel = kFoldBlocks * kFoldSums; // K blocks of such a sum
// Eight epilogue warps that keep 128 sums and 32 products per thread (pair and fold kernel):
// registers move from warps 0..3 to 4..11, 384 x 168 at launch = 128 x 40 + 256 x 232.
constexpr int kRegsLow = 40, kRegsHigh = 232;

constexpr int kScaleBlocks = 8;                 // stream kernel: K blocks of scales fetched at a time

struct ProductArgs {
  CUtensorMap wmap;             // NT, NN: weights [G][n][k]; TN: dy [rows][n]
  CUtensorMap tmap[4];          // NT, NN: token rows, boxes of 128, 64, 32, 16; TN: [0] a [rows][k]
  CUtensorMap omap;             // TN: dw [G][n][k], for stores
  const int32_t* offsets;       // null: one group of all n_rows rows
  int n_groups, n_rows;
  int m_total;                  // output index on the M side: NT n, NN k, TN n
  int n_total;                  // TN: k (the N side)
  int k_blocks;                 // NT, NN: 128-byte blocks of the inner index
  void* out;
  int ld_out;
  int* header;                  // workspace: status word, counters
  float* partials;              // workspace: fp32 sums of cut tiles
  const float *a_scale, *w_scale;   // e4m3: [rows][k_blocks], [G][m blocks][k_blocks]
  int w_scale_rows;             // 128-row blocks of a weight
};

// ------------------------------------------------------------------ scheduling
// Group row offsets, the groups that have rows in the order their tiles are taken, and the
// prefix of those groups' tile counts, in shared memory.
struct GroupTable {
  int32_t off[kMaxProductGroups + 1];
  int32_t pre[kMaxProductGroups + 1];
  int16_t ord[kMaxProductGroups];
  int16_t used;
};

// Tiles of group rows m: as few as hold at most `width` rows each, of nearly equal size.
__device__ __forceinline__ int token_tiles(int m, int width) { return (m + width - 1) / width; }
__device__ __forceinline__ int tile_rows_of(int m, int tiles, int unit) {
  return ((m + tiles - 1) / tiles + unit - 1) / unit * unit;
}

// Fills the table; returns the number of tiles (0, with the status set, for bad offsets).
// Groups with the widest tiles come first (in `classes` classes of width), so that CTAs which
// work side by side have tiles of about one size.  `per_group` > 0: that many tiles for every
// group, in order (TN).  All threads call it.
__device__ int build_groups(const ProductArgs& p, GroupTable& gt, int width, int unit, int classes, int m_blocks,
                            int per_group) {
  const int G = p.n_groups;
  for (int i = threadIdx.x; i <= G; i += blockDim.x)
    gt.off[i] = p.offsets ? p.offsets[i] : (i ? p.n_rows : 0);
  __syncthreads();
  int bad = 0;
  for (int i = threadIdx.x; i < G; i += blockDim.x)
    bad |= gt.off[i] < 0 || gt.off[i + 1] < gt.off[i] || gt.off[i + 1] > p.n_rows;
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) record_status(p.header, kStatusDeviceIndex);
    return 0;
  }
  if (per_group) return per_group * G;
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int count = 0, carry = 0;
    for (int cls = classes - 1; cls >= 0; --cls)
      for (int b = 0; b < G; b += 32) {
        const int g = b + lane;
        const int m = g < G ? gt.off[g + 1] - gt.off[g] : 0;
        int tiles = 0;
        bool mine = m > 0;
        if (mine) {
          tiles = token_tiles(m, width);
          mine = classes == 1 || (tile_rows_of(m, tiles, unit) * classes - 1) / width == cls;
        }
        const uint32_t mask = __ballot_sync(0xffffffffu, mine);
        if (!mask) continue;
        int incl = mine ? tiles * m_blocks : 0;
        const int c = incl;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += v;
        }
        if (mine) {
          const int at = count + __popc(mask & ((1u << lane) - 1u));
          gt.ord[at] = static_cast<int16_t>(g);
          gt.pre[at] = carry + incl - c;
        }
        count += __popc(mask);
        carry += __shfl_sync(0xffffffffu, incl, 31);
      }
    if (lane == 0) {
      gt.pre[count] = carry;
      gt.used = static_cast<int16_t>(count);
    }
  }
  __syncthreads();
  return gt.pre[gt.used];
}

struct Tile {
  int g, mb, nb;                // group, M block, N block (TN)
  int row0, rows;               // NT, NN: first token row and rows; TN: the group's rows
};

// Tile t of the NT / NN products: group by group; inside a group, runs of `run` weight blocks
// sweep all token tiles before the next, so that CTAs at work together share both operands.
__device__ __forceinline__ Tile token_tile(const GroupTable& gt, int t, int width, int unit, int m_blocks,
                                           int run) {
  int lo = 0, hi = gt.used;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (gt.pre[mid] <= t) lo = mid;
    else hi = mid;
  }
  Tile c;
  c.g = gt.ord[lo];
  const int m = gt.off[c.g + 1] - gt.off[c.g];
  const int nt = token_tiles(m, width), per = tile_rows_of(m, nt, unit);
  const int local = t - gt.pre[lo];
  const int strip = local / (nt * run);
  const int wide = min(run, m_blocks - strip * run);
  const int rem = local - strip * nt * run;
  const int tok = rem / wide;
  c.mb = strip * run + rem - tok * wide;
  c.nb = 0;
  c.row0 = gt.off[c.g] + tok * per;
  c.rows = min(per, m - tok * per);
  return c;
}
// Tile t of the TN product: runs of `run` M blocks sweep all N blocks.
__device__ __forceinline__ Tile grad_tile(const GroupTable& gt, int t, int m_blocks, int n_blocks, int run) {
  Tile c;
  c.g = t / (m_blocks * n_blocks);
  const int local = t - c.g * m_blocks * n_blocks;
  const int strip = local / (n_blocks * run);
  const int wide = min(run, m_blocks - strip * run);
  const int rem = local - strip * n_blocks * run;
  c.nb = rem / wide;
  c.mb = strip * run + rem - c.nb * wide;
  c.row0 = gt.off[c.g];
  c.rows = gt.off[c.g + 1] - c.row0;
  return c;
}

// A run of K blocks of one tile.
struct Piece {
  int tile, kb0, kb1;
};

// Stream kernel: the K blocks of all tiles as one sequence, cut into equal pieces, one per CTA --
// or, where there are fewer than half as many tiles as CTAs, every tile cut into the same number
// of parts, one per CTA, so that no CTA has to join two tiles.  Such a part has min_kb K blocks at
// least, 512 inner elements: with fewer the join of more parts costs more than it saves (one row,
// n = 512, k = 7168: bf16 19.1 us with parts of 2 blocks, 12.9 of 4, 11.3 of 8, 12.5 of 16; n = 7168,
// k = 2048, e4m3 10.1 us with 2 or 3, 9.6 with 4, 10.4 with 8).
struct EvenShare {
  int kb, sharers, parts;       // parts > 0: of every tile
  long long total, u, u1;

  __device__ __forceinline__ EvenShare(int me, int n, int n_tiles, int kb_, int min_kb) : kb(kb_) {
    total = static_cast<long long>(n_tiles) * kb;
    sharers = (total + 1) / 2 < n ? static_cast<int>((total + 1) / 2) : n;
    parts = 0;
    u = u1 = 0;
    if (n_tiles > 0 && 2 * n_tiles <= n) {
      parts = max(1, min(n / n_tiles, kb / min_kb));
      if (me < n_tiles * parts) {
        const long long b = static_cast<long long>(me / parts) * kb;
        u = b + kb * (me % parts) / parts;
        u1 = b + kb * (me % parts + 1) / parts;
      }
    } else if (me < sharers) {
      u = total * me / sharers;
      u1 = total * (me + 1) / sharers;
    }
  }
  __device__ __forceinline__ bool next(Piece& c) {
    if (u >= u1) return false;
    const long long t = u / kb;
    c.tile = static_cast<int>(t);
    c.kb0 = static_cast<int>(u - t * kb);
    const long long left = u1 - u;
    c.kb1 = left < kb - c.kb0 ? c.kb0 + static_cast<int>(left) : kb;
    u += c.kb1 - c.kb0;
    return true;
  }
  __device__ __forceinline__ bool cut(const Piece& c) const { return c.kb1 - c.kb0 < kb; }
  // First and last CTA with a piece of tile t.
  __device__ __forceinline__ int owner(long long unit) const {
    return static_cast<int>(((unit + 1) * sharers - 1) / total);
  }
  __device__ __forceinline__ void owners(int t, int& first, int& last) const {
    if (parts) {
      first = t * parts;
      last = first + parts - 1;
    } else {
      const long long b = static_cast<long long>(t) * kb;
      first = owner(b);
      last = owner(b + kb - 1);
    }
  }
};

// Pair and fold kernels: whole tiles me, me + n, ...; the tiles of a last round that would leave
// at least half of the pairs (CTAs) idle are cut into `parts` equal runs of K blocks, one per pair.
// A join costs about what min_kb K blocks do, so a part has that many at least, and there are at
// most four.  Measured: 24 in the pair kernel; 14 in the fold kernel, whose K blocks are twice as
// long (128 rows, n = 4096, k = 7168: 29.0 us in two parts, 25.0 in four; k = 2048 in two parts 20.3
// us against 18.0 whole).
struct RoundShare {
  int me, n, kb, whole, parts, cut_tiles, at;
  bool part_left;               // this pair's part of a cut tile is still to come

  __device__ __forceinline__ RoundShare(int me_, int n_, int n_tiles, int kb_, bool may_cut, int min_kb)
      : me(me_), n(n_), kb(kb_), whole(n_tiles), parts(1), cut_tiles(0), at(me_) {
    const int rest = n_tiles % n;
    if (may_cut && rest > 0) {
      parts = min(min(n / rest, kb / min_kb), 4);
      if (parts > 1) {
        cut_tiles = rest;
        whole = n_tiles - rest;
      }
    }
    part_left = me < cut_tiles * parts;
  }
  __device__ __forceinline__ bool next(Piece& c) {
    if (at < whole) {
      c.tile = at;
      c.kb0 = 0;
      c.kb1 = kb;
      at += n;
      return true;
    }
    if (!part_left) return false;
    part_left = false;
    const int q = me / parts, r = me - q * parts;
    c.tile = whole + q;
    c.kb0 = kb * r / parts;
    c.kb1 = kb * (r + 1) / parts;
    return true;
  }
  __device__ __forceinline__ bool cut(const Piece& c) const { return c.tile >= whole; }
  __device__ __forceinline__ void owners(int t, int& first, int& last) const {
    first = (t - whole) * parts;
    last = first + parts - 1;
  }
};

// ------------------------------------------------------------------ epilogue pieces
// A warp's 16 tokens x 32 output columns (lane = column) to rows of `out`: through the warp's
// shared-memory stage, so that global memory sees 16-byte pieces of rows.  Tokens at or past
// `rows` and columns at or past `cols` are skipped (cols a multiple of 8).
template <typename T>
__device__ __forceinline__ void store_transposed(T* out, size_t ld, int rows, int cols, const float* v,
                                                 void* stage_raw, int lane) {
  T* stage = static_cast<T*>(stage_raw);
  constexpr int kElems = 16 / static_cast<int>(sizeof(T)), kVecs = 32 / kElems;
  constexpr int kRun = 1024 / (32 * static_cast<int>(sizeof(T)));  // tokens that fit 1 KB: 16 or 8
#pragma unroll
  for (int i0 = 0; i0 < 16; i0 += kRun) {
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      if constexpr (sizeof(T) == 4) stage[i * 32 + lane] = v[i0 + i];
      else stage[i * 32 + lane] = __float2bfloat16_rn(v[i0 + i]);
    }
    __syncwarp();
#pragma unroll
    for (int q = lane; q < kRun * kVecs; q += 32) {
      const int r = q / kVecs, c = (q % kVecs) * kElems;
      if (i0 + r < rows && c < cols)
        *reinterpret_cast<uint4*>(out + (i0 + r) * ld + c) = *reinterpret_cast<const uint4*>(stage + r * 32 + c);
    }
    __syncwarp();
  }
}
// A warp's 32 rows (lane = row) x 16 columns to rows of `out`, likewise; 32 bytes of a row at a
// time through 1 KB.
template <typename T>
__device__ __forceinline__ void store_direct(T* out, size_t ld, int rows, int cols, const float* v,
                                             void* stage_raw, int lane) {
  constexpr int kElems = 16 / static_cast<int>(sizeof(T));         // per 16-byte unit
  uint4* stage = static_cast<uint4*>(stage_raw);
#pragma unroll
  for (int c0 = 0; c0 < 16; c0 += 2 * kElems) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float* x = v + c0 + u * kElems;
      uint4 q;
      if constexpr (sizeof(T) == 4) {
        q = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
      } else {
        __nv_bfloat162* b = reinterpret_cast<__nv_bfloat162*>(&q);
#pragma unroll
        for (int e = 0; e < 4; ++e) b[e] = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
      }
      stage[lane * 2 + (u ^ ((lane >> 2) & 1))] = q;               // spread over the banks
    }
    __syncwarp();
#pragma unroll
    for (int i = lane; i < 64; i += 32) {
      const int r = i >> 1, u = i & 1;
      if (r < rows && c0 + u * kElems < cols)
        *reinterpret_cast<uint4*>(out + r * ld + c0 + u * kElems) = stage[r * 2 + (u ^ ((r >> 2) & 1))];
    }
    __syncwarp();
  }
}

// Barrier between the epilogue warps of a CTA, bounded like every other wait.
struct EpilogueSync {
  uint64_t* bar;
  volatile int* abort_flag;
  int* status;
  uint32_t parity = 0;
  __device__ __forceinline__ bool operator()(int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
    const bool ok = mbar_poll_warp(bar, parity, abort_flag, status);
    parity ^= 1u;
    return ok;
  }
};

// After the epilogue warps have written a cut tile's sums: counts this CTA in and says
// whether it is the last of `n`.  False in `ok` if a wait ran out.
__device__ __forceinline__ bool arrive_last(int* header, int counter, int n, EpilogueSync& sync, int* flag,
                                            bool first_thread, int lane, bool& ok) {
  __threadfence();                                   // this thread's sums before the count
  ok = sync(lane);
  if (!ok) return false;
  if (first_thread) {
    unsigned* word = reinterpret_cast<unsigned*>(header) + kCounterWord0 + (counter >> 2);
    const int sh = 8 * (counter & 3);
    const unsigned before = (atomicAdd(word, 1u << sh) >> sh) & 0xFFu;
    const bool last = before == static_cast<unsigned>(n - 1);
    if (last) atomicSub(word, static_cast<unsigned>(n) << sh);   // left zero for the next call
    *flag = last;
  }
  ok = sync(lane);
  if (!ok) return false;
  const bool last = *reinterpret_cast<volatile int*>(flag) != 0;
  if (last) __threadfence();                         // the others' sums after the count
  return last;
}

// A cut tile's fp32 sums in the workspace: four consecutive columns of a row together, rows next
// to one another, [columns / 4][128 rows][4].  `slot` is this thread's row of one part.
__device__ __forceinline__ void write_part(float* slot, int col, const float* v) {   // 4 columns
  __stcg(reinterpret_cast<float4*>(slot + col * 128), make_float4(v[0], v[1], v[2], v[3]));
}
// N columns from `col` of which `valid` count: the sums of parts first .. last, added in order,
// with kDeep parts' loads in flight.
template <int N, int kDeep, class Slot>
__device__ __forceinline__ void join_parts(float* v, Slot slot, int first, int last, int col, int valid) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.f;
  for (int part = first; part <= last; part += kDeep) {
    float4 x[kDeep][N / 4];
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      const float* from = slot(min(part + d, last)) + col * 128;
#pragma unroll
      for (int i = 0; i < N / 4; ++i)
        x[d][i] = part + d <= last && 4 * i < valid ? __ldcg(reinterpret_cast<const float4*>(from + i * 512))
                                                    : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int d = 0; d < kDeep; ++d)
#pragma unroll
      for (int i = 0; i < N / 4; ++i) {
        v[4 * i] += x[d][i].x;
        v[4 * i + 1] += x[d][i].y;
        v[4 * i + 2] += x[d][i].z;
        v[4 * i + 3] += x[d][i].w;
      }
  }
}

// acc += the warp's first `cols` of 128 columns in TMEM, 16 at a time, each load under way during the
// additions of the one before.  (A second form for all 128, without the tests, was 2% slower.)
__device__ __forceinline__ void add_columns(uint32_t tb, int cols, f32x2 (&acc)[64]) {
  uint32_t v[2][16];
  tmem_ld16_begin(tb, v[0]);
  tmem_ld_end(v[0]);
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const bool more = q < 7 && (q + 1) * 16 < cols;
    if (more) tmem_ld16_begin(tb + (q + 1) * 16, v[(q + 1) & 1]);
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      f32x2& a = acc[(q * 16 + i) / 2];
      a = add2(a, pack2(v[q & 1][i], v[q & 1][i + 1]));
    }
    if (!more) break;
    tmem_ld_end(v[(q + 1) & 1]);
  }
}

// The warp's first `cols` of 128 columns, for the level above of a very long sum: acc is put (first) or
// added to a thread's place in the workspace and is zero afterwards, or takes what is there.
__device__ __forceinline__ void lay_aside(float* place, int cols, bool first, f32x2 (&acc)[64]) {
#pragma unroll
  for (int i = 0; i < 128; i += 4) {
    if (i >= cols) break;
    float4* at = reinterpret_cast<float4*>(place + i * 128);
    const float4 x = first ? make_float4(0.f, 0.f, 0.f, 0.f) : __ldcg(at);
    const float2 a = unpack2(acc[i / 2]), b = unpack2(acc[i / 2 + 1]);
    __stcg(at, make_float4(x.x + a.x, x.y + a.y, x.z + b.x, x.w + b.y));
    acc[i / 2] = acc[i / 2 + 1] = both2(0.f);
  }
}
__device__ __forceinline__ void take_back(const float* place, int cols, f32x2 (&acc)[64]) {
#pragma unroll
  for (int i = 0; i < 128; i += 4) {
    if (i >= cols) break;
    const float4 x = __ldcg(reinterpret_cast<const float4*>(place + i * 128));
    acc[i / 2] = add2(acc[i / 2], pack2(x.x, x.y));
    acc[i / 2 + 1] = add2(acc[i / 2 + 1], pack2(x.z, x.w));
  }
}

// Two finite scales whose product is not: the factor of a block has to be finite, for the block's
// products may be zeros.  (Multiplying by one scale after the other where it is not costs registers of
// the fold's loop even if no call needs it: 291 -> 321 us, 8192 rows, n = 4096, k = 7168.)
__device__ __forceinline__ bool scales_overflow(float a, float b) {
  return isinf(a * b) && !isinf(a) && !isinf(b);
}

// ------------------------------------------------------------------ stream kernel
// Groups of few rows: every weight byte is used for a handful of tokens, so HBM bounds it and the
// tile is made for a steady stream.  The weights are the M side (256 rows per tile, two MMAs), the
// tokens the N side (16 or 32), so that a token costs a narrow MMA and not a padded one.  All
// tiles' K blocks form one sequence that is cut evenly over the SMs, whatever the groups are: every
// SM streams the same number of bytes, five stages of 32 KB of weights ahead.
//
// Measured: 64 groups, n = 7168, k = 2048, 512 rows: 6.43 TB/s (0.98 of a copy); one token's 8
// groups of n = 4096, k = 7168 78 us (6.0 TB/s: about 6 us are the start, first loads and the
// join of the cut tiles).  One e4m3 token, n = 7168, k = 2048: 9.6 us, latency: the start of
// the CTA and its first loads, four K blocks, the join of the parts.
template <bool F8, int OP>
struct StreamCfg {
  static constexpr int kMB = 2;                                   // 128-row weight blocks per tile
  static constexpr int kNTok = 32;
  static constexpr uint32_t kA = kMB * kTileA;
  static constexpr uint32_t kStage = kA + kNTok * 128;
  static constexpr int kStages = 5;
  static constexpr int kCols = kMB * kNTok;                       // TMEM columns per buffer
  static constexpr int kBufs = F8 ? 8 : 2;                        // e4m3: one per K block in flight
  static constexpr uint32_t kTmem = F8 ? 512 : 128;
  static constexpr uint32_t kScales = F8 ? 2 * kScaleBlocks * kMB * kNTok * 4 : 0;
  static constexpr uint32_t kStaging = 4 * 2048;
  static constexpr size_t kTileFloats = static_cast<size_t>(kMB) * 128 * kNTok;
  static constexpr uint32_t kSmem =
      1024 + kStages * kStage + 1024 + kScales + kStaging + ((sizeof(GroupTable) + 15) & ~15u);
  static_assert(kBufs * kCols <= static_cast<int>(kTmem) && kSmem <= 227 * 1024, "budget");
};

template <bool F8, int OP, typename OUT>
__global__ void __launch_bounds__(224, 1) stream_kernel(const __grid_constant__ ProductArgs p) {
  using C = StreamCfg<F8, OP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(tiles + C::kStages * C::kStage);
  uint64_t* empty_bar = full_bar + C::kStages;
  uint64_t* tfull_bar = empty_bar + C::kStages;       // [kBufs] accumulators written
  uint64_t* tempty_bar = tfull_bar + C::kBufs;        // [kBufs] accumulators read
  uint64_t* sfull_bar = tempty_bar + C::kBufs;        // [2] scales of kScaleBlocks K blocks
  uint64_t* sempty_bar = sfull_bar + 2;
  uint64_t* epi_bar = sempty_bar + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(epi_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* last_flag = reinterpret_cast<int*>(tmem_slot + 2);
  float* scales = reinterpret_cast<float*>(tiles + C::kStages * C::kStage + 1024);
  uint8_t* staging = reinterpret_cast<uint8_t*>(scales) + C::kScales;
  GroupTable& gt = *reinterpret_cast<GroupTable*>(staging + C::kStaging);
  int* status = p.header;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full_bar[i], 1);
      mbar_init(&empty_bar[i], 1);
    }
    for (int i = 0; i < C::kBufs; ++i) {
      mbar_init(&tfull_bar[i], 1);
      mbar_init(&tempty_bar[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sfull_bar[i], 1);
      mbar_init(&sempty_bar[i], 4);
    }
    mbar_init(epi_bar, 4);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.wmap);
    tma_prefetch_desc(&p.tmap[2]);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmem);
    tmem_relinquish();
  }
  launch_wait();
  launch_begin_next();
  constexpr int kRun = F8 ? 1 : kFoldBlocks;     // K blocks per accumulator
  const int m_blocks = (p.m_total + 128 * C::kMB - 1) / (128 * C::kMB);
  const int n_tiles = build_groups(p, gt, C::kNTok, 16, 1, m_blocks, 0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  EvenShare sched(blockIdx.x, gridDim.x, n_tiles, p.k_blocks, F8 ? 4 : 8);
  Piece c;

  if (warp == 0) {
    // ---------------------------------------------------------- TMA producer
    const bool elected = elect_one();
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    while (ok && sched.next(c)) {
      const Tile t = token_tile(gt, c.tile, C::kNTok, 16, m_blocks, 1);
      const int box = t.rows > 16 ? 32 : 16;
      const CUtensorMap* tm = &p.tmap[box == 32 ? 2 : 3];
      for (int kb = c.kb0; kb < c.kb1; ++kb) {
        ok = mbar_poll_warp(&empty_bar[stage], phase ^ 1u, abort_flag, status);
        if (!ok) break;
        uint8_t* st = tiles + stage * C::kStage;
        uint64_t* bar = &full_bar[stage];
        const int kx = kb * (F8 ? 128 : 64);
        if (elected) {
          mbar_arrive_expect_tx(bar, C::kA + box * 128);
          if (OP == kNT) {
#pragma unroll
            for (int j = 0; j < C::kMB; ++j)
              tma_load_3d(st + j * kTileA, &p.wmap, bar, kx, (t.mb * C::kMB + j) * 128, t.g);
          } else {
#pragma unroll
            for (int j = 0; j < 2 * C::kMB; ++j)
              tma_load_3d(st + j * kBox, &p.wmap, bar, t.mb * C::kMB * 128 + j * 64, kx, t.g);
          }
          tma_load_2d(st + C::kA, tm, bar, kx, t.row0);
        }
        __syncwarp();
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    const bool elected = elect_one();
    int stage = 0;
    uint32_t phase = 0, it = 0;                 // accumulator buffers used so far
    bool ok = true;
    while (ok && sched.next(c)) {
      const Tile t = token_tile(gt, c.tile, C::kNTok, 16, m_blocks, 1);
      const int n_pad = (t.rows + 15) & ~15;
      const uint32_t idesc = F8 ? idesc_e4m3_f32(128, n_pad)
                                : (idesc_bf16_f32(128, n_pad) | (OP == kNN ? kIdescAMajorMN : 0u));
      uint32_t d0 = 0, b = 0;
      for (int kb = c.kb0; kb < c.kb1; ++kb) {
        const int at = (kb - c.kb0) % kRun;
        if (at == 0) {                          // a fresh accumulator buffer
          b = it % C::kBufs;
          ok = mbar_poll_warp(&tempty_bar[b], ((it / C::kBufs) & 1u) ^ 1u, abort_flag, status);
          if (!ok) break;
          d0 = tmem + b * C::kCols;
          ++it;
        }
        ok = mbar_poll_warp(&full_bar[stage], phase, abort_flag, status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t sa = smem_u32(tiles) + stage * C::kStage, sb = sa + C::kA;
        if (elected) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t bd = umma_desc_sw128(sb + kk * 32);
            const uint32_t accumulate = (kk || at) ? 1u : 0u;
#pragma unroll
            for (int j = 0; j < C::kMB; ++j) {
              const uint32_t aj = sa + j * kTileA;
              if (F8) umma_e4m3(d0 + j * C::kNTok, umma_desc_sw128(aj + kk * 32), bd, idesc, accumulate);
              else if (OP == kNT) umma_bf16(d0 + j * C::kNTok, umma_desc_sw128(aj + kk * 32), bd, idesc, accumulate);
              else umma_bf16(d0 + j * C::kNTok, umma_desc_mn_sw128(aj + kk * 2048), bd, idesc, accumulate);
            }
          }
          umma_commit(&empty_bar[stage]);
          if (at == kRun - 1 || kb + 1 == c.kb1) umma_commit(&tfull_bar[b]);
        }
        __syncwarp();
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp == 2) {
    // ---------------------------------------------------------- scales (e4m3)
    // For kScaleBlocks K blocks at a time: lane = token fetches its scales, multiplies them by
    // the weight blocks' and leaves the products as [K block][weight block][token].
    if (F8) {
      uint32_t it = 0;
      bool ok = true, over = false;
      while (ok && sched.next(c)) {
        const Tile t = token_tile(gt, c.tile, C::kNTok, 16, m_blocks, 1);
        const float* sa = p.a_scale + static_cast<size_t>(t.row0 + min(lane, t.rows - 1)) * p.k_blocks;
        for (int kb = c.kb0; kb < c.kb1; kb += kScaleBlocks, ++it) {
          ok = mbar_poll_warp(&sempty_bar[it & 1], ((it >> 1) & 1u) ^ 1u, abort_flag, status);
          if (!ok) break;
          float* dst = scales + (it & 1) * (kScaleBlocks * C::kMB * C::kNTok);
          float s[kScaleBlocks], ws[C::kMB][kScaleBlocks];
#pragma unroll
          for (int q = 0; q < kScaleBlocks; ++q) {
            const int at = min(kb + q, c.kb1 - 1);
            s[q] = __ldg(sa + at);
#pragma unroll
            for (int j = 0; j < C::kMB; ++j)
              ws[j][q] = __ldg(p.w_scale + (static_cast<size_t>(t.g) * p.w_scale_rows +
                                            min(t.mb * C::kMB + j, p.w_scale_rows - 1)) * p.k_blocks + at);
          }
#pragma unroll
          for (int q = 0; q < kScaleBlocks; ++q)
#pragma unroll
            for (int j = 0; j < C::kMB; ++j) dst[(q * C::kMB + j) * C::kNTok + lane] = s[q] * ws[j][q];
          __syncwarp();
          if (lane == 0) mbar_arrive(&sfull_bar[it & 1]);
          float largest = 0.f;
#pragma unroll
          for (int q = 0; q < kScaleBlocks; ++q)
#pragma unroll
            for (int j = 0; j < C::kMB; ++j) largest = fmaxf(largest, fabsf(s[q] * ws[j][q]));
          if (isinf(largest))
#pragma unroll
            for (int q = 0; q < kScaleBlocks; ++q)
#pragma unroll
              for (int j = 0; j < C::kMB; ++j) over |= scales_overflow(s[q], ws[j][q]);
        }
      }
      if (over) record_status(status, kStatusDeviceValue);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------- epilogue
    const int sub = warp & 3;                   // TMEM lane quadrant
    const int m_local = sub * 32 + lane;
    uint8_t* stg = staging + sub * 2048;
    EpilogueSync sync{epi_bar, abort_flag, status};
    uint32_t it = 0, sit = 0;
    bool ok = true;
    while (ok && sched.next(c)) {
      const Tile t = token_tile(gt, c.tile, C::kNTok, 16, m_blocks, 1);
      float acc[C::kMB][2][16];
#pragma unroll
      for (int j = 0; j < C::kMB; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[j][0][i] = acc[j][1][i] = 0.f;
      if (F8) {
        for (int kb = c.kb0; kb < c.kb1; ++kb, ++it) {
          const uint32_t b = it % C::kBufs;
          const int q = (kb - c.kb0) % kScaleBlocks;
          ok = (q != 0 || mbar_poll_warp(&sfull_bar[sit & 1], (sit >> 1) & 1u, abort_flag, status)) &&
               mbar_poll_warp(&tfull_bar[b], (it / C::kBufs) & 1u, abort_flag, status);
          if (!ok) break;
          tc_fence_after();
          const uint32_t tb = tmem + (static_cast<uint32_t>(sub * 32) << 16) + b * C::kCols;
          const float* sc = scales + ((sit & 1) * kScaleBlocks + q) * (C::kMB * C::kNTok);
#pragma unroll
          for (int j = 0; j < C::kMB; ++j) {
            float v0[16], v1[16];
            if (t.rows > 16) tmem_ld16x2(tb + j * C::kNTok, tb + j * C::kNTok + 16, v0, v1);
            else tmem_ld16(tb + j * C::kNTok, v0);
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[j][0][i] = fmaf(sc[j * C::kNTok + i], v0[i], acc[j][0][i]);
            if (t.rows > 16)
#pragma unroll
              for (int i = 0; i < 16; ++i) acc[j][1][i] = fmaf(sc[j * C::kNTok + 16 + i], v1[i], acc[j][1][i]);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&tempty_bar[b]);
            if (q == kScaleBlocks - 1 || kb + 1 == c.kb1) mbar_arrive(&sempty_bar[sit & 1]);
          }
          if (q == kScaleBlocks - 1 || kb + 1 == c.kb1) ++sit;
        }
        if (!ok) break;
      } else {
        for (int kb = c.kb0; kb < c.kb1; kb = c.kb1 - kb > kRun ? kb + kRun : c.kb1, ++it) {
          const uint32_t b = it % C::kBufs;
          ok = mbar_wait_warp(&tfull_bar[b], (it / C::kBufs) & 1u, abort_flag, status);
          if (!ok) break;
          tc_fence_after();
          const uint32_t tb = tmem + (static_cast<uint32_t>(sub * 32) << 16) + b * C::kCols;
#pragma unroll
          for (int j = 0; j < C::kMB; ++j) {
            float v0[16], v1[16];
            if (t.rows > 16) tmem_ld16x2(tb + j * C::kNTok, tb + j * C::kNTok + 16, v0, v1);
            else tmem_ld16(tb + j * C::kNTok, v0);
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[j][0][i] += v0[i];
            if (t.rows > 16)
#pragma unroll
              for (int i = 0; i < 16; ++i) acc[j][1][i] += v1[i];
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty_bar[b]);
        }
        if (!ok) break;
      }
      if (sched.cut(c)) {
        int first, last;
        sched.owners(c.tile, first, last);
        auto slot = [&](int cta) {
          return p.partials + (static_cast<size_t>(cta) * 2 + (cta == first ? 1 : 0)) * C::kTileFloats + m_local * 4;
        };
        float* mine = slot(blockIdx.x);
#pragma unroll
        for (int j = 0; j < C::kMB; ++j)
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            if (i < t.rows) write_part(mine, j * C::kNTok + i, &acc[j][i >> 4][i & 15]);
        if (!arrive_last(p.header, first, last - first + 1, sync, last_flag, m_local == 0, lane, ok)) continue;
#pragma unroll
        for (int j = 0; j < C::kMB; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (h * 16 < t.rows)
              join_parts<16, 4>(acc[j][h], slot, first, last, j * C::kNTok + h * 16, t.rows - h * 16);
      }
#pragma unroll
      for (int j = 0; j < C::kMB; ++j) {
        const int col0 = (t.mb * C::kMB + j) * 128 + sub * 32;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (h * 16 < t.rows && col0 < p.m_total)
            store_transposed<OUT>(static_cast<OUT*>(p.out) + static_cast<size_t>(t.row0 + h * 16) * p.ld_out + col0,
                                  p.ld_out, t.rows - h * 16, p.m_total - col0, acc[j][h], stg, lane);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, C::kTmem);
}

// ------------------------------------------------------------------ pair kernel
// bf16 on larger groups, and every TN product: two CTAs share 256 x 256 tiles (cta_group::2), each
// staging 128 rows of either operand, which halves the shared-memory fill per flop of
// 128-row tiles.  The weight index is the M side and the group's tokens are the N side in steps of
// 32, so a short group costs a narrow MMA; TN has the weight's n index on M, its k index on N.
// Whole rounds of tiles go to the pairs in an order that keeps a few weight blocks and token
// tiles in L2; the K blocks of a partial last round are cut.  Two accumulators of kFoldBlocks K
// blocks take turns: eight epilogue warps add one up in registers, 128 columns per thread, and
// store a finished tile, under the MMAs of the next.
//
// Measured: one group of 8192 rows, n = 4096, k = 7168: 325 us for NT (1480 TFLOP/s), 336 for NN,
// 350-440 for TN.  Alone on a cool GPU the tensor pipe is busy in 93% of the cycles (TN with fp32
// output: 77%); in a loop the 1000 W power limit holds the clock near 1.2 GHz.  fp32 output: 335-357, 370-390 and 430-470.  One
// accumulator for the whole sum, stored as bf16, took 310, 317 and 335-400.  TN of 32 groups x 256
// rows, n = 7168, k = 2048, fp32: 460 us; a tile has four K blocks there for 256 KB of sums, so the
// stores bound it.
constexpr size_t kPartFloats = 128 * 256;       // a CTA's sums of a cut tile

template <int OP>
struct PairCfg {
  static constexpr int kWidth = 256;                              // tokens (TN: columns) per tile
  static constexpr uint32_t kStage = 2 * kTileA;                  // 128 rows of either operand
  static constexpr int kStages = OP == kTN ? 5 : 6;
  static constexpr int kBufs = 2;                                 // accumulators of 256 columns
  static constexpr int kCols = 256;
  static constexpr int kEpi = 8, kEpi0 = 4;                       // epilogue warps, the first of them
  static constexpr int kThreads = 32 * (kEpi0 + kEpi);
  static constexpr uint32_t kWarpStage = OP == kTN ? 4096 : 2048; // TN: one box of a store
  static constexpr uint32_t kStaging = kEpi * kWarpStage;
  static constexpr uint32_t kSmem =
      1024 + kStages * kStage + 1024 + kStaging + ((sizeof(GroupTable) + 15) & ~15u);
  static_assert(kSmem <= 227 * 1024, "budget");
};

// Whether K block kb of a TN tile ends inside a 16-row step of the MMA.
__device__ __forceinline__ bool ragged_block(int rows, int kb) {
  const int left = rows - kb * 64;
  return left < 64 && (left & 15) != 0;
}

// LONG (TN): sums of more than kFoldSums partial sums.
template <int OP, typename OUT, bool LONG>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PairCfg<OP>::kThreads, 1)
    pair_kernel(const __grid_constant__ ProductArgs p) {
  constexpr int kRun = kFoldBlocks;              // K blocks per accumulator
  using C = PairCfg<OP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(tiles + C::kStages * C::kStage);   // the leader's counts
  uint64_t* empty_bar = full_bar + C::kStages;
  uint64_t* land_bar = empty_bar + C::kStages;        // TN: this CTA's loads of a stage
  uint64_t* tfull_bar = land_bar + C::kStages;
  uint64_t* tempty_bar = tfull_bar + C::kBufs;        // the leader's counts
  uint64_t* epi_bar = tempty_bar + C::kBufs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(epi_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* last_flag = reinterpret_cast<int*>(tmem_slot + 2);
  uint8_t* staging = tiles + C::kStages * C::kStage + 1024;
  GroupTable& gt = *reinterpret_cast<GroupTable*>(staging + C::kStaging);
  int* status = p.header;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full_bar[i], OP == kTN ? 2 : 1);     // TN: see the producer
      mbar_init(&empty_bar[i], 1);
      mbar_init(&land_bar[i], 1);
    }
    for (int i = 0; i < C::kBufs; ++i) {
      mbar_init(&tfull_bar[i], 1);
      mbar_init(&tempty_bar[i], 2 * C::kEpi);          // both CTAs' epilogue warps
    }
    mbar_init(epi_bar, C::kEpi);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.wmap);
    tma_prefetch_desc(&p.tmap[0]);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  launch_wait();
  launch_begin_next();
  const int m_blocks = (p.m_total + 255) / 256;
  const int n_blocks = OP == kTN ? (p.n_total + 255) / 256 : 1;
  const int n_tiles = build_groups(p, gt, C::kWidth, 32, 8, m_blocks, OP == kTN ? m_blocks * n_blocks : 0);
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;
  // K blocks of a tile (TN: of the only group; with several, tiles differ and are not cut)
  const int kb_all = OP == kTN ? (n_tiles ? (gt.off[1] - gt.off[0] + 63) / 64 : 1) : p.k_blocks;
  RoundShare sched(pair, n_pairs, n_tiles, kb_all, OP != kTN || p.n_groups == 1, 24);
  // The next piece of work and its tile; a whole TN tile has its own group's K blocks.
  Piece c;
  Tile t;
  bool cut = false;
  auto fetch = [&]() {
    if (!sched.next(c)) return false;
    t = OP == kTN ? grad_tile(gt, c.tile, m_blocks, n_blocks, 8)
                  : token_tile(gt, c.tile, C::kWidth, 32, m_blocks, 8);
    cut = sched.cut(c);
    if (OP == kTN && !cut) c.kb1 = (t.rows + 63) / 64;
    return true;
  };
  // TN: columns of the tile, and the MMA's N
  auto grad_cols = [&]() { return min(256, p.n_total - t.nb * 256); };
  auto grad_n = [&]() { return grad_cols() > 128 ? 256 : 128; };

  if (warp < C::kEpi0) {
    regs_down<kRegsLow>();                       // (one instruction for the whole warpgroup)
    if (warp == 0) {
      // ---------------------------------------------------------- TMA producer (both CTAs)
      const bool elected = elect_one();
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      while (ok && fetch()) {
        const int m0 = t.mb * 256 + rank * 128;
        for (int kb = c.kb0; kb < c.kb1; ++kb) {
          ok = mbar_poll_warp(&empty_bar[stage], phase ^ 1u, abort_flag, status);
          if (!ok) break;
          uint8_t* st = tiles + stage * C::kStage;
          uint8_t* bt = st + kTileA;
          if (OP == kTN) {
            // loads count on the leader's barrier, which the leader's producer arrives on twice;
            // those of a ragged last block count on this CTA's own, and the CTAs' zeroing warps
            // arrive on the leader's, once each, when its rows are in order
            const int half = grad_n() / 2;                          // columns per CTA: 64 or 128
            const int y = t.row0 + kb * 64, x0 = t.nb * 256 + rank * half;
            const bool ragged = ragged_block(t.rows, kb);
            const uint32_t bytes = kTileA + half * 128;
            const uint32_t bar = mapa_shared(ragged ? &land_bar[stage] : &full_bar[stage], ragged ? rank : 0);
            if (elected) {
              if (ragged) {
                mbar_arrive_expect_tx(&land_bar[stage], bytes);
              } else if (leader) {
                mbar_arrive(&full_bar[stage]);
                mbar_arrive_expect_tx(&full_bar[stage], 2 * bytes);
              }
              tma_load_2d_pair(st, &p.wmap, bar, m0, y);
              tma_load_2d_pair(st + kBox, &p.wmap, bar, m0 + 64, y);
              tma_load_2d_pair(bt, &p.tmap[0], bar, x0, y);
              if (half > 64) tma_load_2d_pair(bt + kBox, &p.tmap[0], bar, x0 + 64, y);
            }
          } else {
            const uint32_t bar = mapa_shared(&full_bar[stage], 0);
            const int kx = kb * 64;
            const int n_pad = (t.rows + 31) & ~31;
            // this CTA's half of the token rows, in boxes of 128, 64, 32 and 16 rows
            const int rows = n_pad / 2, y = t.row0 + rank * rows;
            if (elected) {
              if (leader) mbar_arrive_expect_tx(&full_bar[stage], 2 * kTileA + n_pad * 128);
              if (OP == kNT) {
                tma_load_3d_pair(st, &p.wmap, bar, kx, m0, t.g);
              } else {
                tma_load_3d_pair(st, &p.wmap, bar, m0, kx, t.g);
                tma_load_3d_pair(st + kBox, &p.wmap, bar, m0 + 64, kx, t.g);
              }
              for (int bi = 0, off = 0; bi < 4; ++bi) {
                const int box = 128 >> bi;
                while (rows - off >= box) {
                  tma_load_2d_pair(bt + off * 128, &p.tmap[bi], bar, kx, y + off);
                  off += box;
                }
              }
            }
          }
          __syncwarp();
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA issuer (the leader)
      if (leader) {
        const bool elected = elect_one();
        int stage = 0;
        uint32_t phase = 0, it = 0;                // accumulators used so far
        bool ok = true;
        while (ok && fetch()) {
          if (c.kb1 <= c.kb0) continue;                             // TN: a group without rows
          const int n_pad = OP == kTN ? grad_n() : (t.rows + 31) & ~31;
          const uint32_t idesc = idesc_bf16_f32(256, n_pad) | (OP != kNT ? kIdescAMajorMN : 0u) |
                                 (OP == kTN ? kIdescBMajorMN : 0u);
          uint32_t b = 0;
          for (int kb = c.kb0; kb < c.kb1; ++kb) {
            const int at = (kb - c.kb0) % kRun;
            if (at == 0) {                       // a fresh accumulator
              b = it % C::kBufs;
              ok = mbar_poll_warp(&tempty_bar[b], ((it / C::kBufs) & 1u) ^ 1u, abort_flag, status);
              if (!ok) break;
              ++it;
            }
            const uint32_t d = tmem + b * C::kCols;
            ok = OP == kTN && ragged_block(t.rows, kb)
                     ? __all_sync(0xffffffffu, mbar_wait_cluster(&full_bar[stage], phase, abort_flag, status)) != 0
                     : mbar_poll_warp(&full_bar[stage], phase, abort_flag, status);
            if (!ok) break;
            tc_fence_after();
            const uint32_t sa = smem_u32(tiles) + stage * C::kStage, sb = sa + kTileA;
            const int left = OP == kTN ? t.rows - kb * 64 : 64;
            if (elected) {
  #pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                if (OP == kTN && kk * 16 >= left) break;
                const uint64_t ad = OP == kNT ? umma_desc_sw128(sa + kk * 32) : umma_desc_mn_sw128(sa + kk * 2048);
                const uint64_t bd = OP == kTN ? umma_desc_mn_sw128(sb + kk * 2048) : umma_desc_sw128(sb + kk * 32);
                umma_bf16_pair(d, ad, bd, idesc, (at || kk) ? 1u : 0u);
              }
              umma_commit_pair(&empty_bar[stage], 0x3);
              if (at == kRun - 1 || kb + 1 == c.kb1) umma_commit_pair(&tfull_bar[b], 0x3);
            }
            __syncwarp();
            if (++stage == C::kStages) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
      }
      __syncwarp();
    } else if (warp == 2) {
      if (OP == kTN) {
        // -------------------------------------------------------- rows behind the group's last
        // The last K block's rows past the group belong to the next group (or to nobody): in both
        // operands they are overwritten with zeros up to the MMA's 16-row step.
        int stage = 0;
        uint32_t parity = 0;                       // bit s: phase of land_bar[s]
        bool ok = true;
        while (ok && fetch()) {
          const int boxes = 2 + grad_n() / 128;
          for (int kb = c.kb0; kb < c.kb1; ++kb, stage = stage + 1 == C::kStages ? 0 : stage + 1) {
            if (!ragged_block(t.rows, kb)) continue;
            ok = mbar_poll_warp(&land_bar[stage], (parity >> stage) & 1u, abort_flag, status);
            if (!ok) break;
            parity ^= 1u << stage;
            const int left = t.rows - kb * 64;
            uint8_t* st = tiles + stage * C::kStage;
            const int units = (16 - (left & 15)) * 8;               // 16-byte pieces per box
            for (int i = lane; i < units * boxes; i += 32) {
              const int box = i / units;
              *reinterpret_cast<uint4*>(st + box * kBox + left * 128 + (i - box * units) * 16) =
                  make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(mapa_shared(&full_bar[stage], 0));
          }
        }
      }
      __syncwarp();
    }
  } else {
    // ---------------------------------------------------------- epilogue (both CTAs)
    regs_up<kRegsHigh>();
    const int sub = warp & 3;                    // TMEM lane quadrant
    const int m_local = sub * 32 + lane;
    const int from = ((warp - C::kEpi0) >> 2) * 128;             // the warp's 128 columns
    uint8_t* stg = staging + (warp - C::kEpi0) * C::kWarpStage;
    EpilogueSync sync{epi_bar, abort_flag, status};
    uint32_t it = 0;
    bool ok = true;
    auto release = [&](uint32_t b) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_light(mapa_shared(&tempty_bar[b], 0));
    };
    while (ok && fetch()) {
      const int m0 = t.mb * 256 + rank * 128 + sub * 32;          // the warp's first output index
      const int cols = OP == kTN ? grad_cols() : t.rows;          // TMEM columns in use
      const int to = min(cols, from + 128);
      int first = 0, last = 0;
      if (cut) sched.owners(c.tile, first, last);
      auto slot = [&](int owner) {
        return p.partials + (static_cast<size_t>(owner) * 2 + rank) * kPartFloats + m_local * 4;
      };
      // sixteen columns of the finished tile to global memory
      auto finish = [&](const float* v, int n0) {
        if (m0 >= p.m_total) return;
        if (OP == kTN)
          store_direct<OUT>(static_cast<OUT*>(p.out) + (static_cast<size_t>(t.g) * p.m_total + m0) * p.ld_out +
                                t.nb * 256 + n0,
                            p.ld_out, p.m_total - m0, cols - n0, v, stg, lane);
        else
          store_transposed<OUT>(static_cast<OUT*>(p.out) + static_cast<size_t>(t.row0 + n0) * p.ld_out + m0,
                                p.ld_out, cols - n0, p.m_total - m0, v, stg, lane);
      };
      auto emit = [&](const float* v, int n0) {
        if (!cut) {
          finish(v, n0);
        } else {
          float* mine = slot(pair);
#pragma unroll
          for (int i = 0; i < 16; i += 4) write_part(mine, n0 + i, v + i);
        }
      };
      // TN: 32 rows x 128 bytes through a swizzled stage and a TMA store, which leaves out what
      // lies past n and k
      constexpr int kStep = 128 / static_cast<int>(sizeof(OUT));
      auto box_out = [&](const float* v, int n0) {
        if (lane == 0) bulk_wait_read<0>();                       // the store before has left the stage
        __syncwarp();
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          uint4 q;
          if constexpr (kStep == 32) {
            q = make_uint4(__float_as_uint(v[4 * u]), __float_as_uint(v[4 * u + 1]),
                           __float_as_uint(v[4 * u + 2]), __float_as_uint(v[4 * u + 3]));
          } else {
            __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&q);
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = __floats2bfloat162_rn(v[8 * u + 2 * e], v[8 * u + 2 * e + 1]);
          }
          *reinterpret_cast<uint4*>(stg + lane * 128 + ((u ^ (lane & 7)) << 4)) = q;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (m0 < p.m_total) tma_store_3d(&p.omap, stg, t.nb * 256 + n0, m0, t.g);
          bulk_commit();
        }
      };
      const uint32_t lanes = tmem + (static_cast<uint32_t>(sub * 32) << 16);
      f32x2 acc[64];                             // the warp's 128 columns (TN: zeros for no rows)
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = both2(0.f);
      for (int kb = c.kb0; kb < c.kb1; kb += kRun, ++it) {
        const uint32_t b = it % C::kBufs;
        ok = mbar_wait_warp(&tfull_bar[b], (it / C::kBufs) & 1u, abort_flag, status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t tb = lanes + b * C::kCols + from;
        if (from < to) add_columns(tb, to - from, acc);
        release(b);
        const int done = kb + kRun - c.kb0;
        if (LONG && done % kLevel == 0 && done < c.kb1 - c.kb0)
          // (this pair's part of the workspace: its cut tile, if any, comes last and ends there too)
          lay_aside(slot(pair) + from * 128, to - from, done == kLevel, acc);
      }
      if (!ok) break;
      if (LONG && c.kb1 - c.kb0 > kLevel) take_back(slot(pair) + from * 128, to - from, acc);
      auto sums = [&](int i, float* v, auto n) {
#pragma unroll
        for (int e = 0; e < decltype(n)::value / 2; ++e) {
          const float2 f = unpack2(acc[i / 2 + e]);
          v[2 * e] = f.x;
          v[2 * e + 1] = f.y;
        }
      };
      if (OP == kTN && !cut) {
#pragma unroll
        for (int i = 0; i < 128; i += kStep) {
          float v[kStep];
          sums(i, v, std::integral_constant<int, kStep>());
          if (from + i < to) box_out(v, from + i);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 128; i += 16) {
          float v[16];
          sums(i, v, std::integral_constant<int, 16>());
          if (from + i < to) emit(v, from + i);
        }
      }
      if (!cut) continue;
      if (!arrive_last(p.header, 2 * first + rank, last - first + 1, sync, last_flag,
                       warp == C::kEpi0 && lane == 0, lane, ok))
        continue;
      if (OP == kTN) {                           // the stage is about to be written directly
        if (lane == 0) bulk_wait_read<0>();
        __syncwarp();
      }
      for (int n0 = from; n0 < to; n0 += 32) {
        float v[32];
        join_parts<32, 2>(v, slot, first, last, n0, cols - n0);
        finish(v, n0);
        if (n0 + 16 < cols) finish(v + 16, n0 + 16);
      }
    }
    if (OP == kTN && lane == 0) bulk_wait_all();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// ------------------------------------------------------------------ fold kernel
// The e4m3 product on groups of more rows: up to 128 tokens x 256 weight rows per CTA.  Every K
// block's products pass once through the epilogue, acc += (s_a s_w) x products.  Here the tokens
// are the MMA's M side: a thread then holds one token's row, so that the factor of a K block is
// one value per thread and weight block.  (With the weights on M the factor changes from column to
// column; reading 128 factors per thread and K block from shared memory took 1024 of 2100 cycles,
// 446 us at T = 8192, n = 4096, k = 7168.)  Two TMEM buffers of 256 columns take turns: while one
// is folded by eight warps -- 128 fp32 sums per thread, packed two to an instruction, each
// 16-column load under way during the previous one's arithmetic -- the MMAs fill the other.
//
// One commit per K block says both that its products are in TMEM and that its stage is free.  The
// scales come through shared memory, fetched by the two warps that are free otherwise.
//
// Measured at that size: 243 us on a cool GPU (1980 TFLOP/s, 0.75 of cuBLASLt's plain e4m3 rate,
// sustained), 290 us in a run of cases back to back.  A K block takes about 1020 cycles, of which the
// MMAs need 512 at full rate (tensor pipe busy in 51% of the cycles).  Loads alone, with neither MMAs
// nor folds, take 146 us there, loads and MMAs 200 us, loads and folds 200 us: what is left is that
// the two overlap in part only, with the two buffers that TMEM has room for.  On the way (cool): two
// 128-column MMAs and four buffers 312 us (the token operand is read twice), sixteen epilogue warps
// 365 us (twice the waits), scales loaded by the epilogue threads two K blocks ahead 254 us,
// 32-column loads two at a time 318 us (registers spill).  CTA pairs with 256 tokens:
// 245 us, and 450 us where 64 groups have 16 rows each (293 us here); pairs on 128-column tiles
// with four buffers 307 us.
struct FoldCfg {
  static constexpr int kWidth = 128;                              // tokens
  static constexpr uint32_t kStage = 3 * kTileA;                  // 128 token + 256 weight rows: 48 KB
  static constexpr int kStages = 4;
  static constexpr int kCols = 256;                               // per buffer
  static constexpr int kThreads = 384;
  static constexpr uint32_t kWarpStage = 1024;
  static constexpr uint32_t kStaging = 8 * kWarpStage;
  static constexpr int kRowScales = 128 + 2 * 2;                  // per K block: tokens, weight blocks (twice)
  static constexpr uint32_t kScales = 2 * kScaleBlocks * kRowScales * 4;
  static constexpr uint32_t kSmem =
      1024 + kStages * kStage + 1024 + kScales + kStaging + ((sizeof(GroupTable) + 15) & ~15u);
  static_assert(kSmem <= 227 * 1024, "budget");
};

template <typename OUT>
__global__ void __launch_bounds__(FoldCfg::kThreads, 1) fold_kernel(const __grid_constant__ ProductArgs p) {
  using C = FoldCfg;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(tiles + C::kStages * C::kStage);
  uint64_t* done_bar = full_bar + C::kStages;         // a stage's products are in TMEM, the stage is free
  uint64_t* tempty_bar = done_bar + C::kStages;       // [2] buffers read
  uint64_t* sfull_bar = tempty_bar + 2;               // [2] scales of kScaleBlocks K blocks
  uint64_t* sempty_bar = sfull_bar + 2;
  uint64_t* epi_bar = sempty_bar + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(epi_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* last_flag = reinterpret_cast<int*>(tmem_slot + 2);
  float* scales = reinterpret_cast<float*>(tiles + C::kStages * C::kStage + 1024);
  uint8_t* staging = reinterpret_cast<uint8_t*>(scales) + C::kScales;
  GroupTable& gt = *reinterpret_cast<GroupTable*>(staging + C::kStaging);
  int* status = p.header;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full_bar[i], 1);
      mbar_init(&done_bar[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tempty_bar[i], 8);
      mbar_init(&sfull_bar[i], 2);                     // the scale warps
      mbar_init(&sempty_bar[i], 8);
    }
    mbar_init(epi_bar, 8);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.wmap);
    tma_prefetch_desc(&p.tmap[0]);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  launch_wait();
  launch_begin_next();
  const int col_blocks = (p.m_total + 255) / 256;
  const int n_tiles = build_groups(p, gt, C::kWidth, 16, 8, col_blocks, 0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  RoundShare sched(blockIdx.x, gridDim.x, n_tiles, p.k_blocks, true, 14);
  Piece c;
  Tile t;                                        // mb: block of 256 weight rows
  auto fetch = [&]() {
    if (!sched.next(c)) return false;
    t = token_tile(gt, c.tile, C::kWidth, 16, col_blocks, 8);
    return true;
  };
  auto halves = [&]() { return p.m_total - t.mb * 256 > 128 ? 2 : 1; };

  if (warp < 4) {
    regs_down<kRegsLow>();                    // (one instruction for the whole warpgroup)
    if (warp == 0) {
      // -------------------------------------------------------- TMA producer
      const bool elected = elect_one();
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      while (ok && fetch()) {
        const int n_pad = (t.rows + 15) & ~15, nh = halves();
        for (int kb = c.kb0; kb < c.kb1; ++kb) {
          ok = mbar_poll_warp(&done_bar[stage], phase ^ 1u, abort_flag, status);
          if (!ok) break;
          uint8_t* st = tiles + stage * C::kStage;
          uint64_t* bar = &full_bar[stage];
          if (elected) {
            mbar_arrive_expect_tx(bar, nh * kTileA + n_pad * 128);
            tma_load_3d(st + kTileA, &p.wmap, bar, kb * 128, t.mb * 256, t.g);
            if (nh > 1) tma_load_3d(st + 2 * kTileA, &p.wmap, bar, kb * 128, t.mb * 256 + 128, t.g);
            for (int bi = 0, off = 0; bi < 4; ++bi) {             // boxes of 128, 64, 32, 16 rows
              const int box = 128 >> bi;
              while (n_pad - off >= box) {
                tma_load_2d(st + off * 128, &p.tmap[bi], bar, kb * 128, t.row0 + off);
                off += box;
              }
            }
          }
          __syncwarp();
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    } else if (warp == 1) {
      // -------------------------------------------------------- MMA issuer
      // Rows of the token tile that were not loaded hold what an earlier stage left: their
      // products stay in TMEM lanes that nobody stores.
      const bool elected = elect_one();
      int stage = 0;
      uint32_t phase = 0, it = 0;                // buffers used so far
      bool ok = true;
      while (ok && fetch()) {
        const uint32_t idesc = idesc_e4m3_f32(128, 128 * halves());
        for (int kb = c.kb0; kb < c.kb1; ++kb, ++it) {
          const uint32_t b = it & 1u;
          ok = mbar_poll_warp(&full_bar[stage], phase, abort_flag, status) &&
               mbar_poll_warp(&tempty_bar[b], ((it >> 1) & 1u) ^ 1u, abort_flag, status);
          if (!ok) break;
          tc_fence_after();
          const uint32_t sa = smem_u32(tiles) + stage * C::kStage, sb = sa + kTileA;
          if (elected) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_e4m3(tmem + b * C::kCols, umma_desc_sw128(sa + kk * 32), umma_desc_sw128(sb + kk * 32), idesc,
                        kk ? 1u : 0u);
            umma_commit(&done_bar[stage]);
          }
          __syncwarp();
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    } else {
      // -------------------------------------------------------- scales
      // Warps 2 and 3 copy the scales of kScaleBlocks K blocks at a time to [K block][token], with
      // the two weight blocks' behind the tokens' (each warp for itself, to look at their products);
      // rows past the tile repeat its last.
      const int me = (warp - 2) * 32 + lane;
      uint32_t it = 0;
      bool ok = true, over = false;
      while (ok && fetch()) {
        const float* sa0 = p.a_scale + static_cast<size_t>(t.row0 + min(me, t.rows - 1)) * p.k_blocks;
        const float* sa1 = p.a_scale + static_cast<size_t>(t.row0 + min(me + 64, t.rows - 1)) * p.k_blocks;
        const float* sw = p.w_scale + (static_cast<size_t>(t.g) * p.w_scale_rows +
                                       min(2 * t.mb + (lane & 1), p.w_scale_rows - 1)) * p.k_blocks;
        for (int kb = c.kb0; kb < c.kb1; kb += kScaleBlocks, ++it) {
          ok = mbar_poll_warp(&sempty_bar[it & 1], ((it >> 1) & 1u) ^ 1u, abort_flag, status);
          if (!ok) break;
          float* dst = scales + (it & 1) * (kScaleBlocks * C::kRowScales);
          const int last = c.kb1 - 1;
#pragma unroll
          for (int q = 0; q < kScaleBlocks; ++q) {
            cp_async_4(dst + q * C::kRowScales + me, sa0 + min(kb + q, last));
            cp_async_4(dst + q * C::kRowScales + me + 64, sa1 + min(kb + q, last));
          }
          float* w = dst + 128 + 2 * (warp - 2);
          if (lane < 2 * kScaleBlocks)
            cp_async_4(w + (lane >> 1) * C::kRowScales + (lane & 1), sw + min(kb + (lane >> 1), last));
          cp_async_wait_all();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sfull_bar[it & 1]);
#pragma unroll 2
          for (int q = 0; q < kScaleBlocks; ++q) {
            const float a0 = dst[q * C::kRowScales + me], a1 = dst[q * C::kRowScales + me + 64];
            const float w0 = w[q * C::kRowScales], w1 = w[q * C::kRowScales + 1];
            over |= scales_overflow(a0, w0) | scales_overflow(a0, w1) | scales_overflow(a1, w0) |
                    scales_overflow(a1, w1);
          }
        }
      }
      if (over) record_status(status, kStatusDeviceValue);
      __syncwarp();
    }
  } else {
    // ---------------------------------------------------------- epilogue
    regs_up<kRegsHigh>();
    const int sub = warp & 3;                    // TMEM lane quadrant: tokens sub * 32 + lane
    const int half = (warp - 4) >> 2;            // 128-column half of the tile
    uint8_t* stg = staging + (warp - 4) * C::kWarpStage;
    EpilogueSync sync{epi_bar, abort_flag, status};
    uint32_t it = 0, sit = 0;
    bool ok = true;
    while (ok && fetch()) {
      const int col0 = t.mb * 256 + half * 128;  // the warp's first output column
      const int rows = t.rows - sub * 32;        // its rows (<= 0: none)
      const bool mine = half < halves() && rows > 0;
      f32x2 acc[64];                             // 128 sums
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = both2(0.f);
      for (int kb0 = c.kb0; kb0 < c.kb1 && ok; kb0 += kScaleBlocks, ++sit) {
        ok = mbar_poll_warp(&sfull_bar[sit & 1], (sit >> 1) & 1u, abort_flag, status);
        if (!ok) break;
        const float* sc = scales + (sit & 1) * (kScaleBlocks * C::kRowScales);
#pragma unroll 2
        for (int r = 0; r < kScaleBlocks; ++r) {
          if (kb0 + r >= c.kb1) break;
          const uint32_t b = it & 1u;
          const float f = sc[r * C::kRowScales + sub * 32 + lane] * sc[r * C::kRowScales + 128 + half];
          ok = mbar_poll_warp(&done_bar[it % C::kStages], (it / C::kStages) & 1u, abort_flag, status);
          if (!ok) break;
          ++it;
          tc_fence_after();
          if (mine) {
            const uint32_t tb = tmem + (static_cast<uint32_t>(sub * 32) << 16) + b * C::kCols + half * 128;
            const f32x2 gg = both2(f);
            uint32_t v[2][16];
            tmem_ld16_begin(tb, v[0]);
            tmem_ld_end(v[0]);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              if (q < 7) tmem_ld16_begin(tb + (q + 1) * 16, v[(q + 1) & 1]);
#pragma unroll
              for (int i = 0; i < 16; i += 2) {
                f32x2& a = acc[(q * 16 + i) / 2];
                a = fma2(gg, pack2(v[q & 1][i], v[q & 1][i + 1]), a);
              }
              if (q < 7) tmem_ld_end(v[(q + 1) & 1]);
              if (q == 6) {                      // the buffer is free again
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&tempty_bar[b]);
              }
            }
          } else if (lane == 0) {
            mbar_arrive(&tempty_bar[b]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sempty_bar[sit & 1]);
      }
      if (!ok) break;
      auto finish = [&](const float* v, int i) {
        if (mine && col0 + i < p.m_total)
          store_direct<OUT>(static_cast<OUT*>(p.out) + static_cast<size_t>(t.row0 + sub * 32) * p.ld_out + col0 + i,
                            p.ld_out, rows, p.m_total - col0 - i, v, stg, lane);
      };
      auto sixteen = [&](int i, float* v) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 f = unpack2(acc[i / 2 + e]);
          v[2 * e] = f.x;
          v[2 * e + 1] = f.y;
        }
      };
      if (!sched.cut(c)) {
#pragma unroll
        for (int i = 0; i < 128; i += 16) {
          float v[16];
          sixteen(i, v);
          finish(v, i);
        }
        continue;
      }
      int first, last;
      sched.owners(c.tile, first, last);
      auto slot = [&](int owner) { return p.partials + owner * kPartFloats + (sub * 32 + lane) * 4; };
      if (mine) {
        float* to = slot(blockIdx.x);
#pragma unroll
        for (int i = 0; i < 128; i += 16) {
          float v[16];
          sixteen(i, v);
#pragma unroll
          for (int e = 0; e < 16; e += 4) write_part(to, half * 128 + i + e, v + e);
        }
      }
      if (!arrive_last(p.header, first, last - first + 1, sync, last_flag, warp == 4 && lane == 0, lane, ok)) continue;
      for (int i = 0; i < 128 && mine; i += 32) {
        float v[32];
        join_parts<32, 2>(v, slot, first, last, half * 128 + i, 32);
        finish(v, i);
        finish(v + 16, i + 16);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ host
constexpr size_t kProductHeader = 256;
constexpr int kMaxCtas = 148;                   // most CTAs that a launch uses
static_assert(kMaxCtas <= kMaxCounters, "join counters");

size_t product_workspace() {
  const size_t stream = 2 * StreamCfg<true, kNT>::kTileFloats;   // floats per CTA
  return kProductHeader + sizeof(float) * kMaxCtas * (stream > kPartFloats ? stream : kPartFloats);
}

int device_sms() {
  static std::atomic<int> cached[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  const bool keep = dev >= 0 && dev < 64;
  if (keep && (n = cached[dev].load(std::memory_order_relaxed))) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (keep) cached[dev].store(n, std::memory_order_relaxed);
  return n;
}

moe_status check_product(const moe_product_config* c) {
  if (!c || c->n_groups <= 0 || c->n_rows < 0 || c->n <= 0 || c->k <= 0) return MOE_ERR_INVALID_ARG;
  if (c->n_groups > kMaxProductGroups || c->n > 65536 || c->k > 65536 || c->n_rows > (1 << 24))
    return MOE_ERR_UNSUPPORTED;
  if (c->in != MOE_BF16 && c->in != MOE_E4M3_FP32_SCALE) return MOE_ERR_UNSUPPORTED;
  if (c->out != MOE_BF16 && c->out != MOE_F32) return MOE_ERR_UNSUPPORTED;
  if (c->n % 8 || c->k % (c->in == MOE_BF16 ? 8 : 16)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

template <class K>
cudaError_t launch_product_kernel(K kernel, const ProductArgs& a, int grid, int threads, uint32_t smem,
                                  cudaStream_t s) {
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_overlapped(kernel, dim3(grid), threads, smem, s, a);
}

template <bool F8, int OP, typename OUT>
cudaError_t launch_product(const ProductArgs& a, bool stream_tiles, cudaStream_t s) {
  using Pair = PairCfg<OP>;
  const int sms = device_sms();
  if (sms < 2) return cudaErrorInvalidDevice;
  const int ctas = sms < kMaxCtas ? sms : kMaxCtas;
  if constexpr (OP != kTN) {
    if (stream_tiles)
      return launch_product_kernel(stream_kernel<F8, OP, OUT>, a, ctas, 224, StreamCfg<F8, OP>::kSmem, s);
  }
  if constexpr (F8) {
    return launch_product_kernel(fold_kernel<OUT>, a, ctas, FoldCfg::kThreads, FoldCfg::kSmem, s);
  } else {
    // a second level of sums only where a group can have the rows for it: the code for it costs
    // registers (weight gradient of 32 groups x 256 rows: 459 us without, 468 with)
    auto kernel = pair_kernel<OP, OUT, false>;
    if constexpr (OP == kTN)
      if (a.n_rows > 64 * kLevel) kernel = pair_kernel<OP, OUT, true>;
    return launch_product_kernel(kernel, a, ctas / 2 * 2, Pair::kThreads, Pair::kSmem, s);
  }
}
template <bool F8, int OP>
moe_status launch_product(const ProductArgs& a, bool f32, bool stream_tiles, cudaStream_t s) {
  const cudaError_t e = f32 ? launch_product<F8, OP, float>(a, stream_tiles, s)
                            : launch_product<F8, OP, __nv_bfloat16>(a, stream_tiles, s);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// Groups of few rows go to the stream kernel (the host knows the rows' capacity and the groups): at most 32
// rows in all (e4m3: 64, two tiles' rows), or at most eight per group on average, where few groups
// hold more than a tile.  Measured with 64 groups, n = 7168, k = 2048: 8 rows on average 6.43 TB/s, 16
// rows 5.7 (groups above 32 rows read their weights twice), against 6.3 with 32 rows in the pair
// kernel.  One group of 64 rows, n = 4096, k = 7168: e4m3 16.5 us here, 21.8 in the fold kernel (96
// rows, n = 7168, k = 2048: 17.0 against 15.7); bf16 19.8 us here, 17.6 in the pair kernel.
bool few_rows(const moe_product_config& c) {
  return c.n_rows <= (c.in == MOE_BF16 ? 32 : 64) || c.n_rows <= 8 * c.n_groups;
}

moe_status common_checks(const moe_product_config* cfg, const int32_t* offsets, const void* x, const void* y,
                         const void* z, const void* ws, size_t ws_bytes) {
  const moe_status st = check_product(cfg);
  if (st != MOE_OK) return st;
  if (!ws || (!offsets && cfg->n_groups != 1)) return MOE_ERR_INVALID_ARG;
  if (misaligned(x) || misaligned(y) || misaligned(z) || misaligned(ws) || misaligned(offsets, sizeof(int32_t)))
    return MOE_ERR_INVALID_ARG;
  return ws_bytes < product_workspace() ? MOE_ERR_WORKSPACE : MOE_OK;
}

ProductArgs product_args(const moe_product_config& c, const int32_t* offsets, void* out, void* ws) {
  ProductArgs a{};
  a.offsets = offsets;
  a.n_groups = c.n_groups;
  a.n_rows = c.n_rows;
  a.out = out;
  a.header = static_cast<int*>(ws);
  a.partials = reinterpret_cast<float*>(static_cast<char*>(ws) + kProductHeader);
  return a;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_product_workspace_size(const moe_product_config* cfg, size_t* bytes) {
  if (!bytes) return MOE_ERR_INVALID_ARG;
  const moe_status st = check_product(cfg);
  if (st != MOE_OK) return st;
  *bytes = product_workspace();
  return MOE_OK;
}

moe_status moe_grouped_gemm(const moe_product_config* cfg, const int32_t* group_offsets, const void* a,
                            const float* a_scale, const void* w, const float* w_scale, void* y, void* ws,
                            size_t ws_bytes, cudaStream_t stream) {
  const moe_status st = common_checks(cfg, group_offsets, a, w, y, ws, ws_bytes);
  if (st != MOE_OK) return st;
  const bool f8 = cfg->in == MOE_E4M3_FP32_SCALE;
  if (!f8 && (a_scale || w_scale)) return MOE_ERR_INVALID_ARG;
  if (misaligned(a_scale, sizeof(float)) || misaligned(w_scale, sizeof(float))) return MOE_ERR_INVALID_ARG;
  if (cfg->n_rows == 0) return MOE_OK;
  if (!a || !w || !y || (f8 && (!a_scale || !w_scale))) return MOE_ERR_INVALID_ARG;
  ProductArgs p = product_args(*cfg, group_offsets, y, ws);
  const bool few = few_rows(*cfg);
  bool ok = make_tmap_matrix(&p.wmap, w, f8, cfg->n_groups, cfg->n, cfg->k, 128);
  for (int i = few ? 2 : 0; i < 4 && ok; ++i)    // the stream kernel takes boxes of 32 and 16 rows
    ok = f8 ? make_tmap_u8(&p.tmap[i], a, cfg->n_rows, cfg->k, 128u >> i)
            : make_tmap_bf16(&p.tmap[i], a, cfg->n_rows, cfg->k, 128u >> i);
  if (!ok) return MOE_ERR_CUDA;
  p.m_total = p.ld_out = cfg->n;
  p.k_blocks = (cfg->k + (f8 ? 127 : 63)) / (f8 ? 128 : 64);
  p.a_scale = a_scale;
  p.w_scale = w_scale;
  p.w_scale_rows = (cfg->n + 127) / 128;
  const bool f32 = cfg->out == MOE_F32;
  return f8 ? launch_product<true, kNT>(p, f32, few, stream) : launch_product<false, kNT>(p, f32, few, stream);
}

moe_status moe_grouped_gemm_dgrad(const moe_product_config* cfg, const int32_t* group_offsets, const void* dy,
                                  const void* w, void* da, void* ws, size_t ws_bytes, cudaStream_t stream) {
  const moe_status st = common_checks(cfg, group_offsets, dy, w, da, ws, ws_bytes);
  if (st != MOE_OK) return st;
  if (cfg->in != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  if (cfg->n_rows == 0) return MOE_OK;
  if (!dy || !w || !da) return MOE_ERR_INVALID_ARG;
  ProductArgs p = product_args(*cfg, group_offsets, da, ws);
  const bool few = few_rows(*cfg);
  bool ok = make_tmap_matrix(&p.wmap, w, false, cfg->n_groups, cfg->n, cfg->k, 64);
  for (int i = few ? 2 : 0; i < 4 && ok; ++i) ok = make_tmap_bf16(&p.tmap[i], dy, cfg->n_rows, cfg->n, 128u >> i);
  if (!ok) return MOE_ERR_CUDA;
  p.m_total = p.ld_out = cfg->k;
  p.k_blocks = (cfg->n + 63) / 64;
  return launch_product<false, kNN>(p, cfg->out == MOE_F32, few, stream);
}

moe_status moe_grouped_gemm_wgrad(const moe_product_config* cfg, const int32_t* group_offsets, const void* dy,
                                  const void* a, void* dw, void* ws, size_t ws_bytes, cudaStream_t stream) {
  const moe_status st = common_checks(cfg, group_offsets, dy, a, dw, ws, ws_bytes);
  if (st != MOE_OK) return st;
  if (cfg->in != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  if (!dw) return MOE_ERR_INVALID_ARG;
  if (cfg->n_rows == 0) {                        // no rows: every sum is empty
    const size_t bytes = static_cast<size_t>(cfg->n_groups) * cfg->n * cfg->k * (cfg->out == MOE_F32 ? 4 : 2);
    return cudaMemsetAsync(dw, 0, bytes, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  }
  if (!dy || !a) return MOE_ERR_INVALID_ARG;
  ProductArgs p = product_args(*cfg, group_offsets, dw, ws);
  if (!make_tmap_bf16(&p.wmap, dy, cfg->n_rows, cfg->n, 64) ||
      !make_tmap_bf16(&p.tmap[0], a, cfg->n_rows, cfg->k, 64) ||
      !make_tmap_store(&p.omap, dw, cfg->out == MOE_F32, cfg->n_groups, cfg->n, cfg->k))
    return MOE_ERR_CUDA;
  p.m_total = cfg->n;
  p.n_total = p.ld_out = cfg->k;
  p.k_blocks = 0;
  return launch_product<false, kTN>(p, cfg->out == MOE_F32, false, stream);
}

}  // extern "C"
