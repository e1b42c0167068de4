// Products of MX (8-bit, block-scaled) matrices on the sm_100a tensor cores:
// out = residual + alpha * act(X W^T + b) in bf16, and the gated half of the
// feed-forward layer, silu(X Wg^T + bg) * (X Wu^T + bu), in MX form.
//
// X is [M, K], W is [N, K], both e4m3 with an e8m0 scale per 32 values along
// K, so  y[m][n] = sum_b 2^(ex[m][b] + ew[n][b]) * sum_{k in b} x[m][k] w[n][k].
// tcgen05.mma.kind::mxf8f6f4.block_scale does both sums in fp32: one instruction
// covers K = 32, one scale block, and takes the scales from tensor memory.
#include <cudaTypedefs.h>
#include <string.h>

#include "qi21_internal.h"
#include "qi21_mx.cuh"

namespace qi21 {

namespace mx {

constexpr int BK = 128;           // one 128-byte swizzle atom of e4m3, four scale blocks
constexpr int kTileBytes = 512;   // scales of 128 rows x 4 blocks
constexpr int kMaxOut = 4;

// Instruction descriptor of kind::mxf8f6f4: A and B e4m3 (0), K-major, N >> 3 at
// bit 17, scales e8m0 (bit 23), M >> 4 at bit 24; which of a scale word's four
// bytes to use goes to bits 4-5 (B) and 29-30 (A).
__host__ __device__ constexpr uint32_t idesc(int m, int n) {
  return ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(m >> 4) << 24);
}
__device__ __forceinline__ constexpr uint32_t idesc_block(uint32_t b) { return (b << 4) | (b << 29); }

// Shared-memory descriptor of a K-major operand in 128B-swizzled rows of 128
// bytes: 8-row groups 1024 B apart, version 1, layout 2.
__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024u >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// ... and of one scale tile: 32 rows of 16 bytes, 8-row groups 128 B apart, no
// swizzle.
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(128u >> 4) << 32) | ((uint64_t)1 << 46);
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void* map, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* map, uint32_t bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

// One scale tile to tensor memory: row r of 128 goes to lane r % 32 (of every
// warp's lanes) in column r / 32.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}
// D[tmem] (+)= (A * scales) (B * scales)^T over K = 32.
__device__ __forceinline__ void mma_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t sa, uint32_t sb,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
      ::"r"(d), "l"(a), "l"(b), "r"(id), "r"(sa), "r"(sb), "r"(accumulate)
      : "memory");
}

// The same for a CTA pair.  Loads go to this CTA's shared memory and complete on a
// barrier of the pair's first CTA (`bar` is a cluster address); copies and
// products, issued by the first CTA, run in both.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const void* map, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const void* map, uint32_t bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void copy_scales_pair(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}
__device__ __forceinline__ void mma_scaled_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t sa,
                                                uint32_t sb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
      ::"r"(d), "l"(a), "l"(b), "r"(id), "r"(sa), "r"(sb), "r"(accumulate)
      : "memory");
}

// y / (1 + exp(-y)).  The fast exponential's relative error grows with its argument, to about (2 + 1.2 |y|)
// 2^-23, 1e-5 at |y| = 80: below the rounding of the output, 2^-8 (bf16) or 2^-4 (e4m3).  Where 1 + exp(-y)
// exceeds 2^126 (y below -87.3) the quotient is 0 instead of a value below 2^-119.
__device__ __forceinline__ float silu(float y) { return __fdividef(y, 1.f + __expf(-y)); }
// 0.5 y (1 + tanh(u)) = y / (1 + exp(-2u)),  u = sqrt(2/pi) (y + 0.044715 y^3); the same error with 2|u| in
// the place of |y|, and 2^-22 |2u| for the rounding of u.
__device__ __forceinline__ float gelu_tanh(float y) {
  return __fdividef(y, 1.f + __expf(-1.5957691216057308f * fmaf(0.044715f * y * y, y, y)));
}

struct __align__(64) Params {
  CUtensorMap tm_x, tm_w, tm_xs, tm_ws;
  CUtensorMap tm_out[kMaxOut];    // pair kernel: 32-row, 64-byte boxes of out[i], or of q
  CUtensorMap tm_res;             // ... and of the residual
  int32_t M, N, K;
  int32_t n_seg;                  // columns per output segment (swiglu: N / 2)
  int32_t kt;                     // K steps of 128
  int32_t mt, nt;                 // tiles along M and N (CTA pairs)
  int32_t act;
  float alpha;
  __nv_bfloat16* out[kMaxOut];    // [M, n_seg] each
  const __nv_bfloat16* bias;      // [N] or null
  const __nv_bfloat16* residual;  // [M, N] or null (may be out[0])
  uint8_t* q;                     // swiglu: [M, N / 2] e4m3 and its scale tiles
  uint8_t* scale;
  int32_t q_tile_cols;
  uint32_t* status;
};

// ----------------------------------------------------------- few tokens
// A CTA computes 128 features x bn tokens (bn a multiple of 16, at most 128): the features
// (rows of W) take the 128 lanes of tensor memory, so few tokens waste nothing of
// the stream of W, which is what bounds these calls; a warp's store covers 32
// neighbouring features of one token.  The gated form takes a gate block and its up
// block.  With few tiles the K axis is split over a cluster: each CTA leaves its
// partial sums in its shared memory, and each adds up and finishes a share of
// the tokens, reading the others' partials in the order of the split.
//   warp 0     TMA producer
//   warp 1     TMEM owner and MMA issuer
//   warps 2-9  epilogue: one feature per thread, every other sixteen tokens
// Measured on a B200: 1 x 24576 x 4096 in 20.4 us (5.1 TB/s with launch and ramp), 16 x 4096 x 4096
// in 7.9, 77 x 12288 x 4096 gated in 22.9 (4.5 TB/s: its 96 tiles leave 52 of 148 SMs idle, and two parts of K
// would want more SMs than there are), 1 x 4096 x 256 in 3.1.  Bound by HBM for few tokens where there are
// tiles enough, by what an SM takes from L2 (64 bytes a cycle) for many.
//
// Tensor memory and residency: a CTA waits in its allocation while others of the
// SM hold the columns, and CTAs of a cluster wait for one another, so an SM must
// never host CTAs that want more than its 512 columns together.  Shared memory sees to
// that: at most 256 columns with at least 76 KB (two such CTAs fit), or 512 with more
// than 151 KB (nothing else fits beside it).
constexpr int kNarrowThreads = 320;
constexpr int kNarrowMaxStages = 8;
constexpr int kNarrowSlots = 4;
constexpr int kNarrowMaxSmem = 224 * 1024;
constexpr int kW = 128 * BK;

struct Narrow {
  int32_t bn, stages, cols, split, smem;
};

template <bool B>
struct Bool {
  static constexpr bool value = B;
};

struct NarrowBars {
  uint64_t full[kNarrowMaxStages], empty[kNarrowMaxStages], done;
  uint32_t tmem_base;
  int abort_flag;
};

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

template <bool GATED>
__global__ void __launch_bounds__(kNarrowThreads) mx_gemm_narrow(const __grid_constant__ Params p, const Narrow c) {
  constexpr int NW = GATED ? 2 : 1;
  constexpr int kSlot = 4 * NW + 4;  // scale columns of one K step
  extern __shared__ uint8_t smem_raw[];
  __shared__ NarrowBars S;
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  const uint32_t kx = (uint32_t)c.bn * BK;
  const uint32_t sw = base, sx = sw + c.stages * NW * kW, sws = sx + c.stages * kx,
                 sxs = sws + c.stages * NW * kTileBytes;
  const int warp = threadIdx.x >> 5;
  volatile int* abort_flag = &S.abort_flag;
  const int rank = c.split > 1 ? (int)cluster_rank() : 0;
  const int f0 = (int)(blockIdx.x / c.split) * (NW * 128), m0 = blockIdx.y * c.bn;
  const int k_begin = (int)((int64_t)p.kt * rank / c.split), k_end = (int)((int64_t)p.kt * (rank + 1) / c.split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < c.stages; ++s) {
      mbar_init(smem_u32(&S.full[s]), 1);
      mbar_init(smem_u32(&S.empty[s]), 1);
    }
    mbar_init(smem_u32(&S.done), 1);
    S.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&S.tmem_base), c.cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem_base;
  let_next_start();
  first_wait();

  if (warp == 0) {
    if (elect_one_sync()) {
      const uint32_t bytes = NW * (kW + kTileBytes) + kx + kTileBytes;
      int it = 0, st = 0;
      uint32_t ph = 1;
      bool ok = true;
      for (int k = k_begin; k < k_end; ++k, ++it) {
        ok = mbar_wait(smem_u32(&S.empty[st]), ph, abort_flag, p.status, 0x700 | st);
        if (!ok) break;
        const uint32_t bar = smem_u32(&S.full[st]);
        mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          tma_load_2d(sw + (st * NW + w) * kW, &p.tm_w, bar, k * BK, f0 + 128 * w);
          tma_load_3d(sws + (st * NW + w) * kTileBytes, &p.tm_ws, bar, 0, k, (f0 >> 7) + w);
        }
        tma_load_2d(sx + st * kx, &p.tm_x, bar, k * BK, m0);
        tma_load_3d(sxs + st * kTileBytes, &p.tm_xs, bar, 0, k, m0 >> 7);
        if (++st == c.stages) st = 0, ph ^= 1u;
      }
      // every load issued lands before the CTA may exit
      for (st = 0; !ok && st < c.stages; ++st)
        if (it > st) mbar_wait(smem_u32(&S.full[st]), ((it - 1 - st) / c.stages) & 1u, nullptr, nullptr, 0);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (elect_one_sync()) {
      int it = 0, st = 0, slot = 0, old = 0;
      uint32_t ph = 0, old_ph = 0;
      const uint32_t id = idesc(128, c.bn), sf0 = tmem + NW * c.bn;
      for (int k = k_begin; k < k_end; ++k, ++it) {
        bool ok = true;
        if (it >= kNarrowSlots && c.stages > kNarrowSlots) {
          // The scale columns of this slot were last read by the MMAs of step it - kNarrowSlots.
          // (With fewer stages than slots the stage's own reuse waits for them.)
          ok = mbar_wait(smem_u32(&S.empty[old]), old_ph, abort_flag, p.status, 0x720 | st);
          if (++old == c.stages) old = 0, old_ph ^= 1u;
        }
        ok = ok && mbar_wait(smem_u32(&S.full[st]), ph, abort_flag, p.status, 0x710 | st);
        if (!ok) break;
        tc_fence_after();
        const uint32_t sf = sf0 + slot * kSlot;
#pragma unroll
        for (int w = 0; w < NW; ++w) copy_scales(sf + 4 * w, scale_desc(sws + (st * NW + w) * kTileBytes));
        copy_scales(sf + 4 * NW, scale_desc(sxs + st * kTileBytes));
        const uint64_t wd = operand_desc(sw + st * NW * kW), xd = operand_desc(sx + st * kx);
        const int blocks = (p.K - k * BK) >> 5;  // the blocks past K hold nothing
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          if (b >= blocks) break;
#pragma unroll
          for (int w = 0; w < NW; ++w)
            mma_scaled(tmem + w * c.bn, wd + w * (kW >> 4) + 2 * b, xd + 2 * b, id | idesc_block(b), sf + 4 * w,
                       sf + 4 * NW, it > 0 || b > 0);
        }
        mma_commit(smem_u32(&S.empty[st]));
        if (++st == c.stages) st = 0, ph ^= 1u;
        if (++slot == kNarrowSlots) slot = 0;
      }
      // also after a wait that ran out: every MMA issued completes before TMEM is released
      mma_commit(smem_u32(&S.done));
      mbar_wait(smem_u32(&S.done), 0, nullptr, p.status, 0x730);
    }
    __syncwarp();
  }

  const int lane = threadIdx.x & 31, quarter = warp & 3;
  const int j = quarter * 32 + lane;  // feature in the block == TMEM lane
  const int f = f0 + j, last = min(c.bn, p.M - m0);
  const int t0 = warp < 6 ? 0 : 16;  // warps 2-5 and 6-9 take turns
  const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
  bool ok = true;
  if (warp >= 2) {
    // (one vote: what follows under `ok` holds votes and barriers of whole warps)
    ok = mbar_wait(smem_u32(&S.done), 0, abort_flag, p.status, 0x740) && !*abort_flag;
    ok = __all_sync(0xffffffffu, ok);
    tc_fence_after();
  }

  // Sixteen tokens at a time, so that their chains of bias, activation and store overlap (one
  // token at a time cost 90 ns each): the first `n` of y (gated: the gate's sums, u the up
  // projection's) belong to tokens t, t + 1, ...
  float bias = 0.f, bias_u = 0.f;
  const bool live = GATED || f < p.N;
  if (warp >= 2 && p.bias != nullptr && live) {
    bias = __bfloat162float(p.bias[f]);
    if (GATED) bias_u = __bfloat162float(p.bias[f + 128]);
  }
  const int seg = GATED || !live ? 0 : f / p.n_seg;
  const int col = GATED ? (f0 >> 1) + j : f - seg * p.n_seg;
  __nv_bfloat16* out = GATED ? nullptr : p.out[seg] + col;
  auto finish_some = [&](auto all, int t, int n, float (&y)[16], const float (&u)[16]) {
    constexpr bool kAll = decltype(all)::value;  // all sixteen tokens: no tests
    const int64_t row = m0 + t;
    if (GATED) {
      uint8_t* q = p.q + row * p.n_seg + col;
      uint32_t mine = 0;  // lane e keeps the scale byte of token e
#pragma unroll
      for (int e = 0; e < 16; ++e) y[e] = silu(y[e] + bias) * (u[e] + bias_u);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        // a warp's 32 features are one scale block
        const uint32_t byte = mx_scale_byte(__reduce_max_sync(0xffffffffu, abs_bits(y[e])));
        if (kAll || e < n)
          q[(uint64_t)((uint32_t)e) * (uint32_t)p.n_seg] = (uint8_t)mx_cvt2(y[e] * mx_inv_scale(byte), 0.f);
        if (lane == e) mine = byte;
      }
      if (lane < (kAll ? 16 : n)) p.scale[mx_scale_word(row + lane, col >> 7, p.q_tile_cols) + quarter] = (uint8_t)mine;
    } else if (live) {
      float res[16];
      if (p.residual != nullptr) {
        // read and written by the same thread: the residual may be the output
        const __nv_bfloat16* r = p.residual + row * p.N + f;
#pragma unroll
        for (int e = 0; e < 16; ++e)
          res[e] = kAll || e < n ? __bfloat162float(r[(uint64_t)((uint32_t)e) * (uint32_t)p.N]) : 0.f;
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) y[e] += bias;
      if (p.act == QI21_ACT_SILU) {
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] = silu(y[e]);
      } else if (p.act == QI21_ACT_GELU_TANH) {
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] = gelu_tanh(y[e]);
      }
      if (p.residual != nullptr) {
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] = fmaf(p.alpha, y[e], res[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] *= p.alpha;
      }
      __nv_bfloat16* o = out + row * p.n_seg;
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (kAll || e < n) o[(uint64_t)((uint32_t)e) * (uint32_t)p.n_seg] = __float2bfloat16(y[e]);
    }
  };
  auto finish = [&](int t, int n, float (&y)[16], const float (&u)[16]) {
    if (n == 16)
      finish_some(Bool<true>(), t, n, y, u);
    else
      finish_some(Bool<false>(), t, n, y, u);
  };

  if (c.split == 1) {
    for (int t = t0; warp >= 2 && ok && t < last; t += 32) {
      uint32_t v[16], w[16];
      tmem_ld16(lanes + t, v);
      if (GATED) tmem_ld16(lanes + c.bn + t, w);
      tmem_wait_ld();
      float y[16], u[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        y[e] = __uint_as_float(v[e]);
        u[e] = GATED ? __uint_as_float(w[e]) : 0.f;
      }
      finish(t, min(16, last - t), y, u);
    }
  } else {
    // partial sums [w][token][feature], over the operands' buffers (all read by now)
    for (int t = t0; warp >= 2 && t < last; t += 32) {
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        uint32_t v[16];
        tmem_ld16(lanes + w * c.bn + t, v);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e)
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(base + ((w * c.bn + t + e) * 128 + j) * 4), "r"(v[e])
                       : "memory");
      }
    }
    cluster_sync_all();
    const int share = (last + c.split - 1) / c.split, end = min(last, (rank + 1) * share);
    bool reads = true;  // of the others' partials, until this warp's last ones are read
    for (int t = rank * share + t0; warp >= 2 && ok && t < end; t += 32) {
      const int n = min(16, end - t);
      float y[16] = {}, u[16] = {};
      for (int r = 0; r < c.split; ++r) {
        const uint32_t from = cluster_addr(base, r) + (t * 128 + j) * 4;
        float py[16], pu[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          // (all sixteen are read, the last token's again where there are fewer: a test around each load
          // made 64 x 4096 x 4096 take 12.0 us instead of 8.1)
          const uint32_t at = from + min(e, n - 1) * 512;
          py[e] = ld_cluster_f32(at);
          pu[e] = GATED ? ld_cluster_f32(at + c.bn * 512) : 0.f;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          y[e] += py[e];
          u[e] += pu[e];
        }
      }
      if (t + 32 >= end) {
        cluster_arrive();
        reads = false;
      }
      finish(t, n, y, u);
    }
    if (reads) cluster_arrive();
    cluster_wait();  // nobody's partials go away while they are read
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, c.cols);
}

// ---------------------------------------------------------------- CTA pairs
// A pair of CTAs computes 256 tokens x 256 features, each its 128 tokens (TMEM
// lanes) of all 256 features: tcgen05.mma.cta_group::2 reads each CTA's 128 rows
// of X and 128 rows of W, so a CTA loads 32 KB for 128 x 256 x 128 products, two thirds of
// what it would load alone.  Persistent: pair i walks tiles i, i + pairs, ..., M
// fastest in groups of kGroup tiles so that pairs at work together share W and X in L2.
//   warp 0     TMA producer of its CTA's operands (5 stages of K = 128)
//   warp 1     TMEM owner; in the first CTA it issues the scale copies and the MMAs
//   warps 4-11 epilogue: one token per thread, half of its columns
// Tensor memory holds two accumulators of 256 columns that overlap in 64, [0, 256)
// and [192, 448), and the scales of four K steps behind them.  The epilogue drains the
// shared columns first and then lets the next tile's MMAs start, so only that
// part of an epilogue is not hidden.
// Measured on a B200: 4096 x 12288 x 4096 in 149 us, 2.77 PFLOP/s, the tensor pipe busy 75 % of
// the cycles; gated 4096 x 24576 x 4096 in 283 us, 2.91 PFLOP/s, 82 %; 16384 rows of it in 1.11 ms, 1.26
// under the power cap.  Bound by the tensor pipe and the shared memory that it and the TMA share: a
// stage's MMAs take 512 cycles alone, about 600 beside the loads (the same with 4, 5 and 6 stages; with
// stages of K = 256; without the scale copies).  With K below about 1300 (gated: 700) a tile's products are
// done before the epilogue of the one in front, which then sets the pace: 1400 cycles a warp for 32 columns,
// 880 of them arithmetic and packing (4096 x 12288 x 512 in 52 us, gated 4096 x 24576 x 256 in 62, at 18 % of
// the tensor pipe).
constexpr int kWideThreads = 384;
constexpr int kWideStages = 5;
constexpr int kGroup = 16;
constexpr int kOperand = 128 * BK;
constexpr int kWideStageBytes = 2 * kOperand + 3 * kTileBytes;
constexpr uint32_t kAccShift = 192;
constexpr uint32_t kWideScaleCol = 448;
constexpr uint32_t kSlots = 4;  // of 4 (X) + 8 (W) scale columns each
constexpr int kBoxes = 3;

struct __align__(1024) WideSmem {
  uint8_t x[kWideStages][kOperand];
  uint8_t w[kWideStages][kOperand];
  uint8_t stage[8][kBoxes][32 * 64];  // boxes of each epilogue warp (swizzled: 512-byte aligned)
  uint8_t ws[kWideStages][2 * kTileBytes];
  uint8_t xs[kWideStages][kTileBytes];
  float bias[2][256];                // of this tile and the next
  uint64_t full[kWideStages], empty[kWideStages];
  uint64_t acc_full[2], acc_free, drain;
  uint64_t res_full[8][kBoxes];
  uint32_t tmem_base;
  int abort_flag;
};

__device__ __forceinline__ void tile_of(const Params& p, int t, int& m, int& n) {
  const int span = kGroup * p.nt, g = t / span, in = t - g * span;
  const int rows = min(kGroup, p.mt - g * kGroup);
  n = in / rows;
  m = g * kGroup + in - n * rows;
}

// 32 accumulators plus their biases (in shared memory, the same for every thread).
__device__ __forceinline__ void add_bias(float (&y)[32], const uint32_t (&v)[32], const float* bias) {
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    const float4 b = reinterpret_cast<const float4*>(bias)[g];
    y[4 * g] = __uint_as_float(v[4 * g]) + b.x;
    y[4 * g + 1] = __uint_as_float(v[4 * g + 1]) + b.y;
    y[4 * g + 2] = __uint_as_float(v[4 * g + 2]) + b.z;
    y[4 * g + 3] = __uint_as_float(v[4 * g + 3]) + b.w;
  }
}

// Adds the sums of 32 columns in another CTA's shared memory, 512 bytes apart.
__device__ __forceinline__ void add_others(uint32_t (&v)[32], uint32_t from) {
  float o[32];
#pragma unroll
  for (int e = 0; e < 32; ++e) o[e] = ld_cluster_f32(from + e * 512);
#pragma unroll
  for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) + o[e]);
}

// A warp's results leave through boxes of 32 rows x 64 bytes, swizzled as the TMA's
// 64-byte mode does.  16-byte chunk `j` of this lane's row:
__device__ __forceinline__ uint4* box_chunk(uint8_t* box, uint32_t lane, uint32_t j) {
  return reinterpret_cast<uint4*>(box + lane * 64 + ((j ^ ((lane >> 1) & 3u)) << 4));
}
// The box of this warp is written: one lane hands it to the TMA.
__device__ __forceinline__ void store_box(const CUtensorMap* map, uint8_t* box, int c0, int c1) {
  fence_proxy_async_smem();
  __syncwarp();
  if (elect_one_sync()) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(c0),
                 "r"(c1), "r"(smem_u32(box))
                 : "memory");
    bulk_commit_group();
  }
}
// A warp uses its boxes in turn: the one that comes may be written once the TMA has
// read it, that is when at most the last two stores are not.
__device__ __forceinline__ void reuse_box() {
  if (elect_one_sync()) asm volatile("cp.async.bulk.wait_group.read 2;" ::: "memory");
  __syncwarp();
}

// A residual comes the same way: the TMA loads the chunk into the box that its result will leave from,
// one chunk ahead.  (Loads by the threads, 16 bytes of 32 rows each, cost 2.5 us a tile in the L1
// cache: 4096 x 4096 x 256 took 31 us with a residual, 21 without.)
// SPLIT: one tile to a cluster of two pairs, each with half of K, for calls with few tiles.  When
// both are done, the pairs swap halves of the tile's columns through shared
// memory (fp32, [column][token]): pair i finishes columns 128 i .. 128 i + 127 (gated: hidden
// features 64 i .. 64 i + 63), each of its warp groups half of them, adding the other pair's sums.
template <bool GATED, bool SPLIT>
__global__ void __launch_bounds__(kWideThreads, 1) mx_gemm_wide(const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  WideSmem& S = *reinterpret_cast<WideSmem*>(smem_raw + (((raw + 1023u) & ~1023u) - raw));
  const int warp = threadIdx.x >> 5;
  volatile int* abort_flag = &S.abort_flag;
  const uint32_t rank = cluster_rank() & 1u, first = cluster_rank() & ~1u;  // in the pair; the pair's first CTA
  const int part = SPLIT ? (int)(cluster_rank() >> 1) : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kWideStages; ++s) {
      mbar_init(smem_u32(&S.full[s]), 1);
      mbar_init(smem_u32(&S.empty[s]), 1);
    }
    mbar_init(smem_u32(&S.acc_full[0]), 1);
    mbar_init(smem_u32(&S.acc_full[1]), 1);
    mbar_init(smem_u32(&S.acc_free), 16);  // one arrival per epilogue warp of the pair
    mbar_init(smem_u32(&S.drain), 1);
    for (int i = 0; i < 8 * kBoxes; ++i) mbar_init(smem_u32(&S.res_full[0][i]), 1);
    S.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc_pair(smem_u32(&S.tmem_base), 512);
  if (warp == 0 && (threadIdx.x & 31) == 0) {
    tma_prefetch_desc(&p.tm_x);
    tma_prefetch_desc(&p.tm_w);
    tma_prefetch_desc(&p.tm_xs);
    tma_prefetch_desc(&p.tm_ws);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = S.tmem_base;
  let_next_start();
  first_wait();
  const int tiles = p.mt * p.nt, pair = blockIdx.x >> (SPLIT ? 2 : 1), pairs = gridDim.x >> (SPLIT ? 2 : 1);
  const int k_begin = SPLIT && part == 1 ? p.kt / 2 : 0, k_end = SPLIT && part == 0 ? p.kt / 2 : p.kt;

  // registers: 128 x 80 + 256 x 208 of the launch's 384 x 168
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == 0) {
      // ------------------------------------------------------------ producer
      if (elect_one_sync()) {
        uint32_t it = 0, st = 0, ph = 1;
        bool ok = true;
        for (int t = pair; t < tiles && ok; t += pairs) {
          int m, n;
          tile_of(p, t, m, n);
          const int m0 = m * 256 + (int)rank * 128, n0 = n * 256 + (int)rank * 128;
          for (int kb = k_begin; kb < k_end; ++kb, ++it) {
            ok = mbar_wait(smem_u32(&S.empty[st]), ph, abort_flag, p.status, 0x800 | st);
            if (!ok) break;
            // both CTAs' bytes count on the first CTA's barrier
            if (rank == 0) mbar_arrive_expect_tx(smem_u32(&S.full[st]), 2 * kWideStageBytes);
            const uint32_t bar = cluster_addr(smem_u32(&S.full[st]), first);
            tma_load_2d_pair(smem_u32(S.x[st]), &p.tm_x, bar, kb * BK, m0);
            tma_load_2d_pair(smem_u32(S.w[st]), &p.tm_w, bar, kb * BK, n0);
            tma_load_3d_pair(smem_u32(S.xs[st]), &p.tm_xs, bar, 0, kb, m * 2 + (int)rank);
            tma_load_3d_pair(smem_u32(S.ws[st]), &p.tm_ws, bar, 0, kb, n * 2);
            if (++st == kWideStages) st = 0, ph ^= 1u;
          }
        }
        // The last products of every stage free it in both CTAs: their signals land here before this CTA may exit.
        for (st = 0; ok && st < kWideStages; ++st)
          if (it > st)
            ok = mbar_wait(smem_u32(&S.empty[st]), ((it - 1 - st) / kWideStages) & 1u, abort_flag, p.status,
                           0x860 | st);
        if (!ok) {
          // Loads issued must land before the CTAs may exit.  Only the first CTA's
          // barriers see them; give the second one's the time that they need at most.
          if (rank == 0) {
            for (st = 0; st < kWideStages; ++st)
              if (it > st) mbar_wait(smem_u32(&S.full[st]), ((it - 1 - st) / kWideStages) & 1u, nullptr, nullptr, 0);
          } else {
            const uint64_t t0 = global_ns();
            while (global_ns() - t0 < 2000000ull) {
            }
          }
        }
      }
      __syncwarp();
    } else if (warp == 1 && rank == 0) {
      // ---------------------------------------------------------------- MMA
      // One thread runs the whole loop: a stage's products take about 512 cycles, and
      // a warp-wide loop (votes, an elected branch per stage) took longer than that.
      if (elect_one_sync()) {
        uint32_t it = 0, st = 0, ph = 0, slot = 0, tc = 0;
        bool ok = true;
        const uint64_t xd0 = operand_desc(smem_u32(S.x[0])), wd0 = operand_desc(smem_u32(S.w[0]));
        const uint64_t xsd0 = scale_desc(smem_u32(S.xs[0])), wsd0 = scale_desc(smem_u32(S.ws[0]));
        for (int t = pair; t < tiles && ok; t += pairs, ++tc) {
          if (tc > 0) {  // the columns that this accumulator shares with the last one are drained
            ok = mbar_wait_cluster(smem_u32(&S.acc_free), (tc - 1) & 1u, abort_flag, p.status, 0x810);
            if (!ok) break;
          }
          const uint32_t acc = tmem + kAccShift * (tc & 1u);
          for (int kb = k_begin; kb < k_end; ++kb, ++it) {
            // the scale columns of this slot were last read by the MMAs of step it - kSlots
            if (it >= kSlots) {
              const uint32_t was = it - kSlots;
              ok = mbar_wait(smem_u32(&S.empty[was % kWideStages]), (was / kWideStages) & 1u, abort_flag, p.status,
                             0x830 | st);
            }
            ok = ok && mbar_wait(smem_u32(&S.full[st]), ph, abort_flag, p.status, 0x820 | st);
            if (!ok) break;
            tc_fence_after();
            const uint32_t sx = tmem + kWideScaleCol + slot * 12, sw = sx + 4;
            const uint64_t xd = xd0 + st * (kOperand >> 4), wd = wd0 + st * (kOperand >> 4);
            const uint64_t wsd = wsd0 + st * (2 * kTileBytes >> 4);
            copy_scales_pair(sx, xsd0 + st * (kTileBytes >> 4));
            copy_scales_pair(sw, wsd);
            copy_scales_pair(sw + 4, wsd + (kTileBytes >> 4));
            const int blocks = (p.K - kb * BK) >> 5;  // the blocks past K hold nothing
            if (blocks >= 4) {
#pragma unroll
              for (int b = 0; b < 4; ++b)
                mma_scaled_pair(acc, xd + 2 * b, wd + 2 * b, idesc(256, 256) | idesc_block(b), sx, sw,
                                kb > k_begin || b > 0);
            } else {
              for (int b = 0; b < blocks; ++b)
                mma_scaled_pair(acc, xd + 2 * b, wd + 2 * b, idesc(256, 256) | idesc_block(b), sx, sw,
                                kb > k_begin || b > 0);
            }
            mma_commit_pair(smem_u32(&S.empty[st]), first);
            if (kb == k_end - 1) mma_commit_pair(smem_u32(&S.acc_full[tc & 1u]), first);
            if (++st == kWideStages) st = 0, ph ^= 1u;
            if (++slot == kSlots) slot = 0;
          }
        }
        mma_commit_pair(smem_u32(&S.drain), first);
      }
      __syncwarp();
    }
    if (SPLIT) {
      cluster_sync_all();  // the sums are there
      cluster_arrive();    // (these warps read none)
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ----------------------------------------------------------- epilogue
    // Two groups of four warps share a tile's columns: plain, group g takes columns
    // 128 g .. 128 g + 127; gated, the gates and ups of hidden features 64 g .. 64 g + 63.
    const int group = (warp - 4) >> 2;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t free_bar = cluster_addr(smem_u32(&S.acc_free), first);
    const int tid = threadIdx.x & 127, lane = threadIdx.x & 31;
    uint32_t slot = 0, turn = 0;  // the box that comes, and the parity of its use
    bool coming = false;          // its residual is requested
    uint32_t tc = 0;
    bool ok = true;
    // Each thread brings one of its group's 128 biases a tile, requested a tile ahead.
    const int bias_col = GATED ? (tid < 64 ? 64 * group + tid : 64 + 64 * group + tid) : 128 * group + tid;
    auto load_bias = [&](int t) {
      int m, n;
      tile_of(p, t, m, n);
      const int c = n * 256 + bias_col;
      return p.bias != nullptr && c < p.N ? __bfloat162float(p.bias[c]) : 0.f;
    };
    float next_bias = pair < tiles ? load_bias(pair) : 0.f;
    for (int t = pair; t < tiles && ok; t += pairs, ++tc) {
      const uint32_t buf = tc & 1u;
      int m, n;
      tile_of(p, t, m, n);
      const int n0 = n * 256, row0 = m * 256 + (int)rank * 128 + (warp & 3) * 32;
      const int64_t row = row0 + lane;
      const bool live = row < p.M;
      S.bias[buf][bias_col] = next_bias;
      next_bias = t + pairs < tiles ? load_bias(t + pairs) : 0.f;
      const bool holds = !SPLIT && group != (int)buf;
      // plain: the columns of chunk i, the held ones first, and the next chunk that N reaches
      constexpr int kChunks = SPLIT ? 2 : 4;
      auto chunk_col = [&](int i) {
        return SPLIT ? 128 * part + 64 * group + 32 * i : 128 * group + (holds && group == 1 ? 32 * (i ^ 2) : 32 * i);
      };
      const bool add = !GATED && p.residual != nullptr && row0 < p.M;
      auto request = [&](int from, uint32_t box) {
        for (int i = from; i < kChunks; ++i)
          if (n0 + chunk_col(i) < p.N) {
            if (elect_one_sync()) {
              // the box's last store has been read: only the last one of all may not be
              asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
              const uint32_t bar = smem_u32(&S.res_full[warp - 4][box]);
              mbar_arrive_expect_tx(bar, 32 * 64);
              tma_load_2d(smem_u32(S.stage[warp - 4][box]), &p.tm_res, bar, n0 + chunk_col(i), row0);
            }
            __syncwarp();
            return true;
          }
        return false;
      };
      if (add) coming = request(0, slot);
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&S.acc_full[buf]), (tc >> 1) & 1u, abort_flag, p.status,
                                             0x840 | buf));
      if (!ok) {
        if (SPLIT) {
          cluster_sync_all();
          cluster_arrive();
        }
        break;
      }
      tc_fence_after();
      const uint32_t acc = lane_base + kAccShift * buf;
      // The shared columns, the last 64 of buffer 0 (group 1's) and the first 64 of buffer 1
      // (group 0's), leave tensor memory first.  A group without any arrives too: it is
      // done with the last tile.  Nobody arrives where no tile follows: nothing would wait for
      // the signal to land in the first CTA before it exits.
      uint32_t held[2][32];
      if (holds) {
        const uint32_t shared = buf == 0 ? 192 : 0;
        tmem_ld32(acc + shared, held[0]);
        tmem_ld32(acc + shared + 32, held[1]);
        tmem_wait_ld();
      }
      tc_fence_before();
      __syncwarp();
      if (!SPLIT && lane == 0 && t + pairs < tiles) mbar_arrive_cluster(free_bar);
      named_bar_sync(1 + group, 128);  // the biases are there (and the last tile's are no longer read)
      uint32_t others = 0;  // the other pair's sums of this thread's token and this group's first column
      if (SPLIT) {
        const uint32_t mine = smem_u32(S.x[0]) + ((warp & 3) * 32 + lane) * 4;
        // the other pair's columns, half by each group: plain 64 of 128; gated the gates, the ups
        const int from = GATED ? 128 * group + 64 * (1 - part) : 128 * (1 - part) + 64 * group;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t v[32];
          tmem_ld32(acc + from + 32 * i, v);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e)
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(mine + (64 * group + 32 * i + e) * 512), "r"(v[e])
                         : "memory");
        }
        cluster_sync_all();
        others = cluster_addr(mine, cluster_rank() ^ 2u);
      }
      if (GATED) {
        uint8_t* box = S.stage[warp - 4][slot];
        reuse_box();
        uint32_t scales = 0;  // of the row's two blocks
#pragma unroll
        for (int i = 0; i < (SPLIT ? 1 : 2); ++i) {
          const int c = SPLIT ? 64 * part + 32 * group : 64 * group + 32 * i;
          uint32_t v[32], u[32];
          // a held column is an up column in buffer 0, a gate column in buffer 1
          if (!(holds && buf == 1)) tmem_ld32(acc + c, v);
          if (!(holds && buf == 0)) tmem_ld32(acc + 128 + c, u);
          tmem_wait_ld();
          if (SPLIT) {
            add_others(v, others + 32 * group * 512);
            add_others(u, others + (64 + 32 * group) * 512);
            tc_fence_before();
            cluster_arrive();
          }
          if (holds) {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              if (buf == 1) v[e] = held[i][e];
              else u[e] = held[i][e];
            }
          }
          float y[32], up[32];
          add_bias(y, v, S.bias[buf] + c);
          add_bias(up, u, S.bias[buf] + 128 + c);
          uint32_t top = 0;
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            y[e] = silu(y[e]) * up[e];
            top = max(top, abs_bits(y[e]));
          }
          const uint32_t byte = mx_scale_byte(top);
          const float inv = mx_inv_scale(byte);
          scales |= byte << (8 * i);
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            uint4 o;
            o.x = mx_cvt4(y[16 * g] * inv, y[16 * g + 1] * inv, y[16 * g + 2] * inv, y[16 * g + 3] * inv);
            o.y = mx_cvt4(y[16 * g + 4] * inv, y[16 * g + 5] * inv, y[16 * g + 6] * inv, y[16 * g + 7] * inv);
            o.z = mx_cvt4(y[16 * g + 8] * inv, y[16 * g + 9] * inv, y[16 * g + 10] * inv, y[16 * g + 11] * inv);
            o.w = mx_cvt4(y[16 * g + 12] * inv, y[16 * g + 13] * inv, y[16 * g + 14] * inv, y[16 * g + 15] * inv);
            if (!SPLIT)
              *box_chunk(box, lane, 2 * i + g) = o;
            else if (live)
              reinterpret_cast<uint4*>(p.q + row * p.n_seg + (n0 >> 1) + c)[g] = o;
          }
        }
        if (SPLIT) {
          if (live) p.scale[mx_scale_word(row, n, p.q_tile_cols) + 2 * part + group] = (uint8_t)scales;
          continue;
        }
        if (row0 < p.M) {
          store_box(&p.tm_out[0], box, (n0 >> 1) + 64 * group, row0);
          if (++slot == kBoxes) slot = 0, turn ^= 1u;
        }
        if (live)
          *reinterpret_cast<uint16_t*>(p.scale + mx_scale_word(row, n, p.q_tile_cols) + 2 * group) = (uint16_t)scales;
      } else {
        if (SPLIT) {
          // both chunks' sums, own and the other pair's, before anything is stored
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            tmem_ld32(acc + chunk_col(i), held[i]);
            tmem_wait_ld();
            add_others(held[i], others + (64 * group + 32 * i) * 512);
          }
          tc_fence_before();
          cluster_arrive();
        }
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          // 32 columns to a box, the held ones first
          const int c = chunk_col(i);
          if (n0 + c >= p.N) continue;
          // (in the last segment the TMA drops what is past N; a box that another segment ends
          // in is stored by the threads)
          const int seg = p.n_seg == p.N ? 0 : (n0 + c) / p.n_seg, seg_col = n0 + c - seg * p.n_seg;
          const bool boxed = seg_col + 32 <= p.n_seg || n0 + c - seg_col + p.n_seg == p.N;
          uint8_t* box = S.stage[warp - 4][slot];
          const bool more = add && request(i + 1, slot + 1 == kBoxes ? 0 : slot + 1);
          uint32_t v[32];
          if (!SPLIT && !(holds && i < 2)) tmem_ld32(acc + c, v);
          tmem_wait_ld();
          if (SPLIT || (holds && i < 2)) {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = held[i & 1][e];
          }
          float y[32];
          add_bias(y, v, S.bias[buf] + c);
          if (p.act == QI21_ACT_SILU) {
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = silu(y[e]);
          } else if (p.act == QI21_ACT_GELU_TANH) {
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = gelu_tanh(y[e]);
          }
          if (add) {
            ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&S.res_full[warp - 4][slot]), turn, abort_flag, p.status,
                                                   0x850));
            if (!ok) {
              const uint32_t next = slot + 1 == kBoxes ? 0 : slot + 1;
              if (more)
                mbar_wait(smem_u32(&S.res_full[warp - 4][next]), next == 0 ? turn ^ 1u : turn, nullptr, nullptr, 0);
              break;
            }
            coming = more;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const uint4 rr = *box_chunk(box, lane, g);
              const uint32_t rw[4] = {rr.x, rr.y, rr.z, rr.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 rf = unpack_bf16x2(rw[e]);
                y[8 * g + 2 * e] = fmaf(p.alpha, y[8 * g + 2 * e], rf.x);
                y[8 * g + 2 * e + 1] = fmaf(p.alpha, y[8 * g + 2 * e + 1], rf.y);
              }
            }
          } else {
            if (boxed) reuse_box();
            if (p.alpha != 1.f) {
#pragma unroll
              for (int e = 0; e < 32; ++e) y[e] *= p.alpha;
            }
          }
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            uint4 o;
            o.x = pack_bf16x2(y[8 * g], y[8 * g + 1]);
            o.y = pack_bf16x2(y[8 * g + 2], y[8 * g + 3]);
            o.z = pack_bf16x2(y[8 * g + 4], y[8 * g + 5]);
            o.w = pack_bf16x2(y[8 * g + 6], y[8 * g + 7]);
            if (boxed) {
              *box_chunk(box, lane, g) = o;
            } else if (live && n0 + c + 8 * g < p.N) {
              const int col = n0 + c + 8 * g, own = col / p.n_seg;
              *reinterpret_cast<uint4*>(p.out[own] + row * p.n_seg + (col - own * p.n_seg)) = o;
            }
          }
          if (boxed && row0 < p.M) {  // (rows past M are not written)
            store_box(&p.tm_out[seg], box, seg_col, row0);
            if (++slot == kBoxes) slot = 0, turn ^= 1u;
          }
        }
      }
    }
    // (a request that a broken wait left behind lands before the CTA may exit)
    if (coming) mbar_wait(smem_u32(&S.res_full[warp - 4][slot]), turn, nullptr, nullptr, 0);
    if (elect_one_sync()) bulk_wait_read_all();  // the TMA has read what it was given
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    // every MMA issued completes, and its signal has landed in both CTAs, before TMEM is released
    if (elect_one_sync()) mbar_wait(smem_u32(&S.drain), 0, nullptr, p.status, 0x870);
    __syncwarp();
  }
  if (SPLIT)
    cluster_wait();  // for the arrivals behind the reads of the other pair's sums
  else
    cluster_sync_exit();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

}  // namespace mx

// --------------------------------------------------------------- host side
static PFN_cuTensorMapEncodeTiled_v12000 mx_encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e =
        cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q);
    const bool ok = e == cudaSuccess && q == cudaDriverEntryPointSuccess;
    return ok ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr) : nullptr;
  }();
  return fn;
}

// 2-D map of a row-major [rows, K] e4m3 matrix; box 128 (K) x box_rows, 128-byte
// swizzle, zero fill past the ends.
static bool encode_values(CUtensorMap* m, const void* base, uint64_t rows, uint64_t K, uint32_t box_rows) {
  auto fn = mx_encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {K, rows};
  cuuint64_t strides[1] = {K};
  cuuint32_t box[2] = {(cuuint32_t)mx::BK, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 3-D map of the scale tiles of [rows, K]: (512 bytes as 128 words, tile column,
// row group); a box is `groups` tiles of one tile column.  Row groups past the end
// read as zero (a finite scale).
static bool encode_scales(CUtensorMap* m, const void* base, uint64_t rows, uint64_t K, uint32_t groups) {
  auto fn = mx_encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t cols = (K + 127) / 128;
  cuuint64_t dims[3] = {128, cols, (rows + 127) / 128};
  cuuint64_t strides[2] = {mx::kTileBytes, cols * mx::kTileBytes};
  cuuint32_t box[3] = {128, 1, groups};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 2-D map of a row-major result; boxes of 32 rows x 64 bytes, swizzled.
static bool encode_out(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t bytes) {
  auto fn = mx_encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {cols * bytes};
  cuuint32_t box[2] = {64 / bytes, 32};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, bytes == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
            const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// What splitting K costs in the narrow kernel, ns.
static int64_t split_cost(int blocks, int bn) { return 1500 + bn * (blocks == 2 ? 48 : 12); }

// Tokens per tile, stages, TMEM columns and the split of K for few tokens.
template <bool GATED>
static mx::Narrow narrow_config(const MxGemmArgs& a, int kt, int num_sms) {
  constexpr int NW = GATED ? 2 : 1;
  mx::Narrow c;
  c.bn = a.M >= 128 ? 128 : (int)((a.M + 15) / 16) * 16;
  const int cols = NW * c.bn + mx::kNarrowSlots * (4 * NW + 4);
  c.cols = cols <= 256 ? 256 : 512;
  const int stage = NW * (mx::kW + mx::kTileBytes) + c.bn * mx::BK + mx::kTileBytes;
  const int64_t tiles = ((a.N + NW * 128 - 1) / (NW * 128)) * ((a.M + c.bn - 1) / c.bn);
  // Parts of K: a step takes 310 ns; splitting costs barriers and remote reads, more with more
  // tokens, and pays only while SMs would idle (us in 1 / 2 / 4 / 8 parts: 16 x 4096 x 4096, 32 tiles,
  // 12.6 / 8.9 / 7.9 / 14.5; 1 x 320 x 1568 6.3 / 5.7 / 5.3 / 6.3; 75 x 184 x 7456 22 / 15 / 11.1 / 11.0;
  // 128 x 4096 x 1024 5.8 / 6.9 / 7.7 / 13.9).  Of 37 clusters of 4 CTAs, one to an SM, not all found room on
  // the GPCs at once; 32 did.  One CTA per SM takes all of its shared memory for stages
  // (77 x 12288 x 4096 gated: 34 us with half, 25 with all); more tiles than SMs run in twos.
  c.split = 1;
  int64_t best = (int64_t)kt * 310;
  for (int s = 2; s <= 4 && tiles * s <= (s == 4 ? num_sms - 20 : num_sms) && s <= kt; s *= 2) {
    const int64_t cost = (int64_t)((kt + s - 1) / s) * 310 + split_cost(NW, c.bn);
    if (cost < best) {
      best = cost;
      c.split = s;
    }
  }
  const int room = (c.cols == 256 && tiles * c.split > num_sms ? 110 : 220) * 1024;
  c.stages = room / stage < mx::kNarrowMaxStages ? room / stage : mx::kNarrowMaxStages;
  const int least = (c.cols == 256 ? 76 : 152) * 1024;
  c.smem = c.stages * stage;
  if (c.split > 1 && c.smem < NW * c.bn * 512) c.smem = NW * c.bn * 512;  // the partial sums
  c.smem += 1024;
  if (c.smem < least) c.smem = least;
  return c;
}

template <bool GATED>
static cudaError_t launch_narrow(mx::Params& p, const MxGemmArgs& a, cudaStream_t stream, int num_sms) {
  constexpr int NW = GATED ? 2 : 1;
  const mx::Narrow c = narrow_config<GATED>(a, p.kt, num_sms);
  if (!encode_values(&p.tm_x, a.x, a.M, a.K, c.bn) || !encode_values(&p.tm_w, a.w, a.N, a.K, 128) ||
      !encode_scales(&p.tm_xs, a.x_scale, a.M, a.K, 1) || !encode_scales(&p.tm_ws, a.w_scale, a.N, a.K, 1))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t err = allow_smem(mx::mx_gemm_narrow<GATED>, mx::kNarrowMaxSmem, allowed);
  if (err != cudaSuccess) return err;
  const dim3 grid((unsigned)((a.N + NW * 128 - 1) / (NW * 128)) * c.split, (unsigned)((a.M + c.bn - 1) / c.bn));
  return launch_dependent(mx::mx_gemm_narrow<GATED>, grid, mx::kNarrowThreads, c.smem, c.split, stream, p, c);
}

template <bool GATED, bool SPLIT>
static cudaError_t launch_wide(mx::Params& p, const MxGemmArgs& a, cudaStream_t stream, int num_sms) {
  if (!encode_values(&p.tm_x, a.x, a.M, a.K, 128) || !encode_values(&p.tm_w, a.w, a.N, a.K, 128) ||
      !encode_scales(&p.tm_xs, a.x_scale, a.M, a.K, 1) || !encode_scales(&p.tm_ws, a.w_scale, a.N, a.K, 2))
    return cudaErrorInvalidValue;
  if (a.residual != nullptr && !encode_out(&p.tm_res, a.residual, a.M, a.N, 2)) return cudaErrorInvalidValue;
  for (int i = 0; i < a.n_out; ++i)
    if (!encode_out(&p.tm_out[i], GATED ? a.q : a.out[i], a.M, p.n_seg, GATED ? 1 : 2)) return cudaErrorInvalidValue;
  p.mt = (int32_t)((a.M + 255) / 256);
  p.nt = (int32_t)((a.N + 255) / 256);
  const size_t smem = sizeof(mx::WideSmem) + 1024;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t err = allow_smem(mx::mx_gemm_wide<GATED, SPLIT>, (int)smem, allowed);
  if (err != cudaSuccess) return err;
  const int64_t tiles = (int64_t)p.mt * p.nt;
  const int64_t pairs = tiles < num_sms / 2 ? tiles : num_sms / 2;
  const int cluster = SPLIT ? 4 : 2;
  return launch_dependent(mx::mx_gemm_wide<GATED, SPLIT>, dim3((unsigned)(cluster * pairs)), mx::kWideThreads, smem,
                          cluster, stream, p);
}

static int64_t max64(int64_t a, int64_t b) { return a > b ? a : b; }

// Which kernel for more than one tile of tokens: estimates, in ns, of a launch plus the rounds that the
// tiles take over the SMs.  A round of the narrow kernel is its K steps and then its epilogue; of
// the pairs' the longer of the two, as they overlap, except in the first.  The constants are fits to
// measurements on a B200 (us, narrow / pairs / pairs with K split): 1024 x 4096 x 1024 7.5 / 9.2 / -,
// 4096 x 12288 x 512 60 / 52 / -, 512 x 4096 x 4096 14.9 / 16.1 / 13.7, 512 x 4096 x 12288 37 / 36 / 24.7,
// 1024 x 4096 x 12288 49 / 43 / -, 2048 x 4096 x 4096 42 / 31 / -, 4096 x 4096 x 256 with a residual 36 / 25 / -;
// gated 1024 x 2048 x 128 6.2 / 5.6 / -, 333 x 2048 x 4096 19 / 14 / 12.5, 1000 x 4096 x 4096 40 / 28 / -.
// Over 60 random shapes the chosen kernel was 0.8 % slower than the best of the three on average, and the best for 54
// of them (the narrow one for all of them: 16 % slower, the pairs without a split: 32 %); the worst by 32 %, 361 x
// 6152 x 6112 with a residual, whose 147 CTAs of the narrow kernel take 570 ns a step from L2, not the estimate's 352.
MxPlan mx_gemm_plan(const MxGemmArgs& a, int num_sms) {
  const int kt = (int)((a.K + mx::BK - 1) / mx::BK);
  const mx::Narrow c = a.gated ? narrow_config<true>(a, kt, num_sms) : narrow_config<false>(a, kt, num_sms);
  const MxPlan few{QI21_MX_FEW, c.split}, pairs_whole{QI21_MX_PAIRS, 1}, pairs_split{QI21_MX_PAIRS_SPLIT, 2};
  if (a.M <= 128) return few;
  if (a.M > 128 * 65535ll) return pairs_whole;  // more token tiles than a grid's second axis takes
  const int64_t act = a.act != QI21_ACT_NONE ? 2400 : 0;
  const int64_t features = a.gated ? 256 : 128;
  const int64_t ctas = ((a.N + features - 1) / features) * ((a.M + 127) / 128) * c.split;
  const bool twos = !a.gated && ctas > num_sms;  // two CTAs to an SM
  const int64_t at_once = twos ? 2 * num_sms : num_sms, steps = (kt + c.split - 1) / c.split;
  const int64_t rounds = (ctas + at_once - 1) / at_once;
  const int64_t finish = (a.gated ? 4600 : rounds > 1 ? 3300 : 2400) + (act != 0 ? 1300 : 0) +
                         (a.residual == nullptr ? 0 : rounds > 2 ? 4500 : 1500);
  const int64_t narrow = 1500 + (c.split == 1 ? 0 : split_cost(a.gated ? 2 : 1, c.bn)) +
                         rounds * (finish + steps * (a.gated ? 500 : twos ? 450 : 352));
  const int64_t tiles = ((a.M + 255) / 256) * ((a.N + 255) / 256), pairs = num_sms / 2;
  const int64_t drain = (a.gated ? 2700 : 4400) + act + (a.residual != nullptr ? 1000 : 0);
  const int64_t wide = 2200 + drain + kt * 360 + ((tiles + pairs - 1) / pairs - 1) * max64(kt * 365 + 600, drain);
  // (of 37 clusters of four CTAs, one CTA to an SM, not all found room at once; 32 did)
  const int64_t split = 4 * tiles <= num_sms - 20 && kt >= 8 ? 3000 + drain + (kt + 1) / 2 * 360 : INT64_MAX;
  if (split < narrow && split < wide) return pairs_split;
  return wide < narrow ? pairs_whole : few;
}

cudaError_t launch_mx_gemm(const MxGemmArgs& a, cudaStream_t stream, int num_sms) {
  if (a.M == 0 || a.N == 0) return cudaSuccess;
  mx::Params p;
  memset(&p, 0, sizeof(p));
  p.M = (int32_t)a.M;
  p.N = (int32_t)a.N;
  p.K = (int32_t)a.K;
  p.n_seg = (int32_t)(a.gated ? a.N / 2 : a.N / a.n_out);
  p.kt = (int32_t)((a.K + mx::BK - 1) / mx::BK);
  p.act = a.act;
  p.alpha = a.alpha;
  for (int i = 0; i < a.n_out; ++i) p.out[i] = static_cast<__nv_bfloat16*>(a.out[i]);
  p.bias = static_cast<const __nv_bfloat16*>(a.bias);
  p.residual = static_cast<const __nv_bfloat16*>(a.residual);
  p.q = static_cast<uint8_t*>(a.q);
  p.scale = static_cast<uint8_t*>(a.q_scale);
  p.q_tile_cols = p.n_seg / 128;
  p.status = a.status;
  const int32_t kernel = mx_gemm_plan(a, num_sms).kernel;
  if (kernel == QI21_MX_PAIRS)
    return a.gated ? launch_wide<true, false>(p, a, stream, num_sms) : launch_wide<false, false>(p, a, stream, num_sms);
  if (kernel == QI21_MX_PAIRS_SPLIT)
    return a.gated ? launch_wide<true, true>(p, a, stream, num_sms) : launch_wide<false, true>(p, a, stream, num_sms);
  return a.gated ? launch_narrow<true>(p, a, stream, num_sms) : launch_narrow<false>(p, a, stream, num_sms);
}

}  // namespace qi21
