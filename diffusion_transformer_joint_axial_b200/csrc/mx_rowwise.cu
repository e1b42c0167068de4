// Kernels that write MX (8-bit) rows: the plain quantiser and the RMSNorm with
// the residual's addition in front of it.  Both are bound by memory: each
// value is read once in bf16 and written once in 8 bits.  Measured on a B200 whose
// copies run at 6.55 TB/s: quantising 28160 x 4096 takes 54 us (6.5 TB/s), the norm of
// 28160 x 4096 with the addition 119 us (6.8 TB/s, reads and writes mixed 1 : 0.75); without it 65 us
// (5.3 TB/s), where the instructions, 17 per value, take longer than the memory.
//
// The unit of work is a piece of sixteen consecutive values of a row: two
// neighbouring lanes hold one scale block, eight a row's four blocks of one
// scale tile.  (Pieces of eight, whose accesses are one run per warp, took twice the
// shuffles and scale arithmetic per value: 17 against 10.4 us for quantising 4352 x 4096.
// Multiplying in packed pairs, mul.f32x2, was slower too: 13.2 us.)
#include "qi21_internal.h"
#include "qi21_mx.cuh"

namespace qi21 {

namespace {

struct Piece {
  uint32_t v[8];  // bf16 pairs
};

__device__ __forceinline__ Piece load_piece(const __nv_bfloat16* p) {
  Piece c;
  const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
  c.v[0] = a.x, c.v[1] = a.y, c.v[2] = a.z, c.v[3] = a.w;
  c.v[4] = b.x, c.v[5] = b.y, c.v[6] = b.z, c.v[7] = b.w;
  return c;
}

__device__ __forceinline__ void store_piece(__nv_bfloat16* p, const Piece& c) {
  reinterpret_cast<uint4*>(p)[0] = make_uint4(c.v[0], c.v[1], c.v[2], c.v[3]);
  reinterpret_cast<uint4*>(p)[1] = make_uint4(c.v[4], c.v[5], c.v[6], c.v[7]);
}

// Quantises the sixteen values factor * y of this lane and stores them with
// their scales; `top` is the largest |y|, NaN if there is a NaN.  Called by whole
// warps; `live` is false for lanes past the row's end (their blocks read as byte
// 0).  The first lane of a tile's eight stores its four scale bytes.
__device__ __forceinline__ void store_mx(const float2 (&y)[8], float top, float factor, bool live, uint8_t* q,
                                         uint8_t* scale_word) {
  // (rounding is monotonic: the largest product is the product of the largest)
  uint32_t bits = abs_bits(top * factor);
  bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, 1));
  const uint32_t byte = live ? mx_scale_byte(bits) : 0u;
  const float inv = mx_inv_scale(byte);
  uint32_t word = byte | (__shfl_down_sync(0xffffffffu, byte, 2) << 8);
  word |= __shfl_down_sync(0xffffffffu, word, 4) << 16;
  if (live) {
    // factor * 2^-e is exact, except for blocks of tiny values, where it could leave the range
    const float s = byte >= 64u ? factor * inv : factor;
    float2 z[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = make_float2(y[e].x * s, y[e].y * s);
    if (byte < 64u) {
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] = make_float2(z[e].x * inv, z[e].y * inv);
    }
    uint4 o;
    o.x = mx_cvt4(z[0].x, z[0].y, z[1].x, z[1].y);
    o.y = mx_cvt4(z[2].x, z[2].y, z[3].x, z[3].y);
    o.z = mx_cvt4(z[4].x, z[4].y, z[5].x, z[5].y);
    o.w = mx_cvt4(z[6].x, z[6].y, z[7].x, z[7].y);
    *reinterpret_cast<uint4*>(q) = o;
    if ((threadIdx.x & 7) == 0) *reinterpret_cast<uint32_t*>(scale_word) = word;
  }
}

// One thread per piece, eight threads per (row, tile column).
__global__ void __launch_bounds__(256) mx_quantize_kernel(int64_t groups, int32_t K, int32_t tile_cols,
                                                          const __nv_bfloat16* __restrict__ x,
                                                          uint8_t* __restrict__ q, uint8_t* __restrict__ scale) {
  let_next_start();
  first_wait();
  const int64_t g = blockIdx.x * (int64_t)32 + (threadIdx.x >> 3);
  const int64_t row = g / tile_cols;
  const int32_t tc = (int32_t)(g - row * tile_cols), col = tc * 128 + (threadIdx.x & 7) * 16;
  const bool live = g < groups && col < K;
  float2 y[8] = {};
  float top = 0.f;
  if (live) {
    const Piece c = load_piece(x + row * K + col);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y[e] = unpack_bf16x2(c.v[e]);
      top = max3_abs_nan(top, y[e].x, y[e].y);
    }
  }
  store_mx(y, top, 1.f, live, q + row * K + col, scale + mx_scale_word(row, tc, tile_cols));
}

// TR threads per row (256 / TR rows a CTA), C pieces a thread.  First step: h = x
// (+ delta, rounded to bf16 and stored in `sum`), its sum of squares, and h * w (a
// product of two bf16, exact in fp32) with its largest magnitude, held in registers.  Second
// step: (h * w) / sqrt(mean + eps), quantised.  C = 0: rows of any length; the second
// step reads h back (each thread what it wrote).  `sum` may be x or delta: a thread
// reads each value before it writes it.
template <int TR, int C, bool ADD>
__global__ void __launch_bounds__(256) rmsnorm_mx_kernel(int64_t M, int32_t D, int32_t tile_cols,
                                                         const __nv_bfloat16* x, const __nv_bfloat16* delta,
                                                         const __nv_bfloat16* __restrict__ w, float inv_d, float eps,
                                                         __nv_bfloat16* sum, uint8_t* __restrict__ q,
                                                         uint8_t* __restrict__ scale) {
  constexpr int kWarps = TR / 32, kKept = C > 0 ? C : 1;
  __shared__ float part[8];
  let_next_start();
  first_wait();
  const int t = threadIdx.x % TR;
  const int64_t row = blockIdx.x * (int64_t)(256 / TR) + threadIdx.x / TR;
  const int pieces = row < M ? D / 16 : 0;  // (whole warps have none)
  x += row * D;
  q += row * D;
  if (ADD) {
    delta += row * D;
    sum += row * D;
  }
  scale += mx_scale_word(row, 0, tile_cols);

  auto add = [&](int i, Piece& h, const Piece& d) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 a = unpack_bf16x2(h.v[e]), b = unpack_bf16x2(d.v[e]);
      h.v[e] = pack_bf16x2(a.x + b.x, a.y + b.y);
    }
    store_piece(sum + 16 * i, h);
  };
  float2 ss = make_float2(0.f, 0.f);
  auto squares = [&](const float2 (&f)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      ss = make_float2(fmaf(f[e].x, f[e].x, ss.x), fmaf(f[e].y, f[e].y, ss.y));
  };
  auto weigh = [&](float2 (&f)[8], const Piece& g) {
    float most = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 b = unpack_bf16x2(g.v[e]);
      f[e] = make_float2(f[e].x * b.x, f[e].y * b.y);
      most = max3_abs_nan(most, f[e].x, f[e].y);
    }
    return most;
  };
  auto unpack = [](float2 (&f)[8], const Piece& h) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = unpack_bf16x2(h.v[e]);
  };

  float2 y[kKept][8];
  float top[kKept];
  if (C > 0) {
    Piece h[kKept], d[kKept];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = c * TR + t;
      if (i < pieces) {
        h[c] = load_piece(x + 16 * i);
        if (ADD) d[c] = load_piece(delta + 16 * i);
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = c * TR + t;
      if (i < pieces) {
        if (ADD) add(i, h[c], d[c]);
        unpack(y[c], h[c]);
        squares(y[c]);
        top[c] = weigh(y[c], load_piece(w + 16 * i));
      }
    }
  } else {
    for (int i = t; i < pieces; i += TR) {
      Piece h = load_piece(x + 16 * i);
      if (ADD) add(i, h, load_piece(delta + 16 * i));
      unpack(y[0], h);
      squares(y[0]);
    }
  }

  float all = ss.x + ss.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
  if (kWarps > 1) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = all;
    __syncthreads();
    all = part[threadIdx.x / TR * kWarps + (threadIdx.x & (kWarps - 1))];
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
  }
  const float rs = rsqrtf(fmaf(all, inv_d, eps));

  if (C > 0) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = c * TR + t;
      if (c * TR + (t & ~31) < pieces) store_mx(y[c], top[c], rs, i < pieces, q + 16 * i, scale + (i >> 3) * 512);
    }
  } else {
    const __nv_bfloat16* h = ADD ? sum : x;
    for (int base = 0; base < pieces; base += TR) {
      const int i = base + t;
      if (i < pieces) {
        unpack(y[0], load_piece(h + 16 * i));
        top[0] = weigh(y[0], load_piece(w + 16 * i));
      }
      store_mx(y[0], top[0], rs, i < pieces, q + 16 * i, scale + (int64_t)(i >> 3) * 512);
    }
  }
}

template <int TR, int C>
cudaError_t run_rmsnorm_mx(int64_t M, int32_t D, const void* x, const void* delta, const void* w, float eps,
                           void* sum, void* q, void* scale, cudaStream_t stream) {
  constexpr int kRows = 256 / TR;
  return launch_dependent(delta != nullptr ? rmsnorm_mx_kernel<TR, C, true> : rmsnorm_mx_kernel<TR, C, false>,
                          dim3((unsigned)((M + kRows - 1) / kRows)), 256, 0, 1, stream, M, D, (D + 127) / 128,
                          static_cast<const __nv_bfloat16*>(x), static_cast<const __nv_bfloat16*>(delta),
                          static_cast<const __nv_bfloat16*>(w), 1.f / static_cast<float>(D), eps,
                          static_cast<__nv_bfloat16*>(sum),
                          static_cast<uint8_t*>(q), static_cast<uint8_t*>(scale));
}

}  // namespace

cudaError_t launch_mx_quantize(int64_t M, int64_t K, const void* x, void* q, void* scale, cudaStream_t stream) {
  if (M == 0 || K == 0) return cudaSuccess;
  const int32_t tile_cols = (int32_t)((K + 127) / 128);
  const int64_t groups = M * tile_cols;
  return launch_dependent(mx_quantize_kernel, dim3((unsigned)((groups + 31) / 32)), 256, 0, 1, stream, groups,
                          (int32_t)K, tile_cols, static_cast<const __nv_bfloat16*>(x), static_cast<uint8_t*>(q),
                          static_cast<uint8_t*>(scale));
}

cudaError_t launch_rmsnorm_mx(int64_t M, int32_t D, const void* x, const void* delta, const void* w, float eps,
                              void* sum, void* q, void* scale, cudaStream_t stream) {
  if (M == 0) return cudaSuccess;
  // Enough threads to a row for all of it to be in registers, three pieces a thread at
  // most; one piece a thread where that leaves few of them idle (28160 x 4096: 66 us with
  // 256 threads of one piece, 72 with 128 of two; 4352 x 12288: 36 us with 256 of three, 56 with 256 of
  // four).
  const int pieces = D / 16;
  auto run = pieces <= 32    ? run_rmsnorm_mx<32, 1>
             : pieces <= 64  ? run_rmsnorm_mx<64, 1>
             : pieces <= 96  ? run_rmsnorm_mx<32, 3>
             : pieces <= 128 ? run_rmsnorm_mx<128, 1>
             : pieces <= 192 ? run_rmsnorm_mx<64, 3>
             : pieces <= 256 ? run_rmsnorm_mx<256, 1>
             : pieces <= 384 ? run_rmsnorm_mx<128, 3>
             : pieces <= 512 ? run_rmsnorm_mx<256, 2>
             : pieces <= 768 ? run_rmsnorm_mx<256, 3>
                             : run_rmsnorm_mx<256, 0>;
  return run(M, D, x, delta, w, eps, sum, q, scale, stream);
}

}  // namespace qi21
