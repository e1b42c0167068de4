// Kernels that write MX (8-bit) rows: the plain quantiser and the RMSNorm with
// the residual's addition in front of it.  Both are bound by memory: each
// value is read once in bf16 and written once in 8 bits.
#include "qi21_internal.h"
#include "qi21_mx.cuh"

namespace qi21 {

namespace {

// Sixteen consecutive bf16 values of a row: the unit one thread works on.  Two
// neighbouring lanes hold one scale block, eight lanes one tile's four blocks.
struct Chunk {
  uint32_t v[8];
};

__device__ __forceinline__ Chunk load_chunk(const __nv_bfloat16* p) {
  Chunk c;
  const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
  c.v[0] = a.x, c.v[1] = a.y, c.v[2] = a.z, c.v[3] = a.w;
  c.v[4] = b.x, c.v[5] = b.y, c.v[6] = b.z, c.v[7] = b.w;
  return c;
}

__device__ __forceinline__ void store_chunk(__nv_bfloat16* p, const Chunk& c) {
  reinterpret_cast<uint4*>(p)[0] = make_uint4(c.v[0], c.v[1], c.v[2], c.v[3]);
  reinterpret_cast<uint4*>(p)[1] = make_uint4(c.v[4], c.v[5], c.v[6], c.v[7]);
}

// Quantises the sixteen values y of this lane's chunk and stores them with
// their scales.  Called by whole warps; `live` is false for lanes past the row's end
// (their block counts as absent: byte 0).  Lanes 8g..8g+7 hold one tile's
// four blocks of a row, the first of them stores the four bytes.
__device__ __forceinline__ void store_mx(const float (&y)[16], bool live, uint8_t* q, uint8_t* scale_word) {
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 16; ++e) top = max(top, abs_bits(y[e]));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  const uint32_t byte = live ? mx_scale_byte(top) : 0u;
  const float inv = mx_inv_scale(byte);
  if (live) {
    uint4 o;
    o.x = mx_cvt4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
    o.y = mx_cvt4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv);
    o.z = mx_cvt4(y[8] * inv, y[9] * inv, y[10] * inv, y[11] * inv);
    o.w = mx_cvt4(y[12] * inv, y[13] * inv, y[14] * inv, y[15] * inv);
    *reinterpret_cast<uint4*>(q) = o;
  }
  uint32_t word = byte | (__shfl_down_sync(0xffffffffu, byte, 2) << 8);
  word |= __shfl_down_sync(0xffffffffu, word, 4) << 16;
  if (live && (threadIdx.x & 7) == 0) *reinterpret_cast<uint32_t*>(scale_word) = word;
}

// One thread per chunk, eight threads per (row, tile column).
__global__ void __launch_bounds__(256) mx_quantize_kernel(int64_t groups, int32_t K, int32_t tile_cols,
                                                          const __nv_bfloat16* __restrict__ x,
                                                          uint8_t* __restrict__ q, uint8_t* __restrict__ scale) {
  const int64_t g = blockIdx.x * (int64_t)32 + (threadIdx.x >> 3);
  const int64_t row = g / tile_cols;
  const int32_t tc = (int32_t)(g - row * tile_cols), col = tc * 128 + (threadIdx.x & 7) * 16;
  const bool live = g < groups && col < K;
  float y[16] = {};
  if (live) {
    const Chunk c = load_chunk(x + row * K + col);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 f = unpack_bf16x2(c.v[e]);
      y[2 * e] = f.x;
      y[2 * e + 1] = f.y;
    }
  }
  store_mx(y, live, q + row * K + col, scale + mx_scale_word(row, tc, tile_cols));
}

// One CTA per row: h = x (+ delta, rounded to bf16 and stored in `sum`), the sum
// of squares of the stored h, then y = h / sqrt(mean + eps) * w, quantised.  `sum`
// may be x or delta: a thread reads each value before it writes it, and reads it
// back itself.
__global__ void __launch_bounds__(256) rmsnorm_mx_kernel(int32_t D, int32_t tile_cols, const __nv_bfloat16* x,
                                                         const __nv_bfloat16* delta,
                                                         const __nv_bfloat16* __restrict__ w, float eps,
                                                         __nv_bfloat16* sum, uint8_t* __restrict__ q,
                                                         uint8_t* __restrict__ scale) {
  __shared__ float part[8];
  const int64_t row = blockIdx.x;
  const __nv_bfloat16* h = delta != nullptr ? sum : x;
  float ss = 0.f;
  for (int32_t col = threadIdx.x * 16; col < D; col += 256 * 16) {
    Chunk c = load_chunk(x + row * D + col);
    if (delta != nullptr) {
      const Chunk d = load_chunk(delta + row * D + col);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 a = unpack_bf16x2(c.v[e]), b = unpack_bf16x2(d.v[e]);
        c.v[e] = pack_bf16x2(a.x + b.x, a.y + b.y);
      }
      store_chunk(sum + row * D + col, c);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 f = unpack_bf16x2(c.v[e]);
      ss = fmaf(f.x, f.x, fmaf(f.y, f.y, ss));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = ss;
  __syncthreads();
  ss = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss += part[i];
  const float rs = 1.f / sqrtf(ss / static_cast<float>(D) + eps);
  for (int32_t base = 0; base < D; base += 256 * 16) {
    const int32_t col = base + threadIdx.x * 16;
    const bool live = col < D;
    float y[16] = {};
    if (live) {
      const Chunk c = load_chunk(h + row * D + col), g = load_chunk(w + col);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 a = unpack_bf16x2(c.v[e]), b = unpack_bf16x2(g.v[e]);
        y[2 * e] = a.x * rs * b.x;
        y[2 * e + 1] = a.y * rs * b.y;
      }
    }
    store_mx(y, live, q + row * D + col, scale + mx_scale_word(row, col >> 7, tile_cols));
  }
}

}  // namespace

cudaError_t launch_mx_quantize(int64_t M, int64_t K, const void* x, void* q, void* scale, cudaStream_t stream) {
  if (M == 0 || K == 0) return cudaSuccess;
  const int32_t tile_cols = (int32_t)((K + 127) / 128);
  const int64_t groups = M * tile_cols;
  mx_quantize_kernel<<<(unsigned)((groups + 31) / 32), 256, 0, stream>>>(
      groups, (int32_t)K, tile_cols, static_cast<const __nv_bfloat16*>(x), static_cast<uint8_t*>(q),
      static_cast<uint8_t*>(scale));
  note_launch();
  return cudaGetLastError();
}

cudaError_t launch_rmsnorm_mx(int64_t M, int32_t D, const void* x, const void* delta, const void* w, float eps,
                              void* sum, void* q, void* scale, cudaStream_t stream) {
  if (M == 0) return cudaSuccess;
  rmsnorm_mx_kernel<<<(unsigned)M, 256, 0, stream>>>(
      D, (D + 127) / 128, static_cast<const __nv_bfloat16*>(x), static_cast<const __nv_bfloat16*>(delta),
      static_cast<const __nv_bfloat16*>(w), eps, static_cast<__nv_bfloat16*>(sum), static_cast<uint8_t*>(q),
      static_cast<uint8_t*>(scale));
  note_launch();
  return cudaGetLastError();
}

}  // namespace qi21
