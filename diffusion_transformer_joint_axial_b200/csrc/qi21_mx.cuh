// The 8-bit (MX) storage of libqi21: e4m3 values, one e8m0 (power of two)
// scale per 32 consecutive values of a row.
//
// For a block with largest magnitude A the exponent e is the smallest integer
// with A <= 448 * 2^e (448 = the largest e4m3 value, so nothing saturates), at
// least -127; the stored values are x * 2^-e rounded to nearest even, the
// scale byte is e + 127.  An all-zero block stores byte 0 and zeros.  A block
// that holds a NaN or an infinity stores byte 255 and NaN codes: it reads back as
// NaN, and a product with it is NaN.
#pragma once

#include <atomic>

#include "qi21_cluster.cuh"

namespace qi21 {

constexpr uint32_t kMxNanByte = 255;

// Bit pattern of |x|: as unsigned integers these order like the magnitudes,
// with infinity and then the NaNs above every finite value.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// max(top, |a|, |b|) for top >= 0; a NaN anywhere gives a NaN.
__device__ __forceinline__ float max3_abs_nan(float top, float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(top), "f"(fabsf(a)), "f"(fabsf(b)));
  return d;
}

// Scale byte of a block whose largest abs_bits() is `bits`.  With A = m * 2^x,
// 1 <= m < 2, and 448 = 1.75 * 2^8: e = x - 8 if m <= 1.75, else x - 7.  Adding
// 2^21 - 1 to the bits carries into the exponent exactly when the mantissa is
// above 0.75 * 2^23.  (A subnormal A gives byte 0 as it must: e = -127.)
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t bits) {
  if (bits >= 0x7f800000u) return kMxNanByte;
  const uint32_t x = (bits + 0x1fffffu) >> 23;
  return x > 8u ? x - 8u : 0u;
}

// 2^-e of a scale byte: exact, and normal for every byte mx_scale_byte()
// returns below 255 (at most 247).  The NaN byte gives a NaN factor, which turns
// every value of its block into a NaN code.
__device__ __forceinline__ float mx_inv_scale(uint32_t byte) {
  return byte == kMxNanByte ? __uint_as_float(0x7fffffffu) : __uint_as_float((254u - byte) << 23);
}

// Two values to e4m3 (round to nearest even); `lo` in the low byte.
__device__ __forceinline__ uint32_t mx_cvt2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t mx_cvt4(float a, float b, float c, float d) {
  return mx_cvt2(a, b) | (mx_cvt2(c, d) << 16);
}

// Scales lie in tiles of 128 rows x 4 blocks, 512 bytes each, the form in which
// the tensor cores take them: the byte of (row, block) is at
//   tile(row / 128, block / 4) + (row % 32) * 16 + (row % 128) / 32 * 4 + block % 4
// with the tiles of one row group contiguous.  mx_scale_word() is the offset of
// the four bytes of a row in one tile.
__host__ __device__ __forceinline__ int64_t mx_scale_word(int64_t row, int64_t tile_col, int64_t tile_cols) {
  return ((row >> 7) * tile_cols + tile_col) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4;
}

// Launches `kernel` so that its start may overlap the end of the kernel in front of
// it in the stream (see first_wait()); `cluster` > 1: clusters of that many CTAs
// along x.  Repeated calls of 20 us kernels ran 2 us apart closer for it.
template <typename... P, typename... A>
inline cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster,
                                    cudaStream_t stream, const A&... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e != cudaSuccess) return e;
  note_launch();
  return cudaGetLastError();
}

// Raises `kernel`'s dynamic shared memory limit to `bytes` on the current device,
// once for each (the call costs half a microsecond).
template <typename K>
inline cudaError_t allow_smem(K* kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

}  // namespace qi21
