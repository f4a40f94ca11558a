// ft_fp8_quantize: rows to FP8 with one scale per block of 128, the operand
// format of ft_fp8_gemm, ft_grouped_gemm and the FT_FP8 experts.
//
//   s = 2^max(-126, ceil(log2(amax / 448))),   c = e4m3(x / s), ties to even
//
// over blocks of 1 x 128 (activations) or 128 x 128 (weights).  The scale is a
// power of two so that x / s is a shift of the exponent: exact in fp32, which
// leaves the conversion to E4M3 as the only rounding and makes the codes a
// function of the input alone, with no tie decided by a rounded quotient.
// (With s = amax / 448 a quarter percent of bf16 inputs sat on such ties.)  E4M3
// keeps its relative step over 15 binades, so the half binade that a power of
// two gives away on average costs no precision except near the subnormals.
// A block that holds a NaN or an infinity has no scale: s = NaN, codes 0, so
// every product over it is NaN.
//
// The kernels only move bytes: 2 (or 4) in and 1 out per element.  A 16-lane row
// of a wave holds one 1 x 128 block, 8 elements (16 bytes of bf16) per lane,
// and takes the block's maximum with four DPP lane moves.  8192 x 4096 bf16 by
// 1 x 128: 20.4 us, 5.0 TB/s read and written together (a device copy: 5.2);
// a 4096 x 2048 weight by 128 x 128: 7.0 us, of which the launch is about 5.
#include "ft_internal.hpp"
#include "fp8_util.hpp"

namespace ft {

template <typename X>
__global__ __launch_bounds__(256) void fp8_quantize_rows_kernel(const X *__restrict__ x, int64_t ldx, int64_t n, int K,
                                                                int kb, uint8_t *__restrict__ codes, int64_t ldc,
                                                                float *__restrict__ scales) {
  const int64_t b = int64_t(blockIdx.x) * 16 + (threadIdx.x >> 4);
  if (b >= n * kb) return;  // whole 16-lane rows: the lane moves below stay inside one
  const int64_t row = b / kb;
  const int j = int(b % kb), l = threadIdx.x & 15, c = j * kFp8Block + l * 8;
  float v[8];
  if (c < K) {
    fp8_load8(x + row * ldx + c, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
  }
  const uint32_t amax = row16_max_u32(abs_max8(v));
  const Fp8Scale s = fp8_scale(amax);
  if (c < K) *reinterpret_cast<u32x2 *>(codes + row * ldc + c) = fp8_codes8(v, s.inv);
  if (l == 0) scales[row * kb + j] = s.scale;
}

// One 128 x 128 block per workgroup: each 16-lane row takes 8 of its rows.
template <typename X>
__global__ __launch_bounds__(256) void fp8_quantize_tiles_kernel(const X *__restrict__ x, int64_t ldx, int64_t n, int K,
                                                                 int kb, uint8_t *__restrict__ codes, int64_t ldc,
                                                                 float *__restrict__ scales) {
  __shared__ uint32_t s_max[4];
  const int64_t bi = int64_t(blockIdx.x) / kb;
  const int j = int(int64_t(blockIdx.x) % kb), l = threadIdx.x & 15, c = j * kFp8Block + l * 8;
  const int64_t row0 = bi * kFp8Block + (threadIdx.x >> 4);
  float v[8][8];
  uint32_t amax = 0;
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    const int64_t row = row0 + t * 16;
    if (c < K && row < n) {
      fp8_load8(x + row * ldx + c, v[t]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[t][i] = 0.f;
    }
  }
#pragma unroll
  for (int t = 0; t < 8; ++t) amax = max(amax, abs_max8(v[t]));
  amax = wave_max_u32(amax);
  if ((threadIdx.x & 63) == 0) s_max[threadIdx.x >> 6] = amax;
  __syncthreads();
  const Fp8Scale s = fp8_scale(max(max(s_max[0], s_max[1]), max(s_max[2], s_max[3])));
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    const int64_t row = row0 + t * 16;
    if (c < K && row < n) *reinterpret_cast<u32x2 *>(codes + row * ldc + c) = fp8_codes8(v[t], s.inv);
  }
  if (threadIdx.x == 0) scales[bi * kb + j] = s.scale;
}

template <typename X>
static ft_status quantize_launch(const X *x, int64_t ldx, int64_t n, int K, int block_rows, uint8_t *codes, int64_t ldc,
                                 float *scales, hipStream_t stream) {
  const int kb = cdiv(K, kFp8Block);
  if (block_rows == 1) {
    const int64_t grid = cdiv<int64_t>(n * kb, 16);
    hipLaunchKernelGGL((fp8_quantize_rows_kernel<X>), dim3(unsigned(grid)), dim3(256), 0, stream, x, ldx, n, K, kb, codes,
                       ldc, scales);
    FT_LAUNCHED("fp8_quantize_rows_kernel");
  } else {
    const int64_t grid = cdiv<int64_t>(n, kFp8Block) * kb;
    hipLaunchKernelGGL((fp8_quantize_tiles_kernel<X>), dim3(unsigned(grid)), dim3(256), 0, stream, x, ldx, n, K, kb, codes,
                       ldc, scales);
    FT_LAUNCHED("fp8_quantize_tiles_kernel");
  }
  return FT_OK;
}

ft_status fp8_quantize_launch(const void *x, int x_dtype, int64_t ldx, int64_t n, int K, int block_rows, uint8_t *codes,
                              int64_t ldc, float *scales, hipStream_t stream) {
  if (x_dtype == FT_BF16)
    return quantize_launch(static_cast<const uint16_t *>(x), ldx, n, K, block_rows, codes, ldc, scales, stream);
  return quantize_launch(static_cast<const float *>(x), ldx, n, K, block_rows, codes, ldc, scales, stream);
}

}  // namespace ft

using namespace ft;

extern "C" ft_status ft_fp8_quantize(const void *x, int32_t x_dtype, int64_t ldx, int64_t n, int32_t K,
                                     int32_t block_rows, uint8_t *codes, int64_t ldc, float *scales,
                                     hipStream_t stream) {
  FT_REQUIRE(x_dtype == FT_BF16 || x_dtype == FT_F32, "ft_fp8_quantize: x_dtype must be FT_BF16 or FT_F32");
  FT_REQUIRE(block_rows == 1 || block_rows == 128, "ft_fp8_quantize: block_rows must be 1 or 128");
  FT_REQUIRE(n >= 0 && K >= 0, "ft_fp8_quantize: need n >= 0, K >= 0");
  FT_SUPPORTED(K % 16 == 0, "ft_fp8_quantize: K must be a multiple of 16");
  FT_REQUIRE(ldx >= K && ldc >= K, "ft_fp8_quantize: row pitch below K");
  FT_SUPPORTED(n < (int64_t(1) << 31) && n * cdiv(K, kFp8Block) < (int64_t(1) << 28) - 16,  // 2^32 threads of 8 elements
               "ft_fp8_quantize: 2^31 rows, or rows of 2^28 - 16 blocks together, or more");
  if (n == 0 || K == 0) {
    clear_error();
    return FT_OK;
  }
  FT_REQUIRE(x && codes && scales, "ft_fp8_quantize: NULL pointer argument");
  FT_REQUIRE(ldx % 8 == 0 && ldc % 16 == 0 && aligned(x, 16) && aligned(codes, 16) && aligned(scales, 4),
             "ft_fp8_quantize: x and codes must be 16-byte aligned, ldx a multiple of 8, ldc of 16");
  const ft_status st = fp8_quantize_launch(x, x_dtype, ldx, n, K, block_rows, codes, ldc, scales, stream);
  if (st != FT_OK) return st;
  clear_error();
  return FT_OK;
}
