// MXFP4 rows: quantisation and read-back (format in mx_dev.h).
//
// Rows are contiguous and a multiple of 32 long, so a matrix is one run of
// 32-element blocks.  Four lanes take one block, 8 elements each: the block
// maximum is the integer maximum of the magnitudes' bit patterns over the four
// lanes (it orders finite values, infinities and NaN alike), the scale the
// smallest power of two that leaves no element beyond 6, and each lane writes
// its 8 codes as one 4-byte word.  Both are bound by memory: 6.0 and 5.9 TB/s
// over all bytes at 65537 rows of 4096 bf16.
#include "moe_internal.h"
#include "mx_dev.h"
#include "wave_dev.h"

namespace moe {
namespace {

using namespace mx_dev;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// 8 consecutive elements as fp32.
template <bool BF16>
__device__ __forceinline__ void load8(const void* src, int64_t i, float* v) {
  if constexpr (BF16) {
    const u32x4 u = reinterpret_cast<const u32x4*>(src)[i];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(u[j] << 16);
      v[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
    }
  } else {
    const u32x4 a = reinterpret_cast<const u32x4*>(src)[2 * i];
    const u32x4 b = reinterpret_cast<const u32x4*>(src)[2 * i + 1];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = __uint_as_float(a[j]);
      v[4 + j] = __uint_as_float(b[j]);
    }
  }
}

template <bool BF16>
__global__ __launch_bounds__(256) void quantize_mxfp4_kernel(const void* __restrict__ src,
                                                             uint32_t* __restrict__ q,
                                                             uint8_t* __restrict__ scale,
                                                             int64_t n8) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n8) return;                       // whole blocks (4 lanes) leave together
  float v[8];
  load8<BF16>(src, i, v);
  uint32_t a = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) a = max(a, __float_as_uint(v[j]) & 0x7fffffffu);
  a = max(a, (uint32_t)wave_dev::dpp<0xB1>((int)a));   // lane ^ 1
  a = max(a, (uint32_t)wave_dev::dpp<0x4E>((int)a));   // lane ^ 2
  const uint32_t b = block_e8m0(a);
  q[i] = e2m1x8(v, b);
  if ((threadIdx.x & 3) == 0) scale[i >> 2] = (uint8_t)b;
}

// PAST: bf16 stores that leave no line in the caches.
template <bool BF16, bool PAST>
__global__ __launch_bounds__(256) void dequantize_mxfp4_kernel(const uint32_t* __restrict__ q,
                                                               const uint8_t* __restrict__ scale,
                                                               void* __restrict__ dst,
                                                               int64_t n8) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n8) return;
  const uint32_t w = q[i], b = scale[i >> 2];
  // a NaN block reads back as NaN whatever its codes
  const u32x4 v = b == 255 ? u32x4{0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u}
                           : e2m1x8_to_bf16(w, e8m0_float(b));
  if constexpr (BF16) {
    u32x4* p = reinterpret_cast<u32x4*>(dst) + i;
    if constexpr (PAST) __builtin_nontemporal_store(v, p);
    else *p = v;
  } else {
    // every value is a bf16 value: widening is exact
    u32x4* p = reinterpret_cast<u32x4*>(dst) + 2 * i;
    p[0] = u32x4{v[0] << 16, v[0] & 0xffff0000u, v[1] << 16, v[1] & 0xffff0000u};
    p[1] = u32x4{v[2] << 16, v[2] & 0xffff0000u, v[3] << 16, v[3] & 0xffff0000u};
  }
}

}  // namespace

void launch_quantize_mxfp4(int dtype, int64_t n, const void* src, uint8_t* q, uint8_t* scale,
                           hipStream_t s) {
  const int64_t n8 = n / 8;
  if (n8 == 0) return;
  const unsigned grid = (unsigned)((n8 + 255) / 256);
  if (dtype == MOE_DT_BF16)
    quantize_mxfp4_kernel<true><<<grid, 256, 0, s>>>(src, (uint32_t*)q, scale, n8);
  else
    quantize_mxfp4_kernel<false><<<grid, 256, 0, s>>>(src, (uint32_t*)q, scale, n8);
}

void launch_dequantize_mxfp4(int dtype, int64_t n, const uint8_t* q, const uint8_t* scale,
                             void* dst, hipStream_t s) {
  const int64_t n8 = n / 8;
  if (n8 == 0) return;
  const unsigned grid = (unsigned)((n8 + 255) / 256);
  // A result beyond half of the 256 MB last-level cache is not kept for its
  // reader in any case.  Written past the caches against through them, alone
  // and with a pass that reads it: 11.2 / 14.6 and 35.5 / 34.2 us at 64 MB,
  // 41.5 / 67.1 and 147 / 150 at 224 MB, 92 / 156 and 326 / 333 at 512 MB.
  // (fp32 lanes write half lines, which past the caches take 1.5 to 2 times as
  // long.)
  const bool past = 2 * n > (int64_t)128 << 20;
  const uint32_t* w = (const uint32_t*)q;
  if (dtype != MOE_DT_BF16)
    dequantize_mxfp4_kernel<false, false><<<grid, 256, 0, s>>>(w, scale, dst, n8);
  else if (past)
    dequantize_mxfp4_kernel<true, true><<<grid, 256, 0, s>>>(w, scale, dst, n8);
  else
    dequantize_mxfp4_kernel<true, false><<<grid, 256, 0, s>>>(w, scale, dst, n8);
}

}  // namespace moe
