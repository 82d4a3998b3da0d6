// What the grouped GEMM kernels share: the persistent grid, the tile table that
// every workgroup builds from the segment offsets, the waits and copies of the
// LDS rings, and the bf16 epilogue arithmetic.
#pragma once

#include <math.h>

#include <mutex>

#include "moe_internal.h"
#include "wave_dev.h"

namespace moe {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x8 __attribute__((ext_vector_type(8)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// Row tiles that share a weight slice in the tile order (groups of 4, 16 or
// 32 measured 0.5-3% slower on the ragged layers).
constexpr int kGroupM = 8;
constexpr size_t kMaxLdsBytes = 160 * 1024;  // LDS per workgroup on gfx950

// Workgroup ids are dealt round-robin to the 8 XCDs; renumber them so that
// consecutive logical ids share an XCD (and its L2).  Measured 2-5% faster
// than the plain order on the ragged and DeepSeek-shaped layers.
__device__ __forceinline__ int xcd_logical(int bid, int G) {
  return (bid % 8) * (G / 8) + bid / 8;
}

__device__ __forceinline__ float silu(float z) { return z / (1.0f + expf(-z)); }

__device__ __forceinline__ uint16_t to_bf16(float f) {
  return __builtin_bit_cast(uint16_t, (__bf16)f);
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  return (uint32_t)to_bf16(lo) | ((uint32_t)to_bf16(hi) << 16);
}

// ---------------------------------------------------------------- tile tables
// Every workgroup of a grouped-GEMM launch builds the launch's tile table in
// its own LDS from the segment offsets at kernel start: tiles_l[g] = tiles of
// the segments before g (an exclusive prefix), tiles_l[n] = the total.  The
// lengths never leave the device, no separate planning launch runs, and the
// cost is one read of the offsets (L2-resident after the first workgroup)
// and a block scan.
// Tiles of segment g (over both problems) for a cover of tiles bm rows x
// ncols output columns over the segments of length in [min_len, max_len).
template <typename Args>
__device__ __forceinline__ int seg_tiles(const Args& a, int g, int bm, int ncols, int min_len,
                                         int max_len) {
  const int p = g < a.p[0].n_seg ? 0 : 1;
  const auto& P = a.p[p];
  const int s = g - (p ? a.p[0].n_seg : 0);
  const int len = P.seg_offsets ? P.seg_offsets[s + 1] - P.seg_offsets[s] : P.rows;
  if (len < min_len || len >= max_len) return 0;
  if (P.seg_offsets && (unsigned)P.seg_expert[s] >= (unsigned)P.n_w) return 0;
  return ((len + bm - 1) / bm) * ((P.N + ncols - 1) / ncols);
}

// `wsum`: NTHR / 64 + 1 ints of LDS scratch.  Ends with a barrier.
template <int NTHR, typename Args>
__device__ void build_tile_table(const Args& a, int* tiles_l, int* wsum, int bm, int ncols,
                                 int min_len, int max_len) {
  constexpr int NW = NTHR / 64;
  const int n = a.n_seg_total, tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int per = (n + NTHR - 1) / NTHR;
  const int lo = min(n, tid * per), hi = min(n, lo + per);
  int sum = 0;
  for (int g = lo; g < hi; ++g) sum += seg_tiles(a, g, bm, ncols, min_len, max_len);
  const int incl = wave_dev::incl_scan(sum);
  if (lane == 63) wsum[wv] = incl;
  __syncthreads();
  if (tid == 0) {
    int run = 0;
    for (int w = 0; w < NW; ++w) {
      const int t = wsum[w];
      wsum[w] = run;
      run += t;
    }
    wsum[NW] = run;
  }
  __syncthreads();
  int run = wsum[wv] + incl - sum;
  for (int g = lo; g < hi; ++g) {
    tiles_l[g] = run;
    run += seg_tiles(a, g, bm, ncols, min_len, max_len);
  }
  if (tid == 0) tiles_l[n] = wsum[NW];
  __syncthreads();
}

#define MOE_LDS_PTR(p) ((__attribute__((address_space(3))) void*)(p))

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void raw_barrier() { asm volatile("s_barrier" ::: "memory"); }

// Wait until at most `later` stages of this wave's copies (LPW each) are in
// flight; vmcnt takes an immediate, so dispatch on the count.
template <int LPW, int J>
__device__ __forceinline__ void wait_stages(int later) {
  if constexpr (J <= 0) {
    wait_vmcnt<0>();
  } else {
    if (later >= J) wait_vmcnt<J * LPW>();
    else wait_stages<LPW, J - 1>(later);
  }
}

// XOR swizzle of the 16-byte chunk index inside a row piece of KCH chunks,
// chosen so that the 16 lanes reading one MFMA operand column (16 rows, same
// logical chunk) hit distinct 16-byte bank groups of a 256-byte bank row
// (128-byte pieces: measured 3-9% faster than swizzling by row & 7; 256-byte
// pieces, the bf16 activations of 128-deep stages, every row a whole bank row:
// row & 15, 2-4% faster than row & 7).
template <int KCH>
__device__ __forceinline__ int swz(int row) {
  if constexpr (KCH == 16) return row & 15;
  else if constexpr (KCH == 8) return (row >> 1) & 7;
  else return (row >> 2) & 3;
}

// Raw buffer resource over `bytes` bytes at `base` (word 3: the gfx9 raw
// buffer format; loads past `bytes` return zero instead of touching memory).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes,
                                           0x00020000);
}

constexpr int kAuxNT = 2;   // the gfx950 "nt" bit of a buffer access's aux operand

// Persistent grid: as many workgroups as can be resident at once (a larger
// grid would run its excess only after others finish), a multiple of 8 so
// that the XCD remap is a bijection.  The occupancy query's own error (it
// refuses some large-LDS kernels that launch fine) is cleared so that it is
// not reported as a launch failure; `fallback` workgroups per CU are used
// then.  Results are cached per kernel and LDS size.
// (The cache is shared by every host thread that calls the library: guarded.)
template <typename Kern>
int persistent_grid(Kern kernel, size_t dyn_lds, int fallback, int threads = 256) {
  struct Entry { const void* k; size_t lds; int dev; int per_cu; };
  static Entry cache[64];
  static int n_cache = 0;
  static std::mutex mu;
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) dev = 0;
  const void* key = reinterpret_cast<const void*>(kernel);
  int per_cu = 0;
  {
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < n_cache; ++i)
      if (cache[i].k == key && cache[i].lds == dyn_lds && cache[i].dev == dev) per_cu = cache[i].per_cu;
  }
  if (per_cu == 0) {
    if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&per_cu, kernel, threads, dyn_lds) != hipSuccess ||
        per_cu < 1) {
      (void)hipGetLastError();
      per_cu = fallback;
    }
    std::lock_guard<std::mutex> lock(mu);
    if (n_cache < 64) cache[n_cache++] = Entry{key, dyn_lds, dev, per_cu};
  }
  const int g = device_cu_count() * per_cu / 8 * 8;
  return g > 8 ? g : 8;
}

constexpr int kAll = 0x7fffffff;

}  // namespace
}  // namespace moe
