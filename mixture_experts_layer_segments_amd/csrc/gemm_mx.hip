// Grouped SwiGLU experts on MXFP4 weights (format in mx_dev.h), activations
// bf16 or MXFP4:
//
//   GEMM 1: [g | u] = X_s . [W_gate[e] | W_up[e]],  h = silu(g) * u
//   GEMM 2: y = row_scale * (h . W_down[e])
//
// Persistent kernels on the tile tables of gemm_dev.h; a weight is its E2M1
// code times its 1 x 32 block's power of two, exact in bf16, and all sums are
// fp32.
#include "gemm_dev.h"
#include "mx_dev.h"

namespace moe {
namespace {

using namespace mx_dev;

struct MxProblem {
  const void* A;            // [A rows, K] bf16, or E2M1 codes [A rows, K / 2]
  const uint8_t* a_e8;      // E2M1 activations: [A rows, K / 32] scales
  const uint8_t* B;         // [n_w][NB, K / 2] codes
  const uint8_t* b_e8;      // [n_w][NB, K / 32] scales
  uint16_t* C;              // [rows, N] bf16
  uint8_t* Cq;              // E2M1 activations, GEMM 1: h as codes [rows, N / 2]
  uint8_t* c_e8;            //   and scales [rows, N / 32] (C unused)
  const float* scale;       // nullable, by row
  const int32_t* seg_offsets;  // nullable: one segment [0, rows)
  const int32_t* seg_expert;
  const int32_t* a_rows;       // nullable: row r of the problem is row a_rows[r] of A
  int32_t n_seg, rows, N, K;
  int32_t n_w;
  int32_t a_ld_rows;        // rows of A
  int32_t up_off;           // GEMM 1: row offset of W_up inside B
  int64_t b_rows;           // weight rows per expert
};

struct MxArgs {
  MxProblem p[2];
  int32_t n_probs;
  int32_t n_seg_total;
  int32_t tile_bm, tile_ncols, min_len, max_len;   // as GemmArgs
};

// ---------------------------------------------------------------- streaming tiles
// Segments of a few rows: the time is that of reading every active expert's
// codes once (17/32 byte a weight), so the codes go straight from memory to
// the matrix operands, with no LDS and no barrier between a wave's loads.
//
// Tile: 16 activation rows x 16 TN weight rows (GEMM 1: the first half gate
// rows, the second the matching up rows); the four waves of a workgroup split
// K and add their partial sums through LDS at the end.  Work along K goes in
// 128-element slabs.  Of a slab, lane (r, q) = (lane % 16, lane / 16) holds
// elements 32 q .. 32 q + 31 of row r: 16 bytes of codes, one whole scale
// block, loaded by one 16-byte access (the four lanes of a row cover 64
// contiguous bytes, two slabs a 128-byte line).  That is the operand layout of
// the 16x16x128 FP4 matrix instruction; for bf16 activations four 16x16x32
// instructions take the 32 elements in four steps of 8, the activation
// fragment of the same elements beside it (a sum over K is a sum in any
// order).
// A unit: SL slabs of one wave.  Wave w takes units w, w + 4, ... of K, so the
// four waves read 4 SL * 64 contiguous bytes of every row together.
template <bool AF4, int TN, int SL>
struct MxUnit {
  u32x4 w[TN][SL];                     // weight codes
  uint32_t ws[TN][SL];                 // their 4 scale bytes a slab, byte q this lane's
  u32x4 a[SL][AF4 ? 1 : 4];            // activations
  uint32_t as[AF4 ? SL : 1];
};

template <bool AF4, int TN, int SL>
__device__ __forceinline__ void mx_load_a(MxUnit<AF4, TN, SL>& u, const MxProblem& P, bool ok,
                                          uint32_t arow, int slab0, int nslab, int q) {
#pragma unroll
  for (int i = 0; i < SL; ++i) {
    const int sl = slab0 + i;
    const bool in = ok && sl < nslab;
    if constexpr (AF4) {
      const uint8_t* a = (const uint8_t*)P.A + (size_t)arow * (P.K / 2);
      u.a[i][0] = in ? *reinterpret_cast<const u32x4*>(a + sl * 64 + q * 16) : u32x4{0, 0, 0, 0};
      u.as[i] = in ? *reinterpret_cast<const uint32_t*>(P.a_e8 + (size_t)arow * (P.K / 32) + sl * 4)
                   : 0u;
    } else {
      const uint16_t* a = (const uint16_t*)P.A + (size_t)arow * P.K + sl * 128 + q * 32;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        u.a[i][j] = in ? reinterpret_cast<const u32x4*>(a)[j] : u32x4{0, 0, 0, 0};
    }
  }
}

template <bool AF4, int TN, int SL>
__device__ __forceinline__ void mx_load_w(MxUnit<AF4, TN, SL>& u, const uint8_t* Bb,
                                          const uint8_t* Sb, const uint32_t (&brow)[TN], int K,
                                          int slab0, int nslab, int q) {
#pragma unroll
  for (int i = 0; i < SL; ++i) {
    const int sl = slab0 + i;
    if (sl < nslab) {
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        u.w[j][i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(
            Bb + (size_t)(brow[j] * (uint32_t)(K / 2)) + sl * 64 + q * 16));
        u.ws[j][i] = *reinterpret_cast<const uint32_t*>(
            Sb + (size_t)(brow[j] * (uint32_t)(K / 32)) + sl * 4);
      }
    } else {
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        u.w[j][i] = u32x4{0, 0, 0, 0};
        u.ws[j][i] = 0;
      }
    }
  }
}

template <bool AF4, int TN, int SL>
__device__ __forceinline__ void mx_unit_mma(const MxUnit<AF4, TN, SL>& u, f32x4 (&acc)[TN],
                                            int q) {
#pragma unroll
  for (int i = 0; i < SL; ++i) {
    if constexpr (AF4) {
      const u32x4 av = u.a[i][0];
      const i32x8 a = {(int)av[0], (int)av[1], (int)av[2], (int)av[3], 0, 0, 0, 0};
      const int sa = (int)(u.as[i] >> (8 * q));
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const u32x4 wv = u.w[j][i];
        const i32x8 b = {(int)wv[0], (int)wv[1], (int)wv[2], (int)wv[3], 0, 0, 0, 0};
        acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            a, b, acc[j], 4, 4, 0, sa, 0, (int)(u.ws[j][i] >> (8 * q)));
      }
    } else {
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const float sc = e8m0_float((u.ws[j][i] >> (8 * q)) & 0xffu);
#pragma unroll
        for (int m = 0; m < 4; ++m)
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8, u.a[i][m]),
              __builtin_bit_cast(bf16x8, e2m1x8_to_bf16(u.w[j][i][m], sc)), acc[j], 0, 0, 0);
      }
    }
  }
}

template <int MODE, bool AF4, int TN, int SL>
__global__ __launch_bounds__(256) void mx_stream_kernel(MxArgs args) {
  constexpr int NCOLS = 16 * TN / (MODE == 0 ? 2 : 1);   // output columns of a tile
  static_assert(128 % NCOLS == 0, "whole tiles along N (a multiple of 128)");
  static_assert(!(MODE == 0 && AF4) || NCOLS == 32, "a tile holds h's whole 1 x 32 blocks");
  __shared__ f32x4 red[4][TN][64];
  __shared__ int wsum[256 / 64 + 1];
  extern __shared__ int tiles_l[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nst = args.n_seg_total;
  build_tile_table<256>(args, tiles_l, wsum, args.tile_bm, args.tile_ncols, args.min_len,
                        args.max_len);
  const int total = tiles_l[nst];
  const int G = gridDim.x;
  const int r = lane & 15, q = lane >> 4;

  for (int tile = xcd_logical(blockIdx.x, G); tile < total; tile += G) {
    int lo = 0, hi = nst - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tiles_l[mid] <= tile) lo = mid; else hi = mid - 1;
    }
    const int pi = lo < args.p[0].n_seg ? 0 : 1;
    const MxProblem& P = args.p[pi];
    int r0 = 0, len = P.rows, e = 0;
    if (P.seg_offsets) {
      const int s = lo - (pi ? args.p[0].n_seg : 0);
      r0 = P.seg_offsets[s];
      len = P.seg_offsets[s + 1] - r0;
      e = P.seg_expert[s];
    }
    const int mt = (len + 15) / 16;
    const int local = tile - tiles_l[lo];
    const int m0 = (local % mt) * 16, n0 = (local / mt) * NCOLS;
    const int K = P.K, N = P.N, nslab = K / 128;
    const uint8_t* Bb = P.B + (size_t)e * P.b_rows * (K / 2);
    const uint8_t* Sb = P.b_e8 + (size_t)e * P.b_rows * (K / 32);
    uint32_t brow[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j)
      brow[j] = (MODE == 0 && j >= TN / 2 ? P.up_off + n0 + (j - TN / 2) * 16 : n0 + j * 16) + r;
    const bool a_ok = m0 + r < len;
    const int ar = r0 + min(m0 + r, len - 1);
    const uint32_t arow = P.a_rows ? P.a_rows[ar] : ar;

    f32x4 acc[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    MxUnit<AF4, TN, SL> cur, nxt;
    int sl = wv * SL;
    mx_load_a(cur, P, a_ok, arow, sl, nslab, q);
    mx_load_w(cur, Bb, Sb, brow, K, sl, nslab, q);
    while (sl < nslab) {
      sl += 4 * SL;
      mx_load_a(nxt, P, a_ok, arow, sl, nslab, q);
      mx_load_w(nxt, Bb, Sb, brow, K, sl, nslab, q);
      mx_unit_mma(cur, acc, q);
      cur = nxt;
    }

    // the waves' partial sums, then the epilogue on wave 0: lane (r, q) holds
    // rows 4 q .. 4 q + 3 and column r of each 16 x 16 piece
    __syncthreads();
#pragma unroll
    for (int j = 0; j < TN; ++j) red[wv][j][lane] = acc[j];
    __syncthreads();
    if (wv != 0) continue;
    f32x4 v[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j)
      v[j] = acc[j] + red[1][j][lane] + red[2][j][lane] + red[3][j][lane];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = m0 + q * 4 + i;
      if constexpr (MODE == 0 && AF4) {
        // h in bf16, then its 1 x 32 block (two columns a lane) as codes
        const float h0 = __uint_as_float((uint32_t)to_bf16(silu(v[0][i]) * v[2][i]) << 16);
        const float h1 = __uint_as_float((uint32_t)to_bf16(silu(v[1][i]) * v[3][i]) << 16);
        uint32_t a = max(__float_as_uint(h0) & 0x7fffffffu, __float_as_uint(h1) & 0x7fffffffu);
        a = max(a, (uint32_t)wave_dev::dpp<0xB1>((int)a));
        a = max(a, (uint32_t)wave_dev::dpp<0x4E>((int)a));
        a = max(a, (uint32_t)wave_dev::dpp<0x141>((int)a));
        a = max(a, (uint32_t)wave_dev::dpp<0x140>((int)a));
        const uint32_t b = block_e8m0(a);
        // column pairs (r, r + 1) of both halves meet in the even lane
        const float p0 = __builtin_bit_cast(float, wave_dev::dpp<0xB1>(__builtin_bit_cast(int, h0)));
        const float p1 = __builtin_bit_cast(float, wave_dev::dpp<0xB1>(__builtin_bit_cast(int, h1)));
        const float f[8] = {h0, p0, h1, p1, 0.f, 0.f, 0.f, 0.f};
        const uint32_t c = e2m1x8(f, b);
        if (row < len) {
          const size_t at = (size_t)(r0 + row) * N + n0;
          if ((r & 1) == 0) {
            P.Cq[(at + r) / 2] = (uint8_t)c;
            P.Cq[(at + 16 + r) / 2] = (uint8_t)(c >> 8);
          }
          if (r == 0) P.c_e8[at / 32] = (uint8_t)b;
        }
      } else if constexpr (MODE == 0) {
        if (row < len) {
#pragma unroll
          for (int j = 0; j < TN / 2; ++j)
            P.C[(size_t)(r0 + row) * N + n0 + j * 16 + r] =
                to_bf16(silu(v[j][i]) * v[j + TN / 2][i]);
        }
      } else {
        if (row < len) {
          const float sc = P.scale ? P.scale[r0 + row] : 1.0f;
#pragma unroll
          for (int j = 0; j < TN; ++j)
            P.C[(size_t)(r0 + row) * N + n0 + j * 16 + r] = to_bf16(v[j][i] * sc);
        }
      }
    }
  }
}

MxArgs cover(MxArgs g, int bm, int ncols, int min_len, int max_len) {
  g.tile_bm = bm;
  g.tile_ncols = ncols;
  g.min_len = min_len;
  g.max_len = max_len;
  return g;
}

template <int MODE, bool AF4, int TN, int SL>
void launch_stream(const MxArgs& g, int min_len, int max_len, hipStream_t s) {
  auto k = mx_stream_kernel<MODE, AF4, TN, SL>;
  const size_t dyn = (size_t)(g.n_seg_total + 1) * sizeof(int);
  k<<<persistent_grid(k, dyn, 2), 256, dyn, s>>>(
      cover(g, 16, 16 * TN / (MODE == 0 ? 2 : 1), min_len, max_len));
}

template <bool AF4>
void launch_pair(const MxArgs& g1, const MxArgs& g2, hipStream_t s) {
  if constexpr (AF4) {
    launch_stream<0, true, 4, 2>(g1, 1, kAll, s);
    launch_stream<1, true, 2, 2>(g2, 1, kAll, s);
  } else {
    launch_stream<0, false, 2, 2>(g1, 1, kAll, s);
    launch_stream<1, false, 2, 2>(g2, 1, kAll, s);
  }
}

}  // namespace

void launch_grouped_ffn_mx(const moe_config& c, const FfnProblem* probs, int n_probs,
                           hipStream_t s) {
  MxArgs g1{}, g2{};
  int nst = 0;
  for (int p = 0; p < n_probs; ++p) {
    const FfnProblem& P = probs[p];
    MxProblem& a = g1.p[p];
    a.A = P.A;
    a.a_e8 = P.a_e8;
    a.B = (const uint8_t*)P.w13;
    a.b_e8 = P.w13_e8;
    a.C = (uint16_t*)P.h;
    a.Cq = P.h_q;
    a.c_e8 = P.h_e8;
    a.seg_offsets = P.seg_offsets;
    a.seg_expert = P.seg_expert;
    a.a_rows = P.a_rows;
    a.n_seg = P.n_seg;
    a.rows = P.rows;
    a.n_w = P.n_w;
    a.a_ld_rows = P.a_rows ? c.T : P.rows;   // gathered rows come from x
    a.N = P.Iw;
    a.K = c.H;
    a.up_off = P.Iw;
    a.b_rows = 2 * (int64_t)P.Iw;
    MxProblem& b = g2.p[p];
    b = a;
    b.A = P.mx_acts ? (const void*)P.h_q : P.h;
    b.a_e8 = P.h_e8;
    b.Cq = nullptr;
    b.c_e8 = nullptr;
    b.a_rows = nullptr;
    b.a_ld_rows = P.rows;
    b.B = (const uint8_t*)P.w2;
    b.b_e8 = P.w2_e8;
    b.C = (uint16_t*)P.y;
    b.scale = P.row_scale;
    b.N = c.H;
    b.K = P.Iw;
    b.up_off = 0;
    b.b_rows = c.H;
    nst += P.n_seg;
  }
  g1.n_probs = g2.n_probs = n_probs;
  g1.n_seg_total = g2.n_seg_total = nst;
  if (probs[0].mx_acts) launch_pair<true>(g1, g2, s);
  else launch_pair<false>(g1, g2, s);
  MOE_DBG("grouped gemms (MXFP4)");
}

}  // namespace moe
