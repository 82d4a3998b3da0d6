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

// A value that is the same in every lane, said so: what the compiler takes
// for a lane's own it keeps in vector registers, and a buffer described by
// such values is read lane by lane in a loop.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

struct MxArgs {
  MxProblem p[2];
  int32_t n_probs;
  int32_t n_seg_total;
  int32_t tile_bm, tile_ncols, min_len, max_len;   // as GemmArgs
  int32_t* queue;   // ring tiles: [kMxClasses][8], the next tile of each XCD
};

// silu(z) = z / (1 + e^-z) with the hardware's base-2 exponential and
// reciprocal: e^-z = 2^h (1 + l ln 2), h the rounded product z * -log2 e and l
// what its rounding and the constant's left out, so that large |z| lose
// nothing (about 2^-22 in all; h is rounded to bf16 next).  The exponent's z is
// held to +-200, where e^-z is 0 or infinity already, so that no infinity
// meets another.  The reciprocal has no subnormals: below z = -87 the result
// is 0 where the formula's is within 1e-36.
__device__ __forceinline__ float silu_fast(float z) {
  constexpr float c = -1.44269504f, cl = -1.92596299e-8f;
  const float x = __builtin_amdgcn_fmed3f(z, -200.0f, 200.0f);
  const float h = x * c;
  const float l = fmaf(x, cl, fmaf(x, c, -h));
  const float e = __builtin_amdgcn_exp2f(h) * fmaf(l, 0.693147182f, 1.0f);
  return z * __builtin_amdgcn_rcpf(1.0f + e);
}

// Two bf16 in one conversion.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

// ---------------------------------------------------------------- streaming tiles
// Segments of a few rows: the time is that of reading every active expert's
// codes once (17/32 byte a weight).
//
// Tile: 16 activation rows x 16 TN weight rows (GEMM 1: the first half gate
// rows, the second the matching up rows), on KS waves that split K and add
// their partial sums through LDS (a workgroup is 4 / KS tiles).  A stage is
// 256 elements of K, 128 bytes of codes a row: a load instruction reads whole
// 128-byte lines of 8 rows (reading 64-byte pieces of 16 rows, the matrix
// operand's own layout, held the kernel to 3.3 TB/s), each wave turns the
// stage through LDS of its own (no barrier in the K loop) and keeps the next
// four stages' codes and activations in flight in registers.
//
// Of a stage's two 128-element slabs, lane (r, q) = (lane % 16, lane / 16)
// takes elements 32 q .. 32 q + 31 of row r: 16 bytes of codes, one whole
// scale block.  That is the operand layout of the 16x16x128 FP4 matrix
// instruction; for bf16 activations four 16x16x32 instructions take the 32
// elements in four steps of 8, the activation fragment of the same elements
// beside it (a sum over K is a sum in any order).  The E8M0 bytes come four
// stages (32 bytes a row) at a time and go through LDS too.
constexpr int kMxDepth = 4;   // stages in flight

// Byte offsets of a lane's operands at the wave's first stage.  (The whole
// offset goes in the vector offset: the scalar one is no part of the buffer's
// range check, and the last stage of a K that ends inside it reads past the
// last row.)
struct MxSrc {
  __amdgpu_buffer_rsrc_t rb, rs, ra, ras;
  uint32_t w, ws, a, as;
  uint32_t w8;              // 8 weight rows further, in bytes
  uint32_t up;              // GEMM 1: from a gate row to its up row, in bytes
  uint32_t ws_up;           // the same, in scale bytes
};

// Orders a wave's LDS accesses between its own lanes (they execute in order;
// this keeps the compiler from moving a read over another lane's write).
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
}

template <bool AF4>
struct MxActs {
  u32x4 v[2][AF4 ? 1 : 4];
  u32x2 s;                  // FP4: the row's 8 scale bytes of the stage
};

template <bool AF4>
__device__ __forceinline__ void mx_load_a(MxActs<AF4>& a, const MxSrc& s, int stage) {
  if constexpr (AF4) {
    a.v[0][0] = __builtin_amdgcn_raw_buffer_load_b128(s.ra, s.a + stage * 128, 0, 0);
    a.v[1][0] = __builtin_amdgcn_raw_buffer_load_b128(s.ra, s.a + stage * 128 + 64, 0, 0);
    a.s = __builtin_amdgcn_raw_buffer_load_b64(s.ras, s.as + stage * 8, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        a.v[i][j] = __builtin_amdgcn_raw_buffer_load_b128(s.ra, s.a + stage * 512 + i * 256 + j * 16,
                                                          0, 0);
  }
}

template <int MODE, int TN>
__device__ __forceinline__ void mx_load_w(u32x4 (&w)[2 * TN], const MxSrc& s, int stage) {
#pragma unroll
  for (int i = 0; i < 2 * TN; ++i) {
    const bool up = MODE == 0 && i >= TN;
    w[i] = __builtin_amdgcn_raw_buffer_load_b128(
        s.rb, s.w + (stage * 128 + (up ? s.up + (i - TN) * s.w8 : i * s.w8)), 0, kAuxNT);
  }
}

// One stage's products: the codes in `wl` (16 TN rows of 8 chunks, chunk c at
// c ^ swz<8>(row)), this stage's scale dwords at `sl` (8 dwords a row),
// `slabs` of its two slabs inside K.
template <bool AF4, int TN>
__device__ __forceinline__ void mx_stage_mma(const u32x4* wl, const uint32_t* sl,
                                             const MxActs<AF4>& a, int slabs, int r, int q,
                                             f32x4 (&acc)[TN]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (i >= slabs) break;
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const u32x4 w = wl[(j * 16 + r) * 8 + ((4 * i + q) ^ swz<8>(r))];
      const uint32_t sb = sl[(j * 16 + r) * 8 + i] >> (8 * q);
      if constexpr (AF4) {
        const u32x4 v = a.v[i][0];
        acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0},
            i32x8{(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0}, acc[j], 4, 4, 0,
            (int)(a.s[i] >> (8 * q)), 0, (int)sb);
      } else {
        const float sc = e8m0_float(sb & 0xffu);
#pragma unroll
        for (int m = 0; m < 4; ++m)
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8, a.v[i][m]),
              __builtin_bit_cast(bf16x8, e2m1x8_to_bf16(w[m], sc)), acc[j], 0, 0, 0);
      }
    }
  }
}

template <int MODE, bool AF4, int TN, int KS, int WPE>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(WPE)))
void mx_stream_kernel(MxArgs args) {
  constexpr int NCOLS = 16 * TN / (MODE == 0 ? 2 : 1);   // output columns of a tile
  constexpr int NT = 4 / KS;                             // tiles of a workgroup
  static_assert(128 % NCOLS == 0, "whole tiles along N (a multiple of 128)");
  static_assert(!(MODE == 0 && AF4) || NCOLS == 32, "a tile holds h's whole 1 x 32 blocks");
  // a wave's turn buffer: two stages of codes, then four stages' scales
  constexpr int WB_CH = 2 * 16 * TN * 8, WS_CH = 16 * TN * 2;
  __shared__ u32x4 turn[4][WB_CH + WS_CH];
  __shared__ f32x4 red[KS > 1 ? 4 : 1][KS > 1 ? TN : 1][64];
  __shared__ int wsum[256 / 64 + 1];
  extern __shared__ int tiles_l[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = uniform(tid >> 6);
  const int nst = args.n_seg_total;
  build_tile_table<256>(args, tiles_l, wsum, args.tile_bm, args.tile_ncols, args.min_len,
                        args.max_len);
  const int total = tiles_l[nst];
  const int r = lane & 15, q = lane >> 4;
  const int ks = wv % KS;

  const int G = gridDim.x;
  for (int t0 = xcd_logical(blockIdx.x, G) * NT; t0 < total; t0 += G * NT) {
    const int tile = t0 + wv / KS;
    const bool live = tile < total;      // (all true but in the last workgroup)
    int r0 = 0, len = 0, m0 = 0, n0 = 0, pi = 0;
    f32x4 acc[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (live) {
      int lo = 0, hi = nst - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tiles_l[mid] <= tile) lo = mid; else hi = mid - 1;
      }
      lo = uniform(lo);
      pi = lo < args.p[0].n_seg ? 0 : 1;
      const MxProblem& P = args.p[pi];
      int e = 0;
      len = P.rows;
      if (P.seg_offsets) {
        const int s = lo - (pi ? args.p[0].n_seg : 0);
        r0 = uniform(P.seg_offsets[s]);
        len = uniform(P.seg_offsets[s + 1]) - r0;
        e = uniform(P.seg_expert[s]);
      }
      const int mt = (len + 15) / 16;
      const int local = tile - uniform(tiles_l[lo]);
      m0 = (local % mt) * 16;
      n0 = (local / mt) * NCOLS;
      const int K = P.K, nslab = K / 128;
      // this wave's stages: [st0, st0 + ns)
      const int nst_k = (nslab + 1) / 2, per = (nst_k + KS - 1) / KS;
      const int st0 = ks * per, ns = min(per, nst_k - st0);
      MxSrc src;
      const int64_t e_row = (int64_t)e * P.b_rows;
      const uint32_t brow_b = K / 2, srow_b = K / 32, arow_b = AF4 ? K / 2 : K * 2;
      src.rb = buffer_rsrc(P.B + e_row * brow_b, (uint32_t)(P.b_rows * brow_b));
      src.rs = buffer_rsrc(P.b_e8 + e_row * srow_b, (uint32_t)(P.b_rows * srow_b));
      src.w = (uint32_t)(n0 + lane / 8) * brow_b + (lane % 8) * 16 + st0 * 128;
      src.w8 = 8 * brow_b;
      src.up = P.up_off * brow_b;
      // two lanes a row, 16 bytes each
      const int srow = lane / 2;
      src.ws = (uint32_t)(n0 + (MODE == 0 && srow >= 8 * TN ? P.up_off + srow - 8 * TN : srow)) *
                   srow_b + (lane % 2) * 16 + st0 * 8;
      src.ws_up = (MODE == 0 ? P.up_off : 32) * srow_b;
      // a row past the segment takes an offset beyond the buffer (zeros, and no
      // traffic; where a buffer ends within a row of 2^32 bytes it reads a
      // row of it instead: such a row's products are dropped either way)
      const bool a_ok = m0 + r < len;
      const int ar = r0 + min(m0 + r, len - 1);
      const uint32_t arow = P.a_rows ? P.a_rows[ar] : ar;
      src.ra = buffer_rsrc(P.A, (uint32_t)((size_t)P.a_ld_rows * arow_b));
      src.a = a_ok ? arow * arow_b + st0 * (AF4 ? 128 : 512) + q * (AF4 ? 16 : 64)
                   : 0xFFFFFF00u - arow_b;
      src.as = 0;
      if constexpr (AF4) {
        src.ras = buffer_rsrc(P.a_e8, (uint32_t)((size_t)P.a_ld_rows * srow_b));
        src.as = a_ok ? arow * srow_b + st0 * 8 : 0xFFFFFF00u - srow_b;
      }
      if (ns > 0) {
        constexpr int D = kMxDepth;
        u32x4 w[D][2 * TN], sc[TN / 2];
        MxActs<AF4> a[D];
        // (stages past the wave's last repeat it: every load is issued, so that
        // the compiler knows what is in flight at every wait)
        auto load = [&](int d, int st) {
          const int s = min(st, ns - 1);
          mx_load_w<MODE, TN>(w[d], src, s);
          mx_load_a(a[d], src, s);
        };
        auto load_sc = [&](int st) {
#pragma unroll
          for (int i = 0; i < TN / 2; ++i)
            sc[i] =
                __builtin_amdgcn_raw_buffer_load_b128(src.rs, src.ws + (st * 8 + i * src.ws_up), 0, 0);
        };
        u32x4* wl = turn[wv];
        u32x4* sl = wl + WB_CH;
        const int wr = lane / 8, wc = lane % 8;
        auto body = [&](int st, bool more) __attribute__((always_inline)) {
#pragma unroll
          for (int i = 0; i < TN / 2; ++i) sl[i * 64 + lane] = sc[i];
          if (more) load_sc(st + D);
#pragma unroll
          for (int d = 0; d < D; ++d) {
            u32x4* buf = wl + (d & 1) * (16 * TN * 8);
#pragma unroll
            for (int i = 0; i < 2 * TN; ++i) {
              const int row = i * 8 + wr;
              buf[row * 8 + (wc ^ swz<8>(row))] = w[d][i];
            }
            wave_lds_fence();
            if (more) mx_load_w<MODE, TN>(w[d], src, min(st + D + d, ns - 1));
            const int left = nslab - (st0 + st + d) * 2;
            if (st + d < ns)
              mx_stage_mma<AF4, TN>(buf, reinterpret_cast<const uint32_t*>(sl) + d * 2, a[d],
                                    left < 2 ? 1 : 2, r, q, acc);
            if (more) mx_load_a(a[d], src, min(st + D + d, ns - 1));
            wave_lds_fence();
          }
        };
        load_sc(0);
#pragma unroll
        for (int d = 0; d < D; ++d) load(d, d);
        int st = 0;
        for (; st + D < ns; st += D) body(st, true);
        body(st, false);
      }
    }

    // the waves' partial sums, then the epilogue on a tile's first wave: lane
    // (r, q) holds rows 4 q .. 4 q + 3 and column r of each 16 x 16 piece
    f32x4 v[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) v[j] = acc[j];
    if constexpr (KS > 1) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < TN; ++j) red[wv][j][lane] = acc[j];
      __syncthreads();
      if (ks != 0) continue;
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int w = 1; w < KS; ++w) v[j] += red[wv + w][j][lane];
    }
    if (!live) continue;
    const MxProblem& P = args.p[pi];
    const int N = P.N;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = m0 + q * 4 + i;
      if constexpr (MODE == 0 && AF4) {
        // h in bf16, then its 1 x 32 block (two columns a lane) as codes
        const float h0 = __uint_as_float((uint32_t)to_bf16(silu_fast(v[0][i]) * v[2][i]) << 16);
        const float h1 = __uint_as_float((uint32_t)to_bf16(silu_fast(v[1][i]) * v[3][i]) << 16);
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
                to_bf16(silu_fast(v[j][i]) * v[j + TN / 2][i]);
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

// ---------------------------------------------------------------- ring tiles
// Segments of more rows: BM activation rows x 256 weight rows (GEMM 1: 128
// gate rows and the matching 128 up rows) on 8 waves, the operands copied
// straight into an LDS ring of STAGES K stages (waits, copies and their
// completion as in gemm.hip's ring: waves 0-3 issue, explicit vmcnt waits, a
// plain barrier a stage).
//
// A stage holds, per row, 128 bytes of codes (256 elements), in 64-row and in
// FP4 tiles; longer bf16 tiles, where the activations take most of the LDS,
// 256 bytes of bf16 and 64 bytes of codes (128 elements); in 16-byte chunks
// XOR-swizzled by row.  A 64-byte piece costs a request as a whole line does:
// FP4 stages half as deep and twice as many were 15-20% slower, 64-row bf16
// tiles 12% (458 against 409 us for 128 segments of 64 rows, H 4096, I 1536).
// The rows' E8M0 bytes come 16 at a time, those of 512 elements, into two
// slots of their own behind the ring: a 4- or 8-byte piece per stage cost as
// many requests as the codes (10-20% of a launch).
//
// FP4 activations: two 16x16x128 FP4 matrix steps a stage.  Lane (r, q)
// supplies chunk 4 s + q of row r (32 elements, one scale block) and byte
// 4 s + q of the stage's scales.
// bf16 activations: lane (r, q) reads chunk 4 s + q of weight row r, 32 codes
// and one scale, and feeds them to four 16x16x32 steps, 8 at a time, against
// chunk 16 s + 4 q + m of the activation row in step m.  On 64-row tiles the
// eight waves take 32 weight rows each and all the activation rows, so that
// no code is converted twice (4-9% faster than two rows of waves).
//
// What bounds them, measured with a part left out, 32 segments of 2048 rows, H
// 4096, I 1536, FP4 activations (470 + 305 us, 3.3 PFLOP/s): copies and
// stores without the products 365 + 243 us, products and stores without the
// copies 380 + 214, all but the stores 411 + 218.  The copies move 64 KiB a
// stage in about 3500 cycles of a compute unit whatever the rows' stride and
// whether the L2 holds the lines already, the products take 2050.  With bf16
// activations long segments run at 1.2 PFLOP/s, near a large bf16 library
// product's 1.29.
//
// Tiles are chained: when a tile's K loop is done, the copies of the next
// tile's first stages are issued before the output is formed, which is staged
// in the one ring slot they leave free.
// XOR swizzle of the 16-byte chunks of a staged row of KCH chunks (a power of
// two of at most a 256-byte bank row, or two bank rows).  The 64 lanes of a
// 16-byte LDS read are served sixteen at a time, lanes 0-3, 12-15 and 20-27,
// then the other sixteen of 32: of an operand read (row = lane % 16, chunk by
// lane / 16), two sets of rows for two neighbouring chunks.  Each sixteen hit
// distinct 16-byte groups of a bank row.  (Swizzles that spread the sixteen
// rows of one chunk, row & 15 and row / 4 % 4, left a conflict on every read
// of 256- and 64-byte rows: half of the LDS's cycles, 2% of the time.)
template <int KCH>
__device__ __forceinline__ int mx_swz(int row) {
  if constexpr (KCH >= 16) return (row & 11) | ((row >> 1) & 4);
  else if constexpr (KCH == 8) return (row >> 1) & 7;
  else return (row >> 2) & 2;
}

template <bool AF4, int BM, int STAGES_, int WM_>
struct MxRing {
  static constexpr int WAVES_M = WM_, BN = 256, NTHR = 512, NI = 4, STAGES = STAGES_;
  static constexpr int BK = AF4 || BM == 64 ? 256 : 128;  // elements of a stage
  static constexpr int KCA = AF4 ? BK / 32 : BK / 8, KCB = BK / 32;   // chunks per row
  static constexpr int RPA = 64 / KCA, RPB = 64 / KCB;    // rows per 1 KiB copy
  static constexpr int A_CH = BM * KCA, B_CH = BN * KCB, STAGE_CH = A_CH + B_CH;
  static constexpr int SG = 512 / BK;                     // stages of a scale group
  static constexpr int AS_CH = AF4 ? BM : 0;              // chunks of a scale slot: one a row
  static constexpr int SLOT_CH = AS_CH + BN;
  static constexpr int RING_CH = STAGES * STAGE_CH;       // the scale slots follow
  static constexpr int LDS_CH = RING_CH + 2 * SLOT_CH;
  static constexpr int A_IT = BM / RPA / NI, B_IT = BN / RPB / NI;
  static constexpr int LPI = A_IT + B_IT;                 // copies per issuing wave and stage
  static constexpr int S_IT = AF4 ? 2 : 1;                //   and per scale group
  static constexpr int WAVES_N = 8 / WAVES_M;
  static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N;
  static constexpr int TM = WM / 16, TN = WN / 16;
  // weights that no other row tile reads again stream past the caches, where
  // a row's piece is a whole 128-byte line
  static constexpr int B_AUX = (KCB == 8 && BM < 256) ? kAuxNT : 0;
  static_assert((BM / RPA) % NI == 0 && (BN / RPB) % NI == 0, "copy blocks per wave");
  static_assert(STAGES == 2 || STAGES == 3, "stage waits");
};

// Where a tile sits: values of the whole workgroup.
struct MxPlace {
  // (the problem by its number: a pointer into the kernel's arguments, carried
  // around the tile loop, had them copied to scratch memory)
  int pi, e, r0, len, m0, n0;
};

// Reads a value of the whole workgroup that no kernel of this launch writes:
// by the scalar unit, beside the vector memory operations in flight.
__device__ __forceinline__ int scalar_load(const int32_t* p) {
  return *(const __attribute__((address_space(4))) int32_t*)(uintptr_t)p;
}

template <int MODE, int BM>
__device__ __forceinline__ MxPlace mx_ring_place(const MxArgs& args, const int* tiles_l, int tile) {
  MxPlace t;
  int lo = 0, hi = args.n_seg_total - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (uniform(tiles_l[mid]) <= tile) lo = mid; else hi = mid - 1;
  }
  t.pi = lo < args.p[0].n_seg ? 0 : 1;
  const MxProblem& P = args.p[t.pi];
  t.r0 = 0;
  t.len = P.rows;
  t.e = 0;
  if (P.seg_offsets) {
    const int s = lo - (t.pi ? args.p[0].n_seg : 0);
    t.r0 = scalar_load(P.seg_offsets + s);
    t.len = scalar_load(P.seg_offsets + s + 1) - t.r0;
    t.e = scalar_load(P.seg_expert + s);
  }
  const int mt = (t.len + BM - 1) / BM;
  constexpr int ncols = MODE == 0 ? 128 : 256;
  const int nt = (P.N + ncols - 1) / ncols;
  const int local = tile - uniform(tiles_l[lo]);
  const int grp = local / (kGroupM * nt);
  const int first_m = grp * kGroupM;
  const int gm = min(kGroupM, mt - first_m);
  const int lg = local - grp * kGroupM * nt;
  t.m0 = (first_m + lg % gm) * BM;
  t.n0 = (lg / gm) * ncols;
  return t;
}

// The tiles of a class are divided among the XCDs as a static launch would do
// it, rounds of gridDim.x neighbouring tiles in eight parts and what is left
// over evenly, and a workgroup takes the next of its XCD's: the j-th, or -1.
__device__ __forceinline__ int mx_queue_tile(int j, int total) {
  const int G = gridDim.x, per = G / 8, x = blockIdx.x % 8;
  const int full = total / G, rem = total - full * G;
  if (j < full * per) return j / per * G + x * per + j % per;
  const int at = rem * x / 8 + (j - full * per);
  return at < rem * (x + 1) / 8 ? full * G + at : -1;
}

// A tile and this lane's copy sources (byte offsets at k = 0; the weight
// copies of a wave lie at uniform distances).
template <typename R>
struct MxTile : MxPlace {
  int K, up_off;
  bool stream;
  __amdgpu_buffer_rsrc_t ra, rb, rsa, rsb;
  uint32_t va[R::A_IT], vb, vsa, vsb;
  float rs[R::TM];          // GEMM 2: the scales of this lane's output rows
};

template <int MODE, bool AF4, typename R, int BM>
__device__ __forceinline__ void mx_ring_setup(const MxArgs& args, const MxPlace& at,
                                              MxTile<R>& t) {
  const int lane = threadIdx.x & 63;
  const int wvs = uniform(threadIdx.x >> 6);
  static_cast<MxPlace&>(t) = at;
  const MxProblem& P = args.p[t.pi];
  t.K = P.K;
  t.up_off = P.up_off;
  t.stream = t.len <= BM;
  const int K = P.K;
  const uint32_t arow_b = AF4 ? K / 2 : K * 2, brow_b = K / 2, srow_b = K / 32;
  const int64_t e_row = (int64_t)t.e * P.b_rows;
  // (weight rows past the expert's last -- the last column tile of a GEMM 2
  // whose N is an odd multiple of 128 -- lie past the buffers: zeros)
  t.ra = buffer_rsrc(P.A, (uint32_t)((size_t)P.a_ld_rows * arow_b));
  t.rb = buffer_rsrc(P.B + e_row * brow_b, (uint32_t)((size_t)P.b_rows * brow_b));
  if constexpr (AF4) t.rsa = buffer_rsrc(P.a_e8, (uint32_t)((size_t)P.a_ld_rows * srow_b));
  t.rsb = buffer_rsrc(P.b_e8 + e_row * srow_b, (uint32_t)((size_t)P.b_rows * srow_b));
  if constexpr (MODE == 1) {
#pragma unroll
    for (int mi = 0; mi < R::TM; ++mi) {
      const int row = t.m0 + (mi * R::WAVES_M + wvs / R::WAVES_N) * 16 + (lane & 15);
      t.rs[mi] = P.scale ? P.scale[t.r0 + min(row, t.len - 1)] : 1.0f;
    }
  }
  if (wvs >= R::NI) return;
  auto a_src = [&](int row) -> uint32_t {
    const int ar = t.r0 + min(t.m0 + row, t.len - 1);
    return P.a_rows ? P.a_rows[ar] : ar;
  };
#pragma unroll
  for (int i = 0; i < R::A_IT; ++i) {
    const int row = (i * R::NI + wvs) * R::RPA + lane / R::KCA;
    t.va[i] = a_src(row) * arow_b + ((lane % R::KCA) ^ mx_swz<R::KCA>(row)) * 16;
  }
  const int br = wvs * R::RPB + lane / R::KCB;
  t.vb = (uint32_t)(t.n0 + br) * brow_b + ((lane % R::KCB) ^ mx_swz<R::KCB>(br)) * 16;
  // scales: a lane a row, 64 rows a copy (a wave past the activation rows
  // repeats the last 64: every wave issues as many copies)
  t.vsa = 0;
  if constexpr (AF4) t.vsa = a_src(min(wvs, BM / 64 - 1) * 64 + lane) * srow_b;
  const int sr = wvs * 64 + lane;
  t.vsb = (uint32_t)(t.n0 + (MODE == 0 && sr >= R::BN / 2 ? P.up_off + sr - R::BN / 2 : sr)) * srow_b;
}

// This wave's copies of K stage kt, the scales of a new group of stages first.
// (A last stage or group that reaches past K reads on into the next row, or
// zeros past the buffer: those elements enter no product.  The whole offset
// goes in the vector offset, which the buffer's range check covers; the scalar
// one is no part of it.)
template <int MODE, bool AF4, typename R, int BM, int AUX>
__device__ __forceinline__ void mx_ring_issue(const MxTile<R>& t, u32x4* ring, int kt, int wv) {
  if (kt % R::SG == 0) {
    const int g = kt / R::SG;
    u32x4* slot = ring + R::RING_CH + (g & 1) * R::SLOT_CH;
    if constexpr (AF4)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(t.rsa, MOE_LDS_PTR(slot + min(wv, BM / 64 - 1) * 64),
                                               16, t.vsa + g * 16, 0, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(t.rsb, MOE_LDS_PTR(slot + R::AS_CH + wv * 64), 16,
                                             t.vsb + g * 16, 0, 0, 0);
  }
  u32x4* slot = ring + (kt % R::STAGES) * R::STAGE_CH;
#pragma unroll
  for (int i = 0; i < R::A_IT; ++i)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(t.ra, MOE_LDS_PTR(slot + (i * R::NI + wv) * 64), 16,
                                             t.va[i] + kt * (R::KCA * 16), 0, 0, 0);
  const uint32_t brow_b = t.K / 2;
#pragma unroll
  for (int i = 0; i < R::B_IT; ++i) {
    // weight rows i NI RPB further (GEMM 1: the second half are up rows)
    constexpr int RPI = R::NI * R::RPB, HALF = R::BN / 2 / RPI;
    const uint32_t rows = MODE == 0 && i >= HALF ? t.up_off + (i - HALF) * RPI : i * RPI;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        t.rb, MOE_LDS_PTR(slot + R::A_CH + (i * R::NI + wv) * 64), 16,
        t.vb + (rows * brow_b + kt * (R::KCB * 16)), 0, 0, AUX);
  }
}

template <int MODE, bool AF4, typename R, int BM>
__device__ __forceinline__ void mx_ring_stage(const MxTile<R>& t, u32x4* ring, int kt, int wv) {
  if (R::B_AUX && t.stream) mx_ring_issue<MODE, AF4, R, BM, R::B_AUX>(t, ring, kt, wv);
  else mx_ring_issue<MODE, AF4, R, BM, 0>(t, ring, kt, wv);
}

// The first stages of a tile (issuing waves).
template <int MODE, bool AF4, typename R, int BM>
__device__ __forceinline__ void mx_ring_prologue(const MxTile<R>& t, u32x4* ring, int wv) {
  const int KT = (t.K + R::BK - 1) / R::BK;
  mx_ring_stage<MODE, AF4, R, BM>(t, ring, 0, wv);
  if (R::STAGES > 2 && KT > 1) mx_ring_stage<MODE, AF4, R, BM>(t, ring, 1, wv);
}

// Waits until stage kt of KT has landed: at most the copies of the stage
// after it (three stages) may be outstanding and, where `stores` stores of the
// tile before were issued behind this tile's first stages, those too.
// (Vector memory operations of a wave complete in the order of their issue.)
template <typename R, int STORES>
__device__ __forceinline__ void mx_ring_wait(int kt, int KT, bool stores) {
  constexpr int LPI = R::LPI;
  if (stores && kt < R::STAGES - 1) {
    if constexpr (R::STAGES == 2) {
      wait_vmcnt<STORES>();
    } else if (kt == 0) {
      if (KT > 1) wait_vmcnt<STORES + LPI>(); else wait_vmcnt<STORES>();
    } else {
      if (KT > 2) wait_vmcnt<STORES + LPI + (2 % R::SG == 0 ? R::S_IT : 0)>();
      else wait_vmcnt<STORES>();
    }
  } else if constexpr (R::STAGES == 2) {
    wait_vmcnt<0>();
  } else {
    if (kt + 1 >= KT) wait_vmcnt<0>();
    else if ((kt + 1) % R::SG == 0) wait_vmcnt<LPI + R::S_IT>();
    else wait_vmcnt<LPI>();
  }
}

__device__ __forceinline__ i32x8 fp4_operand(u32x4 v) {
  return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
}

// One stage's matrix products over the wave's first NM row fragments (the
// rest lie past the segment) and, with FP4 activations, the stage's first NS
// matrix steps (1 where K ends in the middle of it).
//
// A wave's fragment mi covers rows (mi WAVES_M + wm) 16 .. +15 of the tile, so
// that the live fragments of a partial tile are spread evenly over the
// waves.  Fragment rows are r plus multiples of 16: the swizzle is r's, and a
// wave's fragments lie at constant distances.  Operand reads are placed
// among the products of the fragments before them: two weight fragments
// ahead, the next step's activation fragments over the last products of the
// step before.
template <int MODE, bool AF4, typename R, int NM, int NS>
__device__ __forceinline__ void mx_ring_mma(const u32x4* ring, int kt, int wm, int wn, int lane,
                                            f32x4 (&acc)[R::TM][R::TN]) {
  constexpr int TN = R::TN;
  const u32x4* slot = ring + (kt % R::STAGES) * R::STAGE_CH;
  const int r = lane & 15, q = lane >> 4;
  const int arow = wm * 16 + r;
  const int brow = wn * (MODE == 0 ? R::WN / 2 : R::WN) + r;
  constexpr int AF = R::WAVES_M * 16;   // tile rows between a wave's fragments
  // weight rows of fragment ni from brow
  auto b_at = [](int ni) constexpr {
    return MODE == 1 || ni < TN / 2 ? ni * 16 : R::BN / 2 + (ni - TN / 2) * 16;
  };
  const u32x4* As = slot + arow * R::KCA;
  const u32x4* Bs = slot + R::A_CH + brow * R::KCB;
  const u32x4* sc = ring + R::RING_CH + ((kt / R::SG) & 1) * R::SLOT_CH;
  if constexpr (AF4) {
    // the stage's 8 scale bytes of a row; q and 4 + q are this lane's
    const u32x2* sa2 = reinterpret_cast<const u32x2*>(sc + arow) + (kt & 1);
    const u32x2* sb2 = reinterpret_cast<const u32x2*>(sc + R::AS_CH + brow) + (kt & 1);
    const uint32_t sel = (uint32_t)q | (uint32_t)(4 + q) << 8;
    auto scales = [&](const u32x2* at) -> int {
      const u32x2 v = *at;
      return (int)__builtin_amdgcn_perm(v.y, v.x, sel);
    };
    int sa[NM], sb[TN];
    u32x4 a[2][NM], b[3];
    auto load_a = [&](int s, int mi) {
      a[s][mi] = As[mi * AF * R::KCA + ((s * 4 + q) ^ mx_swz<R::KCA>(r))];
    };
    auto load_b = [&](int x) {
      b[x % 3] = Bs[b_at(x % TN) * R::KCB + (((x / TN) * 4 + q) ^ mx_swz<R::KCB>(r))];
    };
#pragma unroll
    for (int mi = 0; mi < NM; ++mi) sa[mi] = scales(sa2 + mi * AF * 2);
#pragma unroll
    for (int ni = 0; ni < TN; ++ni) sb[ni] = scales(sb2 + b_at(ni) * 2);
#pragma unroll
    for (int mi = 0; mi < NM; ++mi) load_a(0, mi);
    load_b(0);
    load_b(1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int x = 0; x < NS * TN; ++x) {
      const int s = x / TN, ni = x % TN;
      if (x + 2 < NS * TN) load_b(x + 2);
      if (s == 0 && NS == 2) {
        // the NM activation fragments of the second step, over the last products
#pragma unroll
        for (int mi = 0; mi < NM; ++mi)
          if (TN - 1 - mi * TN / NM == ni) load_a(1, mi);
      }
      // weights as the first operand: lane l gets output row l % 16 and
      // columns 4 (l / 16) .. +3 of each 16 x 16 piece
#pragma unroll
      for (int mi = 0; mi < NM; ++mi)
        acc[mi][ni] = s == 0 ? __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                                   fp4_operand(b[x % 3]), fp4_operand(a[0][mi]), acc[mi][ni], 4, 4,
                                   0, sb[ni], 0, sa[mi])
                             : __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                                   fp4_operand(b[x % 3]), fp4_operand(a[1][mi]), acc[mi][ni], 4, 4,
                                   1, sb[ni], 1, sa[mi]);
      __builtin_amdgcn_sched_barrier(0);
    }
  } else {
    const uint32_t* sb1 =
        reinterpret_cast<const uint32_t*>(sc + brow) + kt % R::SG * (R::BK / 128);
    // 128 elements of K at a time
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      u32x4 bc[TN], a[2][NM];
      uint32_t bs[TN];
      auto load_a = [&](int m, int mi) {
        a[m & 1][mi] = As[mi * AF * R::KCA + ((16 * s + 4 * q + m) ^ mx_swz<R::KCA>(r))];
      };
#pragma unroll
      for (int ni = 0; ni < TN; ++ni) {
        bc[ni] = Bs[b_at(ni) * R::KCB + ((4 * s + q) ^ mx_swz<R::KCB>(r))];
        bs[ni] = sb1[b_at(ni) * 4 + s];
      }
#pragma unroll
      for (int mi = 0; mi < NM; ++mi) load_a(0, mi);
      float bf[TN];
#pragma unroll
      for (int ni = 0; ni < TN; ++ni) bf[ni] = e8m0_float((bs[ni] >> (8 * q)) & 0xffu);
      u32x4 b = e2m1x8_to_bf16(bc[0][0], bf[0]);
#pragma unroll
      for (int x = 0; x < 4 * TN; ++x) {
        const int m = x / TN, ni = x % TN;
        if (m < 3) {
#pragma unroll
          for (int mi = 0; mi < NM; ++mi)
            if (mi * TN / NM == ni) load_a(m + 1, mi);
        }
        u32x4 nb = b;
        if (x + 1 < 4 * TN)
          nb = e2m1x8_to_bf16(bc[(x + 1) % TN][(x + 1) / TN], bf[(x + 1) % TN]);
#pragma unroll
        for (int mi = 0; mi < NM; ++mi)
          acc[mi][ni] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, a[m & 1][mi]),
              acc[mi][ni], 0, 0, 0);
        b = nb;
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
}

// Column parts of the output's staging, and the stores that a wave issues.
template <int MODE, typename R, int BM>
constexpr int mx_ring_passes() {
  return BM * (MODE == 0 ? R::BN / 2 : R::BN) / 8 > R::STAGE_CH ? 2 : 1;
}
template <int MODE, bool AF4, typename R, int BM>
constexpr int mx_ring_stores() {
  // FP4 h: codes and scales of 32 rows at a time; else 1 KiB a store
  if (MODE == 0 && AF4) return BM / 32 * 2;
  return R::WM * (MODE == 0 ? R::WN / 2 : R::WN) * 2 / 1024;
}

// The K loop of one tile over the wave's NM live row fragments (0: copies and
// barriers only).  (One loop for each NM, chosen outside it: variants inside
// one loop cost a second set of accumulators where they meet.)
template <int MODE, bool AF4, typename R, int BM, int NM>
__device__ __forceinline__ void mx_ring_kloop(const MxTile<R>& t, u32x4* ring, int wm, int wn,
                                              int wvs, int lane, bool stores,
                                              f32x4 (&acc)[R::TM][R::TN]) {
  const int K = t.K, KT = (K + R::BK - 1) / R::BK;
  auto enter = [&](int kt) {
    if (wvs < R::NI) mx_ring_wait<R, mx_ring_stores<MODE, AF4, R, BM>()>(kt, KT, stores);
    raw_barrier();
    if (kt + R::STAGES - 1 < KT && wvs < R::NI)
      mx_ring_stage<MODE, AF4, R, BM>(t, ring, kt + R::STAGES - 1, wvs);
  };
  const int full = K / R::BK;
  for (int kt = 0; kt < full; ++kt) {
    enter(kt);
    if constexpr (NM > 0) mx_ring_mma<MODE, AF4, R, NM, R::BK / 128>(ring, kt, wm, wn, lane, acc);
  }
  if (R::BK == 256 && full < KT) {
    enter(full);
    if constexpr (NM > 0) mx_ring_mma<MODE, AF4, R, NM, 1>(ring, full, wm, wn, lane, acc);
  }
}

template <int MODE, bool AF4, typename R, int BM, int NM = R::TM>
__device__ __forceinline__ void mx_ring_kloop_live(const MxTile<R>& t, u32x4* ring, int wm, int wn,
                                                   int wvs, int lane, int live, bool stores,
                                                   f32x4 (&acc)[R::TM][R::TN]) {
  if constexpr (NM > 0) {
    if (live < NM)
      return mx_ring_kloop_live<MODE, AF4, R, BM, NM - 1>(t, ring, wm, wn, wvs, lane, live, stores,
                                                          acc);
  }
  mx_ring_kloop<MODE, AF4, R, BM, NM>(t, ring, wm, wn, wvs, lane, stores, acc);
}

// The tile's output through the free ring slot: every wave stages its rows in
// a part of its own, its chunks swizzled by row, in PASSES column
// parts where the slot does not hold them all, and whole 16-byte row chunks go
// out; a chunk past the segment or past N takes an offset beyond the store's
// range and is dropped.  GEMM 1 with FP4 activations: after a barrier, 16
// lanes take one row's 128 columns of h, 4 lanes a 1 x 32 block, and write
// its codes (64 contiguous bytes a row) and scales.
template <int MODE, bool AF4, typename R, int BM>
__device__ __forceinline__ void mx_ring_store(const MxProblem& P, const MxTile<R>& t,
                                              const u32x2* out, u32x4* slot) {
  constexpr int TM = R::TM, WM = R::WM, NPM = MODE == 0 ? R::TN / 2 : R::TN;
  constexpr int COUT = MODE == 0 ? R::WN / 2 : R::WN;
  constexpr int PASSES = mx_ring_passes<MODE, R, BM>();
  constexpr int NP = NPM / PASSES, CPR = COUT / PASSES / 8, RPI = 64 / CPR;
  static_assert(CPR <= 16 && 64 % CPR == 0 && WM % RPI == 0, "output transpose shape");
  static_assert(8 * WM * CPR <= R::STAGE_CH, "the staged output fits a slot");
  static_assert(!(MODE == 0 && AF4) || PASSES == 1, "h's blocks cross the waves' columns");
  // (16 rows' pieces of one chunk spread over a bank row of 256 bytes)
  auto out_swz = [](int rr) { return rr * CPR / 16 % CPR; };
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));   // (addresses formed here, not kept through the K loop)
  const int wv = threadIdx.x >> 6;
  const int wm = wv / R::WAVES_N, wn = wv % R::WAVES_N;
  u32x4* reg = slot + (size_t)wv * WM * CPR;
  const int N = P.N;
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
#pragma unroll
    for (int mi = 0; mi < TM; ++mi) {
      const int rr = mi * 16 + (lane & 15);   // tile row (mi WAVES_M + wm) 16 + lane % 16
#pragma unroll
      for (int ni = 0; ni < NP; ++ni) {
        const int c = ni * 2 + ((lane >> 4) >> 1);
        reinterpret_cast<u32x2*>(reg + rr * CPR + (c ^ out_swz(rr)))[(lane >> 4) & 1] =
            out[mi * NPM + p * NP + ni];
      }
    }
    if constexpr (MODE == 0 && AF4) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      raw_barrier();   // every wave's rows are staged
      const __amdgpu_buffer_rsrc_t rq =
          buffer_rsrc(P.Cq + (size_t)t.r0 * (N / 2), (uint32_t)((size_t)t.len * (N / 2)));
      const __amdgpu_buffer_rsrc_t re =
          buffer_rsrc(P.c_e8 + (size_t)t.r0 * (N / 32), (uint32_t)((size_t)t.len * (N / 32)));
      int tid = threadIdx.x;
      asm volatile("" : "+v"(tid));
      const int cc = tid & 15;                          // this lane's 8 of the 128 columns
      const int swn = cc / CPR, sc = cc % CPR;
#pragma unroll
      for (int it = 0; it < BM / 32; ++it) {
        const int row = it * 32 + (tid >> 4);
        const int frag = row / 16, swm = frag % R::WAVES_M;
        const int rr = frag / R::WAVES_M * 16 + row % 16;
        const u32x4 v =
            slot[(size_t)(swm * R::WAVES_N + swn) * WM * CPR + rr * CPR + (sc ^ out_swz(rr))];
        float f[8];
        uint32_t a = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f[2 * j] = __uint_as_float(v[j] << 16);
          f[2 * j + 1] = __uint_as_float(v[j] & 0xffff0000u);
          a = max(a, max(__float_as_uint(f[2 * j]) & 0x7fffffffu,
                         __float_as_uint(f[2 * j + 1]) & 0x7fffffffu));
        }
        a = max(a, (uint32_t)wave_dev::dpp<0xB1>((int)a));
        a = max(a, (uint32_t)wave_dev::dpp<0x4E>((int)a));
        const uint32_t b = block_e8m0(a);
        const uint32_t codes = e2m1x8(f, b);
        const int grow = t.m0 + row;
        const uint32_t off = grow < t.len
                                 ? ((uint32_t)grow * (uint32_t)N + (uint32_t)(t.n0 + cc * 8)) / 2u
                                 : 0xFFFFFFF0u;
        __builtin_amdgcn_raw_buffer_store_b32(codes, rq, off, 0, 0);
        // (no branch: the waits count every wave's stores)
        __builtin_amdgcn_raw_buffer_store_b8((uint8_t)b, re, (cc & 3) == 0 ? off / 16u : 0xFFFFFFF0u,
                                             0, 0);
      }
    } else {
      wave_lds_fence();
      const __amdgpu_buffer_rsrc_t rc =
          buffer_rsrc(P.C + (size_t)t.r0 * N, (uint32_t)((size_t)t.len * N * 2));
      const int col0 = t.n0 + wn * COUT + p * (COUT / PASSES);
#pragma unroll
      for (int it = 0; it < WM / RPI; ++it) {
        const int rr = it * RPI + lane / CPR, c = lane % CPR;
        const u32x4 v = reg[rr * CPR + (c ^ out_swz(rr))];
        const int row = t.m0 + (rr / 16 * R::WAVES_M + wm) * 16 + rr % 16, col = col0 + c * 8;
        const uint32_t off = (row < t.len && col < N)
                                 ? ((uint32_t)row * (uint32_t)N + (uint32_t)col) * 2u
                                 : 0xFFFFFFF0u;
        __builtin_amdgcn_raw_buffer_store_b128(v, rc, off, 0, MODE == 1 ? kAuxNT : 0);
      }
      wave_lds_fence();
    }
  }
}

constexpr int kMxSmall = 64, kMxBig = 256;

// 16-byte chunks of LDS that the classes of a launch need.
template <bool AF4, int STAGES, bool BIG>
constexpr int mx_ring_lds() {
  constexpr int a = MxRing<AF4, 64, AF4 ? STAGES : 2, AF4 ? 2 : 1>::LDS_CH, b = MxRing<AF4, 128, STAGES, 2>::LDS_CH,
                c = BIG ? MxRing<AF4, 256, 2, 4>::LDS_CH : 0;
  return a > b ? (a > c ? a : c) : (b > c ? b : c);
}

// Every tile of one class: the segments of [min_len, max_len) rows on tiles of
// BM rows, from the class's queue.  The last wave, which issues no copies,
// fetches a tile's number and looks it up while the tile before is computed,
// and leaves the place in `mail`.  (Tiles at a fixed stride, FP4 activations:
// 1712 us against 1600 for 4096 tokens over 256 experts, 1883 against 1774 for
// 16384 over 128; bf16 ones 1494 / 1479 and 924 / 924.  The order in which
// tiles are taken changes no result.)
template <int MODE, bool AF4, int BM, int STAGES, int WAVES_M>
__device__ __forceinline__ void mx_ring_class(const MxArgs& args, u32x4* ring, int* tiles_l,
                                              int min_len, int max_len, int32_t* queue) {
  using R = MxRing<AF4, BM, STAGES, WAVES_M>;
  constexpr int TM = R::TM, TN = R::TN, NPM = MODE == 0 ? TN / 2 : TN;
  constexpr int kFetch = 7;
  const bool fetcher = threadIdx.x == kFetch * 64;
  auto fetch = [&]() -> int {
    return fetcher ? __hip_atomic_fetch_add(queue, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0;
  };
  int ticket = fetch();
  __syncthreads();   // (the class before has left the LDS)
  // (the table's scan borrows the idle ring)
  build_tile_table<512>(args, tiles_l, reinterpret_cast<int*>(ring), BM,
                        MODE == 0 ? R::BN / 2 : R::BN, min_len, max_len);
  const int total = uniform(tiles_l[args.n_seg_total]);
  const int lane = threadIdx.x & 63;
  const int wvs = uniform(threadIdx.x >> 6);
  const int wm = wvs / R::WAVES_N, wn = wvs % R::WAVES_N;
  // (two slots in turn: a slow wave may still read one while the next is left)
  int* mail = tiles_l + args.n_seg_total + 1;
  auto post = [&](int slot) {
    const int tile = mx_queue_tile(uniform(ticket), total);
    MxPlace at{-1, 0, 0, 0, 0, 0};
    if (tile >= 0) at = mx_ring_place<MODE, BM>(args, tiles_l, tile);
    if (lane == 0) {
      int* m = mail + slot * 6;
      m[0] = at.pi;
      m[1] = at.e;
      m[2] = at.r0;
      m[3] = at.len;
      m[4] = at.m0;
      m[5] = at.n0;
    }
  };
  auto read_mail = [&](int slot) -> MxPlace {
    const int* m = mail + slot * 6;
    return {uniform(m[0]), uniform(m[1]), uniform(m[2]), uniform(m[3]), uniform(m[4]), uniform(m[5])};
  };
  if (wvs == kFetch) post(1);
  __syncthreads();   // (and the table's scan has left the ring)
  MxPlace next = read_mail(1);
  if (next.pi < 0) return;
  MxTile<R> t;
  mx_ring_setup<MODE, AF4, R, BM>(args, next, t);
  if (wvs < R::NI) mx_ring_prologue<MODE, AF4, R, BM>(t, ring, wvs);
  ticket = fetch();
  bool stores = false;
  for (int slot = 0;; slot ^= 1) {
    if (wvs == kFetch) post(slot);
    u32x2 outv[TM * NPM];
    {
      f32x4 acc[TM][TN];
#pragma unroll
      for (int mi = 0; mi < TM; ++mi)
#pragma unroll
        for (int ni = 0; ni < TN; ++ni) acc[mi][ni] = f32x4{0.f, 0.f, 0.f, 0.f};
      // row fragments of this wave that hold rows of the segment (a wave with
      // none takes part in the copies and barriers only)
      const int live =
          min(TM, ((t.len - t.m0 + 15) / 16 - wm + R::WAVES_M - 1) / R::WAVES_M);
      mx_ring_kloop_live<MODE, AF4, R, BM>(t, ring, wm, wn, wvs, lane, live, stores, acc);
      // (waited for here: the output is formed behind the next tile's copies,
      // where the wait would be one for the copies)
      if constexpr (MODE == 1) {
#pragma unroll
        for (int mi = 0; mi < TM; ++mi) asm volatile("" : "+v"(t.rs[mi]));
      }
#pragma unroll
      for (int mi = 0; mi < TM; ++mi) {
#pragma unroll
        for (int ni = 0; ni < NPM; ++ni) {
          if (MODE == 0) {
            const f32x4 g = acc[mi][ni], u = acc[mi][ni + TN / 2];
            outv[mi * NPM + ni] =
                u32x2{pack2(silu_fast(g[0]) * u[0], silu_fast(g[1]) * u[1]),
                      pack2(silu_fast(g[2]) * u[2], silu_fast(g[3]) * u[3])};
          } else {
            const f32x4 y = acc[mi][ni];
            const float rs = t.rs[mi];
            outv[mi * NPM + ni] =
                u32x2{pack2(y[0] * rs, y[1] * rs), pack2(y[2] * rs, y[3] * rs)};
          }
        }
      }
    }
    // every wave is done reading the ring, and the mail is there
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    raw_barrier();
    const MxTile<R> done = t;
    next = read_mail(slot);
    const bool more = next.pi >= 0;
    if (more) {
      mx_ring_setup<MODE, AF4, R, BM>(args, next, t);
      if (wvs < R::NI) mx_ring_prologue<MODE, AF4, R, BM>(t, ring, wvs);
    }
    if (more) ticket = fetch();
    // the copies stay before the stores: the waits count on their order
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    mx_ring_store<MODE, AF4, R, BM>(args.p[done.pi], done, outv, ring + (STAGES - 1) * R::STAGE_CH);
    if (!more) break;
    stores = true;
  }
}

constexpr int kMxClasses = 3;

// One grouped GEMM over three classes of segments: up to 64 rows (64-row tiles,
// bound by reading their experts' weights: 5.3 TB/s of codes with FP4
// activations, 3.2 to 4.5 with bf16 ones, whose codes are converted), up to 255
// (128-row tiles; with bf16 activations all longer ones too) and, with FP4
// activations, 256 and more (256-row tiles, bound by the copies and the
// matrix units alike).  Every workgroup works on each class, half of them in
// the opposite order, so that the classes that wait for memory and those that
// compute run side by side (4096 tokens, 256 experts, FP4 activations: 1597
// us, all from the largest class down 1620, from the smallest up 1652).
template <int MODE, bool AF4, int STAGES, bool BIG>
__global__ __launch_bounds__(512, 1) void mx_ring_kernel(MxArgs args) {
  // (the ring and the tile table are the only LDS objects, as in gemm.hip's
  // ring kernel)
  __shared__ __attribute__((aligned(1024))) u32x4 ring[mx_ring_lds<AF4, STAGES, BIG>()];
  extern __shared__ int tiles_l[];
  const int odd = xcd_logical(blockIdx.x, gridDim.x) & 1;
  int32_t* queue = args.queue + blockIdx.x % 8;
  constexpr int n = BIG ? 3 : 2;
  for (int i = 0; i < n; ++i) {
    switch (odd ? i : n - 1 - i) {
      case 0:
        mx_ring_class<MODE, AF4, 64, AF4 ? STAGES : 2, AF4 ? 2 : 1>(args, ring, tiles_l, 1, kMxSmall + 1, queue);
        break;
      case 1:
        mx_ring_class<MODE, AF4, 128, STAGES, 2>(args, ring, tiles_l, kMxSmall + 1,
                                                 BIG ? kMxBig : kAll, queue + 8);
        break;
      default:
        if constexpr (BIG)
          mx_ring_class<MODE, AF4, 256, 2, 4>(args, ring, tiles_l, kMxBig, kAll, queue + 16);
        break;
    }
  }
}

// Clears the queues of one call's two GEMMs (1.4 us; a kernel, so that a
// captured graph holds no memset).
__global__ __launch_bounds__(64) void mx_queue_kernel(int32_t* queue) {
  if (threadIdx.x < 2 * kMxClasses * 8) queue[threadIdx.x] = 0;
}

MxArgs cover(MxArgs g, int bm, int ncols, int min_len, int max_len) {
  g.tile_bm = bm;
  g.tile_ncols = ncols;
  g.min_len = min_len;
  g.max_len = max_len;
  return g;
}

template <int MODE, bool AF4, int TN, int KS, int WPE>
void launch_stream(const MxArgs& g, int min_len, int max_len, hipStream_t s) {
  auto k = mx_stream_kernel<MODE, AF4, TN, KS, WPE>;
  const size_t dyn = (size_t)(g.n_seg_total + 1) * sizeof(int);
  k<<<persistent_grid(k, dyn, 2), 256, dyn, s>>>(
      cover(g, 16, 16 * TN / (MODE == 0 ? 2 : 1), min_len, max_len));
}

// Waves per tile: enough of them to leave each at most 8 stages of K, and more
// where the launch has fewer tiles than the chip takes waves.  us with 4 / 2 /
// 1 waves, 64 tokens, 64 experts: K = 8192 192 / 204 / 205 (bf16 activations),
// 171 / 166 / 186 (FP4); K = 2048 192 / 116 / 104 and 139 / 89 / 82.  One
// token, 8 experts, bf16: K = 7168 28.4 / 27.7 / 41.4, K = 2048 29.5 / 19.1 /
// 16.8.
template <int MODE, bool AF4, int TN, int WPE>
void launch_stream_ks(const MxArgs& g, hipStream_t s) {
  const int64_t ncols = 16 * TN / (MODE == 0 ? 2 : 1);
  int64_t tiles = 0;
  int K = 0;
  for (int p = 0; p < g.n_probs; ++p) {
    const int64_t segs = g.p[p].n_seg < g.p[p].rows ? g.p[p].n_seg : g.p[p].rows;
    tiles += segs * (g.p[p].N / ncols);
    K = g.p[p].K > K ? g.p[p].K : K;
  }
  int ks = K > 4096 ? 4 : K > 2048 ? 2 : 1;
  while (ks < 4 && tiles * ks < (int64_t)device_cu_count() * 4 && K / ks > 512) ks *= 2;
  if (ks == 4) launch_stream<MODE, AF4, TN, 4, WPE>(g, 1, kAll, s);
  else if (ks == 2) launch_stream<MODE, AF4, TN, 2, WPE>(g, 1, kAll, s);
  else launch_stream<MODE, AF4, TN, 1, WPE>(g, 1, kAll, s);
}

// Launches the ring kernel if its LDS holds the launch's tile table beside the
// ring.
template <int MODE, bool AF4, int STAGES, bool BIG>
bool launch_ring(const MxArgs& g, hipStream_t s) {
  const size_t dyn = (size_t)(g.n_seg_total + 1 + 12) * sizeof(int);   // the table and the mail
  if ((size_t)mx_ring_lds<AF4, STAGES, BIG>() * 16 + dyn + 64 > kMaxLdsBytes) return false;
  auto k = mx_ring_kernel<MODE, AF4, STAGES, BIG>;
  k<<<persistent_grid(k, dyn, 1, 512), 512, dyn, s>>>(g);
  return true;
}

// (the smallest rings fit beside the longest table: routed and shared segments)
static_assert(mx_ring_lds<true, 2, false>() * 16 + (kMaxSegments + 2 + 12) * 4 + 64 <= kMaxLdsBytes &&
                  mx_ring_lds<false, 2, false>() * 16 + (kMaxSegments + 2 + 12) * 4 + 64 <= kMaxLdsBytes,
              "every launch has a ring");

template <int MODE, bool AF4>
void launch_gemm(const MxArgs& g, bool few_rows, int longest, hipStream_t s) {
  if (few_rows) {
    // GEMM 1 with FP4 activations takes 32 gate and 32 up rows, so that a tile
    // holds whole 1 x 32 blocks of h; the others 32 weight rows (64, us: bf16
    // activations 200 + 199 against 192 + 104, FP4 GEMM 2 85.6 against 84.2)
    if constexpr (AF4) launch_stream_ks<MODE, AF4, MODE == 0 ? 4 : 2, MODE == 0 ? 2 : 3>(g, s);
    else launch_stream_ks<MODE, AF4, 2, 2>(g, s);
    return;
  }
  // (256-row tiles with FP4 activations only: with bf16 ones 128-row tiles are
  // bound by the matrix units already)
  const bool big = AF4 && longest >= kMxBig;
  if (big && (launch_ring<MODE, AF4, 3, AF4>(g, s) || launch_ring<MODE, AF4, 2, AF4>(g, s))) return;
  if (!launch_ring<MODE, AF4, 3, false>(g, s)) launch_ring<MODE, AF4, 2, false>(g, s);
}

// Streaming tiles for calls of few rows a segment or few rows in all, ring
// tiles for the others.  The ring reads weights as fast from four rows a
// segment on, if its tiles are several to a compute unit; where they are not,
// the streaming tiles, 8 times as many and split over K, fill the chip
// better.  They cross where rows times 128-column tiles of h come to 8 (bf16
// activations) and 16 (FP4) for each unit.  us streaming / ring, rows a segment:
//   H x I                              4          16          64          256
//   4096 x 1536, bf16,   1 expert   22 / 42    28 / 41     27 / 51     71 / 82
//                        8 experts  34 / 49    50 / 50    110 / 55    398 / 126
//                      256 experts 547 / 496 1012 / 558
//                FP4,    1 expert   20 / 36    21 / 36     19 / 39     41 / 60
//                        8 experts  34 / 40    38 / 40     75 / 48    234 / 64
//                      256 experts 436 / 404  624 / 444
//   4096 x 14336, bf16,  1 expert   46 / 113   73 / 113   130 / 125   432 / 254
//                 FP4,   1 expert   46 / 81    56 / 82     81 / 91    260 / 132
// (Segments of very different lengths favour the ring: 256 experts, 4 rows on
// average and 128 at most, 419 / 289 and 283 / 237.)
bool takes_streaming_tiles(const FfnProblem* probs, int n_probs) {
  int64_t rows = 0, segs = 0, tiles = 0;
  for (int p = 0; p < n_probs; ++p) {
    rows += probs[p].rows;
    segs += probs[p].n_seg;
    tiles += (int64_t)probs[p].rows * (probs[p].Iw / 128);
  }
  return rows < 4 * segs || tiles < (probs[0].mx_acts ? 16 : 8) * (int64_t)device_cu_count();
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
  int longest = 0;
  for (int p = 0; p < n_probs; ++p)
    longest = probs[p].max_seg_rows > longest ? probs[p].max_seg_rows : longest;
  const bool few = takes_streaming_tiles(probs, n_probs);
  if (!few) {
    g1.queue = probs[0].queue;
    g2.queue = probs[0].queue + kMxClasses * 8;
    mx_queue_kernel<<<1, 64, 0, s>>>(probs[0].queue);
  }
  if (probs[0].mx_acts) {
    launch_gemm<0, true>(g1, few, longest, s);
    launch_gemm<1, true>(g2, few, longest, s);
  } else {
    launch_gemm<0, false>(g1, few, longest, s);
    launch_gemm<1, false>(g2, few, longest, s);
  }
  MOE_DBG("grouped gemms (MXFP4)");
}

}  // namespace moe
