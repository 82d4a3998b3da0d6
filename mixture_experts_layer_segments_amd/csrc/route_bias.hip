// Top-k routing with a selection bias per expert (balance without an auxiliary
// loss: the bias moves which experts are picked, the weights come from the
// scores alone).
//
//   s_e = sigmoid(l_e), or softmax over the row's unmasked experts
//   c_e = s_e + b_e                      (what is selected on)
//   groups: the topk_group largest sums of a group's best `topn` c
//   winners: the k largest c of the kept groups
//   w_j = s_j [/ sum of the winners' s] * routed_scale
//
// Everything that is compared is in fp64, so that an order of two experts is
// the order of the formulas except within a few 2^-53; ties go to the lower
// id.  (fp32 scores with the near ties routed again in fp64: nearly every batch
// holds a tie near enough, and its wave sets the time.  256 experts in 8
// groups: 13.1 us at 4096 tokens and 19.3 at 16384, against 10.1 and 24.3.)  A
// masked expert (logit at or below the lowest finite fp32, -inf or NaN; or a
// bias of -inf or NaN) is never picked: slots that find no expert left get
// id -1 and weight 0, which the permutation drops.
//
// G lanes (16, 32 or 64) route one token; lane j of them holds experts j VPL ..
// +VPL-1.  A round is the maximum over the lane's own, over the lanes by
// register moves, and the lowest id that holds it.  Bound by issue and, in
// small batches, by the length of the k rounds' chain.
#include <float.h>
#include <math.h>

#include "route_dev.h"
#include "wave_dev.h"

namespace moe {
namespace {

using namespace route_dev;

struct RouteArgs {
  const float* logits;
  const float* bias;
  int T, E, k, score, n_group, topk_group, topn, renorm;
  float routed_scale;
  int32_t* ids;
  float* w;
};

__device__ __forceinline__ double swap32_f64(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)wave_dev::swap_partner<true>((int)(uint32_t)b);
  const uint32_t hi = (uint32_t)wave_dev::swap_partner<true>((int)(uint32_t)(b >> 32));
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// Maximum over every aligned block of P lanes (a power of two), to all of the
// block (no NaN).
__device__ __forceinline__ double block_max(double x, int P) {
  if (P >= 2) x = fmax(x, dpp_f64<0xB1>(x));
  if (P >= 4) x = fmax(x, dpp_f64<0x4E>(x));
  if (P >= 8) x = fmax(x, dpp_f64<0x141>(x));
  if (P >= 16) x = fmax(x, dpp_f64<0x140>(x));
  if (P >= 32) x = fmax(x, swap16_f64(x));
  if (P >= 64) x = fmax(x, swap32_f64(x));
  return x;
}
template <int G>
__device__ __forceinline__ double token_sum(double x) {
  x += dpp_f64<0xB1>(x);
  x += dpp_f64<0x4E>(x);
  x += dpp_f64<0x141>(x);
  x += dpp_f64<0x140>(x);
  if constexpr (G >= 32) x += swap16_f64(x);
  if constexpr (G >= 64) x += swap32_f64(x);
  return x;
}
template <int G>
__device__ __forceinline__ int token_min(int x) {
  x = min(x, wave_dev::dpp<0xB1>(x));
  x = min(x, wave_dev::dpp<0x4E>(x));
  x = min(x, wave_dev::dpp<0x141>(x));
  x = min(x, wave_dev::dpp<0x140>(x));
  if constexpr (G >= 32) x = min(x, wave_dev::swap_partner<false>(x));
  if constexpr (G >= 64) x = min(x, wave_dev::swap_partner<true>(x));
  return x;
}

template <int VPL>
__device__ __forceinline__ double lane_max(const double (&c)[VPL]) {
  double m = c[0];
#pragma unroll
  for (int i = 1; i < VPL; ++i) m = fmax(m, c[i]);
  return m;
}

// In the lanes of `here`, the first value equal to `best` becomes -inf.
template <int VPL>
__device__ __forceinline__ void drop_first(double (&c)[VPL], double best, bool here) {
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const bool hit = here && c[i] == best;
    c[i] = hit ? -INFINITY : c[i];
    here = here && !hit;
  }
}

template <int G, int VPL>
__global__ __launch_bounds__(256) void route_biased_kernel(RouteArgs A) {
  constexpr int TPW = 64 / G;
  const int lane = threadIdx.x & 63;
  const int t0 = __builtin_amdgcn_readfirstlane((blockIdx.x * 4 + (threadIdx.x >> 6)) * TPW);
  if (t0 >= A.T) return;   // the whole wave is past the batch
  // (lanes of a token past the batch route the last one and store nothing)
  const int j = lane % G, base = lane & ~(G - 1), t = min(t0 + lane / G, A.T - 1);
  const int E = A.E, k = A.k, e0 = j * VPL;
  const float* row = A.logits + (size_t)t * E;
  float l[VPL], b[VPL];
  // (16-byte loads where every lane's piece of a row is aligned)
  if (VPL % 4 == 0 && E % 4 == 0 && (((uintptr_t)A.logits | (uintptr_t)A.bias) & 15) == 0) {
#pragma unroll
    for (int i = 0; i < VPL; i += 4) {
      float4 v = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, u = {0.f, 0.f, 0.f, 0.f};
      if (e0 + i < E) {
        v = *reinterpret_cast<const float4*>(row + e0 + i);
        if (A.bias) u = *reinterpret_cast<const float4*>(A.bias + e0 + i);
      }
      l[i] = v.x; l[i + 1] = v.y; l[i + 2] = v.z; l[i + 3] = v.w;
      b[i] = u.x; b[i + 1] = u.y; b[i + 2] = u.z; b[i + 3] = u.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      l[i] = e0 + i < E ? row[e0 + i] : -INFINITY;
      b[i] = e0 + i < E && A.bias ? A.bias[e0 + i] : 0.0f;
    }
  }
  bool live[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    live[i] = l[i] > -FLT_MAX && b[i] > -INFINITY;   // false for NaN
    l[i] = fminf(l[i], FLT_MAX);
  }
  double c[VPL];
  double top = 0.0, denom = 1.0;   // softmax: s = exp(l - top) / denom
  if (A.score == MOE_SCORE_SOFTMAX) {
    double m = -INFINITY, sum = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) m = live[i] ? fmax(m, (double)l[i]) : m;
    top = block_max(m, G);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      c[i] = live[i] ? exp((double)l[i] - top) : 0.0;
      sum += c[i];
    }
    denom = token_sum<G>(sum);
#pragma unroll
    for (int i = 0; i < VPL; ++i) c[i] = live[i] ? c[i] / denom + (double)b[i] : -INFINITY;
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      c[i] = live[i] ? 1.0 / (1.0 + exp(-(double)l[i])) + (double)b[i] : -INFINITY;
  }

  if (A.n_group > 1) {
    const int per = E / A.n_group, P = per / VPL;
    // lane g (the launcher gives a token at least n_group lanes): group g's score
    double gs = -INFINITY;
    double cc[VPL];
    if (per % VPL == 0 && (P & (P - 1)) == 0) {
      // groups are aligned blocks of P lanes: every round takes all groups'
      // next best member at once
      const uint64_t block = (~0ull >> (64 - P)) << (lane & ~(P - 1));
      double s = -INFINITY;
#pragma unroll
      for (int i = 0; i < VPL; ++i) cc[i] = c[i];
      for (int r = 0; r < A.topn; ++r) {
        const double mine = lane_max(cc), best = block_max(mine, P);
        if (best > -INFINITY) s = r == 0 ? best : s + best;
        const uint64_t has = __ballot(mine == best) & block;
        drop_first(cc, best, lane == __ffsll((unsigned long long)has) - 1);
      }
      gs = __shfl(s, base + (j * P) % G);
    } else {
      for (int g = 0; g < A.n_group; ++g) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) cc[i] = (e0 + i) / per == g ? c[i] : -INFINITY;
        double s = -INFINITY;
        for (int r = 0; r < A.topn; ++r) {
          const double mine = lane_max(cc), best = block_max(mine, G);
          if (best > -INFINITY) s = r == 0 ? best : s + best;
          const uint64_t has = __ballot(mine == best) & ((~0ull >> (64 - G)) << base);
          drop_first(cc, best, lane == __ffsll((unsigned long long)has) - 1);
        }
        if (j == g) gs = s;
      }
    }
    // a group is kept when fewer than topk_group others come before it
    int before = 0;
    for (int g = 0; g < A.n_group; ++g) {
      const double o = __shfl(gs, base + g);
      before += (o > gs || (o == gs && g < j)) ? 1 : 0;
    }
    const uint64_t kept = __ballot(j < A.n_group && before < A.topk_group) >> base;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = e0 + i;
      if (e >= E || !((kept >> (e / per)) & 1ull)) c[i] = -INFINITY;
    }
  }

  int my_id = -1;
  for (int r = 0; r < k; ++r) {
    const double best = block_max(lane_max(c), G);
    int id = 0x7fffffff;
#pragma unroll
    for (int i = VPL - 1; i >= 0; --i) id = c[i] == best ? e0 + i : id;
    id = token_min<G>(id);
#pragma unroll
    for (int i = 0; i < VPL; ++i) c[i] = e0 + i == id ? -INFINITY : c[i];
    if (j == r && best > -INFINITY) my_id = id;   // (else no expert is left)
  }

  // the winners' scores, formed again from their logits
  double s = 0.0;
  if (my_id >= 0) {
    const double x = (double)fminf(row[my_id], FLT_MAX);
    s = A.score == MOE_SCORE_SOFTMAX ? exp(x - top) / denom : 1.0 / (1.0 + exp(-x));
  }
  if (A.renorm) {
    const double sum = token_sum<G>(s);
    s = sum > 0.0 ? s / sum : 0.0;
  }
  if (t0 + lane / G < A.T && j < k) {
    A.ids[(size_t)t * k + j] = my_id;
    A.w[(size_t)t * k + j] = (float)(s * (double)A.routed_scale);
  }
}

template <int G, int VPL>
void launch(const RouteArgs& A, hipStream_t s) {
  constexpr int per_block = 4 * (64 / G);
  route_biased_kernel<G, VPL><<<(A.T + per_block - 1) / per_block, 256, 0, s>>>(A);
}

template <int G>
void launch_vpl(const RouteArgs& A, hipStream_t s) {
  const int vpl = (A.E + G - 1) / G;
  if (vpl <= 1) launch<G, 1>(A, s);
  else if (vpl <= 2) launch<G, 2>(A, s);
  else if (vpl <= 4) launch<G, 4>(A, s);
  else if (vpl <= 8) launch<G, 8>(A, s);
  else launch<G, 16>(A, s);
}

}  // namespace

void launch_route_biased(const moe_config& c, const float* logits, const float* bias,
                         float routed_scale, int32_t* ids, float* w, hipStream_t s) {
  const RouteArgs A{logits, bias, c.T, c.E, c.k, c.score, c.n_group, c.topk_group,
                    c.group_score_topn, c.renormalize, routed_scale, ids, w};
  const int need = c.k > c.n_group ? c.k : c.n_group;   // lanes that hold a result
  // More lanes shorten the chain of rounds, fewer issue less per token.  While
  // every SIMD has a wave or less (1024 tokens of 64 lanes, 4096 of 32 being
  // two), the chain is the time.  us with 64 / 32 / 16 lanes, 256 experts in 8
  // groups: 7.0 / 8.2 / 11.6 at 1024 tokens, 11.6 / 10.1 / 11.8 at 4096,
  // 33.7 / 26.3 / 24.3 at 16384; 128 experts, no groups: 4.6 / 4.7 / 5.8,
  // 8.4 / 6.1 / 6.1 and 24.6 / 15.0 / 11.8.
  const int lanes = c.T <= 1024 ? 64 : c.T <= 4096 ? 32 : 16;
  if (lanes <= 16 && need <= 16 && c.E <= 256) launch_vpl<16>(A, s);
  else if (lanes <= 32 && need <= 32 && c.E <= 512) launch_vpl<32>(A, s);
  else launch_vpl<64>(A, s);
}

}  // namespace moe
