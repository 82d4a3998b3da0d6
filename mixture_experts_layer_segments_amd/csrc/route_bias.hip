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
// id.  A masked expert (logit at or below the lowest finite fp32, -inf or NaN;
// or a bias of -inf or NaN) is never picked: slots that find no expert left
// get id -1 and weight 0, which the permutation drops.
//
// One wave routes one token.  Lane l holds experts l * VPL .. +VPL-1, so that
// the lowest lane that holds the maximum also holds the lowest id: a round is
// the fp64 maximum over the lanes (register moves, route_dev.h), a ballot and
// the first set bit.
#include <float.h>
#include <math.h>

#include "route_dev.h"

namespace moe {
namespace {

using namespace route_dev;

// The larger of x and that of the lane 16 (ROW32 false) or 32 lanes away.
template <bool ROW32>
__device__ __forceinline__ double swap_max_f64(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)b, hi = (uint32_t)(b >> 32);
  uint32_t l0, l1, h0, h1;
  if constexpr (ROW32) {
    const auto rl = __builtin_amdgcn_permlane32_swap(lo, lo, false, false);
    const auto rh = __builtin_amdgcn_permlane32_swap(hi, hi, false, false);
    l0 = rl[0]; l1 = rl[1]; h0 = rh[0]; h1 = rh[1];
  } else {
    const auto rl = __builtin_amdgcn_permlane16_swap(lo, lo, false, false);
    const auto rh = __builtin_amdgcn_permlane16_swap(hi, hi, false, false);
    l0 = rl[0]; l1 = rl[1]; h0 = rh[0]; h1 = rh[1];
  }
  return fmax(__builtin_bit_cast(double, ((uint64_t)h0 << 32) | l0),
              __builtin_bit_cast(double, ((uint64_t)h1 << 32) | l1));
}

// Maximum over every aligned block of P lanes (P a power of two), to all of
// the block (no NaN).
template <int P>
__device__ __forceinline__ double block_max_f64(double x) {
  if constexpr (P >= 2) x = fmax(x, dpp_f64<0xB1>(x));
  if constexpr (P >= 4) x = fmax(x, dpp_f64<0x4E>(x));
  if constexpr (P >= 8) x = fmax(x, dpp_f64<0x141>(x));
  if constexpr (P >= 16) x = fmax(x, dpp_f64<0x140>(x));
  if constexpr (P >= 32) x = swap_max_f64<false>(x);
  if constexpr (P >= 64) x = swap_max_f64<true>(x);
  return x;
}

template <int VPL>
__device__ __forceinline__ double lane_max(const double (&c)[VPL]) {
  double m = c[0];
#pragma unroll
  for (int i = 1; i < VPL; ++i) m = fmax(m, c[i]);
  return m;
}

// In the lanes of `here`, the first value equal to `best` becomes -inf;
// returns its slot.
template <int VPL>
__device__ __forceinline__ int take_first(double (&c)[VPL], double best, bool here) {
  int slot = -1;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const bool hit = here && slot < 0 && c[i] == best;
    if (hit) {
      slot = i;
      c[i] = -INFINITY;
    }
  }
  return slot;
}

// Group scores where a group is an aligned block of P lanes: every round
// takes all groups' next best member at once; each lane returns its group's.
template <int VPL, int P>
__device__ __forceinline__ double group_scores_lanes(const double (&c)[VPL], int topn, int lane) {
  double cc[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) cc[i] = c[i];
  const uint64_t block = (P == 64 ? ~0ull : ((1ull << (P & 63)) - 1)) << (lane & ~(P - 1));
  double gs = -INFINITY;
  for (int r = 0; r < topn; ++r) {
    const double mine = lane_max(cc), best = block_max_f64<P>(mine);
    if (best > -INFINITY) gs = r == 0 ? best : gs + best;
    const uint64_t has = __ballot(mine == best) & block;
    take_first(cc, best, lane == __ffsll((unsigned long long)has) - 1);
  }
  return gs;
}

template <int VPL>
__global__ __launch_bounds__(256) void route_biased_kernel(
    const float* __restrict__ logits, const float* __restrict__ bias, int T, int E, int k,
    int score, int n_group, int topk_group, int topn, int renorm, float routed_scale,
    int32_t* __restrict__ ids, float* __restrict__ w) {
  const int lane = threadIdx.x & 63;
  const int t = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  if (t >= T) return;
  const float* row = logits + (size_t)t * E;
  float l[VPL];
  double c[VPL];
  bool live[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane * VPL + i;
    l[i] = e < E ? row[e] : -INFINITY;
    const float b = e < E && bias ? bias[e] : 0.0f;
    live[i] = l[i] > -FLT_MAX && b > -INFINITY;   // false for NaN
    l[i] = fminf(l[i], FLT_MAX);
    c[i] = (double)b;
  }
  double top = 0.0, denom = 1.0;   // softmax: s = exp(l - top) / denom
  if (score == MOE_SCORE_SOFTMAX) {
    double m = -INFINITY, sum = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (live[i]) m = fmax(m, (double)l[i]);
    top = block_max_f64<64>(m);
    double ex[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      ex[i] = live[i] ? exp((double)l[i] - top) : 0.0;
      sum += ex[i];
    }
    denom = wave_sum(sum);
#pragma unroll
    for (int i = 0; i < VPL; ++i) c[i] = live[i] ? ex[i] / denom + c[i] : -INFINITY;
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      c[i] = live[i] ? 1.0 / (1.0 + exp(-(double)l[i])) + c[i] : -INFINITY;
  }

  if (n_group > 1) {
    const int per = E / n_group;
    double gs = -INFINITY;   // lane g: group g's score
    const int P = per % VPL == 0 ? per / VPL : 0;
    if (P > 0 && 64 % P == 0) {
      double s = 0.0;
      switch (P) {
        case 1: s = group_scores_lanes<VPL, 1>(c, topn, lane); break;
        case 2: s = group_scores_lanes<VPL, 2>(c, topn, lane); break;
        case 4: s = group_scores_lanes<VPL, 4>(c, topn, lane); break;
        case 8: s = group_scores_lanes<VPL, 8>(c, topn, lane); break;
        case 16: s = group_scores_lanes<VPL, 16>(c, topn, lane); break;
        default: s = group_scores_lanes<VPL, 32>(c, topn, lane); break;
      }
      gs = __shfl(s, (lane * P) & 63);
    } else {
      // groups that are no lane blocks: one at a time, over the wave
      for (int g = 0; g < n_group; ++g) {
        double cc[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          cc[i] = (lane * VPL + i) / per == g ? c[i] : -INFINITY;
        double s = -INFINITY;
        for (int r = 0; r < topn; ++r) {
          const double mine = lane_max(cc), best = block_max_f64<64>(mine);
          if (!(best > -INFINITY)) break;
          s = r == 0 ? best : s + best;
          const uint64_t has = __ballot(mine == best);
          take_first(cc, best, lane == __ffsll((unsigned long long)has) - 1);
        }
        if (lane == g) gs = s;
      }
    }
    // a group is kept when fewer than topk_group others come before it
    int before = 0;
    for (int g = 0; g < n_group; ++g) {
      const double o = lane_value(gs, g);
      before += (o > gs || (o == gs && g < lane)) ? 1 : 0;
    }
    const uint64_t kept = __ballot(lane < n_group && before < topk_group);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane * VPL + i;
      if (e >= E || !((kept >> (e / per)) & 1ull)) c[i] = -INFINITY;
    }
  }

  int my_id = -1;
  for (int j = 0; j < k; ++j) {
    const double mine = lane_max(c), best = block_max_f64<64>(mine);
    if (!(lane_value(best, 0) > -INFINITY)) break;   // no expert left
    const uint64_t has = __ballot(mine == best);
    const int win = __ffsll((unsigned long long)has) - 1;
    const int slot = take_first(c, best, lane == win);
    const int id = win * VPL + __builtin_amdgcn_readlane(slot, win);
    if (lane == j) my_id = id;
  }

  // the winners' scores, formed again from their logits
  double s = 0.0;
  if (my_id >= 0) {
    const double x = (double)fminf(row[my_id], FLT_MAX);
    s = score == MOE_SCORE_SOFTMAX ? exp(x - top) / denom : 1.0 / (1.0 + exp(-x));
  }
  if (renorm) {
    const double sum = lanes_sum(s, k);
    s = sum > 0.0 ? s / sum : 0.0;
  }
  if (lane < k) {
    ids[(size_t)t * k + lane] = my_id;
    w[(size_t)t * k + lane] = (float)(s * (double)routed_scale);
  }
}

template <int VPL>
void launch_vpl(const moe_config& c, const float* logits, const float* bias, float routed_scale,
                int32_t* ids, float* w, hipStream_t s) {
  route_biased_kernel<VPL><<<(c.T + 3) / 4, 256, 0, s>>>(
      logits, bias, c.T, c.E, c.k, c.score, c.n_group, c.topk_group, c.group_score_topn,
      c.renormalize, routed_scale, ids, w);
}

}  // namespace

void launch_route_biased(const moe_config& c, const float* logits, const float* bias,
                         float routed_scale, int32_t* ids, float* w, hipStream_t s) {
  const int vpl = (c.E + 63) / 64;
  if (vpl <= 1) launch_vpl<1>(c, logits, bias, routed_scale, ids, w, s);
  else if (vpl <= 2) launch_vpl<2>(c, logits, bias, routed_scale, ids, w, s);
  else if (vpl <= 4) launch_vpl<4>(c, logits, bias, routed_scale, ids, w, s);
  else if (vpl <= 8) launch_vpl<8>(c, logits, bias, routed_scale, ids, w, s);
  else launch_vpl<16>(c, logits, bias, routed_scale, ids, w, s);
}

}  // namespace moe
