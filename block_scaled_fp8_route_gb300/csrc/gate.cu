// Router choice: the kr experts of each token and their combine weights, from
// the router's logits.
//
//   s_e   = 1 / (1 + exp(-l_e))  or  exp(l_e - m) / sum_j exp(l_j - m)
//   key_e = s_e + b_e  (balance bias given), or l_e (both scores rise with l)
//   groups of E / G experts: score = max key, or the sum of the two largest
//   s_e + b_e; only the kept_groups best groups take part
//   the kr largest keys, ties to the lowest index; w = s / sum(s chosen) * scale
//
// "GEMM 执行方式" (rainlin-net) §4.2 takes topk_ids / topk_weights as given;
// these are the tensors bsf_route, bsf_dispatch and bsf_combine consume.
//
// One warp per token.  Lane l holds the VPL consecutive experts from l * VPL in registers, so a row of
// logits is read once with wide loads, a group of E / G experts is a run of 32 / G lanes, and the lowest
// lane among equals is the lowest expert.
#include <cfloat>

#include "common.cuh"
#include "host_utils.h"

namespace bsf {
namespace {

constexpr int kGateMaxExperts = 1024;
constexpr int kGateMaxGroups = 32;
constexpr int kGateMaxKr = 32;
constexpr int kGateWarps = 4;           // warps per CTA
constexpr unsigned kAll = 0xffffffffu;
// CTAs per SM: the more warps the better until the registers run out (65533 x 192: 34.3 us with 10 CTAs of
// 48 registers, 40.9 with the 7 that 70 leave; 8192 x 256: 9.9 us with 8, 10.5 with 10, which spill).  The other
// widths, sigmoid + bias, top 8, 65536 and 8192 rows: 64 experts 24.5 and 4.7 us with 12, 24.9 and 5.5 with 8, 24.2
// and 5.4 with 16; 384 experts 75.4 and 12.4 with 4, 83.9 and 16.0 with 3, 72.1 and 12.5 with 5; 512 experts 94.3
// and 16.2 with 4, 103 and 20.9 with 3, 91.3 and 17.0 with 5; 1024 experts 223 and 36.9 with 2, 346 and 51.3
// with 1 (3 would leave 168 registers: 193 and 34.9).
constexpr int gate_ctas(int vpl) { return vpl <= 3 ? 12 : vpl <= 6 ? 10 : vpl <= 8 ? 8 : vpl <= 16 ? 4 : 2; }

struct GateArgs {
  const void* logits;
  int64_t ld;
  const float* bias;
  int64_t T;
  int E, G, kept, kr;
  int kr_lanes;            // power of two >= kr
  int lane_groups;         // a group is 32 / G whole lanes
  int group_shift;         // log2(32 / G) of such groups
  int wide;                // rows may be read with the widest loads (E = 32 VPL, aligned)
  uint32_t group_magic;    // e / (E / G) = (e * group_magic) >> 22 for e < 1024
  int flags;
  float scale;
  int32_t* ids;
  float* weights;
};

__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
// 1 / x of x >= 1 to one unit in the last place (0 above 2**126, where the quotient would be subnormal).
__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float sigmoid(float l) { return reciprocal(1.f + expf(-l)); }

// 2**x to 2 units in the last place (0 below 2**-126).  Only a softmax's sum is built on it, in 3 instructions
// a term instead of the 10 of expf: the argument x * log2(e) is rounded, an error of |x| 2**-24 of the term,
// but terms of large |x| are small ones, and of the sum of E terms it is less than ln(E) 2**-24, one factor of
// every score of the row.  The scores that decide a choice are compared with one another, and at x = -80 a
// rounded argument would cost each of them 2**-18 of its size: they take expf (2 units in the last place;
// 8192 x 256 with a bias, a score per expert: 9.9 us against 9.5).
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
constexpr float kLog2e = 1.4426950408889634f;

// The score of one key for a group's score, at most two a row: one copy, since with more of them inlined rows
// that need none become slower (65533 x 192 by largest logit 35.0 us instead of 34.3; 8192 x 160 in groups by
// their two largest scores 6.6 instead of 6.7).
__device__ __noinline__ float score_of(float k, float m, bool sig) { return sig ? sigmoid(k) : expf(k - m); }

// The VPL logits of this lane (-inf past E); `lane_row` is the row's base plus this lane's first expert.
template <int VPL, bool BF16>
__device__ __forceinline__ void load_row(const GateArgs& p, const char* lane_row, int lane, float (&l)[VPL]) {
  const int e0 = lane * VPL;
  if (BF16) {
    const uint16_t* row = reinterpret_cast<const uint16_t*>(lane_row);
    constexpr int W = VPL % 8 == 0 ? 8 : VPL % 4 == 0 ? 4 : VPL % 2 == 0 ? 2 : 1;   // values per load
    if (W > 1 && p.wide) {
#pragma unroll
      for (int i = 0; i < VPL; i += W) {
        uint32_t w[W >= 2 ? W / 2 : 1];
        if constexpr (W == 8) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + i));
          w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else if constexpr (W == 4) {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(row + i));
          w[0] = v.x, w[1] = v.y;
        } else {
          w[0] = __ldg(reinterpret_cast<const uint32_t*>(row + i));
        }
#pragma unroll
        for (int j = 0; j < W; ++j)
          if (i + j < VPL) l[i + j] = __uint_as_float(j & 1 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        l[i] = e0 + i < p.E ? __uint_as_float(static_cast<uint32_t>(__ldg(row + i)) << 16) : -INFINITY;
    }
  } else {
    const float* row = reinterpret_cast<const float*>(lane_row);
    constexpr int W = VPL % 4 == 0 ? 4 : VPL % 2 == 0 ? 2 : 1;
    if (W > 1 && p.wide) {
#pragma unroll
      for (int i = 0; i < VPL; i += W) {
        if constexpr (W == 4) {
          const float4 v = __ldg(reinterpret_cast<const float4*>(row + i));
          l[i] = v.x, l[i + 1] = v.y, l[i + 2] = v.z, l[i + 3] = v.w;
        } else if constexpr (W == 2) {
          const float2 v = __ldg(reinterpret_cast<const float2*>(row + i));
          l[i] = v.x, l[i + 1] = v.y;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) l[i] = e0 + i < p.E ? __ldg(row + i) : -INFINITY;
    }
  }
}

// Order-preserving unsigned image of a float that is not NaN (-0 as +0); below kFirstFinite for -inf.
constexpr uint32_t kFirstFinite = 0x00800000u;
__device__ __forceinline__ uint32_t order_bits(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}

// c[0] >= c[1] >= ... by Batcher's odd-even merge network (pruned to N; the comparators of an index past N
// would only meet values that sort last).
template <int N>
__device__ __forceinline__ void sort_down(uint32_t (&c)[N]) {
#pragma unroll
  for (int p = 1; p < N; p <<= 1) {
#pragma unroll
    for (int k = p; k >= 1; k >>= 1) {
#pragma unroll
      for (int j = k % p; j + k < N; j += 2 * k) {
#pragma unroll
        for (int i = 0; i < k; ++i) {
          if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const uint32_t hi = max(c[i + j], c[i + j + k]), lo = min(c[i + j], c[i + j + k]);
            c[i + j] = hi;
            c[i + j + k] = lo;
          }
        }
      }
    }
  }
}

// What bounds it: a row is 4 E bytes, but choosing takes a fixed chain of warp operations, so short
// batches are bound by that chain's latency (one token 2.9 us with its launch) and long ones by issue
// slots: about 484 per token of 192 experts in 8 groups (65533 tokens in 34.3 us, 1.5 TB/s, 23 % of the
// copy rate), of which the rounds of the choice and the weights are half whatever E is.  Four lanes per
// token with sorted lists in registers, and one thread per token, took as many slots and twice the latency.
// * A key and its expert share one word: the key's leading bits, then the complement of the expert, so
//   that the words are distinct, a tie goes to the lowest expert, and a maximum names its owner.  Lanes
//   sort their words once (VPL <= 8; two instructions per comparator), and a round of the choice is one
//   reduction and a shift in the lane that gave.  Wider lanes look through all their words in each round.
// * The key's last bits do not fit.  bf16 logits have none there; otherwise, where two neighbours in the
//   order agree in the bits that do fit (about one row in fifty), the row is chosen again by whole keys.
// * Scores are computed only where they decide: with no bias the choice goes by the logits, and only the
//   kr chosen get an exp (plus the sum of a softmax that is not renormalised).
template <int VPL, bool BF16>
__global__ void __launch_bounds__(32 * kGateWarps, gate_ctas(VPL)) gate_kernel(const GateArgs p) {
  pdl_launch_dependents();
  pdl_wait();                                       // (launched as a dependent: nothing is read before)
  __shared__ float s_val[kGateWarps][VPL * 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = p.E;
  const bool sig = p.flags & BSF_GATE_SIGMOID, top2 = p.flags & BSF_GATE_GROUP_TOP2;
  const bool renorm = p.flags & BSF_GATE_RENORMALISE, biased = p.bias != nullptr;
  const bool need_max = !sig && (biased || !renorm || (top2 && p.G > 1));
  const bool need_sum = !sig && (biased || !renorm);
  const int groups = p.G, kr = p.kr;
  float bias[VPL];                                  // (NaN as -inf: such an expert is never chosen)
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    bias[i] = biased && lane * VPL + i < E ? fmaxf(__ldg(p.bias + lane * VPL + i), -INFINITY) : 0.f;

  constexpr int kSize = BF16 ? 2 : 4;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kGateWarps;
  int64_t t = static_cast<int64_t>(blockIdx.x) * kGateWarps + warp;
  if (t >= p.T) return;
  const char* row = static_cast<const char*>(p.logits) + t * p.ld * kSize;
  const int64_t row_step = step * p.ld * kSize;
  float next[VPL];
  load_row<VPL, BF16>(p, row + lane * VPL * kSize, lane, next);
  for (; t < p.T; t += step, row += row_step) {
    float key[VPL];                                 // -inf: not usable (-inf, NaN); +inf as the largest finite float
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = fminf(fmaxf(next[i], -INFINITY), FLT_MAX);
    if (t + step < p.T) load_row<VPL, BF16>(p, row + row_step + lane * VPL * kSize, lane, next);

    float m = 0.f, inv = 1.f;
    if (need_max) {
      m = key[0];
#pragma unroll
      for (int i = 1; i < VPL; ++i) m = fmaxf(m, key[i]);
      m = fmaxf(warp_max(m), -FLT_MAX);            // (finite also where nothing is usable)
    }
    if (need_sum) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) sum += exp2_approx((key[i] - m) * kLog2e);   // exp(-inf) = 0
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
      inv = sum > 0.f ? reciprocal(sum) : 0.f;        // (the largest term is 1)
    }
    auto score = [&](float k) { return sig ? sigmoid(k) : expf(k - m); };
    if (biased) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const float v = fmaf(score(key[i]), inv, bias[i]);
        key[i] = key[i] > -INFINITY ? v : -INFINITY;
      }
    }
    // a group's score from its two largest keys a >= b (scores rise with the logits), -inf where none can be chosen.
    // The sum of two is halved: with biases near the type's lowest value the sum itself would be -inf.
    auto counts = [&](float k) { return biased ? k : score_of(k, m, sig); };
    auto group_score = [&](float a, float b) {
      if (a == -INFINITY || !top2) return a;
      return 0.5f * counts(a) + (b > -INFINITY ? 0.5f * counts(b) : 0.f);
    };

    bool open = true;                               // this lane's experts take part
    if (groups > 1 && p.lane_groups) {
      const int mine = lane >> p.group_shift;
      float gs = key[0];
      if (top2) {
        float a = key[0], b = -INFINITY;
#pragma unroll
        for (int i = 1; i < VPL; ++i) {
          b = fmaxf(b, fminf(a, key[i]));
          a = fmaxf(a, key[i]);
        }
        for (int o = 1; o < 1 << p.group_shift; o <<= 1) {
          const float a2 = __shfl_xor_sync(kAll, a, o), b2 = __shfl_xor_sync(kAll, b, o);
          b = fmaxf(fmaxf(b, b2), fminf(a, a2));
          a = fmaxf(a, a2);
        }
        gs = group_score(a, b);
      } else {
#pragma unroll
        for (int i = 1; i < VPL; ++i) gs = fmaxf(gs, key[i]);
        for (int o = 1; o < 1 << p.group_shift; o <<= 1) gs = fmaxf(gs, __shfl_xor_sync(kAll, gs, o));
      }
      open = false;
      for (int r = 0; r < p.kept; ++r) {
        const float best = warp_max(gs);
        if (best == -INFINITY) break;
        if (mine == (__ffs(__ballot_sync(kAll, gs == best)) - 1) >> p.group_shift) {
          open = true;
          gs = -INFINITY;
        }
      }
    } else if (groups > 1) {
      // groups that end inside a lane: lane g reduces group g from shared memory
      float* val = s_val[warp];
#pragma unroll
      for (int i = 0; i < VPL; ++i) val[lane * VPL + i] = key[i];
      __syncwarp();
      const int per = E / groups;
      float gs = -INFINITY;
      if (lane < groups) {
        float a = -INFINITY, b = -INFINITY;
        for (int i = 0; i < per; ++i) {
          const float v = val[lane * per + i];
          b = fmaxf(b, fminf(a, v));
          a = fmaxf(a, v);
        }
        gs = group_score(a, b);
      }
      __syncwarp();
      uint32_t keep = 0;
      for (int r = 0; r < p.kept; ++r) {
        const float best = warp_max(gs);
        if (best == -INFINITY) break;
        const int g = __ffs(__ballot_sync(kAll, gs == best)) - 1;
        keep |= 1u << g;
        if (lane == g) gs = -INFINITY;
      }
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const uint32_t g = (static_cast<uint32_t>(lane * VPL + i) * p.group_magic) >> 22;
        if (!((keep >> (g & 31)) & 1u)) key[i] = -INFINITY;
      }
    }

    constexpr int kIdBits = VPL == 1 ? 5 : VPL == 2 ? 6 : VPL <= 4 ? 7 : VPL <= 8 ? 8 : VPL <= 16 ? 9 : 10;
    constexpr uint32_t kIdMask = (1u << kIdBits) - 1u;
    uint32_t c[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      c[i] = (order_bits(key[i]) & ~kIdMask) | (kIdMask - static_cast<uint32_t>(lane * VPL + i));
    if constexpr (VPL <= 8) {
      sort_down(c);
      if (!open) c[0] = 0u;                         // a lane that never gives
    } else if (!open) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) c[i] = 0u;
    }
    // round r's word ends up in lane r; one round more shows whether the last choice was clear
    uint32_t mine = 0u, best = 0u;
    for (int r = 0; r <= kr; ++r) {
      uint32_t head = c[0];
      if constexpr (VPL > 8) {
#pragma unroll
        for (int i = 1; i < VPL; ++i) head = max(head, c[i]);
      }
      best = __reduce_max_sync(kAll, head);
      if (best < kFirstFinite) break;
      if (lane == r) mine = best;
      if constexpr (VPL <= 8) {
        if (c[0] == best) {
#pragma unroll
          for (int i = 0; i + 1 < VPL; ++i) c[i] = c[i + 1];
          c[VPL - 1] = 0u;
        }
      } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) c[i] = c[i] == best ? 0u : c[i];
      }
    }
    int my_id = mine && lane < kr ? static_cast<int>(kIdMask - (mine & kIdMask)) : -1;
    if (!BF16 || biased) {
      uint32_t next_word = __shfl_down_sync(kAll, mine, 1);
      if (lane == kr - 1) next_word = best;
      const bool unclear = my_id >= 0 && next_word >= kFirstFinite && ((mine ^ next_word) >> kIdBits) == 0u;
      if (__any_sync(kAll, unclear)) {
        my_id = -1;
        if (!open) {
#pragma unroll
          for (int i = 0; i < VPL; ++i) key[i] = -INFINITY;
        }
        for (int r = 0; r < kr; ++r) {
          float head = key[0];
#pragma unroll
          for (int i = 1; i < VPL; ++i) head = fmaxf(head, key[i]);
          const float most = warp_max(head);
          if (most == -INFINITY) break;
          const int from = __ffs(__ballot_sync(kAll, head == most)) - 1;
          int at = 0;
#pragma unroll
          for (int i = VPL - 1; i >= 0; --i) at = key[i] == most ? i : at;
          const int e = __shfl_sync(kAll, lane * VPL + at, from);
          if (lane == r) my_id = e;
#pragma unroll
          for (int i = 0; i < VPL; ++i)
            if (lane == from && i == at) key[i] = -INFINITY;
        }
      }
    }

    // lane r: the score of choice r, from its logit (still in a cache)
    float l = -INFINITY;
    if (my_id >= 0) {
      const char* at = row + my_id * kSize;
      if (BF16)
        l = __uint_as_float(static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(at))) << 16);
      else
        l = __ldg(reinterpret_cast<const float*>(at));
      l = fminf(l, FLT_MAX);
    }
    // weights that are divided by their sum are taken relative to the largest chosen logit (without a bias the
    // first choice), which a bias may have put so far below the row's that every exp(l - m) would vanish
    if (!sig && renorm) m = biased ? warp_max(l) : __shfl_sync(kAll, l, 0);
    float w = 0.f;
    if (my_id >= 0) w = sig ? sigmoid(l) : expf(l - m) * inv;
    if (renorm) {
      float total = w;
      for (int o = p.kr_lanes >> 1; o > 0; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
      w = total > 0.f ? __fdiv_rn(w, total) : 0.f;
    }
    if (lane < kr) {
      p.ids[t * kr + lane] = my_id;
      p.weights[t * kr + lane] = w * p.scale;
    }
  }
}

template <int VPL>
bsf_status launch_gate(GateArgs a, bool bf16, cudaStream_t s) {
  const int size = bf16 ? 2 : 4;
  const int bytes = VPL * size % 16 == 0 ? 16 : VPL * size % 8 == 0 ? 8 : VPL * size % 4 == 0 ? 4 : 2;
  a.wide = a.E == 32 * VPL && reinterpret_cast<uintptr_t>(a.logits) % bytes == 0 && a.ld * size % bytes == 0;
  a.lane_groups = a.E == 32 * VPL && 32 % a.G == 0;
  while ((a.G << (a.group_shift + 1)) <= 32) ++a.group_shift;
  // one row per warp until every SM has its warps, then each warp goes on with the next row in flight
  const int64_t most = static_cast<int64_t>(sm_count()) * gate_ctas(VPL);
  const int64_t need = (a.T + kGateWarps - 1) / kGateWarps;
  const unsigned blocks = static_cast<unsigned>(need < most ? need : most);
  return launch_dependent(bf16 ? gate_kernel<VPL, true> : gate_kernel<VPL, false>, blocks, 32 * kGateWarps, 0, s, a);
}

}  // namespace
}  // namespace bsf

using namespace bsf;

extern "C" bsf_status bsf_gate(const void* logits, int logits_type, int64_t T, int64_t E, int64_t ld,
                               const float* bias, int64_t groups, int64_t kept_groups, int64_t kr, int flags,
                               float scale, int32_t* topk_ids, float* topk_weights, bsf_stream_t stream) {
  if (T < 0 || E <= 0 || kr <= 0 || groups <= 0 || kept_groups <= 0) return BSF_ERR_INVALID_ARGUMENT;
  if (logits_type != BSF_TYPE_F32 && logits_type != BSF_TYPE_BF16) return BSF_ERR_INVALID_ARGUMENT;
  if (flags & ~(BSF_GATE_SIGMOID | BSF_GATE_GROUP_TOP2 | BSF_GATE_RENORMALISE)) return BSF_ERR_INVALID_ARGUMENT;
  if (groups > E || E % groups || kept_groups > groups || kr > E || ld < E) return BSF_ERR_INVALID_ARGUMENT;
  if (kr > kept_groups * (E / groups)) return BSF_ERR_INVALID_ARGUMENT;
  if (!(scale >= -FLT_MAX && scale <= FLT_MAX)) return BSF_ERR_INVALID_ARGUMENT;
  if (E > kGateMaxExperts || groups > kGateMaxGroups || kr > kGateMaxKr) return BSF_ERR_UNSUPPORTED;
  if (T == 0) return BSF_OK;
  if (!logits || !topk_ids || !topk_weights) return BSF_ERR_INVALID_ARGUMENT;
  const uintptr_t align = logits_type == BSF_TYPE_F32 ? 3 : 1;
  if ((reinterpret_cast<uintptr_t>(logits) & align) || (reinterpret_cast<uintptr_t>(bias) & 3) ||
      (reinterpret_cast<uintptr_t>(topk_ids) & 3) || (reinterpret_cast<uintptr_t>(topk_weights) & 3))
    return BSF_ERR_MISALIGNED;
  if (!fits_rows(T, ld)) return BSF_ERR_UNSUPPORTED;
  GateArgs a = {};
  a.logits = logits;
  a.ld = ld;
  a.bias = bias;
  a.T = T;
  a.E = static_cast<int>(E);
  a.G = static_cast<int>(groups);
  a.kept = static_cast<int>(kept_groups);
  a.kr = static_cast<int>(kr);
  a.kr_lanes = 1;
  while (a.kr_lanes < a.kr) a.kr_lanes *= 2;
  const uint32_t per = static_cast<uint32_t>(E / groups);
  a.group_magic = ((1u << 22) + per - 1) / per;
  a.flags = flags;
  a.scale = scale;
  a.ids = topk_ids;
  a.weights = topk_weights;
  const bool bf16 = logits_type == BSF_TYPE_BF16;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int vpl = (a.E + 31) / 32;
  if (vpl == 1) return launch_gate<1>(a, bf16, s);
  if (vpl == 2) return launch_gate<2>(a, bf16, s);
  if (vpl == 3) return launch_gate<3>(a, bf16, s);
  if (vpl == 4) return launch_gate<4>(a, bf16, s);
  if (vpl == 5) return launch_gate<5>(a, bf16, s);
  if (vpl == 6) return launch_gate<6>(a, bf16, s);
  if (vpl == 7) return launch_gate<7>(a, bf16, s);
  if (vpl == 8) return launch_gate<8>(a, bf16, s);
  if (vpl <= 12) return launch_gate<12>(a, bf16, s);
  if (vpl <= 16) return launch_gate<16>(a, bf16, s);
  return launch_gate<32>(a, bf16, s);
}
