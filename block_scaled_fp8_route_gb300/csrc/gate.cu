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
// One warp per token: lane l holds experts l, l + 32, ... in registers, so a
// row of logits is read once.
#include <cfloat>

#include "common.cuh"
#include "host_utils.h"

namespace bsf {
namespace {

constexpr int kGateMaxExperts = 1024;
constexpr int kGateMaxGroups = 32;
constexpr int kGateMaxKr = 32;
constexpr int kGateWarps = 4;           // tokens per CTA

struct GateArgs {
  const void* logits;
  int64_t ld;
  const float* bias;
  int64_t T;
  int E, G, kept, kr;
  uint32_t group_magic;    // e / (E / G) = (e * group_magic) >> 22 for e < 1024
  float scale;
  int32_t* ids;
  float* weights;
};

// Unsigned image of a float that keeps its order (-0 and +0 the same); 0 = an expert that is not to
// be chosen (no finite or +inf float maps to 0).
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

template <int VPL, bool BF16, bool SIGMOID, bool TOP2, bool RENORM>
__global__ void __launch_bounds__(32 * kGateWarps) gate_kernel(const GateArgs p) {
  pdl_launch_dependents();
  __shared__ float s_val[kGateWarps][VPL * 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kGateWarps + warp;
  if (t >= p.T) return;
  const int E = p.E;
  float s[VPL];
  uint32_t key[VPL];
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 32 * i;
    float l = -INFINITY;
    if (e < E) {
      if (BF16)
        l = __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(p.logits) + t * p.ld + e)) << 16);
      else
        l = __ldg(static_cast<const float*>(p.logits) + t * p.ld + e);
    }
    l = l > -INFINITY ? fminf(l, FLT_MAX) : -INFINITY;     // NaN: not usable
    s[i] = l;
    m = fmaxf(m, l);
  }
  const bool need_score_key = p.bias != nullptr;
  if (SIGMOID) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      key[i] = s[i] > -INFINITY ? order_key(s[i]) : 0u;
      s[i] = key[i] ? __fdiv_rn(1.f, 1.f + expf(-s[i])) : 0.f;
    }
  } else {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      key[i] = s[i] > -INFINITY ? order_key(s[i]) : 0u;
      s[i] = key[i] ? expf(s[i] - m) : 0.f;
      sum += s[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float inv = sum > 0.f ? __fdiv_rn(1.f, sum) : 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) s[i] *= inv;
  }
  if (need_score_key) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + 32 * i;
      if (e < E && key[i]) {
        const float v = s[i] + __ldg(p.bias + e);
        key[i] = v > -INFINITY ? order_key(v) : 0u;
      }
    }
  }
  if (p.G > 1) {
    // group scores: lane g reduces group g from shared memory
    float* val = s_val[warp];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      // a value that orders the group: s (+ b) for the sum of two, the key itself for the maximum
      float v = -INFINITY;
      if (key[i]) v = (TOP2 && !need_score_key) ? s[i] : key_value(key[i]);
      val[lane + 32 * i] = v;
    }
    __syncwarp();
    const int per = E / p.G;
    float gs = -INFINITY;
    if (lane < p.G) {
      float a = -INFINITY, b = -INFINITY;
      for (int i = 0; i < per; ++i) {
        const float v = val[lane * per + i];
        if (TOP2) b = fmaxf(b, fminf(a, v));
        a = fmaxf(a, v);
      }
      gs = TOP2 && b > -INFINITY ? a + b : a;
    }
    int rank = 0;
    for (int g = 0; g < p.G; ++g) {
      const float o = __shfl_sync(0xffffffffu, gs, g);
      rank += (o > gs || (o == gs && g < lane)) ? 1 : 0;
    }
    const uint32_t keep = __ballot_sync(0xffffffffu, lane < p.G && rank < p.kept);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const uint32_t g = (static_cast<uint32_t>(lane + 32 * i) * p.group_magic) >> 22;
      if (!((keep >> (g & 31)) & 1u)) key[i] = 0u;
    }
  }
  // kr rounds: the warp's largest key, the lowest expert that has it
  int my_id = -1;
  float my_s = 0.f;
  for (int r = 0; r < p.kr; ++r) {
    uint32_t best = 0u;
#pragma unroll
    for (int i = 0; i < VPL; ++i) best = max(best, key[i]);
    best = __reduce_max_sync(0xffffffffu, best);
    if (best == 0u) break;
    uint32_t e = 0xFFFFFFFFu;
#pragma unroll
    for (int i = VPL - 1; i >= 0; --i)
      if (key[i] == best) e = lane + 32 * i;
    e = __reduce_min_sync(0xffffffffu, e);
    float se = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (e == static_cast<uint32_t>(lane + 32 * i)) {
        key[i] = 0u;
        se = s[i];
      }
    se = __shfl_sync(0xffffffffu, se, e & 31);
    if (lane == r) {
      my_id = static_cast<int>(e);
      my_s = se;
    }
  }
  float w = my_s;
  if (RENORM) {
    float total = my_s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    w = total > 0.f ? __fdiv_rn(my_s, total) : 0.f;
  }
  if (lane < p.kr) {
    p.ids[t * p.kr + lane] = my_id;
    p.weights[t * p.kr + lane] = w * p.scale;
  }
}

template <int VPL, bool BF16>
void launch_gate(const GateArgs& a, int flags, unsigned blocks, cudaStream_t s) {
  const bool sg = flags & BSF_GATE_SIGMOID, t2 = flags & BSF_GATE_GROUP_TOP2, rn = flags & BSF_GATE_RENORMALISE;
#define BSF_GATE_LAUNCH(S, P, R) gate_kernel<VPL, BF16, S, P, R><<<blocks, 32 * kGateWarps, 0, s>>>(a)
  if (sg) {
    if (t2) { if (rn) BSF_GATE_LAUNCH(true, true, true); else BSF_GATE_LAUNCH(true, true, false); }
    else { if (rn) BSF_GATE_LAUNCH(true, false, true); else BSF_GATE_LAUNCH(true, false, false); }
  } else {
    if (t2) { if (rn) BSF_GATE_LAUNCH(false, true, true); else BSF_GATE_LAUNCH(false, true, false); }
    else { if (rn) BSF_GATE_LAUNCH(false, false, true); else BSF_GATE_LAUNCH(false, false, false); }
  }
#undef BSF_GATE_LAUNCH
}

template <bool BF16>
void launch_gate_width(const GateArgs& a, int flags, unsigned blocks, cudaStream_t s) {
  if (a.E <= 32) launch_gate<1, BF16>(a, flags, blocks, s);
  else if (a.E <= 64) launch_gate<2, BF16>(a, flags, blocks, s);
  else if (a.E <= 128) launch_gate<4, BF16>(a, flags, blocks, s);
  else if (a.E <= 256) launch_gate<8, BF16>(a, flags, blocks, s);
  else if (a.E <= 512) launch_gate<16, BF16>(a, flags, blocks, s);
  else launch_gate<32, BF16>(a, flags, blocks, s);
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
  GateArgs a;
  a.logits = logits;
  a.ld = ld;
  a.bias = bias;
  a.T = T;
  a.E = static_cast<int>(E);
  a.G = static_cast<int>(groups);
  a.kept = static_cast<int>(kept_groups);
  a.kr = static_cast<int>(kr);
  const uint32_t per = static_cast<uint32_t>(E / groups);
  a.group_magic = ((1u << 22) + per - 1) / per;
  a.scale = scale;
  a.ids = topk_ids;
  a.weights = topk_weights;
  const unsigned blocks = static_cast<unsigned>((T + kGateWarps - 1) / kGateWarps);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (logits_type == BSF_TYPE_F32) launch_gate_width<false>(a, flags, blocks, s);
  else launch_gate_width<true>(a, flags, blocks, s);
  return launch_status();
}
