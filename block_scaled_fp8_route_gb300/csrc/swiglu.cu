// SwiGLU of a gate-up product, quantised straight into the FP8 operand of the
// down product:
//
//   h = g / (1 + exp(-g)) * u     (float32, each operation rounded once)
//   q = E4M3(h * 2**-e), e the least integer with max|h| <= 448 * 2**e over a
//   1 x 128 block, kept as a UE8M0 byte (the arithmetic of bsf_quantise_act)
//
// DeepGEMM FP8 article (nxmr.cn), "补偿机制一" (1 x 128 power-of-two scales).
#include "common.cuh"
#include "host_utils.h"
#include "quant_math.cuh"

namespace bsf {
namespace {

// Two float32 values in one 64-bit register: add, mul and fma of a pair cost one issue slot, each half
// rounded once.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t v;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t v;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t v;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
  return v;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// g / (1 + exp(-g)) * u of a pair with |g| <= kPlainGate, from -g: the quotient by the hardware reciprocal, then
// corrected once by its exact remainder (Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990).  For every bf16 g in that range this is the IEEE quotient (the test of both
// branches compares the codes of all of them, with 128 ups each).  Numerator and reciprocal are taken negated: the
// remainder of a zero is +0 either way, and times -r it leaves the sign of a zero quotient as it is.
constexpr float kPlainGate = 80.f;
__device__ __forceinline__ uint64_t swiglu_pair(float minus_g0, float minus_g1, uint64_t u) {
  const uint64_t d = add2(pair(expf(minus_g0), expf(minus_g1)), pair(1.f, 1.f));
  float d0, d1;
  unpair(d, d0, d1);
  const uint64_t minus_r = pair(rcp_approx(-d0), rcp_approx(-d1));
  const uint64_t minus_g = pair(minus_g0, minus_g1);
  const uint64_t q = mul2(minus_g, minus_r);
  return mul2(fma2(fma2(d, q, minus_g), minus_r, q), u);
}

struct RowPiece {
  uint4 gate[2], up[2];
};
// 16 gates and ups at column k0 of a row (zeros from column K on).
__device__ __forceinline__ RowPiece load_piece(const uint16_t* row, int k0, int K) {
  RowPiece r;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const bool in = k0 + 8 * h < K;
    r.gate[h] = in ? __ldcs(reinterpret_cast<const uint4*>(row + k0 + 8 * h)) : make_uint4(0, 0, 0, 0);
    r.up[h] = in ? __ldcs(reinterpret_cast<const uint4*>(row + K + k0 + 8 * h)) : make_uint4(0, 0, 0, 0);
  }
  return r;
}

__device__ __forceinline__ void quantise_piece(const RowPiece& p, bool active, int lane, uint8_t* q_dst,
                                               uint8_t* sf_dst) {
  const uint32_t gw[8] = {p.gate[0].x, p.gate[0].y, p.gate[0].z, p.gate[0].w,
                          p.gate[1].x, p.gate[1].y, p.gate[1].z, p.gate[1].w};
  const uint32_t uw[8] = {p.up[0].x, p.up[0].y, p.up[0].z, p.up[0].w, p.up[1].x, p.up[1].y, p.up[1].z, p.up[1].w};
  __nv_bfloat162 most = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&gw[0]));
#pragma unroll
  for (int i = 1; i < 8; ++i) most = __hmax2_nan(most, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&gw[i])));
  uint64_t v[8];
  if (__low2float(most) <= kPlainGate && __high2float(most) <= kPlainGate) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = swiglu_pair(__uint_as_float((gw[i] << 16) ^ 0x80000000u),
                         __uint_as_float((gw[i] & 0xFFFF0000u) ^ 0x80000000u),
                         pair(__uint_as_float(uw[i] << 16), __uint_as_float(uw[i] & 0xFFFF0000u)));
  } else {
    // gates so large that 1 + exp(-g) may leave the range of the reciprocal, infinities and NaN
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float g0 = __uint_as_float(gw[i] << 16), g1 = __uint_as_float(gw[i] & 0xFFFF0000u);
      v[i] = mul2(pair(__fdiv_rn(g0, __fadd_rn(1.f, expf(-g0))), __fdiv_rn(g1, __fadd_rn(1.f, expf(-g1)))),
                  pair(__uint_as_float(uw[i] << 16), __uint_as_float(uw[i] & 0xFFFF0000u)));
    }
  }
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float a, b;
    unpair(v[i], a, b);
    amax = fmaxf(amax, fmaxf(fabsf(a), fabsf(b)));
  }
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 4));
  const int e = block_exponent(amax);
  if (active) {
    const float s = inv_pow2(e);
    const uint64_t s2 = pair(s, s);
    uint32_t out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b, c, d;
      unpair(mul2(v[2 * i], s2), a, b);
      unpair(mul2(v[2 * i + 1], s2), c, d);
      out[i] = pack4_e4m3(a, b, c, d);
    }
    *reinterpret_cast<uint4*>(q_dst) = make_uint4(out[0], out[1], out[2], out[3]);
  }
  // byte j of the row's word is block j of the group (127 past the last block): one lane of each block
  if ((lane & 7) == 0) sf_dst[lane >> 3] = static_cast<uint8_t>(active ? e + 127 : 127);
}

// One warp per (row, 512 values): lane l covers values 16 l .. 16 l + 15 of the piece, i.e. block l / 8;
// the halves of a lane's 16 values are bounded by K separately (K % 8 == 0), and values from K to the next
// multiple of 128 are stored as zero codes.  A CTA takes 8 * rpw neighbouring rows at piece blockIdx.y,
// warp w rows w, w + 8, ...; a warp looks at the tokens of all its rows at once and loads the next
// routed row's values before it works on the present one's.
//
// Bound by HBM on paper (4 K read, K written a row) and near its limit of issue slots: exp and an IEEE
// division took 48 slots a value (178 us for 65536 routed rows x 2048 of a 98048-row operand); pairs
// of values that share a slot in everything but exp, and a quotient of 3 roundings, leave about 25.
// With the next row's loads in flight that case takes 114 us, 5.9 TB/s, 87 % of the copy rate.
// At most 64 registers (4 CTAs per SM): 3 CTAs 126 us, 5 CTAs (48 registers) 132 us.
__global__ void __launch_bounds__(256, 4) swiglu_quantise_kernel(const uint16_t* __restrict__ y, int64_t T, int K,
                                                                 int64_t ld, uint8_t* __restrict__ q,
                                                                 int32_t* __restrict__ sf, int64_t sf_ld,
                                                                 const int32_t* __restrict__ row_token,
                                                                 const int32_t* __restrict__ rows_used, int rpw) {
  pdl_launch_dependents();
  pdl_wait();                                       // (launched as a dependent: nothing is read before)
  const int Kp = (K + 127) & ~127;
  const int lane = threadIdx.x & 31;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * (8 * rpw) + (threadIdx.x >> 5);
  bool mine = lane < rpw && t0 + 8 * lane < T;
  if (row_token != nullptr && mine) {
    const int token = __ldg(row_token + t0 + 8 * lane);
    mine = t0 + 8 * lane < __ldg(rows_used) && token >= 0;
  }
  uint32_t left = __ballot_sync(0xffffffffu, mine);
  if (left == 0) return;
  const int k0 = blockIdx.y * 512 + lane * 16;
  int64_t t = t0 + 8 * (__ffs(left) - 1);
  RowPiece next = load_piece(y + t * ld, k0, K);
  while (true) {
    const RowPiece now = next;
    uint8_t* q_dst = q + t * Kp + k0;
    uint8_t* sf_dst = reinterpret_cast<uint8_t*>(sf + blockIdx.y * sf_ld + t);
    left &= left - 1;
    if (left) {
      t = t0 + 8 * (__ffs(left) - 1);
      next = load_piece(y + t * ld, k0, K);
    }
    quantise_piece(now, k0 < Kp, lane, q_dst, sf_dst);
    if (!left) break;
  }
}

}  // namespace
}  // namespace bsf

using namespace bsf;

extern "C" bsf_status bsf_swiglu_quantise(const void* y, int64_t T, int64_t K, int64_t ld,
                                          const int32_t* token_of_row, const int32_t* rows_used, uint8_t* q,
                                          int32_t* sf, int64_t sf_ld, bsf_stream_t stream) {
  if (T < 0 || K <= 0 || K % 8 || K > kMaxRowWidth) return BSF_ERR_INVALID_ARGUMENT;
  if (ld < 2 * K) return BSF_ERR_INVALID_ARGUMENT;
  if (T == 0) return BSF_OK;
  if (!y || !q || !sf || (token_of_row == nullptr) != (rows_used == nullptr)) return BSF_ERR_INVALID_ARGUMENT;
  if (sf_ld < T || sf_ld % 4 != 0) return BSF_ERR_INVALID_ARGUMENT;
  if (!aligned16(y) || !aligned16(q) || !aligned16(sf) || ld % 8) return BSF_ERR_MISALIGNED;
  if (!fits_rows(T, ld)) return BSF_ERR_UNSUPPORTED;
  const int64_t groups = ((K + 127) / 128 + 3) / 4;    // <= 2^24 / 512 = 32768, a valid gridDim.y
  // rows per warp: the most, up to 8, that leave 6 CTAs per SM, or 2 where the rows are filtered and most
  // of them may be padding.  More rows per warp hide one row's load under another's arithmetic (60000 x
  // 1536: 99.6 us with 1, 81.8 with 8); fewer keep all SMs busy (500 x 2048: 4.1 us with 1, 8.9 with 8).
  const int64_t least = (token_of_row ? 2 : 6) * static_cast<int64_t>(sm_count());
  int rpw = 8;
  while (rpw > 1 && (T + 8 * rpw - 1) / (8 * rpw) * groups < least) rpw /= 2;
  const dim3 grid(static_cast<unsigned>((T + 8 * rpw - 1) / (8 * rpw)), static_cast<unsigned>(groups));
  return launch_dependent(swiglu_quantise_kernel, grid, 256, 0, reinterpret_cast<cudaStream_t>(stream),
                          static_cast<const uint16_t*>(y), T, static_cast<int>(K), ld, q, sf, sf_ld, token_of_row,
                          rows_used, rpw);
}
