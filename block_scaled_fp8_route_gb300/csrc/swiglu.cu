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

__device__ __forceinline__ float swiglu(float g, float u) {
  return __fmul_rn(__fdiv_rn(g, __fadd_rn(1.f, expf(-g))), u);
}

// One warp per (row, 512 values): lane l covers values 16 l .. 16 l + 15 of the group, i.e. block
// l / 8; the halves of a lane's 16 values are bounded by K separately (K % 8 == 0), and values from
// K to the next multiple of 128 are stored as zero codes.
__global__ void __launch_bounds__(256) swiglu_quantise_kernel(const uint16_t* __restrict__ y, int64_t T, int64_t K,
                                                              int64_t ld, uint8_t* __restrict__ q,
                                                              int32_t* __restrict__ sf, int64_t sf_ld,
                                                              const int32_t* __restrict__ row_token,
                                                              const int32_t* __restrict__ rows_used) {
  pdl_launch_dependents();
  const int64_t Kp = (K + 127) / 128 * 128;
  const int64_t n_groups = (Kp + 511) / 512;
  const int64_t gw = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (gw >= T * n_groups) return;
  const int64_t t = gw / n_groups;
  const int64_t g = gw - t * n_groups;
  if (row_token != nullptr && (t >= __ldg(rows_used) || __ldg(row_token + t) < 0)) return;   // whole warp
  const int64_t k0 = g * 512 + lane * 16;
  float v[16];
  float amax = 0.f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t k = k0 + 8 * h;
    if (k < K) {
      float fg[8], fu[8];
      bf16x8_to_float(__ldg(reinterpret_cast<const uint4*>(y + t * ld + k)), fg);
      bf16x8_to_float(__ldg(reinterpret_cast<const uint4*>(y + t * ld + K + k)), fu);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[8 * h + i] = swiglu(fg[i], fu[i]);
        amax = fmaxf(amax, fabsf(v[8 * h + i]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[8 * h + i] = 0.f;
    }
  }
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 4));
  const int e = block_exponent(amax);
  const bool active = k0 < Kp;
  if (active) {
    const float s = inv_pow2(e);
    uint4 out;
    out.x = pack4_e4m3(v[0] * s, v[1] * s, v[2] * s, v[3] * s);
    out.y = pack4_e4m3(v[4] * s, v[5] * s, v[6] * s, v[7] * s);
    out.z = pack4_e4m3(v[8] * s, v[9] * s, v[10] * s, v[11] * s);
    out.w = pack4_e4m3(v[12] * s, v[13] * s, v[14] * s, v[15] * s);
    *reinterpret_cast<uint4*>(q + t * Kp + k0) = out;
  }
  const uint32_t byte = active ? static_cast<uint32_t>(e + 127) : 127u;
  const uint32_t b0 = __shfl_sync(0xffffffffu, byte, 0);
  const uint32_t b1 = __shfl_sync(0xffffffffu, byte, 8);
  const uint32_t b2 = __shfl_sync(0xffffffffu, byte, 16);
  const uint32_t b3 = __shfl_sync(0xffffffffu, byte, 24);
  if (lane == 0) sf[g * sf_ld + t] = static_cast<int32_t>(b0 | (b1 << 8) | (b2 << 16) | (b3 << 24));
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
  const int64_t warps = T * (((K + 127) / 128 + 3) / 4);
  const int64_t blocks = (warps * 32 + 255) / 256;
  if (blocks > INT32_MAX) return BSF_ERR_UNSUPPORTED;
  swiglu_quantise_kernel<<<static_cast<unsigned>(blocks), 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint16_t*>(y), T, K, ld, q, sf, sf_ld, token_of_row, rows_used);
  return launch_status();
}
