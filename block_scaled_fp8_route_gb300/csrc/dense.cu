// Dense FP8 block-scaled product of one weight matrix (an always-active expert,
// a projection), sm_103a:
//
//   D[r, n] = BF16( sum_k A[r, k] sA[r, k/128] * B[n, k] sB[n/128, k/128]  (+ C[r, n]) )
//
// DeepGEMM FP8 article (nxmr.cn), "补偿机制二": the tensor core applies the
// UE8M0 block scales (kind::mxf8f6f4, one scale per row per 32 K; a 128-wide
// block's byte serves its four K = 32 steps, picked by the scale-factor id).
//
// One weight matrix gives only N / 128 tiles of 128 weight rows, too few for
// 152 SMs, so a tile's K is split over a cluster of S CTAs: each multiplies its
// share of the K-blocks into tensor memory, writes the FP32 partial to its own
// shared memory, and after a cluster barrier every CTA sums a slice of the
// tile's tokens over the S partials through distributed shared memory, in rank
// order (no atomics, no workspace, bit-identical from run to run).
//
// Weights are the MMA's M = 128 rows and tokens its N (16..256), so one token
// costs a 128 x 16 product.
#include "common.cuh"
#include "host_utils.h"
#include "tma_map.h"

namespace bsf {
namespace {

constexpr int kTileW = 128;                     // weight rows per tile
constexpr int kTileK = 128;                     // K per stage
constexpr int kMaxTok = 256;                    // tokens per tile
constexpr int kSfSlots = 4;                     // ring of scale words in tensor memory (512 K each)
constexpr int kSfCols = 16;                     // columns per slot: 4 of weights, up to 8 of tokens at 4
constexpr int kAccCol = kSfSlots * kSfCols;     // accumulator columns start here
constexpr int kThreads = 192;                   // producer, issuer, 4 scale + epilogue warps
constexpr int kMaxStages = 12;
constexpr int kBarBytes = 512;
constexpr int kSmemBytes = 227 * 1024;

struct DenseArgs {
  const int32_t* sfa;
  int64_t sfa_ld;
  const int32_t* sfb;        // [nw][Np]
  int64_t Np;
  const uint16_t* addend;
  int64_t ldc;
  uint16_t* d;
  int64_t ldd;
  int M, N, nkb, nw;
  int chunks, per;           // token chunks per weight tile, tokens of a full chunk (multiple of 16)
  int split, stages;
  uint32_t tmem_cols;
  int tiled;
  int vec4;                  // four neighbouring columns of D (and C) are 8-byte aligned
  int* err;
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t local_smem, uint32_t rank) {
  float4 v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %4, %5;\n\t"
      "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(local_smem), "r"(rank)
      : "memory");
  return v;
}
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort, int* err) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, err));
}
__device__ __forceinline__ void wait_quiet(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer_ns() - t0 > kWaitLimitNs) return;
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    dense_split_kernel(const __grid_constant__ CUtensorMap tmap_b, const __grid_constant__ CUtensorMap tmap_a,
                       const DenseArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int stage_bytes = kTileW * kTileK + p.per * kTileK;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + p.stages * stage_bytes);
  uint64_t* full = bars;
  uint64_t* empty = full + kMaxStages;
  uint64_t* sf_full = empty + kMaxStages;
  uint64_t* sf_empty = sf_full + kSfSlots;
  uint64_t* acc_full = sf_empty + kSfSlots;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_full + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile = blockIdx.x / p.split, rank = blockIdx.x - tile * p.split;
  const int nt = tile / p.chunks, chunk = tile - nt * p.chunks;
  const int tok0 = chunk * p.per;
  const int ntok = min(p.per, p.M - tok0);
  const uint32_t mma_n = (ntok + 15) & ~15;
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.nkb) * rank / p.split);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.nkb) * (rank + 1) / p.split);

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kSfSlots; ++s) {
      mbar_init(&sf_full[s], 4);
      mbar_init(&sf_empty[s], 1);
    }
    mbar_init(acc_full, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmap_b);
    tma_prefetch_desc(&tmap_a);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, p.tmem_cols);
    tmem_relinquish();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  bool have = false;                       // this warp holds a complete accumulator (epilogue warps)
  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      uint32_t stage = 0, phase = 0;
      int issued = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.err)) break;
        uint8_t* dst = smem + stage * stage_bytes;
        mbar_arrive_expect_tx(&full[stage], stage_bytes);
        if (p.tiled)
          tma_load_2d(dst, &tmap_b, &full[stage], 0, (nt * p.nkb + kb) * kTileW);
        else
          tma_load_2d(dst, &tmap_b, &full[stage], kb * kTileK, nt * kTileW);
        tma_load_2d(dst + kTileW * kTileK, &tmap_a, &full[stage], kb * kTileK, tok0);
        ++issued;
        if (++stage == static_cast<uint32_t>(p.stages)) { stage = 0; phase ^= 1u; }
      }
      // no TMA write may be in flight when the CTA exits or reuses its stages
      const int outstanding = issued < p.stages ? issued : p.stages;
      for (int j = 0; j < outstanding; ++j) {
        if (stage == 0) { stage = p.stages; phase ^= 1u; }
        --stage;
        wait_quiet(&full[stage], phase);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      uint32_t stage = 0, phase = 0, slot = 0, sf_phase = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (kb == kb0 || (kb & 3) == 0) {
          if (!mbar_wait(&sf_full[slot], sf_phase, abort_flag, p.err)) { ok = false; break; }
        }
        if (!mbar_wait(&full[stage], phase, abort_flag, p.err)) { ok = false; break; }
        tc_fence_after();
        const uint32_t sfw = tmem_base + slot * kSfCols;
        const uint8_t* src = smem + stage * stage_bytes;
        const uint64_t adesc = smem_desc_k_sw128(smem_u32(src));
        const uint64_t bdesc = smem_desc_k_sw128(smem_u32(src + kTileW * kTileK));
        const uint32_t idesc = idesc_mxf8_e4m3(kTileW, mma_n, kb & 3, kb & 3);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_mxf8(tmem_base + kAccCol, adesc + 2 * k, bdesc + 2 * k, idesc, sfw, sfw + 4, kb != kb0 || k != 0);
        tc_commit(&empty[stage]);
        if (++stage == static_cast<uint32_t>(p.stages)) { stage = 0; phase ^= 1u; }
        if ((kb & 3) == 3) {
          tc_commit(&sf_empty[slot]);
          if (++slot == kSfSlots) { slot = 0; sf_phase ^= 1u; }
        }
      }
      // commits on every way out: TMEM is released only after the issued MMAs are done
      tc_commit(acc_full);
      wait_quiet(acc_full, 0);
      if (!ok) *abort_flag = 1;
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ scale words, then the partial
    // Each of the four warps writes the same words into its own TMEM lane quadrant: column c of a
    // block holds rows lane + 32 c, byte j K-block 4 g + j.
    const int q = warp & 3;
    const uint32_t quad = tmem_base + (static_cast<uint32_t>(32 * q) << 16);
    const int ncols = (mma_n + 31) / 32;
    uint32_t slot = 0, sf_phase = 0;
    bool ok = true;
    for (int g = kb0 >> 2; g <= (kb1 - 1) >> 2; ++g) {
      uint32_t w[4], a[kMaxTok / 32];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        w[c] = static_cast<uint32_t>(__ldg(p.sfb + g * p.Np + nt * kTileW + 32 * c + lane));
#pragma unroll
      for (int c = 0; c < kMaxTok / 32; ++c) {
        const int r = tok0 + lane + 32 * c;
        a[c] = 0x7F7F7F7Fu;
        if (c < ncols && r < p.M) a[c] = static_cast<uint32_t>(__ldg(p.sfa + g * p.sfa_ld + r));
      }
      if (!wait_all(&sf_empty[slot], sf_phase ^ 1u, abort_flag, p.err)) { ok = false; break; }
      tc_fence_after();
      tmem_st_x4(quad + slot * kSfCols, w[0], w[1], w[2], w[3]);
#pragma unroll
      for (int c = 0; c < kMaxTok / 32; ++c)
        if (c < ncols) tmem_st_x1(quad + slot * kSfCols + 4 + c, a[c]);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sf_full[slot]);
      if (++slot == kSfSlots) { slot = 0; sf_phase ^= 1u; }
    }
    if (ok && wait_all(acc_full, 0, abort_flag, p.err)) {
      have = *abort_flag == 0;
      have = __all_sync(0xffffffffu, have);
      tc_fence_after();
      // partial[token][weight row]: every stage has been consumed, so their memory holds it
      float* part = reinterpret_cast<float*>(smem);
      for (int c0 = 0; have && c0 < ntok; c0 += 32) {
        uint32_t r[32];
        tmem_ld_x32(quad + kAccCol + c0, r);
        tmem_wait_ld_regs(r);
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (c0 + j < ntok) part[(c0 + j) * kTileW + 32 * q + lane] = __uint_as_float(r[j]);
      }
    }
    if (!have && lane == 0) *abort_flag = 1;
  }

  tc_fence_before();
  if (p.split > 1) cluster_sync(); else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, p.tmem_cols);
  }
  // ---------------------------------------------------------------- sum over the cluster, store
  if (*abort_flag == 0) {
    const int j0 = ntok * rank / p.split, j1 = ntok * (rank + 1) / p.split;
    const uint32_t base = smem_u32(smem);
    for (int i = threadIdx.x + j0 * 32; i < j1 * 32; i += kThreads) {
      const int j = i >> 5, c = (i & 31) * 4;
      const int n = nt * kTileW + c;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      const uint32_t at = base + (j * kTileW + c) * 4;
      for (int s = 0; s < p.split; ++s) {
        const float4 v = ld_cluster_f4(at, s);
        acc.x += v.x;
        acc.y += v.y;
        acc.z += v.z;
        acc.w += v.w;
      }
      const int64_t row = tok0 + j;
      float f[4] = {acc.x, acc.y, acc.z, acc.w};
      if (p.vec4 && n + 4 <= p.N) {
        if (p.addend) {
          const uint2 cv = *reinterpret_cast<const uint2*>(p.addend + row * p.ldc + n);
          f[0] += __uint_as_float(cv.x << 16);
          f[1] += __uint_as_float(cv.x & 0xFFFF0000u);
          f[2] += __uint_as_float(cv.y << 16);
          f[3] += __uint_as_float(cv.y & 0xFFFF0000u);
        }
        *reinterpret_cast<uint2*>(p.d + row * p.ldd + n) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
      } else {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if (n + x >= p.N) break;
          if (p.addend) f[x] += __uint_as_float(static_cast<uint32_t>(p.addend[row * p.ldc + n + x]) << 16);
          p.d[row * p.ldd + n + x] = static_cast<uint16_t>(pack_bf16x2(f[x], 0.f) & 0xFFFFu);
        }
      }
    }
  }
  // a CTA's shared memory stays until every CTA of the cluster has read it
  if (p.split > 1) cluster_sync();
}

}  // namespace
}  // namespace bsf

using namespace bsf;

extern "C" bsf_status bsf_dense_gemm(const uint8_t* a, const int32_t* sfa, int64_t sfa_ld, int64_t M,
                                     const uint8_t* b, const int32_t* sfb, int64_t N, int64_t K, const void* addend,
                                     int64_t ldc, void* d, int64_t ldd, int flags, bsf_stream_t stream) {
  if (M < 0 || N <= 0 || K <= 0 || K % 128) return BSF_ERR_INVALID_ARGUMENT;
  if (flags & ~BSF_B_TILED) return BSF_ERR_INVALID_ARGUMENT;
  if (M == 0) return BSF_OK;
  if (!a || !sfa || !b || !sfb || !d) return BSF_ERR_INVALID_ARGUMENT;
  if (sfa_ld < M || sfa_ld % 4 || ldd < N || (addend && ldc < N)) return BSF_ERR_INVALID_ARGUMENT;
  if (!aligned16(a) || !aligned16(b) || !aligned16(sfa) || !aligned16(sfb) ||
      (reinterpret_cast<uintptr_t>(d) & 1) || (reinterpret_cast<uintptr_t>(addend) & 1))
    return BSF_ERR_MISALIGNED;
  if (!fits_rows(M, K) || !fits_rows(M, ldd) || (addend && ldc > kMaxRowWidth) || N > kMaxRowWidth || sfa_ld > kMaxRows)
    return BSF_ERR_UNSUPPORTED;
  const int64_t ntn = (N + kTileW - 1) / kTileW, nkb = K / kTileK;
  if (ntn * kTileW * nkb > INT32_MAX) return BSF_ERR_UNSUPPORTED;
  const int64_t chunks = (M + kMaxTok - 1) / kMaxTok;
  const int64_t tiles = ntn * chunks;
  int* err = device_error_ptr();
  if (!err) return BSF_ERR_CUDA;
  int split = 1;
  while (split < 8 && tiles * split * 2 <= sm_count() && nkb >= split * 4) split *= 2;
  if (tiles * split > INT32_MAX) return BSF_ERR_UNSUPPORTED;

  DenseArgs p;
  p.sfa = sfa;
  p.sfa_ld = sfa_ld;
  p.sfb = sfb;
  p.Np = ntn * kTileW;
  p.addend = static_cast<const uint16_t*>(addend);
  p.ldc = ldc;
  p.d = static_cast<uint16_t*>(d);
  p.ldd = ldd;
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.nkb = static_cast<int>(nkb);
  p.nw = static_cast<int>((nkb + 3) / 4);
  p.chunks = static_cast<int>(chunks);
  p.per = static_cast<int>(((M + chunks - 1) / chunks + 15) / 16 * 16);
  // (equal chunks: the last one may be shorter; rounding up to 16 never leaves one empty)
  p.split = split;
  const int stage_bytes = kTileW * kTileK + p.per * kTileK;
  p.stages = (kSmemBytes - 1024 - kBarBytes) / stage_bytes;
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  const int cols = kAccCol + (p.per + 31) / 32 * 32;
  p.tmem_cols = cols <= 128 ? 128 : cols <= 256 ? 256 : 512;
  p.tiled = (flags & BSF_B_TILED) != 0;
  p.vec4 = (reinterpret_cast<uintptr_t>(d) & 7) == 0 && ldd % 4 == 0 &&
           (!addend || ((reinterpret_cast<uintptr_t>(addend) & 7) == 0 && ldc % 4 == 0));
  p.err = err;

  CUtensorMap map_a, map_b;
  if (!make_map(&map_a, a, M, K, p.per)) return BSF_ERR_CUDA;
  if (p.tiled ? !make_map(&map_b, b, p.Np * nkb, 128, kTileW) : !make_map(&map_b, b, p.Np, K, kTileW))
    return BSF_ERR_CUDA;
  static std::atomic<bool> attr_set[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && !attr_set[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(dense_split_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) !=
        cudaSuccess)
      return BSF_ERR_CUDA;
    attr_set[dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(split);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, dense_split_kernel, map_b, map_a, p) != cudaSuccess) {
    cudaGetLastError();
    return BSF_ERR_CUDA;
  }
  return launch_status();
}
