// Matrix product of unquantised operands with bias, activation and residual in its epilogue, sm_103a:
//
//   Y[t, n] = act( sum_k X[t, k] W[n, k] + b[n] ) + R[t, n]
//
// X and W both bf16 or both fp16, FP32 accumulation, Y in bf16, fp16 or float32.  Among others it gives the router's
// logits ("GEMM 执行方式" (rainlin-net) §4.2 takes the top-k of them as given) and the projections around an
// MoE block, added to the residual stream.
//
// As in the dense FP8 product, weights are the MMA's M = 128 rows (256 in a CTA pair) and tokens its N, and the
// forms are chosen by the time each would take (choose_plan):
//
// * Split (few tokens, or few tiles).  A tile's K is split over a cluster of 1 .. 8 CTAs, which exchange their
//   FP32 partials through distributed shared memory and add them in rank order: no atomics, no workspace, the same
//   bits every run.  Bias, activation and residual are applied to the sum, once per element; bias and residual
//   are under way before the cluster's barrier.  Bound by latency (1 x 256 x 7168 6.3 us, of which its 3.7 MB need 0.5;
//   3 x 130 x 264 takes 4.3) or, with weights from HBM, by their stream plus those 4 (37 x 7168 x 4096 15.4 us: 60 MB, 8.8).
// * Pairs (many tokens).  Two CTAs multiply 256 weight rows x up to 256 tokens with one cta_group::2 MMA per 16 K;
//   two accumulators let a tile's epilogue run under the next tile's MMAs.  What an SM takes in from L2, 53 bytes a cycle
//   (the same from its own loads and by multicast), binds these tiles: 256 x 256 x 64 brings each SM 32 KB, 610
//   cycles of loads for 512 of MMAs.  8192 x 7168 x 4096 with bias and residual takes 261-275 us in short runs, 1.75-1.84
//   PFLOP/s, 90-95 % of the measured burst, and 300-330 where the power cap holds; 8192 x 256 x 7168 (tiles of 112 tokens in
//   one round of CTAs) 30.5 us, 986 TFLOP/s; 777 x 4100 x 1416 with gelu 16.0-16.5 us.  With few K-blocks a tile is bound by
//   its epilogue: 8192 x 2048 x 512 21 us, with a residual, whose loads two warps a scheduler do not hide, 31.
#include "cluster.cuh"
#include "common.cuh"
#include "host_utils.h"
#include "tma_map.h"

#include <cuda_fp16.h>
#include <math.h>

namespace bsf {
namespace {

constexpr int kTileW = 128;                     // weight rows per tile and CTA
constexpr int kBlockK = 64;                     // K per block: rows of 128 bytes
constexpr int kRowBytes = 128;
constexpr int kMaxTok = 128;                    // split: tokens per tile
constexpr int kMaxIssuers = 2;
constexpr int kSegment = 1024;                  // values of K that a float32 output's sum takes at once (pairs: two halves)
constexpr int kThreads = 32 * (1 + kMaxIssuers + 4);   // split: loads, issuers, four warps for the accumulators
constexpr int kMaxStages = 12;
constexpr int kBarBytes = 512;
constexpr int kSmemBytes = 227 * 1024;
constexpr int kHalfSmemBytes = 112 * 1024;      // two CTAs per SM

struct Epilogue {
  const void* bias;
  const void* residual;      // of the type of y
  int64_t ldr;
  void* y;
  int64_t ldy;
  int bias_type, act;
  int wide;                  // neighbouring elements of y (and the residual) are aligned together: 4 (split), 2 (pairs)
};

struct SplitArgs {
  Epilogue e;
  int M, N, nkb;
  int chunks, per;           // token chunks per weight tile, tokens of a full chunk (multiple of 16)
  int split, stages;
  int issuers, acc_stride;   // MMA-issuing warps (a power of two), columns between accumulators
  int runs;                  // accumulators of an issuer, one after the other: its sum's parts
  uint32_t tmem_cols, idesc;
  int withhold;              // BSF_DEBUG_WITHHOLD_LOADS, in the last CTA of each cluster
  int* err;
};

__device__ __forceinline__ float load_as_float(const void* p, int64_t i, int type) {
  if (type == BSF_TYPE_F32) return __ldg(static_cast<const float*>(p) + i);
  const uint16_t v = __ldg(static_cast<const uint16_t*>(p) + i);
  return type == BSF_TYPE_BF16 ? __uint_as_float(static_cast<uint32_t>(v) << 16) : __half2float(__ushort_as_half(v));
}

// Values of OUT, two in a word where it has 16 bits.
template <int OUT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if (OUT == BSF_TYPE_BF16) return pack_bf16x2(a, b);
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <int OUT>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if (OUT == BSF_TYPE_BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
// y may be the residual itself, so the residual is read with plain loads.
template <int OUT>
__device__ __forceinline__ float residual_at(const Epilogue& e, int64_t i) {
  if (OUT == BSF_TYPE_F32) return static_cast<const float*>(e.residual)[i];
  return unpack2<OUT>(static_cast<const uint16_t*>(e.residual)[i]).x;
}
template <int OUT>
__device__ __forceinline__ void store_at(const Epilogue& e, int64_t i, float v) {
  if (OUT == BSF_TYPE_F32) static_cast<float*>(e.y)[i] = v;
  else static_cast<uint16_t*>(e.y)[i] = static_cast<uint16_t>(pack2<OUT>(v, 0.f));
}

__device__ __forceinline__ float exp2_approx(float x) {      // 2**x to 2 units in the last place (0 below 2**-126)
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// exp(x) with a rounded argument: off by |x| 2**-24 of it
__device__ __forceinline__ float exp_of(float x) { return exp2_approx(x * 1.4426950408889634f); }

// erfc(|v| / sqrt 2) / 2: with x = |v| / sqrt 2, exp(-x^2) times a polynomial in t = 1 / (1 + 0.3021286 x), a minimax
// fit (Lawson's iteration) of erfc(x) exp(x^2) on 0 .. 14 relative to it, off by 4.5e-8 with its float32 coefficients.
// erfcf would be 2.5 times as many instructions, and a tile's epilogue is not always hidden behind other tiles' products.
// In pairs: one packed instruction takes the place of two.
__device__ __forceinline__ float2 half_erfc(float a, float b) {
  const float t0 = __fdividef(1.f, fmaf(a, 0.21363720167f, 1.f)), t1 = __fdividef(1.f, fmaf(b, 0.21363720167f, 1.f));
  constexpr float c[8] = {0.17041911225827286f,  0.1713477909787805f, 0.15392502081132817f,  0.19541278265418394f,
                          -0.03962212128188006f, 0.4548883512025796f, -0.4179198212295966f, 0.4315029982598405f};
  float q0 = -0.11995414206527316f, q1 = q0;
#pragma unroll
  for (int i = 7; i >= 0; --i) {
    float d0 = c[i], d1 = c[i];
    fma2_f32(d0, d1, q0, q1, t0, t1);
    q0 = d0;
    q1 = d1;
  }
  return make_float2(0.5f * t0 * q0 * exp2_approx(a * a * -0.72134752044448170f),
                     0.5f * t1 * q1 * exp2_approx(b * b * -0.72134752044448170f));
}

// Each activation of N values, in float32 within a few units in the last place of it plus what a rounded argument of
// exp makes (relative: the tails of gelu and of the sigmoids are not differences).  A quotient by more than 2**126 is 0,
// where the exact one is below 2**-119.
template <int N>
__device__ __forceinline__ void activate(float (&v)[N], int act) {
  switch (act) {
    case BSF_ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = v[i] < 0.f ? 0.f : v[i];            // (NaN stays)
      break;
    case BSF_ACT_SILU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = __fdividef(v[i], 1.f + exp_of(-v[i]));
      break;
    case BSF_ACT_GELU:                  // max(v, 0) - |v| erfc(|v| / sqrt 2) / 2, whose second term is 0 from 20 on
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const float a = fminf(fabsf(v[i]), 20.f), b = fminf(fabsf(v[i + 1]), 20.f);
        const float2 e = half_erfc(a, b);
        v[i] = fmaf(-a, e.x, v[i] < 0.f ? 0.f : v[i]);
        v[i + 1] = fmaf(-b, e.y, v[i + 1] < 0.f ? 0.f : v[i + 1]);
      }
      break;
    case BSF_ACT_GELU_TANH:             // 0.5 v (1 + tanh(u)) = v / (1 + exp(-2 u)), u = sqrt(2 / pi) (v + 0.044715 v^3)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float u2 = v[i] * (1.5957691216057308f + 0.07135481627364643f * v[i] * v[i]);
        v[i] = __fdividef(v[i], 1.f + exp_of(-u2));
      }
      break;
    case BSF_ACT_SIGMOID:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = __fdividef(1.f, 1.f + exp_of(-v[i]));
      break;
    default:
      break;
  }
}

// Bias and residual of four weight rows of one token.
struct Beside {
  float b[4], r[4];
};
template <int OUT>
__device__ __forceinline__ Beside beside(const SplitArgs& p, int64_t row, int n) {
  const Epilogue& e = p.e;
  Beside v = {};
  if (n >= p.N) return v;
  if (e.bias) {
#pragma unroll
    for (int x = 0; x < 4; ++x) v.b[x] = load_as_float(e.bias, min(n + x, p.N - 1), e.bias_type);
  }
  if (e.residual) {
    if (e.wide && n + 4 <= p.N) {
      if (OUT == BSF_TYPE_F32) {
        const float4 r = *reinterpret_cast<const float4*>(static_cast<const float*>(e.residual) + row * e.ldr + n);
        v.r[0] = r.x, v.r[1] = r.y, v.r[2] = r.z, v.r[3] = r.w;
      } else {
        const uint2 r = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(e.residual) + row * e.ldr + n);
        const float2 a = unpack2<OUT>(r.x), b = unpack2<OUT>(r.y);
        v.r[0] = a.x, v.r[1] = a.y, v.r[2] = b.x, v.r[3] = b.y;
      }
    } else {
#pragma unroll
      for (int x = 0; x < 4; ++x) v.r[x] = residual_at<OUT>(e, row * e.ldr + min(n + x, p.N - 1));
    }
  }
  return v;
}

// The end of a CTA of a split product: once every CTA of the cluster has its partial part[token][weight row] in its
// shared memory, tokens [j0, j1) of the tile are summed over the S partials in rank order, taken through the epilogue and
// stored.  A thread takes items (token, four weight rows) and has the loads of U of them in flight; those of the first
// items' bias and residual are under way before the barrier.
template <int OUT, int S, int U>
__device__ __forceinline__ void sum_and_store(const SplitArgs& p, uint32_t part, int n0, int tok0, int j0, int j1,
                                              uint32_t tmem_base, volatile int* abort_flag) {
  auto at = [&](int i0, int u) { return min(i0 + u * kThreads, j1 * 32 - 1); };   // (past the end: the last item again)
  Beside with[U];
  const int first = threadIdx.x + j0 * 32;
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (first + u * kThreads < j1 * 32)
      with[u] = beside<OUT>(p, tok0 + (at(first, u) >> 5), n0 + (at(first, u) & 31) * 4);
  tc_fence_before();
  if (S > 1) cluster_sync(); else __syncthreads();
  if (threadIdx.x >> 5 == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, p.tmem_cols);
  }
  if (*abort_flag != 0) return;
  uint32_t base[S];
#pragma unroll
  for (int s = 0; s < S; ++s) base[s] = map_rank(part, s);
  const Epilogue& e = p.e;
  for (int i0 = first; i0 < j1 * 32; i0 += U * kThreads) {
    float4 v[U][S];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int s = 0; s < S; ++s) v[u][s] = ld_cluster_f4(base[s] + at(i0, u) * 16);
    }
    if (i0 != first) {
#pragma unroll
      for (int u = 0; u < U; ++u) with[u] = beside<OUT>(p, tok0 + (at(i0, u) >> 5), n0 + (at(i0, u) & 31) * 4);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kThreads;
      if (i >= j1 * 32) break;
      float f[4] = {v[u][0].x, v[u][0].y, v[u][0].z, v[u][0].w};
#pragma unroll
      for (int s = 1; s < S; ++s) {
        f[0] += v[u][s].x;
        f[1] += v[u][s].y;
        f[2] += v[u][s].z;
        f[3] += v[u][s].w;
      }
      const int n = n0 + (i & 31) * 4;
      if (n >= p.N) continue;
      const int64_t row = tok0 + (i >> 5);
      if (e.bias) {
#pragma unroll
        for (int x = 0; x < 4; ++x) f[x] += with[u].b[x];
      }
      activate(f, e.act);
      if (e.residual) {
#pragma unroll
        for (int x = 0; x < 4; ++x) f[x] += with[u].r[x];
      }
      if (e.wide && n + 4 <= p.N) {
        if (OUT == BSF_TYPE_F32)
          *reinterpret_cast<float4*>(static_cast<float*>(e.y) + row * e.ldy + n) = make_float4(f[0], f[1], f[2], f[3]);
        else
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(e.y) + row * e.ldy + n) =
              make_uint2(pack2<OUT>(f[0], f[1]), pack2<OUT>(f[2], f[3]));
      } else {
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (n + x < p.N) store_at<OUT>(e, row * e.ldy + n + x, f[x]);
      }
    }
  }
}

template <int OUT>
__global__ void __launch_bounds__(kThreads, 2)
    linear_split_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_x,
                        const SplitArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int stage_bytes = (kTileW + p.per) * kRowBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + p.stages * stage_bytes);
  uint64_t* empty = full + kMaxStages;
  uint64_t* acc_full = empty + kMaxStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_full + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile = blockIdx.x / p.split, rank = blockIdx.x - tile * p.split;
  const int nt = tile / p.chunks, chunk = tile - nt * p.chunks;
  const int tok0 = chunk * p.per;
  const int ntok = min(p.per, p.M - tok0);
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.nkb) * rank / p.split);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.nkb) * (rank + 1) / p.split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(acc_full, p.issuers);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmap_w);
    tma_prefetch_desc(&tmap_x);
  }
  pdl_launch_dependents();
  // Dependent launch: while the preceding kernel drains, the first stages of the weights are pulled into L2 (what
  // that kernel may still write is written in L2, too).  No global memory is loaded or stored before it has completed.
  if (threadIdx.x == 0)
    for (int kb = kb0; kb < min(kb1, kb0 + p.stages); ++kb) tma_prefetch_l2(&tmap_w, kb * kBlockK, nt * kTileW);
  pdl_wait();
  if (warp == 1) {
    tmem_alloc(tmem_slot, p.tmem_cols);
    tmem_relinquish();
  }
  __syncwarp();
  tc_fence_before();
  // (the loading warp, whose own thread initialised the barriers, does not wait for the others)
  if (warp != 0) asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
  else asm volatile("bar.arrive 1, %0;" ::"n"(kThreads) : "memory");
  tc_fence_after();
  const uint32_t tmem_base = warp != 0 ? *tmem_slot : 0u;

  bool have = false;                       // this warp may read the accumulators
  if (warp == 0) {
    // ------------------------------------------------------------ loads
    if (lane == 0) {
      uint32_t stage = 0, phase = 0;
      int issued = 0;
      for (int kb = kb0; kb < kb1 && !(p.withhold && rank == p.split - 1); ++kb) {
        if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.err)) break;
        uint8_t* dst = smem + stage * stage_bytes;
        mbar_arrive_expect_tx(&full[stage], stage_bytes);
        tma_load_2d(dst, &tmap_w, &full[stage], kb * kBlockK, nt * kTileW);
        tma_load_2d(dst + kTileW * kRowBytes, &tmap_x, &full[stage], kb * kBlockK, tok0);
        ++issued;
        if (++stage == static_cast<uint32_t>(p.stages)) { stage = 0; phase ^= 1u; }
      }
      // no TMA write may be in flight when the CTA exits or reuses its stages
      const int outstanding = min(issued, p.stages);
      for (int j = 0; j < outstanding; ++j) {
        if (stage == 0) { stage = p.stages; phase ^= 1u; }
        --stage;
        wait_quiet(&full[stage], phase);
      }
    }
    __syncwarp();
  } else if (warp <= kMaxIssuers) {
    // ------------------------------------------------------------ MMA issuers
    // Issuer i takes the K-blocks (kb - kb0) % issuers == i into an accumulator of its own: four narrow MMAs with
    // their wait and commit keep a thread busy longer than the loads of a block take.  The tensor cores cut each sum
    // off, so a long one drifts towards zero; for a float32 output it is taken in runs (issuer_runs), each in
    // columns of its own, which the epilogue adds: 2000 x 256 x 16384 is off by 2.1e-6 in one run and 9.9e-7 in these.
    const int me = warp - 1;
    if (me < p.issuers && lane == 0) {
      uint32_t d_tmem = tmem_base + me * p.runs * p.acc_stride;
      uint32_t stage = me, phase = 0;      // (stages are a multiple of issuers: a stage keeps its issuer)
      bool first = true;
      const int count = (kb1 - kb0 - me + p.issuers - 1) / p.issuers;
      int run = 0, left = count / p.runs;  // K-blocks of the run
      for (int kb = kb0 + me; kb < kb1; kb += p.issuers) {
        if (left == 0) {
          ++run;
          left = static_cast<int>(static_cast<int64_t>(count) * (run + 1) / p.runs) -
                 static_cast<int>(static_cast<int64_t>(count) * run / p.runs);
          d_tmem += p.acc_stride;
          first = true;
        }
        --left;
        if (!mbar_wait(&full[stage], phase, abort_flag, p.err)) break;
        tc_fence_after();
        const uint8_t* src = smem + stage * stage_bytes;
        const uint64_t adesc = smem_desc_k_sw128(smem_u32(src));
        const uint64_t bdesc = smem_desc_k_sw128(smem_u32(src + kTileW * kRowBytes));
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_bf16(d_tmem, adesc + 2 * k, bdesc + 2 * k, p.idesc, !first || k != 0);
        first = false;
        tc_commit(&empty[stage]);
        stage += p.issuers;
        if (stage >= static_cast<uint32_t>(p.stages)) { stage -= p.stages; phase ^= 1u; }
      }
      // commits on every way out: TMEM is released only after the issued MMAs are done
      tc_commit(acc_full);
      wait_quiet(acc_full, 0);
    }
    __syncwarp();
  } else {
    have = wait_all(acc_full, 0, abort_flag, p.err) && *abort_flag == 0;
    have = __all_sync(0xffffffffu, have);
    tc_fence_after();
    // A wait that ran out anywhere in this CTA ends here, and keeps all of its cluster from storing.
    if (!have) {
      if (lane == 0)
        for (int s = 0; s < p.split; ++s) st_cluster_u32(map_rank(smem_u32(const_cast<int*>(abort_flag)), s), 1u);
      __syncwarp();
    }
  }

  // ---------------------------------------------------------------- partial to shared memory, sum, store
  // part[token][weight row] takes the place of the stages, which have all been consumed.
  if (have) {
    const int q = warp & 3;
    const uint32_t quad = tmem_base + (static_cast<uint32_t>(32 * q) << 16);
    float* part = reinterpret_cast<float*>(smem) + 32 * q + lane;
    const int accumulators = p.issuers * p.runs;
    for (int c0 = 0; c0 < ntok; c0 += 32) {      // (whole chunks: the rows past ntok are not read)
      uint32_t r[32], o[32];
      tmem_ld_x32(quad + c0, r);
      if (accumulators > 1) tmem_ld_x32(quad + p.acc_stride + c0, o);
      tmem_wait_ld_regs(r);
      for (int a = 1; a < accumulators; ++a) {
        if (a > 1) tmem_ld_x32(quad + a * p.acc_stride + c0, o);
        tmem_wait_ld_regs(o);
#pragma unroll
        for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) + __uint_as_float(o[j]));
      }
#pragma unroll
      for (int j = 0; j < 32; ++j) part[(c0 + j) * kTileW] = __uint_as_float(r[j]);
    }
  }
  const int j0 = ntok * rank / p.split, j1 = ntok * (rank + 1) / p.split, n0 = nt * kTileW;
  const uint32_t part = smem_u32(smem);
  switch (p.split) {
    case 1: sum_and_store<OUT, 1, 4>(p, part, n0, tok0, j0, j1, tmem_base, abort_flag); break;
    case 2: sum_and_store<OUT, 2, 4>(p, part, n0, tok0, j0, j1, tmem_base, abort_flag); break;
    case 3: sum_and_store<OUT, 3, 2>(p, part, n0, tok0, j0, j1, tmem_base, abort_flag); break;
    case 4: sum_and_store<OUT, 4, 2>(p, part, n0, tok0, j0, j1, tmem_base, abort_flag); break;
    case 5: sum_and_store<OUT, 5, 1>(p, part, n0, tok0, j0, j1, tmem_base, abort_flag); break;
    case 6: sum_and_store<OUT, 6, 1>(p, part, n0, tok0, j0, j1, tmem_base, abort_flag); break;
    case 7: sum_and_store<OUT, 7, 1>(p, part, n0, tok0, j0, j1, tmem_base, abort_flag); break;
    default: sum_and_store<OUT, 8, 1>(p, part, n0, tok0, j0, j1, tmem_base, abort_flag); break;
  }
  // a CTA's shared memory stays until every CTA of the cluster has read it
  if (p.split > 1) cluster_sync();
}

// ---------------------------------------------------------------- CTA pairs: 256 x up to 256 output tiles
constexpr int kPairW = 256;                                // weight rows of a tile (MMA M), 128 per CTA
constexpr int kPairMaxTok = 256;                           // tokens of a tile (MMA N), half staged by each CTA
constexpr int kPairMaxStages = 8;                          // a stage is one or two K-blocks of both operands
// warps: 0 loads, 1 waiter, 2 second MMA issuer (narrow tiles), 3 MMA issuer, 4-11 epilogue
constexpr int kPairWaiter = 1, kPairIssuer2 = 2, kPairIssuer = 3, kPairThreads = 384;
constexpr int kPairBarBytes = 256;

struct PairArgs {
  Epilogue e;
  int M, N, nkb;
  int tiles_m, tiles_n;      // token tiles, weight tiles
  int tok, acc_cols;         // tokens of a tile (a multiple of 16); columns of an accumulator
  int stages, blocks;        // stages, K-blocks in one (2: the barriers of narrow tiles cost as much as their MMAs)
  int nst, segments;         // stages of a tile; runs of them with a sum of their own
  uint32_t idesc;
  int withhold;
  int* err;
};

// Executed by the whole warp, issued by the lane whose `lead` is non-zero.
__device__ __forceinline__ void pair_mma_f16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}

// One past the last stage of segment i.
__device__ __forceinline__ int segment_end(const PairArgs& p, int i) {
  return static_cast<int>(static_cast<int64_t>(p.nst) * (i + 1) / p.segments);
}

// The residual of 32 tokens of one weight row per lane, as finish() takes it: with 16-bit types and aligned rows 16 words
// of two neighbouring rows, of the tokens that the lane will have then, otherwise one value a token.
template <int OUT, bool kResidual>
__device__ __forceinline__ void fetch(const Epilogue& e, uint32_t (&w)[32], int64_t row, int rows, int n, int N) {
  if (!kResidual || rows <= 0 || n >= N) return;
  if (OUT == BSF_TYPE_F32 || !e.wide) {
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const int64_t i = (row + min(j, rows - 1)) * e.ldr + n;
      if (OUT == BSF_TYPE_F32) w[j] = static_cast<const uint32_t*>(e.residual)[i];
      else w[j] = static_cast<const uint16_t*>(e.residual)[i];
    }
    return;
  }
  const int odd = n & 1;
  const uint16_t* from = static_cast<const uint16_t*>(e.residual) + row * e.ldr + (n & ~1);
  if (rows >= 32) {
    from += odd * e.ldr;
#pragma unroll
    for (int j = 0; j < 16; ++j, from += 2 * e.ldr) w[j] = *reinterpret_cast<const uint32_t*>(from);
    return;
  }
#pragma unroll
  for (int j = 0; j < 16; ++j) w[j] = *reinterpret_cast<const uint32_t*>(from + min(2 * j + odd, rows - 1) * e.ldr);
}

// 32 tokens of one weight row per lane -> y.  With 16-bit types two tokens are packed in a word and neighbouring lanes
// exchange words, so that a lane holds two neighbouring rows of one token (one exchange and one byte permutation for two
// values; the residual's words go the other way).  The epilogue's warps are few, two a scheduler, so their instructions
// count: full chunks have no predicates, and rows are stepped through, not multiplied out.
template <int OUT, bool kResidual>
__device__ __forceinline__ void finish(const Epilogue& e, float (&v)[32], const uint32_t (&w)[32], float bias, int64_t row,
                                       int rows, int n, int N) {
  const int odd = n & 1;
  if (e.bias) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] += bias;
  }
  activate(v, e.act);
  if (OUT == BSF_TYPE_F32 || !e.wide) {
    if (n >= N) return;
    if (kResidual) {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] += OUT == BSF_TYPE_F32 ? __uint_as_float(w[j]) : unpack2<OUT>(w[j]).x;
    }
    Epilogue at = e;
    if (OUT == BSF_TYPE_F32) at.y = static_cast<float*>(e.y) + row * e.ldy + n;
    else at.y = static_cast<uint16_t*>(e.y) + row * e.ldy + n;
    if (rows >= 32) {
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        store_at<OUT>(at, 0, v[j]);
        if (OUT == BSF_TYPE_F32) at.y = static_cast<float*>(at.y) + e.ldy;
        else at.y = static_cast<uint16_t*>(at.y) + e.ldy;
      }
      return;
    }
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < rows) store_at<OUT>(at, j * e.ldy, v[j]);
    return;
  }
  // (N is even, so both rows of a word exist or neither does)
  const uint32_t pick = odd ? 0x3276u : 0x5410u;
  uint32_t u[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    float v0 = v[2 * j], v1 = v[2 * j + 1];
    if (kResidual) {
      const float2 r = unpack2<OUT>(__byte_perm(w[j], __shfl_xor_sync(0xffffffffu, w[j], 1), pick));
      v0 += r.x;
      v1 += r.y;
    }
    u[j] = pack2<OUT>(v0, v1);
  }
#pragma unroll
  for (int j = 0; j < 16; ++j) u[j] = __byte_perm(u[j], __shfl_xor_sync(0xffffffffu, u[j], 1), pick);
  if (n >= N) return;
  uint16_t* to = static_cast<uint16_t*>(e.y) + (row + odd) * e.ldy + (n & ~1);
  const int64_t step = 2 * e.ldy;
  if (rows >= 32) {
#pragma unroll
    for (int j = 0; j < 16; ++j, to += step) *reinterpret_cast<uint32_t*>(to) = u[j];
    return;
  }
#pragma unroll
  for (int j = 0; j < 16; ++j, to += step)
    if (2 * j + odd < rows) *reinterpret_cast<uint32_t*>(to) = u[j];
}

template <int OUT, int kIssuers, bool kResidual>
__global__ void __launch_bounds__(kPairThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_x,
                       const PairArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int half_tok = p.tok >> 1;
  // a stage: 128 weight rows of its K-blocks, then half of the tile's tokens of the same
  const int tok_bytes = half_tok * kRowBytes;
  const int stage_bytes = p.blocks * (kTileW * kRowBytes + tok_bytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + p.stages * stage_bytes);          // used in rank 0
  uint64_t* empty = full + kPairMaxStages;
  uint64_t* acc_full = empty + kPairMaxStages;
  uint64_t* acc_empty = acc_full + 2;                                                   // used in rank 0
  uint64_t* mma_done = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int total = p.tiles_m * p.tiles_n;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&acc_full[s], kIssuers);
      mbar_init(&acc_empty[s], 16);
    }
    mbar_init(mma_done, kIssuers);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmap_w);
    tma_prefetch_desc(&tmap_x);
  }
  pdl_launch_dependents();
  pdl_wait();
  if (warp == kPairIssuer) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();                           // barriers of both CTAs are initialised
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t set_cols = kIssuers * p.acc_cols;          // of a set of accumulators, one per issuer

  if (warp == 0) {
    // ------------------------------------------------------------ loads (each CTA its halves)
    // (where a stage is two K-blocks and K has an odd number the last one's second half is zeros, and not multiplied)
    if (lane == 0) {
      uint32_t stage = 0, phase = 0;
      int issued = 0;
      bool ok = !p.withhold;
      for (int t = pair; t < total && ok; t += npairs) {
        const int tm = t % p.tiles_m, tn = t / p.tiles_m;
        const int w_row = (tn * 2 + static_cast<int>(rank)) * kTileW, x_row = tm * p.tok + static_cast<int>(rank) * half_tok;
        for (int kb = 0; kb < p.nkb; kb += p.blocks) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.err)) { ok = false; break; }
          const uint32_t bar = map_rank(smem_u32(&full[stage]), 0);
          uint8_t* dst = smem + stage * stage_bytes;
          uint8_t* tok_dst = dst + p.blocks * kTileW * kRowBytes;
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * stage_bytes);   // both CTAs, both operands
          pair_load_2d(dst, &tmap_w, bar, kb * kBlockK, w_row);
          pair_load_2d(tok_dst, &tmap_x, bar, kb * kBlockK, x_row);
          if (p.blocks == 2) {
            pair_load_2d(dst + kTileW * kRowBytes, &tmap_w, bar, (kb + 1) * kBlockK, w_row);
            pair_load_2d(tok_dst + tok_bytes, &tmap_x, bar, (kb + 1) * kBlockK, x_row);
          }
          ++issued;
          if (++stage == static_cast<uint32_t>(p.stages)) { stage = 0; phase ^= 1u; }
        }
      }
      if (rank == 0) {
        // both CTAs' loads complete on these barriers; rank 1 waits for rank 0 at the last cluster barrier
        const int outstanding = min(issued, p.stages);
        for (int j = 0; j < outstanding; ++j) {
          if (stage == 0) { stage = p.stages; phase ^= 1u; }
          --stage;
          wait_quiet(&full[stage], phase);
        }
      }
    }
    __syncwarp();
  } else if (warp == kPairIssuer || (kIssuers == 2 && warp == kPairIssuer2)) {
    // ------------------------------------------------------------ MMA issuers (rank 0)
    // An issuing thread reads no shared memory between stages: the waiter warp does every wait and hands each stage
    // over through a named barrier whose OR-reduced predicate carries an abort.  With two issuers the stages of
    // a tile go to them in turn, each into an accumulator of its own (narrow tiles are bound by the issue of MMAs).
    const int me = warp == kPairIssuer ? 0 : 1;
    if (rank == 0) {
      const uint32_t lead = lane == 0;
      uint32_t stage = 0, acc = 0;                     // stage: of the tile's next K-blocks, whoever takes them
      bool ok = true;
      for (int t = pair; t < total && ok; t += npairs) {
        uint32_t first = 1;
        int segment = 0, end = segment_end(p, 0);
        for (int st = 0; st < p.nst; ++st) {
          if (OUT == BSF_TYPE_F32 && st == end) {
            pair_commit(&acc_full[acc], lead);
            acc ^= 1u;
            first = 1;
            end = segment_end(p, ++segment);
          }
          if (kIssuers == 1 || (st & 1) == me) {
            if (named_barrier_or(1 + me, 64, false)) { ok = false; break; }
            tc_fence_after();
            const uint32_t d_tmem = tmem_base + acc * set_cols + me * p.acc_cols;
            const uint8_t* src = smem + stage * stage_bytes;
            uint64_t adesc = smem_desc_k_sw128(smem_u32(src));
            uint64_t bdesc = smem_desc_k_sw128(smem_u32(src + p.blocks * kTileW * kRowBytes));
#pragma unroll
            for (int k = 0; k < 4; ++k)
              pair_mma_f16(d_tmem, adesc + 2 * k, bdesc + 2 * k, p.idesc, k == 0 ? first ^ 1u : 1u, lead);
            first = 0;
            if (p.blocks == 2 && 2 * st + 1 < p.nkb) {
              adesc += kTileW * kRowBytes >> 4;
              bdesc += tok_bytes >> 4;
#pragma unroll
              for (int k = 0; k < 4; ++k) pair_mma_f16(d_tmem, adesc + 2 * k, bdesc + 2 * k, p.idesc, 1, lead);
            }
            pair_commit(&empty[stage], lead);
          }
          if (++stage == static_cast<uint32_t>(p.stages)) stage = 0;
        }
        if (!ok) break;
        pair_commit(&acc_full[acc], lead);
        acc ^= 1u;
      }
      pair_commit(mma_done, lead);
      if (lane == 0) wait_quiet(mma_done, 0);
    }
    __syncwarp();
  } else if (warp == kPairWaiter) {
    // ------------------------------------------------------------ waiter (rank 0): the issuers' waits, in their order
    if (rank == 0) {
      uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
      bool good = true;
      int t = pair, st = 0;
      while (t < total) {
        int segment = 0, end = 0;
        for (st = 0; st < p.nst; ++st) {
          if (st == end) {
            good = wait_cluster_all(&acc_empty[acc], acc_phase ^ 1u, abort_flag, p.err);
            if ((acc ^= 1u) == 0u) acc_phase ^= 1u;
            end = segment_end(p, segment++);
          }
          if (good) good = wait_all(&full[stage], phase, abort_flag, p.err);
          if (!good) break;
          named_barrier_or(kIssuers == 1 ? 1 : 1 + (st & 1), 64, false);
          if (++stage == static_cast<uint32_t>(p.stages)) { stage = 0; phase ^= 1u; }
        }
        if (!good) break;
        t += npairs;
      }
      if (!good) {
        // the issuer of this stage is at its barrier or on its way to it, and so is the other one if any later
        // stage is its own (with two issuers every tile has stages of both)
        const int me = kIssuers == 1 ? 0 : st & 1;
        named_barrier_or(1 + me, 64, true);
        if (kIssuers == 2 && (st + 1 < p.nst || t + npairs < total)) named_barrier_or(2 - me, 64, true);
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue: lane = weight row, 32 tokens at a time
    // two warps share a quadrant's tokens
    const int q = warp & 3, ew = warp - 4;
    const int nc = (p.tok + 31) >> 5, c_first = ew < 4 ? 0 : (nc + 1) >> 1, c_last = ew < 4 ? (nc + 1) >> 1 : nc;
    uint32_t acc = 0, acc_phase = 0;
    for (int t = pair; t < total; t += npairs) {
      const int tm = t % p.tiles_m, tn = t / p.tiles_m;
      const int n = tn * kPairW + static_cast<int>(rank) * kTileW + 32 * q + lane;
      const int64_t tok0 = static_cast<int64_t>(tm) * p.tok;
      const int rows = min(p.tok, p.M - static_cast<int>(tok0));
      const float bias = p.e.bias && n < p.N ? load_as_float(p.e.bias, n, p.e.bias_type) : 0.f;
      uint32_t w[32];                       // the residual, in flight while the products run
      fetch<OUT, kResidual>(p.e, w, tok0 + 32 * c_first, rows - 32 * c_first, n, p.N);
      bool ok = wait_all(&acc_full[acc], acc_phase, abort_flag, p.err);
      if (!ok) break;
      tc_fence_after();
      const uint32_t quad = tmem_base + (static_cast<uint32_t>(32 * q) << 16);
      if constexpr (OUT == BSF_TYPE_F32) {
        // The tensor core cuts the running sum off rather than rounding it, so an error grows with the number of terms
        // (8192 x 256 x 7168 in one sum per issuer: 3.8e-6 of the result); sums of kSegment values are added here.
        float v[2][32] = {};
        for (int s = 0; ok && s < p.segments; ++s) {
          if (s > 0) ok = wait_all(&acc_full[acc], acc_phase, abort_flag, p.err);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (c_first + i >= c_last) break;
#pragma unroll
            for (int b = 0; b < kIssuers; ++b) {
              uint32_t r[32];
              tmem_ld_x32(quad + acc * set_cols + b * p.acc_cols + 32 * (c_first + i), r);
              tmem_wait_ld_regs(r);
#pragma unroll
              for (int j = 0; j < 32; ++j) v[i][j] += __uint_as_float(r[j]);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_cluster(map_rank(smem_u32(&acc_empty[acc]), 0));
          if ((acc ^= 1u) == 0u) acc_phase ^= 1u;
        }
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int c = 32 * (c_first + i);
          if (c_first + i >= c_last || c >= rows) break;
          if (i > 0) fetch<OUT, kResidual>(p.e, w, tok0 + c, rows - c, n, p.N);
          finish<OUT, kResidual>(p.e, v[i], w, bias, tok0 + c, min(32, rows - c), n, p.N);
        }
      } else {
        // (16-bit outputs take all of K in the accumulators of the issuers: what they cut off is far below the rounding.
        // 1024 x 2048 x 4096 in bf16: 0.12 % of the outputs are not the one nearest to the exact result, 0.22 % with a
        // library bf16 product, 0.035 % with a rounded float32 one; runs would take 128 registers for their sums)
        const uint32_t taddr = quad + acc * set_cols;
        for (int c = c_first; c < c_last; ++c) {
          uint32_t r[32];
          float v[32];
          tmem_ld_x32(taddr + 32 * c, r);
          tmem_wait_ld_regs(r);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
          if (kIssuers == 2) {
            tmem_ld_x32(taddr + p.acc_cols + 32 * c, r);
            tmem_wait_ld_regs(r);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] += __uint_as_float(r[j]);
          }
          if (c == c_last - 1) {              // the accumulator's last columns are in registers
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_cluster(map_rank(smem_u32(&acc_empty[acc]), 0));
          }
          if (32 * c < rows) {
            uint32_t now[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) now[j] = w[j];
            if (c + 1 < c_last) fetch<OUT, kResidual>(p.e, w, tok0 + 32 * (c + 1), rows - 32 * (c + 1), n, p.N);
            finish<OUT, kResidual>(p.e, v, now, bias, tok0 + 32 * c, min(32, rows - 32 * c), n, p.N);
          }
        }
        if ((acc ^= 1u) == 0u) acc_phase ^= 1u;
      }
    }
    // the issuers' last commits have reached this CTA's barriers too, so none arrives after it exits
    if (warp == 4 && lane == 0) wait_quiet(mma_done, 0);
    __syncwarp();
  }

  tc_fence_before();
  cluster_sync();                           // no load, MMA or remote arrival of the pair is outstanding
  if (warp == kPairIssuer) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(512) : "memory");
  }
}

// 2-D tensor of 16-bit elements [rows, cols] (row pitch ld elements), box {64 cols, box_rows}, 128-byte swizzle; what
// lies past the edges reads as zeros.
bool make_map_16(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t ld, uint32_t box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t box[2] = {kBlockK, box_rows};
  const cuuint32_t estr[2] = {1u, 1u};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// kind::f16, FP32 accumulator, both operands of the same type (0 fp16, 1 bf16), K-major
uint32_t idesc_16(bool bf16, int m, int n) {
  const uint32_t type = bf16 ? 1u : 0u;
  return 1u << 4 | type << 7 | type << 10 | static_cast<uint32_t>(n >> 3) << 17 | static_cast<uint32_t>(m >> 4) << 24;
}

template <int OUT>
const void* kernel_of(int form) {                  // 0 split; 1 and 2 pairs with so many issuers, 3 and 4 with a residual
  switch (form) {
    case 0: return reinterpret_cast<const void*>(linear_split_kernel<OUT>);
    case 1: return reinterpret_cast<const void*>(linear_pair_kernel<OUT, 1, false>);
    case 2: return reinterpret_cast<const void*>(linear_pair_kernel<OUT, 2, false>);
    case 3: return reinterpret_cast<const void*>(linear_pair_kernel<OUT, 1, true>);
    default: return reinterpret_cast<const void*>(linear_pair_kernel<OUT, 2, true>);
  }
}
const void* kernel_of(int out, int form) {
  return out == BSF_TYPE_F32    ? kernel_of<BSF_TYPE_F32>(form)
         : out == BSF_TYPE_BF16 ? kernel_of<BSF_TYPE_BF16>(form)
                                : kernel_of<BSF_TYPE_F16>(form);
}

// Once per device: all kernels may use all shared memory, and the number of CTAs of the split kernel that run at
// once, one per SM, in clusters of 1 .. kMaxSplit (a cluster lives in one GPC, so some sizes leave SMs idle).
constexpr int kMaxSplit = 8;
struct LinearLimits {
  std::atomic<int> ctas[kMaxSplit + 1];
  std::atomic<bool> ready;
};
bsf_status linear_limits(const LinearLimits** out) {
  static LinearLimits limits[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return BSF_ERR_CUDA;
  LinearLimits& l = limits[dev];
  if (!l.ready.load(std::memory_order_acquire)) {      // (racing first calls store the same values)
    for (int type : {BSF_TYPE_F32, BSF_TYPE_BF16, BSF_TYPE_F16})
      for (int form = 0; form < 5; ++form) {
        const void* k = kernel_of(type, form);
        if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) != cudaSuccess ||
            cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) !=
                cudaSuccess)
          return BSF_ERR_CUDA;
      }
    for (int i = 1; i <= kMaxSplit; ++i) {
      DependentLaunch launch(8u * i, kThreads, kSmemBytes, nullptr, i);
      launch.cfg.numAttrs = 1;                           // the cluster alone
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, kernel_of(BSF_TYPE_F32, 0), &launch.cfg) != cudaSuccess || n <= 0) {
        cudaGetLastError();
        return BSF_ERR_CUDA;
      }
      l.ctas[i].store(n * i, std::memory_order_relaxed);
    }
    l.ready.store(true, std::memory_order_release);
  }
  *out = &l;
  return BSF_OK;
}

// Split: the issuers of a CTA, and the accumulators that each needs for runs of kSegment values of a float32 output's
// sum.  TMEM holds 256 columns for each of two CTAs of an SM, 512 for one alone.
int split_issuers(int64_t nkb, int split) { return nkb / split >= kMaxIssuers ? kMaxIssuers : 1; }
int issuer_runs(int64_t nkb, int split, bool f32) {
  const int64_t count = ((nkb + split - 1) / split + split_issuers(nkb, split) - 1) / split_issuers(nkb, split);
  const int64_t runs = f32 ? (count * kBlockK + kSegment - 1) / kSegment : 1;
  return static_cast<int>(runs < 1024 ? runs : 1024);
}
int acc_columns(int64_t per) { return static_cast<int>((per + 31) / 32 * 32); }
bool runs_fit(int64_t nkb, int split, int64_t per, bool f32) {
  return split_issuers(nkb, split) * issuer_runs(nkb, split, f32) * acc_columns(per) <= (per <= 64 ? 256 : 512);
}

// Which kernel a product takes, by the time each would need (nanoseconds).  The constants are fitted to 2200 products
// of 1 .. 8192 tokens, 16 .. 8192 weight rows and K of 64 .. 8192, drawn by their logarithms, with weights that come from
// HBM, each timed in every form that could win (25000 in all), none of them with an activation.  On 1500 others the choice is
// 1.0 % above the best form on average, at worst 18 %; on 9700 with gelu, silu or gelu_tanh 0.9 %, at worst 33 %
// (7592 x 812 x 72 with residual, float32, gelu: 30.1 us in tiles of 80 tokens, 22.7 of 64).  It ranks forms; it is not
// a clock: where the epilogue binds, all forms take up to twice what it says (777 x 4100 x 1416 with gelu 16 us, not
// 10.5; 8192 x 2048 x 512 with residual 31, not 14.4).  Both sides: 64 x 4096 x 4096 takes 12.2 us split and 14.7 in pairs, 256 x 4096 x 4096
// 16.6 and 14.3, 1024 x 256 x 7168 10.9 and 21.0, 777 x 4100 x 1416 33.5 and 13.0.
struct Plan {
  bool pair;
  int tok;                  // pairs: tokens per tile; split: most tokens per tile
  int split;
};
Plan choose_plan(int64_t M, int64_t N, int64_t K, bool f32, bool residual, const LinearLimits& limits) {
  const int64_t nkb = (K + kBlockK - 1) / kBlockK, ntn = (N + kTileW - 1) / kTileW, sms = sm_count(), pairs = sms / 2;
  const double read = 2.0 * K * (M + N) / 8895;        // of both operands from HBM
  Plan best = {false, 64, 1};
  double least = 1e300;
  for (int tok = 64; tok <= kMaxTok; tok += 64) {
    if (tok > 64 && M <= 64) break;
    const int64_t chunks = (M + tok - 1) / tok, per = ((M + chunks - 1) / chunks + 15) / 16 * 16;
    for (int split = 1; split <= kMaxSplit; ++split) {
      const int64_t ctas = ntn * chunks * split, kbs = (nkb + split - 1) / split;
      if (split > 1 && (nkb < 2 * split || ctas > 2 * sms)) break;
      if (!runs_fit(nkb, split, per, f32)) continue;                  // (pairs add runs of any number)
      const int64_t at_once = limits.ctas[split].load(std::memory_order_relaxed);
      const int64_t load = (ctas + at_once - 1) / at_once;            // CTAs of the busiest SM
      const double once = (residual ? 88.4 : 76.4) * per / sqrt(double(split)) + (split > 1 ? 734 + 138 * split : 0);
      // tiles of more than 64 tokens have an SM to themselves, others share one two at a time
      const double busy = per > 64 ? load * (once + 270.0 * kbs)
                                   : load / 2 * (once + 730.0 * kbs) + load % 2 * (once + 293.0 * kbs);
      const double ns = 1498 + (busy > read ? busy : read);
      if (ns < least) {
        least = ns;
        best = {false, tok, split};
      }
    }
  }
  for (int tok = f32 ? kMaxTok : kPairMaxTok; tok >= 64; tok -= 16) {      // (float32 sums live in registers)
    const int64_t tiles = (M + tok - 1) / tok * ((ntn + 1) / 2), waves = (tiles + pairs - 1) / pairs;
    // a K-block: what an SM takes from L2, 53 bytes a cycle, binds every tile (wide ones nearly the tensor cores, too)
    const double loop = tok <= kMaxTok ? (nkb + 1) / 2 * 2 * (152 + 0.682 * tok) : 290.0 * nkb;
    const double store = tok * (2.53 + (f32 ? 4.8 : 0) + (residual ? 4.17 : 0));
    const double busy = waves * (loop > 891 + store ? loop : 891 + store);
    const double ns = 3301 + (busy > read ? busy : read) + store;
    if (ns < least) {
      least = ns;
      best = {true, tok, 1};
    }
  }
  return best;
}

// Tokens of a split tile: equal chunks (the last may be shorter, never empty: (chunks - 1) * per <= (chunks - 1) * tok < T).
int64_t tokens_per_chunk(int64_t T, int64_t chunks) { return ((T + chunks - 1) / chunks + 15) / 16 * 16; }

size_t size_of(int type) { return type == BSF_TYPE_F32 ? 4 : 2; }
bool known(int type) { return type == BSF_TYPE_F32 || type == BSF_TYPE_BF16 || type == BSF_TYPE_F16; }

}  // namespace
}  // namespace bsf

using namespace bsf;

extern "C" bsf_status bsf_linear_form(int64_t T, int64_t N, int64_t K, int y_type, int residual, int64_t* form) {
  if (T <= 0 || N <= 0 || K <= 0 || !known(y_type) || !form) return BSF_ERR_INVALID_ARGUMENT;
  if (!fits_rows(T, N) || K > kMaxRowWidth || T > kMaxRows - 256) return BSF_ERR_UNSUPPORTED;
  const LinearLimits* limits;
  const bsf_status st = linear_limits(&limits);
  if (st != BSF_OK) return st;
  const Plan plan = choose_plan(T, N, K, y_type == BSF_TYPE_F32, residual != 0, *limits);
  const int64_t ntn = (N + kTileW - 1) / kTileW, chunks = (T + plan.tok - 1) / plan.tok;
  form[0] = plan.pair;
  form[1] = plan.pair ? plan.tok : tokens_per_chunk(T, chunks);
  form[2] = plan.split;
  form[3] = chunks * (plan.pair ? (ntn + 1) / 2 : ntn);
  return BSF_OK;
}

extern "C" bsf_status bsf_linear(const void* x, int type, int64_t T, int64_t K, int64_t ldx, const void* w, int64_t N,
                                 int64_t ldw, const void* bias, int bias_type, int activation, const void* residual,
                                 int64_t ldr, void* y, int y_type, int64_t ldy, int flags, bsf_stream_t stream) {
  if (T < 0 || N <= 0 || K <= 0) return BSF_ERR_INVALID_ARGUMENT;
  if ((type != BSF_TYPE_BF16 && type != BSF_TYPE_F16) || !known(y_type) || (bias && !known(bias_type)))
    return BSF_ERR_INVALID_ARGUMENT;
  if (activation < BSF_ACT_NONE || activation > BSF_ACT_SIGMOID) return BSF_ERR_INVALID_ARGUMENT;
  if (flags & ~BSF_DEBUG_WITHHOLD_LOADS) return BSF_ERR_INVALID_ARGUMENT;
  if (T == 0) return BSF_OK;
  if (!x || !w || !y) return BSF_ERR_INVALID_ARGUMENT;
  if (ldx < K || ldw < K || ldy < N || (residual && ldr < N)) return BSF_ERR_INVALID_ARGUMENT;
  const size_t ysize = size_of(y_type);
  if (!aligned16(x) || !aligned16(w) || ldx % 8 || ldw % 8 || reinterpret_cast<uintptr_t>(y) % ysize ||
      reinterpret_cast<uintptr_t>(residual) % ysize || (bias && reinterpret_cast<uintptr_t>(bias) % size_of(bias_type)))
    return BSF_ERR_MISALIGNED;
  if (!fits_rows(T, ldx) || !fits_rows(T, ldy) || (residual && ldr > kMaxRowWidth) || N > kMaxRowWidth ||
      ldw > kMaxRowWidth || T > kMaxRows - 256)
    return BSF_ERR_UNSUPPORTED;
  const int64_t ntn = (N + kTileW - 1) / kTileW, nkb = (K + kBlockK - 1) / kBlockK;
  int* err = device_error_ptr();
  if (!err) return BSF_ERR_CUDA;
  const bool withhold = (flags & BSF_DEBUG_WITHHOLD_LOADS) != 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const LinearLimits* limits;
  const bsf_status st = linear_limits(&limits);
  if (st != BSF_OK) return st;
  const Plan plan = choose_plan(T, N, K, y_type == BSF_TYPE_F32, residual != nullptr, *limits);
  Epilogue e;
  e.bias = bias;
  e.residual = residual;
  e.ldr = ldr;
  e.y = y;
  e.ldy = ldy;
  e.bias_type = bias_type;
  e.act = activation;
  const int64_t group = plan.pair ? 2 : 4;             // elements stored together
  e.wide = reinterpret_cast<uintptr_t>(y) % (group * ysize) == 0 && ldy % group == 0 &&
           (!residual || (reinterpret_cast<uintptr_t>(residual) % (group * ysize) == 0 && ldr % group == 0)) &&
           (!plan.pair || N % 2 == 0);
  CUtensorMap map_w, map_x;
  if (!make_map_16(&map_w, w, N, K, ldw, kTileW)) return BSF_ERR_CUDA;

  if (plan.pair) {
    const int tok = plan.tok;
    const int64_t tiles_m = (T + tok - 1) / tok, tiles_n = (ntn + 1) / 2, tiles = tiles_m * tiles_n;
    if (tiles > INT32_MAX) return BSF_ERR_UNSUPPORTED;
    PairArgs p;
    p.e = e;
    p.M = static_cast<int>(T);
    p.N = static_cast<int>(N);
    p.nkb = static_cast<int>(nkb);
    p.tiles_m = static_cast<int>(tiles_m);
    p.tiles_n = static_cast<int>(tiles_n);
    p.tok = tok;
    p.acc_cols = (tok + 31) / 32 * 32;
    // (each issuer needs a stage of every tile)
    const int issuers = tok <= kMaxTok && nkb > 2 ? 2 : 1;
    // (two sets of accumulators: 2 x 2 x 128 or 2 x 256 columns)
    p.blocks = issuers == 2 ? 2 : 1;
    p.nst = static_cast<int>((nkb + p.blocks - 1) / p.blocks);
    p.segments = y_type == BSF_TYPE_F32 ? (p.nst * p.blocks * kBlockK + kSegment - 1) / kSegment : 1;
    p.idesc = idesc_16(type == BSF_TYPE_BF16, kPairW, tok);
    p.withhold = withhold;
    p.err = err;
    const int stage_bytes = p.blocks * (kTileW + tok / 2) * kRowBytes;
    p.stages = (kSmemBytes - 1024 - kPairBarBytes) / stage_bytes;
    if (p.stages > kPairMaxStages) p.stages = kPairMaxStages;
    if (!make_map_16(&map_x, x, T, K, ldx, tok / 2)) return BSF_ERR_CUDA;
    const int64_t pairs = sm_count() / 2, used = tiles < pairs ? tiles : pairs;
    void* args[] = {&map_w, &map_x, &p};
    return launch_cluster(kernel_of(y_type, issuers + (residual ? 2 : 0)), static_cast<unsigned>(2 * used), kPairThreads, kSmemBytes, 2, s,
                          args);
  }

  const int64_t chunks = (T + plan.tok - 1) / plan.tok, tiles = ntn * chunks;
  if (tiles * plan.split > INT32_MAX) return BSF_ERR_UNSUPPORTED;
  SplitArgs p;
  p.e = e;
  p.M = static_cast<int>(T);
  p.N = static_cast<int>(N);
  p.nkb = static_cast<int>(nkb);
  p.chunks = static_cast<int>(chunks);
  p.per = static_cast<int>(tokens_per_chunk(T, chunks));
  p.split = plan.split;
  const int stage_bytes = (kTileW + p.per) * kRowBytes;
  const size_t smem = p.per <= 64 ? kHalfSmemBytes : kSmemBytes;
  p.stages = (static_cast<int>(smem) - 1024 - kBarBytes) / stage_bytes;
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  p.acc_stride = acc_columns(p.per);
  // (an issuer or a run without a K-block would leave its accumulator unwritten.  The K-blocks of two issuers, of one CTA or
  // of two, differ by at most 1, and runs = ceil(most / 16), so where there are several runs an issuer has at least
  // 16 (runs - 1) K-blocks and each of its runs 8 or more)
  p.issuers = split_issuers(nkb, p.split);
  p.runs = issuer_runs(nkb, p.split, y_type == BSF_TYPE_F32);
  p.stages = p.stages / p.issuers * p.issuers;
  p.tmem_cols = 32;
  while (static_cast<int>(p.tmem_cols) < p.issuers * p.runs * p.acc_stride) p.tmem_cols *= 2;
  p.idesc = idesc_16(type == BSF_TYPE_BF16, kTileW, p.per);
  p.withhold = withhold;
  p.err = err;
  if (!make_map_16(&map_x, x, T, K, ldx, p.per)) return BSF_ERR_CUDA;
  void* args[] = {&map_w, &map_x, &p};
  return launch_cluster(kernel_of(y_type, 0), static_cast<unsigned>(tiles * p.split), kThreads, smem,
                        static_cast<unsigned>(p.split), s, args);
}
