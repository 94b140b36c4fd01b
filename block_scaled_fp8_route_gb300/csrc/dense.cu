// Dense FP8 block-scaled product of one weight matrix (an always-active expert,
// a projection), sm_103a:
//
//   D[r, n] = BF16( sum_k A[r, k] sA[r, k/128] * B[n, k] sB[n/128, k/128]  (+ C[r, n]) )
//
// DeepGEMM FP8 article (nxmr.cn), "补偿机制二": the tensor core applies the
// UE8M0 block scales (kind::mxf8f6f4, one scale per row per 32 K; a 128-wide
// block's byte serves its four K = 32 steps, picked by the scale-factor id).
//
// Weights are the MMA's M = 128 rows (256 in a CTA pair) and tokens its N, so one token costs a 128 x 16
// product.  Two forms, chosen by the time each would take (choose_plan):
//
// * Split (few tokens).  One weight matrix gives only N / 128 tiles of 128 weight rows, too few for 152 SMs
//   that each take about 52 bytes a cycle from L2, so a tile's K is split over a cluster of S CTAs: each
//   multiplies its share of the K-blocks into tensor memory, writes the FP32 partial to its own shared
//   memory, and after a cluster barrier every CTA sums a slice of the tile's tokens over the S partials
//   through distributed shared memory, in rank order (no atomics, no workspace, bit-identical from run
//   to run).  Bound by latency: 1 x 4096 x 7168 takes 7.2 us, of which the 29 MB of weights need 4.3
//   (9.5 us where none of them is in L2).
// * Pairs (many tokens).  Two CTAs multiply 256 weight rows x up to 224 tokens with one cta_group::2 MMA per
//   32 K: each stages 128 weight rows and half of the tokens, so a staged byte feeds twice the products
//   that it would in one CTA, which shared memory could not keep up with.  Two accumulators let a tile's
//   output drain under the next tile's MMAs.  Bound by the tensor cores and, in long runs, by power:
//   8192 x 4096 x 7168 takes 144-149 us, 3.34 PFLOP/s, 87 % of twice the measured bf16 burst rate.
//   Tiles of up to 128 tokens are bound by MMA issue and have two issuing warps.
#include "cluster.cuh"
#include "common.cuh"
#include "host_utils.h"
#include "tma_map.h"

namespace bsf {
namespace {

constexpr int kTileW = 128;                     // weight rows per tile
constexpr int kTileK = 128;                     // K per stage
constexpr int kMaxTok = 128;                    // tokens per tile
constexpr int kSfSlots = 4;                     // ring of scale words in tensor memory (512 K each)
constexpr int kSfCols = 16;                     // columns per slot: 4 of weights, then the tokens' from 4 on
constexpr int kAccCol = kSfSlots * kSfCols;     // accumulator columns start here
constexpr int kMaxIssuers = 2;
constexpr int kThreads = 32 * (1 + kMaxIssuers + 4);   // producer, issuers, 4 scale + epilogue warps
constexpr int kMaxStages = 12;
constexpr int kBarBytes = 512;
constexpr int kSmemBytes = 227 * 1024;
constexpr int kHalfSmemBytes = 112 * 1024;      // two CTAs per SM

struct DenseArgs {
  const int32_t* sfa;
  int64_t sfa_ld;
  const int32_t* sfb;        // [nw][Np]
  int64_t Np;
  const uint16_t* addend;
  int64_t ldc;
  uint16_t* d;
  int64_t ldd;
  int M, N, nkb;
  int chunks, per;           // token chunks per weight tile, tokens of a full chunk (multiple of 16)
  int split, stages;
  int issuers, acc_stride;   // MMA-issuing warps (a power of two), columns between their accumulators
  uint32_t tmem_cols;
  int tiled, withhold;       // withhold: BSF_DEBUG_WITHHOLD_LOADS, in the last CTA of each cluster
  int vec4;                  // four neighbouring columns of D (and C) are 8-byte aligned
  int* err;
};

// Tokens [j0, j1) of a tile: their S partials part[token][weight row], one in each CTA of the cluster,
// summed in rank order and stored.  A thread takes items (token, four weight rows) and has the loads of
// U of them in flight: a load from another CTA's shared memory takes about as long as a whole sum.
template <int S, int U>
__device__ __forceinline__ void sum_and_store(const DenseArgs& p, uint32_t part, int n0, int tok0, int j0, int j1) {
  uint32_t base[S];
#pragma unroll
  for (int s = 0; s < S; ++s) base[s] = map_rank(part, s);
  for (int i0 = threadIdx.x + j0 * 32; i0 < j1 * 32; i0 += U * kThreads) {
    float4 v[U][S];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = min(i0 + u * kThreads, j1 * 32 - 1);     // (past the end: the last item again, not stored)
#pragma unroll
      for (int s = 0; s < S; ++s) v[u][s] = ld_cluster_f4(base[s] + i * 16);
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
      const int64_t row = tok0 + (i >> 5);
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
#pragma unroll 1
        for (int x = 0; x < 4; ++x) {
          if (n + x >= p.N) break;
          const float a = p.addend ? __uint_as_float(static_cast<uint32_t>(p.addend[row * p.ldc + n + x]) << 16) : 0.f;
          p.d[row * p.ldd + n + x] = static_cast<uint16_t>(pack_bf16x2((x & 2 ? x & 1 ? f[3] : f[2] : x & 1 ? f[1] : f[0]) + a, 0.f) & 0xFFFFu);
        }
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads, 2)
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
      mbar_init(&sf_empty[s], p.issuers);
    }
    mbar_init(acc_full, p.issuers);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmap_b);
    tma_prefetch_desc(&tmap_a);
  }
  pdl_launch_dependents();
  // Dependent launch: while the preceding kernel drains, the first stages of the weights are pulled into L2.
  // (Also where that kernel writes them: it writes in L2, so the copies made here cannot go stale.)  No global
  // memory is loaded or stored before it has completed.
  if (warp == 0 && lane == 0) {
    const int most = min(kb1, kb0 + p.stages);
    for (int kb = kb0; kb < most; ++kb) {
      if (p.tiled)
        tma_prefetch_l2(&tmap_b, 0, (nt * p.nkb + kb) * kTileW);
      else
        tma_prefetch_l2(&tmap_b, kb * kTileK, nt * kTileW);
    }
  }
  pdl_wait();
  if (warp == 1) {
    tmem_alloc(tmem_slot, p.tmem_cols);
    tmem_relinquish();
  }
  __syncwarp();
  tc_fence_before();
  // (the producer, whose own thread initialised the barriers, does not wait for the others)
  if (warp != 0) asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
  else asm volatile("bar.arrive 1, %0;" ::"n"(kThreads) : "memory");
  tc_fence_after();
  const uint32_t tmem_base = warp != 0 ? *tmem_slot : 0u;

  bool have = false;                       // this warp holds a complete accumulator (epilogue warps)
  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      uint32_t stage = 0, phase = 0;
      int issued = 0;
      for (int kb = kb0; kb < kb1 && !(p.withhold && rank == p.split - 1); ++kb) {
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
  } else if (warp <= kMaxIssuers) {
    // ------------------------------------------------------------ MMA issuers
    // Issuer i takes the K-blocks kb % issuers == i into an accumulator of its own: a narrow MMA keeps its
    // issuing thread busy for about 75 cycles whatever its N, and each wait about 150, so one thread
    // takes 620 cycles per K-block where the product of up to 64 tokens needs 130.
    const int me = warp - 1;
    if (me < p.issuers && lane == 0) {
      const uint32_t d_tmem = tmem_base + kAccCol + me * p.acc_stride;
      uint32_t slot = 0, sf_phase = 0;
      uint32_t stage = (me - kb0) & (p.issuers - 1), phase = 0;    // of this issuer's first K-block
      bool ok = true, first = true;
      for (int g = kb0 >> 2; g <= (kb1 - 1) >> 2 && ok; ++g) {
        if (!mbar_wait(&sf_full[slot], sf_phase, abort_flag, p.err)) break;
        const uint32_t sfw = tmem_base + slot * kSfCols;
        for (int kb = 4 * g + me; kb < 4 * g + 4; kb += p.issuers) {
          if (kb < kb0 || kb >= kb1) continue;
          if (!mbar_wait(&full[stage], phase, abort_flag, p.err)) { ok = false; break; }
          tc_fence_after();
          const uint8_t* src = smem + stage * stage_bytes;
          const uint64_t adesc = smem_desc_k_sw128(smem_u32(src));
          const uint64_t bdesc = smem_desc_k_sw128(smem_u32(src + kTileW * kTileK));
          const uint32_t idesc = idesc_mxf8_e4m3(kTileW, mma_n, kb & 3, kb & 3);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_mxf8(d_tmem, adesc + 2 * k, bdesc + 2 * k, idesc, sfw, sfw + 4, !first || k != 0);
          first = false;
          tc_commit(&empty[stage]);
          stage += p.issuers;              // (stages are a multiple of issuers)
          if (stage >= static_cast<uint32_t>(p.stages)) { stage -= p.stages; phase ^= 1u; }
        }
        if (!ok) break;
        tc_commit(&sf_empty[slot]);
        if (++slot == kSfSlots) { slot = 0; sf_phase ^= 1u; }
      }
      // commits on every way out: TMEM is released only after the issued MMAs are done
      tc_commit(acc_full);
      wait_quiet(acc_full, 0);
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
    const int g_last = (kb1 - 1) >> 2;
    // the next word is in flight while one is written
    uint32_t w[4], a[kMaxTok / 32];
    auto load = [&](int g) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        w[c] = static_cast<uint32_t>(__ldg(p.sfb + g * p.Np + nt * kTileW + 32 * c + lane));
#pragma unroll
      for (int c = 0; c < kMaxTok / 32; ++c) {
        const int r = tok0 + lane + 32 * c;
        a[c] = 0x7F7F7F7Fu;
        if (c < ncols && r < p.M) a[c] = static_cast<uint32_t>(__ldg(p.sfa + g * p.sfa_ld + r));
      }
    };
    load(kb0 >> 2);
    for (int g = kb0 >> 2; g <= g_last; ++g) {
      uint32_t w0[4], a0[kMaxTok / 32];
#pragma unroll
      for (int c = 0; c < 4; ++c) w0[c] = w[c];
#pragma unroll
      for (int c = 0; c < kMaxTok / 32; ++c) a0[c] = a[c];
      if (g < g_last) load(g + 1);
      if (!wait_all(&sf_empty[slot], sf_phase ^ 1u, abort_flag, p.err)) { ok = false; break; }
      tc_fence_after();
      tmem_st_x4(quad + slot * kSfCols, w0[0], w0[1], w0[2], w0[3]);
#pragma unroll
      for (int c = 0; c < kMaxTok / 32; ++c)
        if (c < ncols) tmem_st_x1(quad + slot * kSfCols + 4 + c, a0[c]);
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
    }
    // A wait that ran out anywhere in this CTA ends here, and keeps all of its cluster from storing sums with its
    // partial.  (The other CTAs, launched with this one, have long been running.)
    if (!have) {
      if (lane == 0)
        for (int s = 0; s < p.split; ++s) st_cluster_u32(map_rank(smem_u32(const_cast<int*>(abort_flag)), s), 1u);
      __syncwarp();
    }
  }

  // ---------------------------------------------------------------- partial to shared memory, sum, store
  // part[token][weight row] takes the place of the stages, which have all been consumed.  (Writing the
  // partials straight into the shared memory of the CTAs that sum them took 0.8 us longer for 64 tokens:
  // it needs another cluster barrier first, and remote 4-byte stores are slow.)
  if (have) {
    const int q = warp & 3;
    const uint32_t quad = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + kAccCol;
    float* part = reinterpret_cast<float*>(smem) + 32 * q + lane;
    for (int c0 = 0; c0 < ntok; c0 += 32) {      // (whole chunks: the rows past ntok are not read)
      uint32_t r[32], o[32];
      tmem_ld_x32(quad + c0, r);
      if (p.issuers == 2) tmem_ld_x32(quad + p.acc_stride + c0, o);
      tmem_wait_ld_regs(r);
      if (p.issuers == 2) {
        tmem_wait_ld_regs(o);
#pragma unroll
        for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) + __uint_as_float(o[j]));
      }
#pragma unroll
      for (int j = 0; j < 32; ++j) part[(c0 + j) * kTileW] = __uint_as_float(r[j]);
    }
  }
  tc_fence_before();
  if (p.split > 1) cluster_sync(); else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, p.tmem_cols);
  }
  if (*abort_flag == 0) {
    const int j0 = ntok * rank / p.split, j1 = ntok * (rank + 1) / p.split, n0 = nt * kTileW;
    const uint32_t part = smem_u32(smem);
    switch (p.split) {
      case 1: sum_and_store<1, 4>(p, part, n0, tok0, j0, j1); break;
      case 2: sum_and_store<2, 4>(p, part, n0, tok0, j0, j1); break;
      case 4: sum_and_store<4, 2>(p, part, n0, tok0, j0, j1); break;
      default: sum_and_store<8, 1>(p, part, n0, tok0, j0, j1); break;
    }
  }
  // a CTA's shared memory stays until every CTA of the cluster has read it
  if (p.split > 1) cluster_sync();
}

// ---------------------------------------------------------------- CTA pairs: 256 x up to 224 output tiles
constexpr int kPairW = 256;                                // weight rows of a tile (MMA M), 128 per CTA
constexpr int kPairMaxTok = 224;                           // tokens of a tile (MMA N), half staged by each CTA
constexpr int kTwoIssuerTok = 128;                         // up to here a pair has two issuing warps
constexpr int kPairMaxStages = 4;                          // a stage is 256 K of both operands
// warps: 0 weight loads, 1 MMA issuer, 2-5 scales, 6-13 epilogue, 14 waiter, 15 token loads, 16 second issuer
constexpr int kPairWaiter = 14, kPairTokLoads = 15, kPairIssuer2 = 16;
constexpr int kBoxBytes = 32 * 64;                         // 32 tokens x 32 bf16 columns of D
constexpr int kPairBarBytes = 512;

struct PairArgs {
  const int32_t* sfa;
  int64_t sfa_ld;
  const int32_t* sfb;
  int64_t Np;
  const uint16_t* addend;
  int64_t ldc;
  uint16_t* d;
  int64_t ldd;
  int M, N, nkb, nw;
  int tiles_m, tiles_n;      // token tiles, weight tiles
  int tok;                   // tokens of a tile: a multiple of 32, at most kPairMaxTok
  int accs;                  // sets of accumulators, one accumulator for each issuer in a set
  int stages;
  int tiled, vec8, withhold;
  int* err;
};

// Executed by the whole warp, issued by the lane whose `lead` is non-zero.
__device__ __forceinline__ void pair_mma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %7, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
          d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(sfa_tmem), "r"(sfb_tmem), "r"(lead)
      : "memory");
}

// kIssuers: MMA-issuing warps, 1 or 2
template <int kIssuers>
__global__ void __launch_bounds__(32 * (15 + kIssuers), 1)
    dense_pair_kernel(const __grid_constant__ CUtensorMap tmap_b, const __grid_constant__ CUtensorMap tmap_a,
                      const __grid_constant__ CUtensorMap tmap_d, const __grid_constant__ CUtensorMap tmap_c,
                      const PairArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int half_tok = p.tok >> 1;
  // a stage: 128 weight rows of two K-blocks, then half of the tile's tokens of the same two
  const int tok_bytes = half_tok * kTileK;
  const int stage_bytes = 2 * (kTileW * kTileK + tok_bytes);
  uint8_t* store = smem + p.stages * stage_bytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(store + 16 * kBoxBytes);                // used in rank 0
  uint64_t* empty = full + kPairMaxStages;
  uint64_t* sf_full = empty + kPairMaxStages;                                           // used in rank 0
  uint64_t* sf_empty = sf_full + kSfSlots;
  uint64_t* acc_full = sf_empty + kSfSlots;
  uint64_t* acc_empty = acc_full + 2;                                                   // used in rank 0
  uint64_t* add_full = acc_empty + 2;                                                   // two per epilogue warp
  uint64_t* mma_done = add_full + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int total = p.tiles_m * p.tiles_n;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kSfSlots; ++s) {
      mbar_init(&sf_full[s], 8);
      mbar_init(&sf_empty[s], kIssuers);
    }
    for (int s = 0; s < p.accs; ++s) {
      mbar_init(&acc_full[s], kIssuers);
      mbar_init(&acc_empty[s], 16);
    }
    for (int s = 0; s < 16; ++s) mbar_init(&add_full[s], 1);
    mbar_init(mma_done, kIssuers);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmap_b);
    tma_prefetch_desc(&tmap_a);
  }
  pdl_launch_dependents();
  pdl_wait();
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();                           // barriers of both CTAs are initialised
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t acc_cols = kIssuers * p.tok;               // of a set of accumulators
  const uint32_t tmem_sf = tmem_base + p.accs * acc_cols;

  if (warp == 0 || warp == kPairTokLoads) {
    // ------------------------------------------------------------ TMA producers (each CTA loads its halves)
    // One warp per operand, two K-blocks per barrier: a load takes its issuing thread about 170 cycles and
    // a wait or commit 100 and more, against 448 cycles of MMAs per K-block.  (Where K has an odd number
    // of blocks the last stage's second half is loaded but not multiplied: past K it is zeros.)
    if (lane == 0) {
      const bool weights = warp == 0;
      uint32_t stage = 0, phase = 0;
      int issued = 0;
      bool ok = !p.withhold;
      for (int t = pair; t < total && ok; t += npairs) {
        const int tm = t % p.tiles_m, tn = t / p.tiles_m;
        const int row = tm * p.tok + static_cast<int>(rank) * half_tok;
        const int wt = tn * 2 + static_cast<int>(rank);               // 128-row weight tile of this CTA
        for (int kb = 0; kb < p.nkb; kb += 2) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.err)) { ok = false; break; }
          const uint32_t bar = map_rank(smem_u32(&full[stage]), 0);
          uint8_t* dst = smem + stage * stage_bytes;
          if (weights) {
            if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * stage_bytes);   // both CTAs, both operands
            if (p.tiled) {                                            // two blocks are one 32 KB run
              pair_load_2d(dst, &tmap_b, bar, 0, (wt * p.nkb + kb) * kTileW);
            } else {
              pair_load_2d(dst, &tmap_b, bar, kb * kTileK, wt * kTileW);
              pair_load_2d(dst + kTileW * kTileK, &tmap_b, bar, (kb + 1) * kTileK, wt * kTileW);
            }
          } else {
            dst += 2 * kTileW * kTileK;
            pair_load_2d(dst, &tmap_a, bar, kb * kTileK, row);
            pair_load_2d(dst + tok_bytes, &tmap_a, bar, (kb + 1) * kTileK, row);
          }
          ++issued;
          if (++stage == static_cast<uint32_t>(p.stages)) { stage = 0; phase ^= 1u; }
        }
      }
      if (rank == 0) {
        // both CTAs' loads complete on these barriers; rank 1 waits for rank 0 at the last cluster barrier
        const int outstanding = issued < p.stages ? issued : p.stages;
        for (int j = 0; j < outstanding; ++j) {
          if (stage == 0) { stage = p.stages; phase ^= 1u; }
          --stage;
          wait_quiet(&full[stage], phase);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1 || warp >= kPairIssuer2) {
    // ------------------------------------------------------------ MMA issuers (rank 0)
    // An issuing thread reads no shared memory between stages: the waiter warp does every wait and hands
    // each stage over through a named barrier whose OR-reduced predicate carries an abort.  An MMA costs its
    // issuing thread about 86 cycles whatever its N, so tiles of up to 128 tokens (64 cycles of tensor work)
    // have two issuers that take a tile's stages in turn, each into an accumulator of its own: in tiles of
    // 128 tokens 512 x 4096 x 7168 takes 17.5 us with two and 20.7 with one, 512 x 256 x 7168 14.4 and 19.1.
    // Wider tiles are slower with two (their accumulators leave no second set, and the tensor cores are the
    // limit): 2500 x 4096 x 7168 takes 53.5 us in tiles of 192 with one, 57.5 with two.
    const int me = warp == 1 ? 0 : 1;
    if (rank == 0) {
      const uint32_t lead = lane == 0;
      uint32_t stage = 0, slot = 0, acc = 0;           // stage: of the tile's next K-block pair, whoever takes it
      bool ok = true;
      for (int t = pair; t < total && ok; t += npairs) {
        const uint32_t d_tmem = tmem_base + acc * acc_cols + me * p.tok;
        uint32_t first = 1;
        for (int kb = 0; kb < p.nkb; kb += 2) {
          if (kIssuers == 1 || ((kb >> 1) & 1) == me) {
            if (named_barrier_or(1 + me, 64, false)) { ok = false; break; }
            tc_fence_after();
            const uint32_t sf = tmem_sf + slot * kSfCols;
            const uint8_t* src = smem + stage * stage_bytes;
            uint64_t adesc = smem_desc_k_sw128(smem_u32(src));
            uint64_t bdesc = smem_desc_k_sw128(smem_u32(src + 2 * kTileW * kTileK));
            uint32_t idesc = idesc_mxf8_e4m3(kPairW, p.tok, kb & 3, kb & 3);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              pair_mma(d_tmem, adesc + 2 * k, bdesc + 2 * k, idesc, sf, sf + 4, k == 0 ? first ^ 1u : 1u, lead);
            first = 0;
            if (kb + 1 < p.nkb) {
              adesc += kTileW * kTileK >> 4;
              bdesc += tok_bytes >> 4;
              idesc = idesc_mxf8_e4m3(kPairW, p.tok, (kb + 1) & 3, (kb + 1) & 3);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                pair_mma(d_tmem, adesc + 2 * k, bdesc + 2 * k, idesc, sf, sf + 4, 1, lead);
            }
            pair_commit(&empty[stage], lead);
          }
          if (++stage == static_cast<uint32_t>(p.stages)) stage = 0;
          if ((kb & 2) || kb + 2 >= p.nkb) {
            pair_commit(&sf_empty[slot], lead);          // (from every issuer, also one that had no stage of it)
            if (++slot == kSfSlots) slot = 0;
          }
        }
        if (!ok) break;
        pair_commit(&acc_full[acc], lead);
        if (++acc == static_cast<uint32_t>(p.accs)) acc = 0;
      }
      pair_commit(mma_done, lead);
      if (lane == 0) wait_quiet(mma_done, 0);
    }
    __syncwarp();
  } else if (warp == kPairWaiter) {
    // ------------------------------------------------------------ waiter (rank 0): the issuers' waits, in their order
    if (rank == 0) {
      uint32_t stage = 0, phase = 0, slot = 0, sf_phase = 0, acc = 0, acc_phase = 0;
      bool good = true;
      int t = pair, kb = 0;
      while (t < total) {
        good = wait_cluster_all(&acc_empty[acc], acc_phase ^ 1u, abort_flag, p.err);
        for (kb = 0; kb < p.nkb; kb += 2) {
          if (good && (kb & 3) == 0) good = wait_cluster_all(&sf_full[slot], sf_phase, abort_flag, p.err);
          if (good) good = wait_all(&full[stage], phase, abort_flag, p.err);
          if (!good) break;
          named_barrier_or(kIssuers == 1 ? 1 : 1 + ((kb >> 1) & 1), 64, false);
          if (++stage == static_cast<uint32_t>(p.stages)) { stage = 0; phase ^= 1u; }
          if ((kb & 2) || kb + 2 >= p.nkb)
            if (++slot == kSfSlots) { slot = 0; sf_phase ^= 1u; }
        }
        if (!good) break;
        if (++acc == static_cast<uint32_t>(p.accs)) { acc = 0; acc_phase ^= 1u; }
        t += npairs;
      }
      if (!good) {
        // the issuer of this stage is at its barrier or on its way to it, and so is the other one if any later
        // stage is its own (with two issuers every tile has stages of both)
        const int me = kIssuers == 1 ? 0 : (kb >> 1) & 1;
        named_barrier_or(1 + me, 64, true);
        if (kIssuers == 2 && (kb + 2 < p.nkb || t + npairs < total)) named_barrier_or(2 - me, 64, true);
      }
    }
  } else if (warp < 6) {
    // ------------------------------------------------------------ scale words (each CTA into its own tensor memory)
    // columns 0-3 of a slot: this CTA's 128 weight rows; from 4: all tokens of the tile
    const int q = warp & 3;
    const uint32_t quad = tmem_sf + (static_cast<uint32_t>(32 * q) << 16);
    const int ncols = p.tok >> 5;
    uint32_t slot = 0, sf_phase = 0;
    // the words of the next slot are in flight while this one's are written: a load's latency is as long as
    // two stages' MMAs, and a slot serves four
    uint32_t w[4], a[kPairMaxTok / 32];
    auto load = [&](int t, int g) {
      const int row = t % p.tiles_m * p.tok + lane;
      const int wrow = t / p.tiles_m * kPairW + static_cast<int>(rank) * 128 + lane;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        w[c] = wrow + 32 * c < p.Np ? static_cast<uint32_t>(__ldg(p.sfb + g * p.Np + wrow + 32 * c)) : 0x7F7F7F7Fu;
#pragma unroll
      for (int c = 0; c < kPairMaxTok / 32; ++c)
        a[c] = c < ncols && row + 32 * c < p.M ? static_cast<uint32_t>(__ldg(p.sfa + g * p.sfa_ld + row + 32 * c))
                                               : 0x7F7F7F7Fu;
    };
    int t = pair, g = 0;
    load(t, g);
    while (true) {
      uint32_t w0[4], a0[kPairMaxTok / 32];
#pragma unroll
      for (int c = 0; c < 4; ++c) w0[c] = w[c];
#pragma unroll
      for (int c = 0; c < kPairMaxTok / 32; ++c) a0[c] = a[c];
      if (++g == p.nw) {
        g = 0;
        t += npairs;
      }
      if (t < total) load(t, g);
      if (!wait_all(&sf_empty[slot], sf_phase ^ 1u, abort_flag, p.err)) break;
      tc_fence_after();
      const uint32_t col = quad + slot * kSfCols;
      tmem_st_x4(col, w0[0], w0[1], w0[2], w0[3]);
      tmem_st_x4(col + 4, a0[0], a0[1], a0[2], a0[3]);
      tmem_st_x2(col + 8, a0[4], a0[5]);
      tmem_st_x1(col + 10, a0[6]);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_cluster(map_rank(smem_u32(&sf_full[slot]), 0));
      if (++slot == kSfSlots) { slot = 0; sf_phase ^= 1u; }
      if (t >= total) break;
    }
  } else {
    // ------------------------------------------------------------ epilogue: lane = weight row, 32 tokens at a time
    // Two warps share a quadrant's tokens.  After one exchange with its neighbour a lane holds two weight
    // rows of one token (4 bytes).  With 16-byte aligned rows of D the 32 x 32 boxes go through this warp's
    // shared memory (64-byte swizzle: 16-byte piece j of token i sits at j ^ (i / 2 % 4)); the addend is
    // loaded the same way, ahead of the accumulator.  TMA cuts the boxes at the edges, but a row only at a
    // multiple of 16 bytes: where N % 8 the last box of a row goes out by elements.
    const int q = warp & 3, ew = warp - 6;
    const int nc = p.tok >> 5, c_first = ew < 4 ? 0 : (nc + 1) >> 1, c_last = ew < 4 ? (nc + 1) >> 1 : nc;
    const int odd = lane & 1;
    uint8_t* bufs = store + ew * 2 * kBoxBytes;
    uint32_t acc = 0, acc_phase = 0, add_phase = 0;        // add_phase: bit b for buffer b
    int box = 0;                            // next box buffer
    for (int t = pair; t < total; t += npairs) {
      const int tm = t % p.tiles_m, tn = t / p.tiles_m;
      const int n0 = tn * kPairW + static_cast<int>(rank) * 128 + 32 * q;
      const int tok0 = tm * p.tok;
      // boxes of this warp that touch D
      const int cuts = n0 < p.N ? min(c_last, (p.M - tok0 + 31) >> 5) - c_first : 0;
      const bool boxed = p.vec8 && (p.N % 8 == 0 || n0 + 32 <= p.N);
      const bool boxed_add = p.addend && boxed && cuts > 0;
      // addend box i of the tile into its buffer (its last store has been read)
      auto load_add = [&](int i) {
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        mbar_arrive_expect_tx(&add_full[ew * 2 + (i & 1)], kBoxBytes);
        tma_load_2d(bufs + (i & 1) * kBoxBytes, &tmap_c, &add_full[ew * 2 + (i & 1)], n0, tok0 + 32 * (c_first + i));
      };
      int loaded = 0;                       // addend boxes of this tile
      if (boxed_add) {
        box = 0;
        loaded = min(2, cuts);
        if (lane == 0)
          for (int i = 0; i < loaded; ++i) load_add(i);
        __syncwarp();
      }
      if (!wait_all(&acc_full[acc], acc_phase, abort_flag, p.err)) {
        // the copies must have landed before this CTA may exit
        for (int i = 0; i < loaded; ++i) wait_landed(&add_full[ew * 2 + i], (add_phase >> i) & 1u, p.err);
        break;
      }
      tc_fence_after();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + acc * acc_cols;
      for (int c = c_first; c < c_last; ++c) {
        uint32_t r[32], r2[32];
        tmem_ld_x32(taddr + 32 * c, r);
        if (kIssuers == 2) tmem_ld_x32(taddr + p.tok + 32 * c, r2);
        tmem_wait_ld_regs(r);
        if (kIssuers == 2) {
          tmem_wait_ld_regs(r2);
#pragma unroll
          for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) + __uint_as_float(r2[j]));
        }
        if (c == c_last - 1) {              // the accumulator's last columns are in registers
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_cluster(map_rank(smem_u32(&acc_empty[acc]), 0));
        }
        if (c - c_first >= cuts) continue;
        if (boxed) {
          uint8_t* buf = bufs + box * kBoxBytes;
          if (boxed_add) {
            wait_landed(&add_full[ew * 2 + box], (add_phase >> box) & 1u, p.err);
            __syncwarp();
            add_phase ^= 1u << box;
          } else {
            if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");  // the box before last is read
            __syncwarp();
          }
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            float v0 = __uint_as_float(r[j]), v1 = __uint_as_float(r[j + 1]);
            const float x = __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, 1);
            v0 = odd ? x : v0;
            v1 = odd ? v1 : x;
            uint32_t* at = reinterpret_cast<uint32_t*>(buf + (j + odd) * 64 + (((lane >> 3) ^ ((j >> 1) & 3)) << 4) +
                                                       (lane & 6) * 2);
            if (boxed_add) {
              const uint32_t a = *at;
              v0 += __uint_as_float(a << 16);
              v1 += __uint_as_float(a & 0xFFFF0000u);
            }
            *at = pack_bf16x2(v0, v1);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tmap_d, buf, n0, tok0 + 32 * c);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            if (boxed_add && loaded < cuts) load_add(loaded);
          }
          ++loaded;
          box ^= 1;
        } else if (n0 + lane < p.N) {
          const int64_t row = tok0 + 32 * c;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            if (row + j < p.M) {
              float f = __uint_as_float(r[j]);
              if (p.addend)
                f += __uint_as_float(static_cast<uint32_t>(p.addend[(row + j) * p.ldc + n0 + lane]) << 16);
              p.d[(row + j) * p.ldd + n0 + lane] = static_cast<uint16_t>(pack_bf16x2(f, 0.f) & 0xFFFFu);
            }
          }
        }
      }
      if (++acc == static_cast<uint32_t>(p.accs)) { acc = 0; acc_phase ^= 1u; }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    // the issuer's last commit has reached this CTA's barriers too, so none arrives after it exits
    if (warp == 6 && lane == 0) wait_quiet(mma_done, 0);
    __syncwarp();
  }

  tc_fence_before();
  cluster_sync();                           // no load, MMA or remote arrival of the pair is outstanding
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(512) : "memory");
  }
}

// Once per device: both kernels may use all shared memory, and the number of CTAs of the split kernel that
// run at once, one per SM, in clusters of 1, 2, 4 and 8 (a cluster lives in one GPC, so 8 leave SMs idle).
struct DeviceLimits {
  std::atomic<int> ctas[4];
  std::atomic<bool> ready;
};
bsf_status device_limits(const DeviceLimits** out) {
  static DeviceLimits limits[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return BSF_ERR_CUDA;
  DeviceLimits& l = limits[dev];
  if (!l.ready.load(std::memory_order_acquire)) {      // (racing first calls store the same values)
    const void* kernels[3] = {reinterpret_cast<const void*>(dense_split_kernel),
                              reinterpret_cast<const void*>(dense_pair_kernel<1>),
                              reinterpret_cast<const void*>(dense_pair_kernel<2>)};
    for (const void* k : kernels) {
      if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) != cudaSuccess ||
          cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) !=
              cudaSuccess)
        return BSF_ERR_CUDA;
    }
    for (int i = 0; i < 4; ++i) {
      DependentLaunch launch(8u << i, kThreads, kSmemBytes, nullptr, 1u << i);
      launch.cfg.numAttrs = 1;                           // the cluster alone
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, kernels[0], &launch.cfg) != cudaSuccess || n <= 0) {
        cudaGetLastError();
        return BSF_ERR_CUDA;
      }
      l.ctas[i].store(n << i, std::memory_order_relaxed);
    }
    l.ready.store(true, std::memory_order_release);
  }
  *out = &l;
  return BSF_OK;
}

// Which kernel a product takes, by the time each would need (nanoseconds).  The constants are fitted to
// products of 1 .. 2600 tokens with 14 weights' widths from 256 to 12288 and 9 inner lengths from 512 to 7168,
// timed in every form that could be the fastest: 10177 with weights that may be in L2 and 5083 with weights
// that come from HBM.  The choice is within 0.5 % and 1.1 % of the best form on average; the worst is 24 %
// (1 x 5120 x 2560 with K over two CTAs and not four).  Both sides, 4096 x 7168: 256 tokens 14.6 us split against 17.7 in
// pairs, 1024 tokens 38.7 against 30.6; 1024 x 1024 takes 1024 tokens in 6.2 us split, 7.2 in pairs.
struct Plan {
  bool pair;
  int tok;                  // pairs: tokens per tile; split: most tokens per tile
  int split;
};
Plan choose_plan(int64_t M, int64_t N, int64_t nkb, const DeviceLimits& limits) {
  const int64_t ntn = (N + kTileW - 1) / kTileW, sms = sm_count(), pairs = sms / 2;
  Plan best = {false, 64, 1};
  int64_t least = INT64_MAX;
  for (int tok = 64; tok <= kMaxTok; tok += 64) {
    if (tok > 64 && M <= 64) break;
    const int64_t chunks = (M + tok - 1) / tok, per = ((M + chunks - 1) / chunks + 15) / 16 * 16;
    for (int i = 0; i < 4; ++i) {
      const int64_t split = int64_t(1) << i, ctas = ntn * chunks * split;
      if (i > 0 && (nkb < 2 * split || ctas > 2 * sms)) break;
      const int64_t at_once = limits.ctas[i].load(std::memory_order_relaxed), kbs = (nkb + split - 1) / split;
      const int64_t load = (ctas + at_once - 1) / at_once;              // CTAs of the busiest SM
      int64_t ns = 3100 + 6 * per + (i > 0 ? 400 + 400 * i : 0);
      if (per > 64)         // one CTA per SM: it cannot start under its predecessor
        ns += 800 + load * kbs * 270 + (load - 1) * 4700;
      else                  // two CTAs on an SM share its 120 bytes a nanosecond from L2
        ns += kbs * (load / 2 * (273 + 32 * per / 15) + load % 2 * 270) + (load - 1) * 1150;
      if (ns < least) {
        least = ns;
        best = {false, tok, static_cast<int>(split)};
      }
    }
  }
  for (int tok = kPairMaxTok; tok >= 96; tok -= 32) {
    const int64_t tiles = (M + tok - 1) / tok * ((ntn + 1) / 2), waves = (tiles + pairs - 1) / pairs;
    // two K-blocks: by the issuing threads, or by the tensor cores and shared memory
    const int64_t issue = tok <= kTwoIssuerTok ? 320 : 470, multiply = (tok <= kTwoIssuerTok ? 30 : 22) * tok / 10;
    const int64_t ns = 4600 + waves * ((nkb + 1) / 2 * (issue > multiply ? issue : multiply) + 13 * tok);
    if (ns < least) {
      least = ns;
      best = {true, tok, 1};
    }
  }
  return best;
}

}  // namespace
}  // namespace bsf

using namespace bsf;

extern "C" bsf_status bsf_dense_gemm(const uint8_t* a, const int32_t* sfa, int64_t sfa_ld, int64_t M,
                                     const uint8_t* b, const int32_t* sfb, int64_t N, int64_t K, const void* addend,
                                     int64_t ldc, void* d, int64_t ldd, int flags, bsf_stream_t stream) {
  if (M < 0 || N <= 0 || K <= 0 || K % 128) return BSF_ERR_INVALID_ARGUMENT;
  if (flags & ~(BSF_B_TILED | BSF_DEBUG_WITHHOLD_LOADS)) return BSF_ERR_INVALID_ARGUMENT;
  if (M == 0) return BSF_OK;
  if (!a || !sfa || !b || !sfb || !d) return BSF_ERR_INVALID_ARGUMENT;
  if (sfa_ld < M || sfa_ld % 4 || ldd < N || (addend && ldc < N)) return BSF_ERR_INVALID_ARGUMENT;
  if (!aligned16(a) || !aligned16(b) || !aligned16(sfa) || !aligned16(sfb) ||
      (reinterpret_cast<uintptr_t>(d) & 1) || (reinterpret_cast<uintptr_t>(addend) & 1))
    return BSF_ERR_MISALIGNED;
  if (!fits_rows(M, K) || !fits_rows(M, ldd) || (addend && ldc > kMaxRowWidth) || N > kMaxRowWidth || sfa_ld > kMaxRows)
    return BSF_ERR_UNSUPPORTED;
  const int64_t ntn = (N + kTileW - 1) / kTileW, nkb = K / kTileK;
  if ((ntn + 2) * kTileW * nkb > INT32_MAX || M > kMaxRows - 256) return BSF_ERR_UNSUPPORTED;
  int* err = device_error_ptr();
  if (!err) return BSF_ERR_CUDA;
  const bool tiled = (flags & BSF_B_TILED) != 0, withhold = (flags & BSF_DEBUG_WITHHOLD_LOADS) != 0;
  const int64_t Np = ntn * kTileW;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const DeviceLimits* limits;
  const bsf_status st = device_limits(&limits);
  if (st != BSF_OK) return st;
  const Plan plan = choose_plan(M, N, nkb, *limits);
  CUtensorMap map_a, map_b;

  if (plan.pair) {
    const int tok = plan.tok;
    const int64_t tiles_m = (M + tok - 1) / tok, tiles_n = (ntn + 1) / 2, tiles = tiles_m * tiles_n;
    if (tiles > INT32_MAX) return BSF_ERR_UNSUPPORTED;
    PairArgs p;
    p.sfa = sfa;
    p.sfa_ld = sfa_ld;
    p.sfb = sfb;
    p.Np = Np;
    p.addend = static_cast<const uint16_t*>(addend);
    p.ldc = ldc;
    p.d = static_cast<uint16_t*>(d);
    p.ldd = ldd;
    p.M = static_cast<int>(M);
    p.N = static_cast<int>(N);
    p.nkb = static_cast<int>(nkb);
    p.nw = static_cast<int>((nkb + 3) / 4);
    p.tiles_m = static_cast<int>(tiles_m);
    p.tiles_n = static_cast<int>(tiles_n);
    p.tok = tok;
    // (each issuer needs a stage of the tile; two sets of accumulators where they and the scales fit)
    const int issuers = tok <= kTwoIssuerTok && nkb > 2 ? 2 : 1;
    p.accs = 2 * issuers * tok + kSfSlots * kSfCols <= 512 ? 2 : 1;
    p.tiled = tiled;
    p.withhold = withhold;
    p.vec8 = aligned16(d) && ldd % 8 == 0 && (!addend || (aligned16(addend) && ldc % 8 == 0));
    const int stage_bytes = 2 * (kTileW + tok / 2) * kTileK;
    p.stages = (kSmemBytes - 1024 - kPairBarBytes - 16 * kBoxBytes) / stage_bytes;
    if (p.stages > kPairMaxStages) p.stages = kPairMaxStages;
    p.err = err;
    CUtensorMap map_d, map_c;
    if (tiled ? !make_map(&map_b, b, Np * nkb, 128, 2 * kTileW) : !make_map(&map_b, b, Np, K, kTileW))
      return BSF_ERR_CUDA;
    if (!make_map(&map_a, a, M, K, tok / 2)) return BSF_ERR_CUDA;
    map_d = map_c = map_a;                           // (not used without 16-byte aligned rows)
    if (p.vec8 && !make_map_bf16(&map_d, d, M, N, ldd)) return BSF_ERR_CUDA;
    if (p.vec8 && addend && !make_map_bf16(&map_c, addend, M, N, ldc)) return BSF_ERR_CUDA;
    const int64_t pairs = sm_count() / 2, used = tiles < pairs ? tiles : pairs;
    void* args[] = {&map_b, &map_a, &map_d, &map_c, &p};
    return launch_cluster(issuers == 2 ? reinterpret_cast<const void*>(dense_pair_kernel<2>)
                                       : reinterpret_cast<const void*>(dense_pair_kernel<1>),
                          static_cast<unsigned>(2 * used), 32 * (15 + issuers), kSmemBytes, 2, s, args);
  }

  const int64_t chunks = (M + plan.tok - 1) / plan.tok, tiles = ntn * chunks;
  if (tiles * plan.split > INT32_MAX) return BSF_ERR_UNSUPPORTED;
  DenseArgs p;
  p.sfa = sfa;
  p.sfa_ld = sfa_ld;
  p.sfb = sfb;
  p.Np = Np;
  p.addend = static_cast<const uint16_t*>(addend);
  p.ldc = ldc;
  p.d = static_cast<uint16_t*>(d);
  p.ldd = ldd;
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.nkb = static_cast<int>(nkb);
  p.chunks = static_cast<int>(chunks);
  // equal chunks (the last may be shorter, never empty: (chunks - 1) * per <= (chunks - 1) * tok < M)
  p.per = static_cast<int>(((M + chunks - 1) / chunks + 15) / 16 * 16);
  p.split = plan.split;
  const int stage_bytes = (kTileW + p.per) * kTileK;
  const size_t smem = p.per <= 64 ? kHalfSmemBytes : kSmemBytes;
  p.stages = (static_cast<int>(smem) - 1024 - kBarBytes) / stage_bytes;
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  p.acc_stride = (p.per + 31) / 32 * 32;
  // (an issuer without a K-block would leave its accumulator unwritten)
  p.issuers = nkb / p.split >= kMaxIssuers ? kMaxIssuers : 1;
  // a stage always goes to the same issuer, whose own waits then see its barrier's phases in order
  p.stages = p.stages / p.issuers * p.issuers;
  const int cols = kAccCol + p.issuers * p.acc_stride;
  p.tmem_cols = cols <= 128 ? 128 : cols <= 256 ? 256 : 512;
  p.tiled = tiled;
  p.withhold = withhold;
  p.vec4 = (reinterpret_cast<uintptr_t>(d) & 7) == 0 && ldd % 4 == 0 &&
           (!addend || ((reinterpret_cast<uintptr_t>(addend) & 7) == 0 && ldc % 4 == 0));
  p.err = err;
  if (tiled ? !make_map(&map_b, b, Np * nkb, 128, kTileW) : !make_map(&map_b, b, Np, K, kTileW)) return BSF_ERR_CUDA;
  if (!make_map(&map_a, a, M, K, p.per)) return BSF_ERR_CUDA;
  void* args[] = {&map_b, &map_a, &p};
  return launch_cluster(reinterpret_cast<const void*>(dense_split_kernel), static_cast<unsigned>(tiles * p.split), kThreads,
                        smem, static_cast<unsigned>(p.split), s, args);
}
