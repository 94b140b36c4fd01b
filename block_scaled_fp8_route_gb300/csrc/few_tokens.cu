// A whole mixture-of-experts layer for a few tokens (1 .. 32), sm_103a, in two kernels:
//
//   [g; u]_te = W13_e x_t                      for every expert e that token t chose
//   h_te      = p_te * g / (1 + exp(-g)) * u
//   z_t       = sum_e W2_e h_te  (+ an expert that every token takes, p = 1)  (+ addend)
//
// "GEMM 执行方式" (rainlin-net) §4.2-§4.4 defines routing, expert products and combine; bsf_dispatch ... bsf_combine
// run them as separate kernels with quantised activations.  Here weights are E4M3 with 128 x 128 UE8M0 scales
// (or bf16) and activations are not quantised.
//
// Such a layer is bound by the chosen experts' weights, which are read once; everything else has to hide
// behind that stream.
// * Work is cut into units of K-blocks, not of experts: every CTA takes the same number of boxes (128
//   weight rows x 128 bytes, 16 KB, a contiguous run of tiled weights) whatever the routing is, fewer where an expert has
//   more than 8 tokens, whose operand then takes longer than its weights.  Each CTA derives routing, units and places
//   from topk_ids itself.
// * The first kernel multiplies gate and up rows of one 128-wide tile by the expert's tokens.  A tile whose
//   K is shared by two or more CTAs leaves that many partial sums; nobody waits for anybody, because
//   the second kernel adds them (in a fixed order) while it forms h.
// * The second kernel, a programmatic dependent, takes whole SMs with up to five stages as the first one's CTAs leave
//   them, does its routing and starts its loads before it waits for the partial sums.  (Half the shared memory for each
//   kernel, so that both are resident and the weights are under way sooner, is no faster with one token and slower with
//   a batch, whose second product then has too little in flight.)  Contraction runs over (expert, i), so a cluster
//   splits one long K and its CTAs exchange one partial of z through distributed shared memory, in rank order.
// * FP8 weights meet unquantised activations on the FP8 tensor cores: a value scaled to its block of 128 is split
//   into E4M3 terms, v = t0 + t1 / 16 (+ t2 / 256), which take two (three) columns of the MMA.  A bf16 value has 8
//   significant bits and each term holds 4, so two terms of x are exact down to 2**-14 of the block's largest value and
//   off by at most 2**-21 of that below.  A float32 h takes three: off by at most 2**-14 of its size or 2**-25 of the
//   block's largest (two would leave 2**-9 and 2**-21, which z's rounding to bf16 does not hide).  bf16 weights meet h as
//   two bf16 terms (2**-17 of it).  The weights go from HBM to the tensor core without passing a register.
//
// Measured with FP8 weights.  128 experts of which a token chooses 8, K 4096, I 1536: 32 tokens read the 2.11 GB of 111
// experts in 300-304 us, 7.0 TB/s; 256 experts, K 7168, I 2048 and a shared one, 5 tokens: 1.69 GB in 236-239 us, 7.1 TB/s; both are
// bound by HBM.  One token of the first layer reads 152 MB in 34 us.  Time stamps of its CTAs (medians): the first kernel's
// routing 1.7, first load and operand 3.1, products 13.2, sums 0.6; the second's start 1.1, routing 2.0, wait for the last
// partial sums 1.1, first operand 2.1, products 7.0, exchange 1.5: 20 us of products in a chain of 13 us of latencies.
// Multiplying less gains next to nothing there (3 of 4 MMAs left out: 1 us).  The third term of h costs 0.1-0.3 us of a
// small layer, 0.6 % of one token, 0.8 % of 32 and 2.2 % where 32 tokens all choose 8 experts (112 -> 114.5 us).
#include <algorithm>
#include <cfloat>

#include "cluster.cuh"
#include "common.cuh"
#include "host_utils.h"
#include "quant_math.cuh"
#include "tma_map.h"

namespace bsf {
namespace {

constexpr int kMaxTokens = 32;
constexpr int kMaxKr = 32;
constexpr int kMaxExperts = 1024;
constexpr int kBoxBytes = 16384;               // 128 weight rows x 128 bytes
constexpr int kMaxStages = 5;                  // a stage: two boxes, the token operand that both meet, its scales
constexpr int kSfBytes = 512;                  // scale bytes of an operand's rows: word r / 32 of row r, byte b for box b
constexpr int kAccCol = 64;                    // tensor memory: 4 columns of ones, 4 per stage and box of scales, sums
constexpr int kParts = 4;                      // most CTAs that share a tile of the first product
// warps: 0 and 3 weight loads, 1 and 2 MMA issuers (one per box each), 4-7 and 8-11 as each kernel needs them
constexpr int kThreads = 384;
constexpr int kBarBytes = 512;                // barriers, tensor memory's place, abort flag, 32 words of groups, a maximum
constexpr int kStages1 = 3;                    // first kernel; with more in flight the SMs share HBM less evenly
constexpr int kUnitTokens = 8;                 // FP8: tokens whose operand the first kernel forms in the time of a load
constexpr int kMostSmem = 227 * 1024;
constexpr int kMaxSplit = 16;

enum { kFp8 = 0, kBf16 = 1 };

struct FewArgs {
  const uint16_t* x;
  int64_t ldx;
  const int32_t* ids;
  const float* weights;
  const int32_t* sf;          // scale words of this kernel's routed weights [E][words][rows], and of the shared ones
  const int32_t* sf_shared;
  float* part;                // partial sums of the first product [kParts][R][2][I], [kParts][T][2][S]
  float* part_shared;
  const uint16_t* addend;
  int64_t ldc;
  uint16_t* z;
  int64_t ldz;
  int T, kr, E, R;            // R = T * kr
  int K, I, S;
  int nkb1;                   // K-blocks of the first product
  int nkb2, nkb2_shared;      // of the second, per expert
  int ctas1;                  // CTAs of the first kernel
  int split, nbox;            // second kernel: CTAs per cluster, 128-row tiles per CTA
  int tables, stage_space;    // bytes of shared memory: tables, then stages
  uint32_t tmem_cols;
  int tiled, withhold, vec4;
  int* err;
};

struct Unit {                 // consecutive K-blocks of one expert (and, in the first kernel, of one tile)
  int a, j, kb0, kb1;         // a: index of the chosen expert, the number of them for the shared one
};

__device__ __forceinline__ void tmem_ld_x8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
// (names the registers of the load that it completes, see tmem_wait_ld_regs)
__device__ __forceinline__ void tmem_wait_ld_regs(uint32_t (&r)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
               :
               : "memory");
}
// Eight tokens' sums of this lane's weight row: the columns of their terms, `rows` apart, all in flight at once.
template <int TERMS>
__device__ __forceinline__ void sum_of_terms(uint32_t taddr, int rows, float (&v)[8]) {
  uint32_t r[TERMS][8];
#pragma unroll
  for (int t = 0; t < TERMS; ++t) tmem_ld_x8(taddr + t * rows, r[t]);
#pragma unroll
  for (int t = 0; t < TERMS; ++t) tmem_wait_ld_regs(r[t]);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    v[k] = __uint_as_float(r[0][k]);
#pragma unroll
    for (int t = 1; t < TERMS; ++t) v[k] += __uint_as_float(r[t][k]);
  }
}
// 32 rows of 16 bytes in shared memory -> four columns of tensor memory, the same in each of the four lane quadrants:
// scale bytes, row r + 32 c of the operand in word c of row r.  The MMAs that the same thread issues next see them.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t smem_addr) {
  uint64_t d = static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);   // no swizzle
  d |= static_cast<uint64_t>(128u >> 4) << 32;                      // stride: 8 rows x 16 bytes
  d |= static_cast<uint64_t>(1u) << 46;                             // descriptor version (tcgen05)
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}
__device__ __forceinline__ void arrive_with(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Eight values f * scale -> E4M3 codes of their leading four bits, and term by term of 16 times what is left (exact in
// float32).
template <int TERMS>
__device__ __forceinline__ void split8(const float (&f)[8], float scale, uint32_t (&code)[TERMS][2]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = f[2 * i] * scale, b = f[2 * i + 1] * scale;
#pragma unroll
    for (int t = 0; t < TERMS; ++t) {
      const __nv_fp8x2_storage_t c = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
      code[t][i >> 1] = i & 1 ? code[t][i >> 1] | static_cast<uint32_t>(c) << 16 : c;
      if (t + 1 < TERMS) {
        const float2 back = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3)));
        a = (a - back.x) * 16.f;
        b = (b - back.y) * 16.f;
      }
    }
  }
}

// x / (1 + exp(-x)); the argument of exp is rounded, an error of |x| 2**-24 of a term that matters up to |x| = 16 only.
__device__ __forceinline__ float silu(float x) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
  return __fdividef(x, 1.f + e);
}

// A block's exponent for split8 and the factor 2**-e: NaN where the block holds an infinity (which E4M3 lacks), as a
// NaN in the block is NaN without it.  At least `least`, so that the products' scales have an exponent.
__device__ __forceinline__ int split_exponent(float amax, int least, float& scale) {
  const int e = max(block_exponent(amax), least);
  scale = amax <= FLT_MAX ? inv_pow2(e) : __uint_as_float(0x7FC00000u);
  return e;
}

// Token operand of one K-block: row r of 128 bytes, 128-byte swizzle.
__device__ __forceinline__ uint8_t* operand_at(uint8_t* slot, int row, int chunk) {
  return slot + row * 128 + ((chunk ^ (row & 7)) << 4);
}

template <int FMT, int PHASE>
__global__ void __launch_bounds__(kThreads, 1)
    few_kernel(const __grid_constant__ CUtensorMap map_routed, const __grid_constant__ CUtensorMap map_shared,
               const FewArgs p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem_raw);                       // per stage and box
  uint64_t* empty = full + 2 * kMaxStages;                                      // per stage and box
  uint64_t* formed = empty + 2 * kMaxStages;                                    // one for each warp that forms operands
  uint64_t* acc_full = formed + 8;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* done = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* groups_of = tmem_slot + 2;              // per 32 experts: chosen ones, further costs << 8, rows << 16
  int* most_tokens = reinterpret_cast<int*>(groups_of + 32);                    // of any chosen expert
  uint8_t* scales = smem_raw + kBarBytes;                                       // [stages][kSfBytes]
  // of each chosen expert: its tokens (bits); expert, first row << 10, further costs of those before it << 21
  uint2* chosen = reinterpret_cast<uint2*>(scales + kMaxStages * kSfBytes);
  float* share = reinterpret_cast<float*>(chosen + min(p.E, p.R) + 1);          // [R] p of each row
  uint8_t* token = reinterpret_cast<uint8_t*>(share + p.R);                     // [R] token of each row
  uint8_t* smem = smem_raw + p.tables;                                          // stages: two boxes and the token operand

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cluster = PHASE == 2 ? static_cast<int>(blockIdx.x) / p.split : 0;
  const int rank = PHASE == 2 ? static_cast<int>(blockIdx.x) - cluster * p.split : 0;
  const int boxes = PHASE == 1 ? 2 : min(p.nbox, p.K / 128 - cluster * p.nbox);
  constexpr int kConvWarps = PHASE == 1 ? 4 : 8;
  constexpr int kShares = PHASE == 1 ? 1 : kConvWarps;       // of forming an operand
  constexpr int kTerms = (FMT == kFp8 ? 1 : 0) + PHASE;      // of a value in the operand

  if (tid == 0) {
    for (int s = 0; s < 2 * kMaxStages; ++s) {
      mbar_init(&full[s], 1 + kShares);    // its load, and all shares of the operand's forming
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kConvWarps; ++s) mbar_init(&formed[s], boxes);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&acc_full[s], boxes);
      mbar_init(&acc_empty[s], 4);
    }
    mbar_init(done, boxes);
    *abort_flag = 0;
    *most_tokens = p.S == 0 ? 1 : p.T;     // (all take the shared expert)
    fence_barrier_init();
    tma_prefetch_desc(&map_routed);
    if (p.S) tma_prefetch_desc(&map_shared);
  }
  // The first kernel lets the second one start once everything before both is complete, so that the second may read
  // topk_ids, topk_weights and weights at once; only the partial sums (and z) wait for the first to end.
  for (int e = tid; e < p.E; e += kThreads) reinterpret_cast<uint32_t*>(smem)[e] = 0u;      // (the masks below)
  if (PHASE == 1) pdl_wait();
  pdl_launch_dependents();

  // What a K-block of the first product costs with n tokens.  Forming an FP8 operand (two terms of each value, a
  // maximum of each block) takes longer than loading its weights beyond 8 tokens: 32 tokens of which all choose one
  // of 64 experts (K 4096, I 1536) take 435 us in CTAs of equal K-blocks and 210 in these, with a shared expert of 1536
  // 435 and 203; the 435 with two stages for such operands, too.  bf16 values are copied (343 either way).  Costs
  // beyond one: at most 3 of an expert, 96 of 32 experts (a byte) and 122 of 1024 assignments (40 experts of 25 tokens, one
  // of 24).
  auto cost = [](uint32_t n) -> uint32_t { return FMT == kFp8 ? (n + kUnitTokens - 1) / kUnitTokens : 1u; };

  // ---------------------------------------------------------------- routing, in every CTA
  // The stages, not yet in use, hold the tables: tokens and first row of every expert, ids and weights.
  {
    uint32_t* mask = reinterpret_cast<uint32_t*>(smem);
    int* first = reinterpret_cast<int*>(mask + kMaxExperts);
    int* ids = first + kMaxExperts;
    float* w = reinterpret_cast<float*>(ids + kMaxTokens * kMaxKr);
    __syncthreads();
    for (int i = tid; i < p.R; i += kThreads) {
      const int id = __ldcg(p.ids + i);
      if (PHASE == 2) w[i] = __ldcg(p.weights + i);
      ids[i] = id;
      if (id >= p.E) {
        if (PHASE == 1 && blockIdx.x == 0) raise_error(p.err, BSF_DEVERR_EXPERT_ID);
      } else if (id >= 0) {
        atomicOr(mask + id, 1u << (i / p.kr));
      }
    }
    __syncthreads();
    const int groups = (p.E + 31) >> 5;
    for (int g = warp; g < groups; g += kThreads / 32) {
      const uint32_t m = g * 32 + lane < p.E ? mask[g * 32 + lane] : 0u;
      const uint32_t n = __popc(m);
      const uint32_t sum = __reduce_add_sync(0xffffffffu, n << 16 | (n ? (cost(n) - 1) << 8 | 1u : 0u));
      const uint32_t most = __reduce_max_sync(0xffffffffu, n);
      if (lane == 0) {
        if (PHASE == 1 || (sum & 0xFF00u)) atomicMax(most_tokens, static_cast<int>(most));
        groups_of[g] = sum;
      }
    }
    __syncthreads();
    for (int g = warp; g < groups; g += kThreads / 32) {
      const int e = g * 32 + lane;
      const uint32_t m = e < p.E ? mask[e] : 0u;
      const uint32_t some = __ballot_sync(0xffffffffu, m != 0u);
      const uint32_t mine = m ? static_cast<uint32_t>(__popc(m)) << 16 | (cost(__popc(m)) - 1) << 8 : 0u;
      uint32_t before = mine;                // rows << 16, further costs << 8, chosen experts
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t below = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += below;
      }
      before += __popc(some & ((1u << lane) - 1u)) - mine;
      uint32_t at = before & 0xFFu, further = before >> 8 & 0xFFu, rows = before >> 16;
      for (int k = 0; k < g; ++k) {
        at += groups_of[k] & 0xFFu;
        further += groups_of[k] >> 8 & 0xFFu;
        rows += groups_of[k] >> 16;
      }
      if (m) {
        chosen[at] = make_uint2(m, static_cast<uint32_t>(e) | rows << 10 | further << 21);
        first[e] = static_cast<int>(rows);
      }
    }
    __syncthreads();
    for (int i = tid; i < p.R; i += kThreads) {
      const int id = ids[i];
      if (id < 0 || id >= p.E) continue;
      const int t = i / p.kr;
      const int row = first[id] + __popc(mask[id] & ((1u << t) - 1u));
      token[row] = static_cast<uint8_t>(t);
      if (PHASE == 2) {
        // an expert named twice by a token is one row with both weights
        float sum = 0.f;
        bool earlier = false;
        for (int k = t * p.kr; k < t * p.kr + p.kr; ++k) {
          if (ids[k] != id) continue;
          earlier |= k < i;
          sum += w[k];
        }
        if (!earlier) share[row] = sum;
      }
    }
  }
  int nchosen = 0, further = 0;
  for (int g = 0; g < (p.E + 31) >> 5; ++g) {
    nchosen += static_cast<int>(groups_of[g] & 0xFFu);
    further += static_cast<int>(groups_of[g] >> 8 & 0xFFu);
  }
  const uint32_t everyone = p.T == 32 ? 0xffffffffu : (1u << p.T) - 1u;
  if (tid == 0) chosen[nchosen] = make_uint2(everyone, static_cast<uint32_t>(further) << 21);
  if (FMT == kFp8)                         // every row has a scale, whether or not it has values
    for (int i = tid; i < kMaxStages * kSfBytes / 4; i += kThreads) reinterpret_cast<uint32_t*>(scales)[i] = 0x7F7F7F7Fu;
  proxy_fence();                           // the tables' place is written by TMA next
  __syncthreads();

  const int tiles = p.I >> 7;              // 128-wide tiles of h per expert
  int u0, u1, per = 1;                     // this CTA's K-blocks
  int first_routed = 0, mine_routed = 0, first_shared = 0;     // (second kernel)
  {
    const int routed = PHASE == 1 ? nchosen * tiles * p.nkb1 : nchosen * p.nkb2;
    const int units = routed + (PHASE == 1 ? (p.S >> 7) * p.nkb1 : p.nkb2_shared);
    const int whole = tiles * p.nkb1;      // K-blocks of an expert
    const int all = (nchosen + further) * whole + (p.S >> 7) * p.nkb1 * static_cast<int>(cost(p.T));   // costs
    // (at least a third of a tile's, so that at most kParts CTAs share one)
    per = max((all + p.ctas1 - 1) / p.ctas1, static_cast<int>(cost(*most_tokens)) * ((p.nkb1 + 2) / 3));
    if (PHASE == 1) {
      // a CTA takes the K-blocks that begin within its `per` costs
      auto cut = [&](int cta) {
        const int at = cta * per;
        if (at >= all) return units;
        int a = min(at / whole, nchosen);
        if (further) {                     // the last expert that begins at or before it
          a = 0;
          for (int hi = nchosen; a < hi;) {
            const int mid = (a + hi + 1) >> 1;
            if ((mid + static_cast<int>(chosen[mid].y >> 21)) * whole <= at) a = mid;
            else hi = mid - 1;
          }
        }
        const int c = static_cast<int>(cost(__popc(chosen[a].x)));
        return a * whole + (at - (a + static_cast<int>(chosen[a].y >> 21)) * whole + c - 1) / c;
      };
      if (all == units) {                  // (one cost each: found without the search, 0.6 us of one token's 33)
        u0 = min(units, static_cast<int>(blockIdx.x) * per);
        u1 = min(units, u0 + per);
      } else {
        u0 = u1 = 0;
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
          u0 = u1;
          u1 = cut(blockIdx.x + k);
        }
      }
    } else {
      // a share of the routed experts' and one of the shared expert's, whose operand takes longer to form
      first_routed = static_cast<int>(static_cast<int64_t>(routed) * rank / p.split);
      mine_routed = static_cast<int>(static_cast<int64_t>(routed) * (rank + 1) / p.split) - first_routed;
      first_shared = p.nkb2_shared * rank / p.split;
      u0 = 0;
      u1 = mine_routed + p.nkb2_shared * (rank + 1) / p.split - first_shared;
    }
  }
  // the costs before a tile, and those of its K-blocks: CTA c of the first kernel has those of c * per and above
  auto costs_before = [&](int a, int j) {
    return ((a + static_cast<int>(chosen[a].y >> 21)) * tiles + j * static_cast<int>(cost(__popc(chosen[a].x)))) * p.nkb1;
  };
  auto unit_at = [&](int u) {
    Unit w;
    if (PHASE == 1) {
      const int item = u / p.nkb1;
      w.a = min(item / tiles, nchosen);
      w.j = item - w.a * tiles;
      w.kb0 = u - item * p.nkb1;
      w.kb1 = min(p.nkb1, w.kb0 + u1 - u);
    } else {
      w.j = 0;
      if (u < mine_routed) {
        w.a = (first_routed + u) / p.nkb2;
        w.kb0 = first_routed + u - w.a * p.nkb2;
        w.kb1 = min(p.nkb2, w.kb0 + mine_routed - u);
      } else {
        w.a = nchosen;
        w.kb0 = first_shared + u - mine_routed;
        w.kb1 = w.kb0 + u1 - u;
      }
    }
    return w;
  };
  // tokens padded to whole groups; the operand has so many rows for each term of a value, 16 k in all
  auto padded = [&](int n) { return kTerms >= 2 ? (n + 7) & ~7 : (n + 15) & ~15; };
  auto operand_rows = [&](int n) { return (kTerms * padded(n) + 15) & ~15; };
  // Stages as large as the most tokens of an expert need: 32 tokens seldom put more than 8 on one, and a larger operand
  // would cost a stage of weights in flight.
  const int most_rows = operand_rows(PHASE == 1 ? *most_tokens : p.T);
  const int stage_bytes = 2 * kBoxBytes + ((most_rows * 128 + 1023) & ~1023);
  const int stages = min(p.stage_space / stage_bytes, PHASE == 1 ? kStages1 : kMaxStages);      // (at most kConvWarps)
  const int acc_stride = (most_rows + 31) & ~31;                   // columns of a sum
  const uint32_t sets = kAccCol + 4 * acc_stride <= static_cast<int>(p.tmem_cols) ? 2u : 1u;   // of sums, first kernel

  // A CTA of the second kernel with at most half as many K-blocks as warps (and no more than stages, so that none is used
  // twice) has several warps form each of them, some tokens each: 10 tokens that all choose 4 experts, K and I 384, 16.2 ->
  // 13.0 us, 32 tokens x 2 of 8 experts, K 2048, I 512, 25.1 -> 23.6.  What a warp's arrival counts makes up for it.
  const int helpers = PHASE == 1 || u1 - u0 > 4 ? 1 : u1 - u0 > 2 ? 2 : u1 - u0 > 1 ? 4 : 8;

  if (warp == 1) {
    tmem_alloc(tmem_slot, p.tmem_cols);
    tmem_relinquish();
  }
  __syncwarp();
  tc_fence_before();
  // (the loads and the operands do not wait for tensor memory, which the first kernel may still hold)
  if (warp == 1 || warp == 2 || warp >= 8) {
    asm volatile("bar.sync 1, %0;" ::"n"(6 * 32) : "memory");
    if (FMT == kFp8) {                     // scales of the weight rows: one (a block's own goes to the tokens' rows)
      if (warp >= 8) {
        tc_fence_after();
        tmem_st_x4(*tmem_slot + (static_cast<uint32_t>(32 * (warp & 3)) << 16), 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu,
                   0x7F7F7F7Fu);
        tmem_wait_st();
        tc_fence_before();
      }
      asm volatile("bar.sync 2, %0;" ::"n"(6 * 32) : "memory");
    }
    tc_fence_after();
  }
  const volatile uint32_t* tmem_at = tmem_slot;      // (read by the warps above; by the others after a later barrier)

  bool have = false;                       // this warp may read the accumulators (second kernel)
  // Each box of a K-block has a loading and an issuing thread of its own: a load with its waits takes a thread about 300
  // cycles, four MMAs with theirs 800, where two boxes' share of HBM is 1400, and less while stages are catching up.
  if (warp == 0 || warp == 3) {
    // ------------------------------------------------------------ weight loads
    const int b = warp == 0 ? 0 : 1;
    if (lane == 0 && b < boxes) {
      const uint64_t once = l2_policy_evict_first();
      uint32_t stage = 0, phase = 0;
      int issued = 0;
      bool ok = !p.withhold;
      for (int u = u0; u < u1 && ok;) {
        const Unit w = unit_at(u);
        const bool shared = w.a == nchosen;
        const CUtensorMap* map = shared ? &map_shared : &map_routed;
        const int e = shared ? 0 : static_cast<int>(chosen[w.a].y & 0x3FFu);
        const int width = shared ? p.S : p.I;                            // of h
        const int row = PHASE == 1 ? (2 * e + b) * width + w.j * 128 : e * p.K + (cluster * p.nbox + b) * 128;
        const int nkb = PHASE == 1 ? p.nkb1 : shared ? p.nkb2_shared : p.nkb2;
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          // (the second kernel's clock starts when the first kernel has ended)
          if (PHASE == 2 && issued == stages) pdl_wait();
          uint64_t* bar = &full[2 * stage + b];
          if (!mbar_wait(&empty[2 * stage + b], phase ^ 1u, abort_flag, p.err)) { ok = false; break; }
          // the stage's operand may be formed anew, too
          if (issued >= stages) mbar_arrive(&formed[(issued - stages) & (kConvWarps - 1)]);
          mbar_arrive_expect_tx(bar, kBoxBytes);
          uint8_t* to = smem + stage * stage_bytes + b * kBoxBytes;
          if (p.tiled)
            tma_load_2d_hint(to, map, bar, 0, row * nkb + kb * 128, once);
          else
            tma_load_2d_hint(to, map, bar, kb * 128, row, once);
          ++issued;
          if (++stage == static_cast<uint32_t>(stages)) { stage = 0; phase ^= 1u; }
        }
        u += w.kb1 - w.kb0;
      }
      // no TMA write may be in flight when the CTA exits or reuses its stages
      const int outstanding = min(issued, stages);
      for (int i = 0; i < outstanding; ++i) {
        if (stage == 0) { stage = stages; phase ^= 1u; }
        --stage;
        wait_quiet(&full[2 * stage + b], phase);
      }
    }
    __syncwarp();
  } else if (warp <= 2) {
    // ------------------------------------------------------------ MMA issuers
    const int b = warp - 1;
    if (lane == 0 && b < boxes) {
      const uint32_t tmem_base = *tmem_at;
      if (PHASE == 2) pdl_wait();
      uint32_t stage = 0, phase = 0, set = 0, set_phase = 0;
      bool ok = true, start = true;
      for (int u = u0; u < u1 && ok;) {
        const Unit w = unit_at(u);
        const int n = operand_rows(PHASE == 1 ? __popc(chosen[w.a].x) : p.T);
        const uint32_t d = tmem_base + kAccCol + (2 * set + b) * acc_stride;
        const uint32_t idesc = FMT == kFp8 ? idesc_mxf8_e4m3(128, n, 0, b) : idesc_bf16(128, n);
        if (PHASE == 1) {
          start = true;
          if (!mbar_wait(&acc_empty[set], set_phase ^ 1u, abort_flag, p.err)) break;
        }
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          if (!mbar_wait(&full[2 * stage + b], phase, abort_flag, p.err)) { ok = false; break; }
          tc_fence_after();
          const uint8_t* at = smem + stage * stage_bytes;
          const uint64_t adesc = smem_desc_k_sw128(smem_u32(at + b * kBoxBytes));
          const uint64_t bdesc = smem_desc_k_sw128(smem_u32(at + 2 * kBoxBytes));
          const uint32_t sf = tmem_base + 4 + (2 * stage + b) * 4;
          if (FMT == kFp8) copy_scales(sf, smem_u32(scales + stage * kSfBytes));
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (FMT == kFp8)
              mma_mxf8(d, adesc + 2 * k, bdesc + 2 * k, idesc, tmem_base, sf, !start || k != 0);
            else
              mma_bf16(d, adesc + 2 * k, bdesc + 2 * k, idesc, !start || k != 0);
          }
          start = false;
          tc_commit(&empty[2 * stage + b]);
          if (++stage == static_cast<uint32_t>(stages)) { stage = 0; phase ^= 1u; }
        }
        u += w.kb1 - w.kb0;
        if (PHASE == 1 && ok) {
          tc_commit(&acc_full[set]);
          if (++set == sets) { set = 0; set_phase ^= 1u; }
        }
      }
      if (PHASE == 2 && ok) tc_commit(&acc_full[0]);
      // on every way out: tensor memory is released only after the issued MMAs are done
      tc_commit(done);
      wait_quiet(done, 0);
    }
    __syncwarp();
  } else if (warp < 4 + kConvWarps) {
    // ------------------------------------------------------------ token operands and scales
    // One warp per K-block: what forms an operand is a chain of latencies (values, a maximum, codes, fences) several
    // times as long as a unit's share of HBM, so as many of them as there are warps are under way at once.
    constexpr int kLanes = FMT == kFp8 ? 16 : 8;             // lanes of eight values per token
    constexpr int kAtOnce = 32 / kLanes;                     // tokens at once
    const int cw = warp - 4, sub = lane & (kLanes - 1), mine = lane / kLanes;
    // exponent of a box's scale (the words of a block's 128 rows are the same)
    auto scale_word = [&](const Unit& w, int b) -> uint32_t {
      if (FMT != kFp8 || b >= boxes) return 0x7F7F7F7Fu;
      const bool sh = w.a == nchosen;
      const int width = sh ? p.S : p.I, e = sh ? 0 : static_cast<int>(chosen[w.a].y & 0x3FFu);
      const int rows = PHASE == 1 ? 2 * width : p.K, inner = PHASE == 1 ? p.K : width;
      const int row = PHASE == 1 ? b * width + w.j * 128 : (cluster * p.nbox + b) * 128;
      const int64_t at = (static_cast<int64_t>(e) * ((inner + 511) >> 9) + (w.kb0 >> 2)) * rows + row;
      return static_cast<uint32_t>(__ldg((sh ? p.sf_shared : p.sf) + at));
    };
    // This lane's eight values of a token as they go into an operand: the terms' codes (or bf16 values), and the
    // exponent of their block.
    struct Terms {
      uint32_t code[kTerms][FMT == kFp8 ? 2 : 4];
      int e;
    };
    auto terms_of = [&](const float (&f)[8], int e0, int e1) {
      Terms r;
      r.e = 0;
      if (FMT == kFp8) {
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[i]));
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        float scale;
        r.e = split_exponent(amax, 4 * kTerms - 130 - min(0, min(e0, e1)), scale);      // (the last term's is -126)
        if constexpr (FMT == kFp8) split8(f, scale, r.code);
      } else if constexpr (FMT == kBf16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t hi = r.code[0][i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
          if constexpr (kTerms == 2)
            r.code[1][i] = pack_bf16x2(f[2 * i] - __uint_as_float(hi << 16), f[2 * i + 1] - __uint_as_float(hi & 0xFFFF0000u));
        }
      }
      return r;
    };
    // ... as row `row` of a stage's operand whose terms are `rows` apart
    auto put = [&](const Terms& r, int stage, int row, int rows, int e0, int e1) {
      uint8_t* to = smem + stage * stage_bytes + 2 * kBoxBytes;
      if constexpr (FMT == kFp8) {
#pragma unroll
        for (int t = 0; t < kTerms; ++t)
          *reinterpret_cast<uint2*>(operand_at(to, t * rows + row, sub >> 1) + (sub & 1) * 8) = make_uint2(r.code[t][0], r.code[t][1]);
        if (sub < kTerms) {                // a term's scales, for box 0 and box 1
          const int at = sub * rows + row, e = r.e + 127 - 4 * sub;
          *reinterpret_cast<uint32_t*>(scales + stage * kSfBytes + (at & 31) * 16 + (at >> 5) * 4) =
              static_cast<uint32_t>(min(e + e0, 254) | min(e + e1, 254) << 8);
        }
      } else {
#pragma unroll
        for (int t = 0; t < kTerms; ++t)
          *reinterpret_cast<uint4*>(operand_at(to, t * rows + row, sub)) = make_uint4(r.code[t][0], r.code[t][1], r.code[t][2], r.code[t][3]);
      }
    };
    auto exponent = [](uint32_t word, int kb) { return static_cast<int>((word >> (8 * (kb & 3))) & 255u) - 127; };
    // K-block i takes the stage of K-block i - stages.  Its end is told (by the loading threads, who wait for it
    // anyway) on a barrier of the warp that formed it: this warp has seen the one before there complete, when it
    // formed K-block i - kConvWarps, and the one after cannot be yet (stages <= kConvWarps), so a parity says which.
    auto wait_stage = [&](int i) {
      const int before = i - stages;
      return before < 0 || wait_all(&formed[before & (kConvWarps - 1)], (before / kConvWarps) & 1, abort_flag, p.err);
    };
    auto publish = [&](int stage) {
      proxy_fence();
      __syncwarp();
      if (lane < boxes) arrive_with(&full[2 * stage + lane], kShares / helpers);
    };

    if (PHASE == 1) {
      // x: the loads of up to kBatch rounds are in flight at once, and while the warp waits for its stage
      constexpr int kBatch = 4;
      constexpr int kStep = kBatch * kAtOnce;
      for (int i = cw; u0 + i < u1; i += kConvWarps) {
        const Unit w = unit_at(u0 + i);
        const uint2 who = chosen[w.a];
        const int n = __popc(who.x), stage = i % stages, rows = padded(n);
        const uint8_t* list = token + (who.y >> 10 & 0x7FFu);
        const bool sh = w.a == nchosen;
        const uint32_t word0 = scale_word(w, 0), word1 = scale_word(w, 1);
        const uint16_t* from = p.x + w.kb0 * (kLanes * 8) + sub * 8;
        bool ok = true;
        const int e0 = exponent(word0, w.kb0), e1 = exponent(word1, w.kb0);
        uint4 v[kBatch];
        auto load = [&](int j0) {
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            const int j = j0 + k * kAtOnce + mine;
            v[k] = make_uint4(0, 0, 0, 0);
            if (j < n) v[k] = __ldg(reinterpret_cast<const uint4*>(from + (sh ? j : list[j]) * p.ldx));
          }
        };
        load(0);
        for (int j0 = 0; j0 < n; j0 += kStep) {
          // A batch's terms side by side, and the next one's loads, before the stage is waited for: a stage held up holds
          // up its own next loads.
          auto term = [&](int k) {
            float f[8];
            bf16x8_to_float(v[k], f);
            return terms_of(f, e0, e1);
          };
          Terms r[kBatch];
          r[0] = term(0);
          const bool more = n - j0 > kAtOnce;
          if (more) {
#pragma unroll
            for (int k = 1; k < kBatch; ++k) r[k] = term(k);
          }
          if (n - j0 > kStep) load(j0 + kStep);
          if (j0 == 0) ok = wait_stage(i);
          if (!ok) break;
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            const int row = j0 + k * kAtOnce + mine;
            if ((k == 0 || more) && row < rows) put(r[k], stage, row, rows, e0, e1);
          }
        }
        if (!ok) break;
        publish(stage);
      }
    } else {
      // h from the first kernel's partial sums, at most kParts of each value, added in the order of the CTAs; tokens
      // that did not choose the expert get zeros
      Unit w = {};
      uint32_t word0 = 0, word1 = 0;
      const int first = cw / helpers, helper = cw - first * helpers;
      if (u0 + first < u1) {               // (there may be no K-block at all, nor scales)
        w = unit_at(u0 + first);
        word0 = scale_word(w, 0);
        word1 = scale_word(w, 1);
      }
      pdl_wait();
      const int rows = padded(p.T);
      for (int i = first; u0 + i < u1; i += kConvWarps) {
        if (i != first) {
          w = unit_at(u0 + i);
          word0 = scale_word(w, 0);
          word1 = scale_word(w, 1);
        }
        const bool sh = w.a == nchosen;
        const uint2 who = chosen[w.a];
        const int n = __popc(who.x), stage = i % stages;
        const int width = sh ? p.S : p.I;
        const int64_t part_step = static_cast<int64_t>(sh ? p.T : p.R) * 2 * width;
        const int at = w.kb0 * (kLanes * 8) + sub * 8;                   // of h
        const int item = w.a * tiles + (at >> 7);
        const int costs = costs_before(w.a, item - w.a * tiles), more = (p.nkb1 - 1) * static_cast<int>(cost(n));
        const int parts = (costs + more) / per - costs / per + 1;
        bool ok = true;
        const int e0 = exponent(word0, w.kb0), e1 = exponent(word1, w.kb0);
        const float* base = (sh ? p.part_shared : p.part) + at;
        constexpr int kRounds = 2;           // of tokens whose loads are in flight together, two parts of each
        // tokens that did not choose the expert, when the stage is free
        auto zeros = [&]() {
          uint8_t* to = smem + stage * stage_bytes + 2 * kBoxBytes;
          for (int z = 4 * helper + (lane >> 3); z < rows; z += 4 * helpers) {
            if (who.x >> z & 1u) continue;
#pragma unroll
            for (int t = 0; t < kTerms; ++t)
              *reinterpret_cast<uint4*>(operand_at(to, t * rows + z, lane & 7)) = make_uint4(0, 0, 0, 0);
          }
        };
        const int j_first = helper * kAtOnce;          // (several warps: a round at a time each)
        if (j_first >= n) zeros();                     // (there are several, so the stage is new)
        for (int j0 = j_first; j0 < n && ok; j0 += helpers > 1 ? helpers * kAtOnce : kRounds * kAtOnce) {
          float g[kRounds][8] = {}, v[kRounds][8] = {}, weight[kRounds];
          int t[kRounds], row[kRounds];
#pragma unroll
          for (int k = 0; k < kRounds; ++k) {
            const int j = j0 + k * kAtOnce + mine;
            row[k] = -1, t[k] = 0, weight[k] = 1.f;
            if (j < n && (k == 0 || helpers == 1)) {
              row[k] = sh ? j : static_cast<int>(who.y >> 10 & 0x7FFu) + j;
              t[k] = sh ? j : token[row[k]];
              if (!sh) weight[k] = share[row[k]];
            }
          }
          // (a single round takes the other one's registers for two more parts)
          const bool narrow = helpers > 1 || n - j0 <= kAtOnce;
          for (int s = 0; s < parts; s += narrow ? 4 : 2) {
            float4 a[kRounds][2][4];
#pragma unroll
            for (int k = 0; k < kRounds; ++k)
#pragma unroll
              for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int i4 = 0; i4 < 4; ++i4) {
                  a[k][q][i4] = make_float4(0.f, 0.f, 0.f, 0.f);
                  const int r = narrow ? row[0] : row[k], part = narrow ? s + 2 * k + q : s + q;
                  if (r >= 0 && part < parts)
                    a[k][q][i4] = __ldcg(reinterpret_cast<const float4*>(base + part * part_step +
                                                                         (2 * static_cast<int64_t>(r) + (i4 >> 1)) * width) + (i4 & 1));
                }
#pragma unroll
            for (int k = 0; k < kRounds; ++k)
#pragma unroll
              for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int i4 = 0; i4 < 2; ++i4) {
                  const float4 x = a[k][q][i4], y = a[k][q][2 + i4];
                  g[k][4 * i4] += x.x, g[k][4 * i4 + 1] += x.y, g[k][4 * i4 + 2] += x.z, g[k][4 * i4 + 3] += x.w;
                  v[k][4 * i4] += y.x, v[k][4 * i4 + 1] += y.y, v[k][4 * i4 + 2] += y.z, v[k][4 * i4 + 3] += y.w;
                }
            static_assert(kRounds == 2 && kParts == 4, "a single round takes all parts");
            if (narrow) {
#pragma unroll
              for (int c = 0; c < 8; ++c) g[0][c] += g[1][c], v[0][c] += v[1][c], g[1][c] = v[1][c] = 0.f;
            }
          }
#pragma unroll
          for (int k = 0; k < kRounds; ++k) {
            if (j0 + k * kAtOnce >= n || (k > 0 && helpers > 1)) break;
#pragma unroll
            for (int c = 0; c < 8; ++c) g[k][c] = silu(g[k][c]) * v[k][c] * weight[k];
            const Terms r = terms_of(g[k], e0, e1);
            if (j0 == j_first && k == 0) {
              ok = wait_stage(i);
              if (!ok) break;
              zeros();
            }
            if (row[k] >= 0) put(r, stage, t[k], rows, e0, e1);
          }
        }
        if (!ok) break;
        publish(stage);
      }
    }
  } else if (PHASE == 1) {
    // ------------------------------------------------------------ first kernel's sums: lane = row of the tile
    const int q = warp & 3;
    const uint32_t tmem_base = *tmem_at;
    uint32_t set = 0, set_phase = 0;
    bool ok = true;
    for (int u = u0; u < u1;) {
      const Unit w = unit_at(u);
      const bool sh = w.a == nchosen;
      const uint2 who = chosen[w.a];
      const int n = __popc(who.x), rows = padded(n);
      const int width = sh ? p.S : p.I;
      const int part = static_cast<int>(blockIdx.x) - costs_before(w.a, w.j) / per;
      const int64_t row0 = static_cast<int64_t>(part) * (sh ? p.T : p.R) + (who.y >> 10 & 0x7FFu);
      float* to = (sh ? p.part_shared : p.part) + row0 * 2 * width + w.j * 128 + 32 * q + lane;
      ok = ok && wait_all(&acc_full[set], set_phase, abort_flag, p.err);
      tc_fence_after();
      const uint32_t acc = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + kAccCol + 2 * set * acc_stride;
      for (int b = 0; b < 2; ++b) {
        for (int c = 0; c < rows; c += 8) {
          float v[8];
          sum_of_terms<kTerms>(acc + b * acc_stride + c, rows, v);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            // (where a wait ran out the sums are marked, so that z cannot look like an answer)
            if (c + k < n) to[(static_cast<int64_t>(c + k) * 2 + b) * width] = ok ? v[k] : __uint_as_float(0x7FC00000u);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[set]);
      if (++set == sets) { set = 0; set_phase ^= 1u; }
      u += w.kb1 - w.kb0;
    }
  }

  if (PHASE == 1) {
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
      tc_fence_after();
      tmem_dealloc(*tmem_at, p.tmem_cols);
    }
    return;
  }

  // ---------------------------------------------------------------- z: partials to shared memory, sum over the cluster
  pdl_wait();                              // (every thread, before it stores)
  __syncthreads();                         // (the place of the accumulators is known to all warps)
  const uint32_t tmem_base = *tmem_at;
  float* sums = reinterpret_cast<float*>(smem);              // [T][boxes][128], in place of the consumed stages
  if (warp >= 4) {
    have = wait_all(&acc_full[0], 0, abort_flag, p.err) && *abort_flag == 0;
    have = __all_sync(0xffffffffu, have);
    tc_fence_after();
    if (!have) {
      // a wait that ran out anywhere in this CTA keeps all of its cluster from storing
      if (lane == 0)
        for (int s = 0; s < p.split; ++s) st_cluster_u32(map_rank(smem_u32(const_cast<int*>(abort_flag)), s), 1u);
      __syncwarp();
    } else if (const int b = (warp - 4) >> 2; b < boxes) {
      const int q = warp & 3, rows = padded(p.T);
      const uint32_t acc = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + kAccCol + b * acc_stride;
      for (int c = 0; c < rows; c += 8) {
        float v[8];
        sum_of_terms<kTerms>(acc + c, rows, v);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (c + k < p.T) sums[((c + k) * boxes + b) * 128 + 32 * q + lane] = u0 < u1 ? v[k] : 0.f;
      }
    }
  }
  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, p.tmem_cols);
  }
  if (*abort_flag == 0) {
    const int quads = p.T * boxes * 32;                      // groups of four neighbouring values of z
    const int i1 = quads * (rank + 1) / p.split;
    const uint32_t mine = smem_u32(sums);
    for (int i = quads * rank / p.split + tid; i < i1; i += kThreads) {
      float4 f = {};
      for (int s0 = 0; s0 < p.split; s0 += 8) {              // in rank order, eight loads at once
        float4 v[8];
#pragma unroll
        for (int s = 0; s < 8; ++s)
          if (s0 + s < p.split) v[s] = ld_cluster_f4(map_rank(mine, s0 + s) + i * 16);
#pragma unroll
        for (int s = 0; s < 8; ++s)
          if (s0 + s < p.split) f.x += v[s].x, f.y += v[s].y, f.z += v[s].z, f.w += v[s].w;
      }
      const int t = i / (boxes * 32), n = cluster * p.nbox * 128 + (i - t * boxes * 32) * 4;
      if (p.vec4) {
        if (p.addend) {
          const uint2 c = *reinterpret_cast<const uint2*>(p.addend + t * p.ldc + n);
          f.x += __uint_as_float(c.x << 16);
          f.y += __uint_as_float(c.x & 0xFFFF0000u);
          f.z += __uint_as_float(c.y << 16);
          f.w += __uint_as_float(c.y & 0xFFFF0000u);
        }
        *reinterpret_cast<uint2*>(p.z + t * p.ldz + n) = make_uint2(pack_bf16x2(f.x, f.y), pack_bf16x2(f.z, f.w));
      } else {
        const float e[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float c = p.addend ? __uint_as_float(static_cast<uint32_t>(p.addend[t * p.ldc + n + k]) << 16) : 0.f;
          p.z[t * p.ldz + n + k] = static_cast<uint16_t>(pack_bf16x2(e[k] + c, 0.f) & 0xFFFFu);
        }
      }
    }
  }
  // a CTA's shared memory stays until every CTA of the cluster has read it
  cluster_sync();
}

// Once per device: shared memory, clusters of up to kMaxSplit CTAs, and how many clusters of each size run at once.
struct FewLimits {
  std::atomic<int> clusters[kMaxSplit + 1];
  std::atomic<bool> ready;
};
template <int FMT>
bsf_status few_limits(const FewLimits** out) {
  static FewLimits limits[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return BSF_ERR_CUDA;
  FewLimits& l = limits[dev];
  if (!l.ready.load(std::memory_order_acquire)) {    // (racing first calls store the same values)
    const void* kernels[2] = {reinterpret_cast<const void*>(few_kernel<FMT, 1>),
                              reinterpret_cast<const void*>(few_kernel<FMT, 2>)};
    for (const void* k : kernels)
      if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem) != cudaSuccess ||
          cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) !=
              cudaSuccess)
        return BSF_ERR_CUDA;
    if (cudaFuncSetAttribute(kernels[1], cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
      return BSF_ERR_CUDA;
    for (int i = 1; i <= kMaxSplit; ++i) {
      DependentLaunch launch(i, kThreads, kMostSmem, nullptr, i);
      launch.cfg.numAttrs = 1;                       // the cluster alone
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, kernels[1], &launch.cfg) != cudaSuccess) {
        cudaGetLastError();
        n = 0;
      }
      l.clusters[i].store(n, std::memory_order_relaxed);
    }
    l.ready.store(true, std::memory_order_release);
  }
  *out = &l;
  return BSF_OK;
}

uint32_t columns_of(int cols) { return cols <= 128 ? 128 : cols <= 256 ? 256 : 512; }

int64_t part_floats(int64_t rows, int64_t width) { return kParts * rows * 2 * width; }

bool few_sizes(int64_t T, int64_t kr, int64_t I, int64_t S) {
  return T >= 0 && T <= kMaxTokens && kr >= 1 && kr <= kMaxKr && I >= 1 && I <= kMaxRowWidth && S >= 0 && S <= kMaxRowWidth;
}

// 16 KB boxes of weights [rows, inner bytes]
bool make_weight_map(CUtensorMap* map, const void* w, int64_t rows, int64_t bytes, bool tiled) {
  return tiled ? make_map(map, w, rows * (bytes / 128), 128, 128) : make_map(map, w, rows, bytes, 128);
}

template <int FMT>
bsf_status launch_few(FewArgs a, const void* w13, const int32_t* sf13, const void* w2, const int32_t* sf2,
                      const void* w13_shared, const int32_t* sf13_shared, const void* w2_shared,
                      const int32_t* sf2_shared, cudaStream_t s) {
  const FewLimits* limits;
  const bsf_status st = few_limits<FMT>(&limits);
  if (st != BSF_OK) return st;
  constexpr int kSize = FMT == kFp8 ? 1 : 2;
  const int sms = sm_count();
  a.nkb1 = a.K * kSize / 128;
  a.nkb2 = a.I * kSize / 128;
  a.nkb2_shared = a.S * kSize / 128;
  a.ctas1 = sms;
  // operand rows of either kernel's terms (one term of bf16 takes whole groups of 16 tokens)
  const int groups = (a.T + 7) / 8 * 8;
  const int rows1 = FMT == kFp8 ? 2 * groups : (a.T + 15) / 16 * 16, rows2 = ((FMT == kFp8 ? 3 : 2) * groups + 15) / 16 * 16;
  const int tables = kBarBytes + kMaxStages * kSfBytes + ((a.E < a.R ? a.E : a.R) + 1) * 8 + a.R * 5;
  a.tables = (tables + 1023) / 1024 * 1024;

  a.stage_space = kStages1 * (2 * kBoxBytes + (rows1 * 128 + 1023) / 1024 * 1024);
  const int space2 = kMostSmem - a.tables;

  // The second kernel: a CTA takes two 128-row tiles of W2, for which the token operand is formed once (one where K is
  // so small that there would be few CTAs), and an SM to itself: 5 stages in each of 96 SMs draw more from HBM than 2 or
  // 3 in twice as many CTAs (32 tokens of 128 experts, K 4096, I 1536: 304 us against 322; 1 token 33.5 against 34.0), and
  // one round of CTAs more than two.  So the contraction is split as far as all clusters surely run at once.
  const int tiles = a.K / 128;
  a.nbox = (tiles + 1) / 2 * kMaxSplit >= 96 ? 2 : 1;
  const int clusters = (tiles + a.nbox - 1) / a.nbox;
  const int64_t most = static_cast<int64_t>(a.E < a.R ? a.E : a.R) * a.nkb2 + a.nkb2_shared;   // K-blocks
  a.split = 1;
  for (int i = 2; i <= kMaxSplit && i <= most; ++i)
    if (limits->clusters[i].load(std::memory_order_relaxed) > clusters) a.split = i;

  CUtensorMap m13, m2, s13, s2;
  if (!make_weight_map(&m13, w13, static_cast<int64_t>(a.E) * 2 * a.I, static_cast<int64_t>(a.K) * kSize, a.tiled) ||
      !make_weight_map(&m2, w2, static_cast<int64_t>(a.E) * a.K, static_cast<int64_t>(a.I) * kSize, a.tiled))
    return BSF_ERR_CUDA;
  s13 = m13;
  s2 = m2;
  if (a.S && (!make_weight_map(&s13, w13_shared, 2 * static_cast<int64_t>(a.S), static_cast<int64_t>(a.K) * kSize, a.tiled) ||
              !make_weight_map(&s2, w2_shared, a.K, static_cast<int64_t>(a.S) * kSize, a.tiled)))
    return BSF_ERR_CUDA;

  a.sf = sf13;
  a.sf_shared = sf13_shared;
  // at least one set of sums for the most tokens; two CTAs share an SM's tensor memory
  const int stride = (rows1 + 31) / 32 * 32;
  a.tmem_cols = columns_of(kAccCol + (kAccCol + 4 * stride <= 256 ? 4 : 2) * stride);
  void* args1[] = {&m13, &s13, &a};
  const bsf_status first = launch_cluster(reinterpret_cast<const void*>(few_kernel<FMT, 1>), a.ctas1, kThreads, a.tables + a.stage_space, 0, s, args1);
  if (first != BSF_OK) return first;
  FewArgs b = a;
  b.stage_space = space2;
  b.sf = sf2;
  b.sf_shared = sf2_shared;
  b.tmem_cols = columns_of(kAccCol + 2 * ((rows2 + 31) / 32 * 32));
  void* args2[] = {&m2, &s2, &b};
  return launch_cluster(reinterpret_cast<const void*>(few_kernel<FMT, 2>), clusters * b.split, kThreads, a.tables + space2, b.split, s, args2);
}

}  // namespace
}  // namespace bsf

using namespace bsf;

extern "C" size_t bsf_few_token_moe_workspace_bytes(int64_t T, int64_t kr, int64_t I, int64_t S) {
  if (!few_sizes(T, kr, I, S)) return 0;
  return static_cast<size_t>(part_floats(T * kr, I) + part_floats(T, S)) * 4 + 16;
}

extern "C" bsf_status bsf_few_token_moe(const void* x, int64_t T, int64_t K, int64_t ldx, const int32_t* topk_ids,
                                        const float* topk_weights, int64_t kr, int64_t E, int64_t I, int weight_type,
                                        const void* w13, const int32_t* sfb13, const void* w2, const int32_t* sfb2,
                                        int64_t S, const void* w13_shared, const int32_t* sfb13_shared,
                                        const void* w2_shared, const int32_t* sfb2_shared, const void* addend,
                                        int64_t ldc, void* z, int64_t ldz, void* workspace, size_t workspace_bytes,
                                        int flags, bsf_stream_t stream) {
  if (T < 0 || K <= 0 || kr <= 0 || E <= 0 || I <= 0 || S < 0) return BSF_ERR_INVALID_ARGUMENT;
  if (K % 128 || I % 128 || S % 128) return BSF_ERR_INVALID_ARGUMENT;
  if (weight_type != BSF_TYPE_E4M3 && weight_type != BSF_TYPE_BF16) return BSF_ERR_INVALID_ARGUMENT;
  if (flags & ~(BSF_B_TILED | BSF_DEBUG_WITHHOLD_LOADS)) return BSF_ERR_INVALID_ARGUMENT;
  if (T > kMaxTokens || kr > kMaxKr || E > kMaxExperts || K > kMaxRowWidth / 2 || !few_sizes(T, kr, I, S))
    return BSF_ERR_UNSUPPORTED;
  if (T == 0) return BSF_OK;
  const bool fp8 = weight_type == BSF_TYPE_E4M3;
  if (!x || !topk_ids || !topk_weights || !w13 || !w2 || !z || !workspace) return BSF_ERR_INVALID_ARGUMENT;
  if (fp8 && (!sfb13 || !sfb2)) return BSF_ERR_INVALID_ARGUMENT;
  if (S && (!w13_shared || !w2_shared || (fp8 && (!sfb13_shared || !sfb2_shared)))) return BSF_ERR_INVALID_ARGUMENT;
  if (ldx < K || ldz < K || (addend && ldc < K)) return BSF_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < bsf_few_token_moe_workspace_bytes(T, kr, I, S)) return BSF_ERR_INVALID_ARGUMENT;
  if (!aligned16(x) || ldx % 8 || !aligned16(w13) || !aligned16(w2) || !aligned16(workspace) ||
      (S && (!aligned16(w13_shared) || !aligned16(w2_shared))))
    return BSF_ERR_MISALIGNED;
  for (const void* q : {static_cast<const void*>(topk_ids), static_cast<const void*>(topk_weights),
                        static_cast<const void*>(sfb13), static_cast<const void*>(sfb2),
                        static_cast<const void*>(sfb13_shared), static_cast<const void*>(sfb2_shared)})
    if (reinterpret_cast<uintptr_t>(q) & 3) return BSF_ERR_MISALIGNED;
  if ((reinterpret_cast<uintptr_t>(z) & 1) || (reinterpret_cast<uintptr_t>(addend) & 1)) return BSF_ERR_MISALIGNED;
  if (ldx > kMaxRowWidth || ldz > kMaxRowWidth || (addend && ldc > kMaxRowWidth)) return BSF_ERR_UNSUPPORTED;
  // weight rows x K-blocks are the boxes' coordinates, K-blocks over all CTAs the units: both 32-bit
  const int64_t per_k = (fp8 ? K : 2 * K) / 128;
  if (!fits_weights(E, 2 * I, 2 * K) || E * I + S > kMaxRows || 2 * (E * I + S) * per_k > INT32_MAX / 2)
    return BSF_ERR_UNSUPPORTED;
  FewArgs a = {};
  a.err = device_error_ptr();
  if (!a.err) return BSF_ERR_CUDA;
  a.x = static_cast<const uint16_t*>(x);
  a.ldx = ldx;
  a.ids = topk_ids;
  a.weights = topk_weights;
  a.part = static_cast<float*>(workspace);
  a.part_shared = a.part + part_floats(T * kr, I);
  a.addend = static_cast<const uint16_t*>(addend);
  a.ldc = ldc;
  a.z = static_cast<uint16_t*>(z);
  a.ldz = ldz;
  a.T = static_cast<int>(T);
  a.kr = static_cast<int>(kr);
  a.E = static_cast<int>(E);
  a.R = static_cast<int>(T * kr);
  a.K = static_cast<int>(K);
  a.I = static_cast<int>(I);
  a.S = static_cast<int>(S);
  a.tiled = (flags & BSF_B_TILED) != 0;
  a.withhold = (flags & BSF_DEBUG_WITHHOLD_LOADS) != 0;
  a.vec4 = (reinterpret_cast<uintptr_t>(z) & 7) == 0 && ldz % 4 == 0 &&
           (!addend || ((reinterpret_cast<uintptr_t>(addend) & 7) == 0 && ldc % 4 == 0));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return fp8 ? launch_few<kFp8>(a, w13, sfb13, w2, sfb2, w13_shared, sfb13_shared, w2_shared, sfb2_shared, s)
             : launch_few<kBf16>(a, w13, sfb13, w2, sfb2, w13_shared, sfb13_shared, w2_shared, sfb2_shared, s);
}
