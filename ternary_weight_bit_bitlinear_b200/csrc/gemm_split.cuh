// gemm_split.cuh -- the ternary product of bitlinear_linear on the
// 5th-generation tensor cores: CTA pairs, split over K inside clusters.
//
// A tile is 256 weight rows x BN tokens.  A pair of CTAs (two SMs) multiplies
// it with tcgen05.mma.cta_group::2, 128 rows in each CTA's tensor memory and
// half of the activations in each CTA's shared memory.  The S pairs of a
// cluster take one tile together: pair k multiplies its share of K, the
// partial sums (int32: their order does not matter) are exchanged through
// distributed shared memory, and pair k finishes BN / S of the tile's tokens.
// Few tiles then still use every SM, and the epilogue is shared too.
//
// Per CTA, the expanded weights live in tensor memory, as in gemm_small.cuh:
//   warp 0       TMA producer: per stage one box of 128 weight rows x G
//                k-blocks (32 packed bytes each, swizzled) and G activation
//                tiles (BN / 2 x 128 int8, 128-byte swizzle);
//   warps 6-13   unpackers, two groups of four (one warp per tensor memory
//                lane quarter, one weight row per lane), stages taken in turn:
//                2-bit fields to 64 (codes+1) in registers, tcgen05.st into
//                the stage's A slot;
//   warp 1       MMA issue, in the even CTA of each pair (whole warp, an
//                elected lane issues): A from both tensor memories, B from
//                both rings; accumulators double-buffered;
//   warps 2-5    epilogue, one per lane quarter: partial sums to the other
//                pairs' CTAs with the same rows, theirs added, then bias,
//                activation, residual and stores (epilogue.cuh).
//
// Why pairs: one CTA per 128-row tile was bound by what TMA brings in (45-50
// bytes a cycle and SM: 12 KB a k-block at 64 tokens, 20 KB at 128); a pair
// brings each activation tile into one of its two CTAs only, and one MMA
// instruction serves both.
//
// The fields are left at the top of their bytes, as unsigned 64 (code + 1):
// shifts to the left run on the FMA pipe, so the masks alone load the integer
// pipe (seven operations there per 16 weights with the fields at the bottom).
// The sums are multiples of 64 and stay in int32: |sum| <= 128 * 128 * K <=
// 2^31 for K <= 131072, reached on the negative side only.
//
// Every wait is bounded (SplitParams::wait_ns).  The CTAs of a cluster meet
// at a cluster barrier before any of them exits, whether or not a wait gave
// up, so nothing arrives in a CTA's shared memory after it is gone.
#pragma once

#include "gemm.cuh"

namespace bl {

constexpr int kSplitGroups = 2;
constexpr int kSplitThreads = (6 + 4 * kSplitGroups) * 32;
constexpr int kSplitMaxPairs = 4;                              // pairs per cluster
constexpr uint32_t kSplitTmemCols = 512;

struct SplitParams {
  CUtensorMap tmA[kGemmMaxProblems];   // packed weights [M][row bytes], box 32 G x 128
  CUtensorMap tmB[kGemmMaxProblems];   // xq [N][K], box 128 x BN / 2
  GemmProblem prob[kGemmMaxProblems];
  Epilogue ep[kGemmMaxProblems];
  int num_problems;
  int total_tiles;
  unsigned long long wait_ns;
};

// A stage is G k-blocks of one tile.  It takes a place in the shared-memory
// ring (packed weights and activations) and an A slot in tensor memory; both
// are free again when its MMAs are done, which one commit tells (a commit
// costs the issuing warp about as much as three MMAs).
__host__ __device__ constexpr int split_stage_kb(int BN) { return BN <= 64 ? 4 : 2; }
template <int BN>
struct SplitCfg {
  static constexpr int G = split_stage_kb(BN);
  static constexpr int kStages = BN <= 64 ? 5 : 6;
  static constexpr int kSlotCols = 32 * G;                     // tensor-memory columns per slot
  static constexpr int kSlots = (static_cast<int>(kSplitTmemCols) - 2 * BN) / kSlotCols;
};

template <int BN>
struct SplitSmem {
  using C = SplitCfg<BN>;
  // multiples of 1024 bytes up to recv
  uint8_t apk[C::kStages][C::G * kGemmBM * kGemmPackedRowBytes];
  uint8_t b[C::kStages][C::G][BN / 2 * kGemmBK];
  // partial sums from the other CTAs of the cluster, four tokens together:
  // [source][token / 4][row], (S - 1) * (BN / S) tokens in all
  int4 recv[BN * (kSplitMaxPairs - 1) / kSplitMaxPairs / 4][kGemmBM];
  float ep_out[4][16 * 32];
  float ep_scale[4][BN];            // per epilogue warp: alpha * amax / 127
  int ep_xsum[4][BN];               // per epilogue warp: activation sums
  uint64_t pfull[C::kStages];       // this CTA's packed weights landed
  uint64_t bfull[C::kStages];       // even CTA: both halves of the activations landed
  uint64_t ready[C::kStages];       // even CTA: the pair's 8 unpack warps are done, one of
                                    // them having seen bfull (the MMA warp waits once a stage)
  uint64_t done[C::kStages];        // MMA commit, both CTAs: the stage and its A slot are free
  uint64_t tfull[2];                // MMA commit, both CTAs
  uint64_t tempty[2];               // even CTA: the pair's 8 epilogue warps
  uint64_t rfull[4];                // per lane quarter: bytes of the S - 1 other CTAs' sums
  uint64_t rempty[4];               // per lane quarter: S - 1 other CTAs have read this one's
  uint64_t join[4];                 // per lane quarter: the last accumulator may be read
  uint64_t drain;                   // MMA commit, both CTAs
  uint32_t tmem_slot;
  int abort;
};
static_assert(sizeof(SplitSmem<32>) + 1024 <= 232448, "shared memory");
static_assert(sizeof(SplitSmem<64>) + 1024 <= 232448, "shared memory");
static_assert(sizeof(SplitSmem<128>) + 1024 <= 232448, "shared memory");

// Stages [first, last) of the tile's K that pair `rank` of `S` takes; k-blocks
// in all.
struct SplitRange {
  int first, last, kblocks;
};
template <int G>
__device__ __forceinline__ SplitRange split_range(int K, int rank, int S) {
  const int kb = (K + kGemmBK - 1) / kGemmBK;
  const int n = (kb + G - 1) / G;
  return {n * rank / S, n * (rank + 1) / S, kb};
}

template <int BN>
__global__ void __launch_bounds__(kSplitThreads, 1)
gemm_split_kernel(const __grid_constant__ SplitParams p) {
  extern __shared__ uint8_t smem_raw[];
  using C = SplitCfg<BN>;
  using Smem = SplitSmem<BN>;
  constexpr int G = C::G;
  constexpr uint32_t kAColBase = 2 * BN;
  const uint32_t base = smem_u32(smem_raw);
  Smem& s = *reinterpret_cast<Smem*>(smem_raw + ((1024u - (base & 1023u)) & 1023u));

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int S = static_cast<int>(cluster_nctarank()) >> 1;   // pairs
  const int rank = static_cast<int>(cluster_ctarank()) >> 1; // this pair
  const int half = static_cast<int>(cluster_ctarank()) & 1;  // this CTA of it
  const int who = static_cast<int>(blockIdx.x) / (2 * S);
  const int nwho = static_cast<int>(gridDim.x) / (2 * S);
  volatile int* abort = &s.abort;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&s.pfull[i], 1);
      mbar_init(&s.bfull[i], 1);
      mbar_init(&s.ready[i], 2 * 4);
      mbar_init(&s.done[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.tfull[i], 1);
      mbar_init(&s.tempty[i], 2 * 4);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s.rfull[i], 1);
      mbar_init(&s.rempty[i], S > 1 ? S - 1 : 1);
      mbar_init(&s.join[i], 1);
    }
    mbar_init(&s.drain, 1);
    s.abort = 0;
    fence_mbar_init();
    for (int i = 0; i < p.num_problems; ++i) {
      tma_prefetch_desc(&p.tmA[i]);
      tma_prefetch_desc(&p.tmB[i]);
    }
  }
  if (warp == 1) {
    tmem_alloc_pair(&s.tmem_slot, kSplitTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();   // every CTA's barriers exist before another one arrives on them
  tc_fence_after();
  const uint32_t tmem_base = s.tmem_slot;
  // The first tile is found before the wait on the preceding kernel (reading
  // the parameters takes 900 cycles the first time), and its first stages'
  // weights go to L2 (a hint: no global memory is read before the wait).
  int tile = who, pi, m_blk, n_blk;
  gemm_locate<BN>(p, tile, pi, m_blk, n_blk);   // who < total_tiles: the grid is no larger
  SplitRange kr = split_range<G>(p.prob[pi].K, rank, S);
  if (threadIdx.x == 0) {
    for (int st = kr.first; st < min(kr.last, kr.first + C::kStages); ++st)
      tma_prefetch_2d(&p.tmA[pi], st * G * kGemmPackedRowBytes,
                      (2 * m_blk + half) * kGemmBM);
  }
  // Moves to this cluster's next tile; false past the last.
  auto next_tile = [&]() {
    tile += nwho;
    if (tile >= p.total_tiles) return false;
    gemm_locate<BN>(p, tile, pi, m_blk, n_blk);
    kr = split_range<G>(p.prob[pi].K, rank, S);
    return true;
  };
  pdl_wait_prior_grid();
  pdl_allow_next_grid();

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    // The two producers of a pair must issue the same loads: the odd CTA's
    // activations complete on the even CTA's barriers, which the even CTA
    // drains.  So they do not follow the CTA's abort flag; both stop at the
    // same stage when the commits (to both CTAs alike) stop.
    const bool leader = elect_one_sync();
    volatile int no_abort = 0;
    uint32_t stage = 0, phase = 0;
    int issued = 0;
    do {
      for (int st = kr.first; st < kr.last; ++st) {
        const int kb0 = st * G, nkb = min(G, kr.kblocks - kb0);
        if (!mbar_wait_warp(&s.done[stage], phase ^ 1u, &no_abort, kDrainLimitNs))
          goto producer_done;
        if (leader) {
          mbar_arrive_expect_tx(&s.pfull[stage], G * (kGemmBM * kGemmPackedRowBytes));
          tma_load_2d(s.apk[stage], &p.tmA[pi], &s.pfull[stage], kb0 * kGemmPackedRowBytes,
                      (2 * m_blk + half) * kGemmBM);
          if (half == 0) mbar_arrive_expect_tx(&s.bfull[stage], nkb * (BN * kGemmBK));
          for (int j = 0; j < nkb; ++j)
            tma_load_2d_pair(s.b[stage][j], &p.tmB[pi], &s.bfull[stage], (kb0 + j) * kGemmBK,
                             n_blk * BN + half * (BN / 2));
        }
        __syncwarp();
        ++issued;
        if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
      }
    } while (next_tile());
  producer_done:
    if (leader) {
      gemm_drain_loads<C::kStages>(s.pfull, issued);
      if (half == 0) gemm_drain_loads<C::kStages>(s.bfull, issued);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (half == 0) {
    const bool leader = elect_one_sync();
    const uint16_t pair_mask = static_cast<uint16_t>(3u << (2 * rank));
    constexpr uint32_t idesc = idesc_u8s8(2 * kGemmBM, BN);
    const uint64_t b_desc0 = smem_desc_k_sw128(smem_u32(s.b[0][0]));
    uint32_t stage = 0, phase = 0, slot = 0;
    int it = 0;
    do {
      const uint32_t db = it & 1, dp = (it >> 1) & 1;
      if (!mbar_wait_warp(&s.tempty[db], dp ^ 1u, abort, p.wait_ns)) break;
      tc_fence_after();
      const uint32_t d_tmem = tmem_base + db * BN;
      bool ok = true;
      for (int st = kr.first; st < kr.last; ++st) {
        const int nkb = min(G, kr.kblocks - st * G);
        if (!mbar_wait_warp(&s.ready[stage], phase, abort, p.wait_ns)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t a_slot = tmem_base + kAColBase + C::kSlotCols * slot;
        const uint64_t bs = b_desc0 + static_cast<uint64_t>((stage * (G * BN / 2 * kGemmBK)) >> 4);
        const uint32_t first = st == kr.first ? 0u : 1u;   // accumulate flag of the first MMA
        // whole stages unrolled with immediate offsets and one condition per MMA
        if (nkb == G) {
#pragma unroll
          for (int j = 0; j < G; ++j)
#pragma unroll
            for (int kk = 0; kk < kGemmBK / 32; ++kk) {
              const uint64_t bd = bs + static_cast<uint64_t>((j * BN / 2 * kGemmBK + 32 * kk) >> 4);
              if (leader)
                mma_i8_ts_pair(d_tmem, a_slot + 32 * j + 8 * kk, bd, idesc,
                               (j | kk) == 0 ? first : 1u);
            }
        } else {
          for (int j = 0; j < nkb; ++j)
#pragma unroll
            for (int kk = 0; kk < kGemmBK / 32; ++kk) {
              const uint64_t bd = bs + static_cast<uint64_t>((j * BN / 2 * kGemmBK + 32 * kk) >> 4);
              if (leader)
                mma_i8_ts_pair(d_tmem, a_slot + 32 * j + 8 * kk, bd, idesc,
                               (j | kk) == 0 ? first : 1u);
            }
        }
        if (leader) mma_commit_mask(&s.done[stage], pair_mask);
        __syncwarp();
        if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
        if (++slot == C::kSlots) slot = 0;
      }
      if (!ok) break;
      if (leader) mma_commit_mask(&s.tfull[db], pair_mask);
      __syncwarp();
      ++it;
    } while (next_tile());
    // Both CTAs learn through `drain` when the pair's last MMAs are done.
    if (leader) mma_commit_mask(&s.drain, pair_mask);
    __syncwarp();
    }
  }

  bool alive = true;   // of the warps from here on: no wait has given up
  int it = 0;          // number of the tile among this cluster's
  const uint32_t quarter = static_cast<uint32_t>(warp & 3);
  if (warp >= 6) {
    // ------------------------------------------------------------ unpackers
    const int group = (warp - 6) >> 2;
    const int u = static_cast<int>(quarter) * 32 + lane;   // weight row within the tile
    // 16-byte chunk c of the row is at c ^ sw (128- or 64-byte swizzle)
    const uint32_t sw = G == 4 ? static_cast<uint32_t>(u & 7) : static_cast<uint32_t>((u >> 1) & 3);
    const uint32_t lane_addr = (quarter * 32u) << 16;
    // The slot of stage number q was stage number q - kSlots' before: free when
    // that one is done, which its place in the ring tells.
    uint32_t stage = 0, phase = 0, slot = 0;
    uint32_t prev = C::kStages - C::kSlots, pphase = 1u;
    int turn = 0;   // group whose stage comes next
    while (true) {
      for (int st = kr.first; st < kr.last; ++st) {
        if (turn == group) {
          if (!mbar_wait_warp(&s.pfull[stage], phase, abort, p.wait_ns) ||
              !mbar_wait_warp(&s.done[prev], pphase, abort, p.wait_ns)) {
            alive = false;
            goto unpack_done;
          }
          tc_fence_after();
          const uint8_t* row = s.apk[stage] + u * (G * kGemmPackedRowBytes);
          uint4 c[2 * G];
#pragma unroll
          for (int q = 0; q < 2 * G; ++q)
            c[q] = *reinterpret_cast<const uint4*>(row + ((static_cast<uint32_t>(q) ^ sw) << 4));
          const uint32_t a_slot = tmem_base + lane_addr + kAColBase + C::kSlotCols * slot;
#pragma unroll
          for (int j = 0; j < G; ++j) {   // k-blocks past K hold zeros: no MMA reads them
            const uint32_t words[8] = {c[2 * j].x,     c[2 * j].y,     c[2 * j].z,
                                       c[2 * j].w,     c[2 * j + 1].x, c[2 * j + 1].y,
                                       c[2 * j + 1].z, c[2 * j + 1].w};
            uint32_t r[32];
#pragma unroll
            for (int w = 0; w < 8; ++w) {   // column 4w + i holds weights 16w + 4i .. +3
              r[4 * w + 0] = (words[w] << 6) & 0xC0C0C0C0u;
              r[4 * w + 1] = (words[w] << 4) & 0xC0C0C0C0u;
              r[4 * w + 2] = (words[w] << 2) & 0xC0C0C0C0u;
              r[4 * w + 3] = words[w] & 0xC0C0C0C0u;
            }
            tmem_st_32x32b_x32(a_slot + 32 * j, r);
          }
          tmem_st_wait();
          if (half == 0 && quarter == 0 &&
              !mbar_wait_warp(&s.bfull[stage], phase, abort, p.wait_ns)) {
            alive = false;
            goto unpack_done;
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(&s.ready[stage], 2 * rank);
        }
        if (++turn == kSplitGroups) turn = 0;
        if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
        if (++prev == C::kStages) { prev = 0; pphase ^= 1u; }
        if (++slot == C::kSlots) slot = 0;
      }
      if (tile + nwho >= p.total_tiles) break;   // the last tile: its epilogue comes next
      ++it;
      next_tile();
    }
  unpack_done:;
  }
  if (warp >= 2 && alive) {
    // ------------------------------------------------------------ epilogue
    // Of the last tile (the only one, where the split leaves each cluster one)
    // the unpack warps take their share: three warps per lane quarter, blocks
    // of 16 tokens in turn.  One warp needs 1400 cycles per block.
    const int own = BN / S;                       // tokens this CTA finishes: a power of two
    const int ls = 31 - __clz(own);
    const int row = static_cast<int>(quarter) * 32 + lane;
    const int part = warp < 6 ? 0 : 1 + ((warp - 6) >> 2);
    // staging block, scales and sums: the unpack warps' in the ring's packed
    // weights, which nothing reads any more once the last accumulator is full
    uint8_t* spare = s.apk[0] + (warp - 6) * (16 * 32 * 4 + BN * 8);
    float* blk = part == 0 ? s.ep_out[quarter] : reinterpret_cast<float*>(spare);
    float* sc = part == 0 ? s.ep_scale[quarter] : reinterpret_cast<float*>(spare + 16 * 32 * 4);
    int* xs = part == 0 ? s.ep_xsum[quarter]
                        : reinterpret_cast<int*>(spare + 16 * 32 * 4 + BN * 4);
    const uint32_t tmem_lane = tmem_base + ((quarter * 32u) << 16);
    do {
      const bool last = tile + nwho >= p.total_tiles;
      const int parts = last ? 1 + kSplitGroups : 1;
      const int t0 = 16 * part;                   // this warp's first block of the CTA's tokens
      const GemmProblem pr = p.prob[pi];
      const Epilogue ep = p.ep[pi];
      const uint32_t db = it & 1, dp = (it >> 1) & 1;
      const uint32_t taddr = tmem_lane + db * BN;
      const int m0 = (2 * m_blk + half) * kGemmBM + static_cast<int>(quarter) * 32;
      const int tok0 = n_blk * BN + rank * own;   // first token this CTA finishes
      const int tend = min(pr.N, tok0 + own);
      // Tokens pair d is sent: those it finishes, in fours, and four at least: a
      // CTA that waited for nothing could run two tiles ahead of the others, and
      // the phases of rempty would be mistaken for one another.
      auto need = [&](int d) {
        return max(4, min(own, (pr.N - n_blk * BN - d * own + 3) & ~3));
      };
      bool armed = false;                         // the bytes to come are announced
      auto announce = [&]() {
        if (lane == 0)
          mbar_arrive_expect_tx(&s.rfull[quarter],
                                static_cast<uint32_t>((S - 1) * need(rank) * 32 * 4));
        armed = true;
      };
      ep_dispatch(ep.dtype, [&](auto type) {
        EpRows<decltype(type), 16> rows;
        rows.begin(ep, m0, pr.M, lane);
        rows.load(ep, tok0 + t0, m0 < pr.M ? tend : 0, rows.res);
        // scale and activation sum of each token, this warp's copy; all loads in
        // flight at once, before the accumulator is waited for
        const float alpha = __ldg(pr.alpha);
        constexpr int kPer = (BN + 31) / 32;
        float am[kPer];
        int xv[kPer];
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          const bool in = tok0 + k * 32 + lane < tend;
          am[k] = in ? __ldg(pr.amax + tok0 + k * 32 + lane) : 0.0f;
          xv[k] = in ? __ldg(pr.xsum + tok0 + k * 32 + lane) : 0;
        }
#pragma unroll
        for (int k = 0; k < kPer; ++k) am[k] = __fmul_rn(alpha, __fdiv_rn(am[k], 127.0f));
        if (part == 0) {
          if (!mbar_wait_warp(&s.tfull[db], dp, abort, p.wait_ns)) {
            alive = false;
            return;
          }
          if (S > 1) {
            announce();
            // the other CTAs have read the sums of the tile before
            if (!mbar_wait_warp(&s.rempty[quarter], static_cast<uint32_t>(it & 1) ^ 1u, abort,
                                p.wait_ns)) {
              alive = false;
              return;
            }
          }
          if (last && lane == 0) mbar_arrive(&s.join[quarter]);
        } else if (!mbar_wait_warp(&s.join[quarter], 0, abort, p.wait_ns)) {
          // (these warps have not followed the phases of the other barriers)
          alive = false;
          return;
        }
        tc_fence_after();
        __syncwarp();
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          sc[k * 32 + lane] = am[k];
          xs[k * 32 + lane] = xv[k];
        }
        __syncwarp();
        if (S > 1) {
#pragma unroll 1
          for (int c0 = t0; c0 < BN; c0 += 16 * parts) {
            if (own >= 16 && (c0 >> ls == rank || (c0 & (own - 1)) >= need(c0 >> ls))) continue;
            uint32_t r[16];
            tmem_ld_32x32b_x16(taddr + c0, r);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              const int d = (c0 + j) >> ls;
              if (d != rank && ((c0 + j) & (own - 1)) < need(d))
                st_async_v4(&s.recv[(((rank < d ? rank : rank - 1) << ls) +
                                     ((c0 + j) & (own - 1))) >> 2][row],
                            &s.rfull[quarter], 2 * d + half, r[j], r[j + 1], r[j + 2], r[j + 3]);
            }
          }
          if (!mbar_wait_warp(&s.rfull[quarter], static_cast<uint32_t>(it & 1), abort,
                              p.wait_ns)) {
            alive = false;
            return;
          }
        }
#pragma unroll 1
        for (int t = t0; t < own; t += 16 * parts) {
          const int n0 = tok0 + t;
          if (n0 >= tend || m0 >= pr.M) break;    // nothing to store from here on
          const int c0 = (rank * own + t) & ~15, off = (rank * own + t) & 15;
          uint32_t r[16];
          tmem_ld_32x32b_x16(taddr + c0, r);
          tmem_ld_wait();
          __syncwarp();                           // the block's last values have been read
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const int q = j - off;                // tokens q .. q + 3 of the block
            if (q >= 0 && q < own) {
              int4 a = make_int4(static_cast<int>(r[j]), static_cast<int>(r[j + 1]),
                                 static_cast<int>(r[j + 2]), static_cast<int>(r[j + 3]));
              for (int o = 0; o < S - 1; ++o) {
                const int4 v = s.recv[((o << ls) + t + q) >> 2][row];
                a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
              }
              const int4 x = *reinterpret_cast<const int4*>(xs + t + q);
              const float4 f = *reinterpret_cast<const float4*>(sc + t + q);
              float* o = blk + q * 32 + lane;
              o[0] = __fmul_rn(__int2float_rn((a.x >> 6) - x.x), f.x);
              o[32] = __fmul_rn(__int2float_rn((a.y >> 6) - x.y), f.y);
              o[64] = __fmul_rn(__int2float_rn((a.z >> 6) - x.z), f.z);
              o[96] = __fmul_rn(__int2float_rn((a.w >> 6) - x.w), f.w);
            }
          }
          __syncwarp();
          uint4 next[decltype(rows)::kIters] = {};
          if (t + 16 * parts < own) rows.load(ep, n0 + 16 * parts, tend, next);
          rows.finish(ep, blk, n0, tend, pr.M);
#pragma unroll
          for (int q = 0; q < decltype(rows)::kIters; ++q) rows.res[q] = next[q];
        }
        if (!last) {   // nobody waits for these after the last tile
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(&s.tempty[db], 2 * rank);
          if (S > 1 && lane < S && lane != rank)
            mbar_arrive_cluster(&s.rempty[quarter], 2 * lane + half);
        }
      });
      if (!alive) {
        // Given up: what the other CTAs may still send has landed before this one
        // exits, or they have given up too.
        if (part == 0 && S > 1) {
          if (!armed) announce();
          mbar_drain(&s.rfull[quarter], static_cast<uint32_t>(it & 1));
        }
        break;
      }
      ++it;
    } while (next_tile());
  }

  // The pair's last MMAs write both tensor memories and read both shared
  // memories: each CTA waits for them, then all meet before anything is freed.
  // (The arrival need not wait for this CTA's stores: what other CTAs were sent
  // they have waited for.)
  if (warp == 1 && lane == 0) mbar_drain(&s.drain, 0);
  tc_fence_before();
  cluster_sync_relaxed();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc_pair(tmem_base, kSplitTmemCols);
  }
}

}  // namespace bl
