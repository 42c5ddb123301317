// gemm_experts.cuh -- one tcgen05 GEMM over all experts of a mixture-of-experts layer: sorted row i
// of expert e times W_e, Y[i, :] = bf16(A[i, :] W_e^T), in MXFP4 (kind::mxf4nvf4, scale_vec::2X)
// or BF16 (kind::f16), fp32 accumulation in tensor memory.
//
// Work split: persistent, warp-specialised, as k_gemm, by one CTA (CG = 1: tiles of 128 rows x 256
// columns) or a pair of CTAs (CG = 2: 256 x 256; each CTA holds its 128 rows of A and of the
// accumulator and half of B's columns, so a tile's operands cross from L2 to shared memory a third
// less often per flop). A tile never spans two experts. The number of tiles and their experts come
// from the plan in device memory, so no launch parameter depends on the routing.
//
// A group's last tile reads rows of the next expert (or, past the last row, the map's zero fill);
// an accumulator row depends on its own A row alone, and rows behind the group's end are not
// stored, so those operands reach no result.
//
// Warps (15 per CTA): 0 TMA producer (A, B, A's scale atoms); 1 MMA issue (the pair's first CTA),
// TMEM allocation; 2 B's scale atoms (MXFP4), or the relay of the pair's second CTA (BF16); 3..6
// scale writers, shared memory -> TMEM (MXFP4); 7..14 epilogue.
// Barriers per stage: full (this CTA's copies landed), ready (in the issuing CTA: the stage may be
// used: every scale writer of the pair has stored its quarter, or, BF16 pairs, both CTAs' copies
// landed), empty (the MMAs that read the stage are done; tcgen05.commit signals both CTAs).
// TMEM (512 columns): MXFP4 256 for the accumulator, from column 256 on one 32-column scale set per
// stage; the two K = 64 steps of a scale atom share the 32-bit cells and select their half by the
// instruction's scale-factor id: B's cells at 8 (step / 2), A's at 16 + 4 (step / 2) + quarter.
// BF16: two accumulators.
// Every wait is bounded, as in k_gemm.
#pragma once

#include "experts.cuh"
#include "gemm.cuh"

namespace arc {

template <int KIND, int CG>
struct ExpertGemmTraits {
  static constexpr bool MX4 = KIND == kGemmMX4;
  static constexpr int BM = 128, BN = 256, TM = BM * CG, B_ROWS = BN / CG;
  static constexpr int A_BYTES = BM * 128, B_BYTES = B_ROWS * 128;
  static constexpr int SFA_BYTES = MX4 ? 2 * 512 : 0, SFB_BYTES = MX4 ? 2 * 2 * 512 : 0;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + SFA_BYTES + SFB_BYTES;
  static constexpr int STAGES = CG == 2 ? 6 : 4;
  static constexpr int ACC_STAGES = MX4 ? 1 : 2;
  static constexpr int SF_COL0 = 256, SF_SET_COLS = 32;
  static constexpr uint32_t IDESC = MX4 ? idesc_mxf4(TM, BN) : idesc_bf16(TM, BN);
  // scale-factor ids of the second K = 64 step of an atom (bytes 2 and 3 of a cell)
  static constexpr uint32_t IDESC_ODD = IDESC | (MX4 ? (2u << 29) | (2u << 4) : 0u);
};

// Shared memory behind the stages: staging 8 x 1 KB, barriers 256 B, first tile of every expert.
template <int KIND, int CG>
constexpr int expert_gemm_smem_bytes(int experts) {
  return ExpertGemmTraits<KIND, CG>::STAGES * ExpertGemmTraits<KIND, CG>::STAGE_BYTES + 8 * kEpiStageBytes + 256 +
         (experts + 1) * 4 + 1024;
}

struct ExpertGemmArgs {
  Plan p;
  int experts;
  int N;
  int ksteps, kstages, katoms;
  int nblk128;  // 128-row blocks of one expert's B scales
  int tiles_n;
  int group_m;
  int box_rows_a, box_rows_b;
  const uint8_t* sfa;
  const uint8_t* sfb;
  __nv_bfloat16* y;
  int64_t ldy;
  uint64_t wait_ns;
  int inject;
};

// ---- cluster and cta_group::2 forms

__device__ __forceinline__ uint32_t cluster_cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Arrive on the barrier at the same place in CTA `rank` of the cluster.
__device__ __forceinline__ void mbar_arrive_cta(uint64_t* bar, uint32_t rank) {
  asm volatile(
      "{\n\t.reg .b32 ra;\n\t"
      "mapa.shared::cluster.u32 ra, %0, %1;\n\t"
      "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [ra];\n\t}\n" ::"r"(smem_u32(bar)),
      "r"(rank)
      : "memory");
}

template <int CG>
__device__ __forceinline__ void tmem_alloc_cg(uint32_t* dst_smem, uint32_t ncols) {
  if constexpr (CG == 1) {
    tmem_alloc(dst_smem, ncols);
    tmem_relinquish();
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void tmem_dealloc_cg(uint32_t taddr, uint32_t ncols) {
  if constexpr (CG == 1)
    tmem_dealloc(taddr, ncols);
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// Commit to this CTA's barrier alone.
template <int CG>
__device__ __forceinline__ void tc_commit_own(uint64_t* bar) {
  if constexpr (CG == 1)
    tc_commit(bar);
  else
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
// Commit to the barrier (of both CTAs of a pair).
template <int CG>
__device__ __forceinline__ void tc_commit_cg(uint64_t* bar) {
  if constexpr (CG == 1)
    tc_commit(bar);
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

template <int KIND, int CG>
__device__ __forceinline__ void expert_mma(uint32_t d_tmem, uint64_t da, uint64_t db, uint32_t sf, int k,
                                           uint32_t accum) {
  using T = ExpertGemmTraits<KIND, CG>;
  if constexpr (T::MX4) {
    const uint32_t idesc = (k & 1) ? T::IDESC_ODD : T::IDESC;
    const uint32_t sfa = sf + 16 + 4 * (k >> 1), sfb = sf + 8 * (k >> 1);
    if constexpr (CG == 1) {
      tc_mma_mxf4(d_tmem, da, db, idesc, sfa, sfb, accum);
    } else {
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "setp.ne.b32 p, %4, 0;\n\t"
          "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}\n" ::
              "r"(d_tmem),
          "l"(da), "l"(db), "r"(idesc), "r"(accum), "r"(sfa), "r"(sfb)
          : "memory");
    }
  } else {
    if constexpr (CG == 1) {
      tc_mma_bf16(d_tmem, da, db, T::IDESC, accum);
    } else {
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "setp.ne.b32 p, %4, 0;\n\t"
          "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
          "l"(da), "l"(db), "r"(T::IDESC), "r"(accum)
          : "memory");
    }
  }
}

__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// Where tile t lies. first[e] = tiles of all column blocks before expert e, in row tiles.
struct ExpertTile {
  int e, im, tn;  // expert, row tile within it, column tile
};
__device__ __forceinline__ ExpertTile expert_tile(int t, const int* first, int experts, int tiles_n, int group_m) {
  const int q = t / tiles_n;
  int lo = 0, hi = experts;  // the expert with first[e] <= q < first[e + 1]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= q)
      lo = mid;
    else
      hi = mid;
  }
  ExpertTile r;
  r.e = lo;
  tile_coords(t - first[lo] * tiles_n, first[lo + 1] - first[lo], tiles_n, group_m, r.im, r.tn);
  return r;
}

template <int KIND, int CG>
__global__ void __launch_bounds__(kGemmThreads, 1)
    k_gemm_experts(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmY, const ExpertGemmArgs g) {
  using T = ExpertGemmTraits<KIND, CG>;
  constexpr bool MX4 = T::MX4;
  constexpr bool RELAY = !MX4 && CG == 2;  // BF16 pairs: warp 2 hands this CTA's landed copies on
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = smem + T::STAGES * T::STAGE_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + 8 * kEpiStageBytes);
  uint64_t* empty = full + T::STAGES;
  uint64_t* ready = empty + T::STAGES;
  uint64_t* acc_full = ready + T::STAGES;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* first = reinterpret_cast<int*>(staging + 8 * kEpiStageBytes + 256);  // [E + 1]
  static_assert((3 * T::STAGES + 5) * 8 + 8 <= 256, "barriers");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_cta_rank() : 0u;
  const int unit = static_cast<int>(blockIdx.x) / CG, units = static_cast<int>(gridDim.x) / CG;
  if (threadIdx.x == 0) {
    for (int s = 0; s < T::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&ready[s], (MX4 ? 4 : 1) * CG);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], 8 * CG);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmY);
  }
  if (warp == 1) tmem_alloc_cg<CG>(tmem_slot, 512);
  pdl_wait();  // the plan and the operands come from earlier kernels
  if (warp == 2) {
    // first row tile of every expert: exclusive sum of ceil(rows / TM)
    int run = 0;
    for (int e0 = 0; e0 <= g.experts; e0 += 32) {
      const int e = e0 + lane;
      int n = 0;
      if (e < g.experts) n = (g.p.offsets[e + 1] - g.p.offsets[e] + T::TM - 1) / T::TM;
      int inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += v;
      }
      if (e <= g.experts) first[e] = run + inc - n;
      run += __shfl_sync(0xFFFFFFFFu, inc, 31);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync_all();  // the other CTA's barriers are initialised
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int ntiles = first[g.experts] * g.tiles_n;

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------------ producer
      uint32_t stage = 0, phase = 0, armed = 0, armed_par = 0;
      bool skip = (g.inject == 1) && blockIdx.x == 0;
      bool ok = true;
      for (int t = unit; t < ntiles && ok; t += units) {
        const ExpertTile at = expert_tile(t, first, g.experts, g.tiles_n, g.group_m);
        const int off = g.p.offsets[at.e], rows = g.p.offsets[at.e + 1] - off;
        const int blk_in = at.im * CG + static_cast<int>(rank);  // 128-row block within the expert
        const int a_row = off + blk_in * 128;
        const int b_row = at.e * g.N + at.tn * T::BN + static_cast<int>(rank) * T::B_ROWS;
        const bool has_a = blk_in * 128 < rows;  // the pair's second half may lie behind the group
        const int64_t sfa_blk = MX4 ? g.p.blocks[at.e] + blk_in : 0;
        const int nb = MX4 ? min(2, g.nblk128 - 2 * at.tn) : 0;
        for (int ks = 0; ks < g.kstages; ++ks) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, g.wait_ns, abort_flag)) {
            ok = false;
            break;
          }
          uint8_t* sA = smem + stage * T::STAGE_BYTES;
          uint8_t* sB = sA + T::A_BYTES;
          if (skip) {
            skip = false;  // failure injection: this stage's loads are never issued
          } else {
            uint32_t bytes = static_cast<uint32_t>((has_a ? g.box_rows_a : 0) + g.box_rows_b) * 128u;
            int natoms = 0;
            if (MX4) {
              natoms = min(2, g.katoms - 2 * ks);
              bytes += static_cast<uint32_t>(natoms * 512 * ((has_a ? 1 : 0) + nb));
            }
            mbar_arrive_expect_tx(&full[stage], bytes);
            const int kx = MX4 ? ks * 128 : ks * 64;
            if (has_a) tma_load_2d(sA, &tmA, &full[stage], kx, a_row);
            tma_load_2d(sB, &tmB, &full[stage], kx, b_row);
            if (MX4 && has_a)
              bulk_load(sB + T::B_BYTES, g.sfa + (sfa_blk * g.katoms + 2 * ks) * 512, natoms * 512, &full[stage]);
            armed |= 1u << stage;
            armed_par = (armed_par & ~(1u << stage)) | (phase << stage);
          }
          if (++stage == T::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (*abort_flag) {
        // let every load this thread issued land before the CTA goes away
        for (int s = 0; s < T::STAGES; ++s)
          if ((armed >> s) & 1u) mbar_wait_teardown(&full[s], (armed_par >> s) & 1u, g.wait_ns);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      // ------------------------------------------------------------------ MMA issue (as k_gemm)
      uint32_t acc = 0, acc_phase = 0, stage = 0, phase = 0;
      bool ok = true;
      constexpr uint64_t kStageDesc = static_cast<uint64_t>(T::STAGE_BYTES >> 4);
      constexpr uint64_t kBDesc = static_cast<uint64_t>(T::A_BYTES >> 4);
      const uint64_t da0 = desc_kmajor_sw128(smem_u32(smem));
      uint64_t da = da0;
      uint32_t sf = tmem + T::SF_COL0;
      for (int t = unit; t < ntiles && ok; t += units) {
        if (!mbar_wait(&acc_empty[acc], acc_phase ^ 1u, g.wait_ns, abort_flag)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem + acc * T::BN;
        for (int ks = 0; ks < g.kstages; ++ks) {
          if (!mbar_wait(MX4 || CG == 2 ? &ready[stage] : &full[stage], phase, g.wait_ns, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t db = da + kBDesc;
          const uint32_t acc0 = ks > 0 ? 1u : 0u;
          const int nk = MX4 ? min(4, g.ksteps - 4 * ks) : 4;
          if (nk == 4) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              expert_mma<KIND, CG>(d_tmem, da + 2 * k, db + 2 * k, sf, k, k > 0 ? 1u : acc0);
          } else {
            for (int k = 0; k < nk; ++k)
              expert_mma<KIND, CG>(d_tmem, da + 2 * k, db + 2 * k, sf, k, k > 0 ? 1u : acc0);
          }
          tc_commit_cg<CG>(&empty[stage]);
          if (++stage == T::STAGES) {
            stage = 0;
            phase ^= 1u;
            da = da0;
            sf = tmem + T::SF_COL0;
          } else {
            da += kStageDesc;
            sf += T::SF_SET_COLS;
          }
        }
        if (!ok) break;
        tc_commit_cg<CG>(&acc_full[acc]);
        if (++acc == T::ACC_STAGES) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      // nothing issued may still be running when the tensor memory is released
      tc_commit_own<CG>(drain);
      mbar_wait_teardown(drain, 0, g.wait_ns);
    }
  } else if (warp == 2) {
    if (MX4 && lane == 0) {
      // B's scale atoms of every stage (all 256 columns, in both CTAs of a pair)
      uint32_t stage = 0, phase = 0, armed = 0, armed_par = 0;
      bool ok = true;
      for (int t = unit; t < ntiles && ok; t += units) {
        const ExpertTile at = expert_tile(t, first, g.experts, g.tiles_n, g.group_m);
        const int64_t blk = static_cast<int64_t>(at.e) * g.nblk128 + 2 * at.tn;
        const int nb = min(2, g.nblk128 - 2 * at.tn);
        for (int ks = 0; ks < g.kstages; ++ks) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, g.wait_ns, abort_flag)) {
            ok = false;
            break;
          }
          const int natoms = min(2, g.katoms - 2 * ks);
          uint8_t* sSFB = smem + stage * T::STAGE_BYTES + T::A_BYTES + T::B_BYTES + T::SFA_BYTES;
          for (int b = 0; b < nb; ++b)
            bulk_load(sSFB + b * 1024, g.sfb + ((blk + b) * g.katoms + 2 * ks) * 512, natoms * 512, &full[stage]);
          armed |= 1u << stage;
          armed_par = (armed_par & ~(1u << stage)) | (phase << stage);
          if (++stage == T::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (*abort_flag) {
        for (int s = 0; s < T::STAGES; ++s)
          if ((armed >> s) & 1u) mbar_wait_teardown(&full[s], (armed_par >> s) & 1u, g.wait_ns);
      }
    }
    if (RELAY && lane == 0) {
      uint32_t stage = 0, phase = 0;
      bool ok = true;
      for (int t = unit; t < ntiles && ok; t += units) {
        for (int ks = 0; ks < g.kstages; ++ks) {
          if (!mbar_wait(&full[stage], phase, g.wait_ns, abort_flag)) {
            ok = false;
            break;
          }
          mbar_arrive_cta(&ready[stage], 0);
          if (++stage == T::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    }
  } else if (warp < kGemmEpiWarp0) {
    if (MX4) {
      // ------------------------------------------------------------------ scale writers
      const int q = warp & 3;
      const uint32_t lane_base = tmem + (static_cast<uint32_t>(q * 32) << 16);
      uint32_t stage = 0, phase = 0;
      bool ok = true;
      for (int t = unit; t < ntiles && ok; t += units) {
        for (int ks = 0; ks < g.kstages; ++ks) {
          const bool got = mbar_wait(&full[stage], phase, g.wait_ns, abort_flag);
          if (!__all_sync(0xFFFFFFFFu, got)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sSFA = smem_u32(smem + stage * T::STAGE_BYTES + T::A_BYTES + T::B_BYTES);
          const uint32_t sSFB = sSFA + T::SFA_BYTES;
          const uint32_t set = lane_base + T::SF_COL0 + T::SF_SET_COLS * stage;
          const int natoms = min(2, g.katoms - 2 * ks);
          uint32_t v[16], a[2];
#pragma unroll
          for (int at = 0; at < 2; ++at) {
            uint4 b0 = make_uint4(0, 0, 0, 0), b1 = b0;
            a[at] = 0;
            if (at < natoms) {
              b0 = lds_u32x4(sSFB + at * 512 + lane * 16);
              b1 = lds_u32x4(sSFB + 1024 + at * 512 + lane * 16);
              a[at] = lds_u32(sSFA + at * 512 + lane * 16 + 4 * q);
            }
            v[8 * at + 0] = b0.x, v[8 * at + 1] = b0.y, v[8 * at + 2] = b0.z, v[8 * at + 3] = b0.w;
            v[8 * at + 4] = b1.x, v[8 * at + 5] = b1.y, v[8 * at + 6] = b1.z, v[8 * at + 7] = b1.w;
          }
          tmem_st_32x32b_x16(set, v);
          tmem_st_32x32b_x1(set + 16 + q, a[0]);
          tmem_st_32x32b_x1(set + 20 + q, a[1]);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (CG == 2)
              mbar_arrive_cta(&ready[stage], 0);
            else
              mbar_arrive(&ready[stage]);
          }
          if (++stage == T::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    }
  } else {
    // -------------------------------------------------------------------- epilogue (as k_gemm)
    const int q = warp & 3;
    const int half = (warp - kGemmEpiWarp0) >> 2;
    constexpr int HB = T::BN / 2;
    uint8_t* stg = staging + (warp - kGemmEpiWarp0) * kEpiStageBytes;
    uint32_t acc = 0, acc_phase = 0;
    for (int t = unit; t < ntiles; t += units) {
      const ExpertTile at = expert_tile(t, first, g.experts, g.tiles_n, g.group_m);
      const int off = g.p.offsets[at.e], end = g.p.offsets[at.e + 1];
      const int row0 = off + (at.im * CG + static_cast<int>(rank)) * 128 + q * 32;
      const int col0 = at.tn * T::BN + half * HB;
      const int nrows = min(32, end - row0);  // of this warp's 32; may be negative
      const bool got = mbar_wait(&acc_full[acc], acc_phase, g.wait_ns, abort_flag, 64);
      if (!__all_sync(0xFFFFFFFFu, got)) break;
      tc_fence_after();
      uint32_t pk[HB / 2];
      if (nrows > 0) {
        const uint32_t tbase = tmem + (static_cast<uint32_t>(q * 32) << 16) + acc * T::BN + half * HB;
#pragma unroll
        for (int c = 0; c < HB / 32; ++c) {
          uint32_t r[32];
          tmem_ld_32x32b_x32(tbase + c * 32, r);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e)
            pk[16 * c + e] = pack_bf16x2_rn(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 2)
          mbar_arrive_cta(&acc_empty[acc], 0);
        else
          mbar_arrive(&acc_empty[acc]);
      }
      if (nrows == 32) {
        // whole 32 x 16 boxes through the warp's staging chunk, clipped at the last column
#pragma unroll
        for (int c = 0; c < HB / 16; ++c) {
          uint4* dst = reinterpret_cast<uint4*>(stg + lane * 32);
          dst[0] = make_uint4(pk[8 * c], pk[8 * c + 1], pk[8 * c + 2], pk[8 * c + 3]);
          dst[1] = make_uint4(pk[8 * c + 4], pk[8 * c + 5], pk[8 * c + 6], pk[8 * c + 7]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (col0 + 16 * c < g.N) tma_store_2d(&tmY, stg, col0 + 16 * c, row0);
            bulk_commit_group();
            bulk_wait_read_all();
          }
          __syncwarp();
        }
      } else if (lane < nrows) {
        // the group ends inside these rows: only its own are stored
        __nv_bfloat16* yrow = g.y + static_cast<int64_t>(row0 + lane) * g.ldy + col0;
#pragma unroll
        for (int j = 0; j < HB / 8; ++j)
          if (col0 + 8 * j < g.N)
            *reinterpret_cast<uint4*>(yrow + 8 * j) = make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
      }
      __syncwarp();
      if (++acc == T::ACC_STAGES) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (lane == 0) bulk_wait_all();
  }
  __syncthreads();
  if (CG == 2) cluster_sync_all();  // nothing of the pair reads this CTA's memory any more
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_cg<CG>(tmem, 512);
  }
}

}  // namespace arc
