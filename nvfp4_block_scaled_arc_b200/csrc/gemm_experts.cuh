// gemm_experts.cuh -- one tcgen05 GEMM over all experts of a mixture-of-experts layer: sorted row i
// of expert e times W_e, Y[i, :] = bf16(W_e row_i), in MXFP4 (kind::mxf4nvf4, scale_vec::2X) or BF16
// (kind::f16), fp32 accumulation in tensor memory.
//
// Operands: the weights are the MMA's M side (256 output features by a pair of CTAs, 128 each), the
// expert's rows its N side. M has one height, N any multiple of 16 up to 256, so a group of rows
// is cut into ceil(rows / 256) tiles of nearly equal height and costs at most 15 rows more than it
// has; with the rows as M an average of half a tile per expert was multiplied for nothing (13 % at
// 1000 rows an expert), and a single token cost a whole 128-row tile. The pair (cta_group::2) holds
// one copy of the tile's rows between its two CTAs, half each, which takes a third of the operand
// bytes per flop off the L2 -> shared memory path against one CTA alone: that path bounds
// the block-scaled product (about 17 TB/s measured for the whole chip).
// A tile never spans two experts. The number of tiles and their experts come from the plan in
// device memory, so no launch parameter depends on the routing. Copies may reach past the group's
// last row (into the next expert's rows, or the map's zero fill): an accumulator column depends on
// its own row alone, and columns behind the group's end are not stored.
//
// Persistent, warp-specialised (15 warps per CTA): 0 producer (weights and rows by TMA, the rows'
// scale bytes); 1 MMA issue (the pair's first CTA), TMEM allocation; 2 the weights' scale atoms
// (MXFP4), or the relay (BF16); 3..6 scale writers, shared memory -> TMEM (MXFP4); 7..14 epilogue.
// Barriers per stage: full (this CTA's copies landed), ready (in the issuing CTA: the stage may be
// used: every scale writer of the pair has stored its quarter, or, BF16, both CTAs' relays have seen
// their copies land), empty (the MMAs that read the stage are done; tcgen05.commit signals both
// CTAs). Arrivals at the other CTA carry no cluster-scope release: what they announce was
// written by TMA or tcgen05.st, whose completion their sender has waited for, and a release per
// stage made the whole product half as fast (908 against 452 us, 8192 rows x 28672 x 4224).
// TMEM (512 columns): MXFP4 256 for the accumulator, from column 256 on one 32-column scale set per
// stage; the two K = 64 steps of a scale atom share the 32-bit cells and select their half by the
// instruction's scale-factor id: the rows' cells at 8 (step / 2) + row / 32 (lane row % 32, in every
// quarter), the weights' at 16 + 4 (step / 2) + quarter. BF16: two accumulators.
// Epilogue: a TMEM lane is an output feature, a column a row of Y; 16 rows x 32 features are turned on their
// way into shared memory (stmatrix; with 16-bit stores from whole lanes 32768 rows of 512 -> 4096 took 93 us
// instead of 85) and stored by TMA.
// Every wait is bounded, as in k_gemm.
#pragma once

#include "experts.cuh"
#include "gemm.cuh"

namespace arc {

// MAXN: rows of a tile, at most. 256 is the general form; 64 (few rows for each expert, where reading the
// weights is the work) leaves room for more stages in flight and for more accumulators.
// BATCH: chunks of Y that an epilogue warp stages and stores together, one fence and one wait for all. Shallow
// products are bound by their epilogue (MXFP4, one accumulator), so that more of them pay for one
// pipeline stage less; deep ones want the stage.
template <int KIND, int MAXN, int BATCH>
struct ExpertGemmTraits {
  static constexpr bool MX4 = KIND == kGemmMX4;
  static constexpr int BM = 128, TM = 256;  // features of a CTA and of the pair
  static constexpr int TN = MAXN;
  static constexpr int W_BYTES = BM * 128, X_BYTES = TN / 2 * 128;
  static constexpr int SFW_BYTES = MX4 ? 2 * 512 : 0, SFX_BYTES = MX4 ? TN * 8 : 0;
  static constexpr int STAGE_BYTES = (W_BYTES + X_BYTES + SFW_BYTES + SFX_BYTES + 1023) / 1024 * 1024;
  static constexpr int STAGES = TN == 256 ? (MX4 && BATCH > 1 ? 5 : 6) : MX4 ? 9 : 10;
  static constexpr int ACC_STAGES = TN == 256 ? (MX4 ? 1 : 2) : 3;
  static constexpr int SF_COL0 = ACC_STAGES * TN, SF_SET_COLS = 32;
  static constexpr uint32_t IDESC0 = MX4 ? idesc_mxf4(TM, 0) : idesc_bf16(TM, 0);  // N is the tile's
  // scale-factor ids of the second K = 64 step of an atom (bytes 2 and 3 of a cell)
  static constexpr uint32_t ODD_STEP = MX4 ? (2u << 29) | (2u << 4) : 0u;
  static_assert(SF_COL0 + (MX4 ? STAGES * SF_SET_COLS : 0) <= 512, "tensor memory");
};

constexpr int kExpertEpiBytes = 16 * 32 * 2;  // 16 rows of Y x 32 features, one per epilogue warp
// Row maps with boxes of 8, 16, 32, 48 .. 128 rows: a stage copies little more of the tile's rows than
// it has.
constexpr int kRowBoxes = 9;
__host__ __device__ constexpr int row_box_index(int rows) { return rows <= 8 ? 0 : (rows + 15) / 16; }
__host__ __device__ constexpr int row_box_height(int index) { return index == 0 ? 8 : 16 * index; }

constexpr int kExpertBarBytes = 384;

// Shared memory behind the stages: staging, barriers, and every expert's first tile, first row and first
// block of scale bytes.
template <int KIND, int MAXN, int BATCH>
constexpr int expert_gemm_smem_bytes(int experts) {
  using T = ExpertGemmTraits<KIND, MAXN, BATCH>;
  return T::STAGES * T::STAGE_BYTES + 8 * BATCH * kExpertEpiBytes +
         kExpertBarBytes + 3 * (experts + 1) * 4 + 1024;
}

struct ExpertGemmArgs {
  Plan p;
  int experts;
  int N;
  int ksteps, kstages, katoms;
  int nblk128;   // 128-row blocks of one expert's weight scales
  int tiles_w;   // feature tiles of an expert
  int group_m;   // raster: row tiles that a column of feature tiles is walked with
  int box_w;     // weight map's box height
  int64_t sfx_rows;  // rows of the scale layout
  const uint8_t* sfx;
  const uint8_t* sfw;
  __nv_bfloat16* y;
  int64_t ldy;
  int64_t slots;
  uint64_t wait_ns;
  int inject;
};

struct ExpertRowMaps {
  CUtensorMap box[kRowBoxes];
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
      "mbarrier.arrive.shared::cluster.b64 _, [ra];\n\t}\n" ::"r"(smem_u32(bar)),
      "r"(rank)
      : "memory");
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// Commit to this CTA's barrier alone, and to the barrier of both CTAs.
__device__ __forceinline__ void tc_commit_own(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

template <class T>
__device__ __forceinline__ void expert_mma(uint32_t d_tmem, uint64_t dw, uint64_t dx, uint32_t idesc, uint32_t sf,
                                           int k, uint32_t accum) {
  if constexpr (T::MX4) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}\n" ::
            "r"(d_tmem),
        "l"(dw), "l"(dx), "r"((k & 1) ? idesc | T::ODD_STEP : idesc), "r"(accum), "r"(sf + 16 + 4 * (k >> 1)),
        "r"(sf + 8 * (k >> 1))
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(dw), "l"(dx), "r"(idesc), "r"(accum)
        : "memory");
  }
}

__device__ __forceinline__ void lds_u32x2(uint32_t addr, uint32_t& a, uint32_t& b) {
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(a), "=r"(b) : "r"(addr));
}
// Four 8 x 8 matrices of 16-bit values, transposed: lane 8 i + r gives the address of matrix i's column r.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}

__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// 16 lanes x 16 consecutive 32-bit columns: lane t of the warp gets, in r[4 c + 2 h] and the next, columns
// 8 c + 2 (t % 4) and the next of TMEM lane t / 4 + 8 h.
__device__ __forceinline__ void tmem_ld_16x256b_x2(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

// Where tile t lies: expert, feature tile, first row within the expert, rows of the expert from
// there on, and the MMA's N (a multiple of 16). first[e] = row tiles before expert e.
struct ExpertTile {
  int e, tw, row, left, n;
};
__device__ __forceinline__ ExpertTile expert_tile(int t, const int* first, const int* offsets, int experts, int tiles_w,
                                                  int group_m) {
  const int q = t / tiles_w;
  int lo = 0, hi = experts;  // the expert with first[e] <= q < first[e + 1]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= q)
      lo = mid;
    else
      hi = mid;
  }
  const int nt = first[lo + 1] - first[lo], rows = offsets[lo + 1] - offsets[lo];
  const int height = ((rows + nt - 1) / nt + 15) & ~15;  // at most 256; (nt - 1) * height < rows
  ExpertTile r;
  int im;
  r.e = lo;
  tile_coords(t - first[lo] * tiles_w, nt, tiles_w, group_m, im, r.tw);
  r.row = im * height;
  r.left = rows - r.row;
  r.n = min(height, (r.left + 15) & ~15);
  return r;
}

template <int KIND, int MAXN, int BATCH>
__global__ void __launch_bounds__(kGemmThreads, 1)
    k_gemm_experts(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ ExpertRowMaps tmX,
                   const __grid_constant__ CUtensorMap tmY, const ExpertGemmArgs g) {
  using T = ExpertGemmTraits<KIND, MAXN, BATCH>;
  constexpr bool MX4 = T::MX4;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = smem + T::STAGES * T::STAGE_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + 8 * BATCH * kExpertEpiBytes);
  uint64_t* empty = full + T::STAGES;
  uint64_t* ready = empty + T::STAGES;
  uint64_t* acc_full = ready + T::STAGES;
  uint64_t* acc_empty = acc_full + T::ACC_STAGES;
  uint64_t* drain = acc_empty + T::ACC_STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* first = reinterpret_cast<int*>(staging + 8 * BATCH * kExpertEpiBytes + kExpertBarBytes);  // [E + 1]
  int* offsets = first + g.experts + 1;                                                          // [E + 1]
  int* blocks = offsets + g.experts + 1;                                                         // [E + 1]
  static_assert((3 * T::STAGES + 2 * T::ACC_STAGES + 1) * 8 + 8 <= kExpertBarBytes, "barriers");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_cta_rank();
  const int unit = static_cast<int>(blockIdx.x >> 1), units = static_cast<int>(gridDim.x >> 1);
  if (threadIdx.x == 0) {
    for (int s = 0; s < T::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&ready[s], MX4 ? 8 : 2);
    }
    for (int a = 0; a < T::ACC_STAGES; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], 16);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmY);
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the other CTA's barriers are initialised
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();  // the plan and the operands come from earlier kernels
  // A buffer that no plan was written to is reported and has no tiles.
  bool bad = false;
  for (int e = threadIdx.x; e <= g.experts; e += kGemmThreads) {
    const int at = g.p.offsets[e], next = g.p.offsets[min(e + 1, g.experts)], blk = MX4 ? g.p.blocks[e] : 0;
    offsets[e] = at;
    blocks[e] = blk;
    bad |= at < 0 || next < at || next > g.slots;
    if (MX4 && !bad) bad = blk < 0 || 128ll * (blk + static_cast<int64_t>((next - at + 127) / 128)) > g.sfx_rows;
  }
  bad = __syncthreads_or(bad);
  if (bad && threadIdx.x == 0) set_status(kStatusInvalidArg);
  if (warp == 2) {
    // first row tile of every expert: exclusive sum of ceil(rows / TN)
    int run = 0;
    for (int e0 = 0; e0 <= g.experts; e0 += 32) {
      const int e = e0 + lane;
      const int n = e < g.experts ? (offsets[e + 1] - offsets[e] + T::TN - 1) / T::TN : 0;
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
  __syncthreads();
  const int ntiles = bad ? 0 : first[g.experts] * g.tiles_w;
  auto tile = [&](int t) { return expert_tile(t, first, offsets, g.experts, g.tiles_w, g.group_m); };

  if (warp == 0) {
    // -------------------------------------------------------------------- producer
    uint32_t stage = 0, phase = 0, armed = 0, armed_par = 0;
    bool skip = (g.inject == 1) && blockIdx.x == 0;
    bool ok = true;
    for (int t = unit; t < ntiles && ok; t += units) {
      const ExpertTile at = tile(t);
      const int w_row = at.e * g.N + at.tw * T::TM + static_cast<int>(rank) * T::BM;
      const int x_row = offsets[at.e] + at.row + static_cast<int>(rank) * (at.n >> 1);
      const int bi = row_box_index(at.n >> 1);  // the smallest box that holds the CTA's half
      const int box_x = static_cast<int>(min(static_cast<int64_t>(row_box_height(bi)), g.slots));
      const CUtensorMap* map_x = &tmX.box[bi];
      const bool has_sfw = MX4 && 2 * at.tw + static_cast<int>(rank) < g.nblk128;
      const uint8_t* sfx = MX4 ? g.sfx + (128ll * blocks[at.e] + at.row) * 8 : nullptr;
      const uint32_t bytes0 =
          static_cast<uint32_t>(g.box_w + box_x) * 128u + (MX4 ? static_cast<uint32_t>(at.n) * 8u : 0u);
      for (int ks = 0; ks < g.kstages; ++ks) {
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&empty[stage], phase ^ 1u, g.wait_ns, abort_flag))) {
          ok = false;
          break;
        }
        if (skip) {
          skip = false;  // failure injection: this stage's loads are never issued
        } else {
          if (elect_one()) {
            uint8_t* sW = smem + stage * T::STAGE_BYTES;
            uint8_t* sX = sW + T::W_BYTES;
            uint32_t bytes = bytes0;
            if (has_sfw) bytes += static_cast<uint32_t>(min(2, g.katoms - 2 * ks)) * 512u;
            mbar_arrive_expect_tx(&full[stage], bytes);
            const int kx = MX4 ? ks * 128 : ks * 64;
            tma_load_2d(sW, &tmW, &full[stage], kx, w_row);
            tma_load_2d(sX, map_x, &full[stage], kx, x_row);
            if (MX4)
              bulk_load(sX + T::X_BYTES + T::SFW_BYTES, sfx, static_cast<uint32_t>(at.n) * 8u, &full[stage]);
          }
          __syncwarp();
          armed |= 1u << stage;
          armed_par = (armed_par & ~(1u << stage)) | (phase << stage);
        }
        sfx += g.sfx_rows * 8;
        if (++stage == T::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (*abort_flag) {
      // let every load of this warp land before the CTA goes away
      for (int s = 0; s < T::STAGES; ++s)
        if ((armed >> s) & 1u) mbar_wait_teardown(&full[s], (armed_par >> s) & 1u, g.wait_ns);
    }
  } else if (warp == 1) {
    if (rank == 0) {
      // ------------------------------------------------------------------ MMA issue
      // The whole warp walks the stages and one elected lane issues: control flow and operands
      // stay warp-uniform.
      uint32_t acc = 0, acc_phase = 0, stage = 0, phase = 0;
      bool ok = true;
      constexpr uint64_t kStageDesc = static_cast<uint64_t>(T::STAGE_BYTES >> 4);
      constexpr uint64_t kXDesc = static_cast<uint64_t>(T::W_BYTES >> 4);
      const uint64_t dw0 = desc_kmajor_sw128(smem_u32(smem));
      uint64_t dw = dw0;
      uint32_t sf = tmem + T::SF_COL0;
      for (int t = unit; t < ntiles && ok; t += units) {
        const uint32_t idesc = T::IDESC0 | (static_cast<uint32_t>(tile(t).n >> 3) << 17);
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&acc_empty[acc], acc_phase ^ 1u, g.wait_ns, abort_flag))) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem + acc * T::TN;
        for (int ks = 0; ks < g.kstages; ++ks) {
          if (!__all_sync(0xFFFFFFFFu, mbar_wait(&ready[stage], phase, g.wait_ns, abort_flag))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t dx = dw + kXDesc;
          const uint32_t acc0 = ks > 0 ? 1u : 0u;
          const int nk = MX4 ? min(4, g.ksteps - 4 * ks) : 4;
          if (elect_one()) {
            if (nk == 4) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                expert_mma<T>(d_tmem, dw + 2 * k, dx + 2 * k, idesc, sf, k, k > 0 ? 1u : acc0);
            } else {
              for (int k = 0; k < nk; ++k)
                expert_mma<T>(d_tmem, dw + 2 * k, dx + 2 * k, idesc, sf, k, k > 0 ? 1u : acc0);
            }
            tc_commit_pair(&empty[stage]);
            if (ks == g.kstages - 1) tc_commit_pair(&acc_full[acc]);
          }
          __syncwarp();
          if (++stage == T::STAGES) {
            stage = 0;
            phase ^= 1u;
            dw = dw0;
            sf = tmem + T::SF_COL0;
          } else {
            dw += kStageDesc;
            sf += T::SF_SET_COLS;
          }
        }
        if (++acc == T::ACC_STAGES) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      // nothing issued may still be running when the tensor memory is released
      if (elect_one()) {
        tc_commit_own(drain);
        mbar_wait_teardown(drain, 0, g.wait_ns);
      }
      __syncwarp();
    }
  } else if (warp == 2) {
    // -------------------------------------------------------------------- weight scales, or relay
    uint32_t stage = 0, phase = 0, armed = 0, armed_par = 0;
    bool ok = true;
    for (int t = unit; t < ntiles && ok; t += units) {
      int64_t blk = 0;
      bool has = false;
      if (MX4) {
        const ExpertTile at = tile(t);
        has = 2 * at.tw + static_cast<int>(rank) < g.nblk128;
        blk = static_cast<int64_t>(at.e) * g.nblk128 + 2 * at.tw + rank;
      }
      const uint8_t* sfw = MX4 ? g.sfw + blk * g.katoms * 512 : nullptr;
      for (int ks = 0; ks < g.kstages; ++ks) {
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(MX4 ? &empty[stage] : &full[stage], MX4 ? phase ^ 1u : phase, g.wait_ns,
                                               abort_flag))) {
          ok = false;
          break;
        }
        if (elect_one()) {
          if (!MX4)
            mbar_arrive_cta(&ready[stage], 0);  // the relay
          else if (has)  // the weights' scale atoms of the stage, beside the producer's copies
            bulk_load(smem + stage * T::STAGE_BYTES + T::W_BYTES + T::X_BYTES, sfw + 1024 * ks,
                      static_cast<uint32_t>(min(2, g.katoms - 2 * ks)) * 512u, &full[stage]);
        }
        __syncwarp();
        if (has) {
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
      for (int s = 0; s < T::STAGES; ++s)
        if ((armed >> s) & 1u) mbar_wait_teardown(&full[s], (armed_par >> s) & 1u, g.wait_ns);
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
          const uint32_t sSFW = smem_u32(smem + stage * T::STAGE_BYTES + T::W_BYTES + T::X_BYTES);
          const uint32_t sSFX = sSFW + T::SFW_BYTES;
          const uint32_t set = lane_base + T::SF_COL0 + T::SF_SET_COLS * stage;
          // what lies behind the tile's rows, features or depth here is never multiplied with a
          // value that reaches a stored result
          uint32_t v[16];
#pragma unroll
          for (int r = 0; r < 8; ++r)
            if (32 * r < T::TN) lds_u32x2(sSFX + (32 * r + lane) * 8, v[r], v[8 + r]);
            else v[r] = v[8 + r] = 0u;
          const uint32_t w0 = lds_u32(sSFW + lane * 16 + 4 * q), w1 = lds_u32(sSFW + 512 + lane * 16 + 4 * q);
          tmem_st_32x32b_x16(set, v);
          tmem_st_32x32b_x1(set + 16 + q, w0);
          tmem_st_32x32b_x1(set + 20 + q, w1);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cta(&ready[stage], 0);
          if (++stage == T::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    }
  } else {
    // -------------------------------------------------------------------- epilogue
    // 8 warps: warp w reads TMEM lane quarter w % 4 (32 features) and every other 16 columns (rows
    // of Y); all of them leave TMEM, rounded, before the first is stored.
    const int q = warp & 3, half = (warp - kGemmEpiWarp0) >> 2;
    uint8_t* stg = staging + (warp - kGemmEpiWarp0) * (BATCH * kExpertEpiBytes);
    const uint32_t stg32 = smem_u32(stg);
    // A staged row is 64 bytes, its 16-byte parts permuted by the map's 64-byte swizzle (part ^ (row / 2) % 4),
    // which keeps the eight rows of a matrix on different banks.
    const uint32_t st_addr = stg32 + (lane & 7) * 64 + 16 * ((lane >> 3) ^ ((lane >> 1) & 3));
    uint32_t acc = 0, acc_phase = 0;
    for (int t = unit; t < ntiles; t += units) {
      const ExpertTile at = tile(t);
      const int f0 = at.tw * T::TM + static_cast<int>(rank) * T::BM + q * 32;
      const int64_t y0 = static_cast<int64_t>(offsets[at.e]) + at.row;
      const bool got = mbar_wait(&acc_full[acc], acc_phase, g.wait_ns, abort_flag, 64);
      if (!__all_sync(0xFFFFFFFFu, got)) break;
      tc_fence_after();
      const uint32_t tbase = tmem + (static_cast<uint32_t>(q * 32) << 16) + acc * T::TN + half * 16;
      constexpr int NC = T::TN / 32;  // 16-row chunks of a warp
      uint32_t pk[8 * NC];
#pragma unroll
      for (int c = 0; c < NC; c += 2) {
        if (32 * c + 16 * half < at.n) {
          uint32_t r[2][2][8];  // chunk, lane half
#pragma unroll
          for (int i = 0; i < 4; ++i)
            tmem_ld_16x256b_x2(tbase + 32 * (c + (i >> 1)) + (static_cast<uint32_t>(16 * (i & 1)) << 16),
                               r[i >> 1][i & 1]);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i)  // pk[8 c + 4 b + m]: rows 8 b .. of the chunk, features 8 m ..
            pk[8 * c + i] = pack_bf16x2_rn(__uint_as_float(r[i >> 3][(i >> 1) & 1][4 * ((i >> 2) & 1) + 2 * (i & 1)]),
                                           __uint_as_float(r[i >> 3][(i >> 1) & 1][4 * ((i >> 2) & 1) + 2 * (i & 1) + 1]));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cta(&acc_empty[acc], 0);
      const int rows = f0 < g.N ? min(at.left, at.n) - 16 * half : 0;  // from the warp's first on
#pragma unroll
      for (int c0 = 0; c0 < NC; c0 += BATCH) {
        if (rows <= 32 * c0) break;
        if (lane < BATCH) bulk_wait_read_all();  // the lane's store of the batch before
        __syncwarp();
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          const int c = c0 + i;
          if (32 * c >= rows) break;
          stmatrix_x4_trans(st_addr + i * kExpertEpiBytes, pk[8 * c], pk[8 * c + 1], pk[8 * c + 2], pk[8 * c + 3]);
          stmatrix_x4_trans(st_addr + i * kExpertEpiBytes + 8 * 64, pk[8 * c + 4], pk[8 * c + 5], pk[8 * c + 6],
                            pk[8 * c + 7]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane < BATCH && rows - 32 * (c0 + lane) >= 16) {  // clipped at the last feature
          tma_store_2d(&tmY, stg + lane * kExpertEpiBytes, f0, static_cast<int32_t>(y0) + 32 * (c0 + lane) + 16 * half);
          bulk_commit_group();
        }
        // where the group ends inside a chunk only its own rows are stored, 16 features a lane
        const int i = (rows >> 5) - c0, nrows = rows & 31;
        if (i < BATCH && nrows > 0 && nrows < 16) {
          const int rr = lane >> 1, f = 16 * (lane & 1);
          if (rr < nrows) {
            __nv_bfloat16* dst = g.y + (y0 + 32 * (c0 + i) + 16 * half + rr) * g.ldy + f0 + f;
            const uint32_t src = stg32 + i * kExpertEpiBytes + rr * 64;
            const uint32_t part = static_cast<uint32_t>(2 * (lane & 1)) ^ ((rr >> 1) & 3);
            const uint4 a = lds_u32x4(src + 16 * part), b = lds_u32x4(src + 16 * (part ^ 1));
            if (f0 + f < g.N) *reinterpret_cast<uint4*>(dst) = a;
            if (f0 + f + 8 < g.N) *reinterpret_cast<uint4*>(dst + 8) = b;
          }
        }
      }
      if (++acc == T::ACC_STAGES) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    // The next kernel may set itself up while the last stores land (a layer of 500 tokens, 4 of 32 experts,
    // 1024 -> 1024: 47.7 -> 45.5 us; 4 tokens, 8 of 64, up: 27.0 -> 26.0 us; a SwiGLU quantizer of 2036 rows
    // behind it starts unevenly spread: 23.2 -> 23.8 us). From the kernel's start on it would take the
    // warps' issue slots for the whole product.
    pdl_launch_dependents();
    if (lane < BATCH) bulk_wait_all();
  }
  __syncthreads();
  cluster_sync_all();  // nothing of the pair reads this CTA's memory any more
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

}  // namespace arc
