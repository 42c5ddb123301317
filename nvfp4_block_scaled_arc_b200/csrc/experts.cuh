// experts.cuh -- the memory-bound kernels of mixture-of-experts layers: the plan (a stable counting
// sort of the slots by expert), tokens copied into sorted order and summed back with their router
// weights, the gradients of both, and the MXFP4 quantizers that write sorted rows.
//
// Slot s = token * k + choice; offsets[e] is the first sorted row of expert e, blocks[e] its first
// 128-row block of scale bytes. Sorted rows are dense (no padding between experts), so everything
// here moves only rows that exist; the scale bytes alone begin a new 128-row block per expert, so
// that a tile's scale bytes always begin on the 16-byte boundary that a bulk copy needs.
#pragma once

#include <cooperative_groups.h>

#include "elementwise.cuh"

namespace arc {

constexpr int kMaxExperts = 512;

// Sections of the plan, each beginning at a multiple of 64 values.
__host__ __device__ constexpr int64_t plan_pad(int64_t n) { return (n + 63) / 64 * 64; }

struct Plan {
  const int32_t* offsets;
  const int32_t* blocks;
  const int32_t* row_of_slot;
  const int32_t* slot_of_row;
  const int32_t* sf_row;
};

__host__ __device__ inline Plan plan_sections(const int32_t* p, int64_t slots, int experts) {
  Plan v;
  v.offsets = p;
  v.blocks = v.offsets + plan_pad(experts + 1);
  v.row_of_slot = v.blocks + plan_pad(experts + 1);
  v.slot_of_row = v.row_of_slot + plan_pad(slots);
  v.sf_row = v.slot_of_row + plan_pad(slots);
  return v;
}

// Whether a plan's entry is a place in [0, n); -1 is none, anything else no plan's (reported, not used).
__device__ __forceinline__ bool plan_place(int64_t v, int64_t n) {
  if (static_cast<uint64_t>(v) < static_cast<uint64_t>(n)) return true;
  if (v != -1) set_status(kStatusInvalidArg);
  return false;
}

// Loads of what an earlier kernel may have written. These kernels begin while that kernel still runs
// and wait for it (griddepcontrol.wait); a non-coherent load, or a plain one through a pointer to
// const that is __restrict__, counts as constant for the whole kernel and could be moved before
// that wait, so there is none here.
__device__ __forceinline__ uint4 ld_v4(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 ld_v4_once(const void* p) {  // read once: not kept in L1
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t ld_u16(const void* p) {
  uint16_t v;
  asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(p));
  return v;
}

// ---------------------------------------------------------------------------------------------
// Plan, in one launch without a grid-wide wait. The slots are cut into parts, one for each cluster
// of CTAs. A cluster counts the ids of all slots per expert (4 bytes a slot from L2, spread over
// its CTAs): those before its part and the others, which gives offsets and the first row of its own
// slots without waiting for another cluster; its CTAs exchange counts through distributed shared
// memory. Then every warp walks its share of the part, 32 slots at a time, and ranks equal ids by
// lane (one vote per bit of the id), which keeps the order of slots within an expert: atomics count,
// none decides a place. Up to 4096 slots one CTA does all. What bounds it is instructions per slot
// and the latency of a dozen barriers: 3.5 us for 8 slots, 9.0 us for 65536 slots of 64 experts (15.1
// us with one cluster), 11.7 us for 131072 slots of 256 (28.0 us; 19.7 us in 16 parts).
// ---------------------------------------------------------------------------------------------

constexpr int kPlanThreads = 1024, kPlanWarps = 32, kPlanCtas = 8, kPlanMaxParts = 8;

// Dynamic shared memory: the part's counts per warp [32][E] and of the CTA [E], all slots' counts
// before the part and from it on [2][E], row bases [E], and what turns a row of an expert into its
// place in the scale layout [E].
__host__ __device__ constexpr size_t plan_smem_bytes(int experts) {
  return static_cast<size_t>(kPlanWarps + 5) * static_cast<size_t>(experts) * 4;
}

template <typename ID>
__device__ __forceinline__ int expert_id(const ID* ids, int64_t ld, int k, int s, int experts) {
  int64_t at = s;
  if (ld != k) {  // rows with a stride: the division costs as much as all else
    const int t = s / k;
    at = t * ld + (s - t * k);
  }
  const ID v = ids[at];
  return v >= 0 && v < experts ? static_cast<int>(v) : -1;
}

// Lanes of the warp whose expert is this lane's (none has e < 0).
__device__ __forceinline__ uint32_t same_expert(int e, int bits) {
  uint32_t peers = __ballot_sync(0xFFFFFFFFu, e >= 0);
  for (int b = 0; b < bits; ++b) {
    const bool set = (e >> b) & 1;
    const uint32_t v = __ballot_sync(0xFFFFFFFFu, set);
    peers &= set ? v : ~v;
  }
  return peers;
}

template <typename ID>
__global__ void __launch_bounds__(kPlanThreads, 1)
    k_expert_plan(const ID* ids, int64_t ld, int slots, int k, int experts, int ctas, int32_t* plan) {
  namespace cg = cooperative_groups;
  extern __shared__ int32_t plan_sm[];
  __shared__ int32_t scan_rows[kPlanWarps], scan_blocks[kPlanWarps];
  cg::cluster_group cluster = cg::this_cluster();
  pdl_launch_dependents();
  int32_t* warp_counts = plan_sm;                    // [32][E]
  int32_t* counts = plan_sm + kPlanWarps * experts;  // [E]
  int32_t* seen = counts + experts;                  // [2][E]
  int32_t* base = seen + 2 * experts;                // [E] first row of this CTA's slots of the expert
  int32_t* sf_shift = base + experts;                // [E] sf_row - row
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = static_cast<int>(blockIdx.x) % ctas, part = static_cast<int>(blockIdx.x) / ctas;
  const int parts = static_cast<int>(gridDim.x) / ctas;
  const uint32_t before_me = (1u << lane) - 1u;
  const int bits = 32 - __clz(experts - 1);  // of an id (0 for one expert)
  for (int i = tid; i < (kPlanWarps + 3) * experts; i += kPlanThreads) warp_counts[i] = 0;
  pdl_wait();  // the ids may come from the kernel before
  __syncthreads();

  // this part's slots, a contiguous range of whole strips of 32 for every warp of the cluster
  const int nwarps = parts * ctas * kPlanWarps;
  const int64_t chunk = (static_cast<int64_t>(slots) + nwarps * 32 - 1) / (nwarps * 32) * 32;
  const int part_lo = static_cast<int>(min(static_cast<int64_t>(slots), part * ctas * kPlanWarps * chunk));
  const int lo = static_cast<int>(min(static_cast<int64_t>(slots), part_lo + (cta * kPlanWarps + warp) * chunk));
  const int hi = static_cast<int>(min(static_cast<int64_t>(slots), lo + chunk));
  int32_t* mine = warp_counts + warp * experts;
  for (int s0 = lo; s0 < hi; s0 += 128) {  // four independent loads in flight
    int e[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int s = s0 + 32 * u + lane;
      e[u] = s < hi ? expert_id(ids, ld, k, s, experts) : -1;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (e[u] >= 0) atomicAdd(&mine[e[u]], 1);
  }
  if (parts > 1) {
    const int share = (slots + ctas - 1) / ctas;
    const int all_hi = min(slots, (cta + 1) * share);
    for (int s0 = cta * share + tid; s0 < all_hi; s0 += 8 * kPlanThreads) {
      int e[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int s = s0 + kPlanThreads * u;
        e[u] = s < all_hi ? expert_id(ids, ld, k, s, experts) : -1;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (e[u] >= 0) atomicAdd(&seen[(s0 + kPlanThreads * u < part_lo ? 0 : experts) + e[u]], 1);
    }
  }
  __syncthreads();
  if (tid < experts) {
    int run = 0;
#pragma unroll 8
    for (int w = 0; w < kPlanWarps; ++w) {
      const int c = warp_counts[w * experts + tid];
      warp_counts[w * experts + tid] = run;
      run += c;
    }
    counts[tid] = run;
    if (parts == 1) seen[experts + tid] = run;
  }
  cluster.sync();
  int total = 0, before = 0;  // thread e < E: rows of expert e, and those of slots before this CTA's
  if (tid < experts) {
#pragma unroll
    for (int c = 0; c < kPlanCtas; ++c) {
      if (c < ctas) {
        const int32_t* there = cluster.map_shared_rank(counts, c);
        const int own = there[tid], bef = there[experts + tid], aft = there[2 * experts + tid];
        total += bef + aft;
        before += bef + (c < cta ? own : 0);
      }
    }
  }
  // exclusive scan over the experts (one thread each)
  const int nblk = (total + 127) >> 7;
  int rows_in = total, blocks_in = nblk;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xFFFFFFFFu, rows_in, o), b = __shfl_up_sync(0xFFFFFFFFu, blocks_in, o);
    if (lane >= o) {
      rows_in += a;
      blocks_in += b;
    }
  }
  if (lane == 31) {
    scan_rows[warp] = rows_in;
    scan_blocks[warp] = blocks_in;
  }
  __syncthreads();
  // every warp scans the 32 warps' sums
  int rows_w = scan_rows[lane], blocks_w = scan_blocks[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xFFFFFFFFu, rows_w, o), b = __shfl_up_sync(0xFFFFFFFFu, blocks_w, o);
    if (lane >= o) {
      rows_w += a;
      blocks_w += b;
    }
  }
  const int all_rows = __shfl_sync(0xFFFFFFFFu, rows_w, 31), all_blocks = __shfl_sync(0xFFFFFFFFu, blocks_w, 31);
  const int rows0 = __shfl_sync(0xFFFFFFFFu, rows_w, warp) - scan_rows[warp];
  const int blocks0 = __shfl_sync(0xFFFFFFFFu, blocks_w, warp) - scan_blocks[warp];
  const int off = rows0 + rows_in - total, blk = blocks0 + blocks_in - nblk;
  int32_t* g_offsets = plan;
  int32_t* g_blocks = g_offsets + plan_pad(experts + 1);
  int32_t* g_row_of_slot = g_blocks + plan_pad(experts + 1);
  int32_t* g_slot_of_row = g_row_of_slot + plan_pad(slots);
  int32_t* g_sf_row = g_slot_of_row + plan_pad(slots);
  if (tid < experts) {
    base[tid] = off + before;
    sf_shift[tid] = 128 * blk - off;
    if (blockIdx.x == 0) {
      g_offsets[tid] = off;
      g_blocks[tid] = blk;
      if (tid == 0) {
        g_offsets[experts] = all_rows;
        g_blocks[experts] = all_blocks;
      }
    }
  }
  __syncthreads();
  for (int s0 = lo; s0 < hi; s0 += 128) {
    int e[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int s = s0 + 32 * u + lane;
      e[u] = s < hi ? expert_id(ids, ld, k, s, experts) : -1;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (s0 + 32 * u >= hi) break;  // the same for the warp
      const int s = s0 + 32 * u + lane;
      const uint32_t peers = same_expert(e[u], bits);
      int row = -1;
      if (e[u] >= 0) row = base[e[u]] + mine[e[u]] + __popc(peers & before_me);
      __syncwarp();  // every lane has read its count before the first of each expert moves it on
      if (e[u] >= 0 && (peers & before_me) == 0u) mine[e[u]] += __popc(peers);
      __syncwarp();
      if (s < hi) g_row_of_slot[s] = row;
      if (e[u] >= 0) {
        g_slot_of_row[row] = s;
        g_sf_row[row] = row + sf_shift[e[u]];
      }
    }
  }
  for (int64_t i = all_rows + static_cast<int64_t>(blockIdx.x) * kPlanThreads + tid; i < slots;
       i += static_cast<int64_t>(gridDim.x) * kPlanThreads) {
    g_slot_of_row[i] = -1;
    g_sf_row[i] = -1;
  }
  cluster.sync();  // no CTA leaves while another may still read its counts
}

// ---------------------------------------------------------------------------------------------
// Sorted rows and back. A group of L lanes (a power of two up to the whole warp, so that narrow rows
// leave no lane idle) takes one token and a segment of L * U 16-byte vectors of it; a lane holds the
// place (and weight) of one of L choices at a time, broadcast by shuffle. At 2048 columns the rows
// move at 0.90 to 1.0 of the copy rate (two choices, the combine: 0.90; eight: 0.96 and more); with 8 choices of
// 256 columns whole warps reached 0.49 (combine) and 0.32 (its gradient), groups 0.79 and 0.91.
// ---------------------------------------------------------------------------------------------

constexpr int kMoveThreads = 256;

// This lane's group and place in it: t the item, v0 the first vector, false behind the last item.
struct MoveLane {
  int64_t t;
  int l, v0;
};
template <int U>
__device__ __forceinline__ MoveLane move_lane(int log_lanes, int nseg) {
  const int lane = threadIdx.x & 31, lanes = 1 << log_lanes;
  const int64_t warp = static_cast<int64_t>(blockIdx.x) * (kMoveThreads / 32) + (threadIdx.x >> 5);
  const int64_t group = (warp << (5 - log_lanes)) + (lane >> log_lanes);
  MoveLane m;
  m.t = nseg == 1 ? group : group / nseg;
  m.l = lane & (lanes - 1);
  m.v0 = static_cast<int>(group - m.t * nseg) * lanes * U + m.l;
  return m;
}

template <int U>
__global__ void __launch_bounds__(kMoveThreads) k_dispatch(const __nv_bfloat16* x, int64_t ldx, int vecs, int log_lanes,
                                                           int nseg, Plan p, int64_t tokens, int k,
                                                           __nv_bfloat16* rows, int64_t ldr) {
  pdl_launch_dependents();
  const int lanes = 1 << log_lanes;
  const MoveLane m = move_lane<U>(log_lanes, nseg);
  const bool valid = m.t < tokens;
  pdl_wait();
  uint4 w[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int v = m.v0 + lanes * u;
    w[u] = valid && v < vecs ? ld_v4_once(x + m.t * ldx + 8 * v) : make_uint4(0, 0, 0, 0);
  }
  for (int j0 = 0; j0 < k; j0 += lanes) {
    const int nj = min(lanes, k - j0);
    const int mine = valid && m.l < nj ? p.row_of_slot[m.t * k + j0 + m.l] : -1;
    for (int j = 0; j < nj; ++j) {
      const int64_t row = __shfl_sync(0xFFFFFFFFu, mine, j, lanes);
      if (!plan_place(row, tokens * k)) continue;
      uint4* dst = reinterpret_cast<uint4*>(rows + row * ldr);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (m.v0 + lanes * u < vecs) dst[m.v0 + lanes * u] = w[u];
    }
  }
}

__device__ __forceinline__ void fma_bf16x8(float (&acc)[8], float w, uint4 v) {
  acc[0] = __fmaf_rn(w, bf16_lo(v.x), acc[0]);
  acc[1] = __fmaf_rn(w, bf16_hi(v.x), acc[1]);
  acc[2] = __fmaf_rn(w, bf16_lo(v.y), acc[2]);
  acc[3] = __fmaf_rn(w, bf16_hi(v.y), acc[3]);
  acc[4] = __fmaf_rn(w, bf16_lo(v.z), acc[4]);
  acc[5] = __fmaf_rn(w, bf16_hi(v.z), acc[5]);
  acc[6] = __fmaf_rn(w, bf16_lo(v.w), acc[6]);
  acc[7] = __fmaf_rn(w, bf16_hi(v.w), acc[7]);
}

// y[t] = bf16( sum_j w_j rows[row_j] [+ add] ): the combine, and with weights of one (weights ==
// nullptr) the gradient of the dispatch. WHOLE: a group is the warp (16384 tokens of 2 x 4096: 64 us,
// against 73 us without that branch taken for the warp as a whole). Otherwise several choices'
// vectors are requested before the first is added (32768 tokens of 8 x 128: 19 against 45 us for a
// warp per token).
template <int U, bool WHOLE>
__global__ void __launch_bounds__(kMoveThreads)
    k_combine(const __nv_bfloat16* rows, int64_t ldr, int vecs, int log_lanes, int nseg, const float* weights,
              int64_t ldw, Plan p, int64_t tokens, int k, const __nv_bfloat16* add, int64_t lda, __nv_bfloat16* y,
              int64_t ldy) {
  pdl_launch_dependents();
  const int lanes = WHOLE ? 32 : 1 << log_lanes;
  const MoveLane m = move_lane<U>(WHOLE ? 5 : log_lanes, nseg);
  const bool valid = m.t < tokens;
  pdl_wait();
  if (WHOLE && !valid) return;
  float acc[U][8];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[u][i] = 0.0f;
  for (int j0 = 0; j0 < k; j0 += lanes) {
    const int nj = min(lanes, k - j0);
    const bool has = valid && m.l < nj;
    const int mine = has ? p.row_of_slot[m.t * k + j0 + m.l] : -1;
    const float wmine = has && weights != nullptr ? weights[m.t * ldw + j0 + m.l] : 1.0f;
    if constexpr (WHOLE) {
#pragma unroll 4
      for (int j = 0; j < nj; ++j) {
        const int64_t row = __shfl_sync(0xFFFFFFFFu, mine, j);
        const float w = __shfl_sync(0xFFFFFFFFu, wmine, j);
        if (!plan_place(row, tokens * k)) continue;
        const __nv_bfloat16* src = rows + row * ldr;
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (m.v0 + 32 * u < vecs) fma_bf16x8(acc[u], w, ld_v4_once(src + 8 * (m.v0 + 32 * u)));
      }
      continue;
    }
    // a choice without a row adds 0 * 0
    constexpr int J = U == 4 ? 2 : 4;
    for (int j = 0; j < nj; j += J) {
      uint4 v[J][U];
      float w[J];
#pragma unroll
      for (int i = 0; i < J; ++i) {
        const int64_t row = __shfl_sync(0xFFFFFFFFu, mine, j + i, lanes);
        w[i] = __shfl_sync(0xFFFFFFFFu, wmine, j + i, lanes);
        const bool ok = j + i < nj && plan_place(row, tokens * k);
        if (!ok) w[i] = 0.0f;
        const __nv_bfloat16* src = rows + row * ldr + 8 * m.v0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          v[i][u] = make_uint4(0, 0, 0, 0);
          if (ok && m.v0 + lanes * u < vecs) v[i][u] = ld_v4_once(src + 8 * lanes * u);
        }
      }
#pragma unroll
      for (int i = 0; i < J; ++i)
#pragma unroll
        for (int u = 0; u < U; ++u) fma_bf16x8(acc[u], w[i], v[i][u]);
    }
  }
  if (!valid) return;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int v = m.v0 + lanes * u;
    if (v >= vecs) continue;
    if (add != nullptr)
      fma_bf16x8(acc[u], 1.0f, *reinterpret_cast<const uint4*>(add + m.t * lda + 8 * v));
    *reinterpret_cast<uint4*>(y + m.t * ldy + 8 * v) =
        make_uint4(pack_bf16x2_rn(acc[u][0], acc[u][1]), pack_bf16x2_rn(acc[u][2], acc[u][3]),
                   pack_bf16x2_rn(acc[u][4], acc[u][5]), pack_bf16x2_rn(acc[u][6], acc[u][7]));
  }
}

// One group per slot: d_rows[row] = bf16(w d_y[t]) and d_w = <d_y[t], rows[row]> (an fp32 sum for each of
// the U vectors of a lane's round, joined by two additions and shuffles: a fixed order; so no chain is
// longer than max(24, 8 ceil(d / 1024)) products, however few lanes take the row. One sum a lane reached 96
// and was hardly faster: 45.7 us each at 4096 tokens of 8 x 2048, 59.1 against 60.0 us at 32768 of 8 x 264). d_rows
// may be rows: each vector is read before the same lane writes it.
__global__ void __launch_bounds__(kMoveThreads)
    k_combine_grad(const __nv_bfloat16* dy, int64_t lddy, const __nv_bfloat16* rows, int64_t ldr, int vecs,
                   int log_lanes, const float* weights, int64_t ldw, Plan p, int64_t tokens, int k,
                   __nv_bfloat16* d_rows, int64_t lddr, float* d_w, int64_t lddw) {
  pdl_launch_dependents();
  const int lanes = 1 << log_lanes;
  const MoveLane m = move_lane<1>(log_lanes, 1);
  const int64_t s = m.t, slots = tokens * k;
  pdl_wait();
  const bool valid = s < slots;
  const int64_t t = valid ? s / k : 0, j = s - t * k;
  const int64_t row = valid ? p.row_of_slot[s] : -1;
  const bool has = plan_place(row, slots);
  constexpr int U = 4;  // vectors in flight: all loaded before the first is written (rows may be d_rows)
  float dots[U] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (has) {
    const float w = weights[t * ldw + j];
    const __nv_bfloat16* a = dy + t * lddy;
    const __nv_bfloat16* b = rows + row * ldr;
    uint4* dst = reinterpret_cast<uint4*>(d_rows + row * lddr);
    for (int v0 = m.l; v0 < vecs; v0 += lanes * U) {
      uint4 g[U], r[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int v = v0 + lanes * u;
        g[u] = r[u] = make_uint4(0, 0, 0, 0);
        if (v < vecs) {
          g[u] = ld_v4(a + 8 * v);
          r[u] = *reinterpret_cast<const uint4*>(b + 8 * v);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t gs[4] = {g[u].x, g[u].y, g[u].z, g[u].w}, rs[4] = {r[u].x, r[u].y, r[u].z, r[u].w};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float g0 = bf16_lo(gs[i]), g1 = bf16_hi(gs[i]);
          dots[u] = __fmaf_rn(g0, bf16_lo(rs[i]), dots[u]);
          dots[u] = __fmaf_rn(g1, bf16_hi(rs[i]), dots[u]);
          o[i] = pack_bf16x2_rn(__fmul_rn(w, g0), __fmul_rn(w, g1));
        }
        if (v0 + lanes * u < vecs) dst[v0 + lanes * u] = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
  float dot = __fadd_rn(__fadd_rn(dots[0], dots[1]), __fadd_rn(dots[2], dots[3]));
  __syncwarp();
  for (int o = lanes >> 1; o; o >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
  if (valid && m.l == 0) d_w[t * lddw + j] = dot;
}

// ---------------------------------------------------------------------------------------------
// MXFP4 quantization into sorted order (format and arithmetic of k_quant_mx_rows). SRC tokens: the
// row of a token is coded once and written to the token's k sorted rows. SRC SwiGLU: row i of
// gate|up gives act = bf16(silu(gate) * up), coded into sorted row i; act never goes to memory. A
// lane takes one block of 32 values (one 16-byte store of codes for each destination). The row's
// scale bytes stay in shared memory for the appended blocks of 32 outlier channels, a lane each,
// whose values are read again (two bytes, or a gate and an up).
// ---------------------------------------------------------------------------------------------

constexpr int kQexTokens = 0, kQexSwiglu = 1;

struct QuantExpertsArgs {
  const __nv_bfloat16* x;  // tokens [T, K], or gate|up [S, 2 K]
  int64_t ldx;
  int64_t n;        // tokens, or slots
  int64_t slots;
  int K, r, kpad;
  int64_t sf_rows;  // rows of the scale layout
  const int32_t* idx;
  Plan p;
  int k, experts;
  uint8_t* codes;
  uint8_t* sf;
};

// silu(g) * u of a bf16 pair each, rounded to bf16: 2^(-g log2 e), one added, the reciprocal, two
// products, in fp32 with the approximate 2^x and reciprocal (2 ulp and 1 ulp). Before the one rounding to
// bf16 (2^-8) the relative error is at most (1.25 max(-g, 0) + 9) 2^-24: the product -g log2 e is off by half
// an ulp and by log2 e's own rounding, together a relative 1.23 |g| 2^-24 of the exponential; 2^x adds
// 4 units of 2^-24, the sum 1, the reciprocal 2, the products 2. That is 2^-20.8 at g >= 0, 2^-19.7 at
// g = -8 and 2^-17.6 at -60, where a value that near to a border between two bf16 values may go to the other
// one. Below g = -87.3 the reciprocal is flushed and the result is 0, where |silu| < 1.1e-36. k_silu_mul's
// correctly rounded quotient would bound the kernel by its arithmetic (162 against 110 us at 8192 x 14336).
__device__ __forceinline__ uint32_t silu_mul_pair(uint32_t g, uint32_t u) {
  const uint64_t g2 = f2_pack(bf16_lo(g), bf16_hi(g));
  constexpr float kNegLog2e = -1.44269504088896341f;
  float x0, x1, r0, r1, a0, a1;
  f2_unpack(f2_mul(g2, f2_pack(kNegLog2e, kNegLog2e)), x0, x1);
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(x0));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(x1));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(__fadd_rn(1.0f, x0)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(__fadd_rn(1.0f, x1)));
  f2_unpack(f2_mul(f2_mul(g2, f2_pack(r0, r1)), f2_pack(bf16_lo(u), bf16_hi(u))), a0, a1);
  return pack_bf16x2_rn(a0, a1);
}

// 32 consecutive values of the source row from channel c on, as 16 bf16 pairs.
template <int SRC>
__device__ __forceinline__ void load_block(const __nv_bfloat16* row, int K, int c, uint32_t (&w)[16]) {
  uint4 g[4], u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) g[i] = ld_v4(row + c + 8 * i);
  if constexpr (SRC == kQexSwiglu) {
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = ld_v4(row + K + c + 8 * i);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t gs[4] = {g[i].x, g[i].y, g[i].z, g[i].w};
    if constexpr (SRC == kQexSwiglu) {
      const uint32_t us[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) w[4 * i + j] = silu_mul_pair(gs[j], us[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) w[4 * i + j] = gs[j];
    }
  }
}

constexpr int kQexMaxWarps = 8;

// Four lanes' scale bytes as one 32-bit word, in every fourth lane.
__device__ __forceinline__ uint32_t join_scales(uint32_t sb) {
  sb |= __shfl_down_sync(0xFFFFFFFFu, sb, 1) << 8;
  return sb | __shfl_down_sync(0xFFFFFFFFu, sb, 2) << 16;
}

// The block of 32 values w coded: its scale byte, codes, and whether it is all zero.
__device__ __forceinline__ uint4 code_block(const uint32_t (&w)[16], uint32_t& sb, bool& zero) {
  uint32_t mw = 0u;
#pragma unroll
  for (int i = 0; i < 16; ++i) mw = __vmaxu2(mw, w[i] & 0x7FFF7FFFu);
  const uint32_t am = max(mw & 0xFFFFu, mw >> 16) << 16;
  sb = mx_scale_byte(am);
  zero = am == 0u;
  if (zero) return make_uint4(0u, 0u, 0u, 0u);
  const float inv = mx_inv_scale(sb);
  uint64_t p[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) p[e] = f2_pack(bf16_lo(w[e]), bf16_hi(w[e]));
  const uint2 lo = mx_encode16(p, inv);
#pragma unroll
  for (int e = 0; e < 8; ++e) p[e] = f2_pack(bf16_lo(w[8 + e]), bf16_hi(w[8 + e]));
  const uint2 hi = mx_encode16(p, inv);
  return make_uint4(lo.x, lo.y, hi.x, hi.y);
}

// E2M1 codes of two values (round to nearest even, saturating at +-6), the first's lowest.
__device__ __forceinline__ uint32_t e2m1x2_rn_sat(float lo, float hi) {
  uint32_t out;
  asm("{\n\t.reg .b8 b;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\t"
      "cvt.u32.u8 %0, b;\n\t}"
      : "=r"(out)
      : "f"(lo), "f"(hi));
  return out;
}

// Residual of an outlier channel with value bits xw in a block of scale byte t, the code formed
// again from both.
__device__ __forceinline__ float outlier_residual(uint32_t xw, uint32_t t) {
  const float xv = __uint_as_float(xw << 16);
  if (t == kMxZeroBlock) return xv;
  return __fsub_rn(xv, __fmul_rn(e2m1_value(e2m1x2_rn_sat(__fmul_rn(xv, mx_inv_scale(t)), 0.0f) & 15u), mx_scale(t)));
}

// The appended block of the warp's 32 residuals: its scale byte, and eight lanes' codes as one 32-bit
// word (the first lane's lowest) in every eighth lane.
__device__ __forceinline__ uint32_t code_residuals(float res, uint32_t& sb) {
  const uint32_t am = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(fabsf(res)));
  sb = mx_scale_byte(am);
  uint32_t code = am == 0u ? 0u : e2m1x2_rn_sat(__fmul_rn(res, mx_inv_scale(sb)), 0.0f) & 15u;
  code |= __shfl_down_sync(0xFFFFFFFFu, code, 1) << 4;
  code |= __shfl_down_sync(0xFFFFFFFFu, code, 2) << 8;
  return code | __shfl_down_sync(0xFFFFFFFFu, code, 4) << 16;
}

// The same for a half warp's 32 residuals, two in each lane: the word in every fourth lane.
__device__ __forceinline__ uint32_t code_residuals(float r0, float r1, uint32_t& sb) {
  uint32_t am = max(__float_as_uint(fabsf(r0)), __float_as_uint(fabsf(r1)));
#pragma unroll
  for (int o = 8; o; o >>= 1) am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, o));
  sb = mx_scale_byte(am);
  const float inv = mx_inv_scale(sb);
  uint32_t code = am == 0u ? 0u : e2m1x2_rn_sat(__fmul_rn(r0, inv), __fmul_rn(r1, inv));
  code |= __shfl_down_sync(0xFFFFFFFFu, code, 1) << 8;
  return code | __shfl_down_sync(0xFFFFFFFFu, code, 2) << 16;
}

// Scale byte kb of place m: 8 bytes (a K = 256 pipeline stage of the product) per row and stage.
__device__ __forceinline__ uint8_t* expert_sf_at(const QuantExpertsArgs& a, int64_t m, int kb) {
  return a.sf + ((kb >> 3) * a.sf_rows + m) * 8 + (kb & 7);
}

// The j-th destination of source row src: its sorted row and scale place, or -1.
template <int SRC>
__device__ __forceinline__ void expert_places(const QuantExpertsArgs& a, int64_t src, int j, int& dst, int& sfr) {
  dst = SRC == kQexTokens ? a.p.row_of_slot[src * a.k + j] : static_cast<int>(src);
  sfr = -1;
  if (!plan_place(dst, a.slots)) dst = -1;
  if (dst >= 0) sfr = a.p.sf_row[dst];
  if (dst >= 0 && !plan_place(sfr, a.sf_rows)) dst = -1;
}

// Sorted rows in use, as the SwiGLU quantizers read them from the plan: a total outside the slots is no
// plan's, is reported (by one thread of the launch) and counts as none.
__device__ __forceinline__ int64_t rows_in_use(const QuantExpertsArgs& a, bool report) {
  const int64_t n = a.p.offsets[a.experts];
  if (static_cast<uint64_t>(n) <= static_cast<uint64_t>(a.slots)) return n;
  if (report) set_status(kStatusInvalidArg);
  return 0;
}

// Stores block b of a row (the coding of it in this lane) to one destination; every lane of the group
// calls it with its own block, b >= nblk where it has none.
__device__ __forceinline__ void store_block(const QuantExpertsArgs& a, int64_t dst, int64_t m, int b, int nblk,
                                            uint4 codes, uint32_t sb, uint32_t joined) {
  uint8_t* crow = a.codes + dst * (a.kpad >> 1);
  if (b < nblk) *reinterpret_cast<uint4*>(crow + 16 * b) = codes;
  if ((b & ~3) + 3 < nblk) {  // the word's four blocks exist
    if ((b & 3) == 0) *reinterpret_cast<uint32_t*>(expert_sf_at(a, m, b)) = joined;
  } else if (b < nblk) {
    *expert_sf_at(a, m, b) = static_cast<uint8_t>(sb);
  }
  // the last block's lane also zeroes the block that pads an odd number of blocks to K_pad
  const int kbz = nblk + (a.r >> 5);
  if (b == nblk - 1 && 32 * kbz < a.kpad) {
    *reinterpret_cast<uint4*>(crow + 16 * kbz) = make_uint4(0, 0, 0, 0);
    *expert_sf_at(a, m, kbz) = 0;
  }
}

// A CTA for each row. The row's scale bytes stay in shared memory for the appended blocks.
template <int SRC>
__global__ void __launch_bounds__(kQexMaxWarps * 32) k_quant_experts(QuantExpertsArgs a) {
  extern __shared__ uint8_t qex_sb[];  // kMxZeroBlock for an all-zero block
  pdl_launch_dependents();  // the GEMM that follows may set itself up meanwhile
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = static_cast<int>(blockDim.x >> 5);
  const int nblk = a.K >> 5, nres = a.r >> 5;
  const int64_t src = blockIdx.x;
  pdl_wait();
  if (SRC == kQexSwiglu && src >= rows_in_use(a, src == 0 && threadIdx.x == 0)) return;
  const __nv_bfloat16* row = a.x + src * a.ldx;
  const int nrows = SRC == kQexTokens ? a.k : 1;
  int dst0 = -1, sfr0 = -1;  // lane j: the j-th destination (32 at a time)
  if (lane < nrows) expert_places<SRC>(a, src, lane, dst0, sfr0);
  // the values of the warp's first appended block
  int oc = -1;
  uint32_t og = 0, ou = 0;
  auto outlier = [&](int rb) {
    oc = a.idx[32 * rb + lane];
    if (static_cast<unsigned>(oc) < static_cast<unsigned>(a.K)) {
      og = ld_u16(row + oc);
      if constexpr (SRC == kQexSwiglu) ou = ld_u16(row + a.K + oc);
    } else {
      oc = -1;
      if (src == 0) set_status(kStatusInvalidArg);
    }
  };
  if (warp < nres) outlier(warp);
  auto each_place = [&](auto&& store) {
    for (int j0 = 0; j0 < nrows; j0 += 32) {
      int dsts = dst0, sfrs = sfr0;
      if (j0) {
        dsts = -1;
        if (j0 + lane < nrows) expert_places<SRC>(a, src, j0 + lane, dsts, sfrs);
      }
      const int nj = min(32, nrows - j0);
      for (int j = 0; j < nj; ++j) {
        const int64_t dst = __shfl_sync(0xFFFFFFFFu, dsts, j), m = __shfl_sync(0xFFFFFFFFu, sfrs, j);
        if (dst >= 0) store(dst, m);
      }
    }
  };
  for (int b0 = 32 * warp; b0 < nblk; b0 += 32 * nwarps) {
    const int b = b0 + lane;
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = 0u;
    if (b < nblk) load_block<SRC>(row, a.K, 32 * b, w);
    uint32_t sb;
    bool zero;
    const uint4 cc = code_block(w, sb, zero);
    if (nres > 0 && b < nblk) qex_sb[b] = static_cast<uint8_t>(zero ? kMxZeroBlock : sb);
    const uint32_t joined = join_scales(sb);
    each_place([&](int64_t dst, int64_t m) { store_block(a, dst, m, b, nblk, cc, sb, joined); });
  }
  if (nres == 0) return;
  __syncthreads();
  for (int rb = warp; rb < nres; rb += nwarps) {
    if (rb != warp) outlier(rb);
    float res = 0.0f;
    if (oc >= 0) res = outlier_residual(SRC == kQexSwiglu ? silu_mul_pair(og, ou) & 0xFFFFu : og, qex_sb[oc >> 5]);
    uint32_t sb;
    const uint32_t code = code_residuals(res, sb);
    const int kb = nblk + rb;
    each_place([&](int64_t dst, int64_t m) {
      if ((lane & 7) == 0)
        *reinterpret_cast<uint32_t*>(a.codes + dst * (a.kpad >> 1) + 16 * kb + (lane >> 1)) = code;
      if (lane == 1) *expert_sf_at(a, m, kb) = static_cast<uint8_t>(sb);
    });
  }
}

// Many rows of at most 32 blocks: a group of 2^log_lanes lanes for each (16 or 32 where there are appended
// blocks), a block in each lane. With a CTA for each row most lanes of narrow rows idle, and the rows
// are bound by instructions (16384 rows of 256: 17.8 against 4.0 us, of 512 with r 64: 18.1 against 11.8 us;
// 131072 SwiGLU rows: 136 against 30 us and 140 against 78 us).
// A half warp takes an appended block, a lane two of its channels; the primary blocks' scale bytes come
// by shuffle. Where a row fills several warps that form is no faster (4096 channels, r 256: 53.5 against
// 55.2 us), nor are several rows a CTA (27.8 against 23.6 us, SwiGLU, 1056 channels).
template <int SRC>
__global__ void __launch_bounds__(kQexMaxWarps * 32) k_quant_experts_narrow(QuantExpertsArgs a, int log_lanes) {
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, lanes = 1 << log_lanes, l = lane & (lanes - 1), hl = lane & 15;
  const int nblk = a.K >> 5, nres = a.r >> 5;
  const int64_t warp = static_cast<int64_t>(blockIdx.x) * kQexMaxWarps + (threadIdx.x >> 5);
  const int64_t src = (warp << (5 - log_lanes)) + (lane >> log_lanes);
  pdl_wait();
  int64_t n = a.n;
  if (SRC == kQexSwiglu) n = rows_in_use(a, src == 0 && l == 0);
  const bool valid = src < n;
  const int nrows = SRC == kQexTokens ? a.k : 1;
  const __nv_bfloat16* row = a.x + src * a.ldx;
  int dst0 = -1, sfr0 = -1;  // lane j of the group: the j-th destination (a group's lanes at a time)
  if (valid && l < nrows) expert_places<SRC>(a, src, l, dst0, sfr0);
  int c0 = -1, c1 = -1;  // the values of an appended block, two a lane
  uint32_t og = 0, ou = 0;
  auto outlier = [&](int at, int shift) {
    const int c = a.idx[at];
    if (static_cast<unsigned>(c) >= static_cast<unsigned>(a.K)) {
      if (src == 0) set_status(kStatusInvalidArg);
      return -1;
    }
    og |= ld_u16(row + c) << shift;
    if constexpr (SRC == kQexSwiglu) ou |= ld_u16(row + a.K + c) << shift;
    return c;
  };
  auto outliers = [&](int rb) {
    c0 = c1 = -1;
    og = ou = 0;
    if (valid && rb < nres) {
      c0 = outlier(32 * rb + 2 * hl, 0);
      c1 = outlier(32 * rb + 2 * hl + 1, 16);
    }
  };
  if (nres > 0) outliers(l >> 4);
  uint32_t w[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] = 0u;
  if (valid && l < nblk) load_block<SRC>(row, a.K, 32 * l, w);
  uint32_t sb;
  bool zero;
  const uint4 cc = code_block(w, sb, zero);
  const uint32_t joined = join_scales(sb);
  auto each_place = [&](auto&& store) {
    for (int j0 = 0; j0 < nrows; j0 += lanes) {
      int dsts = dst0, sfrs = sfr0;
      if (j0) {
        dsts = -1;
        if (valid && j0 + l < nrows) expert_places<SRC>(a, src, j0 + l, dsts, sfrs);
      }
      const int nj = min(lanes, nrows - j0);
      for (int j = 0; j < nj; ++j) {
        const int64_t dst = __shfl_sync(0xFFFFFFFFu, dsts, j, lanes), m = __shfl_sync(0xFFFFFFFFu, sfrs, j, lanes);
        if (dst >= 0) store(dst, m);
      }
    }
  };
  each_place([&](int64_t dst, int64_t m) { store_block(a, dst, m, l, nblk, cc, sb, joined); });
  if (zero) sb = kMxZeroBlock;
  for (int rb0 = 0; rb0 < nres; rb0 += lanes >> 4) {  // a half warp a block
    const int rb = rb0 + (l >> 4), kb = nblk + rb;
    if (rb0) outliers(rb);
    const uint32_t t0 = __shfl_sync(0xFFFFFFFFu, sb, max(c0, 0) >> 5, lanes);
    const uint32_t t1 = __shfl_sync(0xFFFFFFFFu, sb, max(c1, 0) >> 5, lanes);
    const uint32_t xw = SRC == kQexSwiglu ? silu_mul_pair(og, ou) : og;
    const float r0 = c0 >= 0 ? outlier_residual(xw & 0xFFFFu, t0) : 0.0f;
    const float r1 = c1 >= 0 ? outlier_residual(xw >> 16, t1) : 0.0f;
    uint32_t sbr;
    const uint32_t code = code_residuals(r0, r1, sbr);
    each_place([&](int64_t dst, int64_t m) {
      if (rb >= nres) return;
      if ((hl & 3) == 0) *reinterpret_cast<uint32_t*>(a.codes + dst * (a.kpad >> 1) + 16 * kb + hl) = code;
      if (hl == 1) *expert_sf_at(a, m, kb) = static_cast<uint8_t>(sbr);
    });
  }
}

}  // namespace arc
