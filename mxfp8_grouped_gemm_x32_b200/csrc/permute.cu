// Token permutation by expert and top-k combine.
//
// "Efficient MoE Training for Biological Foundation Models", Challenge 1:
// the tokens routed to each expert are gathered into one group (split_sizes
// per expert) so that a single grouped GEMM serves all experts, and the
// expert outputs are added back into token order (the index_add of the
// per-expert loop).  Here the grouping is a stable counting sort of the
// T*k routed slots (slot s = t*k + j) by expert, with every group starting on
// a multiple of 128 rows so that a 128-row GEMM tile never spans two experts.
#include "permute.cuh"

namespace moe {

constexpr int PB = PERM_BLOCK;

__device__ __forceinline__ bool id_ok(int32_t e, int32_t E) { return e >= 0 && e < E; }

// Pass 1: per-block expert histogram; the row maps' empty values (-1 and 0) for
// all rows along the way.
__global__ void __launch_bounds__(PB) perm_hist_kernel(const int32_t* __restrict__ idx, int64_t R,
                                                       int32_t E, int32_t* __restrict__ hist, int64_t rows_cap,
                                                       int32_t* __restrict__ row_to_slot, float* __restrict__ prob_perm) {
  release_dependents();
  dependency_wait(idx);
  extern __shared__ int cnt[];
  for (int64_t i = int64_t(blockIdx.x) * PB + threadIdx.x; i < rows_cap; i += int64_t(gridDim.x) * PB) {
    row_to_slot[i] = -1;
    prob_perm[i] = 0.0f;
  }
  for (int i = threadIdx.x; i < E; i += PB) cnt[i] = 0;
  __syncthreads();
  const int64_t s = int64_t(blockIdx.x) * PB + threadIdx.x;
  if (s < R) {
    const int32_t e = idx[s];
    if (id_ok(e, E))
      atomicAdd(&cnt[e], 1);
    else
      set_status(MOE_ERR_DEVICE_INDEX);
  }
  __syncthreads();
  if (R == 0) return;  // an empty batch: no block of slots, and no room for its counts in the workspace
  for (int i = threadIdx.x; i < E; i += PB) hist[int64_t(blockIdx.x) * E + i] = cnt[i];
}

// Pass 2 (one CTA): split_sizes, 128-aligned group offsets, and the first
// row of every (block, expert) pair relative to its group's start, in place
// in `hist` (the scatter adds the group offset).  PERM_SEGMENTS threads share
// an expert's column of block counts, a run of blocks each, read eight at a
// time so that the loads overlap: once for the runs' sums, once more for the
// prefixes.
constexpr int PERM_SEGMENTS = 4;
__global__ void __launch_bounds__(MOE_MAX_EXPERTS* PERM_SEGMENTS) perm_scan_kernel(int32_t* __restrict__ hist,
                                                                                  int32_t nblocks, int32_t E,
                                                                                  int32_t* __restrict__ split,
                                                                                  int32_t* __restrict__ offs) {
  release_dependents();
  dependency_wait();
  __shared__ int32_t run_sum[PERM_SEGMENTS][MOE_MAX_EXPERTS];
  __shared__ int32_t wsum[MOE_MAX_EXPERTS / 32];
  const int e = threadIdx.x % MOE_MAX_EXPERTS, seg = threadIdx.x / MOE_MAX_EXPERTS, lane = threadIdx.x & 31;
  const int per = (nblocks + PERM_SEGMENTS - 1) / PERM_SEGMENTS;
  const int first = seg * per, last = min(nblocks, first + per);
  int32_t sum = 0;
  if (e < E)
    for (int b0 = first; b0 < last; b0 += 8) {
      int32_t c[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = b0 + i < last ? hist[int64_t(b0 + i) * E + e] : 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += c[i];
    }
  run_sum[seg][e] = sum;
  __syncthreads();
  int32_t before = 0, total = 0;
#pragma unroll
  for (int s = 0; s < PERM_SEGMENTS; ++s) {
    if (s < seg) before += run_sum[s][e];
    total += run_sum[s][e];
  }
  if (e < E)
    for (int b0 = first; b0 < last; b0 += 8) {
      int32_t c[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = b0 + i < last ? hist[int64_t(b0 + i) * E + e] : 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (b0 + i < last) hist[int64_t(b0 + i) * E + e] = before;
        before += c[i];
      }
    }
  // group offsets: exclusive scan of the groups' padded rows (segment 0's warps)
  int32_t padded = 0, incl = 0;
  if (seg == 0) {
    if (e < E) {
      split[e] = total;
      padded = (total + 127) / 128 * 128;
    }
    incl = padded;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t v = __shfl_up_sync(0xFFFFFFFFu, incl, d);
      if (lane >= d) incl += v;
    }
    if (lane == 31) wsum[threadIdx.x >> 5] = incl;
  }
  __syncthreads();
  if (seg == 0 && e < E) {
    int32_t base = 0;
    for (int w = 0; w < int(threadIdx.x >> 5); ++w) base += wsum[w];
    offs[e] = base + incl - padded;
    if (e == E - 1) offs[E] = base + incl;
  }
}

// Pass 3: stable rank of every slot inside its block (warp match + per-warp
// counts), giving its padded row; writes both index maps and the permuted
// routing probability.
__global__ void __launch_bounds__(PB) perm_scatter_kernel(const int32_t* __restrict__ idx,
                                                          const float* __restrict__ prob, int64_t R,
                                                          int32_t E, const int32_t* __restrict__ base,
                                                          const int32_t* __restrict__ offs,
                                                          int32_t* __restrict__ slot_to_row,
                                                          int32_t* __restrict__ row_to_slot,
                                                          float* __restrict__ prob_perm) {
  release_dependents();
  dependency_wait(idx, prob, base, offs);
  extern __shared__ int wcnt[];  // [32 warps][E]
  for (int i = threadIdx.x; i < 32 * E; i += PB) wcnt[i] = 0;
  __syncthreads();
  const int64_t s = int64_t(blockIdx.x) * PB + threadIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int32_t e = -1;
  if (s < R) {
    e = idx[s];
    if (!id_ok(e, E)) e = -1;
  }
  const uint32_t mask = __match_any_sync(0xFFFFFFFFu, e);
  const uint32_t lrank = __popc(mask & ((1u << lane) - 1u));
  if (e >= 0 && lrank == 0) wcnt[warp * E + e] = __popc(mask);
  __syncthreads();
  if (s < R) {
    if (e < 0) {
      slot_to_row[s] = -1;
      return;
    }
    int32_t pre = 0;
    for (int w = 0; w < warp; ++w) pre += wcnt[w * E + e];
    const int32_t row = offs[e] + base[int64_t(blockIdx.x) * E + e] + pre + int32_t(lrank);
    slot_to_row[s] = row;
    row_to_slot[row] = int32_t(s);
    prob_perm[row] = prob[s];
  }
}

// All passes at once for at most PB slots (a decoding batch), in one CTA: the
// same results from one launch instead of five (two fills, histogram, scan,
// scatter), whose launches would take longer than their work: 8 slots of 128
// experts took 21.5 us between events, now 5.9 (events alone: 3).  CTA 0 sorts and
// fills the rows that groups can reach; the others fill the row maps behind them
// (8.0 us when CTA 0 filled them all).
__global__ void __launch_bounds__(PB) perm_small_kernel(const int32_t* __restrict__ idx,
                                                        const float* __restrict__ prob, int32_t R, int32_t E,
                                                        int64_t rows_cap, int64_t reach, int32_t* __restrict__ split,
                                                        int32_t* __restrict__ offs, int32_t* __restrict__ slot_to_row,
                                                        int32_t* __restrict__ row_to_slot,
                                                        float* __restrict__ prob_perm) {
  release_dependents();
  dependency_wait(idx, prob);
  extern __shared__ int wcnt[];  // [warps with slots][E]: counts, then first ranks; then [E] group offsets
  __shared__ int wsum[MOE_MAX_EXPERTS / 32];
  if (blockIdx.x > 0) {
    for (int64_t i = reach + int64_t(blockIdx.x - 1) * PB + threadIdx.x; i < rows_cap; i += int64_t(gridDim.x - 1) * PB) {
      row_to_slot[i] = -1;
      prob_perm[i] = 0.0f;
    }
    return;
  }
  const int nw = (R + 31) >> 5;  // warps with slots
  int* goff = wcnt + nw * E;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int32_t e = -1;
  if (tid < R) {
    e = idx[tid];
    if (!id_ok(e, E)) {
      set_status(MOE_ERR_DEVICE_INDEX);
      e = -1;
    }
  }
  for (int i = tid; i < nw * E; i += PB) wcnt[i] = 0;
  for (int64_t i = tid; i < reach; i += PB) {
    row_to_slot[i] = -1;
    prob_perm[i] = 0.0f;
  }
  __syncthreads();
  uint32_t lrank = 0;
  if (warp < nw) {
    const uint32_t mask = __match_any_sync(0xFFFFFFFFu, e);
    lrank = __popc(mask & ((1u << lane) - 1u));
    if (e >= 0 && lrank == 0) wcnt[warp * E + e] = __popc(mask);
  }
  __syncthreads();
  // thread x: expert x's slots before each warp's, its total and its padded rows
  int32_t total = 0, padded = 0;
  if (tid < MOE_MAX_EXPERTS) {
    if (tid < E) {
      for (int w = 0; w < nw; ++w) {
        const int32_t c = wcnt[w * E + tid];
        wcnt[w * E + tid] = total;
        total += c;
      }
      split[tid] = total;
      padded = (total + 127) / 128 * 128;
    }
    int32_t incl = padded;  // inclusive scan over the warp's experts
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t v = __shfl_up_sync(0xFFFFFFFFu, incl, d);
      if (lane >= d) incl += v;
    }
    if (lane == 31) wsum[warp] = incl;
    padded = incl - padded;  // rows of the warp's experts before this one
    total = incl;
  }
  __syncthreads();
  if (tid < MOE_MAX_EXPERTS) {
    int32_t before = 0;
    for (int w = 0; w < warp; ++w) before += wsum[w];
    if (tid < E) {
      offs[tid] = goff[tid] = before + padded;
      if (tid == E - 1) offs[E] = before + total;
    }
  }
  __syncthreads();
  if (tid < R) {
    if (e < 0) {
      slot_to_row[tid] = -1;
    } else {
      const int32_t row = goff[e] + wcnt[warp * E + e] + int32_t(lrank);
      slot_to_row[tid] = row;
      row_to_slot[row] = tid;
      prob_perm[row] = prob[tid];
    }
  }
}

// out[t] = sum_j y[row(t, j)], fp32 sum in ascending j, 8 columns per thread;
// row(t, j) = t*k + j (rows in slot order) or slot_to_row[t*k + j] (rows in
// permuted order).  FMT: y holds bf16 rows (COMBINE_BF16), fp32 rows
// (COMBINE_F32) or f24 rows (COMBINE_F24: the top 3 bytes of each fp32
// value, see common.cuh).
template <int FMT, int U>
__global__ void __launch_bounds__(256) combine_kernel(const void* __restrict__ yv, const int32_t* __restrict__ slot_to_row,
                                                      int64_t T, int32_t k, int64_t H8, uint4* __restrict__ out) {
  release_dependents();
  dependency_wait(yv, slot_to_row);
  const int64_t n = T * H8;
  for (int64_t i = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; i < n;
       i += int64_t(gridDim.x) * blockDim.x) {
    const int64_t t = i / H8, c = i % H8;
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    // U choices at a time, all their loads in flight, added in order
    for (int j0 = 0; j0 < k; j0 += U) {
      int64_t row[U];
#pragma unroll
      for (int j = 0; j < U; ++j)
        row[j] = j0 + j >= k ? -1 : (slot_to_row ? int64_t(__ldg(slot_to_row + t * k + j0 + j)) : t * k + j0 + j);
      constexpr int W = FMT == COMBINE_F32 ? 8 : (FMT == COMBINE_F24 ? 6 : 4);  // words of eight values
      uint32_t w[U][W];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        if (row[j] < 0) continue;  // past k, or a slot whose expert id was rejected
        if constexpr (FMT == COMBINE_F24) {
          const uint2* y = static_cast<const uint2*>(yv) + (row[j] * H8 + c) * 3;
#pragma unroll
          for (int x = 0; x < 3; ++x) {
            const uint2 v = __ldg(y + x);
            w[j][2 * x] = v.x;
            w[j][2 * x + 1] = v.y;
          }
        } else {
          const uint4* y = static_cast<const uint4*>(yv) + (row[j] * H8 + c) * (W / 4);
#pragma unroll
          for (int x = 0; x < W / 4; ++x) {
            const uint4 v = __ldg(y + x);
            w[j][4 * x] = v.x; w[j][4 * x + 1] = v.y; w[j][4 * x + 2] = v.z; w[j][4 * x + 3] = v.w;
          }
        }
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
        if (row[j] < 0) continue;
        if constexpr (FMT == COMBINE_F32) {
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] += __uint_as_float(w[j][e]);
        } else if constexpr (FMT == COMBINE_F24) {
          uint32_t f[8];
          f24_unpack4(w[j][0], w[j][1], w[j][2], f);
          f24_unpack4(w[j][3], w[j][4], w[j][5], f + 4);
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] += __uint_as_float(f[e]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            acc[2 * e] += bf16lo(w[j][e]);
            acc[2 * e + 1] += bf16hi(w[j][e]);
          }
        }
      }
    }
    out[i] = make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]),
                        pack_bf16x2(acc[4], acc[5]), pack_bf16x2(acc[6], acc[7]));
  }
}

int64_t permute_workspace_bytes(int64_t R, int32_t E) {
  return cdiv(R, PB) * int64_t(E) * 4 + 256;
}

cudaError_t launch_permute_scan_scatter(const int32_t* idx, const float* prob, int64_t R, int32_t E,
                                        int32_t* split, int32_t* offs, int32_t* row_to_slot, int32_t* slot_to_row,
                                        float* prob_perm, void* ws, cudaStream_t st) {
  const int32_t nb = int32_t(cdiv(R, PB));
  int32_t* hist = static_cast<int32_t*>(ws);
  cudaError_t err =
      launch_dependent(perm_scan_kernel, 1, MOE_MAX_EXPERTS * PERM_SEGMENTS, 0, st, hist, nb, E, split, offs);
  if (err == cudaSuccess && nb > 0)
    err = launch_dependent(perm_scatter_kernel, unsigned(nb), PB, 32 * E * sizeof(int), st, idx, prob, R, E, hist, offs,
                           slot_to_row, row_to_slot, prob_perm);
  return err;
}

cudaError_t launch_permute_index(const int32_t* idx, const float* prob, int64_t R, int32_t E,
                                 int64_t rows_cap, int32_t* split, int32_t* offs,
                                 int32_t* row_to_slot, int32_t* slot_to_row, float* prob_perm,
                                 void* ws, cudaStream_t st) {
  if (R > 0 && R <= PB) {
    // no more groups than experts or slots, each within one 128-row tile but for
    // every 128 slots one tile more
    const int64_t most = 128 * ((R < E ? R : int64_t(E)) + R / 128), reach = most < rows_cap ? most : rows_cap;
    const unsigned fill = unsigned(cdiv(rows_cap - reach, 4 * PB));
    return launch_dependent(perm_small_kernel, 1 + fill, PB, (cdiv(R, 32) + 1) * E * sizeof(int), st, idx, prob,
                            int32_t(R), E, rows_cap, reach, split, offs, slot_to_row, row_to_slot, prob_perm);
  }
  // (an empty batch too: one block, no slots)
  const int32_t nb = int32_t(cdiv(R, PB));
  const cudaError_t err = launch_dependent(perm_hist_kernel, unsigned(nb < 1 ? 1 : nb), PB, E * sizeof(int), st, idx, R, E,
                                           static_cast<int32_t*>(ws), rows_cap, row_to_slot, prob_perm);
  if (err != cudaSuccess) return err;
  return launch_permute_scan_scatter(idx, prob, R, E, split, offs, row_to_slot, slot_to_row, prob_perm, ws, st);
}

cudaError_t launch_combine(const void* y, int fmt, const int32_t* slot_to_row, int64_t T, int32_t k, int64_t H,
                           void* out, cudaStream_t st) {
  const int64_t n = T * (H / 8);
  if (n == 0) return cudaSuccess;
  int64_t blocks = cdiv(n, 256);
  if (blocks > 148 * 32) blocks = 148 * 32;
  uint4* o = static_cast<uint4*>(out);
  // Four choices in flight where a small batch leaves the SMs without enough warps
  // to cover the loads' latency (64 tokens, k = 4: 9.2 -> 7.9 us between events);
  // with enough of them the registers cost more (8192 x 4096, k = 2: 48.8 -> 58.8)
  auto pick = [&](auto U) {
    constexpr int u = decltype(U)::value;
    return fmt == COMBINE_F32 ? combine_kernel<COMBINE_F32, u>
                              : (fmt == COMBINE_F24 ? combine_kernel<COMBINE_F24, u> : combine_kernel<COMBINE_BF16, u>);
  };
  const bool few = blocks <= int64_t(device_sm_count()) * 4;
  auto kern = few ? pick(std::integral_constant<int, 4>()) : pick(std::integral_constant<int, 1>());
  return launch_dependent(kern, unsigned(blocks), 256, 0, st, y, slot_to_row, T, k, H / 8, o);
}

}  // namespace moe
