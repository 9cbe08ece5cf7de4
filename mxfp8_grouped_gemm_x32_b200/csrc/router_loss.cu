// Router training: the top-k selection together with the load-balance loss,
// the z-loss and the tokens per expert, and the gradient of the logits.
//
// "Efficient MoE Training for Biological Foundation Models", Challenge 1:
// tokens are routed to k of E experts and the groups' sizes (split_sizes) are
// as uneven as the router makes them; the two losses are what keeps them even
// and the logits small.  With logits z, the softmax s over all E experts, the
// kept experts' probabilities p (a softmax over the kept logits) and n
// unmasked tokens:
//   counts_e = kept slots of expert e,  f_e = counts_e / (n k)
//   balance  = E sum_e f_e (1/n) sum_t s_te      (f carries no gradient)
//   z        = (1/n) sum_t lse_t^2,  lse_t = log sum_e exp z_te
//   dz_te = g_b (E/n) s_te (f_e - sum_j f_j s_tj) + g_z (2/n) lse_t s_te
//         + sum_{i: idx_ti = e} p_ti (dp_ti - sum_j p_tj dp_tj)
// Masked tokens (padding) are selected like any other, so the layer's shapes
// stay, but with probabilities, counts and gradients of zero.
//
// A group of G lanes owns a token, lane g the experts 8g .. 8g+7, so that a row
// of logits is read (and its gradient written) once, 16 or 32 contiguous
// bytes per lane, and stays in registers; G is the smallest power of two with
// 8 G >= E, so a warp works on 32 / G tokens.  The sums over tokens need no
// exchange per token: a lane keeps its experts' sums of s and counts in
// registers over all the tokens its group visits, in fp32; blocks add
// them up in a fixed order and a second kernel adds the blocks, so the results
// do not depend on scheduling.
#include "router_loss.cuh"

namespace moe {

namespace {

constexpr int RL_THREADS = 256;
constexpr int RL_WARPS = RL_THREADS / 32;
// Wide rows (groups of 16 or 32 lanes): four blocks per SM, a token's logits loaded
// when they are needed.  Narrow ones: three, with the next token's logits on their
// way -- more kept experts per lane need more registers (gradient of 262144 x 256:
// 109 against 125 us, x 32: 45 against 41, now 112 and 37).  A lane has places for
// the most experts its group may keep (eight where up to 32 experts share 2 or 4 lanes),
// whatever k is: the gradient's kernels of those widths spill some 130 bytes at 80
// registers, the losses' 28.
template <int G>
constexpr bool RL_WIDE = G >= 16;
template <int G>
constexpr int RL_BLOCKS_PER_SM = RL_WIDE<G> ? 4 : 3;
// most experts that a token of a group of G lanes keeps
template <int G>
constexpr int KEPT_MAX = G < 4 ? 8 * G : 32;
constexpr int RF_CLUSTER = 8, RF_THREADS = 1024;  // the finishing cluster

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

// 2^x by the hardware's instruction: relative error 2^-22, results below 2^-126
// are 0.  As exp(x) = 2^(x log2(e)) the product's rounding adds 2^-24 |x|
// log2(e) -- for softmax terms, which are small where |x| is large.
constexpr float LOG2E = 1.4426950408889634f;
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Squares of lse are summed as (2^-16 lse)^2: fewer than 2^30 of them pass fp32 only
// where their mean does, and only a |lse| below 2^-47 loses bits.  The finishing
// cluster undoes the factor in 64 bits.
constexpr float Z_SCALE = 1.0f / 65536.0f;
constexpr double Z_UNSCALE = 65536.0 * 65536.0;

// Experts 8g..8g+7 of row t; experts past E read as -inf.  `vec`: rows start
// on 16-byte boundaries and E is a multiple of 8.
template <bool BF16>
__device__ __forceinline__ void load_row8(const void* p, int t, int E, int g, bool vec, float* v) {
  const int64_t base = int64_t(t) * E + 8 * g;
  if (8 * g >= E) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = neg_inf();
    return;
  }
  if constexpr (BF16) {
    const uint16_t* q = static_cast<const uint16_t*>(p) + base;
    if (vec) {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(q));
      v[0] = bf16lo(w.x); v[1] = bf16hi(w.x); v[2] = bf16lo(w.y); v[3] = bf16hi(w.y);
      v[4] = bf16lo(w.z); v[5] = bf16hi(w.z); v[6] = bf16lo(w.w); v[7] = bf16hi(w.w);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 8 * g + i < E ? __uint_as_float(uint32_t(__ldg(q + i)) << 16) : neg_inf();
    }
  } else {
    const float* q = static_cast<const float*>(p) + base;
    if (vec) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(q)), b = __ldg(reinterpret_cast<const float4*>(q) + 1);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 8 * g + i < E ? __ldg(q + i) : neg_inf();
    }
  }
}

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  if constexpr (BF16) return __uint_as_float(uint32_t(__ldg(static_cast<const uint16_t*>(p) + i)) << 16);
  return __ldg(static_cast<const float*>(p) + i);
}

// Experts V g .. V g + V - 1 of row t, likewise; V is 4 or a multiple of 8.
template <bool BF16, int V>
__device__ __forceinline__ void load_row(const void* p, int t, int E, int g, bool vec, float* v) {
  if constexpr (V >= 8) {
#pragma unroll
    for (int h = 0; h < V / 8; ++h) load_row8<BF16>(p, t, E, V / 8 * g + h, vec, v + 8 * h);
  } else {
    const int64_t base = int64_t(t) * E + V * g;
    if (vec && V * g < E) {
      if constexpr (BF16) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + base));
        v[0] = bf16lo(w.x); v[1] = bf16hi(w.x); v[2] = bf16lo(w.y); v[3] = bf16hi(w.y);
      } else {
        const float4 a = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + base));
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = V * g + i < E ? load_logit<BF16>(p, base + i) : neg_inf();
    }
  }
}

template <bool BF16>
__device__ __forceinline__ void store_row8(void* p, int t, int E, int g, bool vec, const float* v) {
  const int64_t base = int64_t(t) * E + 8 * g;
  if (8 * g >= E) return;
  if constexpr (BF16) {
    uint16_t* q = static_cast<uint16_t*>(p) + base;
    if (vec) {
      *reinterpret_cast<uint4*>(q) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (8 * g + i < E) q[i] = uint16_t(pack_bf16x2(v[i], 0.0f) & 0xFFFFu);
    }
  } else {
    float* q = static_cast<float*>(p) + base;
    if (vec) {
      *reinterpret_cast<float4*>(q) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(q + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (8 * g + i < E) q[i] = v[i];
    }
  }
}

// Sum and maximum over the G lanes of a group, the same in each of them.
template <int G>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int off = G / 2; off >= 1; off >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, off);
  return x;
}
template <int G>
__device__ __forceinline__ float group_max(float x) {
  if constexpr (G == 32) {
    float m;  // one instruction for the whole warp (sm_100a)
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
    return m;
  } else {
#pragma unroll
    for (int off = G / 2; off >= 1; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, off));
    return x;
  }
}

// A lane's two best candidates among its experts, best first: value and tag, the
// tag one bit (0..7) for the number among the lane's eight with the lane's place
// in the group above it.  Equal values: the lower number first.  NaN stands
// where there is no candidate: it wins no maximum and equals nothing.
struct Best {
  float m1, m2;
  uint32_t t1, t2;
};
__device__ __forceinline__ int tag_expert(uint32_t tag) { return 8 * int(tag >> 8) + __ffs(int(tag & 0xFFu)) - 1; }

// The two best of eight values, by merging sorted pairs (50 instructions; one
// value at a time takes 64).
__device__ __forceinline__ Best best_of8(const float* v, uint32_t place) {
  float a1[4], a2[4];
  uint32_t x1[4], x2[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const bool p = v[2 * j + 1] > v[2 * j];
    a1[j] = p ? v[2 * j + 1] : v[2 * j];
    a2[j] = p ? v[2 * j] : v[2 * j + 1];
    x1[j] = p ? 2u << (2 * j) : 1u << (2 * j);
    x2[j] = p ? 1u << (2 * j) : 2u << (2 * j);
  }
#pragma unroll
  for (int w = 2; w >= 1; w /= 2)
#pragma unroll
    for (int j = 0; j < w; ++j) {
      // lists 2j and 2j + 1: the numbers of the first are below the second's
      const bool p = a1[2 * j + 1] > a1[2 * j];
      const float lose = p ? a1[2 * j] : a1[2 * j + 1], next = p ? a2[2 * j + 1] : a2[2 * j];
      const uint32_t lx = p ? x1[2 * j] : x1[2 * j + 1], nx = p ? x2[2 * j + 1] : x2[2 * j];
      const bool q = next > lose || (!p && next == lose);
      const float top = p ? a1[2 * j + 1] : a1[2 * j];
      const uint32_t tx = p ? x1[2 * j + 1] : x1[2 * j];
      a1[j] = top;
      x1[j] = tx;
      a2[j] = q ? next : lose;
      x2[j] = q ? nx : lx;
    }
  return Best{a1[0], a2[0], x1[0] | place, x2[0] | place};
}

// The two best of the values whose bit in `used` is not set (none of them NaN).
__device__ __forceinline__ Best best_unused(const float* v, uint32_t used, uint32_t place) {
  const float none = __int_as_float(0x7FC00000);
  Best b{none, none, place, place};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if ((used >> i) & 1u) continue;
    if (!(v[i] <= b.m1)) {  // larger, or the first
      b.m2 = b.m1;
      b.t2 = b.t1;
      b.m1 = v[i];
      b.t1 = place | (1u << i);
    } else if (!(v[i] <= b.m2)) {
      b.m2 = v[i];
      b.t2 = place | (1u << i);
    }
  }
  return b;
}

struct LossPartials {
  float* sums;      // [blocks][E]
  int32_t* counts;  // [blocks][E]
  float* z;         // [blocks], squares scaled (Z_SCALE)
  int32_t* n;       // [blocks]
};

// Sum over the block in a fixed order, in thread 0 (the others get anything).
__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, off);
  return x;
}
template <int THREADS>
__device__ __forceinline__ double block_sum(double x, double* warps) {
  x = warp_sum(x);
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = x;
  __syncthreads();
  return warp_sum(int(threadIdx.x) < THREADS / 32 ? warps[threadIdx.x] : 0.0);
}

__device__ __forceinline__ double ld_cluster_f64(const double* p, uint32_t rank) {
  double x;
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(x) : "r"(smem_in_cta(p, rank)) : "memory");
  return x;
}

template <int THREADS>
struct FinishShared {
  double buf[THREADS];
  int32_t ibuf[THREADS];
  double sums[MOE_MAX_EXPERTS], counts[MOE_MAX_EXPERTS];  // this block's
  double zw[32], nw[32], dw[32];                          // of its warps
  double z, n;
};

// The cluster's blocks add the rows of partial sums up, block c the rows c, c + 8,
// ..., eight rows in flight per thread; block 0 then adds the blocks' sums, in
// order, and writes the results.  Sums in 64 bits (counts too, exactly): a few
// hundred terms of any size, and no cost next to the loads.
template <int THREADS>
__device__ __forceinline__ void finish_losses(const RouterLossArgs& a, const LossPartials& part, int blocks,
                                              FinishShared<THREADS>& sh) {
  const int c = int(cluster_ctarank()), tid = threadIdx.x;
  int width = 32;  // threads across the experts, a power of two; the others split the rows
  while (width < a.E) width *= 2;
  const int e = tid & (width - 1), slice = tid / width, slices = THREADS / width;
  double s = 0.0;
  int32_t cnt = 0;
  constexpr int U = 8;
  if (e < a.E)
    for (int b0 = c + RF_CLUSTER * slice; b0 < blocks; b0 += U * RF_CLUSTER * slices) {
      float x[U];
      int32_t y[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int b = b0 + i * RF_CLUSTER * slices;
        x[i] = b < blocks ? part.sums[int64_t(b) * a.E + e] : 0.0f;
        y[i] = b < blocks ? part.counts[int64_t(b) * a.E + e] : 0;
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        s += double(x[i]);
        cnt += y[i];
      }
    }
  double z = 0.0, n = 0.0;
  for (int b = c + RF_CLUSTER * tid; b < blocks; b += RF_CLUSTER * THREADS) {
    z += double(part.z[b]);
    n += double(part.n[b]);  // exact: below 2^53
  }
  sh.buf[tid] = s;
  sh.ibuf[tid] = cnt;
  __syncthreads();
  if (tid < a.E) {
    s = 0.0;
    cnt = 0;
    for (int w = 0; w < slices; ++w) {
      s += sh.buf[w * width + tid];
      cnt += sh.ibuf[w * width + tid];
    }
    sh.sums[tid] = s;
    sh.counts[tid] = double(cnt);
  }
  z = block_sum<THREADS>(z, sh.zw);
  n = block_sum<THREADS>(n, sh.nw);
  if (tid == 0) {
    sh.z = z;
    sh.n = n;
  }
  cluster_sync_all();
  if (c == 0) {
    double dot = 0.0;
    if (tid < a.E) {
      s = n = 0.0;
#pragma unroll
      for (int r = 0; r < RF_CLUSTER; ++r) {
        s += ld_cluster_f64(&sh.sums[tid], uint32_t(r));
        n += ld_cluster_f64(&sh.counts[tid], uint32_t(r));
      }
      a.prob_sums[tid] = float(s);
      a.counts[tid] = int32_t(n);
      dot = s * n;
    }
    dot = block_sum<THREADS>(dot, sh.dw);
    if (tid == 0) {
      z = n = 0.0;
      for (int r = 0; r < RF_CLUSTER; ++r) {
        z += ld_cluster_f64(&sh.z, uint32_t(r));
        n += ld_cluster_f64(&sh.n, uint32_t(r));
      }
      *a.tokens = int32_t(n);
      a.losses[0] = n > 0.0 ? float(double(a.E) * dot / (n * n * double(a.k))) : 0.0f;
      a.losses[1] = n > 0.0 ? float(z * Z_UNSCALE / n) : 0.0f;
    }
  }
  cluster_sync_all();  // no block leaves while its shared memory is read
}

__global__ void __cluster_dims__(RF_CLUSTER, 1, 1) __launch_bounds__(RF_THREADS)
    router_loss_finish_kernel(const RouterLossArgs a, const LossPartials part, const int blocks) {
  __shared__ FinishShared<RF_THREADS> sh;
  finish_losses<RF_THREADS>(a, part, blocks, sh);
}

// Selection: k rounds of a maximum over the group's lanes, each of which offers
// the best of its experts not yet kept.  A lane prepares its two best at once
// and looks again only after both were kept, which for 256 experts and k = 8
// happens about once per token -- a round is then a handful of instructions
// instead of a scan of eight values.  The lane that wins writes the kept value
// and id to shared memory; equal values go to the lowest lane, whose experts
// have the lower ids.
// ONE: a batch so small that a cluster of eight blocks does it all in one launch.
template <bool BF16, int G, bool ONE>
__global__ void __launch_bounds__(RL_THREADS, RL_BLOCKS_PER_SM<G>)
    router_loss_kernel(const RouterLossArgs a, const LossPartials part, const bool vec) {
  constexpr bool AHEAD = !RL_WIDE<G>;
  constexpr int GROUPS = 32 / G;               // tokens per warp
  constexpr int KL = (KEPT_MAX<G> + G - 1) / G;  // kept experts per lane
  __shared__ float2 list[RL_WARPS * GROUPS][KEPT_MAX<G> + 1];  // (value, id as bits) of a token's kept experts
  __shared__ float bsum[RL_WARPS][8 * G];
  __shared__ int32_t bcnt[RL_WARPS][8 * G];
  __shared__ float bz[RL_WARPS];
  __shared__ int32_t bn[RL_WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane & (G - 1), sub = lane / G;
  const uint32_t upto_me = (0xFFFFFFFFu >> (31 - lane)) & ~((1u << (sub * G)) - 1u);  // this group's lanes up to this one
  const int slot = warp * GROUPS + sub;
  const int E = a.E, k = a.k;
  const uint32_t place = uint32_t(g) << 8;
  // bits of the numbers that are no expert
  const uint32_t none = 8 * g >= E ? 0xFFu : (8 * g + 8 <= E ? 0u : (0xFFu << (E - 8 * g)) & 0xFFu);
  float acc[8], zsum = 0.0f;
  int32_t cnt[8], n = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0f, cnt[i] = 0;
  // counts of up to 255 tokens in bytes, then added to the words above
  uint32_t cnt_lo = 0, cnt_hi = 0, tokens = 0;
  auto spill_counts = [&] {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      cnt[i] += int32_t((cnt_lo >> (8 * i)) & 0xFFu);
      cnt[4 + i] += int32_t((cnt_hi >> (8 * i)) & 0xFFu);
    }
    cnt_lo = cnt_hi = tokens = 0;
  };
  constexpr int per = RL_WARPS * GROUPS;  // tokens per block and pass (T < 2^30: 32-bit token numbers)
  // whole warps take part in every round of shuffles: a group past the last
  // token works on the last one and keeps nothing
  const int step = int(gridDim.x) * per;
  int t0 = int(blockIdx.x) * per + warp * GROUPS;
  float next[8];  // AHEAD: the logits of the token after this one are on their way
  if (AHEAD && t0 < a.T) load_row8<BF16>(a.logits, min(t0 + sub, a.T - 1), E, g, vec, next);
  for (; t0 < a.T; t0 += step) {
    const bool in = t0 + sub < a.T;
    const int t = in ? t0 + sub : a.T - 1;
    const bool live = in && (!a.mask || a.mask[t] != 0);
    float v[8];
    if constexpr (AHEAD) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = next[i];
      if (t0 + step < a.T) load_row8<BF16>(a.logits, min(t0 + step + sub, a.T - 1), E, g, vec, next);
    } else {
      load_row8<BF16>(a.logits, t, E, g, vec, v);
    }
    // a NaN among the lane's logits makes this sum NaN (and so may infinities)
    bool nan = false;
    const float probe = ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    if (probe != probe) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (v[i] != v[i]) {
          nan = true;
          v[i] = neg_inf();  // NaN ranks last
        }
    }
    uint32_t used = none;
    Best b = none ? best_unused(v, used, place) : best_of8(v, place);
    float top = group_max<G>(b.m1);
    const float m = top;
    float2* slot_list = list[slot];
    for (int r = 0; r < k; ++r) {
      // the lowest of the group's lanes that hold the maximum
      if ((__ballot_sync(0xFFFFFFFFu, b.m1 == top) & upto_me) == (1u << lane)) {
        slot_list[r] = make_float2(b.m1, __uint_as_float(b.t1));
        used |= b.t1;
        b.m1 = b.m2;
        b.t1 = b.t2;
        b.m2 = __int_as_float(0x7FC00000);
        if (b.m1 != b.m1) b = best_unused(v, used, place);
      }
      top = group_max<G>(b.m1);
    }
    __syncwarp();
    // probabilities of the kept experts; the sum runs over 32 places as a
    // butterfly, kept expert r in place r -- the order of moe_router_topk
    float ex[KL];
    int32_t id[KL];
#pragma unroll
    for (int j = 0; j < KL; ++j) {
      const int r = g + j * G;
      ex[j] = 0.0f;
      if (r < k) {
        const float2 x = list[slot][r];
        ex[j] = expf(x.x - m);
        id[j] = tag_expert(__float_as_uint(x.y));
      }
    }
    float tree[KL];
#pragma unroll
    for (int j = 0; j < KL; ++j) tree[j] = ex[j];
#pragma unroll
    for (int w = KL / 2; w >= 1; w /= 2)
#pragma unroll
      for (int j = 0; j < w; ++j) tree[j] += tree[j + w];
    const float total = group_sum<G>(tree[0]);
    if (in) {
#pragma unroll
      for (int j = 0; j < KL; ++j) {
        const int r = g + j * G;
        if (r < k) {
          a.topk_idx[int64_t(t) * k + r] = id[j];
          a.topk_prob[int64_t(t) * k + r] = live ? ex[j] / total : 0.0f;
        }
      }
    }
    __syncwarp();  // the list is read before the next token's is written
    // softmax over all experts (what is no expert holds -inf and adds 0).  The
    // difference first: m log2(e) overflows where m is near the type's lowest value
    // (a row whose experts are all switched off by it) or its largest
    float se = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = fast_exp2((v[i] - m) * LOG2E);
      se += v[i];
    }
    if (nan) se = __int_as_float(0x7FC00000);
    se = group_sum<G>(se);
    const float lse = live ? m + __logf(se) : 0.0f;  // 3 ulp of log(se) <= log(256): 2^-19.4 absolute
    if (in && g == 0) a.lse[t] = lse;
    if (live) {
      const float inv = __fdividef(1.0f, se);
      const uint32_t kept = used & ~none & 0xFFu;
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = fmaf(v[i], inv, acc[i]);
      // bits 0..3 and 4..7 of `kept` to the bytes of two words
      cnt_lo += ((kept & 15u) * 0x00204081u) & 0x01010101u;
      cnt_hi += ((kept >> 4) * 0x00204081u) & 0x01010101u;
      if (g == 0) {
        zsum = fmaf(Z_SCALE * lse, Z_SCALE * lse, zsum);
        n += 1;
      }
    }
    if (++tokens == 255) spill_counts();
  }
  spill_counts();
  // the block's sums: over the warp's groups by shuffles, over the warps in order
#pragma unroll
  for (int off = G; off < 32; off <<= 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      acc[i] += __shfl_xor_sync(0xFFFFFFFFu, acc[i], off);
      cnt[i] += __shfl_xor_sync(0xFFFFFFFFu, cnt[i], off);
    }
    zsum += __shfl_xor_sync(0xFFFFFFFFu, zsum, off);
    n += __shfl_xor_sync(0xFFFFFFFFu, n, off);
  }
  if (sub == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      bsum[warp][8 * g + i] = acc[i];
      bcnt[warp][8 * g + i] = cnt[i];
    }
    if (g == 0) {
      bz[warp] = zsum;
      bn[warp] = n;
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += RL_THREADS) {
    float s = 0.0f;
    int32_t c = 0;
#pragma unroll
    for (int w = 0; w < RL_WARPS; ++w) {
      s += bsum[w][e];
      c += bcnt[w][e];
    }
    part.sums[int64_t(blockIdx.x) * E + e] = s;
    part.counts[int64_t(blockIdx.x) * E + e] = c;
  }
  if (threadIdx.x == 0) {
    float z = 0.0f;
    int32_t c = 0;
    for (int w = 0; w < RL_WARPS; ++w) {
      z += bz[w];
      c += bn[w];
    }
    part.z[blockIdx.x] = z;
    part.n[blockIdx.x] = c;
  }
  if constexpr (ONE) {
    __shared__ FinishShared<RL_THREADS> sh;
    cluster_sync_all();  // the blocks' partial sums, written to global memory, are there
    finish_losses<RL_THREADS>(a, part, RF_CLUSTER, sh);
  }
}

// Up to eight kept experts of more than 128, three of more than 64 or five of more than 32: sixteen lanes own a token, V
// consecutive experts each (4, 8 or 16 by E), so that a warp works on
// two tokens and what is not per expert -- the probabilities, the sums'
// exchanges -- costs half of what it does with 32 lanes.
// Selection without rounds: at least k experts reach the k-th largest of the
// lanes' maxima, so a bitonic sort of the sixteen maxima (ten exchanges) gives a
// threshold that about ten of 256 random logits pass for k = 8.  Those go to a
// list in ascending order of their ids, one lane takes each, and its place among
// the kept ones is the number of entries that come before it: larger, or equal
// and earlier in the list.  Where more than 16 pass (0.8 % of tokens with 256
// random logits, and rows of equal ones, as padding has them) only the first k of
// those that equal the threshold stay; more than 16 entries are two per lane, more
// than 32 (sixteen large logits in a row) are kept in k rounds over all logits.
// 262144 tokens, this kernel against the one above, us: 256 experts k = 8 114 / 182,
// k = 4 110 / 142, k = 1 108 / 117; 128 experts k = 8 86 / 135, k = 3 83 / 84, k = 2
// 82 / 76, k = 1 82 / 70; 64 experts k = 8 72 / 98, k = 6 71 / 78, k = 4 70 / 62 --
// the work hardly grows with k here, so few kept of few stay with the rounds.  Shorter
// batches, both launches: 4096 tokens 256 experts k = 8 11.8 / 14.8, k = 1 11.3 / 13.8, 128
// experts k = 8 10.3 / 11.8, k = 3 9.7 / 10.3, k = 1 9.7 / 10.2, 64 experts k = 8 10.2 / 11.3, k = 4
// 9.7 / 10.3; 32768 tokens 25.7 / 34.2, 24.1 / 25.6, 19.1 / 26.6, 18.4 / 19.5, 17.9 / 17.4,
// 16.4 / 21.0, 15.8 / 15.5: the same choice within 1 us.  More than eight kept stay with the rounds:
// 262144 tokens, 256 experts, k = 9 192, k = 16 287, k = 32 554.
// 290 warp instructions per token, most of them the selection's (the softmax and its sums need
// some 60), issued 66 % of the time; the first stalls are loads' and shared memory's
// latency.  Three blocks per SM (no spills; with four 44 bytes at sixteen experts per lane) or the
// next row's logits on their way: the same or slower.
constexpr int TOP_LANES = 16, TOP_K = 8, TOP_LIST = 32, TOP_BLOCKS_PER_SM = 4;

template <bool BF16, int V>
__global__ void __launch_bounds__(RL_THREADS, TOP_BLOCKS_PER_SM)
    router_loss_top8_kernel(const RouterLossArgs a, const LossPartials part, const bool vec) {
  constexpr int G = TOP_LANES, GROUPS = 32 / G, E_MAX = G * V;
  __shared__ float2 list[RL_WARPS * GROUPS][TOP_K + 1];  // (value, id as bits) of a token's kept experts, in order
  __shared__ uint8_t ids[RL_WARPS * GROUPS][TOP_LIST];   // experts that reach the threshold
  __shared__ __align__(16) float vals[RL_WARPS * GROUPS][G];  // the first sixteen of them, their logits
  __shared__ float bsum[RL_WARPS][E_MAX];
  __shared__ int32_t bcnt[E_MAX];
  __shared__ float bz[RL_WARPS];
  __shared__ int32_t bn[RL_WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane & (G - 1), sub = lane / G;
  const int slot = warp * GROUPS + sub;
  const int E = a.E, k = a.k;
  for (int e = threadIdx.x; e < E_MAX; e += RL_THREADS) bcnt[e] = 0;
  __syncthreads();
  // bits of the numbers that are experts
  const int have = min(max(E - V * g, 0), V);
  const uint32_t some = (1u << have) - 1u;
  float acc[V], zsum = 0.0f;
  int32_t n = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.0f;
  constexpr int per = RL_WARPS * GROUPS;
  const int step = int(gridDim.x) * per;
  int t0 = int(blockIdx.x) * per + warp * GROUPS;
  for (; t0 < a.T; t0 += step) {
    const bool in = t0 + sub < a.T;
    const int t = in ? t0 + sub : a.T - 1;
    float v[V];
    const bool live = in && (!a.mask || a.mask[t] != 0);
    load_row<BF16, V>(a.logits, t, E, g, vec, v);
    float x = neg_inf();
#pragma unroll
    for (int i = 0; i < V; ++i) x = fmaxf(x, v[i]);  // passes over NaN
#pragma unroll
    for (int size = 2; size <= G; size *= 2)
#pragma unroll
      for (int d = size / 2; d >= 1; d /= 2) {
        const float y = __shfl_xor_sync(0xFFFFFFFFu, x, d);
        x = ((g & d) == 0) == ((g & size) == 0) ? fmaxf(x, y) : fminf(x, y);
      }
    const float m = __shfl_sync(0xFFFFFFFFu, x, 0, G), least = __shfl_sync(0xFFFFFFFFu, x, k - 1, G);
    // softmax over all experts, as in the kernel above
    float ex[V], se = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      ex[i] = fast_exp2((v[i] - m) * LOG2E);
      se += ex[i];
    }
    if (se != se) {  // NaN (or infinities) among the lane's logits
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (v[i] != v[i]) v[i] = neg_inf();  // NaN ranks last
    }
    se = group_sum<G>(se);
    const float lse = live ? m + __logf(se) : 0.0f;
    if (in && g == 0) a.lse[t] = lse;
    if (live) {
      const float inv = __fdividef(1.0f, se);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = fmaf(ex[i], inv, acc[i]);
      if (g == 0) {
        zsum = fmaf(Z_SCALE * lse, Z_SCALE * lse, zsum);
        n += 1;
      }
    }
    uint32_t reach = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) reach |= v[i] >= least ? 1u << i : 0u;
    reach &= some;
    int upto, total;  // entries of the group's lanes up to this one, and of all
    auto count = [&] {
      upto = __popc(reach);
#pragma unroll
      for (int d = 1; d < G; d *= 2) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, upto, d, G);
        if (g >= d) upto += y;
      }
      total = __shfl_sync(0xFFFFFFFFu, upto, G - 1, G);
    };
    count();
    if (__any_sync(0xFFFFFFFFu, total > G)) {
      // equal logits (padding's): of those that equal the threshold the first k suffice
      const uint32_t above = [&] {
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) w |= v[i] > least ? 1u << i : 0u;
        return w & some;
      }();
      uint32_t equal = reach & ~above;
      reach = equal;
      count();
      int spare = k - (upto - __popc(equal));  // places left after the lanes before this one
      uint32_t drop = equal;
      for (; drop != 0 && spare > 0; --spare) drop &= drop - 1u;
      reach = above | (equal & ~drop);
      count();
    }
    auto keep = [&](int r, float value, int id) {
      list[slot][r] = make_float2(value, __int_as_float(id));
      if (live) atomicAdd(&bcnt[id], 1);
    };
    if (!__any_sync(0xFFFFFFFFu, total > TOP_LIST)) {
      for (int at = upto - __popc(reach); reach != 0; reach &= reach - 1u) ids[slot][at++] = uint8_t(V * g + __ffs(int(reach)) - 1);
      const bool more = __any_sync(0xFFFFFFFFu, total > G);
      __syncwarp();
      float value[2];
      int id[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        value[h] = __int_as_float(0x7FC00000);  // no entry: before nothing
        id[h] = 0;
        if (g + h * G < total) {
          id[h] = ids[slot][g + h * G];
          value[h] = fmaxf(load_logit<BF16>(a.logits, int64_t(t) * E + id[h]), neg_inf());
        }
      }
      vals[slot][g] = value[0];
      __syncwarp();
      // larger entries; equal ones are looked for afterwards, by two that come to
      // the same place
      int rank = 0;
#pragma unroll
      for (int j = 0; j < G; j += 4) {
        if (j == 12 && !__any_sync(0xFFFFFFFFu, total > j)) break;
        const float4 w = *reinterpret_cast<const float4*>(&vals[slot][j]);
        rank += (w.x > value[0]) + (w.y > value[0]) + (w.z > value[0]) + (w.w > value[0]);
      }
      if (more) {
        int rank1 = 0;
#pragma unroll
        for (int j = 0; j < G; ++j) {
          const float w0 = vals[slot][j], w1 = __shfl_sync(0xFFFFFFFFu, value[1], j, G);
          rank += w1 > value[0];
          rank1 += (w0 >= value[1]) + (w1 > value[1] || (w1 == value[1] && j < g));
        }
        if (g + G < total && rank1 < k) keep(rank1, value[1], id[1]);
      }
      float2* place = &list[slot][min(rank, TOP_K)];
      const float2 mine = make_float2(value[0], __int_as_float(id[0]));
      if (g < total && rank < k) *place = mine;
      __syncwarp();
      const bool lost = g < total && rank < k && __float_as_int(place->y) != id[0];
      if (__any_sync(0xFFFFFFFFu, lost)) {
#pragma unroll
        for (int j = 0; j < G; ++j) rank += vals[slot][j] == value[0] && j < g;
        if (g < total && rank < k) list[slot][rank] = mine;
      }
      if (g < total && rank < k && live) atomicAdd(&bcnt[id[0]], 1);
    } else {
      uint32_t left = some;
      for (int r = 0; r < k; ++r) {
        float best = __int_as_float(0x7FC00000);
        int who = 0;
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (((left >> i) & 1u) && !(v[i] <= best)) {
            best = v[i];
            who = i;
          }
        const float top = group_max<G>(best);
        // the lowest of the group's lanes that hold the maximum
        const uint32_t hold = __ballot_sync(0xFFFFFFFFu, best == top) >> (sub * G) & ((1u << G) - 1u);
        if (g == __ffs(int(hold)) - 1) {
          keep(r, best, V * g + who);
          left &= ~(1u << who);
        }
      }
    }
    __syncwarp();
    // probabilities of the kept experts, kept expert r in lane r: the sum's order
    // is the butterfly over 32 places of moe_router_topk, whose others are 0
    float p = 0.0f;
    int id = 0;
    if (g < k) {
      const float2 y = list[slot][g];
      p = expf(y.x - m);
      id = __float_as_int(y.y);
    }
    const float psum = group_sum<TOP_K>(p);
    if (in && g < k) {
      a.topk_idx[int64_t(t) * k + g] = id;
      a.topk_prob[int64_t(t) * k + g] = live ? p / psum : 0.0f;
    }
    __syncwarp();  // the list is read before the next token's is written
  }
  // the block's sums: over the warp's two groups by shuffles, over the warps in order
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] += __shfl_xor_sync(0xFFFFFFFFu, acc[i], G);
  zsum += __shfl_xor_sync(0xFFFFFFFFu, zsum, G);
  n += __shfl_xor_sync(0xFFFFFFFFu, n, G);
  if (sub == 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) bsum[warp][V * g + i] = acc[i];
    if (g == 0) {
      bz[warp] = zsum;
      bn[warp] = n;
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += RL_THREADS) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < RL_WARPS; ++w) s += bsum[w][e];
    part.sums[int64_t(blockIdx.x) * E + e] = s;
    part.counts[int64_t(blockIdx.x) * E + e] = bcnt[e];
  }
  if (threadIdx.x == 0) {
    float z = 0.0f;
    int32_t c = 0;
    for (int w = 0; w < RL_WARPS; ++w) {
      z += bz[w];
      c += bn[w];
    }
    part.z[blockIdx.x] = z;
    part.n[blockIdx.x] = c;
  }
}

// Gradient of the logits, on the same lanes.  The k kept logits' gradients are
// scattered to a zeroed row of shared memory, from which every lane adds its
// eight; only where a token lists an expert twice are they added one by one.
template <bool BF16, int G>
__global__ void __launch_bounds__(RL_THREADS, RL_BLOCKS_PER_SM<G>)
    router_bwd_kernel(const RouterBwdArgs a, const bool vec) {
  constexpr bool AHEAD = !RL_WIDE<G>;
  constexpr int GROUPS = 32 / G;
  constexpr int KL = (KEPT_MAX<G> + G - 1) / G;  // kept experts per lane
  __shared__ float share[8 * G];                      // f_e
  __shared__ __align__(16) float add[RL_WARPS * GROUPS][8 * G];  // gradients of a token's kept logits, else 0
  __shared__ uint8_t who[RL_WARPS * GROUPS][8 * G];
  __shared__ float2 list[RL_WARPS * GROUPS][KEPT_MAX<G> + 1];  // (id as bits, gradient of the kept logit)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane & (G - 1), sub = lane / G;
  const int slot = warp * GROUPS + sub;
  const int E = a.E, k = a.k;
  const float n = float(max(*a.tokens, 1));
  for (int e = threadIdx.x; e < 8 * G; e += RL_THREADS) share[e] = e < E ? float(a.counts[e]) / (n * float(k)) : 0.0f;
  for (int i = threadIdx.x; i < RL_WARPS * GROUPS * 8 * G; i += RL_THREADS) (&add[0][0])[i] = 0.0f;
  __syncthreads();
  const float cb = a.dlosses ? a.dlosses[0] * float(E) / n : 0.0f;
  const float cz = a.dlosses ? a.dlosses[1] * 2.0f / n : 0.0f;
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = share[8 * g + i];
  constexpr int per = RL_WARPS * GROUPS;  // tokens per block and pass (T < 2^30: 32-bit token numbers)
  // a token's inputs are loaded while the one before it is worked on
  float next[8], next_lse, p_next[KL], dp_next[KL];
  int32_t id_next[KL];
  bool live_next;
  auto fetch = [&](int t0) {
    const int t = min(t0 + sub, a.T - 1);
    if constexpr (AHEAD) load_row8<BF16>(a.logits, t, E, g, vec, next);
    next_lse = a.lse[t];
    live_next = t0 + sub < a.T && (!a.mask || a.mask[t] != 0);
    if (a.dprob) {
#pragma unroll
      for (int j = 0; j < KL; ++j) {
        const int r = g + j * G;
        p_next[j] = dp_next[j] = 0.0f;
        id_next[j] = 0;
        if (r < k) {
          p_next[j] = a.topk_prob[int64_t(t) * k + r];
          dp_next[j] = a.dprob[int64_t(t) * k + r];
          id_next[j] = a.topk_idx[int64_t(t) * k + r];
        }
      }
    }
  };
  const int step = int(gridDim.x) * per;
  int t0 = int(blockIdx.x) * per + warp * GROUPS;
  if (t0 < a.T) fetch(t0);
  for (; t0 < a.T; t0 += step) {
    const int t = t0 + sub;
    const bool in = t < a.T, live = live_next;
    const float lse = next_lse;
    float d[8], p[KL], dp[KL];
    int32_t id[KL];
    if constexpr (AHEAD) {
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] = next[i];
    } else {
      load_row8<BF16>(a.logits, min(t, a.T - 1), E, g, vec, d);
    }
#pragma unroll
    for (int j = 0; j < KL; ++j) {
      p[j] = p_next[j];
      dp[j] = dp_next[j];
      id[j] = id_next[j];
    }
    if (t0 + step < a.T) fetch(t0 + step);
    // s up to a factor that lse's rounding leaves (up to e^4 at 1e8, E where log E is lost in
    // it), hence the division by their sum
    float fs = 0.0f, one = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      d[i] = fast_exp2((d[i] - lse) * LOG2E);  // 0 where there is no expert
      one += d[i];
      fs = fmaf(d[i], f[i], fs);
    }
    one = group_sum<G>(one);
    fs = group_sum<G>(fs);
    const float inv = __fdividef(1.0f, one), cbs = cb * inv, czs = cz * lse * inv;
    fs *= inv;
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] *= fmaf(cbs, f[i] - fs, czs);
    if (a.dprob) {
      float dot = 0.0f;
#pragma unroll
      for (int j = 0; j < KL; ++j) dot = fmaf(p[j], dp[j], dot);
      dot = group_sum<G>(dot);
#pragma unroll
      for (int j = 0; j < KL; ++j) {
        const int r = g + j * G;
        if (r < k) {
          if (in && uint32_t(id[j]) >= uint32_t(E)) set_status(MOE_ERR_DEVICE_INDEX);
          list[slot][r] = make_float2(__int_as_float(id[j]), p[j] * (dp[j] - dot));
        }
      }
      float* own = add[slot];
      __syncwarp();
      // each kept expert's gradient to its place, and the number r beside it: a
      // number that is read back as another one tells of an id listed twice
#pragma unroll
      for (int j = 0; j < KL; ++j)
        if (g + j * G < k && uint32_t(id[j]) < uint32_t(E)) {
          own[id[j]] = list[slot][g + j * G].y;
          who[slot][id[j]] = uint8_t(g + j * G);
        }
      __syncwarp();
      bool twice = false;
#pragma unroll
      for (int j = 0; j < KL; ++j)
        if (g + j * G < k && uint32_t(id[j]) < uint32_t(E)) twice |= who[slot][id[j]] != uint8_t(g + j * G);
      if (__any_sync(0xFFFFFFFFu, twice)) {
        // in ascending order of r, by the lane that owns the expert
        for (int r = 0; r < k; ++r) {
          const float2 x = list[slot][r];
          const uint32_t i = uint32_t(__float_as_int(x.x)) - 8u * uint32_t(g);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (i == uint32_t(e)) d[e] += x.y;
        }
      } else {
        const float4 lo = reinterpret_cast<const float4*>(own)[2 * g], hi = reinterpret_cast<const float4*>(own)[2 * g + 1];
        d[0] += lo.x; d[1] += lo.y; d[2] += lo.z; d[3] += lo.w;
        d[4] += hi.x; d[5] += hi.y; d[6] += hi.z; d[7] += hi.w;
      }
      __syncwarp();  // read before the next token's values are written; the places go back to 0
#pragma unroll
      for (int j = 0; j < KL; ++j)
        if (g + j * G < k && uint32_t(id[j]) < uint32_t(E)) own[id[j]] = 0.0f;
    }
    if (!live) {
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] = 0.0f;
    }
    if (in) store_row8<BF16>(a.dlogits, t, E, g, vec, d);
  }
}

// Calls f with the group width of E experts as a compile-time number.
template <typename F>
cudaError_t by_group(int32_t E, F f) {
  if (E <= 8) return f(std::integral_constant<int, 1>());
  if (E <= 16) return f(std::integral_constant<int, 2>());
  if (E <= 32) return f(std::integral_constant<int, 4>());
  if (E <= 64) return f(std::integral_constant<int, 8>());
  if (E <= 128) return f(std::integral_constant<int, 16>());
  return f(std::integral_constant<int, 32>());
}

int32_t group_width(int32_t E) {
  int32_t g = 1;
  while (8 * g < E) g *= 2;
  return g;
}

unsigned loss_blocks(int32_t T, int32_t E) {
  const int32_t g = group_width(E);
  const int64_t per = int64_t(RL_WARPS) * (32 / g);
  const int64_t want = cdiv(int64_t(T), per);
  const int64_t cap = int64_t(device_sm_count()) * (g >= 16 ? RL_BLOCKS_PER_SM<16> : RL_BLOCKS_PER_SM<1>);
  return unsigned(want < cap ? want : cap);
}

unsigned top8_blocks(int32_t T) {
  const int64_t want = cdiv(int64_t(T), int64_t(RL_WARPS) * (32 / TOP_LANES));
  const int64_t cap = int64_t(device_sm_count()) * TOP_BLOCKS_PER_SM;
  return unsigned(want < cap ? want : cap);
}

// rows start on 16-byte boundaries and hold whole runs of eight experts
bool rows_vectorised(const void* p, const void* q, int32_t E) {
  return E % 8 == 0 && ((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(q)) & 15u) == 0;
}

}  // namespace

int64_t router_loss_workspace_bytes(int32_t T, int32_t E) {
  (void)T;
  // the most blocks the first kernel is launched with on a device of 1024 SMs
  const int64_t blocks = 1024 * RL_BLOCKS_PER_SM<16>;
  return blocks * (int64_t(E) * 8 + 8);
}

cudaError_t launch_router_losses(const RouterLossArgs& a, bool bf16, void* ws, cudaStream_t st) {
  // One launch where eight blocks need at most two passes over the tokens (512 tokens
  // of four experts: 8.4 us, two launches 10.4); more passes take longer than the
  // second launch
  const bool one = a.T <= 2 * RF_CLUSTER * RL_WARPS * (32 / group_width(a.E));
  const bool top8 = !one && a.k <= TOP_K && (a.E > 128 || (a.E > 64 && a.k >= 3) || (a.E > 32 && a.k >= 5));
  const unsigned blocks = one ? RF_CLUSTER : top8 ? top8_blocks(a.T) : loss_blocks(a.T, a.E);
  LossPartials part;
  part.sums = static_cast<float*>(ws);
  part.counts = reinterpret_cast<int32_t*>(part.sums + int64_t(blocks) * a.E);
  part.z = reinterpret_cast<float*>(part.counts + int64_t(blocks) * a.E);
  part.n = reinterpret_cast<int32_t*>(part.z + blocks);
  const bool vec = rows_vectorised(a.logits, a.logits, a.E);
  if (top8) {
    const auto kernel = a.E <= 4 * TOP_LANES ? (bf16 ? router_loss_top8_kernel<true, 4> : router_loss_top8_kernel<false, 4>)
                        : a.E <= 8 * TOP_LANES ? (bf16 ? router_loss_top8_kernel<true, 8> : router_loss_top8_kernel<false, 8>)
                                             : (bf16 ? router_loss_top8_kernel<true, 16> : router_loss_top8_kernel<false, 16>);
    kernel<<<blocks, RL_THREADS, 0, st>>>(a, part, vec);
    count_launch();
    router_loss_finish_kernel<<<RF_CLUSTER, RF_THREADS, 0, st>>>(a, part, int(blocks));
    count_launch();
    return cudaGetLastError();
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = RF_CLUSTER;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(RL_THREADS);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = one ? 1 : 0;
  const cudaError_t e = by_group(a.E, [&](auto G) {
    constexpr int W = decltype(G)::value;
    if (one)
      return cudaLaunchKernelEx(&cfg, bf16 ? router_loss_kernel<true, W, true> : router_loss_kernel<false, W, true>, a, part,
                                vec);
    return cudaLaunchKernelEx(&cfg, bf16 ? router_loss_kernel<true, W, false> : router_loss_kernel<false, W, false>, a, part,
                              vec);
  });
  if (e != cudaSuccess) return e;
  count_launch();
  if (one) return cudaSuccess;
  router_loss_finish_kernel<<<RF_CLUSTER, RF_THREADS, 0, st>>>(a, part, int(blocks));
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_router_bwd(const RouterBwdArgs& a, bool bf16, cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  const unsigned blocks = loss_blocks(a.T, a.E);
  const bool vec = rows_vectorised(a.logits, a.dlogits, a.E);
  count_launch();
  return by_group(a.E, [&](auto G) {
    if (bf16)
      router_bwd_kernel<true, decltype(G)::value><<<blocks, RL_THREADS, 0, st>>>(a, vec);
    else
      router_bwd_kernel<false, decltype(G)::value><<<blocks, RL_THREADS, 0, st>>>(a, vec);
    return cudaGetLastError();
  });
}

}  // namespace moe
