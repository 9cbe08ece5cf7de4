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
constexpr int RL_BLOCKS_PER_SM = 2;
// most experts that a token of a group of G lanes keeps
template <int G>
constexpr int KEPT_MAX = G < 4 ? 8 * G : 32;
constexpr int RF_CLUSTER = 8;  // blocks of the finishing cluster

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

// Experts 8g..8g+7 of row t; experts past E read as -inf.  `vec`: rows start
// on 16-byte boundaries and E is a multiple of 8.
template <bool BF16>
__device__ __forceinline__ void load_row8(const void* p, int64_t t, int E, int g, bool vec, float* v) {
  const int64_t base = t * E + 8 * g;
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
__device__ __forceinline__ void store_row8(void* p, int64_t t, int E, int g, bool vec, const float* v) {
  const int64_t base = t * E + 8 * g;
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

// Sum over the G lanes of a group, the same in each of them.
template <int G>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int off = G / 2; off >= 1; off >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, off);
  return x;
}

struct LossPartials {
  float* sums;      // [blocks][E]
  int32_t* counts;  // [blocks][E]
  float* z;         // [blocks]
  int32_t* n;       // [blocks]
};

template <bool BF16, int G>
__global__ void __launch_bounds__(RL_THREADS) router_loss_kernel(const RouterLossArgs a, const LossPartials part,
                                                                 const bool vec) {
  constexpr int GROUPS = 32 / G;               // tokens per warp
  __shared__ float list[RL_WARPS * GROUPS][KEPT_MAX<G> + 1];  // unnormalised probabilities of a token's kept experts
  __shared__ int32_t ids[RL_WARPS * GROUPS][KEPT_MAX<G> + 1];
  __shared__ float bsum[RL_WARPS][8 * G];
  __shared__ int32_t bcnt[RL_WARPS][8 * G];
  __shared__ float bz[RL_WARPS];
  __shared__ int32_t bn[RL_WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane & (G - 1), sub = lane / G;
  const int slot = warp * GROUPS + sub;
  const int E = a.E, k = a.k;
  float acc[8], zsum = 0.0f;
  int32_t cnt[8], n = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0f, cnt[i] = 0;
  const int64_t per = int64_t(RL_WARPS) * GROUPS;
  // whole warps take part in every round of shuffles: a group past the last
  // token works on the last one and keeps nothing
  for (int64_t t0 = int64_t(blockIdx.x) * per + warp * GROUPS; t0 < a.T; t0 += int64_t(gridDim.x) * per) {
    const bool in = t0 + sub < a.T;
    const int64_t t = in ? t0 + sub : int64_t(a.T) - 1;
    const bool live = in && (!a.mask || a.mask[t] != 0);
    float v[8];
    load_row8<BF16>(a.logits, t, E, g, vec, v);
    bool nan = false;
    uint32_t used = 0;  // bit i: expert 8g + i is kept or does not exist
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (v[i] != v[i]) {
        nan = true;
        v[i] = neg_inf();  // NaN ranks last
      }
      if (8 * g + i >= E) used |= 1u << i;
    }
    const uint32_t none = used;
    float m = 0.0f, total = 0.0f;
    for (int r = 0; r < k; ++r) {
      float bv = neg_inf();
      int be = 0x7fffffff;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (!((used >> i) & 1u) && (v[i] > bv || be == 0x7fffffff)) {
          bv = v[i];
          be = 8 * g + i;
        }
#pragma unroll
      for (int off = G / 2; off >= 1; off >>= 1) {
        const float ov = __shfl_xor_sync(0xFFFFFFFFu, bv, off);
        const int oe = __shfl_xor_sync(0xFFFFFFFFu, be, off);
        if (ov > bv || (ov == bv && oe < be)) {
          bv = ov;
          be = oe;
        }
      }
      if ((be >> 3) == g) used |= 1u << (be & 7);
      if (r == 0) m = bv;
      const float ex = expf(bv - m);
      total += ex;
      if (g == 0) {
        list[slot][r] = ex;
        ids[slot][r] = be;
      }
    }
    __syncwarp();
    if (in)
      for (int r = g; r < k; r += G) {
        a.topk_idx[t * k + r] = ids[slot][r];
        a.topk_prob[t * k + r] = live ? list[slot][r] / total : 0.0f;
      }
    __syncwarp();
    // softmax over all experts
    float e[8], se = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      e[i] = expf(v[i] - m);
      if ((none >> i) & 1u) e[i] = 0.0f;
      se += e[i];
    }
    if (nan) se = __int_as_float(0x7FC00000);
    se = group_sum<G>(se);
    const float lse = live ? m + logf(se) : 0.0f;
    if (in && g == 0) a.lse[t] = lse;
    if (live) {
      const float inv = 1.0f / se;
      used &= ~none;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        acc[i] += e[i] * inv;
        cnt[i] += int32_t((used >> i) & 1u);
      }
      if (g == 0) {
        zsum += lse * lse;
        n += 1;
      }
    }
  }
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
}

// Sum over the block in a fixed order, the same in every thread.
__device__ __forceinline__ double block_sum(double x, double* buf) {
  __syncthreads();
  buf[threadIdx.x] = x;
  __syncthreads();
  for (int s = RL_THREADS / 2; s >= 1; s >>= 1) {
    if (int(threadIdx.x) < s) buf[threadIdx.x] += buf[threadIdx.x + s];
    __syncthreads();
  }
  return buf[0];
}

// One cluster adds the blocks' rows up: block c owns the experts c, c + 8, ...
// in runs of 32 (lanes) x 8 slices of the rows (warps).  Sums in 64 bits: a
// few hundred terms of any size, and no cost next to the loads.
__global__ void __cluster_dims__(RF_CLUSTER, 1, 1) __launch_bounds__(RL_THREADS)
    router_loss_finish_kernel(const RouterLossArgs a, const LossPartials part, const int blocks) {
  __shared__ double buf[RL_THREADS];
  __shared__ int32_t ibuf[RL_WARPS][32];
  __shared__ double mine;  // this block's part of sum_e counts_e sums_e
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = int(cluster_ctarank());
  double dot = 0.0;
  for (int e0 = 32 * c; e0 < a.E; e0 += 32 * RF_CLUSTER) {
    const int e = e0 + lane;
    double s = 0.0;
    int32_t n = 0;
    if (e < a.E)
      for (int b = warp; b < blocks; b += RL_WARPS) {
        s += double(part.sums[int64_t(b) * a.E + e]);
        n += part.counts[int64_t(b) * a.E + e];
      }
    __syncthreads();
    buf[threadIdx.x] = s;
    ibuf[warp][lane] = n;
    __syncthreads();
    if (warp == 0 && e < a.E) {
      s = 0.0;
      n = 0;
      for (int w = 0; w < RL_WARPS; ++w) {
        s += buf[32 * w + lane];
        n += ibuf[w][lane];
      }
      a.prob_sums[e] = float(s);
      a.counts[e] = n;
      dot += s * double(n);
    }
  }
  const double all = block_sum(dot, buf);
  if (threadIdx.x == 0) mine = all;
  double z = 0.0, n = 0.0;
  if (c == 0) {
    for (int b = threadIdx.x; b < blocks; b += RL_THREADS) {
      z += double(part.z[b]);
      n += double(part.n[b]);  // exact: below 2^53
    }
    z = block_sum(z, buf);
    n = block_sum(n, buf);
  }
  cluster_sync_all();
  if (c == 0 && threadIdx.x == 0) {
    double total = 0.0;
    for (int r = 0; r < RF_CLUSTER; ++r) {
      double other;
      asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(other) : "r"(smem_in_cta(&mine, uint32_t(r))) : "memory");
      total += other;
    }
    *a.tokens = int32_t(n);
    a.losses[0] = n > 0.0 ? float(double(a.E) * total / (n * n * double(a.k))) : 0.0f;
    a.losses[1] = n > 0.0 ? float(z / n) : 0.0f;
  }
  cluster_sync_all();  // no block leaves while its shared memory is read
}

// Gradient of the logits.  A lane's eight gradients go through its own words of
// shared memory so that the token's kept experts can be added by index, in
// ascending order (an expert that a token lists twice gets both).
template <bool BF16, int G>
__global__ void __launch_bounds__(RL_THREADS) router_bwd_kernel(const RouterBwdArgs a, const bool vec) {
  constexpr int GROUPS = 32 / G;
  __shared__ float share[8 * G];                      // f_e
  __shared__ __align__(16) float grad[RL_THREADS][8];
  __shared__ float2 list[RL_WARPS * GROUPS][KEPT_MAX<G> + 1];  // (id as bits, gradient of the kept logit)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane & (G - 1), sub = lane / G;
  const int slot = warp * GROUPS + sub;
  const int E = a.E, k = a.k;
  const float n = float(max(*a.tokens, 1));
  for (int e = threadIdx.x; e < 8 * G; e += RL_THREADS) share[e] = e < E ? float(a.counts[e]) / (n * float(k)) : 0.0f;
  __syncthreads();
  const float cb = a.dlosses ? a.dlosses[0] * float(E) / n : 0.0f;
  const float cz = a.dlosses ? a.dlosses[1] * 2.0f / n : 0.0f;
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = share[8 * g + i];
  const int64_t per = int64_t(RL_WARPS) * GROUPS;
  for (int64_t t0 = int64_t(blockIdx.x) * per + warp * GROUPS; t0 < a.T; t0 += int64_t(gridDim.x) * per) {
    const bool in = t0 + sub < a.T;
    const int64_t t = in ? t0 + sub : int64_t(a.T) - 1;
    const bool live = in && (!a.mask || a.mask[t] != 0);
    float d[8];
    const float lse = a.lse[t];
    load_row8<BF16>(a.logits, t, E, g, vec, d);
    float fs = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      d[i] = 8 * g + i < E ? expf(d[i] - lse) : 0.0f;  // s
      fs = fmaf(d[i], f[i], fs);
    }
    fs = group_sum<G>(fs);
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] *= fmaf(cb, f[i] - fs, cz * lse);
    if (a.dprob) {
      float dot = 0.0f;
      for (int r = g; r < k; r += G) dot = fmaf(a.topk_prob[t * k + r], a.dprob[t * k + r], dot);
      dot = group_sum<G>(dot);
      __syncwarp();
      for (int r = g; r < k; r += G) {
        const int32_t e = a.topk_idx[t * k + r];
        if (in && (e < 0 || e >= E)) set_status(MOE_ERR_DEVICE_INDEX);
        list[slot][r] = make_float2(__int_as_float(e), a.topk_prob[t * k + r] * (a.dprob[t * k + r] - dot));
      }
      float4* own = reinterpret_cast<float4*>(grad[threadIdx.x]);
      own[0] = make_float4(d[0], d[1], d[2], d[3]);
      own[1] = make_float4(d[4], d[5], d[6], d[7]);
      __syncwarp();
      for (int r = 0; r < k; ++r) {
        const float2 x = list[slot][r];
        const int64_t i = int64_t(__float_as_int(x.x)) - 8 * g;  // ids outside [0, E) belong to no lane's experts
        if (i >= 0 && i < 8 && 8 * g + i < E) grad[threadIdx.x][i] += x.y;
      }
      const float4 lo = own[0], hi = own[1];
      d[0] = lo.x; d[1] = lo.y; d[2] = lo.z; d[3] = lo.w;
      d[4] = hi.x; d[5] = hi.y; d[6] = hi.z; d[7] = hi.w;
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

unsigned loss_blocks(int32_t T, int32_t E, int per_sm) {
  const int64_t per = int64_t(RL_WARPS) * (32 / group_width(E));
  const int64_t want = cdiv(int64_t(T), per), cap = int64_t(device_sm_count()) * per_sm;
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
  const int64_t blocks = 1024 * RL_BLOCKS_PER_SM;
  return blocks * (int64_t(E) * 8 + 8);
}

cudaError_t launch_router_losses(const RouterLossArgs& a, bool bf16, void* ws, cudaStream_t st) {
  const unsigned blocks = a.T > 0 ? loss_blocks(a.T, a.E, RL_BLOCKS_PER_SM) : 0;
  LossPartials part;
  part.sums = static_cast<float*>(ws);
  part.counts = reinterpret_cast<int32_t*>(part.sums + int64_t(blocks) * a.E);
  part.z = reinterpret_cast<float*>(part.counts + int64_t(blocks) * a.E);
  part.n = reinterpret_cast<int32_t*>(part.z + blocks);
  if (blocks > 0) {
    const bool vec = rows_vectorised(a.logits, a.logits, a.E);
    cudaError_t e = by_group(a.E, [&](auto G) {
      if (bf16)
        router_loss_kernel<true, decltype(G)::value><<<blocks, RL_THREADS, 0, st>>>(a, part, vec);
      else
        router_loss_kernel<false, decltype(G)::value><<<blocks, RL_THREADS, 0, st>>>(a, part, vec);
      return cudaGetLastError();
    });
    if (e != cudaSuccess) return e;
    count_launch();
  }
  router_loss_finish_kernel<<<RF_CLUSTER, RL_THREADS, 0, st>>>(a, part, int(blocks));
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_router_bwd(const RouterBwdArgs& a, bool bf16, cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  const unsigned blocks = loss_blocks(a.T, a.E, 8);
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
