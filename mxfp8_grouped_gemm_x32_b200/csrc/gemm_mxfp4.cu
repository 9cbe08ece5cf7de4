// Persistent, warp-specialised grouped MXFP4 GEMM for B200 (sm_100a):
// D = (A * SFA) (B * SFB)^T over ragged expert groups, E2M1 operands with one
// E8M0 scale per 32 values along K, fp32 accumulation in TMEM.
//
// "Efficient MoE Training for Biological Foundation Models", Challenge 1 (one
// grouped submission over split_sizes), Challenge 3 / Figure 4 (gate_up GEMM,
// SwiGLU, probability and requantisation in one kernel); here with 4-bit
// operands on tcgen05.mma kind::mxf4.
//
// A 128-byte row of a K tile holds 256 values, so a tile is the MXFP8 one in
// bytes and twice it in K: 128 x 256 outputs per CTA, four K = 64 MMAs per K
// tile, each reading two scale bytes per row (scale_vec::2X) -- half of one
// 128 x 4 scale atom; a K tile loads two atoms per 128 rows.  The last K tile
// loads the atoms and issues the MMAs that K reaches: the operand bytes past K
// are zero filled by TMA and the scale bytes past K are zero (2^-127).
//   warp 0      TMA producer (A, B boxes with 128-byte swizzle; scale atoms by
//               bulk copy) into a 4-stage mbarrier ring
//   warp 1      TMEM owner and MMA issuer (scale atoms to TMEM by tcgen05.cp)
//   warps 2..9  epilogue: accumulator to registers, released, then stored
// Every wait is bounded, as in the MXFP8 kernel: on time-out the kernel records
// MOE_ERR_TIMEOUT, lets its copies and MMAs in flight finish and frees TMEM.
#include "mxfp4.cuh"

namespace moe {

namespace {

// D[tmem] (+)= (A * SFA) (B * SFB)^T, E2M1 operands from shared memory (K = 64
// per instruction), two E8M0 scales per row from TMEM.
__device__ __forceinline__ void tc_mma_mxf4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
          d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa_tmem), "r"(sfb_tmem)
      : "memory");
}

// Instruction descriptor of kind::mxf4: E2M1 x E2M1, both K-major, E8M0
// scales, M x N; the scale-factor ids are 0 or 2 (the byte pair of a column).
__host__ __device__ constexpr uint32_t make_idesc_mxf4(int M, int N, uint32_t a_sf_id, uint32_t b_sf_id) {
  return (b_sf_id & 3u) << 4      // B scale-factor id
         | 1u << 7                // A format E2M1
         | 1u << 10               // B format E2M1
         | uint32_t(N >> 3) << 17 // N / 8
         | 1u << 23               // scale format E8M0
         | uint32_t(M >> 4) << 24 // M / 16
         | (a_sf_id & 3u) << 29;  // A scale-factor id
}

struct Cfg4 {
  static constexpr int BM4 = 128, BN4 = 256, BKB = 128;  // tile rows, columns, bytes of K
  static constexpr int STAGES = 4, EPI_WARPS = 8, LEAD_WARPS = 2;
  static constexpr int THREADS = 32 * (LEAD_WARPS + EPI_WARPS);
  static constexpr int NC = 128;                          // accumulator columns per epilogue warp
  static constexpr uint32_t SFA_COL = 256, SFB_COL = SFA_COL + 8, COLS = 512;
  static constexpr int SMEM_A = BM4 * BKB, SMEM_B = BN4 * BKB, SMEM_SFA = 1024, SMEM_SFB = 2048;
  static constexpr int OFF_A = 0, OFF_B = OFF_A + STAGES * SMEM_A, OFF_SFA = OFF_B + STAGES * SMEM_B;
  static constexpr int OFF_SFB = OFF_SFA + STAGES * SMEM_SFA, OFF_BAR = OFF_SFB + STAGES * SMEM_SFB;
  static constexpr int NUM_BARS = 2 * STAGES + 3;
  static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8, OFF_GO = OFF_MISC + 16;
  static constexpr int STAGE_WARP_BYTES = 2560;
  static constexpr int OFF_STAGE = (OFF_GO + (MOE_MAX_EXPERTS + 1) * 4 + 127) / 128 * 128;
  static constexpr int SMEM_LAUNCH = OFF_STAGE + EPI_WARPS * STAGE_WARP_BYTES + 1024;  // slack for 1 KB alignment
  static_assert(SMEM_LAUNCH <= 232448, "shared memory plan exceeds 227 KB");
};

struct Tile4 {
  int e, m0, n0, row_end;
};

// Tile t of the schedule: experts in order, each expert's row tiles fastest,
// so that CTAs working at the same time share weight panels in L2.
template <int EPI>
__device__ __forceinline__ Tile4 decode_tile4(const Gemm4Args& a, const int* go, int nt, int t) {
  int lo = 0, hi = a.E - 1;  // last expert whose first tile is <= t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((go[mid] >> 7) * nt <= t) lo = mid; else hi = mid - 1;
  }
  const int mt = (go[lo + 1] - go[lo]) >> 7;
  const int local = t - (go[lo] >> 7) * nt;
  const int n_idx = local / mt, m_idx = local - n_idx * mt;
  Tile4 ti;
  ti.e = lo;
  ti.m0 = go[lo] + (m_idx << 7);
  ti.n0 = n_idx * (EPI == EPI4_SWIGLU ? 128 : 256);
  ti.row_end = go[lo] + a.split_sizes[lo];
  return ti;
}

// v holds the warp's accumulator values: EPI4_SWIGLU 64 gate + 64 up columns,
// EPI4_F24_ROWS 128 columns; the warp owns rows 32q.. of the tile and column half `half`.
template <int EPI>
__device__ __forceinline__ void epilogue_tile4(const Gemm4Args& a, const Tile4& ti, uint32_t* v, int q, int half,
                                               int lane, uint32_t* stage) {
  const int r = ti.m0 + 32 * q + lane;
  const bool rv = r < ti.row_end;
  const int N = a.N;
  if constexpr (EPI == EPI4_SWIGLU) {
    const int nb = ti.n0 + 64 * half;
    if (nb >= N || !rv) return;
    const float p = a.prob[r];
    uint32_t hw[8];  // 64 codes
    uint32_t sbs = 0;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      float h[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float g = __uint_as_float(v[32 * b + j]);
        const float u = __uint_as_float(v[64 + 32 * b + j]);
        h[j] = p * __fdividef(g, 1.0f + __expf(-g)) * u;
      }
      const uint32_t sb = e8m0_from_amax_bits_e2m1(__float_as_uint(abs_max_n<32>(h)));
      const float inv = inv_scale_from_e8m0(sb);
#pragma unroll
      for (int j = 0; j < 32; ++j) h[j] *= inv;
#pragma unroll
      for (int j = 0; j < 4; ++j) hw[4 * b + j] = pack8_e2m1(h + 8 * j);
      sbs |= sb << (8 * b);
    }
    // 32 bytes, one sector per row (N is a multiple of 64, so rows start on sectors)
    stg256(a.q_out + int64_t(r) * (N / 2) + nb / 2, hw);
    const int kb0 = nb >> 5;
    uint8_t* sfp = a.sf_out + sf_offset(0, r, kb0, 0, (N + 127) / 128);
    if (nb + 64 == N && (kb0 & 3) == 0)
      *reinterpret_cast<uint32_t*>(sfp) = sbs;  // also zero the two padding blocks of the last atom
    else
      *reinterpret_cast<uint16_t*>(sfp) = uint16_t(sbs);
  } else {
    const int nb = ti.n0 + 128 * half;
    if (nb >= N) return;  // uniform across the warp
    const int ncols = min(128, N - nb);
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const uint32_t u0 = v[4 * i], u1 = v[4 * i + 1], u2 = v[4 * i + 2], u3 = v[4 * i + 3];
      f24_pack4(u0, u1, u2, u3, v[3 * i], v[3 * i + 1], v[3 * i + 2]);
    }
    warp_store_rows<96>(stage, rv ? a.out + (int64_t(r) * N + nb) * 3 : nullptr, v, ncols * 3, lane);
  }
}

template <int EPI>
__global__ void __launch_bounds__(Cfg4::THREADS, 1)
    grouped_mxf4_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                             const Gemm4Args a) {
  using C = Cfg4;
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* empty = full + STAGES;
  uint64_t* acc_full = empty + STAGES;
  uint64_t* acc_empty = acc_full + 1;
  uint64_t* drain = acc_empty + 1;  // MMA completion on the abort path
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  int* go = reinterpret_cast<int*>(smem + C::OFF_GO);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, C::EPI_WARPS);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::COLS);
    tmem_relinquish();
  }
  for (int i = threadIdx.x; i <= a.E; i += C::THREADS) go[i] = a.group_offsets[i];
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int nt = (a.N + (EPI == EPI4_SWIGLU ? 127 : 255)) / (EPI == EPI4_SWIGLU ? 128 : 256);
  const int ntiles = (go[a.E] >> 7) * nt;
  const int KT = (a.K + 127) / 128;      // scale atoms along K
  const int nkt = (a.K + 255) / 256;     // K tiles

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer ----------------
      prefetch_tmap(&tmA);
      prefetch_tmap(&tmB);
      const int b_RT = (a.N + 127) / 128;  // row tiles of a group in B's scale layout
      int stage = 0;
      uint32_t phase = 0, issued = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < ntiles && ok; t += gridDim.x) {
        const Tile4 ti = decode_tile4<EPI>(a, go, nt, t);
        const uint8_t* sfa = a.sfa + int64_t(ti.m0 >> 7) * KT * 512;
        // the two 128-row scale tiles of B: gate and up rows, or two neighbours
        // (rows past N: any tile of the group, their columns are never stored)
        const int rb = ti.n0 >> 7;
        const uint8_t *sfb0, *sfb1;
        if constexpr (EPI == EPI4_SWIGLU) {
          sfb0 = a.sfb + (int64_t(2 * ti.e) * b_RT + rb) * KT * 512;
          sfb1 = sfb0 + int64_t(b_RT) * KT * 512;
        } else {
          sfb0 = a.sfb + (int64_t(ti.e) * b_RT + rb) * KT * 512;
          sfb1 = rb + 1 < b_RT ? sfb0 + int64_t(KT) * 512 : sfb0;
        }
        for (int kt = 0; kt < nkt; ++kt) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag)) { ok = false; break; }
          ++issued;
          uint64_t* bar = &full[stage];
          const uint32_t sfbytes = min(2, KT - 2 * kt) * 512;
          mbar_arrive_expect_tx(bar, uint32_t(a.a_box) * C::BKB + C::SMEM_B + 3 * sfbytes);
          uint8_t* sb = smem + C::OFF_B + stage * C::SMEM_B;
          tma_load_2d(smem + C::OFF_A + stage * C::SMEM_A, &tmA, bar, kt * C::BKB, ti.m0);
          if constexpr (EPI == EPI4_SWIGLU) {
            tma_load_3d(sb, &tmB, bar, kt * C::BKB, ti.n0, 2 * ti.e);
            tma_load_3d(sb + C::SMEM_B / 2, &tmB, bar, kt * C::BKB, ti.n0, 2 * ti.e + 1);
          } else {
            tma_load_3d(sb, &tmB, bar, kt * C::BKB, ti.n0, ti.e);
          }
          uint8_t* ssfa = smem + C::OFF_SFA + stage * C::SMEM_SFA;
          uint8_t* ssfb = smem + C::OFF_SFB + stage * C::SMEM_SFB;
          bulk_load(ssfa, sfa + int64_t(kt) * 1024, sfbytes, bar);
          bulk_load(ssfb, sfb0 + int64_t(kt) * 1024, sfbytes, bar);
          bulk_load(ssfb + 1024, sfb1 + int64_t(kt) * 1024, sfbytes, bar);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      if (*abort_flag) {
        // shutting down early: let the copies of the last armed stages land
        // before the shared memory they write is released
        const uint32_t first = issued > uint32_t(STAGES) ? issued - STAGES : 0u;
        for (uint32_t i = first; i < issued; ++i) mbar_wait_drain(&full[i % STAGES], (i / STAGES) & 1u);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ---------------- MMA issuer ----------------
      int stage = 0;
      uint32_t phase = 0, acc_it = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < ntiles && ok; t += gridDim.x) {
        if (!mbar_wait(acc_empty, (acc_it & 1u) ^ 1u, abort_flag)) break;
        tc_fence_after();
        for (int kt = 0; kt < nkt; ++kt) {
          if (!mbar_wait(&full[stage], phase, abort_flag)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + C::OFF_A + stage * C::SMEM_A);
          const uint32_t sb = smem_u32(smem + C::OFF_B + stage * C::SMEM_B);
          const uint32_t ssfa = smem_u32(smem + C::OFF_SFA + stage * C::SMEM_SFA);
          const uint32_t ssfb = smem_u32(smem + C::OFF_SFB + stage * C::SMEM_SFB);
          const int atoms = min(2, KT - 2 * kt);
          for (int h = 0; h < atoms; ++h) {
            tc_cp_32x128b_warpx4(tmem + C::SFA_COL + 4 * h, make_smem_desc(ssfa + 512 * h, 0, 128, 0));
            tc_cp_32x128b_warpx4(tmem + C::SFB_COL + 8 * h, make_smem_desc(ssfb + 512 * h, 0, 128, 0));
            tc_cp_32x128b_warpx4(tmem + C::SFB_COL + 8 * h + 4, make_smem_desc(ssfb + 1024 + 512 * h, 0, 128, 0));
          }
          const int steps = min(4, (a.K - 256 * kt + 63) / 64);
#pragma unroll
          for (uint32_t kk = 0; kk < 4; ++kk) {
            if (int(kk) >= steps) break;
            const uint32_t h = kk >> 1, id = (kk & 1u) * 2u;
            tc_mma_mxf4(tmem, make_smem_desc(sa + 32 * kk, 16, 1024, 2), make_smem_desc(sb + 32 * kk, 16, 1024, 2),
                        make_idesc_mxf4(C::BM4, C::BN4, id, id), (tmem + C::SFA_COL + 4 * h) | (id << 30),
                        (tmem + C::SFB_COL + 8 * h) | (id << 30), (kt | int(kk)) != 0 ? 1u : 0u);
          }
          tc_commit(&empty[stage]);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        tc_commit(acc_full);
        ++acc_it;
      }
      if (*abort_flag) {
        // shutting down early: every MMA issued so far has to finish writing
        // TMEM before it is freed
        tc_commit(drain);
        mbar_wait_drain(drain, 0);
      }
    }
  } else {
    // ---------------- epilogue warps ----------------
    const int q = warp & 3;                        // TMEM sub-partition this warp may read
    const int half = (warp - C::LEAD_WARPS) >> 2;  // which half of the tile's columns
    uint32_t* stage = reinterpret_cast<uint32_t*>(smem + C::OFF_STAGE + (warp - C::LEAD_WARPS) * C::STAGE_WARP_BYTES);
    uint32_t acc_it = 0;
    uint32_t v[C::NC];
    for (int t = blockIdx.x; t < ntiles; t += gridDim.x) {
      const Tile4 ti = decode_tile4<EPI>(a, go, nt, t);
      if (!mbar_wait(acc_full, acc_it & 1u, abort_flag)) break;
      tc_fence_after();
      const uint32_t tl = tmem + (uint32_t(32 * q) << 16);
      if constexpr (EPI == EPI4_SWIGLU) {  // gate columns 64*half.., up columns 128 + 64*half..
        tmem_ld64(tl + 64 * half, v);
        tmem_ld64(tl + 128 + 64 * half, v + 64);
      } else {
        tmem_ld128(tl + 128 * half, v);
      }
      tc_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty);
      epilogue_tile4<EPI>(a, ti, v, q, half, lane, stage);
      ++acc_it;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::COLS);
  }
}

template <int EPI>
cudaError_t launch_epi4(const CUtensorMap& ma, const CUtensorMap& mb, const Gemm4Args& a, int64_t tiles,
                        cudaStream_t st) {
  static std::atomic<uint64_t> configured{0};
  auto kern = grouped_mxf4_gemm_kernel<EPI>;
  cudaError_t e = ensure_smem_limit(kern, Cfg4::SMEM_LAUNCH, configured);
  if (e != cudaSuccess) return e;
  const int64_t sms = device_sm_count();
  kern<<<unsigned(tiles < sms ? tiles : sms), Cfg4::THREADS, Cfg4::SMEM_LAUNCH, st>>>(ma, mb, a);
  count_launch();
  return cudaGetLastError();
}

}  // namespace

// max_rows: routed rows T*k -- no group is larger, and no more 128-row tiles
// than experts or rows are occupied.
cudaError_t launch_grouped_gemm_mxfp4(int epi, const uint8_t* a_codes, int64_t rows_cap, const uint8_t* b_codes,
                                      Gemm4Args a, int64_t max_rows, cudaStream_t st) {
  // a small batch's groups end within the first rows of their only tile: the
  // A box then covers those (rounded to the swizzle's 8 rows), and the rest of
  // the stage holds anything -- a row of A reaches no row but its own
  a.a_box = max_rows >= 128 ? 128 : int32_t(cdiv(max_rows, 8) * 8);
  const int64_t groups = max_rows < a.E ? max_rows : a.E;
  const int64_t row_tiles = groups + max_rows / 128;  // at most: every group ends inside a tile
  CUtensorMap ma, mb;
  cudaError_t e = make_map_2d(&ma, a_codes, uint64_t(a.K / 2), uint64_t(rows_cap), uint32_t(a.a_box));
  if (e != cudaSuccess) return e;
  if (epi == EPI4_SWIGLU) {
    e = make_map_3d(&mb, b_codes, uint64_t(a.K / 2), uint64_t(a.N), 2 * uint64_t(a.E), 128);
    if (e != cudaSuccess) return e;
    return launch_epi4<EPI4_SWIGLU>(ma, mb, a, row_tiles * cdiv(a.N, 128), st);
  }
  if (epi != EPI4_F24_ROWS) return cudaErrorInvalidValue;
  e = make_map_3d(&mb, b_codes, uint64_t(a.K / 2), uint64_t(a.N), uint64_t(a.E), 256);
  if (e != cudaSuccess) return e;
  return launch_epi4<EPI4_F24_ROWS>(ma, mb, a, row_tiles * cdiv(a.N, 256), st);
}

}  // namespace moe
