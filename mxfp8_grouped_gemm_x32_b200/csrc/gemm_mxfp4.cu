// Persistent, warp-specialised grouped MXFP4 GEMM for B200 (sm_100a):
// D = (A * SFA) (B * SFB)^T over ragged expert groups, E2M1 operands with one
// E8M0 scale per 32 values along K, fp32 accumulation in TMEM.
//
// "Efficient MoE Training for Biological Foundation Models", Challenge 1 (one
// grouped submission over split_sizes), Challenge 3 / Figure 4 (gate_up GEMM,
// SwiGLU, probability and requantisation in one kernel); here with 4-bit
// operands on tcgen05.mma kind::mxf4.
//
// A 128-byte row of a K tile holds 256 values: 128 x 192 outputs per CTA, four
// K = 64 MMAs per K tile, each reading two scale bytes per row (scale_vec::2X),
// half of a column of a 128 x 4 scale atom.  The last K tile issues the MMAs
// that K reaches: the operand bytes past K are zero filled by TMA and the scale
// bytes past K are zero (2^-127).
//   warps 0..3    scales: from shared memory to TMEM through registers
//                 (tcgen05.st); warp w writes lanes 32w.. of every column, so each
//                 of the four reads all scales of the stage
//   warps 4..11   epilogue: two groups of four, each with an accumulator
//   warp 12       TMA producer (A, B boxes with 128-byte swizzle), ring of 4 or 5
//   warp 13       the same for the scales (bulk copies), ring of 6 or 8
//   warp 14       TMEM owner and MMA issuer; a stage is ready when its copies have
//                 landed and the four scale warps have stored its scales
// Mixtral gate_up (3.85 TFLOP) takes 770 us in a burst (5.0 PFLOP/s) and 860 in a
// long run, where the card's power limit sets the rate; down (1.92 TFLOP) 403.
// How it came there, on the same shape:
//   128 x 256 tiles, one accumulator, scales to TMEM by tcgen05.cp (as the MXFP8
//   kernel): 1070 us.  One tcgen05.cp occupies the tensor pipe for some 80 cycles
//   and a K tile needs six, against 4 x 130 for its MMAs; hence the scale warps.
//   Handing the one accumulator over took 1900 cycles per tile, hence two of 192
//   columns (an N = 192 MMA takes 97 cycles; 128 columns remain for the scales).
//   The issuing lane's own instructions took 615 cycles per K tile; with
//   descriptors by addition and barriers looked at ahead it issues four MMAs in 77.
//   Scales read from global memory by the scale warps: 1052; by bulk copies to
//   shared memory, a warp of their own for those: 862 (weights' scales eight copies
//   per K tile); the weights' scales in the order of the tiles, one copy: 783.
// Without its scales the kernel takes 643, without operand copies as well 557:
// what bounds it in a burst is 40 KB per K tile and SM from L2, 71 bytes a cycle.
// CTA pairs (256 x 192, half of B each) read less and were no faster: 808 us, and
// 1440 against 1454 us for a whole forward in a long run.
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

// Eight columns of the warp's 32 TMEM lanes from registers, and the wait for
// all stores of the warp.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// True in one lane of a converged warp.  The issuing warps run their loops with
// all lanes and issue from this one: what they compute stays in the uniform
// registers that tcgen05.mma and TMA take their operands from.  In a branch on the
// lane number every operand is moved there first, some 300 cycles per K tile.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void lds128(const uint8_t* p, uint32_t* r) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  r[0] = v.x; r[1] = v.y; r[2] = v.z; r[3] = v.w;
}

// Whether the phase with `parity` is complete; does not wait.
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// mbar_wait by one lane of a warp (32 lanes' polls of one barrier are taken one
// after the other), with its answer for all of them.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  bool ok = true;
  if (elect_one()) ok = mbar_wait(bar, parity, abort);
  return __all_sync(0xFFFFFFFFu, ok);
}

template <int EPI>
struct Cfg4 {
  static constexpr bool ROWS = EPI == EPI4_F24_ROWS;
  static constexpr int TM = 128, TN = 192, BKB = 128;  // tile rows, columns, bytes of K
  // the rows' staging buffers take the place of a stage and two of the scales' ring
  static constexpr int STAGES = ROWS ? 4 : 5;
  static constexpr int SF_WARPS = 4, EPI_WARPS = 8, PRODUCER = SF_WARPS + EPI_WARPS, SF_PRODUCER = PRODUCER + 1, ISSUER = PRODUCER + 2;
  static constexpr int THREADS = 32 * (ISSUER + 1);
  // TMEM columns: two accumulators, then per stage the scales of A (two atoms
  // of four columns) and of B (two atoms of six columns, eight apart)
  static constexpr uint32_t ACC_STRIDE = TN, SF_COL = 2 * TN, SF_STRIDE = 24, COLS = 512;
  static_assert(SF_COL + STAGES * SF_STRIDE <= COLS, "TMEM plan exceeds 512 columns");
  static constexpr int SMEM_A = TM * BKB, SMEM_B = TN * BKB;
  // scales of a K tile: two 512-byte atoms of A, 48 bytes a lane of B.  Their
  // ring is deeper than the operands': a K tile's scales take one hop more
  // (through the scale warps) to the MMA
  static constexpr int SMEM_SF = 1024 + MXFP4_TILE_SF, SF_RING = ROWS ? 6 : 8;
  static constexpr int OFF_A = 0, OFF_B = OFF_A + STAGES * SMEM_A, OFF_SF = OFF_B + STAGES * SMEM_B;
  static constexpr int OFF_STAGE = OFF_SF + SF_RING * SMEM_SF;
  // per epilogue warp: 32 rows of 32 packed f24 values, twice, the sources of its
  // TMA stores
  static constexpr int STAGE_WARP_BYTES = ROWS ? 2 * 32 * 96 : 0;
  static constexpr int OFF_BAR = OFF_STAGE + EPI_WARPS * STAGE_WARP_BYTES;
  static constexpr int NUM_BARS = 3 * STAGES + 2 * SF_RING + 5;
  static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8, OFF_GO = OFF_MISC + 16;
  static constexpr int SMEM_LAUNCH = OFF_GO + (MOE_MAX_EXPERTS + 1) * 4 + 1024;  // slack for 1 KB alignment
  static_assert(SMEM_LAUNCH <= 232448, "shared memory plan exceeds 227 KB");
};
// columns of D per tile: EPI4_SWIGLU 96 of h (96 gate and 96 up), else all
template <int EPI>
constexpr int TILE_COLS = EPI == EPI4_SWIGLU ? Cfg4<EPI>::TN / 2 : Cfg4<EPI>::TN;

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
  ti.n0 = n_idx * TILE_COLS<EPI>;
  ti.row_end = go[lo] + a.split_sizes[lo];
  return ti;
}

// TMA store of a 32-row, 96-byte box from shared memory, as one bulk group; waits
// until all of the thread's groups but the last have read their sources, or until
// all are complete.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];\n\tcp.async.bulk.commit_group;" ::"l"(
                   map),
               "r"(smem_u32(src)), "r"(c0), "r"(c1)
               : "memory");
}
__device__ __forceinline__ void bulk_wait_read1() { asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// A producer's place in the ring.  The barrier of the stage after the current one
// is looked at as soon as the current one's copies are issued, so that a stage that
// is free by then costs no wait.
template <int STAGES>
struct Ring {
  int stage = 0;
  uint32_t phase = 1;  // parity of the phase before the first: complete
  bool free_seen = true;
  __device__ __forceinline__ bool wait_empty(uint64_t* empty, volatile int* abort) {
    return free_seen || mbar_wait(&empty[stage], phase, abort);
  }
  __device__ __forceinline__ void advance(uint64_t* empty) {
    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
    free_seen = mbar_test_wait(&empty[stage], phase);
  }
};

// Shutting down early: lets the copies of the last armed stages land before the
// shared memory they write is released.
template <int STAGES>
__device__ __forceinline__ void drain_copies(uint64_t* loaded, uint32_t issued) {
  const uint32_t first = issued > uint32_t(STAGES) ? issued - STAGES : 0u;
  for (uint32_t i = first; i < issued; ++i) mbar_wait_drain(&loaded[i % STAGES], (i / STAGES) & 1u);
}

// A tile's epilogue for the warp that owns TMEM lanes 32q..; tl: its lanes and
// the accumulator's first column.  The columns are read as they are needed; the
// last read is followed by done(), which releases the accumulator.
template <int EPI, typename Done>
__device__ __forceinline__ void epilogue_tile4(const Gemm4Args& a, const CUtensorMap* tmY, const Tile4& ti, uint32_t tl,
                                               int q, int lane, uint32_t* stage, uint32_t& turn, Done done) {
  const int N = a.N;
  if constexpr (EPI == EPI4_SWIGLU) {
    const int r = ti.m0 + 32 * q + lane;
    const bool rv = r < ti.row_end;
    // 96 columns of h in three blocks: gate columns 32b.., up columns 96 + 32b..
    const float p = rv ? a.prob[r] : 0.0f;
    const int blocks = min(3, (N - ti.n0) >> 5);
    uint8_t* qr = a.q_out + int64_t(r) * mxfp4_pitch(N) + ti.n0 / 2;
    uint8_t* sfr = a.sf_out + sf_offset(0, r, 0, 0, (N + 127) / 128);
#pragma unroll 1
    for (int b = 0; b < blocks; ++b) {
      __syncwarp();  // lanes without a token skip the arithmetic; the whole warp reads TMEM
      uint32_t g[32], u[32];
      tmem_ld32(tl + 32 * b, g);
      tmem_ld32(tl + 96 + 32 * b, u);
      tc_wait_ld();
      if (b + 1 == blocks) done();
      if (!rv) continue;
      // fast exponential and division, 2^-19 relative together for |gate| below 8: with
      // expf and `/` the kernel takes 869 us instead of 770 (Mixtral), 379 instead of 239
      // (8191 x 2880, k 4), 99 instead of 73 (4096 x 2048, k 8), while a code of h, next to a border
      // between two, comes out as the other neighbour in 3 of 8191 and 6 of 8192 tokens
      float h[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float x = __uint_as_float(g[j]);
        h[j] = p * __fdividef(x, 1.0f + __expf(-x)) * __uint_as_float(u[j]);
      }
      const uint32_t sb = e8m0_from_amax_bits_e2m1(__float_as_uint(abs_max_n<32>(h)));
      const float inv = inv_scale_from_e8m0(sb);
#pragma unroll
      for (int j = 0; j < 32; ++j) h[j] *= inv;
      *reinterpret_cast<uint4*>(qr + 16 * b) =
          make_uint4(pack8_e2m1(h), pack8_e2m1(h + 8), pack8_e2m1(h + 16), pack8_e2m1(h + 24));
      const int kb = (ti.n0 >> 5) + b;
      uint8_t* sp = sfr + int64_t(kb >> 2) * 512 + (kb & 3);
      *sp = uint8_t(sb);
      if (32 * (kb + 1) == N)  // the padding blocks of the last atom
        for (int x = (kb & 3) + 1; x < 4; ++x) sp[x - (kb & 3)] = 0;
    }
  } else {
    // 32 columns at a time: 96 bytes a row into the warp's staging buffer and out
    // by a TMA store of 32 rows (rows past the group's last token are padding
    // rows of the same group; what they hold is never read).  Dropping the sums'
    // low eight bits saves a quarter of the rows' bytes and moves a value by less than
    // 2^-15, 1 / 128 of half a step of the bf16 output
    const int chunks = min(6, (N - ti.n0) >> 5);
    const bool any = ti.m0 + 32 * q < ti.row_end;
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
      __syncwarp();  // lane 0 issues the stores; the whole warp reads TMEM
      uint32_t v[32];
      tmem_ld32(tl + 32 * c, v);
      tc_wait_ld();
      if (c + 1 == chunks) done();
      if (!any) continue;  // uniform across the warp
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t u0 = v[4 * i], u1 = v[4 * i + 1], u2 = v[4 * i + 2], u3 = v[4 * i + 3];
        f24_pack4(u0, u1, u2, u3, v[3 * i], v[3 * i + 1], v[3 * i + 2]);
      }
      if (lane == 0) bulk_wait_read1();  // the buffer's last store, the one before the last, has read it
      __syncwarp();
      uint32_t* buf = stage + turn * (32 * 24);
      turn ^= 1u;
      uint4* row = reinterpret_cast<uint4*>(buf + 24 * lane);
#pragma unroll
      for (int i = 0; i < 6; ++i) row[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tma_store_2d(tmY, buf, (ti.n0 + 32 * c) * 3, ti.m0 + 32 * q);
    }
  }
}

template <int EPI>
__global__ void __launch_bounds__(Cfg4<EPI>::THREADS, 1)
    grouped_mxf4_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA32,
                             const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmY,
                             const Gemm4Args a) {
  using C = Cfg4<EPI>;
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* loaded = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);  // [STAGES] operands landed
  uint64_t* ready = loaded + STAGES;                                  // [STAGES] scales in TMEM
  uint64_t* empty = ready + STAGES;                                   // [STAGES] MMAs done: operands and scales
  uint64_t* sf_loaded = empty + STAGES;                               // [SF_RING] scales landed
  uint64_t* sf_empty = sf_loaded + C::SF_RING;                        // [SF_RING] read by the scale warps
  uint64_t* acc_full = sf_empty + C::SF_RING;  // [2]
  uint64_t* acc_empty = acc_full + 2;          // [2]
  uint64_t* drain = acc_empty + 2;             // MMA completion on the abort path
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  int* go = reinterpret_cast<int*>(smem + C::OFF_GO);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == C::PRODUCER && lane == 0) {
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmA32);
    prefetch_tmap(&tmB);
    if (EPI != EPI4_SWIGLU) prefetch_tmap(&tmY);
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&loaded[s], 1);
      mbar_init(&ready[s], C::SF_WARPS);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < C::SF_RING; ++s) {
      mbar_init(&sf_loaded[s], 1);
      mbar_init(&sf_empty[s], C::SF_WARPS);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], C::EPI_WARPS / 2);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == C::ISSUER) {
    tmem_alloc(tmem_slot, C::COLS);
    tmem_relinquish();
  }
  release_dependents();
  dependency_wait();  // the set-up above overlaps the kernel before this one
  for (int i = threadIdx.x; i <= a.E; i += C::THREADS) go[i] = a.group_offsets[i];
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // all 512 columns were allocated, so they start at column 0
  const uint32_t tmem = 0;
  const int nt = (a.N + TILE_COLS<EPI> - 1) / TILE_COLS<EPI>;
  const int ntiles = (go[a.E] >> 7) * nt;
  const int KT = (a.K + 127) / 128;      // scale atoms along K
  const int nkt = (a.K + 255) / 256;     // K tiles

  if (warp < C::SF_WARPS) {
    // ---------------- scales to TMEM ----------------
    // One lane polls; the others follow it through __syncwarp.  After a time-out the
    // loops run out without waiting.
    const uint32_t tq = tmem + (uint32_t(32 * warp) << 16) + C::SF_COL;
    int stage = 0, slot = 0;
    uint32_t phase = 1, slot_phase = 0;
    bool ok = true, landed = false;
    for (int t = blockIdx.x; t < ntiles; t += gridDim.x) {
      for (int kt = 0; kt < nkt; ++kt) {
        if (lane == 0 && ok && !landed) ok = mbar_wait(&sf_loaded[slot], slot_phase, abort_flag);
        __syncwarp();
        const uint8_t* sf = smem + C::OFF_SF + slot * C::SMEM_SF;
        // (A's second atom in a K tile that K does not reach holds anything; no
        // MMA is issued for it)
        uint32_t wa[8], wb[14];  // B: six words of each of the two atoms, and two that go along with the stores
        lds128(sf + lane * 16, wa);
        lds128(sf + 512 + lane * 16, wa + 4);
#pragma unroll
        for (int i = 0; i < 3; ++i) lds128(sf + 1024 + lane * 48 + 16 * i, wb + 4 * i);
        wb[12] = wb[13] = 0u;
        if (lane == 0 && ok) ok = mbar_wait(&empty[stage], phase, abort_flag);
        __syncwarp();  // (and every lane's loads are done)
        tc_fence_after();
        const uint32_t dst = tq + uint32_t(stage) * C::SF_STRIDE;
        tmem_st8(dst, wa);
        tmem_st8(dst + 8, wb);
        tmem_st8(dst + 16, wb + 6);
        if (lane == 0) mbar_arrive(&sf_empty[slot]);
        if (++slot == C::SF_RING) { slot = 0; slot_phase ^= 1u; }
        if (lane == 0) landed = mbar_test_wait(&sf_loaded[slot], slot_phase);
        __syncwarp();  // the wait is the whole warp's
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ready[stage]);
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
    }
  } else if (warp < C::PRODUCER) {
    // ---------------- epilogue ----------------
    const int q = warp & 3;                     // TMEM sub-partition this warp may read
    const int buf = (warp - C::SF_WARPS) >> 2;  // its accumulator: the CTA's even or odd tiles
    uint32_t* stage = reinterpret_cast<uint32_t*>(smem + C::OFF_STAGE + (warp - C::SF_WARPS) * C::STAGE_WARP_BYTES);
    uint32_t use = 0, turn = 0;  // turn: the staging buffer of the warp's next store
    for (int t = blockIdx.x + buf * gridDim.x; t < ntiles; t += 2 * gridDim.x) {
      const Tile4 ti = decode_tile4<EPI>(a, go, nt, t);
      if (!warp_wait(&acc_full[buf], use & 1u, abort_flag)) break;
      tc_fence_after();
      epilogue_tile4<EPI>(a, &tmY, ti, tmem + (uint32_t(32 * q) << 16) + uint32_t(buf) * C::ACC_STRIDE, q, lane, stage, turn, [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[buf]);
      });
      ++use;
    }
    if (EPI != EPI4_SWIGLU && lane == 0) bulk_wait_done();  // stores still reading the staging buffer
  } else if (warp == C::PRODUCER) {
    // ---------------- TMA producer ----------------
    if (elect_one()) {
      Ring<STAGES> r;
      uint32_t issued = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < ntiles && ok; t += gridDim.x) {
        const Tile4 ti = decode_tile4<EPI>(a, go, nt, t);
        // rows of A that hold tokens, in boxes of 32 unless nearly all do; the
        // rest of the stage holds anything (a row of A reaches no row but its own)
        const int rows = ti.row_end - ti.m0;
        const int boxes = rows > 96 ? 4 : (rows + 31) >> 5;
        const uint32_t bytes = uint32_t(boxes) * 32 * C::BKB + C::SMEM_B;
        for (int kt = 0; kt < nkt; ++kt) {
          if (!r.wait_empty(empty, abort_flag)) { ok = false; break; }
          ++issued;
          uint64_t* bar = &loaded[r.stage];
          mbar_arrive_expect_tx(bar, bytes);
          uint8_t* sa = smem + C::OFF_A + r.stage * C::SMEM_A;
          uint8_t* sb = smem + C::OFF_B + r.stage * C::SMEM_B;
          if constexpr (EPI == EPI4_SWIGLU) {
            tma_load_3d(sb, &tmB, bar, kt * C::BKB, ti.n0, 2 * ti.e);
            tma_load_3d(sb + C::SMEM_B / 2, &tmB, bar, kt * C::BKB, ti.n0, 2 * ti.e + 1);
          } else {
            tma_load_3d(sb, &tmB, bar, kt * C::BKB, ti.n0, ti.e);
          }
          if (boxes == 4)
            tma_load_2d(sa, &tmA, bar, kt * C::BKB, ti.m0);
          else
            for (int b = 0; b < boxes; ++b)
              tma_load_2d(sa + b * 32 * C::BKB, &tmA32, bar, kt * C::BKB, ti.m0 + 32 * b);
          r.advance(empty);
        }
      }
      if (*abort_flag) drain_copies<STAGES>(loaded, issued);
    }
    __syncwarp();
  } else if (warp == C::SF_PRODUCER) {
    // ---------------- scale atoms to shared memory ----------------
    if (elect_one()) {
      Ring<C::SF_RING> r;
      uint32_t issued = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < ntiles && ok; t += gridDim.x) {
        const Tile4 ti = decode_tile4<EPI>(a, go, nt, t);
        const uint8_t* sfa = a.sfa + int64_t(ti.m0 >> 7) * KT * 512;
        const uint8_t* sfb = a.sfb + (int64_t(ti.e) * nt + ti.n0 / TILE_COLS<EPI>) * nkt * MXFP4_TILE_SF;
        for (int kt = 0; kt < nkt; ++kt) {
          if (!r.wait_empty(sf_empty, abort_flag)) { ok = false; break; }
          ++issued;
          uint64_t* bar = &sf_loaded[r.stage];
          const uint32_t atoms = kt + 1 < nkt ? 1024u : uint32_t(KT - 2 * kt) * 512u;
          mbar_arrive_expect_tx(bar, MXFP4_TILE_SF + atoms);
          uint8_t* ss = smem + C::OFF_SF + r.stage * C::SMEM_SF;
          bulk_load(ss, sfa, atoms, bar);
          bulk_load(ss + 1024, sfb, MXFP4_TILE_SF, bar);
          sfa += 1024;
          sfb += MXFP4_TILE_SF;
          r.advance(sf_empty);
        }
      }
      if (*abort_flag) drain_copies<C::SF_RING>(sf_loaded, issued);
    }
    __syncwarp();
  } else {
    // ---------------- MMA issuer ----------------
    // One lane.  Its own instructions are what bounds the kernel when they take
    // longer than the MMAs they issue, so a K tile costs it as few as possible:
    // descriptors by one addition each, whole K tiles apart from the last, and
    // the next stage's barrier looked at behind the MMAs.
    if (elect_one()) {
      const uint64_t da0 = make_smem_desc(smem_u32(smem + C::OFF_A), 16, 1024, 2);
      const uint64_t db0 = make_smem_desc(smem_u32(smem + C::OFF_B), 16, 1024, 2);
      const int nfull = a.K / 256, rest = (a.K - 256 * nfull + 63) / 64;  // MMAs of the last, partial K tile
      int stage = 0;
      uint32_t phase = 0, it = 0;
      bool ok = true, seen = false;
      auto k_tile = [&](uint32_t acc, bool first, int steps) {
        if (!seen && !mbar_wait(&ready[stage], phase, abort_flag)) return false;
        if (!mbar_wait(&loaded[stage], phase, abort_flag)) return false;
        tc_fence_after();
        const uint64_t da = da0 + uint32_t(stage) * (C::SMEM_A >> 4), db = db0 + uint32_t(stage) * (C::SMEM_B >> 4);
        const uint32_t sf = C::SF_COL + uint32_t(stage) * C::SF_STRIDE;
#pragma unroll
        for (uint32_t kk = 0; kk < 4; ++kk) {
          if (int(kk) >= steps) break;
          const uint32_t h = kk >> 1, id = (kk & 1u) * 2u;
          tc_mma_mxf4(acc, da + 2 * kk, db + 2 * kk, make_idesc_mxf4(C::TM, C::TN, id, id), (sf + 4 * h) | (id << 30),
                      (sf + 8 + 8 * h) | (id << 30), kk != 0 ? 1u : uint32_t(!first));
        }
        tc_commit(&empty[stage]);
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        seen = mbar_test_wait(&ready[stage], phase);
        return true;
      };
      for (int t = blockIdx.x; t < ntiles && ok; t += gridDim.x, ++it) {
        const uint32_t buf = it & 1u, acc = buf * C::ACC_STRIDE;
        if (!mbar_wait(&acc_empty[buf], ((it >> 1) & 1u) ^ 1u, abort_flag)) { ok = false; break; }
#pragma unroll 1
        for (int kt = 0; kt < nfull && ok; ++kt) ok = k_tile(acc, kt == 0, 4);
        if (rest && ok) ok = k_tile(acc, nfull == 0, rest);
        if (ok) tc_commit(&acc_full[buf]);
      }
      if (*abort_flag) {
        // shutting down early: every MMA issued so far has to finish writing
        // TMEM before it is freed
        tc_commit(drain);
        mbar_wait_drain(drain, 0);
      }
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::ISSUER) {
    tc_fence_after();
    tmem_dealloc(tmem, C::COLS);
  }
}

// Plain scales [matrices][N][K/32] (gate_up: gate and up matrices in turn) to the
// order the GEMM reads them in, one thread per word of four bytes: for expert e,
// column tile j and K tile kt (256 values) lane l's 48 bytes hold, per 128-value
// atom h, the words of rows l, l + 32, ... of the tile -- gate_up: three of gate
// rows 96 j.. and three of up rows 96 j.., else six of rows 192 j...
__global__ void __launch_bounds__(256) mxfp4_tile_scales_kernel(const uint8_t* __restrict__ plain, int64_t ld, int32_t E,
                                                                int32_t N, int64_t nkb, bool gate_up, int32_t nt,
                                                                int64_t nkt, uint32_t* __restrict__ tiled) {
  const int64_t words = int64_t(E) * nt * nkt * (MXFP4_TILE_SF / 4);
  for (int64_t i = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; i < words; i += int64_t(gridDim.x) * blockDim.x) {
    const int w = int(i % (MXFP4_TILE_SF / 4));
    const int64_t tile = i / (MXFP4_TILE_SF / 4);
    const int64_t kt = tile % nkt, ej = tile / nkt;
    const int64_t e = ej / nt, j = ej % nt;
    const int lane = w / 12, h = (w % 12) / 6, c = w % 6;
    const int64_t matrix = gate_up ? 2 * e + c / 3 : e;
    const int64_t row = gate_up ? 96 * j + 32 * (c % 3) + lane : 192 * j + 32 * c + lane;
    const int64_t kb = 8 * kt + 4 * h;
    uint32_t v = 0;
    if (row < N) {
      const uint8_t* src = plain + (matrix * N + row) * ld + kb;
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (kb + b < nkb) v |= uint32_t(src[b]) << (8 * b);
    }
    tiled[i] = v;
  }
}

template <int EPI>
cudaError_t launch_epi4(const CUtensorMap& ma, const CUtensorMap& ma32, const CUtensorMap& mb, const CUtensorMap& my,
                        const Gemm4Args& a, int64_t tiles, cudaStream_t st) {
  static std::atomic<uint64_t> configured{0};
  auto kern = grouped_mxf4_gemm_kernel<EPI>;
  cudaError_t e = ensure_smem_limit(kern, Cfg4<EPI>::SMEM_LAUNCH, configured);
  if (e != cudaSuccess) return e;
  const int64_t sms = device_sm_count();
  return launch_dependent(kern, unsigned(tiles < sms ? tiles : sms), Cfg4<EPI>::THREADS, Cfg4<EPI>::SMEM_LAUNCH, st, ma,
                          ma32, mb, my, a);
}

// Bytes [rows][inner] (of one of `groups` matrices), rows `pitch` bytes apart, in
// boxes of box_bytes x box_rows; 128-byte boxes are swizzled.
cudaError_t make_map4(CUtensorMap* m, const void* base, int64_t inner, int64_t rows, int64_t groups, int64_t pitch,
                      int box_bytes, int box_rows) {
  EncodeTiledFn fn = get_encode_fn();
  if (!fn) return cudaErrorNotSupported;
  cuuint64_t dims[3] = {cuuint64_t(inner), cuuint64_t(rows), cuuint64_t(groups)};
  cuuint64_t strides[2] = {cuuint64_t(pitch), cuuint64_t(pitch * rows)};
  cuuint32_t box[3] = {cuuint32_t(box_bytes), cuuint32_t(box_rows), 1};
  cuuint32_t es[3] = {1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, groups ? 3 : 2, const_cast<void*>(base), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE,
                  box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_grouped_gemm_mxfp4(int epi, const uint8_t* a_codes, int64_t rows_cap, const uint8_t* b_codes,
                                      int64_t b_pitch, Gemm4Args a, int64_t max_rows, cudaStream_t st) {
  const int64_t groups = max_rows < a.E ? max_rows : a.E;
  const int64_t row_tiles = groups + max_rows / 128;  // at most: every group ends inside a tile
  const int64_t inner = a.K / 2, pitch = mxfp4_pitch(a.K);
  CUtensorMap ma, ma32, mb, my;
  cudaError_t e = make_map4(&ma, a_codes, inner, rows_cap, 0, pitch, 128, Cfg4<EPI4_SWIGLU>::TM);
  if (e == cudaSuccess) e = make_map4(&ma32, a_codes, inner, rows_cap, 0, pitch, 128, 32);
  if (e != cudaSuccess) return e;
  if (epi == EPI4_SWIGLU) {
    e = make_map4(&mb, b_codes, inner, a.N, 2 * int64_t(a.E), b_pitch, 128, TILE_COLS<EPI4_SWIGLU>);
    if (e != cudaSuccess) return e;
    return launch_epi4<EPI4_SWIGLU>(ma, ma32, mb, mb, a, row_tiles * cdiv(a.N, TILE_COLS<EPI4_SWIGLU>), st);
  }
  if (epi != EPI4_F24_ROWS) return cudaErrorInvalidValue;
  e = make_map4(&mb, b_codes, inner, a.N, a.E, b_pitch, 128, TILE_COLS<EPI4_F24_ROWS>);
  if (e == cudaSuccess) e = make_map4(&my, a.out, 3 * int64_t(a.N), rows_cap, 0, 3 * int64_t(a.N), 96, 32);
  if (e != cudaSuccess) return e;
  return launch_epi4<EPI4_F24_ROWS>(ma, ma32, mb, my, a, row_tiles * cdiv(a.N, TILE_COLS<EPI4_F24_ROWS>), st);
}

int64_t mxfp4_tiled_scale_bytes(int64_t E, int64_t N, int64_t K, bool gate_up) {
  return E * cdiv(N, gate_up ? TILE_COLS<EPI4_SWIGLU> : TILE_COLS<EPI4_F24_ROWS>) * cdiv(K, 256) * MXFP4_TILE_SF;
}

cudaError_t launch_mxfp4_tile_scales(const uint8_t* plain, int64_t ld, int32_t E, int32_t N, int64_t K, bool gate_up,
                                     uint8_t* tiled, cudaStream_t st) {
  const int64_t bytes = mxfp4_tiled_scale_bytes(E, N, K, gate_up);
  if (bytes == 0) return cudaSuccess;
  const int64_t want = cdiv(bytes / 4, 256), cap = int64_t(device_sm_count()) * 16;
  mxfp4_tile_scales_kernel<<<unsigned(want < cap ? want : cap), 256, 0, st>>>(
      plain, ld, E, N, K / 32, gate_up, int32_t(cdiv(N, gate_up ? TILE_COLS<EPI4_SWIGLU> : TILE_COLS<EPI4_F24_ROWS>)),
      cdiv(K, 256), reinterpret_cast<uint32_t*>(tiled));
  count_launch();
  return cudaGetLastError();
}

}  // namespace moe
