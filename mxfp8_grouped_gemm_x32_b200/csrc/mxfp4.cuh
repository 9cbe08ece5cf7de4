// MXFP4: E2M1 codes with one E8M0 scale per 32 values -- device helpers and
// launch interfaces of the quantisation kernels and of the grouped GEMM.
#pragma once
#include "gemm.cuh"

namespace moe {

// E8M0 scale byte from the bit pattern of a block's amax: the smallest power
// of two 2^s with amax / 2^s <= 6 (the largest E2M1 magnitude), the rule the
// E4M3 codes use with 448.  amax = m * 2^e with m in [1, 2) gives s = e - 2,
// plus one when m > 1.5; clamped to [-127, 127].  Zero gives byte 0, NaN and
// infinities 0xFF.  (A subnormal amax, e < -126, needs no more than s = -127.)
__device__ __forceinline__ uint32_t e8m0_from_amax_bits_e2m1(uint32_t abits) {
  const uint32_t ef = abits >> 23;
  if (ef == 0xFFu) return 0xFFu;
  const int b = int(ef) - 2 + ((abits & 0x7FFFFFu) > 0x400000u ? 1 : 0);
  return b < 0 || ef == 0u ? 0u : uint32_t(b);
}

// Eight fp32 values -> eight E2M1 codes, value 0 in the lowest four bits
// (round to nearest even, saturating to +-6).
__device__ __forceinline__ uint32_t pack8_e2m1(const float* f) {
  uint32_t r;
  asm("{\n .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}"
      : "=r"(r)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}

// Bytes between rows of the codes that the library lays out itself: whole 128-byte
// lines, so that no 128-byte box row of a TMA load straddles two (2880 values,
// 1440 bytes a row: the GEMMs' loads ran at 38 bytes per cycle and SM, against 71
// for aligned rows).
__host__ __device__ __forceinline__ int64_t mxfp4_pitch(int64_t K) { return (K / 2 + 127) / 128 * 128; }

// Source of the quantiser / destination of the dequantiser: `rows` rows of K
// values per group, contiguous; codes [groups][rows], rows `ldq` bytes apart,
// scales blocked.
struct Mxfp4Args {
  const void* src;
  void* dst;
  uint8_t* q;
  uint8_t* sf;
  int32_t groups;
  int64_t rows, K, ldq;
  FastDiv blocks_div, rows_div;  // K / 32 and rows (set by the launcher)
};
// blocks of 32 values have to be fewer than this (their numbers and a grid's
// stride fit 31 bits)
constexpr int64_t MXFP4_MAX_BLOCKS = (int64_t(1) << 29) - (int64_t(1) << 22);
cudaError_t launch_mxfp4_quant(Mxfp4Args a, bool bf16, cudaStream_t st);
cudaError_t launch_mxfp4_dequant(Mxfp4Args a, bool bf16, cudaStream_t st);

// x [T][H] bf16 -> MXFP4 rows of the permuted order: each token is quantised
// once and written to its rows slot_to_row[t*k + j].  Padding rows of the
// groups are not written (the GEMMs' rows there are never stored).
struct Mxfp4ScatterArgs {
  const uint8_t* src;
  int32_t T, H, k;
  const int32_t* slot_to_row;
  uint8_t* q;   // [rows_cap][H/2], mxfp4_pitch(H) bytes a row
  uint8_t* sf;  // blocked (1, rows_cap, H)
  FastDiv blocks_div;  // H / 32 (set by the launcher)
};
cudaError_t launch_mxfp4_quant_scatter(Mxfp4ScatterArgs a, cudaStream_t st);

// Weight scales in the order the GEMM's tiles read them: per expert, column tile and
// K tile of 256 values 48 bytes for each of 32 lanes, one copy a K tile (the
// blocked order takes up to four, and twice the shared-memory reads).
constexpr int MXFP4_TILE_SF = 32 * 48;
int64_t mxfp4_tiled_scale_bytes(int64_t E, int64_t N, int64_t K, bool gate_up);
cudaError_t launch_mxfp4_tile_scales(const uint8_t* plain, int64_t ld, int32_t E, int32_t N, int64_t K, bool gate_up,
                                     uint8_t* tiled, cudaStream_t st);

// Grouped GEMM on MXFP4 operands over the permuted rows (see gemm_mxfp4.cu).
enum Mxfp4Epi : int {
  EPI4_SWIGLU = 0,    // gate_up: h = p * silu(gate) * up, requantised to MXFP4
  EPI4_F24_ROWS = 1,  // down: the top 24 bits of each fp32 sum, rows in permuted order
};
struct Gemm4Args {
  int32_t E, N, K;      // N: output columns (EPI4_SWIGLU: I); K: contraction length, a multiple of 32
  const int32_t* group_offsets;
  const int32_t* split_sizes;
  const uint8_t* sfa;   // blocked (1, rows_cap, K)
  const uint8_t* sfb;   // tiled (see mxfp4_tiled_scale_bytes)
  const float* prob;
  uint8_t* out;         // EPI4_F24_ROWS: f24 rows [rows_cap][N]
  uint8_t* q_out;       // EPI4_SWIGLU: h codes [rows_cap][N/2], mxfp4_pitch(N) bytes a row
  uint8_t* sf_out;      // EPI4_SWIGLU: blocked (1, rows_cap, N)
};
// a_codes: permuted rows, mxfp4_pitch(K) bytes apart; b_codes: rows b_pitch bytes
// apart.  max_rows: routed rows T*k -- no more 128-row tiles than experts or rows
// are occupied.
cudaError_t launch_grouped_gemm_mxfp4(int epi, const uint8_t* a_codes, int64_t rows_cap, const uint8_t* b_codes,
                                      int64_t b_pitch, Gemm4Args a, int64_t max_rows, cudaStream_t st);

}  // namespace moe
