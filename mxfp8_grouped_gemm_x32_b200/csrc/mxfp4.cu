// MXFP4 quantisation and dequantisation (HBM-bound).
//
// "Efficient MoE Training for Biological Foundation Models", Challenge 2: one
// scaling factor per 32 consecutive values; here with 4-bit E2M1 elements (sign,
// two exponent bits, one mantissa bit: 0, .5, 1, 1.5, 2, 3, 4, 6), two per
// byte, the even element in the low half, and the E8M0 scales and blocked
// scale layout of the MXFP8 tensors.
//
// One thread per block of 32 values: it reads the block with 256-bit loads, finds
// the |max| on its own and writes 16 code bytes (a warp 512 contiguous ones) and
// the scale, four neighbouring threads one word of scales where the rows' blocks
// come in fours.  Rows of any width that is a multiple of 32 need no special
// case, since blocks run on from row to row.  Bound by HBM: 229376 x 4096 bf16
// values (2.4 GB read and written) take 361 us to quantise, the rate of a plain copy
// (6.6 TB/s; four threads per block with shuffles for the |max| 467), and 353 us to
// dequantise.
#include "mxfp4.cuh"

namespace moe {

namespace {

constexpr int Q4_THREADS = 256;

// Block `i` of 32 contiguous values as fp32.  wide: the source starts on a 32-byte boundary.
template <bool BF16>
__device__ __forceinline__ void load32(const void* src, int64_t i, bool wide, float* f) {
  constexpr int W = BF16 ? 16 : 32;  // words
  uint32_t w[W];
  const uint32_t* p = static_cast<const uint32_t*>(src) + i * W;
  if (wide) {
#pragma unroll
    for (int j = 0; j < W / 8; ++j) ldg256(p + 8 * j, w + 8 * j);
  } else {
#pragma unroll
    for (int j = 0; j < W / 4; ++j) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + j);
      w[4 * j] = v.x; w[4 * j + 1] = v.y; w[4 * j + 2] = v.z; w[4 * j + 3] = v.w;
    }
  }
  if constexpr (BF16) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      f[2 * j] = bf16lo(w[j]);
      f[2 * j + 1] = bf16hi(w[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(w[j]);
  }
}

// A block's values -> its codes and scale byte.
__device__ __forceinline__ uint4 encode32(float* f, uint32_t& sb) {
  sb = e8m0_from_amax_bits_e2m1(__float_as_uint(abs_max_n<32>(f)));
  const float inv = inv_scale_from_e8m0(sb);
#pragma unroll
  for (int i = 0; i < 32; ++i) f[i] *= inv;
  return make_uint4(pack8_e2m1(f), pack8_e2m1(f + 8), pack8_e2m1(f + 16), pack8_e2m1(f + 24));
}

// Scale bytes of four neighbouring threads as one word, the same in all four.
__device__ __forceinline__ uint32_t scale_word(uint32_t sb) {
  sb <<= 8 * (threadIdx.x & 3);
  sb |= __shfl_xor_sync(0xFFFFFFFFu, sb, 1);
  return sb | __shfl_xor_sync(0xFFFFFFFFu, sb, 2);
}

// WORDS: K is a multiple of 128, so that the four blocks of a scale word are four
// neighbouring threads, one of which stores it; otherwise every thread stores
// its byte.
template <bool BF16, bool WORDS>
__global__ void __launch_bounds__(Q4_THREADS) mxfp4_quant_kernel(const Mxfp4Args a) {
  const uint32_t KB = a.blocks_div.d;                // blocks per row
  const uint32_t rows = a.rows_div.d;
  const uint32_t n = uint32_t(a.groups) * rows * KB;  // < 2^29 (checked by the launcher)
  const uint32_t RT = (rows + 127) / 128, KT = (KB + 3) / 4;
  const uint32_t stride = gridDim.x * Q4_THREADS;
  const bool wide = (reinterpret_cast<uintptr_t>(a.src) & 31u) == 0;
  // whole warps iterate together (the shuffles need all 32 lanes); with WORDS n is
  // a multiple of four, so a word's threads are in or out together
  for (uint32_t i0 = blockIdx.x * Q4_THREADS + (threadIdx.x & ~31u); i0 < n; i0 += stride) {
    const uint32_t i = i0 + (threadIdx.x & 31);
    const bool in = i < n;
    float f[32];
    load32<BF16>(a.src, in ? i : n - 1, wide, f);
    uint32_t sb;
    const uint4 w = encode32(f, sb);
    if constexpr (WORDS) sb = scale_word(sb);
    if (!in) continue;
    const uint32_t rr = fastdiv(i, a.blocks_div), kb = i - rr * KB;
    *reinterpret_cast<uint4*>(a.q + int64_t(rr) * a.ldq + 16 * kb) = w;
    if (WORDS && (kb & 3)) continue;
    const uint32_t g = fastdiv(rr, a.rows_div), r = rr - g * rows;
    uint8_t* p = a.sf + sf_offset(g, r, kb, RT, KT);
    if constexpr (WORDS) {
      *reinterpret_cast<uint32_t*>(p) = sb;
    } else {
      *p = uint8_t(sb);
      if (kb + 1 == KB)  // the padding blocks of the last scale word
        for (uint32_t x = KB; x < 4 * KT; ++x) a.sf[sf_offset(g, r, x, RT, KT)] = 0;
    }
  }
  // rows past the last one in its 128-row tile: zero scale words
  const uint32_t pad = RT * 128 - rows;
  const int64_t words = int64_t(a.groups) * pad * KT;
  for (int64_t i = blockIdx.x * int64_t(Q4_THREADS) + threadIdx.x; i < words; i += stride) {
    const int64_t kt = i % KT, gr = i / KT;
    *reinterpret_cast<uint32_t*>(a.sf + sf_offset(gr / pad, rows + gr % pad, 4 * kt, RT, KT)) = 0u;
  }
}

// Eight codes (one word) -> fp32 values times the block's scale.
__device__ __forceinline__ void decode8(uint32_t w, float s, float* f) {
  uint32_t h[4];
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
    f[2 * j] = v.x * s;
    f[2 * j + 1] = v.y * s;
  }
}

// Two threads per block: 16 codes in, 32 or 64 contiguous bytes out; a CTA works on
// DQ_HALVES runs of halves and is done, since CTAs that come and go write faster than ones that
// stay (229376 x 4096 to bf16 353 against 431 us, to fp32 630 against 755).
constexpr int DQ_HALVES = 2;  // halves of blocks in flight per thread
template <bool BF16>
__global__ void __launch_bounds__(Q4_THREADS) mxfp4_dequant_kernel(const Mxfp4Args a) {
  const uint32_t KB = a.blocks_div.d, rows = a.rows_div.d;
  const uint32_t n = uint32_t(a.groups) * rows * KB * 2;
  const uint32_t RT = (rows + 127) / 128, KT = (KB + 3) / 4;
  const bool wide = (reinterpret_cast<uintptr_t>(a.dst) & 31u) == 0;
  const uint32_t c = blockIdx.x * (Q4_THREADS * DQ_HALVES);
  uint2 w[DQ_HALVES];
  uint32_t sb[DQ_HALVES];
#pragma unroll
  for (int j = 0; j < DQ_HALVES; ++j) {
    const uint32_t i = c + j * Q4_THREADS + threadIdx.x;
    w[j] = make_uint2(0u, 0u);
    sb[j] = 0u;
    if (i < n) {
      const uint32_t rr = fastdiv(i >> 1, a.blocks_div), kb = (i >> 1) - rr * KB;
      const uint32_t g = fastdiv(rr, a.rows_div), r = rr - g * rows;
      w[j] = __ldg(reinterpret_cast<const uint2*>(a.q + int64_t(rr) * a.ldq + 16 * kb + 8 * (i & 1)));
      sb[j] = __ldg(a.sf + sf_offset(g, r, kb, RT, KT));
    }
  }
#pragma unroll
  for (int j = 0; j < DQ_HALVES; ++j) {
    const uint32_t i = c + j * Q4_THREADS + threadIdx.x;
    if (i >= n) continue;
    // 2^(sb - 127): 2^-127 is a subnormal, 0xFF stands for NaN
    const float s = sb[j] == 0xFFu ? __int_as_float(0x7FC00000)
                                   : (sb[j] == 0u ? 5.877471754111438e-39f : __int_as_float(int(sb[j]) << 23));
    float f[16];
    decode8(w[j].x, s, f);
    decode8(w[j].y, s, f + 8);
    constexpr int W = BF16 ? 8 : 16;
    uint32_t o[W];
#pragma unroll
    for (int e = 0; e < W; ++e) o[e] = BF16 ? pack_bf16x2(f[2 * (e % 8)], f[2 * (e % 8) + 1]) : __float_as_uint(f[e]);
    uint32_t* d = static_cast<uint32_t*>(a.dst) + int64_t(i) * W;
    if (wide) {
#pragma unroll
      for (int e = 0; e < W / 8; ++e) stg256(d + 8 * e, o + 8 * e);
    } else {
#pragma unroll
      for (int e = 0; e < W / 4; ++e)
        reinterpret_cast<uint4*>(d)[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
    }
  }
}

template <bool WORDS>
__global__ void __launch_bounds__(Q4_THREADS) mxfp4_quant_scatter_kernel(const Mxfp4ScatterArgs a) {
  const uint8_t* src = a.src;
  const int32_t* slot_to_row = a.slot_to_row;
  release_dependents();
  dependency_wait(src, slot_to_row);
  const uint32_t KB = a.blocks_div.d, KT = (KB + 3) / 4;
  const uint32_t n = uint32_t(a.T) * KB;  // < 2^29 (checked by the launcher)
  const int64_t pitch = mxfp4_pitch(a.H);
  const uint32_t stride = gridDim.x * Q4_THREADS;
  const bool wide = (reinterpret_cast<uintptr_t>(src) & 31u) == 0;
  for (uint32_t i0 = blockIdx.x * Q4_THREADS + (threadIdx.x & ~31u); i0 < n; i0 += stride) {
    const uint32_t i = i0 + (threadIdx.x & 31);
    const bool in = i < n;
    const uint32_t b = in ? i : n - 1;
    const uint32_t t = fastdiv(b, a.blocks_div), kb = b - t * KB;
    const int32_t* rows = slot_to_row + int64_t(t) * a.k;
    float f[32];
    load32<true>(src, b, wide, f);
    const int32_t first = __ldg(rows);
    uint32_t sb;
    const uint4 w = encode32(f, sb);
    if constexpr (WORDS) sb = scale_word(sb);
    if (!in) continue;
    for (int j0 = 0; j0 < a.k; j0 += 4) {
      int32_t rw[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) rw[x] = j0 + x == 0 ? first : (j0 + x < a.k ? __ldg(rows + j0 + x) : -1);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if (rw[x] < 0) continue;  // past k, or a slot whose expert id was rejected
        const int64_t r = rw[x];
        *reinterpret_cast<uint4*>(a.q + r * pitch + 16 * kb) = w;
        uint8_t* p = a.sf + sf_offset(0, r, kb, 0, KT);
        if constexpr (WORDS) {
          if ((kb & 3) == 0) *reinterpret_cast<uint32_t*>(p) = sb;
        } else {
          *p = uint8_t(sb);
          if (kb + 1 == KB)  // the padding blocks of the last scale word
            for (uint32_t y = KB; y < 4 * KT; ++y) a.sf[sf_offset(0, r, y, 0, KT)] = 0;
        }
      }
    }
  }
}

unsigned q4_blocks(int64_t threads, int per_sm) {
  const int64_t want = cdiv(threads, Q4_THREADS), cap = int64_t(device_sm_count()) * per_sm;
  return unsigned(want < 1 ? 1 : (want < cap ? want : cap));
}

}  // namespace

cudaError_t launch_mxfp4_quant(Mxfp4Args a, bool bf16, cudaStream_t st) {
  const int64_t blocks = int64_t(a.groups) * a.rows * (a.K / 32);
  if (blocks == 0) return cudaSuccess;
  a.blocks_div = make_fastdiv(uint32_t(a.K / 32));
  a.rows_div = make_fastdiv(uint32_t(a.rows));
  const unsigned grid = q4_blocks(blocks, 16);
  const bool words = a.K % 128 == 0;
  if (bf16)
    (words ? mxfp4_quant_kernel<true, true> : mxfp4_quant_kernel<true, false>)<<<grid, Q4_THREADS, 0, st>>>(a);
  else
    (words ? mxfp4_quant_kernel<false, true> : mxfp4_quant_kernel<false, false>)<<<grid, Q4_THREADS, 0, st>>>(a);
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_mxfp4_dequant(Mxfp4Args a, bool bf16, cudaStream_t st) {
  const int64_t blocks = int64_t(a.groups) * a.rows * (a.K / 32);
  if (blocks == 0) return cudaSuccess;
  a.blocks_div = make_fastdiv(uint32_t(a.K / 32));
  a.rows_div = make_fastdiv(uint32_t(a.rows));
  const unsigned grid = unsigned(cdiv(2 * blocks, Q4_THREADS * DQ_HALVES));
  if (bf16)
    mxfp4_dequant_kernel<true><<<grid, Q4_THREADS, 0, st>>>(a);
  else
    mxfp4_dequant_kernel<false><<<grid, Q4_THREADS, 0, st>>>(a);
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_mxfp4_quant_scatter(Mxfp4ScatterArgs a, cudaStream_t st) {
  const int64_t blocks = int64_t(a.T) * (a.H / 32);
  if (blocks == 0) return cudaSuccess;
  if (blocks >= MXFP4_MAX_BLOCKS) return cudaErrorInvalidValue;
  a.blocks_div = make_fastdiv(uint32_t(a.H / 32));
  return launch_dependent(a.H % 128 == 0 ? mxfp4_quant_scatter_kernel<true> : mxfp4_quant_scatter_kernel<false>,
                          q4_blocks(blocks, 16), Q4_THREADS, 0, st, a);
}

}  // namespace moe
