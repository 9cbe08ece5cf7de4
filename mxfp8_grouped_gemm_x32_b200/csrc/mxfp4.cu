// MXFP4 quantisation and dequantisation (HBM-bound).
//
// "Efficient MoE Training for Biological Foundation Models", Challenge 2: one
// scaling factor per 32 consecutive values; here with 4-bit E2M1 elements (sign,
// two exponent bits, one mantissa bit: 0, .5, 1, 1.5, 2, 3, 4, 6), two per
// byte, the even element in the low half, and the E8M0 scales and blocked
// scale layout of the MXFP8 tensors.
//
// One thread per 8 values (a unit) and four lanes per block (the block's |max|
// by two shuffles): a warp reads 512 (bf16) or 1024 (fp32) contiguous bytes and
// writes 128 contiguous code bytes, and rows of any width that is a multiple
// of 32 need no special case, since units run on from row to row.  Bound by
// HBM: a thread works on Q4_UNROLL units whose loads are all in flight.
#include "mxfp4.cuh"

namespace moe {

namespace {

constexpr int Q4_THREADS = 256;
constexpr int Q4_UNROLL = 4;
constexpr uint32_t Q4_CHUNK = Q4_THREADS * Q4_UNROLL;  // units of a block and pass

template <bool BF16>
__device__ __forceinline__ void load8(const void* src, int64_t unit, float* f) {
  if constexpr (BF16) {
    const uint4 v = __ldg(static_cast<const uint4*>(src) + unit);
    f[0] = bf16lo(v.x); f[1] = bf16hi(v.x); f[2] = bf16lo(v.y); f[3] = bf16hi(v.y);
    f[4] = bf16lo(v.z); f[5] = bf16hi(v.z); f[6] = bf16lo(v.w); f[7] = bf16hi(v.w);
  } else {
    const float4 a = __ldg(static_cast<const float4*>(src) + 2 * unit);
    const float4 b = __ldg(static_cast<const float4*>(src) + 2 * unit + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
}

// Eight values of a block -> codes and the block's scale byte (the same in its four lanes).
__device__ __forceinline__ uint32_t encode8(float* f, uint32_t& sb) {
  float m = abs_max_n<8>(f);
  m = abs_max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  m = abs_max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
  sb = e8m0_from_amax_bits_e2m1(__float_as_uint(m));
  const float inv = inv_scale_from_e8m0(sb);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] *= inv;
  return pack8_e2m1(f);
}

// WORDS: K is a multiple of 128, so that the four blocks of a scale word are 16
// neighbouring lanes, which store it at once; otherwise every block stores its
// byte.
template <bool BF16, bool WORDS>
__global__ void __launch_bounds__(Q4_THREADS) mxfp4_quant_kernel(const Mxfp4Args a) {
  const uint32_t U = a.units_div.d, KB = U / 4;                   // units and blocks per row
  const uint32_t rows = a.rows_div.d;
  const uint32_t n = uint32_t(a.groups) * rows * U;               // < 2^31 (checked by the launcher)
  const uint32_t RT = (rows + 127) / 128, KT = (KB + 3) / 4;
  const uint32_t stride = gridDim.x * Q4_THREADS;
  // n is a multiple of four (of 16 with WORDS): a block's lanes are in or out
  // together, and those that are out hold zeros through the shuffles
  for (uint32_t c = blockIdx.x * Q4_CHUNK; c < n; c += gridDim.x * Q4_CHUNK) {
    float f[Q4_UNROLL][8];
#pragma unroll
    for (int j = 0; j < Q4_UNROLL; ++j) {
      const uint32_t i = c + j * Q4_THREADS + threadIdx.x;
      if (i < n) {
        load8<BF16>(a.src, i, f[j]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[j][e] = 0.0f;
      }
    }
#pragma unroll
    for (int j = 0; j < Q4_UNROLL; ++j) {
      const uint32_t i = c + j * Q4_THREADS + threadIdx.x;
      uint32_t sb;
      const uint32_t w = encode8(f[j], sb);
      const uint32_t rr = fastdiv(i, a.units_div), u = i - rr * U;
      if constexpr (WORDS) {
        sb <<= 2 * (i & 12u);  // the block's byte of the word
        sb |= __shfl_xor_sync(0xFFFFFFFFu, sb, 4);
        sb |= __shfl_xor_sync(0xFFFFFFFFu, sb, 8);
      }
      if (i >= n) continue;
      *reinterpret_cast<uint32_t*>(a.q + int64_t(rr) * a.ldq + 4 * u) = w;
      if (u & (WORDS ? 15u : 3u)) continue;
      const uint32_t g = fastdiv(rr, a.rows_div), r = rr - g * rows, kb = u >> 2;
      uint8_t* p = a.sf + sf_offset(g, r, kb, RT, KT);
      if constexpr (WORDS) {
        *reinterpret_cast<uint32_t*>(p) = sb;
      } else {
        *p = uint8_t(sb);
        if (kb + 1 == KB)  // the padding blocks of the last scale word
          for (uint32_t x = KB; x < 4 * KT; ++x) a.sf[sf_offset(g, r, x, RT, KT)] = 0;
      }
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
__device__ __forceinline__ void decode8(uint32_t w, uint32_t sb, float* f) {
  // 2^(sb - 127): 2^-127 is a subnormal, 0xFF stands for NaN
  const float s = sb == 0xFFu ? __int_as_float(0x7FC00000) : (sb == 0u ? 5.877471754111438e-39f : __int_as_float(int(sb) << 23));
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

template <bool BF16>
__global__ void __launch_bounds__(Q4_THREADS) mxfp4_dequant_kernel(const Mxfp4Args a) {
  const uint32_t U = a.units_div.d, rows = a.rows_div.d;
  const uint32_t n = uint32_t(a.groups) * rows * U;
  const uint32_t RT = (rows + 127) / 128, KT = (U / 4 + 3) / 4;
  for (uint32_t c = blockIdx.x * Q4_CHUNK; c < n; c += gridDim.x * Q4_CHUNK) {
    uint32_t w[Q4_UNROLL], sb[Q4_UNROLL];
#pragma unroll
    for (int j = 0; j < Q4_UNROLL; ++j) {
      const uint32_t i = c + j * Q4_THREADS + threadIdx.x;
      w[j] = sb[j] = 0u;
      if (i < n) {
        const uint32_t rr = fastdiv(i, a.units_div), u = i - rr * U;
        const uint32_t g = fastdiv(rr, a.rows_div), r = rr - g * rows;
        w[j] = __ldg(reinterpret_cast<const uint32_t*>(a.q + int64_t(rr) * a.ldq + 4 * u));
        sb[j] = __ldg(a.sf + sf_offset(g, r, u >> 2, RT, KT));
      }
    }
#pragma unroll
    for (int j = 0; j < Q4_UNROLL; ++j) {
      const uint32_t i = c + j * Q4_THREADS + threadIdx.x;
      if (i >= n) continue;
      float f[8];
      decode8(w[j], sb[j], f);
      if constexpr (BF16) {
        static_cast<uint4*>(a.dst)[i] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                   pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
      } else {
        float4* d = static_cast<float4*>(a.dst) + 2 * int64_t(i);
        d[0] = make_float4(f[0], f[1], f[2], f[3]);
        d[1] = make_float4(f[4], f[5], f[6], f[7]);
      }
    }
  }
}

// UNROLL units a thread; small batches take one, to spread over the SMs.
template <int UNROLL>
__global__ void __launch_bounds__(Q4_THREADS) mxfp4_quant_scatter_kernel(const Mxfp4ScatterArgs a) {
  const uint32_t U = a.units_div.d, KB = U / 4, KT = (KB + 3) / 4;
  const uint32_t n = uint32_t(a.T) * U;  // < 2^31 (checked by the launcher)
  constexpr uint32_t CHUNK = Q4_THREADS * UNROLL;
  for (uint32_t c = blockIdx.x * CHUNK; c < n; c += gridDim.x * CHUNK) {
    float f[UNROLL][8];
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) {
      const uint32_t i = c + j * Q4_THREADS + threadIdx.x;
      if (i < n) {
        load8<true>(a.src, i, f[j]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[j][e] = 0.0f;
      }
    }
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) {
      const uint32_t i = c + j * Q4_THREADS + threadIdx.x;
      uint32_t sb;
      const uint32_t w = encode8(f[j], sb);
      if (i >= n) continue;
      const uint32_t t = fastdiv(i, a.units_div), u = i - t * U, kb = u >> 2;
      const bool lead = (u & 3) == 0, last = lead && kb + 1 == KB;
      const int32_t* rows = a.slot_to_row + int64_t(t) * a.k;
      for (int j0 = 0; j0 < a.k; j0 += 4) {
        int32_t rw[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) rw[x] = j0 + x < a.k ? __ldg(rows + j0 + x) : -1;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if (rw[x] < 0) continue;  // past k, or a slot whose expert id was rejected
          const int64_t r = rw[x];
          *reinterpret_cast<uint32_t*>(a.q + r * mxfp4_pitch(a.H) + u * 4) = w;
          if (lead) {
            a.sf[sf_offset(0, r, kb, 0, KT)] = uint8_t(sb);
            if (last)
              for (uint32_t p = KB; p < 4 * KT; ++p) a.sf[sf_offset(0, r, p, 0, KT)] = 0;
          }
        }
      }
    }
  }
}

unsigned q4_blocks(int64_t units, int64_t per_block) {
  const int64_t want = cdiv(units, per_block), cap = int64_t(device_sm_count()) * 8;
  return unsigned(want < 1 ? 1 : (want < cap ? want : cap));
}

}  // namespace

cudaError_t launch_mxfp4_quant(Mxfp4Args a, bool bf16, cudaStream_t st) {
  const int64_t units = int64_t(a.groups) * a.rows * (a.K / 8);
  if (units == 0) return cudaSuccess;
  a.units_div = make_fastdiv(uint32_t(a.K / 8));
  a.rows_div = make_fastdiv(uint32_t(a.rows));
  const unsigned blocks = q4_blocks(units, Q4_CHUNK);
  const bool words = a.K % 128 == 0;
  if (bf16)
    (words ? mxfp4_quant_kernel<true, true> : mxfp4_quant_kernel<true, false>)<<<blocks, Q4_THREADS, 0, st>>>(a);
  else
    (words ? mxfp4_quant_kernel<false, true> : mxfp4_quant_kernel<false, false>)<<<blocks, Q4_THREADS, 0, st>>>(a);
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_mxfp4_dequant(Mxfp4Args a, bool bf16, cudaStream_t st) {
  const int64_t units = int64_t(a.groups) * a.rows * (a.K / 8);
  if (units == 0) return cudaSuccess;
  a.units_div = make_fastdiv(uint32_t(a.K / 8));
  a.rows_div = make_fastdiv(uint32_t(a.rows));
  if (bf16)
    mxfp4_dequant_kernel<true><<<q4_blocks(units, Q4_CHUNK), Q4_THREADS, 0, st>>>(a);
  else
    mxfp4_dequant_kernel<false><<<q4_blocks(units, Q4_CHUNK), Q4_THREADS, 0, st>>>(a);
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_mxfp4_quant_scatter(Mxfp4ScatterArgs a, cudaStream_t st) {
  const int64_t units = int64_t(a.T) * (a.H / 8);
  if (units == 0) return cudaSuccess;
  if (units >= MXFP4_MAX_UNITS - (int64_t(1) << 24)) return cudaErrorInvalidValue;
  a.units_div = make_fastdiv(uint32_t(a.H / 8));
  if (units >= int64_t(device_sm_count()) * 4 * Q4_CHUNK)
    mxfp4_quant_scatter_kernel<Q4_UNROLL><<<q4_blocks(units, Q4_CHUNK), Q4_THREADS, 0, st>>>(a);
  else
    mxfp4_quant_scatter_kernel<1><<<q4_blocks(units, Q4_THREADS), Q4_THREADS, 0, st>>>(a);
  count_launch();
  return cudaGetLastError();
}

}  // namespace moe
