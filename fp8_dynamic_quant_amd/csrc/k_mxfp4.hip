// Microscaled 4-bit blocks: quantisation, its inverse, and the product that reads them.
//
// A block is 32 consecutive elements that share one UE8M0 scale 2^e (byte e + 127); an
// element is E2M1 (sign, two exponent bits of bias 1, one fraction bit: 0, 0.5, 1, 1.5, 2,
// 3, 4, 6 and their negatives), two to a byte, the even element in the low nibble.  The
// scales have the layout of the 8-bit blocks: four bytes to an int32 word, one word for the
// 128 elements that a matrix instruction takes, [G, ceil(D / 128), align4(T)].
#include "wq_device.h"
#include "wq_kernels.h"

namespace wq {

typedef unsigned v2u __attribute__((ext_vector_type(2)));
typedef unsigned v4u __attribute__((ext_vector_type(4)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

// e = max(-127, smallest e with 2^e >= a / 6) for the bf16 pattern of a finite a >= 0.  With
// a = 2^(E-127) (1 + F/128): 6 = 1.5 * 2^2, so e = E - 129, one more when 1 + F/128 > 1.5.  A
// subnormal a (E = 0) gives at most -128 and so the clamp, as a / 6 < 2^-128 asks.
__device__ __forceinline__ int e2m1_exp(uint32_t a) {
  const int e = (int)(a >> 7) - 129 + ((a & 0x7Fu) > 0x40u ? 1 : 0);
  return e < -127 ? -127 : e;
}

// One wave for 512 consecutive elements of a row: lane l takes 8 of them (16 bytes read, 4
// written), four lanes a block, 16 lanes a scale word.
__global__ __launch_bounds__(256) void k_group_quant_mxfp4(const uint16_t* __restrict__ x, int64_t T, int G, int D,
                                                           uint8_t* __restrict__ xq, int32_t* __restrict__ xs) {
  const int lane = threadIdx.x & 63;
  const int HG = D / 32, PH = (HG + 3) / 4, PW = (PH + 3) / 4;
  const int64_t TA = (T + 3) / 4 * 4;
  const int64_t wid = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (wid >= TA * G * PW) return;
  const int pw = (int)(wid % PW);
  const int64_t tg = wid / PW;
  const int g = (int)(tg % G);
  const int64_t t = tg / G;
  const int p = 4 * pw + (lane >> 4);         // this 16-lane row's scale word
  const int h = 4 * p + ((lane >> 2) & 3);    // this quad's block
  int byte = 0;
  if (t < T && p < PH && h < HG) {
    const int64_t off = (t * G + g) * (int64_t)D + (int64_t)h * 32 + (lane & 3) * 8;
    const v4u u = *reinterpret_cast<const v4u*>(x + off);
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) a = max(a, max(u[i] & 0x7FFFu, (u[i] >> 16) & 0x7FFFu));
    // max over the quad: swap neighbours, then pairs (exec covers whole quads here)
    a = max(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0xB1, 0xF, 0xF, false));
    a = max(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0x4E, 0xF, 0xF, false));
    uint32_t q = 0;
    if (a < 0x7F80u) {
      const int e = e2m1_exp(a);
      byte = e + 127;
      const float s = ldexpf(1.0f, e);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(v2bf, (uint32_t)u[0]), s, 0);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(v2bf, (uint32_t)u[1]), s, 1);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(v2bf, (uint32_t)u[2]), s, 2);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(v2bf, (uint32_t)u[3]), s, 3);
    } else {
      byte = 255;  // a NaN or an infinity among the 32: the scale's NaN, codes zero
    }
    *reinterpret_cast<uint32_t*>(xq + off / 2) = q;
  }
  // the row's four quad bytes (0 for blocks past HG) form the word; lane 16 r writes it
  const int base = lane & ~15;
  const int b1 = __shfl(byte, base + 4, 64), b2 = __shfl(byte, base + 8, 64), b3 = __shfl(byte, base + 12, 64);
  if ((lane & 15) == 0 && p < PH) {
    const uint32_t word = (uint32_t)byte | ((uint32_t)b1 << 8) | ((uint32_t)b2 << 16) | ((uint32_t)b3 << 24);
    xs[((int64_t)g * PH + p) * TA + t] = (int32_t)word;
  }
}

hipError_t launch_group_quant_mxfp4(const uint16_t* x, int64_t T, int G, int D, uint8_t* xq, int32_t* xs,
                                    hipStream_t st) {
  const int HG = D / 32, PH = (HG + 3) / 4, PW = (PH + 3) / 4;
  const int64_t TA = (T + 3) / 4 * 4;
  const int64_t waves = TA * G * PW;
  if (waves == 0) return hipSuccess;
  hipLaunchKernelGGL(k_group_quant_mxfp4, dim3((unsigned)((waves + 3) / 4)), dim3(256), 0, st, x, T, G, D, xq, xs);
  return hipGetLastError();
}

// y = code * 2^(byte - 127), exact in bf16: two significant bits, and the least magnitude
// 0.5 * 2^-127 is a bf16 subnormal.  Byte 255 gives NaN.  Eight elements a lane.
__global__ __launch_bounds__(256) void k_group_dequant_mxfp4(const uint8_t* __restrict__ xq,
                                                             const int32_t* __restrict__ xs, int64_t T, int G, int D,
                                                             uint16_t* __restrict__ y) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;  // 8 elements
  const int per = D / 8;
  const int64_t tg = i / per;
  const int d8 = (int)(i % per);
  const int g = (int)(tg % G);
  const int64_t t = tg / G;
  if (t >= T) return;
  const int PH = (D / 32 + 3) / 4;
  const int64_t TA = (T + 3) / 4 * 4;
  const int h = d8 / 4;
  const uint32_t byte = ((uint32_t)xs[((int64_t)g * PH + h / 4) * TA + t] >> (8 * (h & 3))) & 0xFFu;
  const uint32_t q = *reinterpret_cast<const uint32_t*>(xq + i * 4);
  v4u o;
  if (byte == 255) {
    o = v4u{0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u};
  } else {
    const float s = ldexpf(1.0f, (int)byte - 127);
    o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 0));
    o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 1));
    o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 2));
    o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 3));
  }
  *reinterpret_cast<v4u*>(y + i * 8) = o;
}

hipError_t launch_group_dequant_mxfp4(const uint8_t* xq, const int32_t* xs, int64_t T, int G, int D, uint16_t* y,
                                      hipStream_t st) {
  const int64_t n = T * G * (D / 8);
  if (n == 0) return hipSuccess;
  hipLaunchKernelGGL(k_group_dequant_mxfp4, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, xq, xs, T, G, D, y);
  return hipGetLastError();
}

// ---- product -----------------------------------------------------------------------------
// y[m, g, n] = sum over 32-deep blocks of 2^(ea + eb) sum a b, by
// v_mfma_scale_f32_16x16x128_f8f6f4: its 128-deep step is one scale word of each operand.
// Operand layout (measured with one-hot inputs): lane group q (lanes 16q .. 16q+15) holds, of
// a 4-bit operand, K 32q .. 32q+31 in its first four registers; of an 8-bit operand K 16q ..
// 16q+15 in the first four and 64+16q .. 64+16q+15 in the last four; the scale operand of lane
// group s applies to K 32s .. 32s+31 of either.

template <bool A8>
__device__ __forceinline__ v8i load_a_frag(const uint8_t* row, int kb, int q) {
  if constexpr (A8) {
    const v4i lo = *reinterpret_cast<const v4i*>(row + kb * 128 + q * 16);
    const v4i hi = *reinterpret_cast<const v4i*>(row + kb * 128 + 64 + q * 16);
    return v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  } else {
    const v4i lo = *reinterpret_cast<const v4i*>(row + kb * 64 + q * 16);
    return v8i{lo[0], lo[1], lo[2], lo[3], 0, 0, 0, 0};
  }
}

__device__ __forceinline__ v8i load_w_frag(const uint8_t* row, int kb, int q) {
  const v4i lo = *reinterpret_cast<const v4i*>(row + kb * 64 + q * 16);
  return v8i{lo[0], lo[1], lo[2], lo[3], 0, 0, 0, 0};
}

// A wave makes 16 rows x 16 columns over all of K, operands straight from memory.
template <bool A8>
__global__ __launch_bounds__(256) void k_mx4_plain(Mx4Args p) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int nx = (p.N / 16 + 3) / 4;  // workgroups across the columns
  const int g = blockIdx.y, m0 = (int)(blockIdx.x / nx) * 16, n0 = ((int)(blockIdx.x % nx) * 4 + wv) * 16;
  if (n0 >= p.N) return;
  const int cl = lane & 15, q = lane >> 4, KT = p.K >> 7;
  const int row = min(m0 + cl, p.M - 1);
  const uint8_t* A = p.a + g * p.a_batch_stride + row * p.lda;
  const uint8_t* W = p.w + g * p.w_batch_stride + (int64_t)(n0 + cl) * (p.K / 2);
  const int32_t* SA = p.a_scale + (int64_t)g * KT * p.a_tokens + row;
  const int32_t* SW = p.w_scale + (int64_t)g * KT * p.N + n0 + cl;
  v4f acc{0.0f, 0.0f, 0.0f, 0.0f};
  for (int kb = 0; kb < KT; ++kb) {
    const v8i a = load_a_frag<A8>(A, kb, q), w = load_w_frag(W, kb, q);
    const int sa = (SA[kb * p.a_tokens] >> (8 * q)) & 0xFF, sw = (SW[(int64_t)kb * p.N] >> (8 * q)) & 0xFF;
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, w, acc, A8 ? 0 : 4, 4, 0, sa, 0, sw);
  }
  // the matrix results are pinned before the per-lane stores: the compiler may otherwise move
  // a matrix instruction into the branch, where part of its lanes are off
  asm volatile("" : "+v"(acc));
  uint16_t* Y = p.y + g * p.y_batch_stride;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = m0 + 4 * q + i;  // output layout: column lane % 16, row 4 (lane / 16) + i
    if (m < p.M) Y[m * p.ldy + n0 + cl] = (uint16_t)f32_to_bf16_nan(acc[i]);
  }
}

hipError_t launch_mx4(const Mx4Args& a, bool a8, hipStream_t st) {
  const int64_t wgs = (int64_t)((a.N / 16 + 3) / 4) * ((a.M + 15) / 16);
  if (wgs >= ((int64_t)1 << 31)) return hipErrorInvalidValue;
  const dim3 grid((unsigned)wgs, (unsigned)a.batch);
  if (a8)
    hipLaunchKernelGGL(k_mx4_plain<true>, grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL(k_mx4_plain<false>, grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace wq
