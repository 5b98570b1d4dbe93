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

}  // namespace wq
