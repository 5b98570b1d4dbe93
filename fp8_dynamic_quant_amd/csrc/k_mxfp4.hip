// Microscaled 4-bit blocks: quantisation, its inverse, and the product that reads them.
//
// A block is 32 consecutive elements that share one UE8M0 scale 2^e (byte e + 127); an
// element is E2M1 (sign, two exponent bits of bias 1, one fraction bit: 0, 0.5, 1, 1.5, 2,
// 3, 4, 6 and their negatives), two to a byte, the even element in the low nibble.  The
// scales have the layout of the 8-bit blocks: four bytes to an int32 word, one word for the
// 128 elements that a matrix instruction takes, [G, ceil(D / 128), align4(T)].
#include "wq_device.h"
#include "wq_mx4_kv.h"

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

// Both kernels: a wave takes 512 consecutive elements of one group in four consecutive tokens, a
// workgroup 16 tokens of them.  Lane l holds 8 elements (16 bytes of bf16, 4 of codes) of each token,
// four lanes a block, 16 lanes a scale word; the four tokens' words are 16 consecutive bytes (a word a
// token, written by itself, and one token a wave took 38.6 us instead of 31 for both kernels on 8192
// tokens of 4096).  Memory bounds both: quantising and back at that size moves 152 MB, 4.9 TB/s, the
// rate of a large copy; one token of 8 x 4096 takes 4.2 us for both, which is launch and one latency.
// x and codes are read, y is written once: streaming accesses.  Codes and scales stay cached for the
// product that reads them.
struct Share {
  int g, p, h;   // group; this 16-lane row's scale word, this quad's block
  int64_t t0;    // the first of the wave's four tokens
  bool word, block;
};
__device__ __forceinline__ Share share_of(int G, int D) {
  const int lane = threadIdx.x & 63, HG = D / 32, PH = (HG + 3) / 4;
  const uint32_t PW = (uint32_t)(PH + 3) / 4, across = (uint32_t)G * PW;
  const uint32_t block = blockIdx.x + (blockIdx.y << kGridXLog), rows = block / across, in = block % across;
  Share s;
  s.g = (int)(in / PW);
  s.t0 = (int64_t)rows * 16 + (threadIdx.x >> 6) * 4;
  s.p = 4 * (int)(in % PW) + (lane >> 4);
  s.h = 4 * s.p + ((lane >> 2) & 3);
  s.word = s.p < PH;
  s.block = s.h < HG;
  return s;
}
hipError_t share_grid(int64_t T, int G, int D, dim3* grid) {
  const int64_t blocks = (T + 15) / 16 * G * (((int64_t)D / 32 + 15) / 16);
  if (blocks >= ((int64_t)1 << 31)) return hipErrorInvalidValue;
  *grid = folded_grid(blocks);
  return hipSuccess;
}

__global__ __launch_bounds__(256) void k_group_quant_mxfp4(const uint16_t* __restrict__ x, int64_t T, int G, int D,
                                                           uint8_t* __restrict__ xq, int32_t* __restrict__ xs) {
  const Share s = share_of(G, D);
  if (s.t0 >= T) return;  // whole waves
  const int64_t TA = (T + 3) / 4 * 4, step = (int64_t)G * D;
  const int64_t off = (s.t0 * G + s.g) * D + (int64_t)s.h * 32 + (threadIdx.x & 3) * 8;
  v4u u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    u[i] = v4u{0, 0, 0, 0};
    if (s.block && s.t0 + i < T) u[i] = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(x + off + i * step));
  }
  v4u words;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t a = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) a = max(a, max(u[i][j] & 0x7FFFu, (u[i][j] >> 16) & 0x7FFFu));
    // max over the quad: swap neighbours, then pairs
    a = max(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0xB1, 0xF, 0xF, false));
    a = max(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0x4E, 0xF, 0xF, false));
    const bool there = s.block && s.t0 + i < T;
    uint32_t q = 0;
    int byte = 0;
    if (there && a < 0x7F80u) {
      const int e = e2m1_exp(a);
      byte = e + 127;
      const float f = ldexpf(1.0f, e);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(v2bf, (uint32_t)u[i][0]), f, 0);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(v2bf, (uint32_t)u[i][1]), f, 1);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(v2bf, (uint32_t)u[i][2]), f, 2);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(v2bf, (uint32_t)u[i][3]), f, 3);
    } else if (there) {
      byte = 255;  // a NaN or an infinity among the 32: the scale's NaN, codes zero
    }
    if (there) *reinterpret_cast<uint32_t*>(xq + (off + i * step) / 2) = q;
    // the row's four quad bytes (0 for blocks past the last and tokens past T) form the word
    const int base = threadIdx.x & 48;
    words[i] = (uint32_t)byte | (uint32_t)__shfl(byte, base + 4, 64) << 8 | (uint32_t)__shfl(byte, base + 8, 64) << 16 |
               (uint32_t)__shfl(byte, base + 12, 64) << 24;
  }
  if ((threadIdx.x & 15) == 0 && s.word)
    *reinterpret_cast<v4u*>(xs + ((int64_t)s.g * ((D / 32 + 3) / 4) + s.p) * TA + s.t0) = words;
}

hipError_t launch_group_quant_mxfp4(const uint16_t* x, int64_t T, int G, int D, uint8_t* xq, int32_t* xs,
                                    hipStream_t st) {
  if (T == 0 || G == 0 || D == 0) return hipSuccess;
  dim3 grid;
  const hipError_t e = share_grid(T, G, D, &grid);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_group_quant_mxfp4, grid, dim3(256), 0, st, x, T, G, D, xq, xs);
  return hipGetLastError();
}

// y = code * 2^(byte - 127), exact in bf16: two significant bits, and the least magnitude
// 0.5 * 2^-127 is a bf16 subnormal.  Byte 255 gives NaN.
__global__ __launch_bounds__(256) void k_group_dequant_mxfp4(const uint8_t* __restrict__ xq,
                                                             const int32_t* __restrict__ xs, int64_t T, int G, int D,
                                                             uint16_t* __restrict__ y) {
  const Share s = share_of(G, D);
  if (s.t0 >= T || !s.block) return;
  const int64_t TA = (T + 3) / 4 * 4, step = (int64_t)G * D;
  const int64_t off = (s.t0 * G + s.g) * D + (int64_t)s.h * 32 + (threadIdx.x & 3) * 8;
  const v4u words = *reinterpret_cast<const v4u*>(xs + ((int64_t)s.g * ((D / 32 + 3) / 4) + s.p) * TA + s.t0);
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    q[i] = s.t0 + i < T ? __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(xq + (off + i * step) / 2)) : 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t byte = (words[i] >> (8 * (s.h & 3))) & 0xFFu;
    const float f = ldexpf(1.0f, (int)byte - 127);
    v4u o;
    o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[i], f, 0));
    o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[i], f, 1));
    o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[i], f, 2));
    o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[i], f, 3));
    if (byte == 255) o = v4u{0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u};
    if (s.t0 + i < T) __builtin_nontemporal_store(o, reinterpret_cast<v4u*>(y + off + i * step));
  }
}

hipError_t launch_group_dequant_mxfp4(const uint8_t* xq, const int32_t* xs, int64_t T, int G, int D, uint16_t* y,
                                      hipStream_t st) {
  if (T == 0 || G == 0 || D == 0) return hipSuccess;
  dim3 grid;
  const hipError_t e = share_grid(T, G, D, &grid);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_group_dequant_mxfp4, grid, dim3(256), 0, st, xq, xs, T, G, D, y);
  return hipGetLastError();
}

}  // namespace wq
