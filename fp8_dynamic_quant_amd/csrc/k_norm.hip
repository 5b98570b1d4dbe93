// The residual's addition, the root-mean-square norm of the sum, and its rows in 8 bits.
//
//   h = RN_bf16(x + residual),  v = (h * inv) * gamma,  inv = 1 / sqrt(f32(sum h^2 / K) + eps)
//
// and v's rows as int8 with a scale for each, or as E4M3 with a UE8M0 scale for 128 or 32 elements
// in the packed words that the products read.  The sum of squares is taken in 64 bits (the squares
// of bf16 numbers are exact there) and rounded once to 32; every other step is one rounding in 32.
// One pass over memory: a row's sums h stay in registers, packed in bf16, from the first load to
// the codes.  Bound by memory with many rows, by latency with few: 8192 rows of 4096 in E4M3 with a
// scale for 32 45.7 us (5.2 TB/s read and written, what a copy reaches), 1000 rows of 2064 in int8 with
// the norm itself 8.0 (2.3 TB/s), 64 rows and one row of 4096 3.6, of which 3 are the launch, the loads'
// latency and two reductions.
#include "wq_dma.h"
#include "wq_layer.h"

namespace wq {

namespace {

typedef unsigned v2u __attribute__((ext_vector_type(2)));
typedef unsigned v4u __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) { return f32_to_bf16_nan(a) | f32_to_bf16_nan(b) << 16; }

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
template <int CTRL>
__device__ __forceinline__ double dpp_add(double v) {
  const uint64_t u = __double_as_longlong(v);
  return v + __longlong_as_double((int64_t)((uint64_t)dpp<CTRL>((uint32_t)(u >> 32)) << 32 | dpp<CTRL>((uint32_t)u)));
}
// the sum over a wave, in every lane: pairs, quads, half rows and rows of 16 lanes, then the rows
__device__ __forceinline__ double wave_total(double v) {
  v = dpp_add<0xB1>(v);
  v = dpp_add<0x4E>(v);
  v = dpp_add<0x141>(v);
  v = dpp_add<0x140>(v);
  const uint64_t u = __double_as_longlong(v);
  double r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = __longlong_as_double((int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), 16 * i) << 32 |
                                          (uint32_t)__builtin_amdgcn_readlane((int)u, 16 * i)));
  return (r[0] + r[1]) + (r[2] + r[3]);
}
// the largest of a row of 16 lanes, of a quad
__device__ __forceinline__ uint32_t quad_most(uint32_t v) {
  v = max(v, dpp<0xB1>(v));
  return max(v, dpp<0x4E>(v));
}
__device__ __forceinline__ uint32_t row16_most(uint32_t v) {
  v = quad_most(v);
  v = max(v, dpp<0x141>(v));
  return max(v, dpp<0x140>(v));
}
__device__ __forceinline__ uint32_t wave_most(uint32_t v) {
  v = row16_most(v);
  return max(max((uint32_t)__builtin_amdgcn_readlane((int)v, 0), (uint32_t)__builtin_amdgcn_readlane((int)v, 16)),
             max((uint32_t)__builtin_amdgcn_readlane((int)v, 32), (uint32_t)__builtin_amdgcn_readlane((int)v, 48)));
}

// 1 / sqrt(f32(ss / K) + eps).  ss / K is one correctly rounded division in 64 bits, as a product
// with RN(1 / K) and one step by the exact remainder (Markstein's theorem: the reciprocal is
// correctly rounded, and K's significand is not all ones).  NaN for a row that holds a NaN or an
// infinity: only then is the sum not finite (65536 squares below 2^256).
__device__ __forceinline__ float rms_inverse(double ss, double k, double inv_k, float eps) {
  const double q = ss * inv_k;
  const float ms = (float)__builtin_fma(__builtin_fma(-q, k, ss), inv_k, q);
  const float inv = __fdiv_rn(1.0f, sqrtf(__fadd_rn(ms, eps)));
  return __builtin_isfinite(ss) ? inv : __uint_as_float(0x7FC00000u);
}

// the smallest e >= -127 with 448 * 2^e >= a, for a finite pattern: 448 = 1.75 * 2^8
__device__ __forceinline__ int e4m3_exp(uint32_t a) {
  return max((int)(a >> 23) - 135 + ((a & 0x7FFFFFu) > 0x600000u ? 1 : 0), -127);
}

// W waves a row, CH pieces of eight elements a lane: piece i of thread t is i * 64 W + t, so that a
// wave's piece is 512 consecutive elements.
template <int KIND, int W, int CH>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void k_add_rms_quant(NormArgs a) {
  constexpr int kRowThreads = 64 * W, kRows = W == 1 ? 4 : 1;
  __shared__ double sums[W];
  __shared__ uint32_t most[W];
  const int t = W == 1 ? threadIdx.x & 63 : threadIdx.x, lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int64_t block = blockIdx.x + ((int64_t)blockIdx.y << kGridXLog);
  const int64_t row = block * kRows + (W == 1 ? __builtin_amdgcn_readfirstlane(wv) : 0);
  if (row >= a.M) return;
  const int C = a.K / 8;
  const uint16_t* x = a.x + row * a.ldx;
  const uint16_t* r = a.residual + row * a.ldr;
  // ---- the sum, and its squares
  constexpr bool kGammaHeld = CH <= 4;  // beyond that the registers do not hold it as well
  v4u h[CH], u[CH], gm[kGammaHeld ? CH : 1];
#pragma unroll
  for (int i = 0; i < CH; ++i) h[i] = *reinterpret_cast<const v4u*>(x + 8 * min(i * kRowThreads + t, C - 1));
  if (a.residual) {
#pragma unroll
    for (int i = 0; i < CH; ++i) u[i] = *reinterpret_cast<const v4u*>(r + 8 * min(i * kRowThreads + t, C - 1));
  }
  auto gamma = [&](int i) __attribute__((always_inline)) {
    return *reinterpret_cast<const v4u*>(a.gamma + 8 * min(i * kRowThreads + t, C - 1));
  };
  if constexpr (kGammaHeld) {
#pragma unroll
    for (int i = 0; i < CH; ++i) gm[i] = gamma(i);
  }
  double ss = 0.0;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = i * kRowThreads + t;
    if (a.residual) {
#pragma unroll
      for (int j = 0; j < 4; ++j) h[i][j] = pack_bf16(low(h[i][j]) + low(u[i][j]), high(h[i][j]) + high(u[i][j]));
    }
    if (c >= C) h[i] = v4u{0, 0, 0, 0};
    if (a.sum && c < C) *reinterpret_cast<v4u*>(a.sum + row * a.lds + 8 * c) = h[i];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      ss = __builtin_fma((double)low(h[i][j]), (double)low(h[i][j]), ss);
      ss = __builtin_fma((double)high(h[i][j]), (double)high(h[i][j]), ss);
    }
  }
  ss = wave_total(ss);
  if constexpr (W > 1) {
    if (lane == 0) sums[wv] = ss;
    __syncthreads();
    ss = sums[0];
#pragma unroll
    for (int w = 1; w < W; ++w) ss += sums[w];
  }
  const float inv = rms_inverse(ss, (double)a.K, a.inv_k, a.eps);
  auto normed = [&](int i, float (&v)[8]) __attribute__((always_inline)) {
    const v4u gi = kGammaHeld ? gm[kGammaHeld ? i : 0] : gamma(i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __fmul_rn(__fmul_rn(low(h[i][j]), inv), low(gi[j]));
      v[2 * j + 1] = __fmul_rn(__fmul_rn(high(h[i][j]), inv), high(gi[j]));
    }
  };
  auto magnitude = [&](const float (&v)[8]) __attribute__((always_inline)) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[e]) & 0x7FFFFFFFu);
    return m;
  };
  auto store_y = [&](int c, const float (&v)[8]) __attribute__((always_inline)) {
    if (a.y && c < C)
      *reinterpret_cast<v4u*>(a.y + row * a.ldy + 8 * c) =
          v4u{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
  };
  uint8_t* codes = a.xq + row * a.K;
  // ---- codes
  if constexpr (KIND == kNormInt8) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = i * kRowThreads + t;
      float v[8];
      normed(i, v);
      store_y(c, v);
      // (lanes past the row hold zeros, or NaN where a norm of zeros or gamma's last pieces are not finite)
      if (c < C) m = max(m, magnitude(v));
    }
    m = wave_most(m);
    if constexpr (W > 1) {
      if (lane == 0) most[wv] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < W; ++w) m = max(m, most[w]);
    }
    const bool bad = m >= 0x7F800000u;
    const float s = bad ? __uint_as_float(0x7FC00000u) : __fdiv_rn(__uint_as_float(m), 127.0f);
    const float rs = recip_refined(s);
    if (t == 0) static_cast<float*>(a.xs)[row] = s;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = i * kRowThreads + t;
      float v[8];
      normed(i, v);
      if (c < C) *reinterpret_cast<uint2*>(codes + 8 * c) = bad ? uint2{0u, 0u} : quant8(v, s, rs);
    }
  } else {
    const int PH = KIND == kNormE4m3 ? (a.K + 511) / 512 : (a.K + 127) / 128;
    const int64_t TA = (a.M + 3) / 4 * 4;
    int32_t* words = static_cast<int32_t*>(a.xs);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = i * kRowThreads + t;
      float v[8];
      normed(i, v);
      store_y(c, v);
      // a block is 16 or 4 whole lanes, all in the row or none
      const uint32_t m = KIND == kNormE4m3 ? row16_most(magnitude(v)) : quad_most(magnitude(v));
      const bool bad = m >= 0x7F800000u;
      const int e = e4m3_exp(m);
      const float f = __uint_as_float((uint32_t)(127 - e) << 23);  // 2^-e, e in [-127, 120]
      uint32_t lo = 0, hi = 0;
      lo = __builtin_amdgcn_cvt_pk_fp8_f32(__fmul_rn(v[0], f), __fmul_rn(v[1], f), lo, false);
      lo = __builtin_amdgcn_cvt_pk_fp8_f32(__fmul_rn(v[2], f), __fmul_rn(v[3], f), lo, true);
      hi = __builtin_amdgcn_cvt_pk_fp8_f32(__fmul_rn(v[4], f), __fmul_rn(v[5], f), hi, false);
      hi = __builtin_amdgcn_cvt_pk_fp8_f32(__fmul_rn(v[6], f), __fmul_rn(v[7], f), hi, true);
      if (c < C) *reinterpret_cast<v2u*>(codes + 8 * c) = bad ? v2u{0u, 0u} : v2u{lo, hi};
      const uint32_t byte = c >= C ? 0u : bad ? 255u : (uint32_t)(e + 127);
      uint32_t word;
      int p;
      bool mine;
      if constexpr (KIND == kNormE4m3) {
        word = (uint32_t)__builtin_amdgcn_readlane((int)byte, 0) | (uint32_t)__builtin_amdgcn_readlane((int)byte, 16) << 8 |
               (uint32_t)__builtin_amdgcn_readlane((int)byte, 32) << 16 | (uint32_t)__builtin_amdgcn_readlane((int)byte, 48) << 24;
        p = c >> 6;
        mine = lane == 0;
      } else {
        // the four quads' bytes to the row's first lane
        const int base = lane & ~15;
        word = byte | (uint32_t)__shfl((int)byte, base + 4, 64) << 8 | (uint32_t)__shfl((int)byte, base + 8, 64) << 16 |
               (uint32_t)__shfl((int)byte, base + 12, 64) << 24;
        p = c >> 4;
        mine = (lane & 15) == 0;
      }
      if (mine && p < PH) {
        words[p * TA + row] = (int32_t)word;
        if (row == a.M - 1)
          for (int64_t pad = a.M; pad < TA; ++pad) words[p * TA + pad] = 0;
      }
    }
  }
}

template <int KIND, int W, int CH>
hipError_t launch(const NormArgs& a, hipStream_t st) {
  constexpr int kRows = W == 1 ? 4 : 1;
  hipLaunchKernelGGL((k_add_rms_quant<KIND, W, CH>), folded_grid((a.M + kRows - 1) / kRows), dim3(W == 1 ? 256 : 64 * W), 0, st, a);
  return hipGetLastError();
}

// A row's threads: enough that a lane has four pieces at most while a workgroup can be that large; of
// rows that do not fill the chip a piece each, where latency is all (K = 4096 and 7168, E4M3, by one
// piece and as many rows take it: 64 rows 3.9 and 4.4, 4.4 and 4.9 us; 512 rows of 4096 5.4 and 5.7;
// 1000 rows of 2064 8.2 and 8.0; 8192 rows of 4096 46.8 and 46.2).
template <int KIND>
hipError_t launch_kind(const NormArgs& a, int num_cu, hipStream_t st) {
  const int C = a.K / 8;
  if (a.M <= 2 * num_cu && C > 256 && C <= 1024) return C <= 512 ? launch<KIND, 8, 1>(a, st) : launch<KIND, 16, 1>(a, st);
  if (C <= 64) return launch<KIND, 1, 1>(a, st);
  if (C <= 256) return launch<KIND, 4, 1>(a, st);
  if (C <= 512) return launch<KIND, 4, 2>(a, st);
  if (C <= 1024) return launch<KIND, 4, 4>(a, st);
  if (C <= 2048) return launch<KIND, 8, 4>(a, st);
  if (C <= 4096) return launch<KIND, 16, 4>(a, st);
  return launch<KIND, 16, 8>(a, st);
}

}  // namespace

hipError_t launch_add_rms_quant(const NormArgs& a, int kind, int num_cu, hipStream_t st) {
  if (kind == kNormInt8) return launch_kind<kNormInt8>(a, num_cu, st);
  return kind == kNormE4m3 ? launch_kind<kNormE4m3>(a, num_cu, st) : launch_kind<kNormMx>(a, num_cu, st);
}

}  // namespace wq
