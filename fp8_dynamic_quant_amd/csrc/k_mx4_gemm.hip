// Products on 4-bit weights in 32-element blocks:
//   y[m, g, n] = sum over 32-deep blocks of 2^(ea + eb) sum a b
// with E2M1 or E4M3 activations, by the block-scaled matrix instructions, whose 128-deep step
// is one scale word (four UE8M0 bytes) of either operand.  f32 sums, one rounding to bf16.
//
// Operand layout (measured on gfx950 with one-hot inputs and distinct block scales).  Lane
// groups q: of 16 lanes for v_mfma_scale_f32_16x16x128_f8f6f4, of 32 for 32x32x64 (Q = 4 or 2
// groups).  Of a 4-bit operand, lane group q holds K 32q .. 32q+31 in its first four registers;
// of an 8-bit one K 16q .. 16q+15 in its first four and 16 Q + 16q .. +15 in its last four.  The
// scale operand of lane group s applies to K 32s .. 32s+31 of either.
#include <type_traits>

#include "wq_dma.h"
#include "wq_kernels.h"
#include "wq_mx4_kv.h"

namespace wq {

namespace {

typedef unsigned v2u __attribute__((ext_vector_type(2)));
typedef unsigned v4u __attribute__((ext_vector_type(4)));

__device__ __forceinline__ v8i regs4(const v4i lo) { return v8i{lo[0], lo[1], lo[2], lo[3], 0, 0, 0, 0}; }
__device__ __forceinline__ v8i regs8(const v4i lo, const v4i hi) {
  return v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}

// ---- few rows: the weights stream past ------------------------------------------------------
// A workgroup makes up to 16 rows x 16 CT columns of one group over all of K: eight waves
// take eight runs of 128-deep steps, operands straight from memory into registers (each byte of
// the weights is read once), and add their f32 sums in LDS in wave order.  What bounds it is the
// latency of one round of loads, at large sizes the weights' stream: M=1 N=1024 K=4096 takes 3.1 us
// (1.7 of them any kernel's), M=1 G=8 N=1024 K=4096 5.5 us (17.8 MB, 3.25 TB/s), M=1 N=8192 K=8192
// 8.4 us (4.2 TB/s).
constexpr int kFewWaves = 8, kFewSteps = 4;  // and steps whose operands are in flight together

template <bool A8, int CT>
__global__ __launch_bounds__(64 * kFewWaves) void k_mx4_few(Mx4Args p) {
  __shared__ float red[kFewWaves][CT * 4][64];
  const int t = threadIdx.x, lane = t & 63;
  const int wv = __builtin_amdgcn_readfirstlane(t >> 6);
  const int cl = lane & 15, q = lane >> 4;
  // workgroups go to the XCDs in turn: each XCD takes a run of consecutive slices of columns, so that
  // a group's rows come into as few L2s as can be
  const int S = gridDim.x, all = S * gridDim.y, id = blockIdx.x + S * blockIdx.y;
  const int item = (all & 7) == 0 ? (id & 7) * (all >> 3) + (id >> 3) : id;
  const int g = item / S, n0 = item % S * 16 * CT, M = p.M, N = p.N, KT = p.K >> 7;
  const int k_lo = KT * wv / kFewWaves, k_hi = KT * (wv + 1) / kFewWaves;
  const uint8_t* A = p.a + g * p.a_batch_stride + q * 16;
  const uint8_t* W = p.w + g * p.w_batch_stride + q * 16;
  const int32_t* SA = p.a_scale + (int64_t)g * KT * p.a_tokens;
  const int32_t* SW = p.w_scale + (int64_t)g * KT * N;
  // rows behind the last read the last, columns likewise: they feed outputs that are not stored
  const int row = min(cl, M - 1);
  const uint8_t* ar = A + row * p.lda;
  const uint8_t* wr[CT];
  int col[CT];
#pragma unroll
  for (int j = 0; j < CT; ++j) {
    col[j] = min(n0 + 16 * j + cl, N - 1);
    wr[j] = W + (int64_t)col[j] * (p.K / 2);
  }
  v4f acc[CT];
#pragma unroll
  for (int j = 0; j < CT; ++j) acc[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  constexpr int F = kFewSteps;
  for (int k0 = k_lo; k0 < k_hi; k0 += F) {
    v4i w[F][CT], lo[F], hi[F];
    int sa[F], sw[F][CT];
#pragma unroll
    for (int s = 0; s < F; ++s) {
      const int kb = min(k0 + s, k_hi - 1);  // loads of steps past the run are not used
#pragma unroll
      for (int j = 0; j < CT; ++j) {
        w[s][j] = *reinterpret_cast<const v4i*>(wr[j] + kb * 64);
        sw[s][j] = SW[(int64_t)kb * N + col[j]];
      }
      sa[s] = SA[kb * p.a_tokens + row];
      lo[s] = *reinterpret_cast<const v4i*>(ar + kb * (A8 ? 128 : 64));
      if constexpr (A8) hi[s] = *reinterpret_cast<const v4i*>(ar + kb * 128 + 64);
    }
    __builtin_amdgcn_sched_barrier(0);  // every load above before the first use
#pragma unroll
    for (int s = 0; s < F; ++s) {
      if (k0 + s < k_hi) {  // uniform
        const v8i a = A8 ? regs8(lo[s], hi[s]) : regs4(lo[s]);
#pragma unroll
        for (int j = 0; j < CT; ++j)
          acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              a, regs4(w[s][j]), acc[j], A8 ? 0 : 4, 4, 0, (uint32_t)sa[s] >> (8 * q), 0, (uint32_t)sw[s][j] >> (8 * q));
      }
    }
  }
#pragma unroll
  for (int j = 0; j < CT; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) red[wv][j * 4 + r][lane] = acc[j][r];
  __syncthreads();
  uint16_t* Y = p.y + g * p.y_batch_stride;
  for (int e = t; e < CT * 4 * 64; e += 64 * kFewWaves) {
    const int ln = e & 63, r = (e >> 6) & 3, j = e >> 8;
    // output layout: column lane % 16, row 4 (lane / 16) + r
    const int m = 4 * (ln >> 4) + r, n = n0 + 16 * j + (ln & 15);
    float v = red[0][e >> 6][ln];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) v += red[w][e >> 6][ln];
    if (m < M && n < N) Y[m * p.ldy + n] = (uint16_t)f32_to_bf16_nan(v);
  }
}

// ---- many rows: tiles -----------------------------------------------------------------------
// 64 WM x 64 WN outputs for a workgroup of four waves (2 x 2, 32 WM x 32 WN each, of 32 x 32
// instructions).  128-deep slices of both operands and of their scale words go global -> LDS
// by DMA into a ring of S stages, S - 1 ahead; two workgroups share a CU, so that one's
// epilogue runs beside the other's matrix instructions.  With KS = 2 a second four waves take the
// odd slices (a slice of a 64 x 64 tile is a chain of wait, barrier, LDS read and two dependent
// instructions, which two halves go through side by side: M=64 G=8 N=1024 K=4096 11.8 -> 10.6 us),
// and their sums are added through LDS.
// What bounds it: with large tiles no single unit (M=8192 N=32768 K=1024: 202 us alone at 2.0 GHz, 233 -
// 260 in a row; matrix instructions take 32 % of the cycles, others 30, LDS reads 25 and DMA writes about 13 %), but
// the chain of wait, barrier, LDS reads and instructions that two waves a SIMD go through (a quarter
// of their time they wait for loads, 38 % to issue), beside 537 MB of output; with 8-bit activations
// matrix instructions take 53 % (297 us in a row).  256 x 256 tiles, which read less
// from L2, were no faster: 269.  With small tiles the chain of a slice, and CUs without a tile:
// M=64 G=8 N=1024 K=4096 has 128 tiles, 10.6 us, 2.0 TB/s.  Outputs are stored past the caches: they
// would drive out operands (269 -> 250 us at M=8192).
//
// A 4-bit row's slice is 64 bytes, four chunks of 16; four rows make a 256-byte line of LDS
// (all its banks), and a chunk is XORed with bits 2..3 of its row, so that sixteen rows read at
// one chunk meet sixteen different bank groups.  An 8-bit row's slice is 128 bytes, eight chunks,
// XORed with bits 1..3.
template <int B>
__device__ __forceinline__ int chunk_swz(int row) { return B == 64 ? (row >> 2) & 3 : (row >> 1) & 7; }
template <int B>
__device__ __forceinline__ int lds_at(int row, int c) { return row * B + ((c ^ chunk_swz<B>(row)) << 4); }

template <bool A8, int WM, int WN, int S, int KS>
struct Ring {
  static constexpr int kBM = 64 * WM, kBN = 64 * WN;
  static constexpr int kARow = A8 ? 128 : 64;          // bytes of a row's slice
  static constexpr int kA = kBM * kARow, kW = kBN * 64, kS = (kBM + kBN) * 4;
  static constexpr int kStage = kA + kW + kS;
  static constexpr int kNA = kA / 4096, kNW = kW / 4096, kNS = (kBM + kBN + 255) / 256;  // DMAs of a wave
  static constexpr int kDma = kNA + kNW + kNS;
  static constexpr int kOut = kBM * kBN * 2;           // the bf16 tile, staged in the ring's place
  static constexpr int kSum = (KS - 1) * kBM * kBN * 4; // sums of the waves behind the first four
  static constexpr int kBytes = KS * S * kStage > kOut + kSum ? KS * S * kStage : kOut + kSum;
};

template <bool A8, int WM, int WN, int S, int KS>
__global__ __launch_bounds__(256 * KS, 2) void k_mx4_tile(Mx4Args p, int tiles_m, int tiles_n, int per_xcd) {
  using R = Ring<A8, WM, WN, S, KS>;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int t = threadIdx.x, lane = t & 63;
  const int wv = __builtin_amdgcn_readfirstlane(t >> 6) & 3, wm = wv >> 1, wn = wv & 1;
  const int ks = KS == 1 ? 0 : __builtin_amdgcn_readfirstlane(t >> 8);
  const int M = p.M, N = p.N, KT = p.K >> 7, ST = (KT + KS - 1) / KS;  // slices, steps
  // workgroups go to the XCDs in turn; each XCD takes a run of consecutive tiles, in groups of
  // eight tile rows, so that what its L2 holds is used by its neighbours
  const int per_group = tiles_m * tiles_n;
  const int64_t id = (int64_t)(blockIdx.x & 7) * per_xcd + (blockIdx.x >> 3);
  if (id >= (int64_t)per_group * p.batch) return;
  const int g = (int)(id / per_group), in_g = (int)(id % per_group);
  const int band = in_g / (8 * tiles_n), rows8 = min(8, tiles_m - 8 * band), in_b = in_g - band * 8 * tiles_n;
  const int m0 = (8 * band + in_b % rows8) * R::kBM, n0 = in_b / rows8 * R::kBN;

  const uint8_t* A = p.a + g * p.a_batch_stride + (int64_t)m0 * p.lda;
  const uint8_t* W = p.w + g * p.w_batch_stride + (int64_t)n0 * (p.K / 2);
  const int32_t* SA = p.a_scale + (int64_t)g * KT * p.a_tokens + m0;
  const int32_t* SW = p.w_scale + (int64_t)g * KT * N + n0;
  // lane offsets of this wave's DMA instructions wv, wv + 4, ...: position 64 i + lane of the
  // slice in LDS is a row's chunk; rows behind the last read the last
  uint32_t aoff[R::kNA], woff[R::kNW], soff[R::kNS];
#pragma unroll
  for (int i = 0; i < R::kNA; ++i) {
    constexpr int per = R::kARow / 16;
    const int pos = (wv + 4 * i) * 64 + lane, r = pos / per, c = (pos % per) ^ chunk_swz<R::kARow>(r);
    aoff[i] = (uint32_t)(min(r, M - 1 - m0) * (int)p.lda + c * 16);
  }
#pragma unroll
  for (int i = 0; i < R::kNW; ++i) {
    const int pos = (wv + 4 * i) * 64 + lane, r = pos / 4, c = (pos % 4) ^ chunk_swz<64>(r);
    woff[i] = (uint32_t)(min(r, N - 1 - n0) * (p.K / 2) + c * 16);
  }
  constexpr int kWordDmas = (R::kBM + R::kBN) / 64;  // the rows' words first, then the columns'
#pragma unroll
  for (int i = 0; i < R::kNS; ++i) {
    const int d = (wv + 4 * i) % kWordDmas, r = d * 64 + lane;
    soff[i] = (uint32_t)(d < WM ? min(r, M - 1 - m0) : min(r - R::kBM, N - 1 - n0)) * 4u;
  }
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_ptr_u8)smem;
  auto issue = [&](int step, int stage) __attribute__((always_inline)) {
    const int kt = KS == 1 ? step : min(KS * step + ks, KT - 1);
    const uint32_t st = lds0 + (stage * KS + ks) * R::kStage;
    const uint8_t* a = A + (int64_t)kt * R::kARow;
    const uint8_t* w = W + (int64_t)kt * 64;
#pragma unroll
    for (int i = 0; i < R::kNA; ++i) dma16(a, aoff[i], st + (wv + 4 * i) * 1024);
#pragma unroll
    for (int i = 0; i < R::kNW; ++i) dma16(w, woff[i], st + R::kA + (wv + 4 * i) * 1024);
#pragma unroll
    for (int i = 0; i < R::kNS; ++i) {
      const int d = (wv + 4 * i) % kWordDmas;
      const int32_t* s = d < WM ? SA + kt * p.a_tokens : SW + (int64_t)kt * N;
      dma4(s, soff[i], st + R::kA + R::kW + d * 256);
    }
  };

  v16f acc[WM][WN];
#pragma unroll
  for (int i = 0; i < WM; ++i)
#pragma unroll
    for (int j = 0; j < WN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
  const int l32 = lane & 31, h = lane >> 5;
  const int ar = wm * 32 * WM + l32, wr = wn * 32 * WN + l32;
  auto multiply = [&](int stage) __attribute__((always_inline)) {
    const uint8_t* sa = smem + (stage * KS + ks) * R::kStage;
    const uint8_t* sw = sa + R::kA;
    const uint32_t* ss = reinterpret_cast<const uint32_t*>(sw + R::kW);
    uint32_t xa[WM], xw[WN];
#pragma unroll
    for (int i = 0; i < WM; ++i) xa[i] = ss[ar + 32 * i] >> (8 * h);
#pragma unroll
    for (int j = 0; j < WN; ++j) xw[j] = ss[R::kBM + wr + 32 * j] >> (8 * h);
    v4i al[2][WM], ah[2][WM], wf[2][WN];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int i = 0; i < WM; ++i) {
        if constexpr (A8) {
          al[s][i] = *reinterpret_cast<const v4i*>(sa + lds_at<128>(ar + 32 * i, 4 * s + h));
          ah[s][i] = *reinterpret_cast<const v4i*>(sa + lds_at<128>(ar + 32 * i, 4 * s + 2 + h));
        } else {
          al[s][i] = *reinterpret_cast<const v4i*>(sa + lds_at<64>(ar + 32 * i, 2 * s + h));
        }
      }
#pragma unroll
      for (int j = 0; j < WN; ++j) wf[s][j] = *reinterpret_cast<const v4i*>(sw + lds_at<64>(wr + 32 * j, 2 * s + h));
    }
    // the weights are the first operand: a lane ends with four consecutive columns of a row
#pragma unroll
    for (int i = 0; i < WM; ++i)
#pragma unroll
      for (int j = 0; j < WN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            regs4(wf[0][j]), A8 ? regs8(al[0][i], ah[0][i]) : regs4(al[0][i]), acc[i][j], 4, A8 ? 0 : 4, 0, xw[j], 0, xa[i]);
#pragma unroll
    for (int i = 0; i < WM; ++i)
#pragma unroll
      for (int j = 0; j < WN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            regs4(wf[1][j]), A8 ? regs8(al[1][i], ah[1][i]) : regs4(al[1][i]), acc[i][j], 4, A8 ? 0 : 4, 2, xw[j], 2, xa[i]);
  };

  // steps 0 .. S - 2 are sent ahead (past the last one, the last again: never read)
#pragma unroll
  for (int s = 0; s < S - 1; ++s) issue(min(s, ST - 1), s);
  int kt = 0, stage = 0;
  for (; kt + S - 1 < ST; ++kt) {
    wait_vm<R::kDma*(S - 2)>();  // this wave's share of slice kt has landed
    lds_barrier();               // everyone's has, and slice kt - 1 has been read by all
    const int next = stage == 0 ? S - 1 : stage - 1;
    issue(kt + S - 1, next);
    multiply(stage);
    stage = stage + 1 == S ? 0 : stage + 1;
  }
  // the last steps, nothing left to send
  auto last = [&](auto left) __attribute__((always_inline)) {
    constexpr int L = decltype(left)::value;  // steps behind this one
    if (kt + L == ST - 1) {
      wait_vm<R::kDma * L>();
      lds_barrier();
      if (KS == 1 || L > 0 || KS * kt + ks < KT) multiply(stage);
      stage = stage + 1 == S ? 0 : stage + 1;
      ++kt;
    }
  };
  if constexpr (S >= 4) last(std::integral_constant<int, 2>{});
  if constexpr (S >= 3) last(std::integral_constant<int, 1>{});
  last(std::integral_constant<int, 0>{});

  // ---- bf16, through LDS: a wave's tile is 32 WM rows of 64 WN bytes, its chunks of 16 bytes
  // XORed with the row, so that both the 8-byte writes (a row a lane) and the reads of whole
  // rows meet all banks; then 16 bytes a lane to memory
  lds_barrier();
  if constexpr (KS == 2) {  // the second half of the slices' sums come through LDS
    v4f* sum = reinterpret_cast<v4f*>(smem + R::kOut) + wv * (WM * WN * 4 * 64) + lane;
    if (ks == 1) {
#pragma unroll
      for (int e = 0; e < WM * WN * 4; ++e) {
        const v16f& c = acc[e / 4 / WN][e / 4 % WN];
        sum[e * 64] = v4f{c[e % 4 * 4], c[e % 4 * 4 + 1], c[e % 4 * 4 + 2], c[e % 4 * 4 + 3]};
      }
    }
    __syncthreads();
    if (ks == 1) return;
#pragma unroll
    for (int e = 0; e < WM * WN * 4; ++e) {
      const v4f c = sum[e * 64];
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[e / 4 / WN][e / 4 % WN][e % 4 * 4 + r] += c[r];
    }
  }
  constexpr int RB = 64 * WN, CH = RB / 16;
  uint8_t* so = smem + wv * (32 * WM * RB);
  auto out_at = [&](int r, int c) { return r * RB + ((c ^ (CH == 16 ? r & 15 : CH == 8 ? (r >> 1) & 7 : (r >> 2) & 3)) << 4); };
#pragma unroll
  for (int i = 0; i < WM; ++i)
#pragma unroll
    for (int j = 0; j < WN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t w0 = f32_to_bf16_nan(acc[i][j][4 * q]) | f32_to_bf16_nan(acc[i][j][4 * q + 1]) << 16;
        const uint32_t w1 = f32_to_bf16_nan(acc[i][j][4 * q + 2]) | f32_to_bf16_nan(acc[i][j][4 * q + 3]) << 16;
        *reinterpret_cast<v2u*>(so + out_at(32 * i + l32, 4 * j + q) + 8 * h) = v2u{w0, w1};
      }
  constexpr int RPI = 64 / CH;  // rows of one store instruction
  const int mw = m0 + wm * 32 * WM, n = n0 + wn * 32 * WN + (lane % CH) * 8;
  uint16_t* Y = p.y + g * p.y_batch_stride + n;
#pragma unroll
  for (int k = 0; k < 32 * WM / RPI; ++k) {
    const int r = k * RPI + lane / CH;
    const v4u v = *reinterpret_cast<const v4u*>(so + out_at(r, lane % CH));
    if (mw + r < M && n < N) __builtin_nontemporal_store(v, reinterpret_cast<v4u*>(Y + (int64_t)(mw + r) * p.ldy));
  }
}

template <bool A8, int CT>
hipError_t few(const Mx4Args& a, hipStream_t st) {
  const dim3 grid((unsigned)((a.N + 16 * CT - 1) / (16 * CT)), (unsigned)a.batch);
  hipLaunchKernelGGL((k_mx4_few<A8, CT>), grid, dim3(64 * kFewWaves), 0, st, a);
  return hipGetLastError();
}

template <bool A8, int WM, int WN, int S, int KS>
hipError_t tile(const Mx4Args& a, hipStream_t st) {
  using R = Ring<A8, WM, WN, S, KS>;
  const int64_t tm = (a.M + R::kBM - 1) / R::kBM, tn = (a.N + R::kBN - 1) / R::kBN;
  const int64_t total = tm * tn * a.batch, per_xcd = (total + 7) / 8;
  // threads of a launch are counted in 32 bits (beyond that the operands alone are 200 GB)
  if (per_xcd * 8 * 256 * KS >= ((int64_t)1 << 32)) return hipErrorInvalidValue;
  const void* kernel = reinterpret_cast<const void*>(k_mx4_tile<A8, WM, WN, S, KS>);
  hipError_t e = set_lds_limit(kernel, R::kBytes);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_mx4_tile<A8, WM, WN, S, KS>), dim3((unsigned)(per_xcd * 8)), dim3(256 * KS), R::kBytes, st, a, (int)tm,
                     (int)tn, (int)per_xcd);
  return hipGetLastError();
}

template <bool A8>
hipError_t launch(const Mx4Args& a, int path, hipStream_t st) {
  switch (path) {
    case 1: return few<A8, 1>(a, st);
    case 2: return few<A8, 2>(a, st);
    case 3: return tile<A8, 1, 1, 4, 2>(a, st);
    case 4: return tile<A8, 1, 2, 4, 1>(a, st);
    default: return tile<A8, 2, 4, A8 ? 2 : 3, 1>(a, st);
  }
}

}  // namespace

int mx4_path(int M, int N, int batch, int num_cu) {
  // Tiles of 64 x 64, 64 x 128 or 128 x 256: the largest that still give every CU one, since what a
  // CU reads for an output shrinks with the tile (64 x 64 against 64 x 128, us: M=64 G=8 N=1024
  // K=4096 10.6 / 14.1, M=1000 N=2064 K=1152 13.8 / 9.2; 64 x 128 against 128 x 256: M=2048 N=4096
  // K=4096 36.7 / 28.0, M=8192 N=32768 K=1024 308 / 246).
  const int64_t narrow = (int64_t)((M + 63) / 64) * ((N + 63) / 64) * batch;
  // Up to 16 rows the streaming kernel, unless 64-column tiles fill the chip by themselves (streaming
  // against tiles, us: M=16 G=8 N=1024 K=4096 6.7 / 8.9, M=1 N=8192 K=8192 8.5 / 12.0; at 256 tiles
  // M=1 N=16384 K=4096 7.9 / 8.1, M=16 8.9 / 8.3; at 512 M=1 N=32768 K=1024 11.2 / 5.9, M=16
  // K=8192 40.6 / 34.5).  32 columns to a workgroup where two a CU remain, else 16 (16 against 32:
  // M=16 G=8 N=1024 K=4096 8.3 / 6.7, M=1 N=1024 K=4096 3.1 / 4.1).
  if (M <= 16 && narrow < num_cu) return (int64_t)N / 16 * batch >= 2 * num_cu ? 2 : 1;
  const int64_t large = (int64_t)((M + 127) / 128) * ((N + 255) / 256) * batch;
  if (large >= num_cu) return 5;
  const int64_t small = (int64_t)((M + 63) / 64) * ((N + 127) / 128) * batch;
  return small >= num_cu ? 4 : 3;
}

hipError_t launch_mx4(const Mx4Args& a, bool a8, int num_cu, hipStream_t st) {
  const int path = mx4_path(a.M, a.N, a.batch, num_cu);
  return a8 ? launch<true>(a, path, st) : launch<false>(a, path, st);
}

}  // namespace wq
