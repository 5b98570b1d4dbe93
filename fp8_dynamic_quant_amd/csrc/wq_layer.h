// Launch interface of what stands between a layer's products: the residual's norm in 8 bits, turned
// keys and queries, and attention behind a shared prefix.
#pragma once

#include "wq_mx4_kv.h"

namespace wq {

// The residual's addition, RMSNorm and 8-bit rows (k_norm.hip).
enum { kNormInt8 = 0, kNormE4m3 = 1, kNormMx = 2 };
struct NormArgs {
  const uint16_t* x;        // bf16 [M][K], row stride ldx
  int64_t ldx;
  const uint16_t* residual; // bf16 [M][K], row stride ldr, or null
  int64_t ldr;
  const uint16_t* gamma;    // bf16 [K]
  float eps;
  double inv_k;             // RN(1 / K)
  int64_t M;
  int K;
  uint16_t* sum;            // bf16 [M][K], row stride lds, or null
  int64_t lds;
  uint16_t* y;              // bf16 [M][K], row stride ldy, or null
  int64_t ldy;
  uint8_t* xq;              // codes [M][K]
  void* xs;                 // f32 [M], or words [ceil(K / (4 block))][align4(M)]
};
hipError_t launch_add_rms_quant(const NormArgs& a, int kind, int num_cu, hipStream_t st);

// Append with turned keys, and turned queries (k_kv_rotated.hip).
struct TurnArgs {
  const float* angles;      // [positions][2][rot / 2]: cosines, then sines
  int64_t positions;
  int rot;                  // elements turned, a multiple of 16
  const uint16_t* q;        // bf16 [T][H * R * D], row stride ldq, or null
  int64_t ldq;
  uint16_t* q_out;          // row stride ldo
  int64_t ldo;
  int R;
};
hipError_t launch_kv_append_rotated(const KvArgs& c, bool i8, bool pairs, const uint16_t* k_new, int64_t ldk,
                                    const uint16_t* v_new, int64_t ldv, const TurnArgs& r, hipStream_t st);

// Attention of sequences that share their first pages (k_kv_shared.hip).
size_t kv_shared_workspace(const KvArgs& c, int R, int num_cu);
int kv_shared_path(const KvArgs& c, int R, int num_cu);
hipError_t launch_kv_attention_shared(KvAttnArgs a, bool i8, const int32_t* group, const int32_t* shared, int num_cu,
                                      void* ws, hipStream_t st);

}  // namespace wq
