// Launch interface of the 4-bit blocks, the products on them, and the paged 8-bit cache.  Apart
// from wq_kernels.h, whose text the headline kernel's tracked profiles are keyed by.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

namespace wq {

// A launch counts its threads along each axis in 32 bits: of more workgroups than this, x counts
// kGridX at a time and y the rest (append, which has no axis left, takes several launches).
constexpr uint32_t kGridXLog = 22, kGridX = 1u << kGridXLog;
inline dim3 folded_grid(int64_t blocks) {
  return dim3(blocks < kGridX ? (unsigned)blocks : kGridX, (unsigned)((blocks + kGridX - 1) >> kGridXLog));
}

// Microscaled 4-bit blocks (k_mxfp4.hip): bf16 [T, G, D] -> E2M1 pairs [T, G, D/2] and UE8M0
// words [G, ceil(D/128), align4(T)], and back (D % 32 == 0)
hipError_t launch_group_quant_mxfp4(const uint16_t* x, int64_t T, int G, int D, uint8_t* xq, int32_t* xs,
                                    hipStream_t st);
hipError_t launch_group_dequant_mxfp4(const uint8_t* xq, const int32_t* xs, int64_t T, int G, int D, uint16_t* y,
                                      hipStream_t st);
// Product on 4-bit weights (k_mx4_gemm.hip), N % 16 == 0, K % 128 == 0, lda < 2^23.
struct Mx4Args {
  const uint8_t* a;        // rows of E2M1 pairs (K/2 bytes) or E4M3 codes (K bytes)
  int64_t lda;             // bytes between rows
  int64_t a_batch_stride;  // bytes between groups
  const int32_t* a_scale;  // [batch][K/128][a_tokens]
  int64_t a_tokens;
  const uint8_t* w;        // [batch][N][K/2]
  int64_t w_batch_stride;  // bytes between groups
  const int32_t* w_scale;  // [batch][K/128][N]
  uint16_t* y;             // bf16
  int64_t ldy, y_batch_stride;
  int M, N, K, batch;
};
// a8: E4M3 activation codes instead of E2M1 pairs
hipError_t launch_mx4(const Mx4Args& a, bool a8, int num_cu, hipStream_t st);
// its kernel, as wq_mx4_path numbers them
int mx4_path(int M, int N, int batch, int num_cu);

// The paged 8-bit cache (k_kv.hip).  A page holds P tokens of every head: k [page][H][P][D],
// v [page][H][D][P], one UE8M0 byte for each (page, head) of either.
struct KvArgs {
  void* k;
  void* v;
  uint8_t* k_scale;
  uint8_t* v_scale;
  const int32_t* table;     // [B][table_stride], the first max_pages entries of a row used
  int64_t table_stride;
  int pages, H, P, D, max_pages;
  uint32_t page_recip;      // ceil(2^32 / (P / 16)): token groups of 16 to pages without a division
  const int64_t* offsets;   // [B + 1]: rows of each sequence
  const int32_t* lens;      // [B]: tokens of each sequence, the new rows among them
  int B;
  int64_t T;                // rows in all
};
hipError_t launch_kv_append(const KvArgs& c, bool i8, const uint16_t* k_new, int64_t ldk, const uint16_t* v_new,
                            int64_t ldv, hipStream_t st);
// an item that several workgroups share (k_kv_join): its parts' slots, and the rows it is of
struct KvJoin {
  int parts, first_slot, h, tile, row0, rows, spare[2];
};
struct KvAttnArgs {
  KvArgs c;
  const uint16_t* q;        // bf16 [T][Hq * D], row stride ldq
  int64_t ldq;
  uint16_t* out;            // bf16 [T][Hq * D], row stride ldo
  int64_t ldo;
  float* lse;               // [T][Hq] or null
  float scale;
  int R;                    // query heads of each cache head
  int causal;
  // set by the launcher: workgroups that share the work, its least share in steps, whether items
  // are cut, the steps that an item counts besides its own, the rows of a tile, and for items that are cut the parts' unnormalised sums
  // [runs][2][tile_rows][D], running maxima (log2) and sums [runs][2][tile_rows], and [runs] joins
  int runs, least, cut, fixed, tile_rows;
  float* part;
  float2* stat;
  KvJoin* joins;
};
bool kv_head_dim_ok(int64_t D);
// how a call of these sizes runs, as wq_kv_attention_path numbers it, and the bytes that joining
// cut items takes
int kv_attention_path(const KvArgs& c, int R, int num_cu);
size_t kv_attention_workspace(const KvArgs& c, int R, int num_cu);
hipError_t launch_kv_attention(KvAttnArgs a, bool i8, int num_cu, void* ws, hipStream_t st);

}  // namespace wq
