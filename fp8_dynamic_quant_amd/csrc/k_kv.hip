// A paged cache of keys and values in 8 bits, and attention over it.
//
// A page holds P tokens of every head, as codes (E4M3, or int8) and one UE8M0 byte for each
// (page, head) of keys and of values: x = code * 2^(byte - 127).  Keys lie [page][H][P][D],
// values [page][H][D][P]: the matrix instruction contracts q k over D and p v over tokens,
// and wants eight consecutive terms of a contraction from each lane, so with this layout both
// come from memory in operand order and nothing is transposed when they are read.
#include "wq_device.h"
#include "wq_kernels.h"

namespace wq {

namespace {

typedef unsigned v2u __attribute__((ext_vector_type(2)));
typedef unsigned v4u __attribute__((ext_vector_type(4)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int kRowTile = 16;   // rows (of one cache head's queries) of a tile
constexpr int kTokTile = 64;   // tokens of a wave's step
constexpr int kAttnWaves = 4;

// The sequence of slot `item` when sequence b owns the slots from offsets[b] * mul / div +
// per * b on (the host knows neither a sequence's rows nor its length, so every sequence gets
// as many slots as it can need): the last b whose first slot is not behind `item`.  Offsets are
// read as 0 .. T, whatever they hold.
struct SeqSlot {
  int b;
  int64_t row0, rows;  // its rows
  int64_t j;           // the slot's place among its slots
};
__device__ __forceinline__ int64_t seq_offset(const KvArgs& c, int b) {
  return min(max(c.offsets[b], (int64_t)0), c.T);
}
__device__ __forceinline__ SeqSlot find_slot(const KvArgs& c, int64_t item, int mul, int div, int per) {
  int lo = 0, hi = c.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (seq_offset(c, mid) * mul / div + (int64_t)per * mid <= item) lo = mid;
    else hi = mid - 1;
  }
  SeqSlot s;
  s.b = lo;
  s.row0 = seq_offset(c, lo);
  s.rows = seq_offset(c, lo + 1) - s.row0;
  s.j = item - (s.row0 * mul / div + (int64_t)per * lo);
  if (s.j < 0) s.j = s.rows = 0;  // offsets that do not begin at 0: rows before the first sequence
  return s;
}

// ---- append -------------------------------------------------------------------------------

// Exponent of a block with the largest magnitude a (a finite bf16 pattern): the smallest e with
// 2^e >= a / c, at least -127.  c = 448 = 1.75 * 2^8 (E4M3), 127 = 1.984375 * 2^6 (int8).
template <bool I8>
__device__ __forceinline__ int block_exp(uint32_t a) {
  const int E = (int)(a >> 7);
  const uint32_t F = a & 0x7Fu;  // a = 2^(E-127) (1 + F/128)
  const int e = I8 ? E - 133 + (F > 0x7Eu ? 1 : 0) : E - 135 + (F > 0x60u ? 1 : 0);
  return e < -127 ? -127 : e;
}

template <bool I8>
__device__ __forceinline__ uint32_t encode(float y) {
  if constexpr (I8) {
    return (uint32_t)(int)rintf(y) & 0xFFu;
  } else {
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y, y, 0, false) & 0xFFu;
  }
}

// a held code at a larger scale: its value times 2^d, d < 0, rounded once more.  int8 codes stay
// within a unit of the exact quotient however often a page's scale grows: each growth at least
// halves what the earlier roundings left (1/2 + 1/4 + ...).
template <bool I8>
__device__ __forceinline__ uint32_t rescale(uint32_t code, int d) {
  if constexpr (I8) {
    return (uint32_t)(int)rintf(ldexpf((float)(int8_t)code, d)) & 0xFFu;
  } else {
    if ((code & 0x7Fu) == 0x7Fu) return code;  // E4M3's NaN
    return encode<false>(ldexpf(__builtin_amdgcn_cvt_f32_fp8((int)code, 0), d)) & 0xFFu;
  }
}

// One workgroup for the new rows of one sequence in one page of one head, keys (side 0) or
// values (side 1).
template <bool I8>
__global__ __launch_bounds__(256) void k_kv_append(KvArgs c, const uint16_t* k_new, int64_t ldk, const uint16_t* v_new,
                                                   int64_t ldv) {
  __shared__ uint32_t red[4];
  const int t = threadIdx.x, h = blockIdx.y, side = blockIdx.z;
  const SeqSlot s = find_slot(c, blockIdx.x, 1, c.P, 2);
  if (s.rows <= 0) return;
  const int64_t len = c.lens[s.b], start = len - s.rows;
  const int64_t pg = max(start, (int64_t)0) / c.P + s.j;
  const int64_t lo = max(start, pg * c.P), hi = min(len, (pg + 1) * c.P);
  if (lo >= hi || pg >= c.max_pages) return;
  const int page = c.table[s.b * c.table_stride + pg];
  if (page < 0 || page >= c.pages) return;
  const int D = c.D, P = c.P, s0 = (int)(lo - pg * P), n = (int)(hi - lo);
  const int64_t ld = side ? ldv : ldk;
  const uint16_t* x = (side ? v_new : k_new) + (s.row0 + (lo - start)) * ld + (int64_t)h * D;
  // largest magnitude of the new rows
  const int per = D / 8;
  uint32_t a = 0;
  for (int i = t; i < n * per; i += 256) {
    const v4u u = *reinterpret_cast<const v4u*>(x + (i / per) * ld + (i % per) * 8);
#pragma unroll
    for (int j = 0; j < 4; ++j) a = max(a, max(u[j] & 0x7FFFu, (u[j] >> 16) & 0x7FFFu));
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) a = max(a, (uint32_t)__shfl_xor((int)a, o, 64));
  if ((t & 63) == 0) red[t >> 6] = a;
  __syncthreads();
  a = max(max(red[0], red[1]), max(red[2], red[3]));
  uint8_t* scale = (side ? c.v_scale : c.k_scale) + (int64_t)page * c.H + h;
  const int old = s0 > 0 ? *scale : 0;
  const int byte = max(old, a < 0x7F80u ? block_exp<I8>(a) + 127 : 255);
  __syncthreads();  // every thread has read the old byte
  if (t == 0) *scale = (uint8_t)byte;
  uint8_t* codes = static_cast<uint8_t*>(side ? c.v : c.k) + ((int64_t)page * c.H + h) * P * D;
  // keys: slot-major rows of D; values: D rows of P slots
  const int slot_step = side ? 1 : D, d_step = side ? P : 1;
  if (s0 > 0 && old < byte && byte != 255) {
    for (int i = t; i < s0 * D; i += 256) {
      uint8_t* at = side ? codes + (int64_t)(i / s0) * P + i % s0 : codes + i;
      *at = (uint8_t)rescale<I8>(*at, old - byte);
    }
  }
  for (int i = t; i < n * per; i += 256) {
    const int r = i / per, d = (i % per) * 8;
    const v4u u = *reinterpret_cast<const v4u*>(x + r * ld + d);
    uint8_t* at = codes + (s0 + r) * slot_step + d * d_step;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float v = __uint_as_float((j & 1) ? u[j / 2] & 0xFFFF0000u : u[j / 2] << 16);
      at[j * d_step] = byte == 255 ? 0 : (uint8_t)encode<I8>(ldexpf(v, 127 - byte));
    }
  }
}

// ---- attention -----------------------------------------------------------------------------

// eight codes -> eight bf16, exact (E4M3 has 4 significant bits, int8 at most 7)
template <bool I8>
__device__ __forceinline__ v8bf widen8(uint32_t lo, uint32_t hi) {
  v4u o;
  if constexpr (I8) {
    const uint32_t w[2] = {lo, hi};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x = w[i / 2] >> (16 * (i & 1));
      const uint32_t f0 = __float_as_uint((float)(int8_t)(x & 0xFF)), f1 = __float_as_uint((float)(int8_t)((x >> 8) & 0xFF));
      o[i] = __builtin_amdgcn_perm(f1, f0, 0x07060302u);  // the high halves: exact
    }
  } else {
    o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false));
    o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true));
    o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false));
    o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true));
  }
  return __builtin_bit_cast(v8bf, o);
}

// 2^(byte - 127); byte 255 is NaN, byte 0 the subnormal 2^-127
__device__ __forceinline__ float scale_of(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7FC00000u) : byte == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(byte << 23);
}

// max / sum over the four lane groups that share a row (lanes l, l + 16, l + 32, l + 48)
__device__ __forceinline__ float groups_max(float v) {
  v = fmaxf(v, __shfl_xor(v, 16, 64));
  return fmaxf(v, __shfl_xor(v, 32, 64));
}
__device__ __forceinline__ float groups_sum(float v) {
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

// A workgroup takes 16 rows of one sequence and cache head (row = new token * R + query head
// of the group) and one of `splits` parts of the keys they see; its four waves take 64-token
// steps in turn, each with its own running maximum and sum, joined at the end in LDS.
//
// Lane l: j = l % 16, g = l / 16.  A step's tokens are 16-token groups g = 0 .. 3, each inside
// one page (P % 16 == 0).
//  * s^T = k q^T in four 16-token instructions t: the lane that supplies k row i takes token
//    16 (i / 4) + 4 t + i % 4, so that the results, rows 4 g + r of column j, are tokens
//    16 g + 4 t + r of row j: lane group g ends with the 16 consecutive tokens of its group.
//  * o^T += v^T p^T: the lane supplies p of exactly those 16 tokens, from its own registers,
//    and v of the same 16 tokens: 16 consecutive bytes of a value row.  No exchange of lanes.
//  * the scales are one number for the lane's tokens: keys' multiplies s, values' multiplies p.
template <int D, bool I8>
__global__ __launch_bounds__(64 * kAttnWaves) void k_kv_attention(KvAttnArgs a) {
  constexpr int ND = D / 16, NC = D / 64;
  __shared__ float o_lds[kAttnWaves][kRowTile][D + 4];
  __shared__ float m_lds[kAttnWaves][kRowTile], l_lds[kAttnWaves][kRowTile];
  const KvArgs& c = a.c;
  const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int h = blockIdx.y, split = blockIdx.z, R = a.R;
  const SeqSlot s = find_slot(c, blockIdx.x, R, kRowTile, 1);
  const int64_t r0 = s.j * kRowTile, nrows = s.rows * R;
  if (r0 >= nrows) return;
  const int64_t len = c.lens[s.b];
  const int64_t seen = min(max(len, (int64_t)0), (int64_t)c.max_pages * c.P);  // tokens that the table can hold
  // rows behind the last read the last and see no key
  const int64_t rr = r0 + j, rc = min(rr, nrows - 1);
  const int64_t tok = s.row0 + rc / R;
  const int head = h * R + (int)(rc % R);
  auto limit_of = [&](int64_t row) -> int64_t {
    return a.causal ? min(max(len - s.rows + row / R + 1, (int64_t)0), seen) : seen;
  };
  const int64_t limit = rr < nrows ? limit_of(rc) : 0;
  const int64_t last = limit_of(min(r0 + kRowTile, nrows) - 1);   // the tile's longest row
  const int64_t steps = (last + kTokTile - 1) / kTokTile;
  const int64_t t_lo = steps * split / a.splits, t_hi = steps * (split + 1) / a.splits;

  v8bf qf[NC][2];
  {
    const uint16_t* q = a.q + tok * a.ldq + (int64_t)head * D + 16 * g;
#pragma unroll
    for (int cc = 0; cc < NC; ++cc)
#pragma unroll
      for (int m = 0; m < 2; ++m) qf[cc][m] = *reinterpret_cast<const v8bf*>(q + 64 * cc + 8 * m);
  }
  const float to_log2 = a.scale * 1.44269504088896340736f;
  const int32_t* table = c.table + s.b * c.table_stride;
  const int64_t page_bytes = (int64_t)c.P * D;
  float mx = -INFINITY, sum = 0.0f;
  v4f o[ND];
#pragma unroll
  for (int i = 0; i < ND; ++i) o[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  for (int64_t step = t_lo + wv; step < t_hi; step += kAttnWaves) {
    const int64_t tok0 = step * kTokTile;
    // this lane group's page; a token group past the end, or a page number outside the cache,
    // reads page 0 and is masked
    const int64_t gt = tok0 + 16 * g;
    int page = gt < seen ? table[gt / c.P] : -1;
    const bool there = page >= 0 && page < c.pages;
    page = there ? page : 0;
    const int slot = (int)(gt % c.P);
    const int64_t base = ((int64_t)page * c.H + h) * page_bytes;
    const int64_t kv_at = (int64_t)page * c.H + h;
    const float ks = scale_of(c.k_scale[kv_at]) * to_log2;
    const float vs = scale_of(c.v_scale[kv_at]);
    // the page and slot of the token group that this lane reads keys of
    const int kg = j >> 2;
    const int64_t kbase = ((int64_t)__shfl(page, kg * 16, 64) * c.H + h) * page_bytes;
    const int kslot = (int)((tok0 + 16 * kg) % c.P) + (j & 3);
    const uint8_t* kp = static_cast<const uint8_t*>(c.k) + kbase + (int64_t)kslot * D + 16 * g;
    v4f sc[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      sc[t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int cc = 0; cc < NC; ++cc) {
        const v4u kk = *reinterpret_cast<const v4u*>(kp + 4 * t * D + 64 * cc);
        sc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8<I8>(kk[0], kk[1]), qf[cc][0], sc[t], 0, 0, 0);
        sc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8<I8>(kk[2], kk[3]), qf[cc][1], sc[t], 0, 0, 0);
      }
    }
    // scores in units of log2, masked
    float top = -INFINITY;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float v = sc[t][r] * ks;
        sc[t][r] = there && gt + 4 * t + r < limit ? v : -INFINITY;
        top = fmaxf(top, sc[t][r]);
      }
    top = groups_max(top);
    const float mn = fmaxf(mx, top);
    const float base_m = mn == -INFINITY ? 0.0f : mn;
    const float alpha = __builtin_amdgcn_exp2f(mx - base_m);
    mx = mn;
    float part = 0.0f;
    v8bf pf[2];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float e = __builtin_amdgcn_exp2f(sc[t][r] - base_m);
        part += e;
        // rounded to bf16 with the values' scale on it (a power of two: no further rounding);
        // a masked token's weight is zero whatever its page's scale holds
        pf[t >> 1][(t & 1) * 4 + r] = (__bf16)(sc[t][r] == -INFINITY ? 0.0f : e * vs);
      }
    sum = sum * alpha + part;
    const uint8_t* vp = static_cast<const uint8_t*>(c.v) + base + (int64_t)j * c.P + slot;
    const int64_t rest = seen - gt;  // the group's slots from `rest` on hold anything: read as zero
    const int valid = !there || rest <= 0 ? 0 : rest >= 16 ? 16 : (int)rest;
#pragma unroll
    for (int i = 0; i < ND; ++i) {
      v4u vv = *reinterpret_cast<const v4u*>(vp + (int64_t)16 * i * c.P);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const int keep = valid - 4 * w;
        vv[w] = keep >= 4 ? vv[w] : keep <= 0 ? 0u : vv[w] & ((1u << (8 * keep)) - 1u);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) o[i][r] *= alpha;
      o[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8<I8>(vv[0], vv[1]), pf[0], o[i], 0, 0, 0);
      o[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8<I8>(vv[2], vv[3]), pf[1], o[i], 0, 0, 0);
    }
  }
  sum = groups_sum(sum);
#pragma unroll
  for (int i = 0; i < ND; ++i) *reinterpret_cast<v4f*>(&o_lds[wv][j][16 * i + 4 * g]) = o[i];
  if (g == 0) {
    m_lds[wv][j] = mx;
    l_lds[wv][j] = sum;
  }
  __syncthreads();
  // join the waves: thread -> (row, 16-th of D)
  const int row = threadIdx.x >> 4, dq = (threadIdx.x & 15) * (D / 16);
  if (r0 + row >= nrows) return;
  float M = m_lds[0][row];
#pragma unroll
  for (int w = 1; w < kAttnWaves; ++w) M = fmaxf(M, m_lds[w][row]);
  const float Mb = M == -INFINITY ? 0.0f : M;
  float L = 0.0f, wgt[kAttnWaves];
#pragma unroll
  for (int w = 0; w < kAttnWaves; ++w) {
    wgt[w] = __builtin_amdgcn_exp2f(m_lds[w][row] - Mb);
    L += wgt[w] * l_lds[w][row];
  }
  float acc[D / 16];
#pragma unroll
  for (int d = 0; d < D / 16; ++d) {
    acc[d] = 0.0f;
#pragma unroll
    for (int w = 0; w < kAttnWaves; ++w) acc[d] += wgt[w] * o_lds[w][row][dq + d];
  }
  const int64_t orow = r0 + row;
  if (a.splits == 1) {
    const float inv = M == -INFINITY ? 0.0f : 1.0f / L;
    uint16_t* out = a.out + (s.row0 + orow / R) * a.ldo + (int64_t)(h * R + orow % R) * D + dq;
#pragma unroll
    for (int d = 0; d < D / 16; ++d) out[d] = (uint16_t)f32_to_bf16_nan(acc[d] * inv);
    if (a.lse && dq == 0)
      a.lse[(s.row0 + orow / R) * (int64_t)(c.H * R) + h * R + orow % R] =
          M == -INFINITY ? -INFINITY : (M + __builtin_amdgcn_logf(L)) * 0.69314718055994530942f;
  } else {
    const int64_t at = (((int64_t)blockIdx.x * c.H + h) * a.splits + split) * kRowTile + row;
    float* part = a.part + at * D + dq;
#pragma unroll
    for (int d = 0; d < D / 16; ++d) part[d] = acc[d];
    if (dq == 0) a.stat[at] = float2{M, L};
  }
}

// The parts of one row tile, joined in order: one workgroup for each (row tile, cache head).
template <int D>
__global__ __launch_bounds__(256) void k_kv_join(KvAttnArgs a) {
  const KvArgs& c = a.c;
  const int h = blockIdx.y, R = a.R;
  const SeqSlot s = find_slot(c, blockIdx.x, R, kRowTile, 1);
  const int64_t r0 = s.j * kRowTile, nrows = s.rows * R;
  const int row = threadIdx.x >> 4, dq = (threadIdx.x & 15) * (D / 16);
  if (r0 + row >= nrows) return;
  const int64_t at = ((int64_t)blockIdx.x * c.H + h) * a.splits * kRowTile + row;
  float M = -INFINITY;
  for (int i = 0; i < a.splits; ++i) M = fmaxf(M, a.stat[at + (int64_t)i * kRowTile].x);
  const float Mb = M == -INFINITY ? 0.0f : M;
  float L = 0.0f, acc[D / 16];
#pragma unroll
  for (int d = 0; d < D / 16; ++d) acc[d] = 0.0f;
  for (int i = 0; i < a.splits; ++i) {
    const float2 st = a.stat[at + (int64_t)i * kRowTile];
    const float w = __builtin_amdgcn_exp2f(st.x - Mb);
    L += w * st.y;
    const float* part = a.part + (at + (int64_t)i * kRowTile) * D + dq;
#pragma unroll
    for (int d = 0; d < D / 16; ++d) acc[d] += w * part[d];
  }
  const int64_t orow = r0 + row;
  const float inv = M == -INFINITY ? 0.0f : 1.0f / L;
  uint16_t* out = a.out + (s.row0 + orow / R) * a.ldo + (int64_t)(h * R + orow % R) * D + dq;
#pragma unroll
  for (int d = 0; d < D / 16; ++d) out[d] = (uint16_t)f32_to_bf16_nan(acc[d] * inv);
  if (a.lse && dq == 0)
    a.lse[(s.row0 + orow / R) * (int64_t)(c.H * R) + h * R + orow % R] =
        M == -INFINITY ? -INFINITY : (M + __builtin_amdgcn_logf(L)) * 0.69314718055994530942f;
}

}  // namespace

hipError_t launch_kv_append(const KvArgs& c, bool i8, const uint16_t* k_new, int64_t ldk, const uint16_t* v_new,
                            int64_t ldv, hipStream_t st) {
  const dim3 grid((unsigned)(c.T / c.P + 2 * (int64_t)c.B), (unsigned)c.H, 2);
  if (i8)
    hipLaunchKernelGGL(k_kv_append<true>, grid, dim3(256), 0, st, c, k_new, ldk, v_new, ldv);
  else
    hipLaunchKernelGGL(k_kv_append<false>, grid, dim3(256), 0, st, c, k_new, ldk, v_new, ldv);
  return hipGetLastError();
}

bool kv_head_dim_ok(int64_t D) { return D == 64 || D == 128 || D == 256; }

template <int D>
static hipError_t attention_of(const KvAttnArgs& a, bool i8, unsigned tiles, hipStream_t st) {
  const dim3 grid(tiles, (unsigned)a.c.H, (unsigned)a.splits), block(64 * kAttnWaves);
  if (i8)
    hipLaunchKernelGGL((k_kv_attention<D, true>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((k_kv_attention<D, false>), grid, block, 0, st, a);
  if (a.splits > 1) hipLaunchKernelGGL(k_kv_join<D>, dim3(tiles, (unsigned)a.c.H), dim3(256), 0, st, a);
  return hipGetLastError();
}

static int64_t row_tiles(const KvArgs& c, int R) { return c.T * R / kRowTile + c.B; }

// Parts of the keys: enough workgroups for the chip, while the longest sequence that the table
// can hold keeps a step for each wave of a part.
int kv_attention_splits(const KvArgs& c, int R, int num_cu) {
  const int64_t wgs = row_tiles(c, R) * c.H;
  const int64_t most = ((int64_t)c.max_pages * c.P + kTokTile * kAttnWaves - 1) / (kTokTile * kAttnWaves);
  return (int)max((int64_t)1, min((2 * (int64_t)num_cu + wgs - 1) / wgs, min(most, (int64_t)65535)));
}

size_t kv_attention_workspace(const KvArgs& c, int R, int num_cu) {
  const int splits = kv_attention_splits(c, R, num_cu);
  return splits == 1 ? 0 : (size_t)(row_tiles(c, R) * c.H * kRowTile * splits) * (c.D * 4 + 8);
}

hipError_t launch_kv_attention(KvAttnArgs a, bool i8, int num_cu, void* ws, hipStream_t st) {
  const int64_t tiles = row_tiles(a.c, a.R);
  a.splits = kv_attention_splits(a.c, a.R, num_cu);
  a.part = static_cast<float*>(ws);
  a.stat = a.splits > 1 ? reinterpret_cast<float2*>(a.part + tiles * a.c.H * kRowTile * a.splits * a.c.D) : nullptr;
  if (a.c.D == 64) return attention_of<64>(a, i8, (unsigned)tiles, st);
  if (a.c.D == 128) return attention_of<128>(a, i8, (unsigned)tiles, st);
  return attention_of<256>(a, i8, (unsigned)tiles, st);
}

}  // namespace wq
