// The cut of attention behind a shared prefix into runs, in whole numbers: what the kernels and the
// host go by.  It needs no device, so that its test builds it for the CPU.
#pragma once

#include <cstdint>

namespace wq {

constexpr int kShareSeqs = 512;  // sequences of one launch (their plan is held in LDS)
constexpr int kShareWaves = 8;   // waves of a workgroup

enum { kNarrow = 0, kWide = 1 };
constexpr int kNarrowRows = 16;
__host__ __device__ constexpr int wide_rows(int D) { return D == 256 ? 128 : 256; }
// rows of the workspace for the narrow runs of a workgroup (a wave does not hold a head of 256)
__host__ __device__ constexpr int narrow_slots(int D) { return D == 256 ? 0 : kShareWaves * kNarrowRows; }

// units of a run, by kind: fewer leave more parts to join.  (8 sequences of 50 own tokens behind 1000:
// 15.2 us, with {8, 4} 18.4; 64 of 500 behind 8192, whose runs are longer than either: 41.)
constexpr uint32_t kLeast[2] = {5, 2};
// units that an item counts besides its steps: a run of either kind has 7 to 9 us of its own (plan, first
// loads, parts) beside 2 to 2.7 us a step, and an item inside it 2 to 4.  (2 and 4 instead: from 4 %
// quicker to 5 % slower over twelve shapes.)
__host__ __device__ __forceinline__ uint32_t fixed_units(int kind) { return kind == kNarrow ? 4u : 6u; }

// The items of `rows` rows (tokens times R) over `steps` steps
struct Kind {
  int kind;
  uint32_t tile, tiles, steps, units;  // rows of a tile; tiles; units of an item
};
template <int D>
__host__ __device__ __forceinline__ Kind kind_of(uint32_t rows, uint32_t steps) {
  Kind k;
  k.kind = D < 256 && rows <= (uint32_t)kNarrowRows ? kNarrow : kWide;
  k.tile = k.kind == kNarrow ? kNarrowRows : wide_rows(D);
  k.tiles = (rows + k.tile - 1) / k.tile;
  k.steps = steps;
  k.units = steps + fixed_units(k.kind);
  return k;
}

struct Axis {
  uint32_t units, per, runs;
  static __host__ __device__ __forceinline__ Axis cut(uint32_t units, uint32_t runs, uint32_t least) {
    const uint32_t even = (units + runs - 1) / runs, per = even > least ? even : least;
    return Axis{units, per, (units + per - 1) / per};
  }
};
struct SharePlan {
  Axis axis[2];
};
// The two axes, by `all` workgroups (two at least): as many take wide runs as those units ask for, the
// waves of the others narrow ones.
//
// A narrow unit of one wave takes about 5 / 4 of the time of a wide one of eight.  (Weighed by 1/2, 1,
// 5/4, 2: 402, 257, 234, 238 us at 256 sequences of 1500 own tokens behind 32768, 32 heads of 128.
// Every workgroup taking both kinds, half of them one first and half the other: 238 us there, but
// 53 us, not 41, at 64 sequences of 500 own tokens behind 8192, where each waits for its slowest wave.)
__host__ __device__ __forceinline__ SharePlan cut_axes(uint32_t narrow, uint32_t wide, uint32_t all) {
  const uint64_t weight = ((uint64_t)narrow * 5 + 4 * kShareWaves - 1) / (4 * kShareWaves);
  const uint32_t share = (uint32_t)((uint64_t)all * wide / (wide + weight + 1));
  const uint32_t some = share < 1 ? 1 : share < all - 1 ? share : all - 1;
  SharePlan p;
  p.axis[kWide] = Axis::cut(wide, narrow == 0 ? all : some, kLeast[kWide]);
  const uint32_t taken = p.axis[kWide].runs < all - 1 ? p.axis[kWide].runs : all - 1;
  p.axis[kNarrow] = Axis::cut(narrow, (all - taken) * kShareWaves, kLeast[kNarrow]);
  return p;
}

// step p of an item lies at its unit fixed + p: a run that begins at or before that and ends behind it
// takes the step.  The steps in front of unit x:
__host__ __device__ __forceinline__ uint32_t step_at(const Kind& k, uint32_t x) {
  const uint32_t f = fixed_units(k.kind), n = x <= f ? 0u : x - f;
  return n < k.steps ? n : k.steps;
}

// The parts of an item whose first unit is i0: its first run, how many, and the place of row `row` in a
// tile, marked by kind.
struct Parts {
  uint32_t run, count, at;
};
__host__ __device__ __forceinline__ Parts parts_of(const Kind& k, const SharePlan& p, uint32_t i0, uint32_t row) {
  const uint32_t per = k.kind == kNarrow ? p.axis[kNarrow].per : p.axis[kWide].per, first = i0 + fixed_units(k.kind);
  const uint32_t run = first / per;
  return Parts{run, (first + k.steps - 1) / per - run + 1, row % k.tile | (uint32_t)k.kind << 15};
}

// Rows of the workspace: two for every output row (of its own tokens' item and the shared ones', where
// a run begins the item), and a tile for every run, which begins inside no other item.
__host__ __device__ __forceinline__ int64_t first_slot(int64_t keys, int64_t key, bool of_group) { return (of_group ? keys : 0) + key; }
template <int D>
__host__ __device__ __forceinline__ int64_t run_slot(int64_t keys, uint32_t all, int kind, uint32_t run, uint32_t row) {
  const int64_t narrow = 2 * keys, wide = narrow + (int64_t)all * narrow_slots(D);
  return row + (kind == kNarrow ? narrow + (int64_t)run * kNarrowRows : wide + (int64_t)run * wide_rows(D));
}
__host__ __device__ __forceinline__ int64_t share_slots(int64_t keys, uint32_t all, int D) {
  return 2 * keys + (int64_t)all * (narrow_slots(D) + wide_rows(D));
}

}  // namespace wq
