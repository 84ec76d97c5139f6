// Layout of feature rows (irreps blocks in mul_ir order) as the row operators' kernels take it.
#pragma once

#include <cstdint>

#include "../../include/e3b.h"

namespace e3b {

constexpr int FR_MAXB = 32;             // irrep blocks at most
constexpr int FR_MAX_L = 500;            // degree of a block at most
constexpr int64_t FR_MAX_DIM = 1 << 20;  // columns of a row at most

struct RowBlock {
  int32_t col0;        // first column
  int32_t mul, d;      // channels, components (2 l + 1)
  int32_t group_cols;  // columns of one group: mul / groups * d
  int32_t chan0;       // index of its first channel among all channels
  int32_t bias0;       // index of its first channel among the even scalars, -1 for other irreps
};

struct RowLayout {
  int32_t n_blocks, groups, dim, n_channels, n_scalars;
  RowBlock blk[FR_MAXB];
  int32_t n_groups() const { return n_blocks * groups; }
};

// Dropout as the kernels take it: a channel stays when its word is >= thr.
struct DropArgs {
  const int64_t* state;  // device {seed, offset}, or NULL: the values below
  uint32_t k0, k1, offset;
  uint32_t thr;
  uint32_t row0;         // added to the row index in the counter
  double scale;          // 1 / (1 - p)
};

// Validate `drop` (NULL: no dropout) for N rows; *on tells whether anything is dropped.
e3_status drop_args(const e3_dropout_spec* drop, int64_t N, DropArgs* out, bool* on);
// f is not NULL and its device is current.
e3_status check_features_device(const e3_features* f);

}  // namespace e3b

struct e3_features {
  int device = 0;
  e3_dtype dtype = E3_F32;
  e3b::RowLayout lay{};
};
