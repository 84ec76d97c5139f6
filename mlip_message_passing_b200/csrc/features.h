// Layout of feature rows (irreps blocks in mul_ir order) as the row operators' kernels take it.
#pragma once

#include <cstdint>
#include <string>
#include <vector>

#include "../../include/e3b.h"

#if !defined(__CUDACC__) && !defined(__host__)
#define __host__
#define __device__
#endif

namespace e3b {

constexpr int FR_MAXB = 32;             // irrep blocks at most
constexpr int FR_MAX_L = 127;           // degree of a block at most
constexpr int64_t FR_MAX_DIM = 32768;   // columns of a row at most

// One term of an irreps string: multiplicity, degree, parity (+1 / -1).
struct IrrepT {
  int mul, l, p;
};
// Terms of an irreps string (host.cpp); false with the reason in *why when it is malformed.
bool parse_irreps(const char* s, std::vector<IrrepT>* out, std::string* why);

struct RowBlock {
  int32_t col0;        // first column
  int32_t mul, d;      // channels, components (2 l + 1)
  int32_t group_cols;  // columns of one group: mul / groups * d
  int32_t chan0;       // index of its first channel among all channels
  int32_t bias0;       // index of its first channel among the even scalars, -1 for other irreps
  uint32_t div_d, div_group;  // reciprocals of d and group_cols (fast_div)
};
// x / n = umulhi(x, reciprocal(n)) for 1 < n and x n < 2^32; 0 stands for n = 1.
inline uint32_t reciprocal(uint32_t n) { return n > 1 ? uint32_t(0xFFFFFFFFu / n) + 1u : 0u; }

struct RowLayout {
  int32_t n_blocks, groups, dim, n_channels, n_scalars;
  uint32_t div_groups;
  RowBlock blk[FR_MAXB];
  __host__ __device__ int32_t n_groups() const { return n_blocks * groups; }
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
// Tiles of the group norm (group_norm.cu), once per features.
void make_tiles(e3_features* f);
// f is not NULL and its device is current.
e3_status check_features_device(const e3_features* f);

// A cut of a row's vector columns into tiles of at most tx.
struct TileSet {
  int tx = 0, groups = 0;      // widest tile, most groups of a tile
  bool cut = false;            // some group lies in several tiles
  std::vector<int32_t> first;  // first vector column of each tile, then the end
  std::vector<int32_t> scalars;  // vector columns of even scalars in each tile
  int n() const { return int(first.size()) - 1; }
};

}  // namespace e3b

struct e3_features {
  int device = 0;
  e3_dtype dtype = E3_F32;
  e3b::RowLayout lay{};
  int vec = 1;                   // group norm: columns of a vector
  bool cluster_ok = false;       // group norm: the tiles for long segments suit clusters
  int wide = 0;                  // widest group in vectors
  // tiles for 2^i row lanes of a segment, for segments of one row, for clusters, for long segments
  e3b::TileSet local[10], rows, narrow, grid;
};
