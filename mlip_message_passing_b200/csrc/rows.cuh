// Device helpers of the feature-row operators: 16-byte vectors of a row, the place of a column in
// the irreps layout, and the counter-based dropout decisions.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "features.h"

namespace e3b {

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) RowVec {
  T v[VEC];
};

template <typename T, int VEC>
__device__ __forceinline__ RowVec<T, VEC> load_row(const T* p) {
  return *reinterpret_cast<const RowVec<T, VEC>*>(p);
}
template <typename T, int VEC>
__device__ __forceinline__ void store_row(T* p, const RowVec<T, VEC>& v) {
  *reinterpret_cast<RowVec<T, VEC>*>(p) = v;
}

__host__ __device__ __forceinline__ uint32_t fast_div(uint32_t x, uint32_t recip) {
#ifdef __CUDA_ARCH__
  return recip ? __umulhi(x, recip) : x;
#else
  return recip ? uint32_t((uint64_t(x) * recip) >> 32) : x;
#endif
}

// The same for rows that are not needed again: they leave L2 first.
template <typename T, int VEC>
__device__ __forceinline__ void store_row_last(T* p, const RowVec<T, VEC>& v) {
  if constexpr (sizeof(v) == 16) {
    int4 q;
    memcpy(&q, &v, 16);
    __stcs(reinterpret_cast<int4*>(p), q);
  } else if constexpr (sizeof(v) == 8) {
    int2 q;
    memcpy(&q, &v, 8);
    __stcs(reinterpret_cast<int2*>(p), q);
  } else {
    static_assert(VEC == 1, "one vector or one element");
    __stcs(p, v.v[0]);
  }
}

// Block of a column.
__host__ __device__ __forceinline__ int block_of(const RowLayout& L, int col) {
  int b = 0;
  while (b + 1 < L.n_blocks && col >= L.blk[b + 1].col0) ++b;
  return b;
}
// Group index (over all blocks) of a column.
__host__ __device__ __forceinline__ int group_of(const RowLayout& L, int col) {
  const int b = block_of(L, col);
  return b * L.groups + int(fast_div(uint32_t(col - L.blk[b].col0), L.blk[b].div_group));
}

// Philox4x32-10 (Salmon et al., "Parallel random numbers: as easy as 1, 2, 3"): ten rounds of two
// 32 x 32 -> 64 bit products on the counter, the key raised by a constant each round.
__device__ __forceinline__ uint4 philox10(uint4 c, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p0 = uint64_t(0xD2511F53u) * c.x, p1 = uint64_t(0xCD9E8D57u) * c.z;
    c = make_uint4(uint32_t(p1 >> 32) ^ c.y ^ k0, uint32_t(p1), uint32_t(p0 >> 32) ^ c.w ^ k1, uint32_t(p0));
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return c;
}

// The dropout of one thread's vector column: its quad of channels and the word of each element.
// With 16-byte vectors all elements of a vector lie in one quad (a quad of channels spans
// 4 (2l+1) columns, counted from the block's start, which is a vector boundary).
template <int VEC>
struct DropCol {
  uint32_t quad, block;
  uint32_t bytes;  // byte i: 1 << (word of element i)
  uint32_t k0, k1, offset, thr, row0;

  __device__ __forceinline__ void init(const RowLayout& L, const DropArgs& a, int col) {
    const int b = block_of(L, col);
    const uint32_t o = uint32_t(col - L.blk[b].col0);
    block = uint32_t(b);
    quad = fast_div(o, L.blk[b].div_d) >> 2;
    bytes = 0;
#pragma unroll
    for (int i = 0; i < VEC; ++i) bytes |= 1u << ((fast_div(o + i, L.blk[b].div_d) & 3u) + 8 * i);
    k0 = a.k0;
    k1 = a.k1;
    offset = a.offset;
    if (a.state != nullptr) {
      const uint64_t s = uint64_t(a.state[0]);
      k0 = uint32_t(s);
      k1 = uint32_t(s >> 32);
      offset = uint32_t(a.state[1]);
    }
    thr = a.thr;
    row0 = a.row0;
  }
  // byte i is not 0: element i of this column's vector in `row` stays
  __device__ __forceinline__ uint32_t keep(int64_t row) const {
    const uint4 w = philox10(make_uint4(quad, row0 + uint32_t(row), block, offset), k0, k1);
    const uint32_t m = uint32_t(w.x >= thr) | uint32_t(w.y >= thr) << 1 | uint32_t(w.z >= thr) << 2 |
                       uint32_t(w.w >= thr) << 3;
    return (m * 0x01010101u) & bytes;
  }
  static __device__ __forceinline__ bool kept(uint32_t k, int i) { return (k & (0xFFu << (8 * i))) != 0; }
};

}  // namespace e3b
