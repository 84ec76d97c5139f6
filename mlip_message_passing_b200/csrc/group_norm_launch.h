// Launchers of the group norm, one translation unit per form.
#pragma once

#include <atomic>

#include "group_norm.cuh"

namespace e3b {

static_assert(sizeof(NormArgs) <= 4096, "kernel arguments");

// Threads of a CTA of the local kernel when every segment is one row: rows are wide, batches short (256 threads
// leave a third of them idle on 2048 columns with one group per block).
constexpr int GN_ROW_THREADS = 512;
// (Segment, group) pairs of a batch of one-row segments at most (twice as many for floats, whose tiles may have 512
// groups of one column): 8 segments a thread of one-element vectors of doubles take 160 KB for rows and sums, and 24
// bytes a pair for the forward's coefficients.
constexpr int GN_ROW_ITEMS = 2048;

struct GnConfig {
  bool local = false;
  bool one_row = false;   // local: no segment has more than one row
  const TileSet* tiles = nullptr;
  size_t ws_bytes = 0;
};
// Rows of a segment that a thread of the local kernel holds, and segments per thread when every segment is
// one row: what leaves two or three CTAs to an SM (per thread and row 16, 32, 48 bytes of shared memory).
// 8, 4 and 2 rows with a second set of slots were slower: 142 us instead of 97 on one-row segments (forward),
// 113 instead of 92 on molecules (forward and backward).
__host__ __device__ constexpr int gn_reg_rows(int op) { return op == GN_FWD ? 16 : op == GN_BWD ? 8 : 4; }
__host__ __device__ constexpr int gn_reg_segments(int op, int vec) {
  return vec == 1 ? (op == GN_DBL ? 2 : 8) : op == GN_DBL ? 1 : 4;
}

// Chunks and workspace of the grid kernel on `ctas` resident CTAs; returns the bytes needed.
size_t gn_grid_layout(NormArgs* a, int op, int64_t ctas);
// Workspace of the local kernel on `ctas` CTAs: their column sums, then (clusters) a counter by tile.
size_t gn_column_bytes(const NormArgs& a, int op, int vec, int64_t ctas);
size_t gn_local_layout(const NormArgs& a, int op, int vec, int64_t ctas);
// Shares out `room` resident CTAs (clusters) among the tiles of the local kernel, `batches` of segments each.
void gn_share(NormArgs* a, int op, const TileSet& t, int64_t batches, int64_t room);
// Most CTAs that any kernel here keeps resident on an SM (sizes workspaces).
constexpr int GN_MAX_RESIDENT = 8;

e3_status gn_launch_fwd(NormArgs& a, const GnConfig& c, bool f64, int vec, bool drop, void* ws, cudaStream_t s);
e3_status gn_launch_bwd(NormArgs& a, const GnConfig& c, bool f64, int vec, bool drop, void* ws, cudaStream_t s);
e3_status gn_launch_dbl(NormArgs& a, const GnConfig& c, bool f64, int vec, bool drop, void* ws, cudaStream_t s);

// CTAs of `kernel` that are resident together on the current device (found once per device).
template <typename K>
int gn_resident(K kernel, size_t smem, std::atomic<int64_t>* cache, bool cluster, int threads = GN_THREADS) {
  int dev = 0;
  cudaGetDevice(&dev);
  // the cache holds the answer for the last size asked for; layouts that take turns ask again at each call
  const int64_t hit = dev < 64 ? cache[dev].load(std::memory_order_relaxed) : 0;
  int n = hit >> 32 == int64_t(smem) ? int(hit & 0xFFFFFFFF) : 0;
  if (n == 0) {
    int per = 0;
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024) != cudaSuccess)
      return 0;
    if (cluster && cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
      return 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, smem) != cudaSuccess) return 0;
    n = std::min(per, GN_MAX_RESIDENT) * sm_count();
    if (dev < 64) cache[dev].store(int64_t(smem) << 32 | n, std::memory_order_relaxed);
  }
  return n;
}

template <typename K>
e3_status gn_start(K kernel, const NormArgs& a, dim3 grid, size_t smem, bool meet, int cluster, cudaStream_t s,
                   int threads = GN_THREADS) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  unsigned n = 0;
  if (meet) {
    attr[n].id = cudaLaunchAttributeCooperative;
    attr[n++].val.cooperative = 1;
  }
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = unsigned(cluster);
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, a);
  if (err != cudaSuccess) return fail(E3_ERR_CUDA, "group norm launch failed: %s", cudaGetErrorString(err));
  return E3_OK;
}

template <typename T, int VEC, int OP, bool DROP, int R, int M, bool CL, int NT = GN_THREADS>
e3_status gn_run_local(NormArgs& a, const GnConfig& c, void* ws, cudaStream_t s) {
  static std::atomic<int64_t> cache[64];
  const size_t smem = GnLocal<T, VEC, OP, R, M, CL, NT>::smem(a);
  auto kernel = gn_local_kernel<T, VEC, OP, DROP, R, M, CL, NT>;
  const int q = gn_resident(kernel, smem, cache, CL, NT);
  int64_t room = q / a.cs;  // CTAs, or clusters, that are resident together
  if (CL) {
    static std::atomic<int64_t> clusters[64][5];  // like gn_resident's cache
    int dev = 0, size = 0;
    cudaGetDevice(&dev);
    while ((1 << size) < a.cs) ++size;
    const int64_t hit = dev < 64 ? clusters[dev][size].load(std::memory_order_relaxed) : 0;
    int n = hit >> 32 == int64_t(smem) ? int(hit & 0xFFFFFFFF) : 0;
    if (n == 0) {
      cudaLaunchConfig_t cfg{};
      cfg.gridDim = dim3(unsigned(a.cs));
      cfg.blockDim = dim3(GN_THREADS);
      cfg.dynamicSmemBytes = smem;
      cudaLaunchAttribute attr;
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = unsigned(a.cs);
      attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      if (q == 0 || cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) n = 0;
      if (dev < 64) clusters[dev][size].store(int64_t(smem) << 32 | n, std::memory_order_relaxed);
    }
    room = std::min<int64_t>(room, n);
    // no cluster waits for another
    if (n > 0) room = std::max<int64_t>(room, a.n_tiles);
  }
  if (room < a.n_tiles) return fail(E3_ERR_CUDA, "group norm: no room for the kernel on this device");
  const int64_t batch = int64_t(a.j) * M;
  gn_share(&a, OP, *c.tiles, (a.B + batch - 1) / batch, room);
  const int64_t ctas = a.start[a.n_tiles];
  if (gn_local_layout(a, OP, VEC, ctas) > c.ws_bytes) return fail(E3_ERR_SHAPE, "group norm: workspace too small");
  const bool columns = OP != GN_FWD && (a.gw != nullptr || a.gb != nullptr);
  a.colpart = columns ? static_cast<double*>(ws) : nullptr;
  a.meet = columns && !(CL && ctas == int64_t(a.n_tiles) * a.cs);
  if (CL && a.meet) {
    a.tickets = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + gn_column_bytes(a, OP, VEC, ctas));
    if (cudaMemsetAsync(a.tickets, 0, sizeof(int32_t) * size_t(a.n_tiles), s) != cudaSuccess)
      return fail(E3_ERR_CUDA, "group norm: zeroing the counters failed");
  }
  const dim3 grid = a.even ? dim3(unsigned(a.start[1]), unsigned(a.n_tiles)) : dim3(unsigned(ctas));
  return gn_start(kernel, a, grid, smem, !CL && a.meet, a.cs, s, NT);
}

template <typename T, int VEC, int OP, bool DROP>
e3_status gn_run(NormArgs& a, const GnConfig& c, void* ws, cudaStream_t s) {
  if (c.local) {
    if (c.one_row) return gn_run_local<T, VEC, OP, DROP, 1, gn_reg_segments(OP, VEC), false, GN_ROW_THREADS>(a, c, ws, s);
    if (a.cs > 1) return gn_run_local<T, VEC, OP, DROP, gn_reg_rows(OP), 1, true>(a, c, ws, s);
    return gn_run_local<T, VEC, OP, DROP, gn_reg_rows(OP), 1, false>(a, c, ws, s);
  }
  static std::atomic<int64_t> cache[64];
  constexpr size_t smem = GnGrid<T, VEC, OP>::smem;
  auto kernel = gn_grid_kernel<T, VEC, OP, DROP>;
  const int q = gn_resident(kernel, smem, cache, false);
  if (q < a.n_tiles) return fail(E3_ERR_CUDA, "group norm: no room for the kernel on this device");
  if (gn_grid_layout(&a, OP, q) > c.ws_bytes)
    return fail(E3_ERR_SHAPE, "group norm: workspace too small");
  char* base = static_cast<char*>(ws);
  a.part = base;
  a.tickets = reinterpret_cast<int32_t*>(base + reinterpret_cast<size_t>(a.tickets));
  a.coef = base + reinterpret_cast<size_t>(a.coef);
  const bool columns = OP != GN_FWD && (a.gw != nullptr || a.gb != nullptr);
  a.colpart = columns ? reinterpret_cast<double*>(base + reinterpret_cast<size_t>(a.colpart)) : nullptr;
  return gn_start(kernel, a, dim3(unsigned(a.chunks) * unsigned(a.n_tiles)), smem, true, 1, s);
}

template <int OP>
e3_status gn_launch(NormArgs& a, const GnConfig& c, bool f64, int vec, bool drop, void* ws, cudaStream_t s) {
#define GN_CASE(T, V) return drop ? gn_run<T, V, OP, true>(a, c, ws, s) : gn_run<T, V, OP, false>(a, c, ws, s)
  if (f64) {
    if (vec == 2) GN_CASE(double, 2);
    GN_CASE(double, 1);
  }
  if (vec == 4) GN_CASE(float, 4);
  if (vec == 2) GN_CASE(float, 2);
  GN_CASE(float, 1);
#undef GN_CASE
}

}  // namespace e3b
