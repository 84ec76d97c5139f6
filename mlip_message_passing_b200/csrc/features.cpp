// Feature layouts (host): the irreps string of a row, its groups, and the arguments of a dropout.
#include "features.h"

#include <cuda_runtime.h>

#include <cmath>
#include <memory>
#include <new>
#include <string>
#include <vector>

#include "internal.h"

using namespace e3b;

extern "C" e3_status e3_features_create(const char* irreps, int32_t groups, e3_dtype dtype, e3_features** out) {
  clear_error();
  if (out == nullptr) return fail(E3_ERR_INVALID_ARG, "features is NULL");
  *out = nullptr;
  if (dtype != E3_F32 && dtype != E3_F64) return fail(E3_ERR_INVALID_ARG, "bad dtype");
  if (groups < 1) return fail(E3_ERR_INVALID_ARG, "groups must be positive, got %d", int(groups));
  std::vector<IrrepT> ir;
  std::string why;
  if (!parse_irreps(irreps, &ir, &why)) return fail(E3_ERR_IRREPS_PARSE, "irreps: %s", why.c_str());
  if (ir.size() > size_t(FR_MAXB)) return fail(E3_ERR_UNSUPPORTED, "more than %d irrep blocks", FR_MAXB);
  std::unique_ptr<e3_features> f(new (std::nothrow) e3_features);
  if (!f) return fail(E3_ERR_INVALID_ARG, "out of host memory");
  int64_t col = 0;
  RowLayout& L = f->lay;
  L.n_blocks = int32_t(ir.size());
  L.groups = groups;
  L.div_groups = reciprocal(uint32_t(groups));
  for (size_t i = 0; i < ir.size(); ++i) {
    const IrrepT& t = ir[i];
    if (t.l > FR_MAX_L) return fail(E3_ERR_UNSUPPORTED, "degree %d is above %d", t.l, FR_MAX_L);
    if (t.mul % groups != 0)
      return fail(E3_ERR_SHAPE, "multiplicity %d of block %d is not divisible into %d groups", t.mul, int(i), int(groups));
    const bool scalar = t.l == 0 && t.p > 0;
    RowBlock& b = L.blk[i];
    b.col0 = int32_t(col);
    b.mul = t.mul;
    b.d = 2 * t.l + 1;
    b.chan0 = L.n_channels;
    b.bias0 = scalar ? L.n_scalars : -1;
    col += int64_t(t.mul) * b.d;
    if (col > FR_MAX_DIM) return fail(E3_ERR_UNSUPPORTED, "rows of more than %lld columns", (long long)FR_MAX_DIM);
    b.group_cols = t.mul / groups * b.d;
    b.div_d = reciprocal(uint32_t(b.d));
    b.div_group = reciprocal(uint32_t(b.group_cols));
    L.n_channels += t.mul;
    if (scalar) L.n_scalars += t.mul;
  }
  L.dim = int32_t(col);
  f->dtype = dtype;
  make_tiles(f.get());
  // without a device the layout can still be described (host checks); the calls refuse it
  if (cudaGetDevice(&f->device) != cudaSuccess) {
    cudaGetLastError();
    f->device = -1;
  }
  *out = f.release();
  return E3_OK;
}

extern "C" e3_status e3_features_destroy(e3_features* f) {
  delete f;
  return E3_OK;
}

extern "C" e3_status e3_features_info(const e3_features* f, int64_t* dim, int64_t* n_channels, int64_t* n_scalars,
                                      int64_t* n_groups) {
  clear_error();
  if (f == nullptr) return fail(E3_ERR_INVALID_ARG, "features is NULL");
  if (dim) *dim = f->lay.dim;
  if (n_channels) *n_channels = f->lay.n_channels;
  if (n_scalars) *n_scalars = f->lay.n_scalars;
  if (n_groups) *n_groups = f->lay.n_groups();
  return E3_OK;
}

e3_status e3b::check_features_device(const e3_features* f) {
  if (f == nullptr) return fail(E3_ERR_INVALID_ARG, "features is NULL");
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return fail(E3_ERR_CUDA, "cudaGetDevice failed");
  if (dev != f->device)
    return fail(E3_ERR_INVALID_ARG, "features belong to device %d but device %d is current", f->device, dev);
  return E3_OK;
}

e3_status e3b::drop_args(const e3_dropout_spec* drop, int64_t N, DropArgs* out, bool* on) {
  *out = DropArgs{};
  *on = false;
  if (drop == nullptr) return E3_OK;
  if (!(drop->p >= 0.0 && drop->p < 1.0)) return fail(E3_ERR_INVALID_ARG, "dropout p = %g is not in [0, 1)", drop->p);
  if (drop->row0 < 0 || drop->row0 > (int64_t(1) << 32) - N)
    return fail(E3_ERR_SHAPE, "dropout rows %lld .. + %lld pass 2^32", (long long)drop->row0, (long long)N);
  if (drop->state == nullptr && drop->offset >= (uint64_t(1) << 32))
    return fail(E3_ERR_INVALID_ARG, "dropout offset passes 2^32");
  if (reinterpret_cast<uintptr_t>(drop->state) & 7u) return fail(E3_ERR_INVALID_ARG, "state is not 8-byte aligned");
  out->state = drop->state;
  out->k0 = uint32_t(drop->seed);
  out->k1 = uint32_t(drop->seed >> 32);
  out->offset = uint32_t(drop->offset);
  out->thr = uint32_t(std::floor(drop->p * 4294967296.0));
  out->row0 = uint32_t(drop->row0);
  out->scale = 1.0 / (1.0 - drop->p);
  *on = drop->p > 0.0;
  return E3_OK;
}
