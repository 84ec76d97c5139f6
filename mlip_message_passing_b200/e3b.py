"""Thin PyTorch binding of the C ABI in ``include/e3b.h`` (``libe3b.so``).

Every function here only checks and marshals arguments (device, dtype, shape, contiguity),
then calls the library on the current CUDA stream; all arithmetic runs in the library's CUDA
kernels.  If the shared library is missing this module fails to import: there is no CPU path.
"""

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libe3b.so")

E3_OK, E3_ERR_INVALID_ARG, E3_ERR_IRREPS_PARSE, E3_ERR_INSTRUCTION, E3_ERR_UNSUPPORTED, \
    E3_ERR_SHAPE, E3_ERR_INDEX, E3_ERR_CUDA, E3_ERR_TIMEOUT = range(9)
STATUS_NAMES = ["OK", "INVALID_ARG", "IRREPS_PARSE", "INSTRUCTION", "UNSUPPORTED", "SHAPE", "INDEX",
                "CUDA", "TIMEOUT"]
_DTYPES = {torch.float32: 0, torch.float64: 1}
_SH_NORMS = {"component": 0, "integral": 1, "norm": 2}
_ACTS = {None: 0, "silu": 1}

# every symbol include/e3b.h declares
SYMBOLS = [
    "e3_plan_create", "e3_plan_destroy", "e3_plan_info", "e3_plan_irreps_out", "e3_plan_paths",
    "e3_device_status", "e3_cg_dense", "e3_supported", "e3_tp_forward", "e3_tp_backward",
    "e3_spherical_harmonics", "e3_csr_workspace_size", "e3_csr_build", "e3_gather_rows",
    "e3_conv_forward", "e3_conv_backward", "e3_last_error", "e3_csr_build_static",
    "e3_backward_workspace_size", "e3_spherical_harmonics_backward", "e3_morton_workspace_size",
    "e3_morton_order", "e3_invert_permutation", "e3_remap_ids", "e3_conv_workspace_size",
    "e3_conv_topology_size", "e3_conv_topology_build", "e3_set_test_knobs", "e3_add_rows",
    "e3_conv_topology_build_ordered", "e3_radial_prep_size", "e3_radial_prepare", "e3_radial_weights",
    "e3_spherical_harmonics_double_backward", "e3_plan_status", "e3_features_create", "e3_features_destroy",
    "e3_features_info", "e3_dropout", "e3_group_norm_workspace_size", "e3_group_norm_forward",
    "e3_group_norm_backward", "e3_group_norm_double_backward",
]


class E3Error(RuntimeError):
    def __init__(self, status, message):
        self.status = status
        name = STATUS_NAMES[status] if 0 <= status < len(STATUS_NAMES) else str(status)
        super().__init__(f"e3b {name}: {message}")


class Instruction(ctypes.Structure):
    _fields_ = [("i_in1", ctypes.c_int32), ("i_in2", ctypes.c_int32), ("i_out", ctypes.c_int32),
                ("has_weight", ctypes.c_int32), ("path_weight", ctypes.c_double)]


class DropoutSpec(ctypes.Structure):
    _fields_ = [("p", ctypes.c_double), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64),
                ("state", ctypes.c_void_p), ("row0", ctypes.c_int64)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m mlip_message_passing_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64, D, VP = ctypes.c_char_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double, ctypes.c_void_p
    sig = {
        "e3_plan_create": [P, P, P, ctypes.POINTER(Instruction), I32, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                           ctypes.POINTER(VP)],
        "e3_plan_destroy": [VP],
        "e3_plan_info": [VP, ctypes.POINTER(I64), ctypes.POINTER(I64), ctypes.POINTER(I64), ctypes.POINTER(I64),
                         ctypes.POINTER(I32)],
        "e3_plan_irreps_out": [VP, ctypes.c_char_p, ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t)],
        "e3_plan_paths": [VP, ctypes.POINTER(I32), ctypes.POINTER(D)],
        "e3_device_status": [VP],
        "e3_plan_status": [VP, VP],
        "e3_cg_dense": [I32, I32, I32, ctypes.POINTER(D)],
        "e3_supported": [],
        "e3_tp_forward": [VP, I64, VP, VP, VP, VP, VP],
        "e3_tp_backward": [VP, I64, VP, VP, VP, VP, VP, VP, VP, VP, ctypes.c_size_t, VP],
        "e3_backward_workspace_size": [I64, ctypes.POINTER(ctypes.c_size_t)],
        "e3_spherical_harmonics": [I32, I64, VP, ctypes.c_int, ctypes.c_int, VP, VP],
        "e3_spherical_harmonics_backward": [I32, I64, VP, ctypes.c_int, VP, ctypes.c_int, VP, VP],
        "e3_spherical_harmonics_double_backward": [I32, I64, VP, ctypes.c_int, VP, VP, ctypes.c_int, VP, VP, VP],
        "e3_csr_workspace_size": [I64, I64, ctypes.POINTER(ctypes.c_size_t)],
        "e3_csr_build": [I64, I64, VP, VP, VP, VP, VP, VP, VP, ctypes.c_size_t, VP],
        "e3_csr_build_static": [I64, I64, VP, VP, VP, VP, VP, VP, VP],
        "e3_gather_rows": [I64, I64, I64, VP, VP, VP, VP],
        "e3_add_rows": [I64, I64, I64, ctypes.c_int, VP, VP, VP, VP],
        "e3_radial_prep_size": [I32, I32, ctypes.POINTER(ctypes.c_size_t)],
        "e3_radial_prepare": [I32, I32, VP, VP, ctypes.c_size_t, VP],
        "e3_radial_weights": [I64, VP, D, I32, I32, I32, VP, VP, I32, VP, VP],
        "e3_conv_forward": [VP, I64, I64, VP, VP, VP, VP, VP, ctypes.c_int, VP, D, VP, VP, VP, ctypes.c_size_t,
                            VP],
        "e3_conv_workspace_size": [VP, I64, I64, ctypes.POINTER(ctypes.c_size_t)],
        "e3_conv_topology_size": [I64, I64, ctypes.POINTER(ctypes.c_size_t)],
        "e3_conv_topology_build": [I64, I64, VP, VP, VP, ctypes.c_size_t, VP],
        "e3_conv_topology_build_ordered": [I64, I64, VP, VP, VP, VP, ctypes.c_size_t, VP],
        "e3_conv_backward": [VP, I64, I64, VP, VP, VP, VP, VP, VP, VP, VP, ctypes.c_int, VP, VP, D, VP, VP, VP,
                             VP, VP, ctypes.c_size_t, VP],
        "e3_morton_workspace_size": [I64, ctypes.POINTER(ctypes.c_size_t)],
        "e3_morton_order": [I64, VP, ctypes.c_int, ctypes.POINTER(D), ctypes.POINTER(D), VP, VP, ctypes.c_size_t,
                            VP],
        "e3_invert_permutation": [I64, VP, VP, VP],
        "e3_remap_ids": [I64, VP, I64, VP, VP, VP],
        "e3_set_test_knobs": [I64, I32],
        "e3_features_create": [P, I32, ctypes.c_int, ctypes.POINTER(VP)],
        "e3_features_destroy": [VP],
        "e3_features_info": [VP, ctypes.POINTER(I64), ctypes.POINTER(I64), ctypes.POINTER(I64), ctypes.POINTER(I64)],
        "e3_dropout": [VP, I64, VP, VP, ctypes.POINTER(DropoutSpec), VP, VP],
        "e3_group_norm_workspace_size": [VP, I64, I64, I64, ctypes.POINTER(ctypes.c_size_t)],
        "e3_group_norm_forward": [VP, I64, I64, VP, I64, VP, VP, VP, D, ctypes.c_int, ctypes.POINTER(DropoutSpec), VP,
                                  VP, VP, ctypes.c_size_t, VP],
        "e3_group_norm_backward": [VP, I64, I64, VP, I64, VP, VP, VP, VP, ctypes.c_int, ctypes.POINTER(DropoutSpec),
                                   VP, VP, VP, VP, VP, ctypes.c_size_t, VP],
        "e3_group_norm_double_backward": [VP, I64, I64, VP, I64, VP, VP, VP, VP, ctypes.c_int,
                                          ctypes.POINTER(DropoutSpec), VP, VP, VP, VP, VP, VP, VP, VP, VP,
                                          ctypes.c_size_t, VP],
        "e3_last_error": [],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_char_p if name in ("e3_last_error", "e3_supported") else ctypes.c_int
    return lib


lib = _load()


def _check(status):
    if status != E3_OK:
        raise E3Error(status, lib.e3_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _need(t, name, dtype, shape, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def supported():
    """Degree triples (Lx, Ly, Lo) with compiled kernels."""
    return [tuple(int(v) for v in s.split(",")) for s in lib.e3_supported().decode().split()]


def cg_dense(l1, l2, l3):
    """The library's real CG tensor (ladder construction) as a float64 CPU tensor."""
    out = (ctypes.c_double * ((2 * l1 + 1) * (2 * l2 + 1) * (2 * l3 + 1)))()
    _check(lib.e3_cg_dense(l1, l2, l3, out))
    return torch.tensor(list(out), dtype=torch.float64).reshape(2 * l1 + 1, 2 * l2 + 1, 2 * l3 + 1)


def device_status():
    """Synchronise the current stream; raise E3Error if a kernel recorded an error."""
    _check(lib.e3_device_status(_stream()))


class Plan:
    """A tensor-product plan (irreps, instructions, dtype) bound to the current CUDA device.

    ``irreps_out`` with ``instructions=None`` filters the enumerated output irreps; pass
    ``lmax_out`` instead to keep every output irrep of degree <= lmax_out.
    ``instructions``: list of (i_in1, i_in2, i_out[, path_weight]) tuples.
    """

    def __init__(self, irreps_in1, irreps_in2, irreps_out=None, instructions=None, lmax_out=None,
                 dtype=torch.float32, mode="uvu", shared_weights=False):
        if lmax_out is not None:
            if irreps_out is not None or instructions is not None:
                raise ValueError("give lmax_out or irreps_out/instructions, not both")
            irreps_out = "+".join(f"1x{l}{p}" for l in range(lmax_out + 1) for p in "eo")
        modes = {"uvu": 0, "uvw": 1, "uuu": 2, "uuw": 3}
        if mode not in modes:
            raise ValueError(f"unknown mode {mode!r}")
        if dtype not in _DTYPES:
            raise ValueError("dtype must be torch.float32 or torch.float64")
        n = 0
        arr = None
        if instructions is not None:
            n = len(instructions)
            arr = (Instruction * n)()
            for i, ins in enumerate(instructions):
                pw = float(ins[3]) if len(ins) > 3 else -1.0
                arr[i] = Instruction(int(ins[0]), int(ins[1]), int(ins[2]), 1, pw)
        handle = ctypes.c_void_p()
        self._handle = None
        _check(lib.e3_plan_create(irreps_in1.encode(), irreps_in2.encode(),
                                  None if irreps_out is None else irreps_out.encode(), arr, n, modes[mode],
                                  _DTYPES[dtype], 1 if shared_weights else 0, ctypes.byref(handle)))
        self._handle = handle
        self.dtype = dtype
        self.shared_weights = shared_weights
        self.device = torch.device("cuda", torch.cuda.current_device())
        d1, d2, do, wn = (ctypes.c_int64() for _ in range(4))
        npth = ctypes.c_int32()
        _check(lib.e3_plan_info(handle, ctypes.byref(d1), ctypes.byref(d2), ctypes.byref(do), ctypes.byref(wn),
                                ctypes.byref(npth)))
        self.dim_in1, self.dim_in2, self.dim_out = d1.value, d2.value, do.value
        self.weight_numel, self.n_paths = wn.value, npth.value
        need = ctypes.c_size_t()
        _check(lib.e3_plan_irreps_out(handle, None, 0, ctypes.byref(need)))
        buf = ctypes.create_string_buffer(need.value)
        _check(lib.e3_plan_irreps_out(handle, buf, need.value, None))
        self.irreps_out = buf.value.decode()
        lls = (ctypes.c_int32 * (3 * self.n_paths))()
        al = (ctypes.c_double * self.n_paths)()
        _check(lib.e3_plan_paths(handle, lls, al))
        self.paths = [tuple(lls[3 * p:3 * p + 3]) for p in range(self.n_paths)]
        self.alphas = list(al)
        self.irreps_in1, self.irreps_in2 = irreps_in1, irreps_in2

    def __del__(self):
        if getattr(self, "_handle", None) and lib is not None:
            try:
                lib.e3_plan_destroy(self._handle)
            except Exception:  # interpreter shutdown
                pass
            self._handle = None

    @property
    def handle(self):
        return self._handle

    def status(self):
        """Synchronise the current stream; raise E3Error if a kernel of a call made with this plan
        recorded an error since the last read (e3_plan_status)."""
        _check(lib.e3_plan_status(self._handle, _stream()))

    def _w_shape(self, rows):
        return (self.weight_numel,) if self.shared_weights else (rows, self.weight_numel)


def tp_forward(plan, x, y, w, out=None):
    """out[b] = TP(x[b], y[b], w[b]) (e3_tp_forward)."""
    B = x.shape[0]
    dev, dt = plan.device, plan.dtype
    _need(x, "x", dt, (B, plan.dim_in1), dev)
    _need(y, "y", dt, (B, plan.dim_in2), dev)
    _need(w, "w", dt, plan._w_shape(B), dev)
    if out is None:
        out = torch.empty((B, plan.dim_out), dtype=dt, device=dev)
    _need(out, "out", dt, (B, plan.dim_out), dev)
    _check(lib.e3_tp_forward(plan.handle, B, _ptr(x), _ptr(y), _ptr(w), _ptr(out), _stream()))
    return out


def tp_backward(plan, x, y, w, grad_out, need_x=True, need_y=True, need_w=True):
    """(grad_x, grad_y, grad_w) of <grad_out, TP(x, y, w)> (e3_tp_backward); skipped ones are None."""
    B = x.shape[0]
    dev, dt = plan.device, plan.dtype
    _need(x, "x", dt, (B, plan.dim_in1), dev)
    _need(y, "y", dt, (B, plan.dim_in2), dev)
    _need(w, "w", dt, plan._w_shape(B), dev)
    _need(grad_out, "grad_out", dt, (B, plan.dim_out), dev)
    gx = torch.empty_like(x) if need_x else None
    gy = torch.empty_like(y) if need_y else None
    gw = torch.empty_like(w) if need_w else None
    ws = backward_workspace(B, dev)
    _check(lib.e3_tp_backward(plan.handle, B, _ptr(x), _ptr(y), _ptr(w), _ptr(grad_out), _ptr(gx), _ptr(gy),
                              _ptr(gw), _ptr(ws), ws.numel(), _stream()))
    return gx, gy, gw


def conv_workspace(plan, n_nodes, n_edges, device):
    """Device workspace for e3_conv_forward / e3_conv_backward, from torch's allocator."""
    nbytes = ctypes.c_size_t()
    _check(lib.e3_conv_workspace_size(plan.handle, n_nodes, n_edges, ctypes.byref(nbytes)))
    return torch.empty(nbytes.value, dtype=torch.uint8, device=device)


def backward_workspace(n, device):
    """Device workspace for e3_tp_backward (n = B) / e3_conv_backward (n = N), from torch's allocator."""
    nbytes = ctypes.c_size_t()
    _check(lib.e3_backward_workspace_size(n, ctypes.byref(nbytes)))
    return torch.empty(nbytes.value, dtype=torch.uint8, device=device)


def spherical_harmonics(lmax, vec, sh_norm="component", out=None):
    """[n, (lmax+1)^2] real harmonics of vec [n, 3] (e3_spherical_harmonics)."""
    if vec.dtype not in _DTYPES:
        raise ValueError("vec must be float32 or float64")
    n = vec.shape[0]
    _need(vec, "vec", vec.dtype, (n, 3), vec.device)
    if out is None:
        out = torch.empty((n, (lmax + 1) ** 2), dtype=vec.dtype, device=vec.device)
    _need(out, "out", vec.dtype, (n, (lmax + 1) ** 2), vec.device)
    _check(lib.e3_spherical_harmonics(lmax, n, _ptr(vec), _SH_NORMS[sh_norm], _DTYPES[vec.dtype], _ptr(out),
                                      _stream()))
    return out


def spherical_harmonics_backward(lmax, vec, grad_y, sh_norm="component", out=None):
    """[n, 3] gradient of sum(grad_y * Y(vec)) with respect to vec (e3_spherical_harmonics_backward)."""
    if vec.dtype not in _DTYPES:
        raise ValueError("vec must be float32 or float64")
    n = vec.shape[0]
    _need(vec, "vec", vec.dtype, (n, 3), vec.device)
    _need(grad_y, "grad_y", vec.dtype, (n, (lmax + 1) ** 2), vec.device)
    if out is None:
        out = torch.empty((n, 3), dtype=vec.dtype, device=vec.device)
    _need(out, "out", vec.dtype, (n, 3), vec.device)
    _check(lib.e3_spherical_harmonics_backward(lmax, n, _ptr(vec), _SH_NORMS[sh_norm], _ptr(grad_y),
                                               _DTYPES[vec.dtype], _ptr(out), _stream()))
    return out


def spherical_harmonics_double_backward(lmax, vec, grad_y, u, sh_norm="component"):
    """(d_grad_y, d_vec): the backward of grad_vec = J(vec)^T grad_y for upstream u
    (e3_spherical_harmonics_double_backward)."""
    n = vec.shape[0]
    for t_, nm, sh_ in ((vec, "vec", (n, 3)), (grad_y, "grad_y", (n, (lmax + 1) ** 2)), (u, "u", (n, 3))):
        _need(t_, nm, vec.dtype, sh_, vec.device)
    d_gy = torch.empty((n, (lmax + 1) ** 2), dtype=vec.dtype, device=vec.device)
    d_vec = torch.empty((n, 3), dtype=vec.dtype, device=vec.device)
    _check(lib.e3_spherical_harmonics_double_backward(lmax, n, _ptr(vec), _SH_NORMS[sh_norm], _ptr(grad_y), _ptr(u),
                                                      _DTYPES[vec.dtype], _ptr(d_gy), _ptr(d_vec), _stream()))
    return d_gy, d_vec


class _ShFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, vec, lmax, sh_norm):
        ctx.lmax, ctx.sh_norm = lmax, sh_norm
        ctx.save_for_backward(vec)
        return spherical_harmonics(lmax, vec, sh_norm)

    @staticmethod
    def backward(ctx, g):
        (vec,) = ctx.saved_tensors
        return _ShBwdFn.apply(vec, g.contiguous(), ctx.lmax, ctx.sh_norm), None, None


class _ShBwdFn(torch.autograd.Function):
    """grad_vec = J(vec)^T grad_y as a differentiable function of (vec, grad_y)."""

    @staticmethod
    def forward(ctx, vec, gy, lmax, sh_norm):
        ctx.lmax, ctx.sh_norm = lmax, sh_norm
        ctx.save_for_backward(vec, gy)
        return spherical_harmonics_backward(lmax, vec, gy, sh_norm)

    @staticmethod
    def backward(ctx, u):
        vec, gy = ctx.saved_tensors
        d_gy, d_vec = spherical_harmonics_double_backward(ctx.lmax, vec, gy, u.contiguous(), ctx.sh_norm)
        return d_vec, d_gy, None, None


def sh(lmax, vec, sh_norm="component"):
    """Twice-differentiable real harmonics of vec [n, 3]."""
    return _ShFn.apply(vec, lmax, sh_norm)


def morton_order(pos, lo, extent):
    """int32 [N] node order along the Morton curve of pos [N, 3] inside the box [lo, lo + extent)
    (e3_morton_order): perm[i] is the id of the i-th node on the curve."""
    if pos.dtype not in _DTYPES:
        raise ValueError("pos must be float32 or float64")
    N = pos.shape[0]
    _need(pos, "pos", pos.dtype, (N, 3), pos.device)
    nbytes = ctypes.c_size_t()
    _check(lib.e3_morton_workspace_size(N, ctypes.byref(nbytes)))
    ws = torch.empty(nbytes.value, dtype=torch.uint8, device=pos.device)
    perm = torch.empty(N, dtype=torch.int32, device=pos.device)
    lo3, ext3 = (ctypes.c_double * 3)(*map(float, lo)), (ctypes.c_double * 3)(*map(float, extent))
    _check(lib.e3_morton_order(N, _ptr(pos), _DTYPES[pos.dtype], lo3, ext3, _ptr(perm), _ptr(ws), ws.numel(),
                               _stream()))
    return perm


def invert_permutation(perm):
    """inv with inv[perm[i]] = i (e3_invert_permutation)."""
    _need(perm, "perm", torch.int32, (perm.shape[0],), perm.device)
    inv = torch.empty_like(perm)
    _check(lib.e3_invert_permutation(perm.shape[0], _ptr(perm), _ptr(inv), _stream()))
    return inv


def remap_ids(ids, mapping):
    """mapping[ids] for int32 tensors (e3_remap_ids)."""
    _need(ids, "ids", torch.int32, (ids.shape[0],), ids.device)
    _need(mapping, "mapping", torch.int32, (mapping.shape[0],), ids.device)
    out = torch.empty_like(ids)
    _check(lib.e3_remap_ids(ids.shape[0], _ptr(ids), mapping.shape[0], _ptr(mapping), _ptr(out), _stream()))
    return out


def reorder_graph(pos, lo, extent, src, dst):
    """Morton renumbering of a graph: (perm, inv, src', dst') with src' = inv[src], dst' = inv[dst].
    Node rows of the new numbering are rows[perm] (gather_rows); results map back with rows[inv]."""
    perm = morton_order(pos, lo, extent)
    inv = invert_permutation(perm)
    return perm, inv, remap_ids(src, inv), remap_ids(dst, inv)


def csr_build(n_nodes, src, dst):
    """(perm_dst, row_ptr_dst, perm_src, row_ptr_src) of an int32 edge list (e3_csr_build)."""
    E = src.shape[0]
    dev = src.device
    _need(src, "src", torch.int32, (E,), dev)
    _need(dst, "dst", torch.int32, (E,), dev)
    nbytes = ctypes.c_size_t()
    _check(lib.e3_csr_workspace_size(n_nodes, E, ctypes.byref(nbytes)))
    ws = torch.empty((nbytes.value + 255) // 4 + 64, dtype=torch.int32, device=dev)
    off = (-ws.data_ptr()) % 256 // 4
    wsv = ws[off:]
    perm_dst = torch.empty(E, dtype=torch.int32, device=dev)
    perm_src = torch.empty(E, dtype=torch.int32, device=dev)
    rp_dst = torch.empty(n_nodes + 1, dtype=torch.int32, device=dev)
    rp_src = torch.empty(n_nodes + 1, dtype=torch.int32, device=dev)
    _check(lib.e3_csr_build(n_nodes, E, _ptr(src), _ptr(dst), _ptr(perm_dst), _ptr(rp_dst), _ptr(perm_src),
                            _ptr(rp_src), _ptr(wsv), nbytes.value, _stream()))
    return perm_dst, rp_dst, perm_src, rp_src


def gather_rows(perm, t, out=None):
    """out[i] = t[perm[i]] for a contiguous tensor t (e3_gather_rows)."""
    n = perm.shape[0]
    _need(perm, "perm", torch.int32, (n,), t.device)
    if not t.is_contiguous():
        raise ValueError("t must be contiguous")
    if out is None:
        out = torch.empty((n,) + tuple(t.shape[1:]), dtype=t.dtype, device=t.device)
    row_bytes = t.element_size() * (t[0].numel() if t.dim() > 1 else 1)
    _check(lib.e3_gather_rows(n, t.shape[0], row_bytes, _ptr(perm), _ptr(t), _ptr(out), _stream()))
    return out


def add_rows_(out, idx, t):
    """out[idx[i]] += t[i] for distinct int32 indices (e3_add_rows); returns out."""
    n = idx.shape[0]
    _need(idx, "idx", torch.int32, (n,), out.device)
    if out.dtype not in _DTYPES:
        raise ValueError("out must be float32 or float64")
    _need(t, "t", out.dtype, (n,) + tuple(out.shape[1:]), out.device)
    if not out.is_contiguous():
        raise ValueError("out must be contiguous")
    row = out[0].numel() if out.dim() > 1 else 1
    _check(lib.e3_add_rows(n, out.shape[0], row, _DTYPES[out.dtype], _ptr(idx), _ptr(t), _ptr(out), _stream()))
    return out


class Radial:
    """The radial network w = SiLU(f(|v|) W1) W2 (Bessel basis x polynomial envelope) with W2 laid
    out once for the tensor cores (e3_radial_prepare); call ``weights(edge_vec)`` per step."""

    def __init__(self, w1, w2, cutoff, envelope_p=6):
        if w1.dtype != torch.float32 or w2.dtype != torch.float32:
            raise ValueError("the radial network runs in float32")
        if not (w1.is_contiguous() and w2.is_contiguous()) or w1.device != w2.device or w1.device.type != "cuda":
            raise ValueError("w1, w2 must be contiguous CUDA tensors on one device")
        self.n_basis, self.hidden = w1.shape
        if w2.shape[0] != self.hidden:
            raise ValueError("w2 must be [hidden, n_out]")
        self.n_out = w2.shape[1]
        self.cutoff, self.p, self.w1 = float(cutoff), int(envelope_p), w1
        nbytes = ctypes.c_size_t()
        _check(lib.e3_radial_prep_size(self.hidden, self.n_out, ctypes.byref(nbytes)))
        self.prep = torch.empty(nbytes.value, dtype=torch.uint8, device=w1.device)
        _check(lib.e3_radial_prepare(self.hidden, self.n_out, _ptr(w2), _ptr(self.prep), nbytes.value, _stream()))

    def weights(self, edge_vec, out=None):
        E = edge_vec.shape[0]
        _need(edge_vec, "edge_vec", torch.float32, (E, 3), self.w1.device)
        if out is None:
            out = torch.empty((E, self.n_out), dtype=torch.float32, device=self.w1.device)
        _need(out, "out", torch.float32, (E, self.n_out), self.w1.device)
        _check(lib.e3_radial_weights(E, _ptr(edge_vec), self.cutoff, self.n_basis, self.p, self.hidden, _ptr(self.w1),
                                     _ptr(self.prep), self.n_out, _ptr(out), _stream()))
        return out


class Graph:
    """A fixed topology in receiver order: CSR arrays plus src/dst permuted once (E3J,
    section E.2.2: CSR receiver aggregation).  ``perm_dst[i]`` is the original id of the
    i-th edge in receiver order; use ``to_receiver_order`` on per-edge arrays.  ``order``: an
    optional int32 permutation of the nodes in which the kernels process rows (for example the
    Morton order of the positions, ``morton_order``); results do not depend on it."""

    def __init__(self, n_nodes, src, dst, order=None):
        self.n_nodes = int(n_nodes)
        self.n_edges = int(src.shape[0])
        self.perm_dst, self.row_ptr_dst, self.perm_src, self.row_ptr_src = csr_build(self.n_nodes, src, dst)
        self.src = gather_rows(self.perm_dst, src)
        self.dst = gather_rows(self.perm_dst, dst)
        # the convolution's work units (rows cut into segments), built once for the topology
        nbytes = ctypes.c_size_t()
        _check(lib.e3_conv_topology_size(self.n_nodes, self.n_edges, ctypes.byref(nbytes)))
        self.topo = torch.empty(nbytes.value, dtype=torch.uint8, device=src.device)
        if order is not None:
            _need(order, "order", torch.int32, (self.n_nodes,), src.device)
        _check(lib.e3_conv_topology_build_ordered(self.n_nodes, self.n_edges, _ptr(self.row_ptr_dst),
                                                  _ptr(self.row_ptr_src), _ptr(order), _ptr(self.topo),
                                                  self.topo.numel(), _stream()))

    def to_receiver_order(self, t):
        return gather_rows(self.perm_dst, t.contiguous())


def conv_forward(plan, graph, x, w, y=None, edge_vec=None, sh_norm="component", out_scale=1.0, out=None):
    """out[n] = out_scale * sum_{e: dst_e = n} TP(x[src_e], Y_e, w_e) (e3_conv_forward).
    Edge arrays (w, y or edge_vec) are in the graph's receiver order."""
    N, E = graph.n_nodes, graph.n_edges
    dev, dt = plan.device, plan.dtype
    _need(x, "x", dt, (N, plan.dim_in1), dev)
    _need(w, "w", dt, plan._w_shape(E), dev)
    if (y is None) == (edge_vec is None):
        raise ValueError("give exactly one of y and edge_vec")
    if y is not None:
        _need(y, "y", dt, (E, plan.dim_in2), dev)
    else:
        _need(edge_vec, "edge_vec", dt, (E, 3), dev)
    if out is None:
        out = torch.empty((N, plan.dim_out), dtype=dt, device=dev)
    _need(out, "out", dt, (N, plan.dim_out), dev)
    ws = conv_workspace(plan, N, E, dev)
    _check(lib.e3_conv_forward(plan.handle, N, E, _ptr(graph.row_ptr_dst), _ptr(graph.src), _ptr(x), _ptr(y),
                               _ptr(edge_vec), _SH_NORMS[sh_norm], _ptr(w), float(out_scale), _ptr(out),
                               _ptr(graph.topo), _ptr(ws), ws.numel(), _stream()))
    return out


def conv_backward(plan, graph, x, w, grad_out, y=None, edge_vec=None, sh_norm="component", out_scale=1.0,
                  need_x=True, need_y=True, need_w=True):
    """(grad_x, grad_y, grad_w) of <grad_out, conv_forward(...)> (e3_conv_backward)."""
    N, E = graph.n_nodes, graph.n_edges
    dev, dt = plan.device, plan.dtype
    _need(x, "x", dt, (N, plan.dim_in1), dev)
    _need(w, "w", dt, (E, plan.weight_numel), dev)
    _need(grad_out, "grad_out", dt, (N, plan.dim_out), dev)
    if (y is None) == (edge_vec is None):
        raise ValueError("give exactly one of y and edge_vec")
    if y is not None:
        _need(y, "y", dt, (E, plan.dim_in2), dev)
    else:
        _need(edge_vec, "edge_vec", dt, (E, 3), dev)
    gx = torch.empty_like(x) if need_x else None
    gy = torch.empty((E, plan.dim_in2), dtype=dt, device=dev) if need_y else None
    gw = torch.empty_like(w) if need_w else None
    ws = conv_workspace(plan, N, E, dev)
    _check(lib.e3_conv_backward(plan.handle, N, E, _ptr(graph.row_ptr_dst), _ptr(graph.src), _ptr(graph.dst),
                                _ptr(graph.row_ptr_src), _ptr(graph.perm_src), _ptr(x), _ptr(y), _ptr(edge_vec),
                                _SH_NORMS[sh_norm], _ptr(w), _ptr(grad_out), float(out_scale), _ptr(gx),
                                _ptr(gy), _ptr(gw), _ptr(graph.topo), _ptr(ws), ws.numel(), _stream()))
    return gx, gy, gw


def _accumulate(acc, t):
    """acc + t for same-shape tensors through the library (e3_add_rows with the identity rows)."""
    if t is None:
        return acc
    if acc is None:
        return t.contiguous().clone()
    n = acc.shape[0]
    idx = torch.arange(n, dtype=torch.int32, device=acc.device)
    return add_rows_(acc.contiguous(), idx, t.contiguous())


class _ConvFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, y, w, plan, graph, out_scale):
        ctx.plan, ctx.graph, ctx.out_scale = plan, graph, out_scale
        ctx.save_for_backward(x, y, w)
        return conv_forward(plan, graph, x, w, y=y, out_scale=out_scale)

    @staticmethod
    def backward(ctx, g):
        x, y, w = ctx.saved_tensors
        gx, gy, gw = _ConvBwdFn.apply(x, y, w, g.contiguous(), ctx.plan, ctx.graph, ctx.out_scale,
                                      tuple(ctx.needs_input_grad[:3]))
        return gx, gy, gw, None, None, None


class _ConvBwdFn(torch.autograd.Function):
    """The convolution's backward as a differentiable function of (x, y, w, grad_out), so that the
    convolution is twice differentiable (xnn, "Run Models on Fused GPU Kernels", Training: force
    training runs through the fast path).  The convolution F(x, y, w) is linear in each argument,
    so with B_x, B_y, B_w its three gradients and upstream (u_x, u_y, u_w) for them,
        d/dg = F(u_x, y, w) + F(x, u_y, w) + F(x, y, u_w)
        d/dx = B_x(x, u_y, w, g) + B_x(x, y, u_w, g)
        d/dy = B_y(u_x, y, w, g) + B_y(x, y, u_w, g)
        d/dw = B_w(u_x, y, w, g) + B_w(x, u_y, w, g)
    (e.g. <u_y, B_y(x, w, g)> = <g, F(x, u_y, w)>, whose x-gradient is B_x with y -> u_y), each
    term one call of the library's forward or backward kernels, sums by e3_add_rows."""

    @staticmethod
    def forward(ctx, x, y, w, g, plan, graph, out_scale, needs):
        ctx.plan, ctx.graph, ctx.out_scale = plan, graph, out_scale
        ctx.save_for_backward(x, y, w, g)
        gx, gy, gw = conv_backward(plan, graph, x, w, g, y=y, out_scale=out_scale, need_x=needs[0], need_y=needs[1],
                                   need_w=needs[2])
        return gx, gy, gw

    @staticmethod
    def backward(ctx, ux, uy, uw):
        x, y, w, g = ctx.saved_tensors
        P, G, s = ctx.plan, ctx.graph, ctx.out_scale
        nx, ny, nw, ng = ctx.needs_input_grad[:4]
        ux = None if ux is None else ux.contiguous()
        uy = None if uy is None else uy.contiguous()
        uw = None if uw is None else uw.contiguous()
        dx = dy = dw = dg = None
        if ng:
            if ux is not None:
                dg = _accumulate(dg, conv_forward(P, G, ux, w, y=y, out_scale=s))
            if uy is not None:
                dg = _accumulate(dg, conv_forward(P, G, x, w, y=uy, out_scale=s))
            if uw is not None:
                dg = _accumulate(dg, conv_forward(P, G, x, uw, y=y, out_scale=s))
        if uy is not None and (nx or nw):  # y -> u_y: its x- and w-gradients
            bx, _, bw = conv_backward(P, G, x, w, g, y=uy, out_scale=s, need_x=nx, need_y=False, need_w=nw)
            dx, dw = _accumulate(dx, bx), _accumulate(dw, bw)
        if uw is not None and (nx or ny):  # w -> u_w: its x- and y-gradients
            bx, by, _ = conv_backward(P, G, x, uw, g, y=y, out_scale=s, need_x=nx, need_y=ny, need_w=False)
            dx, dy = _accumulate(dx, bx), _accumulate(dy, by)
        if ux is not None and (ny or nw):  # x -> u_x: its y- and w-gradients
            _, by, bw = conv_backward(P, G, ux, w, g, y=y, out_scale=s, need_x=False, need_y=ny, need_w=nw)
            dy, dw = _accumulate(dy, by), _accumulate(dw, bw)
        return dx, dy, dw, dg, None, None, None, None


def conv(plan, graph, x, y, w, out_scale=1.0):
    """Twice-differentiable convolution with respect to x, y (harmonics) and w."""
    return _ConvFn.apply(x, y, w, plan, graph, out_scale)


class _ConvVecFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, vec, w, plan, graph, out_scale, sh_norm):
        ctx.plan, ctx.graph, ctx.out_scale, ctx.sh_norm = plan, graph, out_scale, sh_norm
        ctx.save_for_backward(x, vec, w)
        return conv_forward(plan, graph, x, w, edge_vec=vec, sh_norm=sh_norm, out_scale=out_scale)

    @staticmethod
    def backward(ctx, g):
        x, vec, w = ctx.saved_tensors
        need_vec = ctx.needs_input_grad[1]
        gx, gy, gw = conv_backward(ctx.plan, ctx.graph, x, w, g.contiguous(), edge_vec=vec, sh_norm=ctx.sh_norm,
                                   out_scale=ctx.out_scale, need_x=ctx.needs_input_grad[0], need_y=need_vec,
                                   need_w=ctx.needs_input_grad[2])
        lmax = int(ctx.plan.dim_in2 ** 0.5 + 0.5) - 1  # harmonics irreps 1x0e+1x1o+... of dim (lmax+1)^2
        gvec = spherical_harmonics_backward(lmax, vec, gy, ctx.sh_norm) if need_vec else None
        return gx, gvec, gw, None, None, None, None


def conv_vec(plan, graph, x, edge_vec, w, out_scale=1.0, sh_norm="component"):
    """Differentiable convolution with harmonics computed in the kernels from edge vectors
    (receiver order): gradients with respect to x, edge_vec (through the harmonics) and w."""
    return _ConvVecFn.apply(x, edge_vec, w, plan, graph, out_scale, sh_norm)


class Features:
    """The layout of feature rows [N, dim] for ``group_norm`` and ``dropout``: an irreps string in the
    mul_ir layout (any multiplicities and degrees), the number of groups into which every block's
    channels are cut, and the rows' dtype; bound to the current CUDA device (e3_features_create).

    ``n_channels`` weights (one per copy of an irrep), ``n_scalars`` biases (0e channels only),
    ``n_groups`` groups over all blocks."""

    def __init__(self, irreps, groups=1, dtype=torch.float32):
        if dtype not in _DTYPES:
            raise ValueError("dtype must be torch.float32 or torch.float64")
        handle = ctypes.c_void_p()
        self._handle = None
        _check(lib.e3_features_create(irreps.encode(), int(groups), _DTYPES[dtype], ctypes.byref(handle)))
        self._handle = handle
        self.irreps, self.groups, self.dtype = irreps, int(groups), dtype
        vals = [ctypes.c_int64() for _ in range(4)]
        _check(lib.e3_features_info(handle, *(ctypes.byref(v) for v in vals)))
        self.dim, self.n_channels, self.n_scalars, self.n_groups = (v.value for v in vals)
        self.index = torch.cuda.current_device() if torch.cuda.is_available() else None
        self.device = None if self.index is None else torch.device("cuda", self.index)
        self.workspace_bytes = {}  # sizes by (rows, segments, max_rows)

    def __del__(self):
        if getattr(self, "_handle", None) and lib is not None:
            try:
                lib.e3_features_destroy(self._handle)
            except Exception:  # interpreter shutdown
                pass
            self._handle = None

    @property
    def handle(self):
        return self._handle


class Segments:
    """Rows of a batch cut into structures: segment s holds rows row_ptr[s] .. row_ptr[s+1] - 1 of
    ``n_rows``; rows from row_ptr[-1] on are padding.  ``row_ptr``: int32 CUDA tensor [B + 1] starting
    at 0.  ``max_rows``: an upper bound on a segment's rows if the host knows one: it selects the
    kernels (a bound that does not hold is reported by ``device_status``)."""

    def __init__(self, row_ptr, n_rows, max_rows=None):
        if not isinstance(row_ptr, torch.Tensor) or row_ptr.dim() != 1 or row_ptr.shape[0] < 2:
            raise ValueError("row_ptr must be a one-dimensional tensor of at least two entries")
        if row_ptr.device.type != "cuda":
            raise ValueError("row_ptr must be a CUDA tensor")
        _need(row_ptr, "row_ptr", torch.int32, row_ptr.shape, row_ptr.device)
        if n_rows < 0 or (max_rows is not None and max_rows < 0):
            raise ValueError("n_rows and max_rows must not be negative")
        self.row_ptr, self.n_rows = row_ptr, int(n_rows)
        self.n_segments = row_ptr.shape[0] - 1
        # every segment empty: any positive bound holds
        self.max_rows = 0 if max_rows is None else max(1, int(max_rows))

    @classmethod
    def from_counts(cls, counts, n_rows=None, device=None):
        """From the rows of each segment (host numbers); ``n_rows`` above their sum adds padding rows."""
        counts = [int(c) for c in counts]
        if not counts or min(counts) < 0:
            raise ValueError("counts must be a non-empty list of non-negative numbers")
        total = sum(counts)
        n_rows = total if n_rows is None else int(n_rows)
        if total > n_rows:
            raise ValueError(f"counts add up to {total} rows of {n_rows}")
        if n_rows > 2 ** 31 - 65536:
            raise ValueError("n_rows passes 2^31 - 65536")
        ptr = torch.zeros(len(counts) + 1, dtype=torch.int32)
        ptr[1:] = torch.tensor(counts, dtype=torch.int64).cumsum(0)
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
        return cls(ptr.to(device), n_rows, max_rows=max(counts))


def _rows(t, name, features, shape):
    """`_need` for the operands of the row operators, with the common case first: these calls take a few
    microseconds on small inputs."""
    if not (type(t) is torch.Tensor and t.dtype is features.dtype and t.shape == shape and t.is_contiguous()
            and t.is_cuda and t.get_device() == features.index):
        _need(t, name, features.dtype, shape, features.device)
    return t.data_ptr()


def _opt_rows(t, name, features, shape):
    return None if t is None else _rows(t, name, features, shape)


def _operand(t):
    """A gradient as the C calls take it: autograd hands over strided ones, and slices of a larger gradient
    that do not start on a 16-byte boundary."""
    if t is None:
        return None
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _row_stream(features):
    """The current stream's handle; the features' device has to be current (the library checks it)."""
    return torch._C._cuda_getCurrentRawStream(features.index)


def _drop_spec(features, p, rng, row0):
    """The C dropout argument (by reference), or None when nothing is dropped."""
    if p == 0:
        return None
    p = float(p)
    if not 0.0 <= p < 1.0:
        raise ValueError(f"p must be in [0, 1), got {p}")
    if rng is None:
        raise ValueError("dropout needs rng: a seed, a (seed, offset) pair or an int64 CUDA tensor [2]")
    if not -2 ** 63 <= int(row0) < 2 ** 63:
        raise ValueError("row0 must fit 64 bits")
    if isinstance(rng, torch.Tensor):
        _need(rng, "rng", torch.int64, (2,), features.device)
        return ctypes.byref(DropoutSpec(p, 0, 0, rng.data_ptr(), int(row0)))
    seed, offset = rng if isinstance(rng, (tuple, list)) else (rng, 0)
    seed, offset = int(seed), int(offset)
    if not -2 ** 63 <= seed < 2 ** 64 or not 0 <= offset < 2 ** 32:
        raise ValueError("the seed must fit 64 bits, the offset 32")
    return ctypes.byref(DropoutSpec(p, seed % 2 ** 64, offset, None, int(row0)))


def dropout_forward(features, x, p, rng, residual=None, row0=0, out=None):
    """Dropout of whole channels of rows x [N, dim], plus ``residual`` if given (e3_dropout).
    ``rng``: a seed, a (seed, offset) pair, or an int64 CUDA tensor [seed, offset] read when the kernel
    runs (for captured programs).  ``row0``: index of the first row in a larger, sharded array.
    ``out`` may be x or residual.  The mask depends on rng, row and channel only, so the gradient
    with respect to x is this call on the gradient."""
    N = x.shape[0]
    shape = (N, features.dim)
    px = _rows(x, "x", features, shape)
    pr = _opt_rows(residual, "residual", features, shape)
    if out is None:
        out = torch.empty_like(x)
    _check(lib.e3_dropout(features.handle, N, px, pr, _drop_spec(features, p, rng, row0),
                          _rows(out, "out", features, shape), _row_stream(features)))
    return out


class _DropoutFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, features, p, rng, row0):
        ctx.features, ctx.p, ctx.row0, ctx.has_residual = features, p, row0, residual is not None
        ctx.rng = None if isinstance(rng, torch.Tensor) else rng
        ctx.save_for_backward(*([rng] if isinstance(rng, torch.Tensor) else []))
        return dropout_forward(features, x, p, rng, residual=residual, row0=row0)

    @staticmethod
    def backward(ctx, g):
        rng = ctx.saved_tensors[0] if ctx.saved_tensors else ctx.rng
        gx = None
        if ctx.needs_input_grad[0]:
            gx = _DropoutFn.apply(_operand(g), None, ctx.features, ctx.p, rng, ctx.row0)
        return gx, g if ctx.has_residual else None, None, None, None, None


def dropout(features, x, p, rng, residual=None, row0=0):
    """Differentiable (any order) dropout of whole channels plus an optional residual; see
    ``dropout_forward``.  An rng tensor must keep its values until the backward has run."""
    return _DropoutFn.apply(x, residual, features, p, tuple(rng) if isinstance(rng, list) else rng, row0)


def _norm_args(features, x, weight, bias, segments, act):
    """(N, B, row_ptr, max_rows, x, weight, bias) as the C calls take them."""
    N = x.shape[0]
    px = _rows(x, "x", features, (N, features.dim))
    pw = _opt_rows(weight, "weight", features, (features.n_channels,))
    pb = _opt_rows(bias, "bias", features, (features.n_scalars,))
    if act not in _ACTS:
        raise ValueError(f"act must be None or 'silu', got {act!r}")
    if segments is None:
        return N, 1, None, N, px, pw, pb
    if segments.n_rows != N:
        raise ValueError(f"x has {N} rows, the segments were made for {segments.n_rows}")
    if segments.row_ptr.get_device() != features.index:
        raise ValueError(f"segments are on {segments.row_ptr.device}, expected {features.device}")
    return N, segments.n_segments, segments.row_ptr.data_ptr(), segments.max_rows, px, pw, pb


def _norm_workspace(features, N, B, max_rows):
    """(tensor or None, pointer, bytes); a new buffer each time, so that calls in flight never share one."""
    n = features.workspace_bytes.get((N, B, max_rows))
    if n is None:
        nbytes = ctypes.c_size_t()
        _check(lib.e3_group_norm_workspace_size(features.handle, N, B, max_rows, ctypes.byref(nbytes)))
        if len(features.workspace_bytes) > 4096:
            features.workspace_bytes.clear()
        n = features.workspace_bytes[(N, B, max_rows)] = nbytes.value
    if n == 0:
        return None, None, 0
    ws = torch.empty(n, dtype=torch.uint8, device=features.device)
    return ws, ws.data_ptr(), n


def group_norm_forward(features, x, weight=None, bias=None, segments=None, eps=1e-5, act=None, p=0.0, rng=None,
                       row0=0, out=None):
    """(y, stats): group norm of rows x [N, dim] over the segments (None: one segment of all rows), then
    the activation on the 0e channels, then dropout (e3_group_norm_forward).  ``stats`` [B, n_groups, 2]
    float64 holds (mean, 1 / deviation) for the backward.  Padding rows of y are zero.  ``row0`` is for the dropout
    alone: a structure's statistics need all of its rows in one call."""
    N, B, row_ptr, max_rows, px, pw, pb = _norm_args(features, x, weight, bias, segments, act)
    if out is None:
        out = torch.empty_like(x)
    stats = torch.empty((B, features.n_groups, 2), dtype=torch.float64, device=features.device)
    ws, pws, n = _norm_workspace(features, N, B, max_rows)
    _check(lib.e3_group_norm_forward(features.handle, N, B, row_ptr, max_rows, px, pw, pb, eps, _ACTS[act],
                                     _drop_spec(features, p, rng, row0), _rows(out, "out", features, x.shape),
                                     stats.data_ptr(), pws, n, _row_stream(features)))
    return out, stats


def _norm_stats(features, stats, B):
    return _need(stats, "stats", torch.float64, (B, features.n_groups, 2), features.device).data_ptr()


def group_norm_backward(features, x, stats, grad_y, weight=None, bias=None, segments=None, act=None, p=0.0, rng=None,
                        row0=0, need_x=True, need_weight=True, need_bias=True):
    """(grad_x, grad_weight, grad_bias) of <grad_y, y> (e3_group_norm_backward); skipped ones are None.
    Arguments as the forward's, with its ``stats``."""
    N, B, row_ptr, max_rows, px, pw, pb = _norm_args(features, x, weight, bias, segments, act)
    dt, dev = features.dtype, features.device
    gx = torch.empty_like(x) if need_x else None
    gw = torch.empty(features.n_channels, dtype=dt, device=dev) if need_weight else None
    gb = torch.empty(features.n_scalars, dtype=dt, device=dev) if need_bias else None
    ws, pws, n = _norm_workspace(features, N, B, max_rows)
    _check(lib.e3_group_norm_backward(features.handle, N, B, row_ptr, max_rows, px, _norm_stats(features, stats, B),
                                      pw, pb, _ACTS[act], _drop_spec(features, p, rng, row0),
                                      _rows(grad_y, "grad_y", features, x.shape), _ptr(gx), _ptr(gw), _ptr(gb), pws,
                                      n, _row_stream(features)))
    return gx, gw, gb


def group_norm_double_backward(features, x, stats, grad_y, weight=None, bias=None, u_x=None, u_weight=None,
                               u_bias=None, segments=None, act=None, p=0.0, rng=None, row0=0, need_grad_y=True,
                               need_x=True, need_weight=True, need_bias=True):
    """(d_grad_y, d_x, d_weight, d_bias): the backward of ``group_norm_backward`` for upstream gradients
    u_x, u_weight, u_bias of its three results, None being zero (e3_group_norm_double_backward)."""
    N, B, row_ptr, max_rows, px, pw, pb = _norm_args(features, x, weight, bias, segments, act)
    dt, dev = features.dtype, features.device
    pg = _rows(grad_y, "grad_y", features, x.shape)
    pux = _opt_rows(u_x, "u_x", features, x.shape)
    puw = _opt_rows(u_weight, "u_weight", features, (features.n_channels,))
    pub = _opt_rows(u_bias, "u_bias", features, (features.n_scalars,))
    dg = torch.empty_like(x) if need_grad_y else None
    dx = torch.empty_like(x) if need_x else None
    dw = torch.empty(features.n_channels, dtype=dt, device=dev) if need_weight else None
    db = torch.empty(features.n_scalars, dtype=dt, device=dev) if need_bias else None
    ws, pws, n = _norm_workspace(features, N, B, max_rows)
    _check(lib.e3_group_norm_double_backward(features.handle, N, B, row_ptr, max_rows, px,
                                             _norm_stats(features, stats, B), pw, pb, _ACTS[act],
                                             _drop_spec(features, p, rng, row0), pg, pux, puw, pub, _ptr(dg), _ptr(dx),
                                             _ptr(dw), _ptr(db), pws, n, _row_stream(features)))
    return dg, dx, dw, db


class _NormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, features, segments, eps, act, p, rng, row0):
        ctx.features, ctx.rng = features, rng
        ctx.kw = dict(segments=segments, act=act, p=p, row0=row0)
        y, stats = group_norm_forward(features, x, weight, bias, eps=eps, rng=rng, **ctx.kw)
        # the row pointer too: one that changes before the backward is refused, as a changed x is
        ctx.save_for_backward(x, weight, bias, stats, rng if isinstance(rng, torch.Tensor) else None,
                              None if segments is None else segments.row_ptr)
        return y

    @staticmethod
    def backward(ctx, g):
        x, weight, bias, stats, rng, _ = ctx.saved_tensors
        gx, gw, gb = _NormBwdFn.apply(x, weight, bias, _operand(g), stats, ctx.features,
                                      ctx.rng if rng is None else rng, tuple(ctx.needs_input_grad[:3]), ctx.kw)
        return gx, gw, gb, None, None, None, None, None, None, None


class _NormBwdFn(torch.autograd.Function):
    """The group norm's backward as a differentiable function of (x, weight, bias, grad_y)."""

    @staticmethod
    def forward(ctx, x, weight, bias, g, stats, features, rng, needs, kw):
        ctx.features, ctx.rng, ctx.kw = features, rng, kw
        ctx.save_for_backward(x, weight, bias, g, stats, rng if isinstance(rng, torch.Tensor) else None,
                              None if kw["segments"] is None else kw["segments"].row_ptr)
        ctx.set_materialize_grads(False)
        return group_norm_backward(features, x, stats, g, weight, bias, rng=rng, need_x=needs[0],
                                   need_weight=needs[1], need_bias=needs[2], **kw)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, ux, uw, ub):
        x, weight, bias, g, stats, rng, _ = ctx.saved_tensors
        nx, nw, nb, ng = ctx.needs_input_grad[:4]
        dg, dx, dw, db = group_norm_double_backward(
            ctx.features, x, stats, g, weight, bias, u_x=_operand(ux), u_weight=_operand(uw),
            u_bias=_operand(ub), rng=ctx.rng if rng is None else rng, need_grad_y=ng, need_x=nx, need_weight=nw,
            need_bias=nb, **ctx.kw)
        return dx, dw, db, dg, None, None, None, None, None


def group_norm(features, x, weight=None, bias=None, segments=None, eps=1e-5, act=None, p=0.0, rng=None, row0=0):
    """Twice-differentiable group norm with activation and dropout (x, weight, bias; see
    ``group_norm_forward``).  An rng tensor, and the segments' row pointer, must keep their values until the
    backward has run."""
    rng = tuple(rng) if isinstance(rng, list) else rng  # a list could change before the backward
    return _NormFn.apply(x, weight, bias, features, segments, eps, act, p, rng, row0)
