"""Pins of the feature-row oracle: the generator against its published known answers, derivatives
against central differences, equivariance, the closed forms of the norm, and host refusals of the
library's entry points (no GPU)."""

import ctypes

import numpy as np
import pytest

import oracle

IRREPS = "4x0e+2x0o+6x1o+2x2e"
PTR = [0, 5, 5, 6, 11]   # one empty segment, one of a single row; rows 11.. are padding
N = 13


# Known answers of Philox4x32-10 (the vectors published with the generator).
@pytest.mark.parametrize("ctr,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_philox_known_answers(ctr, key, want):
    assert tuple(oracle.philox4x32(ctr, key)) == want


def test_dropout_rate_and_sharding():
    f = oracle.dropout_factor(IRREPS, 400, 0.3, seed=77, offset=3)
    assert set(np.unique(f)) == {0.0, 1.0 / 0.7}
    kept = np.concatenate(oracle.dropout_keep(IRREPS, 400, 0.3, seed=77, offset=3), axis=1)
    assert abs(kept.mean() - 0.7) < 4.0 * np.sqrt(0.21 / kept.size)
    # components of a channel go together; a shard's rows are the whole call's rows
    v = f[:, 6:24].reshape(400, 6, 3)
    assert np.all(v == v[:, :, :1])
    assert np.array_equal(oracle.dropout_factor(IRREPS, 50, 0.3, seed=77, offset=3, row0=120), f[120:170])
    assert not np.array_equal(oracle.dropout_factor(IRREPS, 50, 0.3, seed=77, offset=4), f[:50])


def _inputs(seed=0):
    rng = np.random.default_rng(seed)
    dim = oracle.parse_irreps(IRREPS).dim
    return (rng.standard_normal((N, dim)) + 0.5, 1.0 + 0.3 * rng.standard_normal(14), 0.3 * rng.standard_normal(4),
            rng.standard_normal((N, dim)), rng)


def _directional(f, args, dirs, h=1e-6):
    plus = f(*[a + h * d for a, d in zip(args, dirs)])
    minus = f(*[a - h * d for a, d in zip(args, dirs)])
    return (plus - minus) / (2.0 * h)


@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_norm_derivatives_match_differences(act, p):
    x, w, b, g, rng = _inputs()
    factor = oracle.dropout_factor(IRREPS, N, p, seed=5) if p else None
    kw = dict(act=act, factor=factor)
    loss = lambda x_, w_, b_: float((oracle.group_norm(IRREPS, 2, PTR, x_, w_, b_, **kw) * g).sum())
    gx, gw, gb = oracle.group_norm_backward(IRREPS, 2, PTR, x, g, w, b, **kw)
    ux, uw, ub = rng.standard_normal(x.shape), rng.standard_normal(w.shape), rng.standard_normal(b.shape)
    want = _directional(loss, (x, w, b), (ux, uw, ub))
    assert abs((gx * ux).sum() + (gw * uw).sum() + (gb * ub).sum() - want) < 1e-7 * max(1.0, abs(want))

    def phi(x_, w_, b_, g_):
        a = oracle.group_norm_backward(IRREPS, 2, PTR, x_, g_, w_, b_, **kw)
        return float((a[0] * ux).sum() + (a[1] * uw).sum() + (a[2] * ub).sum())

    dg, dx, dw, db = oracle.group_norm_double_backward(IRREPS, 2, PTR, x, g, w, b, ux, uw, ub, **kw)
    for i, (a, d) in enumerate(((x, dx), (w, dw), (b, db), (g, dg))):
        dirs = [np.zeros_like(t) for t in (x, w, b, g)]
        dirs[i] = rng.standard_normal(a.shape)
        want = _directional(phi, (x, w, b, g), dirs)
        assert abs((d * dirs[i]).sum() - want) < 1e-6 * max(1.0, abs(want)), i


def test_norm_closed_forms():
    x, w, b, _, _ = _inputs(3)
    y = oracle.group_norm(IRREPS, 2, PTR, x, eps=1e-12)
    s = y[:5, :2]                       # first group of the even scalars: mean 0, mean square 1
    assert abs(s.mean()) < 1e-12 and abs(np.mean(s ** 2) - 1.0) < 1e-9
    v = y[:5, 6:15]                     # first group of the vectors: mean square 1, mean kept
    assert abs(np.mean(v ** 2) - 1.0) < 1e-9
    assert np.allclose(v / np.sqrt(np.mean(v ** 2)), x[:5, 6:15] / np.sqrt(np.mean(x[:5, 6:15] ** 2)))
    assert np.all(y[11:] == 0.0)
    one = oracle.group_norm("1x0e", 1, [0, 1], np.array([[7.0]]), bias=np.array([0.25]))
    assert one[0, 0] == 0.25            # a single value: its own mean


def test_norm_commutes_with_rotations_and_inversion():
    x, w, b, _, _ = _inputs(4)
    rng = np.random.default_rng(9)
    R, _ = np.linalg.qr(rng.standard_normal((3, 3)))   # acts on the l = 1 blocks (any orthonormal basis of R^3)
    Q, _ = np.linalg.qr(rng.standard_normal((5, 5)))   # a norm of the l = 2 components is all that is used

    def act(t):
        o = t.copy()
        o[:, 4:6] *= -1.0
        o[:, 6:24] = (t[:, 6:24].reshape(N, 6, 3) @ R.T).reshape(N, 18)
        o[:, 24:34] = (t[:, 24:34].reshape(N, 2, 5) @ Q.T).reshape(N, 10)
        return o

    f = oracle.dropout_factor(IRREPS, N, 0.25, seed=1)
    a = oracle.group_norm(IRREPS, 2, PTR, act(x), w, b, act="silu", factor=f)
    assert np.allclose(a, act(oracle.group_norm(IRREPS, 2, PTR, x, w, b, act="silu", factor=f)), atol=1e-12)


# ------------------------------------------------------------------ library refusals (host) ---

@pytest.fixture(scope="module")
def e3b():
    from mlip_message_passing_b200 import e3b
    return e3b


@pytest.mark.parametrize("irreps,groups,code", [
    ("8x0e+8x1q", 1, "IRREPS_PARSE"),
    ("", 1, "IRREPS_PARSE"),
    ("8x0e", 0, "INVALID_ARG"),
    ("8x0e+6x1o", 4, "SHAPE"),
    ("+".join(["1x0e"] * 33), 1, "UNSUPPORTED"),
    ("1000000x20e", 1, "UNSUPPORTED"),
    ("1x501e", 1, "UNSUPPORTED"),
])
def test_features_refusals(e3b, irreps, groups, code):
    with pytest.raises(e3b.E3Error) as err:
        e3b.Features(irreps, groups=groups)
    assert e3b.STATUS_NAMES[err.value.status] == code


def test_features_layout(e3b):
    import torch
    f = e3b.Features("25x0e + 7x0o + 11x1o + 5x2e + 3x0e", groups=1, dtype=torch.float64)
    assert (f.dim, f.n_channels, f.n_scalars, f.n_groups) == (25 + 7 + 33 + 25 + 3, 51, 28, 5)
    with pytest.raises(ValueError):
        e3b.Features("8x0e", dtype=torch.float16)


def test_dropout_argument_refusals(e3b):
    f = e3b.Features("8x0e")
    for p in (-0.1, 1.0, 1.5, float("nan")):
        with pytest.raises(ValueError):
            e3b._drop_spec(f, p, 1, 0)
    with pytest.raises(ValueError):
        e3b._drop_spec(f, 0.5, None, 0)
    with pytest.raises(ValueError):
        e3b._drop_spec(f, 0.5, (1, 2 ** 32), 0)
    with pytest.raises(ValueError):
        e3b._drop_spec(f, 0.5, 2 ** 64, 0)
    assert e3b._drop_spec(f, 0.0, None, 0) is None


def test_segments_refusals(e3b):
    import torch
    for bad in ([], [3, -1]):
        with pytest.raises(ValueError):
            e3b.Segments.from_counts(bad, device="cpu")
    with pytest.raises(ValueError):
        e3b.Segments.from_counts([3, 4], n_rows=6, device="cpu")
    with pytest.raises(ValueError):
        e3b.Segments.from_counts([2 ** 31], device="cpu")
    with pytest.raises(ValueError):   # host tensors are refused
        e3b.Segments(torch.zeros(3, dtype=torch.int32), 4)


def test_workspace_size_of_extreme_shapes(e3b):
    nb = ctypes.c_size_t()
    f = e3b.Features("64x0e+64x1o", groups=8)
    for n, b, m in ((0, 1, 0), (1, 1, 1), (2 ** 31 - 65536, 1, 0), (1, 100000, 1), (100000, 100000, 1)):
        assert e3b.lib.e3_group_norm_workspace_size(f.handle, n, b, m, ctypes.byref(nb)) == e3b.E3_OK
        assert nb.value < 2 ** 33
    assert e3b.lib.e3_group_norm_workspace_size(f.handle, 2 ** 31 - 65535, 1, 0, ctypes.byref(nb)) == e3b.E3_ERR_SHAPE
    assert e3b.lib.e3_group_norm_workspace_size(f.handle, -1, 1, 0, ctypes.byref(nb)) == e3b.E3_ERR_SHAPE
    assert e3b.lib.e3_group_norm_workspace_size(f.handle, 5, 0, 0, ctypes.byref(nb)) == e3b.E3_ERR_SHAPE
    assert e3b.lib.e3_group_norm_workspace_size(None, 5, 1, 0, ctypes.byref(nb)) == e3b.E3_ERR_INVALID_ARG
