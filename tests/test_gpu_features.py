"""Feature-row operators (group norm with an activation, counter-based dropout) against the float64
oracle, at the sizes and masks where they can go wrong.

Tolerances, elementwise, in half steps of the type (2^-24 for float32, 2^-53 for float64) times the sum
of the absolute values of the terms that make up an output (the oracle's ``scale=True``):
* a thread adds at most 64 rows in the rows' type before it goes on in double: 64 half steps for a
  column sum, and 4 x 64 where a thread adds its four columns into one sum (double backward);
* the pointwise part rounds fewer than 32 times (centre 2, scale, weight, bias, the sigmoid with a
  2-ulp exponential and a 2-ulp division, its derivatives, the result).
So 96 for the forward and the backward, 288 for the double backward."""

import numpy as np
import pytest
import torch

import oracle
from mlip_message_passing_b200 import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF = {torch.float32: 2.0 ** -24, torch.float64: 2.0 ** -53}
NP = {torch.float32: np.float32, torch.float64: np.float64}


@pytest.fixture(scope="module")
def e3b():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from mlip_message_passing_b200 import e3b
    return e3b


def _close(got, want, size, steps, dtype, what):
    got = got.detach().cpu().double().numpy()
    bound = steps * HALF[dtype] * size + 1e-30
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (what, int(bad.sum()), float(np.nanmax(np.abs(got - want) / bound)))


def _data(irreps, N, dtype, seed, offset=0.0, scale=1.0):
    rng = np.random.default_rng(seed)
    blocks = oracle.parse_irreps(irreps)
    n_ch = sum(b.mul for b in blocks)
    n_sc = sum(b.mul for b in blocks if b.l == 0 and b.p == 1)
    t = lambda *s: rng.standard_normal(s).astype(NP[dtype])
    d = dict(x=t(N, blocks.dim) * NP[dtype](scale) + NP[dtype](offset), w=1 + NP[dtype](0.3) * t(n_ch),
             b=NP[dtype](0.3) * t(n_sc), g=t(N, blocks.dim), ux=t(N, blocks.dim), uw=t(n_ch), ub=t(n_sc))
    return {k: np.ascontiguousarray(v) for k, v in d.items()}


def _check_all(e3b, irreps, groups, counts, pad, dtype, act, p, seed, hint="max", data=None):
    N = sum(counts) + pad
    ptr = np.concatenate([[0], np.cumsum(counts)])
    d = _data(irreps, N, dtype, seed) if data is None else data
    f = e3b.Features(irreps, groups=groups, dtype=dtype)
    seg = e3b.Segments.from_counts(counts, n_rows=N)
    if hint != "max":
        seg.max_rows = hint
    if len(counts) == 1 and pad == 0 and hint == "max":
        seg = None
    t = {k: torch.as_tensor(v, device=DEV) for k, v in d.items()}
    if pad:  # what padding rows hold is never looked at
        for k in ("x", "g", "ux"):
            t[k][N - pad:] = float("nan")
    rng = (seed + 2 ** 40, 7)
    factor = oracle.dropout_factor(irreps, N, p, rng[0], rng[1]) if p else None
    kw = dict(segments=seg, act=act, p=p, rng=rng if p else None)
    y, stats = e3b.group_norm_forward(f, t["x"], t["w"], t["b"], **kw)
    gx, gw, gb = e3b.group_norm_backward(f, t["x"], stats, t["g"], t["w"], t["b"], **kw)
    dbl = e3b.group_norm_double_backward(f, t["x"], stats, t["g"], t["w"], t["b"], u_x=t["ux"], u_weight=t["uw"],
                                         u_bias=t["ub"], **kw)
    e3b.device_status()
    okw = dict(act=act, factor=factor, scale=True)
    _close(y, *oracle.group_norm(irreps, groups, ptr, d["x"], d["w"], d["b"], **okw), 96, dtype, "y")
    ref = oracle.group_norm_backward(irreps, groups, ptr, d["x"], d["g"], d["w"], d["b"], **okw)
    for i, (got, what) in enumerate(((gx, "gx"), (gw, "gw"), (gb, "gb"))):
        _close(got, ref[i], ref[i + 3], 96, dtype, what)
    ref = oracle.group_norm_double_backward(irreps, groups, ptr, d["x"], d["g"], d["w"], d["b"], d["ux"], d["uw"],
                                            d["ub"], **okw)
    for i, (got, what) in enumerate(zip(dbl, ("dg", "dx", "dw", "db"))):
        _close(got, ref[i], ref[i + 4], 288, dtype, what)
    if pad:
        for got in (y, gx, dbl[0], dbl[1]):
            assert bool((got[N - pad:] == 0).all())
    return y, stats


LAYOUTS = [("64x0e+64x1o+64x2e", 8), ("128x0e+128x1o", 8), ("64x0e", 8), ("25x0e+7x0o+11x1o+5x2e", 1), ("1x0e", 1),
           ("4x0e+4x3o", 2), ("3x1o", 3), ("8x1o+8x0e+4x2e+12x0e", 4), ("30x0e+10x1o", 1)]


@pytest.mark.parametrize("irreps,groups", LAYOUTS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.float64])
@pytest.mark.parametrize("counts,pad", [([1], 0), ([37], 0), ([5, 0, 1, 17, 2, 9, 0], 3)])
def test_norm_small_segments(e3b, irreps, groups, dtype, counts, pad):
    _check_all(e3b, irreps, groups, counts, pad, dtype, "silu", 0.0, seed=sum(counts) + groups)


@pytest.mark.parametrize("irreps,groups", LAYOUTS)
@pytest.mark.parametrize("dtype,act,p", [(torch.float32, None, 0.3), (torch.float64, "silu", 0.15),
                                         (torch.float32, "silu", 0.15)])
def test_norm_with_dropout(e3b, irreps, groups, dtype, act, p):
    _check_all(e3b, irreps, groups, [11, 40, 3], 2, dtype, act, p, seed=groups)


@pytest.mark.parametrize("irreps,groups", LAYOUTS[:4])
@pytest.mark.parametrize("counts,pad", [([2500], 0), ([900, 1, 0, 1200, 33], 9)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float64])
def test_norm_long_segments(e3b, irreps, groups, counts, pad, dtype):
    _check_all(e3b, irreps, groups, counts, pad, dtype, "silu", 0.0, seed=3)


@pytest.mark.parametrize("irreps,groups", [LAYOUTS[0], LAYOUTS[3]])
@pytest.mark.parametrize("counts,pad,hint", [
    ([5, 0, 1, 17, 2, 9, 0, 60], 3, 0),    # no hint: the kernels for long segments on short ones
    ([150, 0, 301, 40], 5, 400),           # a bound that is not tight
    ([70, 0, 3, 64], 5, 2000),             # nor this one: clusters with idle CTAs
    ([1] * 200, 0, "max"),                 # every row by itself
    ([0, 0, 0], 4, "max"),                 # nothing but padding
])
def test_norm_hints_and_rows(e3b, irreps, groups, counts, pad, hint):
    _check_all(e3b, irreps, groups, counts, pad, torch.float32, "silu", 0.0, seed=21, hint=hint)


@pytest.mark.parametrize("irreps,groups,dtype", [("30x0e+30x1o+30x2e", 1, torch.float32),
                                                  ("31x0e+7x3o", 1, torch.float32), ("30x0e+30x1o", 1, torch.float64)])
def test_norm_rows_that_take_turns(e3b, irreps, groups, dtype):
    """Many segments with more rows than a block's slots: their rows take the slots in turns."""
    _check_all(e3b, irreps, groups, [60, 3, 41, 0, 64] * 40, 7, dtype, "silu", 0.1, seed=9)


def test_norm_many_tiny_rows(e3b):
    """Rows narrower than a warp, thousands of one-row segments: many segments per block."""
    _check_all(e3b, "4x0e+4x1o", 4, [1] * 700, 3, torch.float32, "silu", 0.0, seed=9)
    _check_all(e3b, "1x0e", 1, [1] * 1500, 0, torch.float64, None, 0.0, seed=9)
    _check_all(e3b, "3x0e+1x1o", 1, [1, 0] * 600, 0, torch.float32, "silu", 0.4, seed=9)


@pytest.mark.parametrize("irreps,groups", [("64x0e+64x1o+64x2e", 8), ("40x0e+40x1o", 4)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float64])
@pytest.mark.parametrize("act", [None, "silu"])
def test_norm_more_segments_than_blocks(e3b, irreps, groups, dtype, act):
    """With many segments the tiles of scalars, which take longer, get more blocks.  Row results are those of the
    segments taken 100 at a time, bit for bit; the parameters' gradients add up to float64 sums: each side is off
    by 288 half steps of the sum of its terms' absolute values, of which there are 5 a row at most, below 64 each
    (factors of unit variance)."""
    counts, per = [1 + i % 7 for i in range(2000)], 100
    N = sum(counts)
    f = e3b.Features(irreps, groups=groups, dtype=dtype)
    gen = torch.Generator(DEV).manual_seed(11)
    x, g, ux = (torch.randn(N, f.dim, device=DEV, dtype=dtype, generator=gen) for _ in range(3))
    w, b, uw, ub = (torch.randn(n, device=DEV, dtype=dtype, generator=gen).clamp(-2, 2)
                    for n in (f.n_channels, f.n_scalars) * 2)

    def run(lo, counts):
        n = sum(counts)
        seg = e3b.Segments.from_counts(counts)
        seg.max_rows = 7
        kw = dict(segments=seg, act=act, p=0.2, rng=(3, 1), row0=lo)
        at = slice(lo, lo + n)
        xs, gs, us = (t[at].clone() for t in (x, g, ux))
        y, st = e3b.group_norm_forward(f, xs, w, b, **kw)
        gx, gw, gb = e3b.group_norm_backward(f, xs, st, gs, w, b, **kw)
        dg, dx, dw, db = e3b.group_norm_double_backward(f, xs, st, gs, w, b, u_x=us, u_weight=uw, u_bias=ub, **kw)
        return (y, gx, dg, dx), (gw, gb, dw, db)

    rows, params = run(0, counts)
    sums = [torch.zeros(t.shape, device=DEV, dtype=torch.float64) for t in params]
    at = 0
    for i in range(0, len(counts), per):
        part_rows, part_params = run(at, counts[i:i + per])
        n = part_rows[0].shape[0]
        for whole, part in zip(rows, part_rows):
            assert torch.equal(whole[at:at + n], part)
        for t, part in zip(sums, part_params):
            t += part.double()
        at += n
    for t, whole in zip(sums, params):
        assert float((t - whole.double()).abs().max()) <= 2 * 288 * HALF[dtype] * 64 * 5 * N
    e3b.device_status()


def test_norm_bound_that_is_too_small_is_reported(e3b):
    """Rows of a segment beyond what the bound selected are skipped and the status word says so."""
    f = e3b.Features("8x0e+8x1o", groups=2)
    x = torch.randn(500, 32, device=DEV)
    seg = e3b.Segments.from_counts([200, 300])
    for bound in (1, 2, 7):
        seg.max_rows = bound
        e3b.group_norm_forward(f, x, segments=seg)
        with pytest.raises(e3b.E3Error) as err:
            e3b.device_status()
        assert err.value.status == e3b.E3_ERR_INDEX


def test_norm_wide_groups(e3b):
    """Groups wider than a block of threads: only the kernels for long segments hold them."""
    _check_all(e3b, "700x1o+300x0e", 1, [30, 0, 7], 1, torch.float32, "silu", 0.2, seed=2)
    _check_all(e3b, "257x0e", 1, [6], 0, torch.float32, None, 0.0, seed=2)
    _check_all(e3b, "2x100e", 1, [4], 0, torch.float64, None, 0.0, seed=2)


@pytest.mark.parametrize("counts", [[40] * 6, [3000]])
def test_norm_offset_and_outlier_data(e3b, counts):
    """Scalars far from zero and one value far from the rest: the variance keeps its digits.  The data
    is rounded to float32 before both sides see it; 1e4 +- 1 moves by 2^-11 of its spread."""
    irreps, groups, N = "16x0e+4x1o", 2, sum(counts)
    d = _data(irreps, N, torch.float32, 5)
    d["x"][:, :16] += np.float32(1e4)
    d["x"][0, 0] = np.float32(1e4 + 500.0)
    _check_all(e3b, irreps, groups, counts, 0, torch.float32, "silu", 0.0, seed=5, data=d)


def test_norm_nan_stays_in_its_group(e3b):
    f = e3b.Features("8x0e+8x1o", groups=2)
    x = torch.randn(30, 32, device=DEV, generator=torch.Generator(DEV).manual_seed(1))
    x[4, 1] = float("nan")
    x[14, 20] = float("inf")
    y, _ = e3b.group_norm_forward(f, x, segments=e3b.Segments.from_counts([10, 10, 10]))
    bad = ~torch.isfinite(y)
    assert bool(bad[:10, :4].all()) and int(bad[:10, 4:].sum()) == 0
    assert int(bad[10:20, :20].sum()) == 0 and bool(bad[14, 20])
    assert int(bad[20:].sum()) == 0


def test_norm_defaults_and_optional_gradients(e3b):
    irreps, counts = "16x0e+8x1o", [9, 12]
    d = _data(irreps, 21, torch.float32, 8)
    f, seg = e3b.Features(irreps, groups=4), e3b.Segments.from_counts([9, 12])
    t = {k: torch.as_tensor(v, device=DEV) for k, v in d.items()}
    y, stats = e3b.group_norm_forward(f, t["x"], segments=seg, eps=1e-3)
    ptr = np.concatenate([[0], np.cumsum(counts)])
    _close(y, *oracle.group_norm(irreps, 4, ptr, d["x"], eps=1e-3, scale=True), 96, torch.float32, "y")
    full = e3b.group_norm_backward(f, t["x"], stats, t["g"], segments=seg)
    for needs in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (0, 0, 0)):
        part = e3b.group_norm_backward(f, t["x"], stats, t["g"], segments=seg, need_x=needs[0], need_weight=needs[1],
                                       need_bias=needs[2])
        for a, b, n in zip(part, full, needs):
            assert (a is None) if not n else torch.equal(a, b)
    full = e3b.group_norm_double_backward(f, t["x"], stats, t["g"], segments=seg, u_x=t["ux"])
    for k in range(4):
        part = e3b.group_norm_double_backward(f, t["x"], stats, t["g"], segments=seg, u_x=t["ux"], need_grad_y=k == 0,
                                              need_x=k == 1, need_weight=k == 2, need_bias=k == 3)
        assert torch.equal(part[k], full[k]) and sum(v is not None for v in part) == 1
    ref = oracle.group_norm_double_backward(irreps, 4, ptr, d["x"], d["g"], eps=1e-3, u_weight=d["uw"], scale=True)
    got = e3b.group_norm_double_backward(f, t["x"], stats, t["g"], segments=seg, u_weight=t["uw"])
    for i in range(4):
        _close(got[i], ref[i], ref[i + 4], 288, torch.float32, i)
    # no rows at all
    y, stats = e3b.group_norm_forward(f, t["x"][:0])
    gx, gw, gb = e3b.group_norm_backward(f, t["x"][:0], stats, t["g"][:0])
    assert y.shape == (0, 40) and gx.shape == (0, 40) and not gw.any() and not gb.any()


def test_norm_repeatable_across_calls_and_streams(e3b):
    f = e3b.Features("64x0e+64x1o+64x2e", groups=8)
    gen = torch.Generator(DEV).manual_seed(3)
    x, g = (torch.randn(3000, f.dim, device=DEV, generator=gen) for _ in range(2))
    for seg in (None, e3b.Segments.from_counts([30] * 100)):
        def run():
            y, st = e3b.group_norm_forward(f, x, segments=seg, act="silu", p=0.1, rng=5)
            return (y, *e3b.group_norm_backward(f, x, st, g, segments=seg, act="silu", p=0.1, rng=5),
                    *e3b.group_norm_double_backward(f, x, st, g, u_x=g, segments=seg, act="silu", p=0.1, rng=5))
        a = run()
        side = [torch.cuda.Stream() for _ in range(2)]
        res = []
        torch.cuda.synchronize()
        for s in side:  # two calls at once, each with its own workspace
            with torch.cuda.stream(s):
                res.append(run())
        torch.cuda.synchronize()
        for r in res:
            assert all(torch.equal(u, v) for u, v in zip(a, r))
    e3b.device_status()


def test_norm_bad_row_pointer_is_reported(e3b):
    """Decreasing, too large or shifted row pointers: rows stay in range (the kernels clamp them) and
    the status word says so; a good call afterwards is clean."""
    f = e3b.Features("8x0e+8x1o", groups=2)
    x = torch.randn(40, 32, device=DEV)
    for ptr in ([0, 30, 20, 40], [0, 20, 41], [2, 20, 40], [0, -5, 40]):
        for hint in (40, None):
            seg = e3b.Segments(torch.tensor(ptr, dtype=torch.int32, device=DEV), 40, max_rows=hint)
            _, stats = e3b.group_norm_forward(f, x, segments=seg)
            with pytest.raises(e3b.E3Error) as err:
                e3b.device_status()
            assert err.value.status == e3b.E3_ERR_INDEX
            e3b.group_norm_backward(f, x, stats, x, segments=seg)
            with pytest.raises(e3b.E3Error):
                e3b.device_status()
    e3b.group_norm_forward(f, x, segments=e3b.Segments.from_counts([20, 20]))
    e3b.device_status()


def test_refusals(e3b):
    f = e3b.Features("8x0e+8x1o", groups=2)
    x = torch.randn(10, 32, device=DEV)
    ok = torch.ones(16, device=DEV)
    for bad in (x.double(), x.cpu(), x[:, :31], torch.randn(32, 10, device=DEV).t()):
        with pytest.raises(ValueError):
            e3b.group_norm_forward(f, bad)
        with pytest.raises(ValueError):
            e3b.dropout_forward(f, bad, 0.1, 1)
    with pytest.raises(ValueError):
        e3b.group_norm_forward(f, x, weight=ok[:8])
    with pytest.raises(ValueError):
        e3b.group_norm_forward(f, x, bias=ok)
    with pytest.raises(ValueError):
        e3b.group_norm_forward(f, x, act="gelu")
    with pytest.raises(ValueError):
        e3b.group_norm_forward(f, x, segments=e3b.Segments.from_counts([4, 5]))
    with pytest.raises(ValueError):
        e3b.group_norm_forward(f, x, p=0.5)
    with pytest.raises(ValueError):
        e3b.dropout_forward(f, x, 0.5, torch.zeros(2, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        e3b.dropout_forward(f, x, 0.5, 1, residual=x[:9])
    with pytest.raises(ValueError):
        e3b.group_norm_backward(f, x, torch.zeros(1, 4, 2, device=DEV), x)
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(e3b.E3Error) as err:
            e3b.group_norm_forward(f, x, eps=eps)
        assert err.value.status == e3b.E3_ERR_INVALID_ARG
    for row0 in (-1, 2 ** 32 - 9):
        with pytest.raises(e3b.E3Error) as err:
            e3b.dropout_forward(f, x, 0.5, 1, row0=row0)
        assert err.value.status == e3b.E3_ERR_SHAPE
    # a view that starts off a 16-byte boundary
    odd = e3b.Features("3x0e")
    with pytest.raises(e3b.E3Error) as err:
        e3b.dropout_forward(odd, torch.randn(5, 3, device=DEV)[1:], 0.1, 1)
    assert err.value.status == e3b.E3_ERR_INVALID_ARG


# ------------------------------------------------------------------------------- dropout ---

@pytest.mark.parametrize("irreps", ["64x0e+64x1o+64x2e", "25x0e+7x0o+11x1o+5x2e", "1x0e", "3x1o", "4x0e+4x3o+2x1e",
                                    "300x1o"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float64])
@pytest.mark.parametrize("N,p,residual", [(1, 0.5, False), (67, 0.1, True), (130, 0.0, True), (40, 0.999, False)])
def test_dropout(e3b, irreps, dtype, N, p, residual):
    f = e3b.Features(irreps, dtype=dtype)
    rng = np.random.default_rng(N)
    x, r = (rng.standard_normal((N, f.dim)).astype(NP[dtype]) for _ in range(2))
    fac = oracle.dropout_factor(irreps, N, p, 2 ** 63 + 11, 4, row0=5)
    got = e3b.dropout_forward(f, torch.as_tensor(x, device=DEV), p, (2 ** 63 + 11, 4), row0=5,
                              residual=torch.as_tensor(r, device=DEV) if residual else None)
    want = x * fac + (r if residual else 0.0)
    # the factor, the product and the sum round once each
    _close(got, want, np.abs(x * fac) + np.abs(want), 2, dtype, "out")
    if not residual:
        assert np.array_equal(got.cpu().numpy() == 0, fac == 0)


def test_dropout_in_place_state_and_shards(e3b):
    f = e3b.Features("64x0e+64x1o")
    x = torch.randn(500, f.dim, device=DEV)
    want = e3b.dropout_forward(f, x, 0.4, (9, 2))
    state = torch.tensor([9, 2], dtype=torch.int64, device=DEV)
    assert torch.equal(e3b.dropout_forward(f, x, 0.4, state), want)
    parts = [e3b.dropout_forward(f, x[a:b].contiguous(), 0.4, state, row0=a) for a, b in ((0, 123), (123, 500))]
    assert torch.equal(torch.cat(parts), want)
    for other in ((10, 2), (9, 3), (9 + 2 ** 32, 2)):
        assert not torch.equal(e3b.dropout_forward(f, x, 0.4, other), want)
    y = x.clone()
    assert e3b.dropout_forward(f, y, 0.4, (9, 2), out=y) is y and torch.equal(y, want)
    y = x.clone()
    e3b.dropout_forward(f, x, 0.4, (9, 2), residual=y, out=y)
    assert torch.equal(y, want + x)
    bad = x.clone()
    bad[want == 0] = float("nan")     # a dropped value gives 0 whatever it is
    assert torch.equal(e3b.dropout_forward(f, bad, 0.4, (9, 2)), want)
    # a negative seed is its two's complement, as an int64 state holds it
    neg = torch.tensor([-3, 1], dtype=torch.int64, device=DEV)
    assert torch.equal(e3b.dropout_forward(f, x, 0.4, neg), e3b.dropout_forward(f, x, 0.4, (2 ** 64 - 3, 1)))
    assert torch.equal(e3b.dropout_forward(f, x, 0.4, neg), e3b.dropout_forward(f, x, 0.4, (-3, 1)))


def test_dropout_autograd(e3b):
    f = e3b.Features("8x0e+8x1o", dtype=torch.float64)
    x, r, g = (torch.randn(20, 32, device=DEV, dtype=torch.float64, requires_grad=True) for _ in range(3))
    y = e3b.dropout(f, x, 0.3, 5, residual=r)
    gx, gr = torch.autograd.grad(y, (x, r), g, create_graph=True)
    assert torch.equal(gr, g) and torch.equal(gx.detach(), e3b.dropout_forward(f, g.detach(), 0.3, 5))
    (gg,) = torch.autograd.grad(gx, g, x.detach())
    assert torch.equal(gg, e3b.dropout_forward(f, x.detach(), 0.3, 5))


# -------------------------------------------------------------------------------- offsets ---

def test_rows_beyond_32_bit_offsets(e3b):
    """1.1 M rows of 2048 columns: 2.25e9 values, offsets pass 2^31.  The last structure is checked
    against the oracle, dropout's last rows against its mask."""
    irreps, N, last = "128x0e+128x1o+128x2e+128x3o", 1_100_000, 50
    f = e3b.Features(irreps, groups=16)
    x = torch.empty(N, f.dim, device=DEV)
    for a in range(0, N, 100_000):
        x[a:a + 100_000].normal_(generator=torch.Generator(DEV).manual_seed(a))
    tail = x[N - last:].cpu().numpy()
    for hint in (None, 2):
        seg = e3b.Segments(torch.tensor([0, N - last, N], dtype=torch.int32, device=DEV), N, max_rows=None)
        y, _ = e3b.group_norm_forward(f, x, segments=seg, act="silu", p=0.5, rng=(3, 1))
        fac = oracle.dropout_factor(irreps, last, 0.5, 3, 1, row0=N - last)
        ref = oracle.group_norm(irreps, 16, [0, last], tail, act="silu", factor=fac, scale=True)
        _close(y[N - last:], *ref, 96, torch.float32, hint)
        del y
    out = e3b.dropout_forward(f, x, 0.5, (3, 1), out=x)
    assert np.array_equal(out[N - last:].cpu().numpy(), (tail * fac).astype(np.float32))
    e3b.device_status()
    del x, out
    torch.cuda.empty_cache()


# ------------------------------------------------------------------------- run together ---

@pytest.mark.parametrize("counts", [[20, 0, 700, 30], [20, 9000, 30], [7, 8, 0, 9] * 50, [1] * 300])
def test_captured_layer_replays_with_new_masks(e3b, counts):
    """norm + dropout, forward and backward, recorded into two CUDA graphs (one layer each) and replayed
    with another seed: the results of the eager calls.  Clusters, the grid, one CTA, one row each."""
    f = e3b.Features("32x0e+32x1o", groups=4)
    n = sum(counts) + 10
    seg = e3b.Segments.from_counts(counts, n_rows=n)
    gen = torch.Generator(DEV).manual_seed(0)
    x, g = (torch.randn(n, f.dim, device=DEV, generator=gen) for _ in range(2))
    state = torch.tensor([1, 0], dtype=torch.int64, device=DEV)

    def layer(src, rng):
        y, st = e3b.group_norm_forward(f, src, segments=seg, act="silu", p=0.2, rng=rng)
        z = e3b.dropout_forward(f, y, 0.2, rng, residual=src)
        gx, gw, gb = e3b.group_norm_backward(f, src, st, g, segments=seg, act="silu", p=0.2, rng=rng)
        return y, z, gx, gw, gb

    layer(x, state)
    torch.cuda.synchronize()
    graphs, outs = [], []
    src = x
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = layer(src, state)
        graphs.append(graph)
        outs.append(out)
        src = out[1]
    for seed in (1, 42):
        state[0] = seed
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        a = layer(x, (seed, 0))
        b = layer(a[1], (seed, 0))
        for got, want in zip(outs, (a, b)):
            assert all(torch.equal(u, v) for u, v in zip(got, want))
    e3b.device_status()
    del graphs


def test_autograd_defaults_and_changed_state(e3b):
    """No weight or bias; only some leaves need gradients; a grad that is not contiguous; a third
    derivative and a state that changed before the backward are refused."""
    f = e3b.Features("8x0e+4x1o", groups=2, dtype=torch.float64)
    gen = torch.Generator(DEV).manual_seed(4)
    x, g = (torch.randn(30, f.dim, device=DEV, dtype=torch.float64, generator=gen) for _ in range(2))
    seg = e3b.Segments.from_counts([10, 20])
    leaf = x.clone().requires_grad_(True)
    y = e3b.group_norm(f, leaf, segments=seg, act="silu")
    (gx,) = torch.autograd.grad(y, leaf, g.t().contiguous().t(), create_graph=True)
    _, st = e3b.group_norm_forward(f, x, segments=seg, act="silu")
    want = e3b.group_norm_backward(f, x, st, g, segments=seg, act="silu")
    assert torch.equal(gx.detach(), want[0])
    (dx,) = torch.autograd.grad(gx.square().sum(), leaf, create_graph=True)
    ref = e3b.group_norm_double_backward(f, x, st, g, u_x=2 * want[0], segments=seg, act="silu")
    assert torch.equal(dx.detach(), ref[1])
    with pytest.raises(RuntimeError):
        torch.autograd.grad(dx.sum(), leaf)
    w = torch.ones(f.n_channels, device=DEV, dtype=torch.float64, requires_grad=True)
    y = e3b.group_norm(f, x, w, segments=seg)
    (gw,) = torch.autograd.grad(y, w, g)
    _, st = e3b.group_norm_forward(f, x, w.detach(), segments=seg)
    assert torch.equal(gw, e3b.group_norm_backward(f, x, st, g, w.detach(), segments=seg)[1])
    state = torch.tensor([3, 0], dtype=torch.int64, device=DEV)
    for call in (lambda: e3b.group_norm(f, leaf, segments=seg, p=0.5, rng=state),
                 lambda: e3b.dropout(f, leaf, 0.5, state)):
        y = call()
        state += 1
        with pytest.raises(RuntimeError):
            torch.autograd.grad(y, leaf, g)


def test_norm_writes_over_its_input(e3b):
    """out=x: every value is read before it is written, whichever kernel runs."""
    f = e3b.Features("64x0e+64x1o", groups=8)
    for counts in ([30] * 20, [1] * 50, [2000], [20_000, 5]):
        seg = e3b.Segments.from_counts(counts)
        x = torch.randn(sum(counts), f.dim, device=DEV, generator=torch.Generator(DEV).manual_seed(1))
        want, _ = e3b.group_norm_forward(f, x, segments=seg, act="silu")
        y, _ = e3b.group_norm_forward(f, x, segments=seg, act="silu", out=x)
        assert y is x and torch.equal(x, want)


def _box(n, mul, seed):
    g = W.graph_inputs(n, mul, 1, 1, 1, seed=seed, dtype=np.float64)
    return {k: torch.as_tensor(g[k], device=DEV) for k in ("src", "dst", "vec", "x", "w")}


def test_layer_with_convolution_force_training(e3b):
    """conv -> group norm (SiLU, dropout) -> dropout with a residual -> energy; forces are the gradient
    with respect to the edge vectors, and a loss on them is differentiated again: directional
    central differences in float64 (step 1e-5: truncation and rounding below 1e-6 of the scale)."""
    n, mul = 400, 8
    d = _box(n, mul, seed=3)
    plan = e3b.Plan(W.irreps_str(mul, 1), W.sh_irreps(1), lmax_out=2, dtype=torch.float64)
    graph = e3b.Graph(n, d["src"], d["dst"])
    f = e3b.Features(plan.irreps_out, groups=2, dtype=torch.float64)
    seg = e3b.Segments.from_counts([150, 60, 190])
    gen = torch.Generator(DEV).manual_seed(2)
    rnd = lambda *s: torch.randn(s, device=DEV, dtype=torch.float64, generator=gen)
    vec = graph.to_receiver_order(d["vec"])
    wts = rnd(d["src"].shape[0], plan.weight_numel)
    gamma, beta = 1 + 0.2 * rnd(f.n_channels), 0.2 * rnd(f.n_scalars)
    readout, target = rnd(n, f.dim), rnd(d["src"].shape[0], 3)

    def forces(x, v, gm, bt, create):
        h = e3b.conv(plan, graph, x, e3b.sh(1, v), wts, out_scale=0.2)
        y = e3b.group_norm(f, h, gm, bt, segments=seg, act="silu", p=0.2, rng=(8, 1))
        z = e3b.dropout(f, y, 0.1, (8, 2), residual=h)
        energy = (torch.tanh(z) * readout).sum()
        (fv,) = torch.autograd.grad(energy, v, create_graph=create)
        return energy, fv

    def loss(x, v, gm, bt, create=False):
        v = v.requires_grad_(True)
        energy, fv = forces(x, v, gm, bt, create=True)
        return energy + ((fv - target) ** 2).sum() * 0.01

    args = [d["x"].clone(), vec.clone(), gamma, beta]
    leaves = [a.clone().requires_grad_(True) for a in args]
    grads = torch.autograd.grad(loss(*leaves), leaves)
    for i in range(4):
        u = rnd(*args[i].shape)
        h = 1e-5
        num = []
        for sgn in (1, -1):
            moved = [a.clone() for a in args]
            moved[i] = moved[i] + sgn * h * u
            num.append(float(loss(*moved).detach()))
        want, got = (num[0] - num[1]) / (2 * h), float((grads[i] * u).sum())
        assert abs(got - want) <= 1e-5 * max(1.0, abs(want), float(grads[i].abs().max())), i
    e3b.device_status()


def test_gradients_that_start_off_a_vector_boundary(e3b):
    """The gradient of a concatenation is a slice that starts anywhere: 6 floats into a buffer here."""
    f = e3b.Features("3x0e+1x1o")
    gen = torch.Generator(DEV).manual_seed(4)
    first, x, res = (torch.randn(n, f.dim, device=DEV, generator=gen, requires_grad=True) for n in (1, 5, 5))
    coef = torch.randn(6, f.dim, device=DEV, generator=gen)

    def run(op, join):
        y = op()
        loss = (torch.cat([first, y]) * coef).sum() if join else (y * coef[1:].clone()).sum()
        (gx,) = torch.autograd.grad(loss + (y ** 2).sum(), x, create_graph=True)
        return gx.detach(), torch.autograd.grad((torch.cat([first, gx]) * coef).sum() if join
                                                else (gx * coef[1:].clone()).sum(), x, allow_unused=True)[0]

    for op in (lambda: e3b.group_norm(f, x, act="silu"), lambda: e3b.dropout(f, x, 0.3, 5, residual=res)):
        for got, want in zip(run(op, True), run(op, False)):
            assert torch.equal(got, want)
    y = e3b.group_norm(f, x)
    (gx,) = torch.autograd.grad((torch.cat([first, y]) * coef).sum(), x)  # the slice itself, added to nothing
    want, _, _ = e3b.group_norm_backward(f, x.detach(), e3b.group_norm_forward(f, x.detach())[1], coef[1:].clone())
    assert torch.equal(gx, want)
