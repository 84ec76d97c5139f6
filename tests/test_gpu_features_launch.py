"""Launch forms and rare calls of the feature-row operators: what a captured call launches, sums of many rows,
extreme values, parameters anywhere in memory, rows beyond 32-bit offsets in every kernel.

Tolerances are in half steps of the type (2^-24 for float32) times the sum of the absolute values of the terms
that make up an output, unless a test derives its own."""

import ctypes

import numpy as np
import pytest
import torch

import oracle
from test_gpu_features import _check_all, _close

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def e3b():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from mlip_message_passing_b200 import e3b
    return e3b


def _kernel_nodes(graph):
    """(cooperative, CTAs of a cluster) of every kernel node of a captured graph, by the driver's graph calls."""
    cu = ctypes.CDLL("libcuda.so.1")
    handle = ctypes.c_void_p(graph.raw_cuda_graph())
    n = ctypes.c_size_t()
    assert cu.cuGraphGetNodes(handle, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert cu.cuGraphGetNodes(handle, nodes, ctypes.byref(n)) == 0
    out = []
    for node in nodes:
        kind = ctypes.c_int()
        assert cu.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        if kind.value != 0:  # a kernel
            continue
        value = {}
        for attr in (2, 4):  # cooperative, cluster dimension
            v = (ctypes.c_uint * 16)()
            assert cu.cuGraphKernelNodeGetAttribute(ctypes.c_void_p(node), attr, v) == 0
            value[attr] = list(v)
        x, y, z = value[4][:3]
        out.append((bool(value[2][0]), max(1, x) * max(1, y) * max(1, z)))
    return out


@pytest.mark.parametrize("irreps,groups,counts", [
    ("32x0e+16x1o+8x2e", 4, [40, 0, 80]), ("16x0e+8x1o", 2, [300, 170]), ("64x0e+64x1o+64x2e", 8, [700])])
def test_clusters_do_not_meet_across_the_grid(e3b, irreps, groups, counts):
    """Segments held by clusters: the call is captured and not run, and no launch has both a cluster dimension
    and the right to a grid barrier."""
    f, seg = e3b.Features(irreps, groups=groups), e3b.Segments.from_counts(counts)
    n = sum(counts)
    x, g, u = (torch.zeros(n, f.dim, device=DEV) for _ in range(3))
    stats = torch.zeros(len(counts), f.n_groups, 2, dtype=torch.float64, device=DEV)
    e3b.group_norm_forward(f, x[:0].contiguous())  # sets the device's status word up
    kw = dict(segments=seg, act="silu")
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        e3b.group_norm_forward(f, x, **kw)
        e3b.group_norm_backward(f, x, stats, g, **kw)
        e3b.group_norm_double_backward(f, x, stats, g, u_x=u, **kw)
    nodes = _kernel_nodes(graph)
    assert len(nodes) == 3 and sum(cluster > 1 for _, cluster in nodes) >= 2, nodes
    assert not any(coop and cluster > 1 for coop, cluster in nodes), nodes
    del graph


def test_clusters_share_a_tile(e3b):
    """Several clusters to a tile leave their column sums and the last to come adds them: the same bits in every
    run, on two streams at once and in a replayed graph, and the oracle's values."""
    irreps, groups, counts = "16x0e+8x1o", 2, [300, 0, 170, 450]
    f, seg = e3b.Features(irreps, groups=groups), e3b.Segments.from_counts(counts)
    n = sum(counts)
    rng = np.random.default_rng(2)
    xn, gn, un = (rng.standard_normal((n, f.dim)).astype(np.float32) for _ in range(3))
    x, g, u = (torch.as_tensor(t, device=DEV) for t in (xn, gn, un))
    kw = dict(segments=seg, act="silu", p=0.2, rng=(6, 1))

    def run():
        _, st = e3b.group_norm_forward(f, x, **kw)
        return (*e3b.group_norm_backward(f, x, st, g, **kw), *e3b.group_norm_double_backward(f, x, st, g, u_x=u, **kw))

    want = run()
    okw = dict(act="silu", factor=oracle.dropout_factor(irreps, n, 0.2, 6, 1), scale=True)
    ptr = np.concatenate([[0], np.cumsum(counts)])
    first = oracle.group_norm_backward(irreps, groups, ptr, xn, gn, **okw)
    second = oracle.group_norm_double_backward(irreps, groups, ptr, xn, gn, u_x=un, **okw)
    # 96 and 288: a thread's float sums of at most 64 rows (of four columns) and at most 32 pointwise roundings
    for got, ref, size, steps in (*((want[i], first[i], first[i + 3], 96) for i in range(3)),
                                  *((want[i + 3], second[i], second[i + 4], 288) for i in range(4))):
        assert (np.abs(got.cpu().double().numpy() - ref) <= steps * 2.0 ** -24 * size + 1e-30).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = run()
    side = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        res = []
        for s in side:
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                res.append(run())
        for s in side:
            torch.cuda.current_stream().wait_stream(s)
        graph.replay()
        res.append(kept)
        torch.cuda.synchronize()
        for r in res:
            assert all(torch.equal(a, b) for a, b in zip(r, want))
    e3b.device_status()
    del graph


@pytest.mark.parametrize("irreps,groups", [("512x0e", 512), ("256x0e+256x0o", 256), ("1024x0e", 1024),
                                           ("+".join(["16x0o"] * 32), 16), ("+".join(["100x0e"] * 5), 100)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float64])
def test_one_row_segments_of_many_groups(e3b, irreps, groups, dtype):
    """Hundreds of one-column groups to a tile: the coefficients of a batch have to fit shared memory."""
    _check_all(e3b, irreps, groups, [1] * 20, 3, dtype, "silu", 0.1, seed=6)


def test_parameter_gradients_of_segments_that_take_turns(e3b):
    """5032 segments of 64 rows, whose rows take a thread's slots in turns: the weight gradients of a column are sums of
    N equal terms t = 1 + 2^-16 (1 - 2^-6).  A float32 sum of them drops 2^-16 of every term once it is above 256, so a
    thread that went on for more than 64 rows before its sums go to double would be off by up to 180 half steps.
    With 64 rows it is off by 64 half steps at most, and by 32 for the pointwise part."""
    irreps, B = "85x1o", 5032
    f, seg = e3b.Features(irreps), e3b.Segments.from_counts([64] * B)
    n, t = 64 * B, 1 + 2.0 ** -16 * (1 - 2.0 ** -6)
    one = torch.ones(n, f.dim, device=DEV)
    x = one.clone()
    x[1::2] = -1  # sums of z u vanish, z = x: the mean square is 1
    kw = dict(segments=seg, act=None)
    _, stats = e3b.group_norm_forward(f, x, eps=1e-30, segments=seg)
    bound = (64 + 32) * 2.0 ** -24 * n * 3 * t  # a channel has three columns
    _, gw, _ = e3b.group_norm_backward(f, x, stats, x * t, need_x=False, **kw)
    assert float((gw.double() - n * 3 * t).abs().max()) <= bound
    _, _, dw, _ = e3b.group_norm_double_backward(f, x, stats, one * t, u_x=one, **kw)
    assert float((dw.double() - n * 3 * t).abs().max()) <= bound
    e3b.device_status()


def test_eps_that_vanishes_in_the_rows_type_is_refused(e3b):
    """1e-50 is 0 as a float32 and 1e39 infinite: a constant group would become NaN.  float64 rows take both."""
    for dtype in (torch.float32, torch.float64):
        f = e3b.Features("8x0e+8x1o", groups=2, dtype=dtype)
        x = torch.zeros(10, 32, device=DEV, dtype=dtype)
        for eps in (1e-50, 1e39):
            if dtype is torch.float32:
                with pytest.raises(e3b.E3Error) as err:
                    e3b.group_norm_forward(f, x, eps=eps)
                assert err.value.status == e3b.E3_ERR_INVALID_ARG
            else:
                assert not bool(e3b.group_norm_forward(f, x, eps=eps)[0].any())
        y, _ = e3b.group_norm_forward(f, x, eps=1e-44)  # a subnormal float32 number
        assert not bool(y.any())


@pytest.mark.parametrize("counts,hint", [([10, 10, 10], "max"), ([10, 10, 10], 0), ([1] * 30, "max"), ([30], "max")])
def test_infinite_mean_square_gives_zero(e3b, counts, hint):
    """A value whose square no float32 holds: r = 1 / sqrt(inf) = 0, so its group is t = bias, not NaN, and takes no
    part in the gradients; the other groups are what they are without it."""
    f, seg = e3b.Features("8x0e+8x1o", groups=2), e3b.Segments.from_counts(counts)
    if hint != "max":
        seg.max_rows = hint
    gen = torch.Generator(DEV).manual_seed(1)
    x, g, u = (torch.randn(30, 32, device=DEV, generator=gen) for _ in range(3))
    b = torch.randn(8, device=DEV, generator=gen)
    big = x.clone()
    big[4, 1] = 1e25    # scalars, first group
    big[4, 20] = -1e25  # vectors, second group
    first = next(i for i, e in enumerate(np.cumsum(counts)) if e > 4)
    lo, hi = sum(counts[:first]), sum(counts[:first + 1])
    bad = torch.zeros(30, 32, dtype=torch.bool, device=DEV)
    bad[lo:hi, :4] = True
    bad[lo:hi, 20:] = True
    out = []
    for src in (x, big):
        y, st = e3b.group_norm_forward(f, src, None, b, segments=seg)
        gx = e3b.group_norm_backward(f, src, st, g, None, b, segments=seg)[0]
        dg, dx, _, _ = e3b.group_norm_double_backward(f, src, st, g, None, b, u_x=u, segments=seg)
        out.append((y, gx, dg, dx))
    for a, c in zip(*out):
        assert torch.equal(a[~bad], c[~bad])
    y, gx, dg, dx = out[1]
    assert torch.equal(y[lo:hi, :4], b[:4].expand(hi - lo, 4)) and not bool(y[lo:hi, 20:].any())
    for t in (gx, dg, dx):
        assert not bool(t[bad].any())
    e3b.device_status()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float64])
def test_parameters_anywhere_in_a_flat_buffer(e3b, dtype):
    """Weights, biases and their upstream gradients are slices of one buffer that start off every vector boundary."""
    f, seg = e3b.Features("5x0e+3x1o", dtype=dtype), e3b.Segments.from_counts([4, 0, 9])
    gen = torch.Generator(DEV).manual_seed(1)
    flat = torch.randn(60, device=DEV, dtype=dtype, generator=gen)
    w, b, uw, ub = flat[1:9], flat[9:14], flat[23:31], flat[31:36]
    x, g, u = (torch.randn(13, f.dim, device=DEV, dtype=dtype, generator=gen) for _ in range(3))

    def run(w, b, uw, ub):
        y, st = e3b.group_norm_forward(f, x, w, b, segments=seg, act="silu")
        return (y, *e3b.group_norm_backward(f, x, st, g, w, b, segments=seg, act="silu"),
                *e3b.group_norm_double_backward(f, x, st, g, w, b, u, uw, ub, segments=seg, act="silu"))

    for got, want in zip(run(w, b, uw, ub), run(*(t.clone() for t in (w, b, uw, ub)))):
        assert torch.equal(got, want)
    leaf = flat.clone().requires_grad_(True)
    y = e3b.group_norm(f, x, leaf[1:9], leaf[9:14], segments=seg, act="silu")
    (grad,) = torch.autograd.grad(y, leaf, g)
    _, st = e3b.group_norm_forward(f, x, w, b, segments=seg, act="silu")
    _, gw, gb = e3b.group_norm_backward(f, x, st, g, w, b, segments=seg, act="silu")
    want = torch.zeros_like(flat)
    want[1:9], want[9:14] = gw, gb
    assert torch.equal(grad, want)


def test_first_row_beyond_32_bits_is_refused(e3b):
    """row0 near 2^63 (where row0 + N overflows) and past 64 bits: not a mask of another row."""
    f = e3b.Features("8x0e")
    x = torch.ones(10, 8, device=DEV)
    for call in (lambda r: e3b.dropout_forward(f, x, 0.5, 1, row0=r),
                 lambda r: e3b.group_norm_forward(f, x, p=0.5, rng=1, row0=r)):
        for row0 in (2 ** 63 - 1, 2 ** 63 - 10, 2 ** 32 - 9, 2 ** 32, -1, -2 ** 63):
            with pytest.raises(e3b.E3Error) as err:
                call(row0)
            assert err.value.status == e3b.E3_ERR_SHAPE
        for row0 in (2 ** 63, 2 ** 64, 2 ** 64 + 5, -2 ** 63 - 1):
            with pytest.raises(ValueError):
                call(row0)
        call(2 ** 32 - 10)


def test_bad_row_pointers_of_the_longest_arrays(e3b):
    """N = 2^31 - 65536 rows and pointers beyond them: a segment's clamped end stays inside [0, N], though start plus
    the rows that a cluster holds (65536) passes 2^31."""
    f, n = e3b.Features("1x0e"), 2 ** 31 - 65536
    x = torch.zeros(n, 1, device=DEV)
    ptr = torch.tensor([0, 2 ** 31 - 1, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    y, _ = e3b.group_norm_forward(f, x, segments=e3b.Segments(ptr, n, max_rows=65536))
    with pytest.raises(e3b.E3Error) as err:
        e3b.device_status()
    assert err.value.status == e3b.E3_ERR_INDEX
    assert not bool(y[:65536].any())
    del x, y
    torch.cuda.empty_cache()


def test_row_pointer_that_changed_before_the_backward_is_refused(e3b):
    """A row pointer in a buffer that the next batch overwrites: the gradient of the earlier batch would be taken over
    other segments.  Both derivatives refuse it."""
    f = e3b.Features("8x0e+4x1o", groups=2)
    gen = torch.Generator(DEV).manual_seed(4)
    x, g = (torch.randn(30, f.dim, device=DEV, generator=gen) for _ in range(2))
    ptr = torch.tensor([0, 10, 30], dtype=torch.int32, device=DEV)
    seg = e3b.Segments(ptr, 30, max_rows=20)
    for second in (False, True):
        leaf = x.clone().requires_grad_(True)
        y = e3b.group_norm(f, leaf, segments=seg, act="silu")
        if second:
            (y,) = torch.autograd.grad(y, leaf, g, create_graph=True)
        ptr[1] = 12
        with pytest.raises(RuntimeError):
            torch.autograd.grad(y, leaf, g)
        ptr[1] = 10


def test_generator_list_that_counts_on(e3b):
    """rng as a list [seed, offset] that the caller advances after the call: the backward drops what the forward did."""
    f = e3b.Features("8x0e+4x1o", groups=2)
    gen = torch.Generator(DEV).manual_seed(4)
    x, g = (torch.randn(30, f.dim, device=DEV, generator=gen) for _ in range(2))
    for op in (lambda t, rng: e3b.dropout(f, t, 0.5, rng), lambda t, rng: e3b.group_norm(f, t, p=0.5, rng=rng)):
        grads = []
        for rng in ([3, 0], (3, 0)):
            leaf = x.clone().requires_grad_(True)
            y = op(leaf, rng)
            if isinstance(rng, list):
                rng[1] += 1
            grads.append(torch.autograd.grad(y, leaf, g)[0])
        assert torch.equal(*grads)


def test_tiles_that_end_inside_a_channel(e3b):
    """Long segments of 2048 columns: two tiles of 1024, and column 1024 is one of channel 102 of the 2e block."""
    _check_all(e3b, "128x0e+128x1o+128x2e+128x3o", 16, [300, 0, 40], 2, torch.float32, "silu", 0.0, seed=8, hint=0)


def _gradient_sizes(irreps, groups, counts, t, act, factor):
    """float64 weight and bias gradients of the norm's first and second derivative, and the size of each on which
    rounding acts: the same sums with every term replaced by the sum of its parts' absolute values.  (The activation's
    derivatives are products of the sigmoid, below 1, with 1 + t (1 - s) and 2 + t (1 - 2 s).)"""
    seg = torch.repeat_interleave(torch.arange(len(counts), device=DEV), torch.tensor(counts, device=DEV))
    n = torch.tensor(counts, device=DEV, dtype=torch.float64).clamp(min=1)
    out, ch, sc = {k: [] for k in ("gw", "gb", "dw", "db", "gw_", "gb_", "dw_", "db_")}, 0, 0
    col = 0
    for ir in oracle.parse_irreps(irreps):
        d, scalar = 2 * ir.l + 1, ir.l == 0 and ir.p == 1
        take = lambda v: v[:, col:col + ir.mul * d].reshape(v.shape[0], groups, -1, d)
        chan = lambda v, first: v[first:first + ir.mul].reshape(1, groups, -1, 1)

        def mean(v):
            s = torch.zeros(len(counts), groups, device=DEV, dtype=torch.float64)
            s.index_add_(0, seg, v.sum(dim=(2, 3)))
            return (s / (n * (ir.mul // groups * d))[:, None])[seg][:, :, None, None]

        x, g, u, m = take(t["x"]), take(t["g"]), take(t["ux"]), take(factor)
        w, uw = chan(t["w"], ch), chan(t["uw"], ch)
        b, ub = (chan(t[k], sc) if scalar else torch.zeros(1, 1, 1, 1, device=DEV, dtype=torch.float64) for k in ("b", "ub"))
        mu = mean(x) if scalar else 0 * mean(x)
        r = torch.rsqrt(mean((x - mu) ** 2) + 1e-5)
        z, za = (x - mu) * r, (x.abs() + mu.abs()) * r
        tt, ta = w * z + b, w.abs() * za + b.abs()
        on = scalar and act
        s = torch.sigmoid(tt)
        d1, d2 = (s * (1 + tt * (1 - s)), s * (1 - s) * (2 + tt * (1 - 2 * s))) if on else (1.0, 0.0)
        h, ha = m * g * d1, m * g.abs() * ((1 + ta) if on else 1.0)
        m1, m1a = (mean(u), mean(u.abs())) if scalar else (0.0, 0.0)
        zd, zda = r * (u - m1 - z * mean(z * u)), r * (u.abs() + m1a + za * mean(za * u.abs()))
        td, tda = w * zd + uw * z + ub, w.abs() * zda + uw.abs() * za + ub.abs()
        q, qa = m * g * d2 * td, m * g.abs() * ((2 + ta) if on else 0.0) * tda
        add = lambda v: v.expand(x.shape).sum(dim=(0, 3)).reshape(-1)
        for k, v in (("gw", h * z), ("gw_", ha * za), ("dw", q * z + h * zd), ("dw_", qa * za + ha * zda)):
            out[k].append(add(v))
        if scalar:
            for k, v in (("gb", h), ("gb_", ha), ("db", q), ("db_", qa)):
                out[k].append(add(v))
        ch, sc, col = ch + ir.mul, sc + (ir.mul if scalar else 0), col + ir.mul * d
    return {k: torch.cat(v) for k, v in out.items()}


@pytest.mark.parametrize("irreps,groups", [("64x0e+64x1o+64x2e", 8), ("40x0e+40x1o", 4), ("25x0e+7x0o+11x1o+5x2e", 1)])
@pytest.mark.parametrize("act,p", [(None, 0.0), ("silu", 0.2)])
def test_parameter_gradients_of_many_segments(e3b, irreps, groups, act, p):
    """More segments than blocks, and tiles with different numbers of blocks: every block's column sums have to come
    in.  96 half steps of the terms' absolute values for the first derivative (64 rows of a thread in float32, at most
    32 pointwise roundings), 288 for the second (four columns to a thread's group sums).  One block's share, some 27
    of 8000 rows, has a signed sum of about 5 in 6400: 8e-4, against 6e-6 and 1.7e-5."""
    counts = [1 + i % 7 for i in range(2000)]
    N = sum(counts)
    f = e3b.Features(irreps, groups=groups)
    seg = e3b.Segments.from_counts(counts)
    gen = torch.Generator(DEV).manual_seed(5)
    t = {k: torch.randn(*s, device=DEV, generator=gen) for k, s in
         (("x", (N, f.dim)), ("g", (N, f.dim)), ("ux", (N, f.dim)), ("w", (f.n_channels,)), ("b", (f.n_scalars,)),
          ("uw", (f.n_channels,)), ("ub", (f.n_scalars,)))}
    kw = dict(segments=seg, act=act, p=p, rng=(3, 1) if p else None)
    _, st = e3b.group_norm_forward(f, t["x"], t["w"], t["b"], **kw)
    got = dict(zip(("gw", "gb"), e3b.group_norm_backward(f, t["x"], st, t["g"], t["w"], t["b"], **kw)[1:]))
    got.update(zip(("dw", "db"), e3b.group_norm_double_backward(f, t["x"], st, t["g"], t["w"], t["b"], t["ux"], t["uw"],
                                                                t["ub"], **kw)[2:]))
    wide = e3b.Features(irreps, dtype=torch.float64)
    factor = torch.ones(N, f.dim, device=DEV, dtype=torch.float64)
    if p:
        factor = e3b.dropout_forward(wide, factor, p, (3, 1))
    ref = _gradient_sizes(irreps, groups, counts, {k: v.double() for k, v in t.items()}, act, factor)
    for k, steps in (("gw", 96), ("gb", 96), ("dw", 288), ("db", 288)):
        worst = float(((got[k].double() - ref[k]).abs() / (steps * 2.0 ** -24 * ref[k + "_"] + 1e-30)).max())
        assert worst <= 1, (k, worst)
    e3b.device_status()


@pytest.mark.parametrize("rows", [1, 25])
def test_short_segments_beyond_32_bit_offsets(e3b, rows):
    """1.1 M rows of 2048 columns (2.25e9 values) in one-row segments and in segments of 25 rows: the kernels that
    hold a segment in one block, all three forms.  The last segments against the oracle."""
    irreps, N, last = "128x0e+128x1o+128x2e+128x3o", 1_100_000, 25
    f = e3b.Features(irreps, groups=16)
    seg = e3b.Segments(torch.arange(0, N + 1, rows, dtype=torch.int32, device=DEV), N, max_rows=rows)

    def fill(seed):
        t = torch.empty(N, f.dim, device=DEV)
        for a in range(0, N, 100_000):
            t[a:a + 100_000].normal_(generator=torch.Generator(DEV).manual_seed(a + seed))
        return t

    x, g, u = fill(0), fill(1), fill(2)
    xn, gn, un = (t[N - last:].cpu().numpy() for t in (x, g, u))
    ptr = np.arange(0, last + 1, rows)
    kw = dict(segments=seg, act="silu", p=0.5, rng=(3, 1))
    okw = dict(act="silu", factor=oracle.dropout_factor(irreps, last, 0.5, 3, 1, row0=N - last), scale=True)
    y, st = e3b.group_norm_forward(f, x, **kw)
    _close(y[N - last:], *oracle.group_norm(irreps, 16, ptr, xn, **okw), 96, torch.float32, "y")
    del y
    gx, _, _ = e3b.group_norm_backward(f, x, st, g, **kw)
    ref = oracle.group_norm_backward(irreps, 16, ptr, xn, gn, **okw)
    _close(gx[N - last:], ref[0], ref[3], 96, torch.float32, "gx")
    del gx
    dg, dx, _, _ = e3b.group_norm_double_backward(f, x, st, g, u_x=u, **kw)
    ref = oracle.group_norm_double_backward(irreps, 16, ptr, xn, gn, u_x=un, **okw)
    for i, (got, what) in enumerate(((dg, "dg"), (dx, "dx"))):
        _close(got[N - last:], ref[i], ref[i + 4], 288, torch.float32, what)
    e3b.device_status()
    del x, g, u, st, dg, dx
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float64])
@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("hint", ["max", 0])
def test_groups_of_one_scalar_have_no_gradient(e3b, dtype, act, hint):
    """One-row segments, one 0e channel to a group: z = 0 whatever x is, so the first derivative is 0 and the second
    has none with respect to x, exactly, although r = 316 multiplies what is left of differences there.  The other
    columns are those of the oracle."""
    irreps, groups, n = "4x0e+8x1o+4x0e", 4, 300
    f, seg = e3b.Features(irreps, groups=groups, dtype=dtype), e3b.Segments.from_counts([1] * n)
    if hint != "max":
        seg.max_rows = hint
    gen = torch.Generator(DEV).manual_seed(7)
    x, g, u = (torch.randn(n, f.dim, device=DEV, dtype=dtype, generator=gen) for _ in range(3))
    w, b, uw, ub = (torch.randn(k, device=DEV, dtype=dtype, generator=gen) for k in (f.n_channels, f.n_scalars) * 2)
    kw = dict(segments=seg, act=act)
    y, st = e3b.group_norm_forward(f, x, w, b, **kw)
    gx, _, _ = e3b.group_norm_backward(f, x, st, g, w, b, **kw)
    scalar = torch.ones(f.dim, dtype=torch.bool, device=DEV)
    scalar[4:28] = False
    assert not bool(gx[:, scalar].any())
    for ups in (dict(u_x=u), dict(u_x=u, u_weight=uw, u_bias=ub), dict(u_weight=uw, u_bias=ub)):
        dg, dx, _, _ = e3b.group_norm_double_backward(f, x, st, g, w, b, **ups, **kw)
        assert not bool(dx[:, scalar].any())
        ref = oracle.group_norm_double_backward(irreps, groups, np.arange(n + 1), *(t.cpu().numpy() for t in (x, g, w, b)),
                                                act=act, scale=True, **{k: t.cpu().numpy() for k, t in ups.items()})
        _close(dg, ref[0], ref[4], 288, dtype, "dg")
        _close(dx, ref[1], ref[5], 288, dtype, "dx")
    e3b.device_status()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float64])
def test_one_row_segments_of_the_most_groups(e3b, dtype):
    """32768 one-column groups, the most that a row can have: 64 tiles of 512 for floats, more for doubles, which leave
    them to the kernel for long segments.  y = x / sqrt(x^2 + eps): at most 8 roundings, the root's step included."""
    f = e3b.Features("32768x0o", groups=32768, dtype=dtype)
    x = torch.randn(40, f.dim, device=DEV, dtype=dtype, generator=torch.Generator(DEV).manual_seed(2))
    y, st = e3b.group_norm_forward(f, x, segments=e3b.Segments.from_counts([1] * 40))
    want = x.double() / torch.sqrt(x.double() ** 2 + 1e-5)
    half = 2.0 ** -24 if dtype is torch.float32 else 2.0 ** -53
    assert float(((y.double() - want).abs() / want.abs()).max()) <= 8 * half
    gx, _, _ = e3b.group_norm_backward(f, x, st, x, segments=e3b.Segments.from_counts([1] * 40))
    # grad_x = r (c - z (c z)) with c = x, in terms of r x = y: y (1 - y^2); the difference cancels, so against y
    assert float(((gx.double() - want * (1 - want ** 2)).abs() / want.abs()).max()) <= 16 * half
    e3b.device_status()
