"""Workloads of the feature-row operators: group norm with an activation (forward, training pass,
force-training pass) and counter-based dropout.

Every case is one pass over node or edge feature rows [N, dim] in the mul_ir layout (irrep blocks
in order, inside a block [channel][component]).  ``run`` computes a pass in its plain form with
elementary torch operations, or, when the module's ``own`` is true, through the library's public
calls.  ``exact`` is the definition in float64, written on its own.

Group norm: every irrep block's channels are cut into ``groups`` groups; statistics are taken over
all rows of a segment (a structure of the batch) and all components of a group.  Even scalars (0e)
are centred, get a bias and the activation; every other irrep is only scaled by its root mean
square and a weight per channel, which keeps the result equivariant.  Rows outside every segment
(padding) give zero rows.

Dropout: one decision per (row, channel), shared by the channel's 2l+1 components, from
Philox4x32-10 (Salmon, Moraes, Dror, Shaw: "Parallel random numbers: as easy as 1, 2, 3") with
key = seed and counter (channel / 4, row, block, offset); word (channel % 4) >= floor(p 2^32) keeps
the channel and scales it by 1 / (1 - p).
"""

import math

import numpy as np
import torch

own = False

EPS = 1e-5
DTYPES = {"f32": torch.float32, "f64": torch.float64}


# ------------------------------------------------------------------------------------- cases ---

def listed():
    return [
        # one small box of 400 atoms, 64 channels of degrees 0..2: an inference step, launch latency counts
        dict(name="norm_box_fwd", op="norm_fwd", irreps="64x0e+64x1o+64x2e", groups=8, rows=400, segs=1,
             pad=0, dtype="f32", act=True, p=0.0),
        # training on a batch of molecules (ragged, padded to a fixed row count), dropout in the epilogue
        dict(name="norm_molecules_train", op="norm_train", irreps="128x0e+128x1o", groups=8, rows=17_600, segs=512,
             pad=211, dtype="f32", act=True, p=0.1),
        # training step on one water box of 3000 atoms
        dict(name="norm_waterbox_train", op="norm_train", irreps="64x0e+64x1o+64x2e", groups=8, rows=3000, segs=1,
             pad=0, dtype="f32", act=True, p=0.0),
        # inference on the large graph: 24000 atoms, 128 channels of degrees 0..3
        dict(name="norm_large_fwd", op="norm_fwd", irreps="128x0e+128x1o+128x2e+128x3o", groups=16, rows=24_000,
             segs=1, pad=0, dtype="f32", act=True, p=0.0),
        # training on the large graph with dropout in the epilogue
        dict(name="norm_large_train", op="norm_train", irreps="128x0e+128x1o+128x2e+128x3o", groups=16, rows=24_000,
             segs=1, pad=0, dtype="f32", act=True, p=0.2),
        # edge embeddings of the radial network's width, a few structures with many edges each
        dict(name="norm_edges_train", op="norm_train", irreps="64x0e", groups=8, rows=420_000, segs=6,
             pad=1000, dtype="f32", act=True, p=0.0),
        # every node normalised by itself (a layer norm of its irreps)
        dict(name="norm_nodes_fwd", op="norm_fwd", irreps="128x0e+128x1o+128x2e+128x3o", groups=1, rows=24_000,
             segs=24_000, pad=0, dtype="f32", act=False, p=0.0),
        # force training on the water box: the norm's backward is itself differentiated
        dict(name="norm_waterbox_force", op="norm_force", irreps="64x0e+64x1o+64x2e", groups=8, rows=3000, segs=1,
             pad=0, dtype="f32", act=True, p=0.0),
        # odd multiplicities in double precision, several small structures, force training
        dict(name="norm_odd_force_f64", op="norm_force", irreps="25x0e+7x0o+11x1o+5x2e", groups=1, rows=4111,
             segs=37, pad=0, dtype="f64", act=True, p=0.15),
        # dropout of a small box's rows: launch latency counts
        dict(name="dropout_box", op="dropout", irreps="64x0e+64x1o+64x2e", rows=400, dtype="f32", p=0.1,
             residual=False),
        # residual branch of a layer on the large graph
        dict(name="dropout_large_residual", op="dropout", irreps="128x0e+128x1o+128x2e+128x3o", rows=24_000,
             dtype="f32", p=0.1, residual=True),
        # dropout of edge embeddings: one decision per value
        dict(name="dropout_edges", op="dropout", irreps="64x0e", rows=1_200_000, dtype="f32", p=0.25,
             residual=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_train", "norm_force", "dropout"])
    dtype = "f64" if rng.random() < 0.25 else "f32"
    lmax = rng.randint(0, 3)
    if rng.random() < 0.35:  # odd multiplicities, one group
        groups = 1
        muls = [rng.randint(1, 80) | 1 for _ in range(lmax + 1)]
    else:
        groups = rng.choice([1, 2, 4, 8, 16])
        muls = [groups * _log_int(rng, 1, 128 // groups)] * (lmax + 1)
    parity = lambda l: "e" if l % 2 == 0 or rng.random() < 0.2 else "o"
    irreps = "+".join(f"{m}x{l}{parity(l)}" for l, m in enumerate(muls))
    dim = sum(m * (2 * l + 1) for l, m in enumerate(muls))
    limit = {"norm_fwd": 48_000_000, "norm_train": 40_000_000, "norm_force": 16_000_000, "dropout": 60_000_000}[op]
    if dtype == "f64":
        limit //= 2
    rows = _log_int(rng, 200, max(400, min(400_000, limit // dim)))
    if op == "dropout":
        return dict(op=op, irreps=irreps, rows=rows, dtype=dtype, p=round(rng.uniform(0.02, 0.6), 3),
                    residual=rng.random() < 0.5)
    segs = rng.choice([1, rng.randint(2, 12), max(1, rows // rng.randint(12, 60)), rows])
    pad = rng.choice([0, rng.randint(1, max(1, rows // 50))]) if 1 < segs < rows else 0
    return dict(op=op, irreps=irreps, groups=groups, rows=rows, segs=segs, pad=pad, dtype=dtype,
                act=rng.random() < 0.7, p=rng.choice([0.0, round(rng.uniform(0.02, 0.6), 3)]))


# ------------------------------------------------------------------------------------ inputs ---

def _blocks(irreps):
    """[(multiplicity, components, is an even scalar, first column)] of an irreps string."""
    out, col = [], 0
    for term in irreps.split("+"):
        mul, rest = term.strip().split("x")
        mul, d = int(mul), 2 * int(rest[:-1]) + 1
        out.append((mul, d, rest == "0e", col))
        col += mul * d
    return out


def _dim(irreps):
    return sum(m * d for m, d, _, _ in _blocks(irreps))


def _counts(case, seed):
    """Rows of each segment: between about 0.3 and 1.7 times the average, one of them empty."""
    B, n = case["segs"], case["rows"] - case["pad"]
    if B == 1:
        return [n]
    if B == case["rows"]:
        return [1] * B
    g = np.random.default_rng(seed)
    w = g.uniform(0.3, 1.7, B)
    if B >= 8:
        w[int(g.integers(B))] = 0.0
    edge = np.floor(np.cumsum(w) / w.sum() * n + 0.5).astype(np.int64)
    edge[-1] = n
    return np.diff(np.concatenate([[0], edge])).tolist()


def _inputs(case, seed):
    dev, dt = torch.device("cuda"), DTYPES[case["dtype"]]
    gen = torch.Generator(device=dev).manual_seed(seed)
    N, D = case["rows"], _dim(case["irreps"])

    def normal(*shape):
        return torch.randn(shape, generator=gen, dtype=dt, device=dev)

    st = dict(case=case, rng=((seed * 2654435761 + 12345) % 2 ** 62, seed % 1000), x=normal(N, D))
    if case["op"] == "dropout":
        st["residual"] = normal(N, D) if case["residual"] else None
        return st
    # features with a scale and, for the scalars, an offset per channel, as a convolution leaves them
    blocks = _blocks(case["irreps"])
    for mul, d, scalar, c0 in blocks:
        v = st["x"][:, c0:c0 + mul * d].view(N, mul, d)
        v *= torch.exp(0.5 * normal(mul, 1))
        if scalar:
            v += normal(mul, 1)
    n_ch, n_sc = sum(b[0] for b in blocks), sum(b[0] for b in blocks if b[2])
    st["weight"] = 1.0 + 0.2 * normal(n_ch)
    st["bias"] = 0.2 * normal(n_sc)
    if case["op"] != "norm_fwd":
        st["g"] = normal(N, D)
    if case["op"] == "norm_force":
        st["ux"] = normal(N, D)
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    norm, dt = case["op"] != "dropout", DTYPES[case["dtype"]]
    counts = _counts(case, seed) if norm else None
    if own:
        from mlip_message_passing_b200 import e3b
        st["features"] = e3b.Features(case["irreps"], groups=case["groups"] if norm else 1, dtype=dt)
        if norm:
            one = len(counts) == 1 and not case["pad"]
            st["segments"] = None if one else e3b.Segments.from_counts(counts, n_rows=case["rows"])
    elif norm:
        st["n"] = torch.tensor(counts, dtype=torch.int64, device="cuda")
        st["seg"] = torch.repeat_interleave(torch.arange(len(counts), device="cuda"), st["n"])
    return st


# ------------------------------------------------------------------------------- plain forms ---

M0, M1, W0, W1, MASK = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85, 0xFFFFFFFF


def _keep(irreps, rows, p, rng, device):
    """Per block, the [rows, channels] truth values of the channels that stay."""
    seed, offset = rng
    thr = math.floor(p * 2.0 ** 32)
    out = []
    for b, (mul, _, _, _) in enumerate(_blocks(irreps)):
        quads = (mul + 3) // 4
        c0 = torch.arange(quads, device=device).expand(rows, quads)
        c1 = torch.arange(rows, device=device)[:, None].expand(rows, quads)
        c2 = torch.full((rows, quads), b, device=device)
        c3 = torch.full((rows, quads), offset & MASK, device=device)
        k0, k1 = seed & MASK, (seed >> 32) & MASK
        for _ in range(10):
            p0, p1 = c0 * M0, c2 * M1  # low 64 bits; the shifted high half is masked
            c0, c1, c2, c3 = ((p1 >> 32) & MASK) ^ c1 ^ k0, p1 & MASK, ((p0 >> 32) & MASK) ^ c3 ^ k1, p0 & MASK
            k0, k1 = (k0 + W0) & MASK, (k1 + W1) & MASK
        out.append(torch.stack([c0, c1, c2, c3], dim=-1).reshape(rows, 4 * quads)[:, :mul] >= thr)
    return out


def _plain_dropout(st):
    case, x = st["case"], st["x"]
    out = torch.empty_like(x)
    scale = 1.0 / (1.0 - case["p"])
    for (mul, d, _, c0), keep in zip(_blocks(case["irreps"]), _keep(case["irreps"], x.shape[0], case["p"], st["rng"],
                                                                  x.device)):
        v = x[:, c0:c0 + mul * d].reshape(-1, mul, d)
        r = torch.where(keep[:, :, None], v * scale, torch.zeros_like(v)).reshape(-1, mul * d)
        out[:, c0:c0 + mul * d] = r if st["residual"] is None else r + st["residual"][:, c0:c0 + mul * d]
    return out


def _sigmoid(t):
    return 1.0 / (1.0 + torch.exp(-t))


class _Block:
    """One irrep block of a group-norm pass: [rows, groups, channels, components] views and the
    segment means."""

    def __init__(self, st, mul, d, scalar, c0):
        self.case, self.st = st["case"], st
        self.mul, self.d, self.scalar, self.c0 = mul, d, scalar, c0
        self.seg, self.rows = st["seg"], st["seg"].shape[0]
        self.groups = self.case["groups"]
        self.size = (st["n"] * (mul * d // self.groups)).clamp(min=1).to(torch.float64)[:, None]

    def take(self, t):
        return t[:self.rows, self.c0:self.c0 + self.mul * self.d].reshape(self.rows, self.groups, -1, self.d)

    def put(self, out, t):
        out[:self.rows, self.c0:self.c0 + self.mul * self.d] = t.reshape(self.rows, -1)

    def mean(self, t):
        """Mean over a segment's rows and a group's values, spread back over the rows; long sums in 64 bits."""
        s = torch.zeros((self.st["n"].shape[0], self.groups), dtype=torch.float64, device=t.device)
        s.index_add_(0, self.seg, t.sum(dim=(2, 3)).to(torch.float64))
        return (s / self.size).to(t.dtype)[self.seg][:, :, None, None]

    def channel(self, v, first):
        return v[first:first + self.mul].reshape(1, self.groups, -1, 1)

    def center(self, t):
        return t - self.mean(t) if self.scalar else t


def _plain_norm(st):
    case, x, w, b = st["case"], st["x"], st["weight"], st["bias"]
    y = torch.zeros_like(x)
    train, force = case["op"] == "norm_train", case["op"] == "norm_force"
    gx, dg, dx = (torch.zeros_like(x) for _ in range(3)) if train or force else (None,) * 3
    gw, gb = torch.zeros_like(w), torch.zeros_like(b)
    keeps = _keep(case["irreps"], x.shape[0], case["p"], st["rng"], x.device) if case["p"] > 0 else None
    ch = sc = 0
    for i, (mul, d, scalar, c0) in enumerate(_blocks(case["irreps"])):
        B = _Block(st, mul, d, scalar, c0)
        xc = B.center(B.take(x))
        r = torch.rsqrt(B.mean(xc * xc) + EPS)
        z = xc * r
        gamma = B.channel(w, ch)
        t = gamma * z + (B.channel(b, sc) if scalar else 0.0)
        act = scalar and case["act"]
        s = _sigmoid(t) if act else None
        m = 1.0
        if keeps is not None:
            k = keeps[i][:B.rows].reshape(B.rows, B.groups, -1, 1)
            m = k.to(x.dtype) * (1.0 / (1.0 - case["p"]))
        B.put(y, m * (t * s if act else t))
        if train or force:
            d1 = s * (1.0 + t * (1.0 - s)) if act else 1.0
            g = B.take(st["g"])
            h = m * g * d1
            c = gamma * h
            mcz = B.mean(c * z)
            B.put(gx, r * (B.center(c) - z * mcz))
            if train:
                gw[ch:ch + mul] = (h * z).sum(dim=(0, 3)).reshape(-1)
                if scalar:
                    gb[sc:sc + mul] = h.sum(dim=(0, 3)).reshape(-1)
        if force:
            u = B.take(st["ux"])
            m2 = B.mean(z * u)
            zd = r * (B.center(u) - z * m2)
            td = gamma * zd
            B.put(dg, m * d1 * td)
            q = m * g * (s * (1.0 - s) * (2.0 + t * (1.0 - 2.0 * s))) * td if act else torch.zeros_like(td)
            C = gamma * q - r * m2 * c - r * mcz * u
            B.put(dx, r * (B.center(C) - z * B.mean(z * C)) - r * z * B.mean(c * zd))
            gw[ch:ch + mul] = (q * z + h * zd).sum(dim=(0, 3)).reshape(-1)
            if scalar:
                gb[sc:sc + mul] = q.sum(dim=(0, 3)).reshape(-1)
        ch += mul
        sc += mul if scalar else 0
    if train:
        return y, gx, gw, gb
    if force:
        return y, gx, dg, dx, gw, gb
    return y


def _own_norm(st):
    from mlip_message_passing_b200 import e3b
    case, f, x, w, b = st["case"], st["features"], st["x"], st["weight"], st["bias"]
    kw = dict(segments=st["segments"], act="silu" if case["act"] else None, p=case["p"],
              rng=st["rng"] if case["p"] > 0 else None)
    y, stats = e3b.group_norm_forward(f, x, w, b, eps=EPS, **kw)
    if case["op"] == "norm_fwd":
        return y
    if case["op"] == "norm_train":
        gx, gw, gb = e3b.group_norm_backward(f, x, stats, st["g"], w, b, **kw)
        return y, gx, gw, gb
    gx, _, _ = e3b.group_norm_backward(f, x, stats, st["g"], w, b, need_weight=False, need_bias=False, **kw)
    dg, dx, gw, gb = e3b.group_norm_double_backward(f, x, stats, st["g"], w, b, u_x=st["ux"], **kw)
    return y, gx, dg, dx, gw, gb


def run(state):
    if state["case"]["op"] == "dropout":
        if own:
            from mlip_message_passing_b200 import e3b
            return e3b.dropout_forward(state["features"], state["x"], state["case"]["p"], state["rng"],
                                       residual=state["residual"])
        return _plain_dropout(state)
    return _own_norm(state) if own else _plain_norm(state)


# -------------------------------------------------------------------------------------- work ---

def work(case):
    size = 4 if case["dtype"] == "f32" else 8
    blocks = _blocks(case["irreps"])
    n = case["rows"] * _dim(case["irreps"])
    params = sum(b[0] for b in blocks) + sum(b[0] for b in blocks if b[2])
    scalars = case["rows"] * sum(m for m, _, s, _ in blocks if s) if case.get("act") else 0
    # a generator call (10 rounds of 2 products and 4 exclusive ors) serves four channels
    random = case["rows"] * sum((b[0] + 3) // 4 for b in blocks) * 60 if case["p"] > 0 else 0
    if case["op"] == "dropout":
        return {"bytes": n * size * (3 if case["residual"] else 2), "flops": n * 2 + random}
    # arrays read and written, operations a value, operations a scalar's activation and derivatives
    arrays, per, act = {"norm_fwd": (2, 8, 5), "norm_train": (4, 22, 18), "norm_force": (7, 60, 40)}[case["op"]]
    extra = {"norm_fwd": 1, "norm_train": 2, "norm_force": 2}[case["op"]]
    return {"bytes": n * size * arrays + params * size * extra, "flops": n * per + scalars * act + random}


# ------------------------------------------------------------------------------------- exact ---

def _exact_factor(irreps, rows, p, rng):
    """[rows, dim] float64 dropout factors, the generator in unsigned 32-bit words on the host."""
    seed, offset = rng
    u32, u64 = np.uint32, np.uint64
    cols = []
    for b, (mul, d, _, _) in enumerate(_blocks(irreps)):
        quads = -(-mul // 4)
        words = np.empty((rows, quads, 4), dtype=u32)
        step = max(1, (1 << 16) // quads)
        for r0 in range(0, rows, step):
            r1 = min(rows, r0 + step)
            ctr = [np.broadcast_to(np.arange(quads, dtype=u32), (r1 - r0, quads)),
                   np.broadcast_to(np.arange(r0, r1, dtype=u32)[:, None], (r1 - r0, quads)),
                   np.full((r1 - r0, quads), b, dtype=u32), np.full((r1 - r0, quads), offset % 2 ** 32, dtype=u32)]
            key = [seed % 2 ** 32, (seed // 2 ** 32) % 2 ** 32]
            for _ in range(10):
                a = ctr[0].astype(u64) * u64(M0)
                c = ctr[2].astype(u64) * u64(M1)
                ctr = [(c >> u64(32)).astype(u32) ^ ctr[1] ^ u32(key[0]), c.astype(u32),
                       (a >> u64(32)).astype(u32) ^ ctr[3] ^ u32(key[1]), a.astype(u32)]
                key = [(key[0] + W0) % 2 ** 32, (key[1] + W1) % 2 ** 32]
            words[r0:r1] = np.stack(ctr, axis=-1)
        keep = words.reshape(rows, 4 * quads)[:, :mul] >= u32(int(p * 2 ** 32))
        cols.append(torch.from_numpy(keep).cuda().double().div_(1.0 - p).repeat_interleave(d, dim=1))
    return torch.cat(cols, dim=1)


def exact(case, seed):
    if case["op"] == "norm_force" and case["rows"] * _dim(case["irreps"]) > 40_000_000:
        return None
    st = _inputs(case, seed)
    x = st["x"].double()
    N, D = x.shape
    f = _exact_factor(case["irreps"], N, case["p"], st["rng"]) if case["p"] > 0 else None
    if case["op"] == "dropout":
        y = x * f if f is not None else x
        return y if st["residual"] is None else y + st["residual"].double()

    # columns: group, channel, bias index (the last one for "none"), centred or not
    group, chan, bidx, cent = [], [], [], []
    ng = nch = nsc = 0
    for mul, d, scalar, _ in _blocks(case["irreps"]):
        per = mul // case["groups"]
        for u in range(mul):
            group += [ng + u // per] * d
            chan += [nch + u] * d
            bidx += [nsc + u if scalar else -1] * d
            cent += [1.0 if scalar else 0.0] * d
        ng += case["groups"]
        nch += mul
        nsc += mul if scalar else 0
    dev = x.device
    group, chan, bidx = (torch.tensor(v, device=dev) for v in (group, chan, bidx))
    cent = torch.tensor(cent, dtype=torch.float64, device=dev)
    counts = torch.tensor(_counts(case, seed), device=dev)
    rows = int(counts.sum())
    seg = torch.repeat_interleave(torch.arange(len(counts), device=dev), counts)
    size = counts.clamp(min=1).double()[:, None] * torch.bincount(group, minlength=ng).double()[None, :]

    def spread_mean(t):
        cols = torch.zeros(rows, ng, dtype=torch.float64, device=dev).index_add(1, group, t)
        tot = torch.zeros(len(counts), ng, dtype=torch.float64, device=dev).index_add(0, seg, cols)
        return (tot / size).index_select(0, seg).index_select(1, group)

    order = case["op"] != "norm_fwd"
    xr = x[:rows].clone().requires_grad_(order)
    w = st["weight"].double().requires_grad_(order)
    b = st["bias"].double().requires_grad_(order)
    xc = xr - spread_mean(xr) * cent
    z = xc / torch.sqrt(spread_mean(xc * xc) + EPS)
    t = z * w[chan] + torch.cat([b, torch.zeros(1, dtype=torch.float64, device=dev)])[bidx] * cent
    y = torch.where(cent.bool(), t / (1.0 + torch.exp(-t)), t) if case["act"] else t
    if f is not None:
        y = y * f[:rows]

    def full(v):
        return torch.cat([v.detach(), torch.zeros(N - rows, D, dtype=torch.float64, device=dev)])

    if not order:
        return full(y)
    g = st["g"][:rows].double().requires_grad_(True)
    if case["op"] == "norm_train":
        gx, gw, gb = torch.autograd.grad(y, (xr, w, b), g, allow_unused=True)
        return full(y), full(gx), gw, torch.zeros_like(b) if gb is None else gb
    (gx,) = torch.autograd.grad(y, xr, g, create_graph=True)
    dg, dx, gw, gb = torch.autograd.grad(gx, (g, xr, w, b), st["ux"][:rows].double(), allow_unused=True)
    return (full(y), full(gx), full(dg), full(dx), gw.detach(),
            torch.zeros_like(b).detach() if gb is None else gb.detach())
