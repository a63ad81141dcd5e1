"""The norms around a block and their gradients, against 64 bits.

Tolerances, relative to the formulas in fp64 on the same stored inputs:
  - rstd: a sum of d squares in fp32 (at most 16 terms in a thread, then 5 + 32
    partial sums: under 64 roundings of 2^-24) and rsqrtf (2 units of 2^-23);
    the square root halves the first: REL = 40 * 2^-24 covers both;
  - an output is a handful of fp32 products and one rounding to the storage
    type, half a step of it (bf16 2^-8 of the value, fp32 2^-24);
  - h is the norm of z as stored, so the reference takes the kernel's own z.
"""
import ctypes

import numpy as np
import pytest
import torch

from routing_dispatch_expert_sigmoid_b200 import ops

REL = 40 * 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
EPS = 1e-5


def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def f64(t):
    return t.detach().to(torch.float64)


class Case:
    """Inputs of one call: tokens T of d values, which parts there are."""

    def __init__(self, T, d, dtype, post=True, pre=True, span=0, alpha=0.75, weights=True, seed=0,
                 device=None, normed=True):
        g = torch.Generator(device="cpu").manual_seed(seed + T * 31 + d)
        dt = DT[dtype]
        r = lambda *s, k=1.0: (torch.randn(s, generator=g) * k).to(dt).to(device)  # noqa: E731
        self.T, self.d, self.dtype, self.dt, self.dev = T, d, dtype, dt, device
        self.post, self.pre, self.span, self.alpha, self.normed = post, pre, span, alpha, normed
        self.x = r(T, d, k=2.0)
        self.y = r(T, d, k=0.5) if post else None
        self.w_post = 1 + r(d, k=0.2) if post and normed and weights else None
        self.w_pre = 1 + r(d, k=0.2) if pre and weights else None
        self.gate = r(-(-T // span), d) if span else None
        self.dz, self.dh = r(T, d), r(T, d)
        self.cfg = ops.norm_config(T, d, dtype, EPS, EPS, alpha, span, normed)

    def full_gate(self):
        if self.gate is None:
            return 1.0
        return f64(self.gate)[torch.arange(self.T, device=self.dev) // self.span]

    def wide(self, dt=None):
        return torch.full((self.T, self.d), -7, dtype=dt or self.dt, device=self.dev)

    def vec(self, n):
        return torch.full((n,), -7.0, device=self.dev)

    def forward(self, codes=False):
        o = dict(z=self.wide() if self.post else None, h=self.wide() if self.pre else None,
                 rstd_post=self.vec(self.T) if self.post and self.normed else None,
                 rstd_pre=self.vec(self.T) if self.pre else None)
        if codes:
            o.update(hq=self.wide(torch.int8), h_scale=self.vec(self.T))
        ops.moe_norm(self.cfg, self.x, y=self.y, w_post=self.w_post, gate=self.gate,
                     w_pre=self.w_pre, **o)
        return o

    def backward(self, o, dz=True, **override):
        ng = self.gate.shape[0] if self.gate is not None else 0
        out = dict(dx=self.wide(), dy=self.wide() if self.post else None,
                   dw_post=self.vec(self.d) if self.post and self.normed else None,
                   dgate=self.vec(ng * self.d).view(ng, self.d) if ng else None,
                   dw_pre=self.vec(self.d) if self.pre else None)
        out.update(override)
        ops.moe_norm_backward(self.cfg, dz=self.dz if dz else None,
                              dh=self.dh if self.pre else None,
                              z=(o["z"] if self.post else self.x) if self.pre else None, y=self.y,
                              w_post=self.w_post, gate=self.gate, w_pre=self.w_pre,
                              rstd_post=o["rstd_post"], rstd_pre=o["rstd_pre"],
                              ws=ops.norm_workspace(self.cfg), **out)
        return out


def rms(v, w):
    n = v * torch.rsqrt(v.square().mean(1, keepdim=True) + EPS)
    return n if w is None else n * w


def near(got, ref, tol, what):
    err = (f64(got) - ref).abs()
    bad = err > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} off, worst {float((err / tol.clamp(min=1e-300)).max()):.2f} of the tolerance"


def check_forward(c, o):
    """z, h and the statistics against fp64; h from the kernel's own z."""
    x = f64(c.x)
    w_post = None if c.w_post is None else f64(c.w_post)
    w_pre = None if c.w_pre is None else f64(c.w_pre)
    z = x
    if c.post:
        y = f64(c.y)
        term = c.full_gate() * (rms(y, w_post) if c.normed else y)
        ref = c.alpha * x + term
        # roundings: rstd, three products and the sum (each 2^-24 of its operands)
        tol = HALF[c.dtype] * ref.abs() + (REL + 8 * 2.0 ** -24) * (term.abs() + (c.alpha * x).abs())
        near(o["z"], ref, tol, "z")
        if c.normed:
            near(o["rstd_post"], torch.rsqrt(y.square().mean(1) + EPS),
                 REL * torch.rsqrt(y.square().mean(1) + EPS), "rstd_post")
        z = f64(o["z"])
    if c.pre:
        ref = rms(z, w_pre)
        near(o["h"], ref, (HALF[c.dtype] + REL + 8 * 2.0 ** -24) * ref.abs() + 1e-300, "h")
        r = torch.rsqrt(z.square().mean(1) + EPS)
        near(o["rstd_pre"], r, REL * r, "rstd_pre")


def ref_backward(c, o, dz=True):
    """fp64 gradients by differentiation, at the stored z."""
    out, grad = {}, f64(c.dz) if dz else None
    if c.pre:
        v = f64(o["z"] if c.post else c.x).requires_grad_()
        w = (torch.ones(c.d, device=c.dev, dtype=torch.float64) if c.w_pre is None
             else f64(c.w_pre)).requires_grad_()
        dv, out["dw_pre"] = torch.autograd.grad(rms(v, w), (v, w), f64(c.dh))
        grad = dv if grad is None else grad + dv
    out["g"] = grad
    if not c.post:
        out["dx"] = grad
        return out
    x, y = f64(c.x).requires_grad_(), f64(c.y).requires_grad_()
    w = (torch.ones(c.d, device=c.dev, dtype=torch.float64) if c.w_post is None
         else f64(c.w_post)).requires_grad_()
    leaves = [x, y, w]
    if c.gate is not None:
        gate = f64(c.gate).requires_grad_()
        leaves.append(gate)
        full = gate[torch.arange(c.T, device=c.dev) // c.span]
    else:
        full = 1.0
    n = rms(y, w) if c.normed else y * w
    got = torch.autograd.grad(c.alpha * x + full * n, leaves, grad)
    out.update(zip(("dx", "dy", "dw_post", "dgate"), got))
    return out


def check_backward(c, o, out, dz=True):
    ref = ref_backward(c, o, dz)
    # Each element is a few products and two means over the row.  The means are
    # fp32 sums of d products (64 roundings) of terms of at most the row's size;
    # their error enters every element times v or u, of order one (at most
    # sqrt(d) for a single element, so the row's own size is taken): an
    # allowance of 128 * 2^-24 of the row's largest gradient, and of it times
    # the largest |u| or |v| for the elements that the mean is multiplied by.
    slack = 128 * 2.0 ** -24
    size = f64(c.dz).abs().amax(1, keepdim=True)
    big = 1.0
    if c.pre:
        z = f64(o["z"] if c.post else c.x)
        v = z * torch.rsqrt(z.square().mean(1, keepdim=True) + EPS)
        r = torch.rsqrt(z.square().mean(1, keepdim=True) + EPS)
        wmax = 1.0 if c.w_pre is None else float(c.w_pre.abs().max())
        size = size + r * f64(c.dh).abs().amax(1, keepdim=True) * wmax * (1 + v.abs())
    near(out["dx"], ref["dx"], HALF[c.dtype] * ref["dx"].abs() + slack * size, "dx")
    if c.post:
        y = f64(c.y)
        r = torch.rsqrt(y.square().mean(1, keepdim=True) + EPS) if c.normed else torch.ones_like(y[:, :1])
        u = y * r
        cw = 1.0 if c.w_post is None else f64(c.w_post).abs().max()
        gmax = 1.0 if c.gate is None else f64(c.gate).abs().max()
        big = r * cw * gmax * size.amax(1, keepdim=True) * (1 + u.abs())
        near(out["dy"], ref["dy"], HALF[c.dtype] * ref["dy"].abs() + slack * big, "dy")
    # sums over tokens: fp32 sums of T terms whose magnitudes are summed here;
    # at most 2 + log-free T / CTAs + 16 + 16 sequential roundings: T bounds them
    for name in ("dw_post", "dw_pre", "dgate"):
        if out.get(name) is None:
            continue
        if name == "dw_pre":
            z = f64(o["z"] if c.post else c.x)
            terms = f64(c.dh).abs() * (z * torch.rsqrt(z.square().mean(1, keepdim=True) + EPS)).abs()
        else:
            y = f64(c.y)
            u = (y * torch.rsqrt(y.square().mean(1, keepdim=True) + EPS)).abs() if c.normed else y.abs()
            w = 1.0 if (name == "dw_post" or c.w_post is None) else f64(c.w_post).abs()
            gt = c.full_gate() if name == "dw_post" else 1.0
            gt = gt.abs() if torch.is_tensor(gt) else gt
            terms = size * u * w * gt
        if name == "dgate":
            tot = torch.zeros_like(ref["dgate"]).index_add_(
                0, torch.arange(c.T, device=c.dev) // c.span, terms)
        else:
            tot = terms.sum(0)
        near(out[name], ref[name], (min(c.T, 64) + 128) * 2.0 ** -24 * tot + 1e-300, name)


SIZES = [(1, 8), (3, 264), (5, 1024), (130, 2880), (7, 4096), (2, 7168), (3, 8192), (600, 512), (1500, 40)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("T,d", SIZES)
@pytest.mark.parametrize("parts", ("both", "post", "pre"))
def test_forward_and_backward(dtype, T, d, parts):
    c = Case(T, d, dtype, post=parts != "pre", pre=parts != "post", span=3 if parts == "both" else 0,
             device=dev())
    o = c.forward()
    check_forward(c, o)
    check_backward(c, o, c.backward(o))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("T,d", [(1, 8), (33, 264), (300, 4096)])
@pytest.mark.parametrize("pre", (False, True))
@pytest.mark.parametrize("span", (0, 1, 10, 400))
def test_residual_without_a_post_norm(dtype, T, d, pre, span):
    c = Case(T, d, dtype, pre=pre, span=span, normed=False, device=dev())
    o = c.forward()
    check_forward(c, o)
    check_backward(c, o, c.backward(o))


@pytest.mark.gpu
@pytest.mark.parametrize("d", (16384, 12288))
def test_longest_rows(d):
    c = Case(301, d, "bf16", span=100, device=dev())
    o = c.forward(codes=True)
    check_forward(c, o)
    check_backward(c, o, c.backward(o))
    c = Case(5, d // 2, "f32", span=2, device=dev())
    o = c.forward(codes=True)
    check_forward(c, o)
    check_backward(c, o, c.backward(o))


@pytest.mark.gpu
@pytest.mark.parametrize("span", (1, 2, 7, 64, 999, 1000, 1001, 5000, 2 ** 31 - 1))
@pytest.mark.parametrize("d", (128, 4096))
def test_gate_spans(span, d):
    """One gate row for each token, for several, for a sequence, for all."""
    c = Case(1000, d, "bf16", span=span, device=dev())
    o = c.forward()
    check_forward(c, o)
    check_backward(c, o, c.backward(o))


@pytest.mark.gpu
@pytest.mark.parametrize("T", (148, 149, 296, 700, 4001))
def test_gate_rows_across_the_ranges_of_ctas(T):
    for span in (T // 3, T // 148 + 1, 5, T - 1):
        c = Case(T, 512, "f32", span=span, pre=False, device=dev())
        o = c.forward()
        check_backward(c, o, c.backward(o))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("bf16", "f32"))
def test_optional_parts(dtype):
    d = dev()
    c = Case(33, 256, dtype, weights=False, device=d)          # no weights: ones
    o = c.forward()
    check_forward(c, o)
    check_backward(c, o, c.backward(o))
    out = c.backward(o, dz=False)                              # nothing arrives at z
    full = dict(out)
    ref = ref_backward(c, o, dz=False)
    check_backward(c, o, out, dz=False)
    # sums that are not wanted, and no workspace for none of them
    out = c.backward(o, dz=False, dw_post=None, dw_pre=None)
    assert torch.equal(out["dx"], full["dx"]) and torch.equal(out["dy"], full["dy"])
    c2 = Case(33, 256, dtype, span=4, device=d)
    o2 = c2.forward()
    a, b = c2.backward(o2), c2.backward(o2, dw_post=None, dw_pre=None)
    assert torch.equal(a["dgate"], b["dgate"]) and torch.equal(a["dx"], b["dx"])
    del ref
    # without y, dz None: the plain norm's gradient
    c3 = Case(9, 264, dtype, post=False, device=d)
    o3 = c3.forward()
    check_backward(c3, o3, c3.backward(o3, dz=False), dz=False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("bf16", "f32"))
def test_fused_call_equals_the_steps_in_turn(dtype):
    """One call gives what the residual step, the plain norm and the row
    quantiser give in three; in-place buffers change nothing."""
    d = dev()
    c = Case(77, 1032, dtype, span=10, device=d)
    o = c.forward(codes=True)
    z, h = c.wide(), c.wide()
    ops.moe_norm(c.cfg, c.x, y=c.y, w_post=c.w_post, gate=c.gate, z=z)
    alone = ops.norm_config(c.T, c.d, dtype, EPS, EPS)
    ops.moe_norm(alone, z, w_pre=c.w_pre, h=h)
    assert torch.equal(z, o["z"]) and torch.equal(h, o["h"])
    hf = h.float()
    scale = hf.abs().amax(1) / torch.full((c.T,), 127.0, device=d)
    codes = (hf / scale[:, None]).round().clamp(-127, 127)
    assert torch.equal(scale, o["h_scale"]) and torch.equal(codes.to(torch.int8), o["hq"])
    hq, hs = c.wide(torch.int8), c.vec(c.T)                    # codes without h
    ops.moe_norm(c.cfg, c.x, y=c.y, w_post=c.w_post, gate=c.gate, w_pre=c.w_pre, z=z, hq=hq,
                 h_scale=hs)
    assert torch.equal(hq, o["hq"]) and torch.equal(hs, o["h_scale"])
    x, y = c.x.clone(), c.y.clone()
    ops.moe_norm(c.cfg, x, y=y, w_post=c.w_post, gate=c.gate, w_pre=c.w_pre, z=x, h=y)
    assert torch.equal(x, o["z"]) and torch.equal(y, o["h"])
    out = c.backward(o)
    dz, dh = c.dz.clone(), c.dh.clone()
    c.dz, c.dh = dz, dh
    got = c.backward(o, dx=dz, dy=dh)
    assert all(torch.equal(out[n], got[n]) for n in out)


@pytest.mark.gpu
def test_rows_of_zeros_and_non_finite_values():
    d = dev()
    for dtype in ("bf16", "f32"):
        c = Case(6, 520, dtype, device=d)
        c.x[0], c.y[0] = 0, 0
        c.x[1, 5], c.y[2, 7] = float("nan"), float("inf")
        c.x[3, 1] = float("inf")
        o = c.forward(codes=True)
        assert (o["z"][0] == 0).all() and (o["h"][0] == 0).all()
        assert (o["hq"][0] == 0).all() and o["h_scale"][0] == 1
        for t in (1, 2, 3):
            assert o["h_scale"][t].isnan() and (o["hq"][t] == 0).all()
            assert not o["h"][t].isfinite().all()
        assert o["h"][4:].isfinite().all() and o["h_scale"][4:].isfinite().all()
        clean = Case(6, 520, dtype, device=d)
        want = clean.forward(codes=True)
        for n in ("z", "h", "hq", "h_scale"):
            assert torch.equal(o[n][4:], want[n][4:])


@pytest.mark.gpu
def test_backward_matches_differences():
    """Central differences of the fp64 forward pass along random directions:
    step 1e-5, truncation 1e-10 of the third derivative, rounding 1e-11."""
    d = dev()
    c = Case(4, 24, "f32", span=3, device=d)
    o = c.forward()
    out = c.backward(o)
    leaves = dict(dx=c.x, dy=c.y, dw_post=c.w_post, dgate=c.gate, dw_pre=c.w_pre)

    def loss(v):
        gate = v["dgate"][torch.arange(c.T, device=d) // c.span]
        z = c.alpha * v["dx"] + gate * rms(v["dy"], v["dw_post"])
        return (z * f64(c.dz)).sum() + (rms(z, v["dw_pre"]) * f64(c.dh)).sum()

    base = {n: f64(t) for n, t in leaves.items()}
    g = torch.Generator(device="cpu").manual_seed(9)
    for n in leaves:
        for _ in range(3):
            u = torch.randn(base[n].shape, generator=g, dtype=torch.float64).to(d)
            up = loss(dict(base, **{n: base[n] + 1e-5 * u}))
            down = loss(dict(base, **{n: base[n] - 1e-5 * u}))
            fd = float((up - down) / 2e-5)
            got = float((f64(out[n]) * u).sum())
            scale = float((f64(out[n]).abs() * u.abs()).sum())
            assert abs(got - fd) <= 1e-5 * scale + 1e-6


@pytest.mark.gpu
def test_graph_replay_on_a_side_stream():
    d = dev()
    c = Case(50, 640, "bf16", span=20, device=d)
    o = c.forward()
    want = c.backward(o)
    ws = ops.norm_workspace(c.cfg)
    got_o = {n: torch.empty_like(t) for n, t in o.items()}
    got = {n: torch.empty_like(t) for n, t in want.items()}

    def both():
        ops.moe_norm(c.cfg, c.x, y=c.y, w_post=c.w_post, gate=c.gate, w_pre=c.w_pre, **got_o)
        ops.moe_norm_backward(c.cfg, dz=c.dz, dh=c.dh, z=got_o["z"], y=c.y, w_post=c.w_post,
                              gate=c.gate, w_pre=c.w_pre, rstd_post=got_o["rstd_post"],
                              rstd_pre=got_o["rstd_pre"], ws=ws, **got)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        both()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            both()
        for _ in range(3):
            for t in (*got.values(), *got_o.values()):
                t.fill_(3)
            graph.replay()
            side.synchronize()
            assert all(torch.equal(got[n], want[n]) for n in want)
            assert all(torch.equal(got_o[n], o[n]) for n in o)
    del graph


# ---- refusals (no GPU needed) ---------------------------------------------------
FAKE = 0x7F0000000000  # 16-byte aligned, never dereferenced: validation fails first
P = ctypes.byref


@pytest.mark.parametrize("kw,expect", [
    (dict(T=-1), -1), (dict(d=0), -1), (dict(d=4), -4), (dict(d=16392), -2), (dict(dtype=5), -2),
    (dict(gate_span=-1), -1), (dict(post_norm=2), -1), (dict(eps_post=0.0), -1), (dict(eps_pre=float("nan")), -1),
    (dict(eps_pre=-1e-6), -1), (dict(eps_post=float("inf")), -1), (dict(dtype=0, d=8196), -2),
    (dict(dtype=0, d=6), -4),
])
def test_config_refusals(kw, expect):
    c = ops.norm_config(4, 64)
    for n, v in kw.items():
        setattr(c, n, v)
    L, n = ops.lib(), ctypes.c_size_t(0)
    assert L.moe_norm(P(c), P(ops.MoeNormIo()), None) == expect
    assert L.moe_norm_backward(P(c), P(ops.MoeNormGradIo()), None, 0, None) == expect
    assert L.moe_norm_workspace_size(P(c), P(n)) == expect


def _io(cls, names, **kw):
    io = cls()
    for i, n in enumerate(names.split()):
        setattr(io, n, FAKE + 4096 * (i + 1))
    for n, v in kw.items():
        setattr(io, n, v)
    return io


@pytest.mark.parametrize("names,kw,span,expect", [
    ("y z h", {}, 0, -1),                                    # no x
    ("x", {}, 0, -1),                                        # nothing to compute
    ("x y h", {}, 0, -1),                                    # y without z
    ("x z h", {}, 0, -1),                                    # z without y
    ("x w_post h", {}, 0, -1),                               # a post-norm weight without y
    ("x y z w_pre", {}, 0, -1),                              # a pre-norm weight without h
    ("x y z", {}, 4, -1),                                    # a span without a gate
    ("x y z gate", {}, 0, -1),                               # a gate without a span
    ("x h gate", {}, 4, -1),                                 # a gate without y
    ("x hq", {}, 0, -1), ("x h h_scale", {}, 0, -1),         # codes and scales go together
    ("x h rstd_post", {}, 0, -1), ("x y z rstd_pre", {}, 0, -1),
    ("x y z h", dict(h=FAKE, z=FAKE), 0, -1),                # one buffer for two outputs
    ("x h", dict(x=FAKE + 8), 0, -4), ("x y z h", dict(y=FAKE + 4), 0, -4),
    ("x hq h_scale", dict(hq=FAKE + 8), 0, -4), ("x hq h_scale", dict(h_scale=FAKE + 2), 0, -4),
    ("x h rstd_pre", dict(rstd_pre=FAKE + 1), 0, -4),
])
def test_forward_refusals(names, kw, span, expect):
    c = ops.norm_config(4, 64, gate_span=span)
    assert ops.lib().moe_norm(P(c), P(_io(ops.MoeNormIo, names, **kw)), None) == expect


@pytest.mark.parametrize("names,kw,span,expect", [
    ("y rstd_post dx dy", {}, 0, -1),                        # no gradient arrives
    ("dz z dx", {}, 0, -1),                                  # neither norm
    ("dh rstd_pre dx", {}, 0, -1),                           # dh without z
    ("dh z dx", {}, 0, -1),                                  # dh without its statistic
    ("dz y dx dy", {}, 0, -1),                               # y without its statistic
    ("dz y rstd_post dx", {}, 0, -1),                        # no dy
    ("dh z rstd_pre dx dy", {}, 0, -1),                      # dy without y
    ("dz y rstd_post dy", {}, 0, -1),                        # no dx
    ("dz y rstd_post dx dy", dict(dx=FAKE, dy=FAKE), 0, -1),
    ("dz y rstd_post dx dy dgate", {}, 0, -1), ("dz y rstd_post dx dy dw_pre", {}, 0, -1),
    ("dh z rstd_pre dx dw_post", {}, 0, -1), ("dh z rstd_pre dx gate", {}, 3, -1),
    ("dz y rstd_post dx dy", dict(dx=FAKE + 8), 0, -4), ("dh z rstd_pre dx", dict(z=FAKE + 2), 0, -4),
    ("dz y rstd_post dx dy dw_post", {}, 0, -3),             # no workspace
])
def test_backward_refusals(names, kw, span, expect):
    c = ops.norm_config(4, 64, gate_span=span)
    io = _io(ops.MoeNormGradIo, names, **kw)
    assert ops.lib().moe_norm_backward(P(c), P(io), None, 0, None) == expect


def test_refusals_without_a_post_norm():
    c = ops.norm_config(4, 64, post_norm=False)
    L = ops.lib()
    for extra in ("w_post", "rstd_post"):
        assert L.moe_norm(P(c), P(_io(ops.MoeNormIo, "x y z " + extra)), None) == -1
    for extra in ("w_post", "rstd_post", "dw_post"):
        io = _io(ops.MoeNormGradIo, "dz y dx dy " + extra)
        assert L.moe_norm_backward(P(c), P(io), FAKE, 1 << 30, None) == -1


def test_workspace_refusals_and_empty_batch():
    c = ops.norm_config(300, 64, gate_span=10)
    need = ops.norm_workspace_size(c)
    assert need > 0 and need % 16 == 0
    io = _io(ops.MoeNormGradIo, "dz y gate rstd_post dx dy dgate")
    L = ops.lib()
    assert L.moe_norm_backward(P(c), P(io), FAKE, need - 1, None) == -3
    assert L.moe_norm_backward(P(c), P(io), FAKE + 8, need, None) == -4
    assert L.moe_norm(P(c), None, None) == -1
    assert L.moe_norm_backward(P(c), None, None, 0, None) == -1
    c.T = 0
    assert L.moe_norm(P(c), P(ops.MoeNormIo()), None) == 0
    assert L.moe_norm_backward(P(c), P(ops.MoeNormGradIo()), None, 0, None) == 0


def test_binding_refuses_wrong_tensors():
    c = ops.norm_config(4, 64)
    with pytest.raises(ops.MoeError, match="x is on cpu"):
        ops.moe_norm(c, torch.zeros(4, 64, dtype=torch.bfloat16))
    with pytest.raises(ops.MoeError, match="dx is missing"):
        ops.moe_norm_backward(c)


@pytest.mark.gpu
def test_binding_refuses_wrong_device_tensors():
    d = dev()
    c = ops.norm_config(4, 64)
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=d)
    h = torch.zeros_like(x)
    for bad in (x.float(), x[:2], torch.zeros(64, 4, dtype=torch.bfloat16, device=d).t()):
        with pytest.raises(ops.MoeError, match="x has to be"):
            ops.moe_norm(c, bad, h=h)
