"""General gating and the gradient of the combine weights, against 64 bits.

Forward: the selection has to equal that of the scores computed in fp64 from
the same fp32 logits and biases, including tokens whose experts are closer
than fp32 scores can tell; weights within their rounding (derived below).
Backward: against the formula's gradient by fp64 differentiation and against
central differences of the fp64 forward pass.
"""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from parity import assert_out_close, gpu_inputs, oracle_cf
from routing_dispatch_expert_sigmoid_b200 import ops
from routing_dispatch_expert_sigmoid_b200.workloads import WORKLOADS, make_inputs, to_numpy

MODES = ("softmax", "softmax_renorm", "sigmoid", "sigmoid_renorm")
# E, k, groups, kept groups, scores summed for a group
SHAPES = [(8, 2, 1, 1, 1), (33, 4, 1, 1, 1), (64, 6, 8, 3, 2), (128, 8, 4, 2, 1), (160, 6, 8, 3, 1),
          (256, 8, 8, 4, 2), (384, 7, 4, 4, 3), (512, 16, 1, 1, 1), (1024, 32, 2, 1, 8),
          (40, 1, 4, 1, 8), (5, 5, 1, 1, 1)]
# fp32 weights, relative: expf within 2 units of 2^-23 (4 of 2^-24), its
# argument's rounding at most 16 of 2^-24 for |l| <= 8, one rounding each for
# the sum 1 + e, the quotient and the scale, at most 37 for a sum of 1024
# terms; numerator and denominator together stay under 128 * 2^-24.
W_REL = 2.0 ** -17


def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def ref_scores(l64, mode):
    """fp64 scores; rows that are all -inf score 0."""
    with np.errstate(over="ignore", invalid="ignore"):
        if mode.startswith("sigmoid"):
            return 1.0 / (1.0 + np.exp(-l64))
        m = l64.max(1, keepdims=True)
        e = np.where(np.isneginf(m), 0.0, np.exp(l64 - np.where(np.isneginf(m), 0.0, m)))
        s = e.sum(1, keepdims=True)
        return e / np.where(s == 0, 1.0, s)


def ref_gate(l32, mode, k, bias=None, kt=None, groups=1, keep=1, top=1, scale=1.0):
    l64 = l32.astype(np.float64)
    T, E = l64.shape
    s = ref_scores(l64, mode)
    u = s if bias is None else s + bias.astype(np.float64)[None]
    order_by = l64 if bias is None else u
    alive = np.ones((T, E), bool)
    if groups > 1:
        per = np.sort(u.reshape(T, groups, E // groups), axis=2)[:, :, ::-1][:, :, :top].sum(2)
        if bias is None and top == 1:
            per = l64.reshape(T, groups, -1).max(2)
        rank = np.argsort(np.argsort(-per, axis=1, kind="stable"), axis=1, kind="stable")
        alive = np.repeat(rank < keep, E // groups, axis=1)
    # candidates by key, the experts of dropped groups behind all others
    idx = np.lexsort((np.broadcast_to(np.arange(E), (T, E)), -order_by, ~alive), axis=1)[:, :k]
    w = np.take_along_axis(s, idx, 1)
    if kt is not None:
        pad = np.arange(k)[None] >= kt[:, None]
        w, idx = np.where(pad, 0.0, w), np.where(pad, -1, idx)
    if mode.endswith("renorm"):
        if mode.startswith("sigmoid"):
            # shares by their logarithms, log s = -log(1 + e^-l): rows of equal
            # logits below -745 have equal shares although fp64 sigmoids vanish
            lg = -np.logaddexp(0.0, -np.take_along_axis(l64, idx, 1))
            lg = np.where(idx < 0, -np.inf, lg)
            big = lg.max(1, keepdims=True)
            w = np.where(np.isneginf(lg), 0.0, np.exp(lg - np.where(np.isneginf(big), 0.0, big)))
        tot = w.sum(1, keepdims=True)
        w = np.where(tot > 0, w / np.where(tot > 0, tot, 1.0), 0.0)
    return idx.astype(np.int32), scale * w


def run_gate(cfg, logits, bias, kt, device):
    idx = torch.full((cfg.T, cfg.k_max), -7, dtype=torch.int32, device=device)
    w = torch.full((cfg.T, cfg.k_max), -7.0, device=device)
    up = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(device)  # noqa: E731
    ops.moe_gate(cfg, up(logits), up(bias), up(kt), idx, w)
    return idx.cpu().numpy(), w.cpu().numpy()


@pytest.mark.gpu
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"E{s[0]}k{s[1]}g{s[2]}")
@pytest.mark.parametrize("bias", (False, True))
def test_forward_matches_64_bits(mode, shape, bias):
    d = dev()
    E, k, groups, keep, top = shape
    for T, ragged in ((1, False), (203, True)):
        rng = np.random.default_rng(E * 7 + T)
        l = np.clip(rng.standard_normal((T, E)) * 1.5, -8, 8).astype(np.float32)
        b = (rng.standard_normal(E) * 0.05).astype(np.float32) if bias else None
        kt = rng.integers(1, k + 1, T).astype(np.int32) if ragged else None
        cfg = ops.gate_config(T, E, k, mode, groups, keep, top, 2.5)
        idx, w = run_gate(cfg, l, b, kt, d)
        ridx, rw = ref_gate(l, mode, k, b, kt, groups, keep, top, 2.5)
        assert (idx == ridx).all(), np.argwhere(idx != ridx)[:4].tolist()
        np.testing.assert_allclose(w, rw, rtol=W_REL, atol=0)
        ops.moe_check_errors()


@pytest.mark.gpu
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("groups", (1, 4))
def test_order_of_experts_closer_than_fp32_scores(mode, groups):
    """Logits a unit in the last place apart give scores that fp32 rounds to
    one value or to the wrong order; biases that all but cancel the difference
    of two scores do the same.  Equal logits stay in index order."""
    d = dev()
    T, E, k = 64, 128, 8
    rng = np.random.default_rng(5)
    l = rng.standard_normal((T, E)).astype(np.float32)
    l[:32, 1::2] = np.nextafter(l[:32, ::2], np.float32(9), dtype=np.float32)
    l[32:48] = np.round(l[32:48] * 2) / 2  # many equal logits
    b = np.zeros(E, np.float32)
    s = ref_scores(l[48:49].astype(np.float64), mode)[0]
    b[:] = (s.max() - s).astype(np.float32)  # row 48: every key equal but for the rounding of b
    l[49:] = l[48] + rng.integers(-1, 2, (T - 49, E)).astype(np.float32) * 2.0 ** -23
    cfg = ops.gate_config(T, E, k, mode, groups, min(groups, 2), 2 if groups > 1 else 1)
    for bias in (b, np.zeros(E, np.float32), None):
        idx, w = run_gate(cfg, l, bias, None, d)
        ridx, rw = ref_gate(l, mode, k, bias, None, groups, min(groups, 2), 2 if groups > 1 else 1)
        assert (idx == ridx).all(), np.argwhere(idx != ridx)[:4].tolist()
        np.testing.assert_allclose(w, rw, rtol=W_REL, atol=0)
    ops.moe_check_errors()


@pytest.mark.gpu
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("groups", (1, 2))
def test_masked_and_non_finite_rows(mode, groups):
    d = dev()
    E, k = 64, 6
    rng = np.random.default_rng(11)
    l = rng.standard_normal((7, E)).astype(np.float32)
    l[1, rng.permutation(E)[:E - 3]] = -np.inf          # three experts left for six slots
    l[2] = -np.inf                                      # nothing left
    l[3] = np.finfo(np.float32).min                     # the type's lowest value everywhere
    l[4] = -200.0 - np.arange(E)                        # sigmoids far below fp32's range
    l[5, 9], l[6, 3] = np.nan, np.inf
    b = (rng.standard_normal(E) * 0.05).astype(np.float32)
    b[5] = -np.inf                                      # an expert that is never wanted
    cfg = ops.gate_config(7, E, k, mode, groups, groups, 1)
    for bias in (None, b):
        idx, w = run_gate(cfg, l, bias, None, d)
        ridx, rw = ref_gate(l[:5], mode, k, bias, None, groups, groups, 1)
        assert (idx[:5] == ridx).all()
        if mode == "sigmoid_renorm":  # fp64 sigmoids of row 4 keep their ratios
            assert np.isfinite(rw[4]).all() and rw[4].sum() > 0.99
        # fp32's smallest numbers are 2^-149 apart; row 4's arguments of exp are
        # up to 263, whose rounding is 263 * 2^-24 of the result
        np.testing.assert_allclose(w[:5], rw, rtol=2.0 ** -15, atol=2.0 ** -148)
        assert np.isnan(w[5:]).all()
        for t in (5, 6):
            assert len(set(idx[t])) == k and (idx[t] >= 0).all() and (idx[t] < E).all()
        assert bias is None or not (idx[[0, 2, 3, 4]] == 5).any()
    ops.moe_check_errors()


@pytest.mark.gpu
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("shape", [(64, 6, 8, 3, 2), (96, 5, 3, 2, 1), (256, 8, 4, 2, 2), (512, 16, 1, 1, 1),
                                   (1024, 32, 8, 5, 3)], ids=lambda s: f"E{s[0]}k{s[1]}g{s[2]}")
def test_keys_far_apart(mode, shape):
    """Logits and biases over many orders of magnitude; the first and the last
    expert as the largest and the smallest of their rows."""
    d = dev()
    E, k, groups, keep, top = shape
    T = 64
    rng = np.random.default_rng(E + 1)
    l = (rng.standard_normal((T, E)) * np.array([1.0, 12.0, 40.0, 1e4])[:, None].repeat(T // 4, 0)).astype(np.float32)
    l[::4, 0], l[::4, E - 1] = l[::4].max(1) + 1, l[::4].min(1) - 1
    l[1::4, E - 1], l[1::4, 0] = l[1::4].max(1) + 1, l[1::4].min(1) - 1
    b = (rng.standard_normal(E) * 10.0 ** rng.integers(-6, 38, E)).astype(np.float32)
    b[rng.permutation(E)[:E // 4]] = 0
    gated = ops.gate_config(T, E, k, mode, groups, keep, 1)
    idx, _ = run_gate(gated, l, None, None, d)
    assert (idx == ref_gate(l, mode, k, None, None, groups, keep, 1)[0]).all()
    rows = T // 4  # scores that fp64 keeps apart
    cfg = ops.gate_config(rows, E, k, mode, groups, keep, top)
    for bias in (None, b):
        idx, _ = run_gate(cfg, l[:rows], bias, None, d)
        assert (idx == ref_gate(l[:rows], mode, k, bias, None, groups, keep, top)[0]).all()
    ops.moe_check_errors()


@pytest.mark.gpu
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("bias", (False, True))
@pytest.mark.parametrize("shape", [(72, 7, 1, 1, 1), (512, 32, 1, 1, 1), (1024, 32, 1, 1, 1), (1024, 32, 8, 4, 2)],
                         ids=lambda s: f"E{s[0]}k{s[1]}g{s[2]}")
def test_many_equal_experts(mode, bias, shape):
    """Logits and biases of few different values: from two to all of a token's
    experts share the last place, those of the lowest index get it."""
    d = dev()
    E, k, groups, keep, top = shape
    rng = np.random.default_rng(E + k)
    values = np.array([2.0, 3.0, 12.0, 50.0, 1e9])
    l = rng.standard_normal((40, E))
    step = 3.0 / values[np.arange(40) % 5][:, None]
    l = (np.round(l / step) * step).astype(np.float32)
    b = (rng.integers(-1, 2, E) * 0.25).astype(np.float32) if bias else None
    cfg = ops.gate_config(40, E, k, mode, groups, keep, top)
    idx, _ = run_gate(cfg, l, b, None, d)
    ridx, _ = ref_gate(l, mode, k, b, None, groups, keep, top)
    assert (idx == ridx).all(), np.argwhere(idx != ridx)[:4].tolist()
    ops.moe_check_errors()


@pytest.mark.gpu
def test_budget_out_of_range_is_flagged():
    d = dev()
    cfg = ops.gate_config(3, 16, 4, "softmax")
    l = np.random.default_rng(0).standard_normal((3, 16)).astype(np.float32)
    idx, _ = run_gate(cfg, l, None, np.array([4, 0, 9], np.int32), d)
    with pytest.raises(ops.MoeError):
        ops.moe_check_errors()
    ridx, _ = ref_gate(l, "softmax", 4, None, np.array([4, 1, 4]))  # taken as 1 and k_max
    assert (idx == ridx).all()


def ref_grad(l32, idx, dw, mode, scale):
    """fp64 gradient by differentiation of the weights' formula."""
    l = torch.from_numpy(l32).to(torch.float64).requires_grad_()
    s = torch.sigmoid(l) if mode.startswith("sigmoid") else torch.softmax(l, 1)
    it = torch.from_numpy(idx).long()
    w = torch.gather(s, 1, it.clamp(min=0)) * (it >= 0)
    if mode.endswith("renorm"):
        w = w / w.sum(1, keepdim=True)
    g, = torch.autograd.grad((scale * w * torch.from_numpy(dw).double()).sum(), l)
    return g.numpy()


def run_grad(cfg, l, idx, dw, device):
    out = torch.full((cfg.T, cfg.E), -7.0, device=device)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(device)  # noqa: E731
    ops.moe_gate_backward(cfg, up(l), up(idx), up(dw), out)
    return out.cpu().numpy()


@pytest.mark.gpu
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"E{s[0]}k{s[1]}g{s[2]}")
def test_backward_matches_64_bits(mode, shape):
    d = dev()
    E, k, groups, keep, top = shape
    for T in (1, 75):
        rng = np.random.default_rng(E + T)
        l = np.clip(rng.standard_normal((T, E)) * 1.5, -8, 8).astype(np.float32)
        kt = rng.integers(1, k + 1, T).astype(np.int32)
        idx, _ = ref_gate(l, mode, k, None, kt, groups, keep, top)
        dw = rng.standard_normal((T, k)).astype(np.float32)
        dw[idx < 0] = np.nan  # gradients of empty slots are not read into anything
        cfg = ops.gate_config(T, E, k, mode, groups, keep, top, 1.7)
        got = run_grad(cfg, l, idx, dw, d)
        ref = ref_grad(l, idx, np.where(idx < 0, 0, dw), mode, 1.7)
        # every element is a sum of at most k + 1 products of factors at most 1
        # (shares, scores) with g: absolute error W_REL * (1 + k) * max|g|
        tol = W_REL * (1 + k) * 1.7 * np.nanmax(np.abs(dw), axis=1, keepdims=True)
        assert (np.abs(got - ref) <= tol).all(), np.abs(got - ref).max()
        if mode != "softmax":  # untouched experts get exact zeros
            hit = np.zeros((T, E), bool)
            np.put_along_axis(hit, np.where(idx < 0, idx[:, :1], idx), True, 1)
            assert (got[~hit] == 0).all()
    ops.moe_check_errors()


@pytest.mark.gpu
@pytest.mark.parametrize("mode", MODES)
def test_backward_matches_differences(mode):
    """Central differences of the fp64 weights at step h: truncation below
    h^2 * max|w'''| < 1e-10, rounding below 2^-52 / h: both far below 1e-5."""
    d = dev()
    T, E, k, h = 3, 24, 4, 1e-5
    rng = np.random.default_rng(3)
    l = rng.standard_normal((T, E)).astype(np.float32)
    idx, _ = ref_gate(l, mode, k)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    cfg = ops.gate_config(T, E, k, mode)
    got = run_grad(cfg, l, idx, dw, d)

    def loss(l64):
        s = ref_scores(l64, mode)
        w = np.take_along_axis(s, idx, 1)
        if mode.endswith("renorm"):
            w = w / w.sum(1, keepdims=True)
        return (w * dw).sum(1)

    for e in range(E):
        step = np.zeros(E)
        step[e] = h
        l64 = l.astype(np.float64)
        fd = (loss(l64 + step) - loss(l64 - step)) / (2 * h)
        assert np.abs(got[:, e] - fd).max() <= 1e-5 + W_REL * (1 + k) * np.abs(dw).max()


@pytest.mark.gpu
@pytest.mark.parametrize("fixed,general,scale", [("topk_softmax", "softmax_renorm", 1.0),
                                                 ("softmax_topk_renorm", "softmax_renorm", 1.0),
                                                 ("sigmoid_grouped", "sigmoid_renorm", 2.5)])
def test_fixed_modes_share_the_gradient(fixed, general, scale):
    """The three fixed modes weight as the renormalised general ones do."""
    d = dev()
    T, E, k = 37, 64, 6
    rng = np.random.default_rng(8)
    l = rng.standard_normal((T, E)).astype(np.float32)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    idx, w = run_gate(ops.gate_config(T, E, k, fixed, 8, 4, 2, 2.5), l, None, None, d)
    kw = (8, 4, 2) if fixed == "sigmoid_grouped" else (1, 1, 1)
    gidx, gw = run_gate(ops.gate_config(T, E, k, general, *kw, scale), l, None, None, d)
    assert (idx == gidx).all()
    np.testing.assert_allclose(w, gw, rtol=2 * W_REL)
    a = run_grad(ops.gate_config(T, E, k, fixed, 8, 4, 2, 2.5), l, idx, dw, d)
    b = run_grad(ops.gate_config(T, E, k, general, *kw, scale), l, idx, dw, d)
    assert (a == b).all()


@pytest.mark.gpu
@pytest.mark.parametrize("mode", MODES)
def test_backward_repeated_and_bad_indices(mode):
    """A repeated index gets the sum of its gradients, the same one every time;
    an index outside the experts is flagged and adds nothing."""
    d = dev()
    T, E, k = 5, 33, 6
    rng = np.random.default_rng(2)
    l = rng.standard_normal((T, E)).astype(np.float32)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    idx = rng.integers(0, E, (T, k)).astype(np.int32)
    idx[0], idx[1, 3:] = 7, 2
    idx[4] = -1                                       # no slot at all
    cfg = ops.gate_config(T, E, k, mode)
    got = run_grad(cfg, l, idx, dw, d)
    ref = ref_grad(l[:4], idx[:4], dw[:4], mode, 1.0)
    assert np.abs(got[:4] - ref).max() <= W_REL * (1 + k) * k * np.abs(dw).max()
    assert (got[4] == 0).all()
    for _ in range(3):
        assert (run_grad(cfg, l, idx, dw, d) == got).all()
    ops.moe_check_errors()
    bad = idx.copy()
    bad[2, 1], bad[3, 0] = E, -2
    got = run_grad(cfg, l, bad, dw, d)
    with pytest.raises(ops.MoeError):
        ops.moe_check_errors()
    skipped = np.where((bad >= E) | (bad < -1), -1, bad)
    ref = ref_grad(l[:4], skipped[:4], np.where(skipped < 0, 0, dw)[:4], mode, 1.0)
    assert np.abs(got[:4] - ref).max() <= W_REL * (1 + k) * k * np.abs(dw).max()


@pytest.mark.gpu
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("T", (60, 300))
def test_layer_in_the_general_modes(mode, T):
    """moe_route and moe_layer take the general modes: the gating of their own
    logits is moe_gate's bit for bit, the layout and the layer's output are the
    oracle's for that routing."""
    d = dev()
    w = WORKLOADS["dsv3_prefill"].scaled(T=T, d=256, E=64, f=136, f_shared=72, gating=mode,
                                         capacity_factor=1.25)
    hin = make_inputs(w, 4, device="cpu")
    inp = gpu_inputs(w, 4, d, hin)
    cfg = ops.config(w)
    rb, out, ws = ops.route_buffers(cfg), torch.empty_like(inp["x"]), ops.workspace(cfg)
    ops.moe_layer(cfg, inp["x"], inp["Wr"], inp["logit_bias"], inp["sel_bias"],
                  inp["k_per_token"], inp["W1"], inp["W3"], inp["W2"], inp["Ws1"], inp["Ws3"],
                  inp["Ws2"], out, rb, ws)
    ops.moe_check_errors()
    l32 = rb["logits"].cpu().numpy()
    idx, wts = run_gate(cfg, l32, hin["sel_bias"].numpy(), None, d)
    assert (rb["topk_idx"].cpu().numpy() == idx).all()
    assert (rb["topk_w"].cpu().numpy() == wts).all()
    ridx, rw = ref_gate(l32, mode, w.k_max, hin["sel_bias"].numpy(), None, w.n_groups,
                        w.topk_groups, w.group_score_topk, w.routed_scale)
    assert (idx == ridx).all()
    np.testing.assert_allclose(wts, rw, rtol=W_REL)
    lay = oracle.capacity_dispatch(idx, w.E, oracle_cf(w))
    for key in ("counts", "kept", "offsets", "slot_row"):
        assert (rb[key].cpu().numpy() == lay[key]).all(), key
    ref = oracle.layer_tokens(np.arange(T, dtype=np.int32), to_numpy(hin["x"]),
                              *[to_numpy(hin[n]) for n in ("W1", "W3", "W2")], idx, wts,
                              lay["slot_row"], *[to_numpy(hin[n]) for n in ("Ws1", "Ws3", "Ws2")])
    assert_out_close(out, ref)
    # moe_route alone gives the same routing
    rb2 = ops.route_buffers(cfg)
    ops.moe_route(cfg, inp["x"], inp["Wr"], inp["logit_bias"], inp["sel_bias"], None, rb2,
                  ops.workspace(cfg, ops.WS_ROUTE))
    ops.moe_check_errors()
    assert torch.equal(rb["topk_idx"], rb2["topk_idx"]) and torch.equal(rb["topk_w"], rb2["topk_w"])


@pytest.mark.gpu
def test_graph_replay_on_a_side_stream():
    d = dev()
    T, E, k = 50, 128, 8
    cfg = ops.gate_config(T, E, k, "sigmoid_renorm", 4, 2, 2, 2.5)
    g = torch.Generator(device=d).manual_seed(1)
    l, l2 = (torch.randn((T, E), generator=g, device=d) for _ in range(2))
    bias = torch.randn(E, generator=g, device=d) * 0.05
    dw = torch.randn((T, k), generator=g, device=d)

    def both(lg, idx, w, dl):
        ops.moe_gate(cfg, lg, bias, None, idx, w)
        ops.moe_gate_backward(cfg, lg, idx, dw, dl)

    def buffers():
        return (torch.empty((T, k), dtype=torch.int32, device=d), torch.empty((T, k), device=d),
                torch.empty((T, E), device=d))

    want = [buffers(), buffers()]
    both(l, *want[0])
    both(l2, *want[1])
    static, got = l.clone(), buffers()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        both(static, *got)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            both(static, *got)
        for src, ref in ((l, want[0]), (l2, want[1]), (l, want[0])):
            static.copy_(src)
            graph.replay()
            side.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, ref))
    ops.moe_check_errors()
    del graph


# ---- refusals (no GPU needed) ---------------------------------------------------
FAKE = 0x7F0000000000  # 16-byte aligned, never dereferenced: validation fails first


@pytest.mark.parametrize("kw,expect", [
    (dict(E=0), -1), (dict(k_max=33), -1), (dict(n_groups=3), -1), (dict(n_groups=0), -1),
    (dict(topk_groups=9), -1), (dict(topk_groups=1, k_max=9), -1), (dict(group_score_topk=0), -1),
    (dict(gating=7), -2), (dict(T=-1), -1),
])
def test_config_refusals(kw, expect):
    cfg = ops.gate_config(4, 64, 4, "sigmoid", 8, 4, 2)
    for name, v in kw.items():
        setattr(cfg, name, v)
    L, c = ops.lib(), ctypes.byref(cfg)
    assert L.moe_gate(c, FAKE, None, None, FAKE, FAKE, None) == expect
    assert L.moe_gate_backward(c, FAKE, FAKE, FAKE, FAKE, None) == expect


def test_pointer_refusals():
    cfg = ops.gate_config(4, 64, 4, "softmax")
    L, c = ops.lib(), ctypes.byref(cfg)
    good = [FAKE] * 5
    for i, may_lack in enumerate((False, True, True, False, False)):
        a = list(good)
        a[i] = FAKE + 2
        assert L.moe_gate(c, *a, None) == -4
        if not may_lack:
            a[i] = None
            assert L.moe_gate(c, *a, None) == -1
    for i in range(4):
        a = good[:4]
        a[i] = None
        assert L.moe_gate_backward(c, *a, None) == -1
        a[i] = FAKE + 1
        assert L.moe_gate_backward(c, *a, None) == -4
    cfg.T = 0  # an empty batch touches nothing
    assert L.moe_gate(c, None, None, None, None, None, None) == 0
    assert L.moe_gate_backward(c, None, None, None, None, None) == 0


def test_binding_refuses_wrong_tensors():
    cfg = ops.gate_config(4, 64, 4, "softmax")
    l, idx, w = torch.zeros(4, 64), torch.zeros(4, 4, dtype=torch.int32), torch.zeros(4, 4)
    for args in ((l, None, None, idx, w), (None, None, None, idx, w)):
        with pytest.raises(ops.MoeError, match="logits"):
            ops.moe_gate(cfg, *args)  # host memory, a missing tensor
    with pytest.raises(ops.MoeError, match="logits"):
        ops.moe_gate_backward(cfg, l, idx, w, l)


@pytest.mark.gpu
def test_binding_refuses_wrong_device_tensors():
    d = dev()
    cfg = ops.gate_config(4, 64, 4, "softmax")
    l, idx, w = torch.zeros(4, 64, device=d), torch.zeros(4, 4, dtype=torch.int32, device=d), torch.zeros(4, 4, device=d)
    for bad in (l.double(), torch.zeros(4, 65, device=d), torch.zeros(64, 4, device=d).t()):
        with pytest.raises(ops.MoeError, match="logits"):
            ops.moe_gate(cfg, bad, None, None, idx, w)
    with pytest.raises(ops.MoeError, match="topk_idx"):
        ops.moe_gate(cfg, l, None, None, idx.long(), w)
