"""The block around a layer: pre-norm, layer, post-norm or plain residual step.

moe_block and moe_block_int8 have to give bit for bit what their pieces give
in turn (each piece is tested against 64 bits in a file of its own), also in
place, from a graph, and with the gate and the residual scale.
"""
import ctypes

import pytest
import torch

from parity import gpu_inputs
from routing_dispatch_expert_sigmoid_b200 import ops
from routing_dispatch_expert_sigmoid_b200.workloads import WORKLOADS, make_inputs

CASES = {
    "mixtral_decode": WORKLOADS["mixtral_decode"].scaled(T=5, d=512, f=1024),
    "dsv3_prefill": WORKLOADS["dsv3_prefill"].scaled(T=300, d=256, E=64, f=144, f_shared=80),
    "general_gating": WORKLOADS["qwen3_prefill"].scaled(T=257, d=192, E=16, k_max=4, f=208,
                                                        gating="softmax"),
    "one_token": WORKLOADS["mixtral_decode"].scaled(T=1, d=256, f=256),
    "f32": WORKLOADS["tiny_f32"].scaled(T=70),
}


def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


class Block:
    def __init__(self, w, post_norm, span, device):
        self.w, self.inp = w, gpu_inputs(w, 3, device, make_inputs(w, 3, device="cpu"))
        self.x, dt = self.inp["x"], self.inp["x"].dtype
        g = torch.Generator(device="cpu").manual_seed(7)
        r = lambda *s, k: (torch.randn(s, generator=g) * k).to(dt).to(device)  # noqa: E731
        self.w_pre = 1 + r(w.d, k=0.1)
        self.w_post = 1 + r(w.d, k=0.1) if post_norm else None
        self.gate = r(-(-w.T // span), w.d, k=0.5) if span else None
        self.cfg = ops.config(w)
        self.norm = ops.norm_config(w.T, w.d, w.dtype, 1e-5, 1e-6, 0.8, span, post_norm)
        self.route = [self.inp[n] for n in ("Wr", "logit_bias", "sel_bias", "k_per_token")]

    def weights(self, int8):
        i = self.inp
        if not int8:
            return [i[n] for n in ("W1", "W3", "W2", "Ws1", "Ws3", "Ws2")]
        return [ops.int8_weight_set(i["W1"], i["W3"], i["W2"]),
                ops.int8_weight_set(i["Ws1"], i["Ws3"], i["Ws2"]) if self.w.f_shared else None]

    def pieces(self, weights, int8):
        c = self.cfg
        h, y, out = (torch.empty_like(self.x) for _ in range(3))
        pre = ops.norm_config(self.w.T, self.w.d, self.w.dtype, eps_pre=1e-6)
        ops.moe_norm(pre, self.x, w_pre=self.w_pre, h=h)
        if int8:
            ops.moe_layer_int8(c, h, *self.route, *weights, y, None,
                               ops.workspace(c, ops.WS_LAYER_INT8))
        else:
            ops.moe_layer(c, h, *self.route, *weights, y, None, ops.workspace(c))
        ops.moe_norm(self.norm, self.x, y=y, w_post=self.w_post, gate=self.gate, z=out)
        return out

    def block(self, weights, int8, x, out, ws, route_out=None):
        f = ops.moe_block_int8 if int8 else ops.moe_block
        f(self.cfg, self.norm, x, self.w_pre, self.w_post, self.gate, *self.route, *weights, out,
          route_out, ws)


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(CASES))
@pytest.mark.parametrize("int8", (False, True))
@pytest.mark.parametrize("post_norm,span", [(True, 0), (True, 64), (False, 0), (False, 1000)])
def test_block_equals_its_pieces(name, int8, post_norm, span):
    w = CASES[name]
    if int8 and w.dtype == "f32":
        pytest.skip("int8 experts need bf16 activations")
    b = Block(w, post_norm, span, dev())
    weights = b.weights(int8)
    want = b.pieces(weights, int8)
    ws = ops.workspace(b.cfg, ops.WS_BLOCK_INT8 if int8 else ops.WS_BLOCK)
    out, rb = torch.full_like(b.x, -7), ops.route_buffers(b.cfg)
    b.block(weights, int8, b.x, out, ws, rb)
    ops.moe_check_errors()
    assert torch.equal(out, want)
    assert int(rb["offsets"][-1]) == int(rb["kept"].sum())
    x = b.x.clone()
    b.block(weights, int8, x, x, ws)  # in place
    ops.moe_check_errors()
    assert torch.equal(x, want)


@pytest.mark.gpu
@pytest.mark.parametrize("int8", (False, True))
def test_graph_replay_on_a_side_stream(int8):
    b = Block(CASES["mixtral_decode"], True, 2, dev())
    weights = b.weights(int8)
    want = b.pieces(weights, int8)
    ws = ops.workspace(b.cfg, ops.WS_BLOCK_INT8 if int8 else ops.WS_BLOCK)
    static, out = b.x.clone(), torch.empty_like(b.x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        b.block(weights, int8, static, out, ws)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            b.block(weights, int8, static, out, ws)
        for _ in range(2):
            out.zero_()
            graph.replay()
            side.synchronize()
            assert torch.equal(out, want)
    ops.moe_check_errors()
    del graph


# ---- refusals (no GPU needed) ---------------------------------------------------
FAKE = 0x7F0000000000  # 16-byte aligned, never dereferenced: validation fails first
P = ctypes.byref


def _call(cfg, norm, norms, int8, x=FAKE, out=FAKE, Wr=FAKE, ws=FAKE, ws_bytes=1 << 45, W2=FAKE):
    L = ops.lib()
    if int8:
        w = ops.MoeInt8Weights(FAKE, FAKE, W2, FAKE, FAKE, FAKE)
        return L.moe_block_int8(P(cfg), P(norm), P(norms), x, Wr, None, None, None, P(w), P(w),
                                out, None, ws, ws_bytes, None)
    return L.moe_block(P(cfg), P(norm), P(norms), x, Wr, None, None, None, FAKE, FAKE, W2, FAKE,
                       FAKE, FAKE, out, None, ws, ws_bytes, None)


@pytest.mark.parametrize("int8", (False, True))
def test_refusals(int8):
    w = WORKLOADS["dsv3_decode"]
    cfg, norm, bn = ops.config(w), ops.norm_config(w.T, w.d), ops.MoeBlockNorms()
    for kw in (dict(T=w.T + 1), dict(d=w.d + 16), dict(dtype=0)):
        n = ops.norm_config(w.T, w.d)
        for k, v in kw.items():
            setattr(n, k, v)
        assert _call(cfg, n, bn, int8) == -1          # the layer's and the norms' sizes differ
    assert _call(cfg, norm, bn, int8, x=None) == -1 and _call(cfg, norm, bn, int8, out=None) == -1
    assert _call(cfg, norm, bn, int8, x=FAKE + 8) == -4
    assert _call(cfg, norm, bn, int8, Wr=None) == -1  # the layer's own arguments
    assert _call(cfg, norm, bn, int8, W2=None) == -1
    assert _call(cfg, norm, ops.MoeBlockNorms(gate=FAKE), int8) == -1    # a gate without a span
    assert _call(cfg, ops.norm_config(w.T, w.d, gate_span=4), bn, int8) == -1
    assert _call(cfg, ops.norm_config(w.T, w.d, post_norm=False), ops.MoeBlockNorms(w_post=FAKE),
                 int8) == -1
    assert _call(cfg, norm, ops.MoeBlockNorms(w_pre=FAKE + 4), int8) == -4
    kind = ops.WS_BLOCK_INT8 if int8 else ops.WS_BLOCK
    need = ops.moe_workspace_size(cfg, kind)
    layer = ops.moe_workspace_size(cfg, ops.WS_LAYER_INT8 if int8 else ops.WS_LAYER)
    assert need >= layer + 2 * w.T * w.d * 2 + (w.T * w.d if int8 else 0)
    assert _call(cfg, norm, bn, int8, ws_bytes=need - 1) == -3
    assert _call(cfg, norm, bn, int8, ws=None) == -3
    cfg.T = norm.T = 0
    assert _call(cfg, norm, bn, int8, x=None, out=None, Wr=None, ws=None, ws_bytes=0) == 0
    if int8:
        cfg, norm = ops.config(w.scaled(dtype="f32")), ops.norm_config(w.T, w.d, "f32")
        assert _call(cfg, norm, bn, int8) == -2
