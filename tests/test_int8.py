"""Int8 products against exact arithmetic.

Codes and scales have to equal the definition bit for bit (fp32 divisions done
on the CPU).  The sums are integers, computed here in fp64, which holds them
exactly; a plain product is then two fp32 multiplications and has to be equal
bit for bit.  SwiGLU goes through the fast exponential and division: for
|g| <= 80 at most 2 + 1.16 * 80 units of 2^-23 and 2 more, under 2^-16
relative, beside half a step of bf16 (2^-8 of the value).
"""
import ctypes
import os

import pytest
import torch

from parity import check_routing_bit_exact, gpu_inputs
from routing_dispatch_expert_sigmoid_b200 import ops
from routing_dispatch_expert_sigmoid_b200.workloads import WORKLOADS, make_inputs

SWIGLU_REL = 2.0 ** -8 + 2.0 ** -16
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


@pytest.fixture(params=("default", "swap", "pair", "gemv"))
def engine(request):
    old = os.environ.pop("MOE_INT8_ENGINE", None)
    if request.param != "default":
        os.environ["MOE_INT8_ENGINE"] = request.param
    yield request.param
    os.environ.pop("MOE_INT8_ENGINE", None)
    if old is not None:
        os.environ["MOE_INT8_ENGINE"] = old


def ref_codes(x):
    """Codes (int8) and scales (fp32) of the rows of a host tensor."""
    x = x.to(torch.float32)
    top = x.abs().amax(-1) if x.shape[-1] else torch.zeros(x.shape[:-1])
    s = top / torch.full_like(top, 127.0)
    fine = torch.isfinite(x).all(-1)
    div = torch.where(fine & (s != 0), s, torch.ones_like(s))
    q = (x / div[..., None]).round().clamp(-127, 127)
    q = torch.where(fine[..., None], q, torch.zeros_like(q))
    return q.to(torch.int8), torch.where(fine, div, torch.full_like(div, float("nan")))


def same(a, b):
    a, b = a.cpu(), b.cpu()
    return a.shape == b.shape and bool(((a == b) | (a.isnan() & b.isnan())).all())


# ---- codes ----------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("rows,K", [(1, 8), (3, 136), (70, 1024), (5, 2056), (9, 4096), (300, 7168),
                                    (2, 16384), (3, 20000), (2, 131056), (5000, 64)])
def test_row_codes_are_the_definition(dtype, rows, K):
    d = dev()
    g = torch.Generator().manual_seed(rows + K)
    x = torch.randn((rows, K), generator=g) * torch.exp(torch.randn((rows, 1), generator=g) * 4)
    x = x.to(DT[dtype])
    if rows > 2:  # many exact halves: multiples of half a code
        x[1] = (torch.randint(-254, 255, (K,), generator=g) / 2).to(DT[dtype])
        x[1, 0] = 127
    q, s = ref_codes(x)
    gq = torch.full((rows, K), -7, dtype=torch.int8, device=d)
    gs = torch.full((rows,), -7.0, device=d)
    ops.moe_quantize_rows_int8(x.to(d), gq, gs)
    assert same(gs, s) and torch.equal(gq.cpu(), q)
    ops.moe_check_errors()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("K", (64, 5000 * 8))
def test_row_codes_of_special_rows(dtype, K):
    d = dev()
    g = torch.Generator().manual_seed(1)
    x = torch.randn((9, K), generator=g)
    x[0] = 0
    x[1, 3] = float("inf")
    x[2, 4] = float("nan")
    x[3] = x[3] * 1e-39                       # subnormal values
    x[4] = 0
    x[4, 7] = 1e-44                           # the scale underflows to zero or its last bits
    x[5] = 3e38                               # the type's range
    x[6] = -x[6].abs()
    x[7, 9] = float("-inf")
    x = x.to(DT[dtype])
    q, s = ref_codes(x)
    gq, gs = torch.empty((9, K), dtype=torch.int8, device=d), torch.empty(9, device=d)
    ops.moe_quantize_rows_int8(x.to(d), gq, gs)
    assert same(gs, s) and torch.equal(gq.cpu(), q)


@pytest.mark.gpu
def test_weight_codes_are_the_definition():
    d = dev()
    g = torch.Generator().manual_seed(31)
    W = (torch.randn(3, 112, 48, generator=g) * torch.rand(3, 1, 48, generator=g) * 4).bfloat16()
    W[0, :, 7] = 0
    W[1, 3, 9] = 3e4
    W[2, :, 11] = 1e-39
    W[2, 5, 12] = float("nan")
    q, s = ops.moe_quantize_int8(W.to(d))
    rq, rs = ref_codes(W.transpose(1, 2))
    assert torch.equal(q.cpu(), rq) and same(s, rs)
    q2, s2 = ops.moe_quantize_int8(W[1].to(d))
    assert torch.equal(q2.cpu(), rq[1]) and same(s2, rs[1])


# ---- products -------------------------------------------------------------------
def operands(rows, K, N, sizes, swiglu, device, seed=0, extreme=False):
    g = torch.Generator().manual_seed(seed + rows * 7 + K + N)
    G = len(sizes) if sizes else 1
    r = lambda *s: torch.randint(-128 if extreme else -127, 128, s, generator=g, dtype=torch.int32).to(torch.int8)  # noqa: E731
    sc = lambda *s: (torch.rand(s, generator=g) + 0.5) * 1e-3  # noqa: E731
    o = dict(xq=r(rows, K), xs=sc(rows), W1=r(G, N, K), s1=sc(G, N), W3=None, s3=None)
    if extreme:
        o["xq"][0], o["W1"][0, 0] = -128, -128
    if swiglu:
        o["W3"], o["s3"] = r(G, N, K), sc(G, N)
    o["offsets"] = None
    if sizes:
        o["offsets"] = torch.tensor([0] + list(sizes)).cumsum(0).to(torch.int32)
    return o, {k: None if v is None else v.to(device) for k, v in o.items()}


def ref_product(o, rows, sizes, which):
    """fp32 y of W1 or W3, exactly as it has to come out; rows behind the groups are NaN."""
    W, s = o["W" + which], o["s" + which]
    y = torch.full((rows, W.shape[1]), float("nan"))
    row = 0
    for g, n in enumerate(sizes or [rows]):
        a = o["xq"][row:row + n].double() @ W[g].double().T
        y[row:row + n] = a.float() * (o["xs"][row:row + n, None] * s[g][None])
        row += n
    return y


def check_product(o, dv, rows, K, N, sizes, swiglu, out_dtype, device):
    G = len(sizes) if sizes else 1
    lin = ops.int8_linear(rows, K, N, G, out_dtype=out_dtype, swiglu=swiglu)
    out = torch.full((rows, N), -7.0, dtype=DT[out_dtype], device=device)
    ops.moe_gemm_int8(lin, dv["xq"], dv["xs"], dv["offsets"], dv["W1"], dv["s1"], dv["W3"],
                      dv["s3"], out)
    ops.moe_check_errors()
    got = out.cpu()
    live = sum(sizes) if sizes else rows
    assert (got[live:] == -7).all(), "rows behind the last group were written"
    got = got[:live]
    y = ref_product(o, rows, sizes, "1")[:live]
    if not swiglu:
        want = y.to(DT[out_dtype])
        assert torch.equal(got, want), f"{int((got != want).sum())} of {got.numel()} differ"
        return
    u = ref_product(o, rows, sizes, "3")[:live].double()
    ref = y.double() / (1 + torch.exp(-y.double())) * u
    assert not y.numel() or float(y.abs().max()) <= 80
    err = (got.double() - ref).abs()
    # results under bf16's normal range (2^-126) round in steps of 2^-133
    assert (err <= SWIGLU_REL * ref.abs() + 2.0 ** -133).all(), (err / ref.abs()).flatten()[:4].tolist()


SHAPES = [  # rows, K, N
    (1, 16, 8), (1, 7168, 2048), (2, 272, 120), (15, 128, 256), (16, 1040, 136), (17, 2048, 264),
    (33, 144, 1000), (64, 4096, 512), (65, 512, 128), (100, 7168, 96), (128, 256, 384),
    (129, 1024, 8), (3, 528, 40), (4, 14336, 64), (5, 4096, 264), (8, 8192, 512), (8, 8208, 104), (255, 400, 256), (256, 768, 264), (257, 128, 520), (600, 2064, 1032),
]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,K,N", SHAPES)
@pytest.mark.parametrize("form", ("f32", "bf16", "swiglu"))
def test_one_matrix(rows, K, N, form, engine):
    d = dev()
    o, dv = operands(rows, K, N, None, form == "swiglu", d)
    if form == "swiglu":  # gates of order one: |g| stays under 80
        o["xs"] /= K ** 0.5
        dv["xs"] = o["xs"].to(d)
    check_product(o, dv, rows, K, N, None, form == "swiglu", "f32" if form == "f32" else "bf16", d)


GROUPS = [  # rows of each group
    [5], [0, 3, 0, 1], [16, 17, 31, 32, 33, 0, 64], [1] * 40, [0] * 8, [300, 2, 0, 129, 256],
    [127, 128, 129, 257], [0, 0, 700], [1, 0, 2, 0, 0, 1, 0, 0], [0] * 60 + [9, 0, 0, 1, 1], [40, 0, 0, 0, 0, 0, 0, 0, 0, 8],
]


@pytest.mark.gpu
@pytest.mark.parametrize("sizes", GROUPS, ids=lambda s: "_".join(map(str, s[:8])))
@pytest.mark.parametrize("form", ("f32", "bf16", "swiglu"))
@pytest.mark.parametrize("K,N", [(400, 264), (1024, 120)])
def test_groups(sizes, form, K, N, engine):
    d = dev()
    rows = sum(sizes) + 7  # some rows behind the last group
    o, dv = operands(rows, K, N, sizes, form == "swiglu", d)
    if form == "swiglu":
        o["xs"] /= K ** 0.5
        dv["xs"] = o["xs"].to(d)
    check_product(o, dv, rows, K, N, sizes, form == "swiglu", "f32" if form == "f32" else "bf16", d)


@pytest.mark.gpu
def test_many_groups_and_the_longest_sums(engine):
    d = dev()
    g = torch.Generator().manual_seed(3)
    sizes = torch.randint(0, 4, (1024,), generator=g).tolist()
    o, dv = operands(sum(sizes), 128, 16, sizes, False, d)
    check_product(o, dv, sum(sizes), 128, 16, sizes, False, "f32", d)
    o, dv = operands(2, 131056, 16, None, False, d, extreme=True)  # every product 2^14 in one sum
    check_product(o, dv, 2, 131056, 16, None, False, "f32", d)


@pytest.mark.gpu
@pytest.mark.parametrize("offsets", ([0, 5, 3, 10], [0, -1, 4, 10], [0, 4, 8, 11], [1 << 30, 0, 0, 0]))
def test_bad_offsets_are_flagged(offsets, engine):
    d = dev()
    o, dv = operands(10, 128, 64, [3, 3, 4], False, d)
    lin = ops.int8_linear(10, 128, 64, 3, out_dtype="f32")
    out = torch.full((10, 64), -7.0, device=d)
    ops.moe_gemm_int8(lin, dv["xq"], dv["xs"], torch.tensor(offsets, dtype=torch.int32, device=d),
                      dv["W1"], dv["s1"], None, None, out)
    with pytest.raises(ops.MoeError):
        ops.moe_check_errors()
    assert (out == -7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("sizes", (None, [0, 9, 30, 1]))
def test_linear_is_codes_then_product(dtype, sizes, engine):
    d = dev()
    rows, K, N = (sum(sizes) + 3 if sizes else 70), 528, 200
    g = torch.Generator().manual_seed(5)
    x = torch.randn((rows, K), generator=g).to(DT[dtype])
    o, dv = operands(rows, K, N, sizes, True, d)
    G = len(sizes) if sizes else 1
    lin = ops.int8_linear(rows, K, N, G, dtype=dtype, swiglu=True)
    q, s = torch.empty((rows, K), dtype=torch.int8, device=d), torch.empty(rows, device=d)
    ops.moe_quantize_rows_int8(x.to(d), q, s)
    a, b = (torch.full((rows, N), -7.0, dtype=torch.bfloat16, device=d) for _ in range(2))
    w = (dv["offsets"], dv["W1"], dv["s1"], dv["W3"], dv["s3"])
    ops.moe_gemm_int8(lin, q, s, *w, a)
    ops.moe_linear_int8(lin, x.to(d), *w, b, ops.int8_workspace(lin))
    ops.moe_check_errors()
    assert torch.equal(a, b)


@pytest.mark.gpu
def test_non_finite_rows_stay_in_their_rows():
    d = dev()
    g = torch.Generator().manual_seed(5)
    x = torch.randn((40, 256), generator=g).bfloat16().to(d)
    _, dv = operands(40, 256, 64, None, False, d)
    lin = ops.int8_linear(40, 256, 64, out_dtype="f32")
    out, bad = torch.empty((40, 64), device=d), torch.empty((40, 64), device=d)
    ws = ops.int8_workspace(lin)
    ops.moe_linear_int8(lin, x, None, dv["W1"], dv["s1"], None, None, out, ws)
    x2 = x.clone()
    x2[3, 7], x2[11, 0] = float("nan"), float("inf")
    ops.moe_linear_int8(lin, x2, None, dv["W1"], dv["s1"], None, None, bad, ws)
    keep = [i for i in range(40) if i not in (3, 11)]
    assert bad[3].isnan().all() and bad[11].isnan().all() and torch.equal(out[keep], bad[keep])


# ---- experts and layers -------------------------------------------------------------
def _set64(hin, names):
    """Dequantised weights [G, K, N] in fp64 from the definition's codes."""
    out = []
    for n in names:
        W = hin[n] if hin[n].dim() == 3 else hin[n][None]
        q, s = ref_codes(W.transpose(1, 2))
        out.append((q.double() * s.double()[..., None]).transpose(1, 2))
    return out


def ffn64(x, W1, W3, W2):
    """The int8 FFN of rows x (bf16) with one expert's dequantised weights: codes of
    x, SwiGLU, h rounded to bf16, codes of h, down projection."""
    dq = lambda v: (lambda q, s: q.double() * s.double()[:, None])(*ref_codes(v))  # noqa: E731
    a = dq(x)
    g, u = a @ W1, a @ W3
    h = (g / (1 + torch.exp(-g)) * u).to(torch.bfloat16)
    return dq(h) @ W2, h


# The kernel's h may round to the other neighbour in bf16 where its fp32 value
# lies next to the middle (one in 2^8 of the elements at most), and a changed
# largest element moves a row's scale by 2^-8: every code of that row is then
# rounded anew, an error of at most one code step, max|h| / 127, on each of its
# f elements with independent signs.  Against the fp64 chain the output is
# therefore compared with a bound on the relative Frobenius norm of the
# quantisation noise itself: a step of max|h| / 127 is uniform noise of 0.29
# steps; max|h| is under 30 times h's RMS for f <= 4096, so 30 / 127 * 0.29 =
# 0.07 of the output.  Rows whose h has the kernel's own codes are exact
# products and are tested above.
FFN_FROB = 0.07
FFN_CASES = {
    "prefill": WORKLOADS["mixtral_prefill"].scaled(T=300, d=256, f=384),
    "decode": WORKLOADS["mixtral_decode"].scaled(T=5, d=512, f=1024),
    "ragged": WORKLOADS["mixtral_prefill"].scaled(T=200, d=272, f=400),
    "drops": WORKLOADS["qwen3_prefill"].scaled(T=150, d=192, E=16, k_max=4, f=208,
                                               capacity_factor=0.25),
    "shared": WORKLOADS["dsv3_prefill"].scaled(T=130, d=256, E=64, f=144, f_shared=80),
    "general": WORKLOADS["dsv3_decode"].scaled(T=64, d=384, E=64, f=144, f_shared=96,
                                               gating="softmax"),
    "one_token": WORKLOADS["mixtral_decode"].scaled(T=1, d=256, f=256),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(FFN_CASES))
def test_layer(name, engine):
    """moe_layer_int8: routing bit for bit, the output that of its own pieces bit for
    bit, and the fp64 chain within the quantisation noise; the codes of x handed
    in change nothing."""
    d = dev()
    w = FFN_CASES[name]
    hin = make_inputs(w, 0, device="cpu")
    inp = gpu_inputs(w, 0, d, hin)
    cfg = ops.config(w)
    experts = ops.int8_weight_set(inp["W1"], inp["W3"], inp["W2"])
    shared = ops.int8_weight_set(inp["Ws1"], inp["Ws3"], inp["Ws2"]) if w.f_shared else None
    ws, rb = ops.workspace(cfg, ops.WS_LAYER_INT8), ops.route_buffers(cfg)
    out = torch.empty_like(inp["x"])
    head = (cfg, inp["x"], inp["Wr"], inp["logit_bias"], inp["sel_bias"], inp["k_per_token"],
            experts, shared)
    ops.moe_layer_int8(*head, out, rb, ws)
    ops.moe_check_errors()
    if w.gating != "softmax":
        check_routing_bit_exact(w, hin, rb)
    xq = torch.empty((w.T, w.d), dtype=torch.int8, device=d)
    xs = torch.empty(w.T, device=d)
    ops.moe_quantize_rows_int8(inp["x"], xq, xs)
    out2 = torch.empty_like(out)
    ops.moe_layer_int8(*head, out2, None, ws, xq=xq, x_scale=xs)
    ops.moe_check_errors()
    assert torch.equal(out, out2)

    # the pieces: dispatch, expert FFN, combine
    rows = w.T * w.k_max
    x_perm = torch.zeros((rows, w.d), dtype=torch.bfloat16, device=d)
    ops.moe_dispatch(cfg, inp["x"], rb["offsets"], rb["row_src"], x_perm)
    y = torch.full((rows, w.d), -7.0, device=d)
    ops.moe_expert_ffn_int8(cfg, x_perm, rb["offsets"], experts, y,
                            ops.workspace(cfg, ops.WS_EXPERT_FFN_INT8))
    ops.moe_check_errors()
    off = rb["offsets"].tolist()
    assert (y[off[-1]:] == -7).all()
    W1, W3, W2 = _set64(hin, ("W1", "W3", "W2"))
    ref = torch.zeros((rows, w.d), dtype=torch.float64)
    for e in range(w.E):
        if off[e + 1] > off[e]:
            ref[off[e]:off[e + 1]] = ffn64(x_perm[off[e]:off[e + 1]].cpu(), W1[e], W3[e], W2[e])[0]
    got = y[:off[-1]].double().cpu()
    ref = ref[:off[-1]]
    if off[-1]:
        assert float((got - ref).norm()) <= FFN_FROB * float(ref.norm())
    y_sh = None
    if w.f_shared:
        # the shared expert through the same calls: one group of T rows
        c1 = ops.MoeConfig.from_buffer_copy(cfg)
        c1.E, c1.k_max, c1.f, c1.gating, c1.n_groups = 1, 1, w.f_shared, 0, 1
        y_sh = torch.empty((w.T, w.d), device=d)
        ops.moe_expert_ffn_int8(c1, inp["x"], torch.tensor([0, w.T], dtype=torch.int32, device=d),
                                {k: v[None] for k, v in shared.items()}, y_sh,
                                ops.workspace(c1, ops.WS_EXPERT_FFN_INT8))
    out3 = torch.empty_like(out)
    ops.moe_combine(cfg, y, rb["slot_row"], rb["topk_w"], y_sh, out3)
    ops.moe_check_errors()
    assert torch.equal(out, out3)


@pytest.mark.gpu
def test_block_of_norm_layer_and_norm():
    """The operators as a block uses them: pre-norm with codes, int8 layer in a
    general gating mode on those codes, post-norm with gate and residual; equal to
    the same chain in which the layer quantises for itself, and near the bf16
    layer's block (the distance is that of the weights' and rows' codes)."""
    d = dev()
    w = WORKLOADS["dsv3_prefill"].scaled(T=300, d=512, E=64, f=256, f_shared=256,
                                         gating="sigmoid_renorm")
    hin = make_inputs(w, 2, device="cpu")
    inp = gpu_inputs(w, 2, d, hin)
    g = torch.Generator(device=d).manual_seed(1)
    r = lambda *s, k=1.0: (torch.randn(s, generator=g, device=d) * k).bfloat16()  # noqa: E731
    w_pre, w_post, gate = 1 + r(w.d, k=0.1), 1 + r(w.d, k=0.1), r(1, w.d, k=0.5)
    x = inp["x"]
    cfg = ops.config(w)
    pre = ops.norm_config(w.T, w.d)
    post = ops.norm_config(w.T, w.d, gate_span=w.T)
    h, hq, hs = torch.empty_like(x), torch.empty((w.T, w.d), dtype=torch.int8, device=d), torch.empty(w.T, device=d)
    ops.moe_norm(pre, x, w_pre=w_pre, h=h, hq=hq, h_scale=hs)
    experts = ops.int8_weight_set(inp["W1"], inp["W3"], inp["W2"])
    shared = ops.int8_weight_set(inp["Ws1"], inp["Ws3"], inp["Ws2"])
    head = (cfg, h, inp["Wr"], inp["logit_bias"], inp["sel_bias"], None, experts, shared)
    ws = ops.workspace(cfg, ops.WS_LAYER_INT8)
    outs = []
    for kw in (dict(xq=hq, x_scale=hs), {}):
        y, z = torch.empty_like(x), torch.empty_like(x)
        ops.moe_layer_int8(*head, y, None, ws, **kw)
        ops.moe_norm(post, x, y=y, w_post=w_post, gate=gate, z=z)
        outs.append(z)
    assert torch.equal(*outs)
    y, z = torch.empty_like(x), torch.empty_like(x)
    ops.moe_layer(cfg, h, inp["Wr"], inp["logit_bias"], inp["sel_bias"], None, inp["W1"], inp["W3"],
                  inp["W2"], inp["Ws1"], inp["Ws3"], inp["Ws2"], y, None, ops.workspace(cfg))
    ops.moe_norm(post, x, y=y, w_post=w_post, gate=gate, z=z)
    ops.moe_check_errors()
    ref = y.double()
    # three products of codes, each operand's noise 0.29 steps of max / 127 with
    # max under 5 RMS for rows and columns of 256 to 512 normal values (30 for h):
    # 0.012 each for x, W1, W3, W2 and 0.07 for h
    y8 = torch.empty_like(x)
    ops.moe_layer_int8(*head, y8, None, ws)
    assert float((y8.double() - ref).norm()) <= 0.12 * float(ref.norm())
    zdiff = float((outs[0].double() - z.double()).norm())
    assert zdiff <= 0.12 * float((z.double() - x.double()).norm()) + 2.0 ** -8 * float(z.double().norm())


@pytest.mark.gpu
def test_graph_replay_on_a_side_stream():
    d = dev()
    w = WORKLOADS["mixtral_decode"].scaled(T=16, d=512, f=1024, gating="softmax")
    inp, nxt = (make_inputs(w, s, device=d) for s in (0, 1))
    cfg = ops.config(w)
    experts = ops.int8_weight_set(inp["W1"], inp["W3"], inp["W2"])
    ws = ops.workspace(cfg, ops.WS_LAYER_INT8)

    def layer(x, out):
        ops.moe_layer_int8(cfg, x, inp["Wr"], inp["logit_bias"], None, None, experts, None, out,
                           None, ws)

    want = [torch.empty_like(inp["x"]) for _ in range(2)]
    layer(inp["x"], want[0])
    layer(nxt["x"], want[1])
    static, out = inp["x"].clone(), torch.empty_like(inp["x"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        layer(static, out)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            layer(static, out)
        for src, ref in ((inp["x"], want[0]), (nxt["x"], want[1])):
            static.copy_(src)
            out.zero_()
            graph.replay()
            side.synchronize()
            assert torch.equal(out, ref)
    ops.moe_check_errors()
    del graph


@pytest.mark.gpu
@pytest.mark.parametrize("rows,K,N", [(1, 4096, 256), (64, 2048, 40000)])
def test_waits_that_run_out_are_reported(rows, K, N, monkeypatch):
    """The swap engine's pipeline waits with no time at all: the call ends, the
    error word says so, and the next call is right again."""
    d = dev()
    o, dv = operands(rows, K, N, None, False, d)
    lin = ops.int8_linear(rows, K, N, out_dtype="f32")
    out = torch.empty((rows, N), device=d)
    args = (lin, dv["xq"], dv["xs"], None, dv["W1"], dv["s1"], None, None, out)
    monkeypatch.setenv("MOE_INT8_ENGINE", "swap")
    monkeypatch.setenv("MOE_WAIT_LIMIT_NS", "0")
    ops.moe_gemm_int8(*args)
    monkeypatch.delenv("MOE_WAIT_LIMIT_NS")
    with pytest.raises(ops.MoeError):
        ops.moe_check_errors()
    check_product(o, dv, rows, K, N, None, False, "f32", d)


# ---- refusals (no GPU needed) ---------------------------------------------------
FAKE = 0x7F0000000000  # 16-byte aligned, never dereferenced: validation fails first
P = ctypes.byref


@pytest.mark.parametrize("kw,expect", [
    (dict(rows=-1), -1), (dict(K=0), -1), (dict(N=0), -1), (dict(G=0), -1), (dict(G=1025), -1),
    (dict(swiglu=2), -1), (dict(dtype=3), -2), (dict(out_dtype=-1), -2),
    (dict(swiglu=1, out_dtype=0), -2), (dict(K=24), -4), (dict(N=12), -4), (dict(K=131072), -2),
    (dict(rows=(1 << 30) + 1), -2), (dict(N=(1 << 24) + 8), -2),
    (dict(rows=1 << 30, N=1 << 16), -2),  # 2^25 row steps x 513 column tiles
])
def test_linear_config_refusals(kw, expect):
    lin = ops.int8_linear(4, 64, 16)
    for n, v in kw.items():
        setattr(lin, n, v)
    L, n = ops.lib(), ctypes.c_size_t(0)
    assert L.moe_int8_workspace_size(P(lin), P(n)) == expect
    assert L.moe_gemm_int8(P(lin), *[None] * 9) == expect
    assert L.moe_linear_int8(P(lin), *[None] * 8, 0, None) == expect


def test_linear_pointer_refusals():
    L = ops.lib()
    lin = ops.int8_linear(4, 64, 16, G=2, swiglu=True)
    good = [FAKE] * 8  # xq, scale, offsets, W1, s1, W3, s3, out
    for i in range(8):
        a = list(good)
        a[i] = None
        assert L.moe_gemm_int8(P(lin), *a, None) == -1
        a[i] = FAKE + 2
        assert L.moe_gemm_int8(P(lin), *a, None) == -4
    lin.swiglu = 0  # W3 with the plain form
    assert L.moe_gemm_int8(P(lin), *good, None) == -1
    ws = ctypes.c_size_t(ops.int8_workspace_size(lin) - 256)
    lin_args = [FAKE, FAKE, FAKE, FAKE, None, None, FAKE]
    assert L.moe_linear_int8(P(lin), *lin_args, FAKE, ws, None) == -3
    assert L.moe_linear_int8(P(lin), *lin_args, None, 1 << 30, None) == -3
    assert L.moe_linear_int8(P(lin), *lin_args, FAKE + 8, 1 << 30, None) == -4
    lin.rows = 0  # no rows: nothing is touched
    assert L.moe_gemm_int8(P(lin), *[None] * 9) == 0
    assert L.moe_linear_int8(P(lin), *[None] * 8, 0, None) == 0


def test_quantiser_refusals():
    L = ops.lib()
    assert L.moe_quantize_int8(FAKE, 2, 64, 24, FAKE, FAKE, None) == -4
    assert L.moe_quantize_int8(FAKE, 2, 40, 32, FAKE, FAKE, None) == -4
    assert L.moe_quantize_int8(FAKE, -1, 64, 32, FAKE, FAKE, None) == -1
    assert L.moe_quantize_int8(FAKE, 0, 64, 32, None, None, None) == 0
    assert L.moe_quantize_int8(FAKE, 70000, 64, 32, FAKE, FAKE, None) == -2
    assert L.moe_quantize_rows_int8(FAKE, 1, 3, 12, FAKE, FAKE, None) == -4
    assert L.moe_quantize_rows_int8(FAKE, 0, 3, 6, FAKE, FAKE, None) == -4
    assert L.moe_quantize_rows_int8(FAKE, 2, 3, 16, FAKE, FAKE, None) == -2
    assert L.moe_quantize_rows_int8(FAKE, 1, -3, 16, FAKE, FAKE, None) == -1
    assert L.moe_quantize_rows_int8(FAKE, 1, (1 << 30) + 1, 16, FAKE, FAKE, None) == -2
    assert L.moe_quantize_rows_int8(FAKE + 8, 1, 3, 16, FAKE, FAKE, None) == -4
    assert L.moe_quantize_rows_int8(FAKE, 1, 3, 16, FAKE, None, None) == -1
    assert L.moe_quantize_rows_int8(None, 1, 0, 16, None, None, None) == 0


def _wset(**kw):
    v = dict(W1=FAKE, W3=FAKE, W2=FAKE, s1=FAKE, s3=FAKE, s2=FAKE)
    v.update(kw)
    return ops.MoeInt8Weights(*[v[k] for k in ("W1", "W3", "W2", "s1", "s3", "s2")])


def test_layer_refusals():
    L = ops.lib()
    w = _wset()

    def call(c, experts=w, shared=w, xq=None, xs=None, ws=1 << 40, ev=None, n=0, x=FAKE):
        return L.moe_layer_int8(P(c), x, xq, xs, FAKE, None, None, None,
                                None if experts is None else P(experts),
                                None if shared is None else P(shared), FAKE, None, FAKE, ws, None,
                                ev, n)

    base = WORKLOADS["dsv3_decode"]
    for kw, expect in ((dict(dtype="f32"), -2), (dict(d=7160), -4), (dict(f=2040), -4),
                       (dict(f_shared=2040), -4), (dict(d=131072), -2), (dict(f=131072), -2),
                       (dict(f_shared=131072), -2)):
        assert call(ops.config(base.scaled(**kw))) == expect
    c = ops.config(base)
    assert call(c, experts=None) == -1 and call(c, shared=None) == -1
    assert call(c, ev=None, n=3) == -1
    assert call(c, xq=FAKE) == -1 and call(c, xs=FAKE) == -1 and call(c, xq=FAKE + 8, xs=FAKE) == -4
    assert call(c, experts=_wset(s2=FAKE + 4)) == -4 and call(c, experts=_wset(W3=0)) == -1
    need = ops.moe_workspace_size(c, ops.WS_LAYER_INT8)
    assert call(c, ws=need - 1) == -3
    assert ops.moe_workspace_size(c, ops.WS_EXPERT_FFN_INT8) < need
    n = ctypes.c_size_t(0)
    assert L.moe_workspace_size(P(c), 7, P(n)) == -1
    assert L.moe_expert_ffn_int8(P(c), FAKE, FAKE, None, FAKE, FAKE, 1 << 40, None) == -1
    c.T = 0
    assert call(c, x=None) == 0


def test_binding_refuses_wrong_tensors():
    lin = ops.int8_linear(4, 64, 16)
    with pytest.raises(ops.MoeError, match="xq is on cpu"):
        ops.moe_gemm_int8(lin, torch.zeros(4, 64, dtype=torch.int8), None, None, None, None, None,
                          None, None)


@pytest.mark.gpu
def test_binding_refuses_wrong_device_tensors():
    d = dev()
    lin = ops.int8_linear(4, 64, 16)
    W, s = torch.zeros(1, 16, 64, dtype=torch.int8, device=d), torch.ones(1, 16, device=d)
    x, out = torch.zeros(4, 64, dtype=torch.bfloat16, device=d), torch.zeros(4, 16, dtype=torch.bfloat16, device=d)
    ws = ops.int8_workspace(lin)
    for a in ((x.float(), W, out), (x, W.transpose(1, 2), out), (x, W.view(torch.uint8), out),
              (x, W, out.float()), (x, W[:, :8], out)):
        with pytest.raises(ops.MoeError, match="contiguous"):
            ops.moe_linear_int8(lin, a[0], None, a[1], s, None, None, a[2], ws)
