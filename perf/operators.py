"""Cases of the layer's 8-bit integer products, block norms and general gating, with their plain forms.

Three operators of a Mixture-of-Experts block:

  product   rows times int8 weights, the rows brought to int8 codes with one scale each, the weights held
            as codes with one scale per output channel; one matrix, or one for each expert over rows
            grouped by expert; plain, or the SwiGLU pair silu(x W1) * (x W3)
  norm      the norms around a block: z = alpha * x + gate * (w_post * rms(y)), h = w_pre * rms(z), in one
            pass, and its backward pass
  gate      top-k gating: softmax or sigmoid scores, a selection bias, groups, weights renormalised or
            not, and the gradient of the weights with respect to the logits

`own` False: elementary torch operations.  `own` True: the library's entry points.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
DTYPES = {"bf16": BF16, "f32": F32}


# ---------------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------------
def listed():
    return [
        # one new token through a dense projection of a DeepSeek-V3-shaped shared expert
        dict(name="product_one_token", op="product", rows=1, K=7168, N=2048, G=1, zipf=0.0, dtype="bf16", out="bf16", swiglu=False),
        # a decode batch of 64 tokens, top-2 of 8: the up projection, a stream of expert weights
        dict(name="product_decode_up", op="product", rows=128, K=4096, N=14336, G=8, zipf=0.5, dtype="bf16", out="bf16", swiglu=True),
        # 16384 tokens, top-8 of 128 fine-grained experts, ragged groups: the up projection of a prefill
        dict(name="product_prefill_up", op="product", rows=131072, K=2048, N=768, G=128, zipf=0.17, dtype="bf16", out="bf16", swiglu=True),
        # 8192 tokens, top-2 of 8: the down projection of a prefill, fp32 rows for the combine; an odd number of rows
        dict(name="product_prefill_down", op="product", rows=16381, K=14336, N=4096, G=8, zipf=0.5, dtype="bf16", out="f32", swiglu=False),
        # a decode batch: residual and post-norm of one block with the pre-norm of the next
        dict(name="norm_decode", op="norm", T=16, d=4096, dtype="bf16", post=True, pre=True, gate_span=0, alpha=1.0, backward=False),
        # a prefill with a per-channel gate and a scaled residual
        dict(name="norm_prefill", op="norm", T=8192, d=7168, dtype="bf16", post=True, pre=True, gate_span=8192, alpha=0.9, backward=False),
        # a training step's backward pass, one gate row for each sequence, the last one short
        dict(name="norm_train", op="norm", T=16381, d=4096, dtype="bf16", post=True, pre=True, gate_span=2048, alpha=1.0, backward=True),
        # a small fp32 layer's backward pass with a gate value of its own for every token
        dict(name="norm_train_f32", op="norm", T=777, d=2880, dtype="f32", post=True, pre=False, gate_span=1, alpha=1.0, backward=True),
        # a decode batch: sigmoid scores, a bias for balance, 4 of 8 groups, top-8 of 256, renormalised
        dict(name="gate_decode", op="gate", T=128, E=256, k=8, k_min=8, score="sigmoid", renorm=True, groups=8, keep=4, top=2, bias=True, scale=2.5, backward=False),
        # a prefill: softmax scores with a bias, weights kept as the scores are
        dict(name="gate_prefill", op="gate", T=16384, E=128, k=8, k_min=8, score="softmax", renorm=False, groups=1, keep=1, top=1, bias=True, scale=1.0, backward=False),
        # a training step, 512 sub-experts, 8 to 16 for each token, softmax over all of them
        dict(name="gate_train_softmax", op="gate", T=8191, E=512, k=16, k_min=8, score="softmax", renorm=False, groups=1, keep=1, top=1, bias=False, scale=1.0, backward=True),
        # a training step of the sigmoid form
        dict(name="gate_train_sigmoid", op="gate", T=16384, E=256, k=8, k_min=8, score="sigmoid", renorm=True, groups=8, keep=4, top=2, bias=True, scale=2.5, backward=True),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(("product", "norm", "gate"))
    if op == "product":
        while True:
            c = dict(op=op, rows=_log_int(rng, 1, 131072), K=_log_int(rng, 256, 14336, 16), N=_log_int(rng, 256, 14336, 8),
                     G=rng.choice((1, 1, 4, 8, 32, 64, 128)), zipf=round(rng.uniform(0.0, 0.5), 2), dtype="bf16" if rng.random() < 0.75 else "f32",
                     out=rng.choice(("bf16", "f32")), swiglu=rng.random() < 0.5)
            if c["swiglu"]:
                c["out"] = "bf16"
            weights = c["G"] * c["N"] * c["K"] * (2 if c["swiglu"] else 1)
            per_row = c["N"] * c["K"] * (2 if c["swiglu"] else 1)
            if weights <= 900_000_000 and c["rows"] * per_row <= 900_000_000_000 and c["rows"] * max(c["K"], c["N"]) <= 250_000_000:
                return c
    if op == "norm":
        while True:
            post = rng.random() < 0.8
            c = dict(op=op, T=_log_int(rng, 1, 32768), d=_log_int(rng, 256, 8192, 8), dtype="bf16" if rng.random() < 0.75 else "f32", post=post,
                     pre=not post or rng.random() < 0.7, gate_span=0, alpha=round(rng.uniform(0.5, 1.0), 3), backward=rng.random() < 0.5)
            if post and rng.random() < 0.7:
                c["gate_span"] = rng.choice((1, _log_int(rng, 2, max(2, c["T"])), c["T"]))
            if c["T"] * c["d"] <= 58_000_000:
                return c
    while True:
        E = rng.choice((8, 16, 40, 60, 64, 128, 160, 256, 384, 512))
        groups = rng.choice([n for n in (1, 1, 2, 4, 8) if E % n == 0 and E // n >= 4])
        k = rng.randint(1, min(16, E // 2))
        c = dict(op=op, T=_log_int(rng, 1, 32768), E=E, k=k, k_min=rng.randint(1, k) if rng.random() < 0.3 else k, score=rng.choice(("softmax", "sigmoid")),
                 renorm=rng.random() < 0.5, groups=groups, keep=rng.randint(1, groups), top=rng.randint(1, 3) if groups > 1 else 1, bias=rng.random() < 0.6,
                 scale=round(rng.uniform(0.5, 3.0), 2), backward=rng.random() < 0.5)
        if k <= c["keep"] * (E // groups) and c["T"] * E <= 4_200_000:
            return c


# ---------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------
def _sizes(rows, G, zipf):
    """Rows of each group, largest first: a Zipf law over the groups, rounded so that they add up."""
    share = [(i + 1.0) ** -zipf for i in range(G)]
    total = sum(share)
    ends, run = [0], 0.0
    for s in share:
        run += s
        ends.append(int(round(rows * run / total)))
    ends[-1] = rows
    return [b - a for a, b in zip(ends, ends[1:])]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def normal(*shape, dtype=F32, std=1.0):
        return torch.randn(shape, generator=g, device=dev).mul_(std).to(dtype)

    if case["op"] == "product":
        rows, K, N, G = case["rows"], case["K"], case["N"], case["G"]
        sizes = _sizes(rows, G, case["zipf"])
        sizes = [sizes[i] for i in torch.randperm(G, generator=g, device=dev).tolist()]
        # activations as a norm leaves them: unit variance, a few channels several times as large
        x = normal(rows, K)
        x *= 1.0 + 5.0 * (torch.rand(K, generator=g, device=dev) < 0.01)
        s = dict(case=case, x=x.to(DTYPES[case["dtype"]]), sizes=sizes, most=max(sizes))
        s["offsets"] = torch.tensor([0] + sizes, device=dev).cumsum(0).to(torch.int32) if G > 1 else None
        for name in ("1", "3") if case["swiglu"] else ("1",):
            codes = torch.empty((G, N, K), dtype=torch.int8, device=dev)
            for i in range(G):  # normal weights: the largest of a channel is about four standard deviations
                codes[i] = torch.randn((N, K), generator=g, device=dev).mul_(127.0 / 4.2).round_().clamp_(-127, 127)
            s["W" + name] = codes
            s["s" + name] = (0.8 + 0.4 * torch.rand((G, N), generator=g, device=dev)) * (4.2 / 127.0 / math.sqrt(K))
        return s
    if case["op"] == "norm":
        T, d, dt = case["T"], case["d"], DTYPES[case["dtype"]]
        s = dict(case=case, x=normal(T, d, dtype=dt, std=2.0), y=normal(T, d, dtype=dt, std=0.7) if case["post"] else None)
        s["w_post"] = (1.0 + normal(d, std=0.1)).to(dt) if case["post"] else None
        s["w_pre"] = (1.0 + normal(d, std=0.1)).to(dt) if case["pre"] else None
        span = case["gate_span"]
        s["gate"] = normal(-(-T // span), d, dtype=dt, std=0.5) if span else None
        if case["backward"]:  # what a forward pass leaves, and the gradients that arrive
            z, _, rstd_post, rstd_pre = _norm_plain(s)
            s.update(z=z, rstd_post=rstd_post, rstd_pre=rstd_pre)
            s["dz"] = normal(T, d, dtype=dt) if case["post"] else None
            s["dh"] = normal(T, d, dtype=dt) if case["pre"] else None
        return s
    T, E, k = case["T"], case["E"], case["k"]
    s = dict(case=case)
    rank = torch.randperm(E, generator=g, device=dev).to(F32) + 1.0
    s["logits"] = normal(T, E) - 0.3 * rank.log()
    s["sel_bias"] = normal(E, std=0.05) if case["bias"] else None
    s["k_per_token"] = torch.randint(case["k_min"], k + 1, (T,), generator=g, device=dev, dtype=torch.int32) if case["k_min"] < k else None
    if case["backward"]:
        s["topk_idx"], _ = _gate_plain(s)
        s["dtopk_w"] = normal(T, k)
    return s


# ---------------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------------
def run(state):
    op, backward = state["case"]["op"], state["case"].get("backward")
    if own:
        return _own_product(state) if op == "product" else _own_norm(state) if op == "norm" else _own_gate(state)
    if op == "product":
        return _product_plain(state)
    if op == "norm":
        return _norm_backward_plain(state) if backward else dict(zip("zh", _norm_plain(state)[:2]))
    return _gate_backward_plain(state) if backward else dict(zip(("topk_idx", "topk_w"), _gate_plain(state)))


# ---- plain forms ----------------------------------------------------------------------------------
def _product_plain(s):
    case, x = s["case"], s["x"].to(F32)
    top = x.abs().amax(1)
    scale = top / torch.full_like(top, 127.0)  # a division: by a Python number it would be a product with 1 / 127
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    codes = (x / scale[:, None]).round().clamp(-127, 127)
    G, rows = case["G"], case["rows"]
    if G > 1:  # the rows of each group side by side, the short groups filled up with zeros
        off = s["offsets"].to(torch.int64)
        row = torch.arange(rows, device=x.device)
        group = torch.searchsorted(off[1:], row, right=True)
        at = group * s["most"] + row - off[group]
        a = torch.zeros((G * s["most"], case["K"]), device=x.device)
        a[at] = codes
        a = a.view(G, s["most"], case["K"])
    else:
        a = codes[None]

    def times(W, sc):
        y = torch.matmul(a, W.to(F32).transpose(1, 2))
        y = y * sc[:, None, :]
        y = y.view(-1, case["N"])[at] if G > 1 else y[0]
        return y * scale[:, None]

    y = times(s["W1"], s["s1"])
    if case["swiglu"]:
        y = y / (1.0 + torch.exp(-y)) * times(s["W3"], s["s3"])
    return y.to(DTYPES[case["out"]])


def _gate_rows(s):
    """The gate of every token, fp32 [T, d]; 1.0 without one."""
    if s["gate"] is None:
        return 1.0
    at = torch.arange(s["case"]["T"], device=s["gate"].device) // s["case"]["gate_span"]
    return s["gate"].to(F32)[at]


EPS = 1e-6


def _norm_plain(s):
    """(z, h, rstd_post, rstd_pre): z None without a post-norm, h None without a pre-norm."""
    case, dt = s["case"], DTYPES[s["case"]["dtype"]]
    x, z, h, rstd_post, rstd_pre = s["x"].to(F32), None, None, None, None
    if case["post"]:
        y = s["y"].to(F32)
        rstd_post = 1.0 / torch.sqrt((y * y).mean(1) + EPS)
        z = (case["alpha"] * x + _gate_rows(s) * (y * rstd_post[:, None] * s["w_post"].to(F32))).to(dt)
    if case["pre"]:
        v = (s["x"] if z is None else z).to(F32)
        rstd_pre = 1.0 / torch.sqrt((v * v).mean(1) + EPS)
        h = (v * rstd_pre[:, None] * s["w_pre"].to(F32)).to(dt)
    return z, h, rstd_post, rstd_pre


def _norm_backward_plain(s):
    case, dt, out = s["case"], DTYPES[s["case"]["dtype"]], {}
    d = case["d"]
    grad = s["dz"].to(F32) if s["dz"] is not None else 0.0
    if case["pre"]:
        v = (s["x"] if s["z"] is None else s["z"]).to(F32) * s["rstd_pre"][:, None]
        dh = s["dh"].to(F32)
        out["dw_pre"] = (dh * v).sum(0)
        dv = dh * s["w_pre"].to(F32)
        grad = grad + s["rstd_pre"][:, None] * (dv - v * ((dv * v).sum(1, keepdim=True) / d))
    if not case["post"]:
        return dict(out, dx=grad.to(dt))
    out["dx"] = (case["alpha"] * grad).to(dt)
    v = s["y"].to(F32) * s["rstd_post"][:, None]
    w = s["w_post"].to(F32)
    if s["gate"] is not None:
        span, T = case["gate_span"], case["T"]
        part = grad * v * w
        n = s["gate"].shape[0]
        if n * span > T:
            part = torch.cat((part, part.new_zeros(n * span - T, d)))
        out["dgate"] = part.view(n, span, d).sum(1)
    dn = grad * _gate_rows(s)
    out["dw_post"] = (dn * v).sum(0)
    dv = dn * w
    out["dy"] = (s["rstd_post"][:, None] * (dv - v * ((dv * v).sum(1, keepdim=True) / d))).to(dt)
    return out


def _scores(case, logits):
    """The scores, in 64 bits: a selection looks at differences that 32 bits lose."""
    l64 = logits.to(torch.float64)
    if case["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l64))
    e = torch.exp(l64 - l64.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _gate_plain(s):
    case, E, k = s["case"], s["case"]["E"], s["case"]["k"]
    score = _scores(case, s["logits"])
    key = score if s["sel_bias"] is None else score + s["sel_bias"].to(torch.float64)
    n = case["groups"]
    if n > 1:
        per = key.view(-1, n, E // n)
        group = per.sort(dim=2, descending=True)[0][:, :, :case["top"]].sum(2)
        kept = group.sort(dim=1, descending=True, stable=True)[1][:, :case["keep"]]
        mask = torch.zeros_like(group).scatter_(1, kept, 1.0)
        key = torch.where(mask[:, :, None] > 0, per, torch.full_like(per, -math.inf)).view(-1, E)
    idx = key.sort(dim=1, descending=True, stable=True)[1][:, :k]
    w = score.gather(1, idx)
    if s["k_per_token"] is not None:
        live = torch.arange(k, device=idx.device)[None, :] < s["k_per_token"][:, None]
        w = torch.where(live, w, torch.zeros_like(w))
        idx = torch.where(live, idx, torch.full_like(idx, -1))
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return idx.to(torch.int32), (case["scale"] * w).to(F32)


def _gate_backward_plain(s):
    case, logits = s["case"], s["logits"]
    live = s["topk_idx"] >= 0
    at = s["topk_idx"].clamp(min=0).to(torch.int64)
    g = torch.where(live, case["scale"] * s["dtopk_w"], torch.zeros_like(s["dtopk_w"]))
    zero = torch.zeros_like(logits)
    if case["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-logits))
    else:
        e = torch.exp(logits - logits.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    chosen = torch.where(live, score.gather(1, at), torch.zeros_like(g))
    if case["renorm"]:
        total = chosen.sum(1, keepdim=True)
        g = torch.where(live, (g - (g * chosen / total).sum(1, keepdim=True)) / total, torch.zeros_like(g))
    ds = zero.scatter_add(1, at, g)
    if case["score"] == "sigmoid":
        return ds * score * (1.0 - score)
    return score * (ds - (ds * score).sum(1, keepdim=True))


# ---- the library ----------------------------------------------------------------------------------
def _kept(s, make):
    """What a program keeps beside its inputs: descriptors, workspaces and output buffers."""
    if "kept" not in s:
        s["kept"] = make()
    return s["kept"]


def _own_product(s):
    from routing_dispatch_expert_sigmoid_b200 import ops
    case = s["case"]

    def make():
        lin = ops.int8_linear(case["rows"], case["K"], case["N"], case["G"], dtype=case["dtype"], out_dtype=case["out"], swiglu=case["swiglu"])
        return lin, torch.empty((case["rows"], case["N"]), dtype=DTYPES[case["out"]], device=s["x"].device), ops.int8_workspace(lin)

    lin, out, ws = _kept(s, make)
    ops.moe_linear_int8(lin, s["x"], s["offsets"], s["W1"], s["s1"], s.get("W3"), s.get("s3"), out, ws)
    return out


def _own_norm(s):
    from routing_dispatch_expert_sigmoid_b200 import ops
    case = s["case"]
    T, d, dt, dev = case["T"], case["d"], DTYPES[case["dtype"]], s["x"].device

    def make():
        cfg = ops.norm_config(T, d, dtype=case["dtype"], eps_post=EPS, eps_pre=EPS, residual_scale=case["alpha"], gate_span=case["gate_span"])
        wide = lambda want: torch.empty((T, d), dtype=dt, device=dev) if want else None  # noqa: E731
        if not case["backward"]:
            return cfg, wide(case["post"]), wide(case["pre"])
        vec = lambda want, *n: torch.empty(n, dtype=F32, device=dev) if want else None  # noqa: E731
        gate = s["gate"]
        return (cfg, wide(True), wide(case["post"]), vec(case["post"], d), vec(gate is not None, *(gate.shape if gate is not None else ())),
                vec(case["pre"], d), ops.norm_workspace(cfg))

    kept = _kept(s, make)
    if not case["backward"]:
        cfg, z, h = kept
        ops.moe_norm(cfg, s["x"], y=s["y"], w_post=s["w_post"], gate=s["gate"], w_pre=s["w_pre"], z=z, h=h)
        return dict(z=z, h=h)
    cfg, dx, dy, dw_post, dgate, dw_pre, ws = kept
    ops.moe_norm_backward(cfg, dz=s["dz"], dh=s["dh"], z=s["z"] if case["post"] else s["x"], y=s["y"], w_post=s["w_post"], gate=s["gate"], w_pre=s["w_pre"],
                          rstd_post=s["rstd_post"], rstd_pre=s["rstd_pre"], dx=dx, dy=dy, dw_post=dw_post, dgate=dgate, dw_pre=dw_pre, ws=ws)
    out = dict(dx=dx, dy=dy, dw_post=dw_post, dgate=dgate, dw_pre=dw_pre)
    return {k: v for k, v in out.items() if v is not None}


def _own_gate(s):
    from routing_dispatch_expert_sigmoid_b200 import ops
    case, dev = s["case"], s["logits"].device
    T, E, k = case["T"], case["E"], case["k"]

    def make():
        cfg = ops.gate_config(T, E, k, gating=case["score"] + ("_renorm" if case["renorm"] else ""), n_groups=case["groups"], topk_groups=case["keep"],
                              group_score_topk=case["top"], routed_scale=case["scale"])
        if case["backward"]:
            return cfg, torch.empty((T, E), device=dev)
        return cfg, torch.empty((T, k), dtype=torch.int32, device=dev), torch.empty((T, k), device=dev)

    kept = _kept(s, make)
    if case["backward"]:
        cfg, dlogits = kept
        ops.moe_gate_backward(cfg, s["logits"], s["topk_idx"], s["dtopk_w"], dlogits)
        return dlogits
    cfg, idx, w = kept
    ops.moe_gate(cfg, s["logits"], s["sel_bias"], s["k_per_token"], idx, w)
    return dict(topk_idx=idx, topk_w=w)


# ---------------------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------------------
def work(case):
    if case["op"] == "product":
        rows, K, N, n = case["rows"], case["K"], case["N"], 2 if case["swiglu"] else 1
        used = sum(v > 0 for v in _sizes(rows, case["G"], case["zipf"]))
        size = {"bf16": 2, "f32": 4}
        return {"bytes": rows * K * size[case["dtype"]] + used * n * N * (K + 4) + rows * N * size[case["out"]], "flops": 2 * rows * N * K * n}
    if case["op"] == "norm":
        T, d, b = case["T"], case["d"], 2 if case["dtype"] == "bf16" else 4
        gates = -(-T // case["gate_span"]) if case["gate_span"] else 0
        post, pre = int(case["post"]), int(case["pre"])
        vec = (post + pre + gates) * d * b
        if not case["backward"]:  # x, and y; z and h
            return {"bytes": T * d * b * (1 + 2 * post + pre) + vec, "flops": T * d * (6 * post + 4 * pre)}
        # dz and y, dh and z; dx and dy
        moved = T * d * b * (2 * post + 2 * pre + 1 + post) + vec + 4 * d * (post + pre + gates) + 4 * T * (post + pre)
        return {"bytes": moved, "flops": T * d * (10 * post + 8 * pre)}
    T, E, k = case["T"], case["E"], case["k"]
    # the logits; indices and weights, or indices, their gradients and the gradient of the logits
    return {"bytes": T * E * 4 * (2 if case["backward"] else 1) + T * k * 8, "flops": T * E * 8}


# ---------------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    f64 = lambda t: t.to(torch.float64)  # noqa: E731
    if case["op"] == "product":
        # a row's scale is the fp32 quotient of its largest magnitude and 127; the codes are the
        # whole numbers nearest to the fp32 quotients of the row and its scale
        out = torch.empty((case["rows"], case["N"]), dtype=torch.float64, device=s["x"].device)
        row = 0
        for g, n in enumerate(s["sizes"]):
            if n:
                x = f64(s["x"][row:row + n])
                sc = f64((x.abs().amax(1) / 127.0).to(F32))[:, None]
                sc[sc == 0] = 1.0
                codes = torch.clamp(torch.round(f64((x / sc).to(F32))), -127, 127)
                y = codes @ f64(s["W1"][g]).T * sc * f64(s["s1"][g])
                if case["swiglu"]:
                    y = y * torch.sigmoid(y) * (codes @ f64(s["W3"][g]).T * sc * f64(s["s3"][g]))
                out[row:row + n] = y
                row += n
        return out
    if case["op"] == "norm":
        T = case["T"]
        gate = 1.0
        if s["gate"] is not None:
            gate = f64(s["gate"]).repeat_interleave(case["gate_span"], 0)[:T]
        rms = lambda v, w: v * torch.rsqrt(v.square().mean(1, keepdim=True) + EPS) * w  # noqa: E731
        if not case["backward"]:
            z = case["alpha"] * f64(s["x"]) + gate * rms(f64(s["y"]), f64(s["w_post"])) if case["post"] else None
            # h is the norm of z as it is stored
            kept = f64(s["x"]) if z is None else f64(z.to(DTYPES[case["dtype"]]))
            return dict(z=z, h=rms(kept, f64(s["w_pre"])) if case["pre"] else None)
        # by differentiation of the forward formulas at the stored z
        out, grad = {}, None if s["dz"] is None else f64(s["dz"])
        with torch.enable_grad():
            if case["pre"]:
                v = f64(s["z"] if case["post"] else s["x"]).requires_grad_()
                w = f64(s["w_pre"]).requires_grad_()
                dv, out["dw_pre"] = torch.autograd.grad(rms(v, w), (v, w), f64(s["dh"]))
                grad = dv if grad is None else grad + dv
            if not case["post"]:
                return dict(out, dx=grad)
            x, y, w = (f64(s[n]).requires_grad_() for n in ("x", "y", "w_post"))
            leaf = f64(s["gate"]).requires_grad_() if s["gate"] is not None else None
            full = 1.0 if leaf is None else leaf.repeat_interleave(case["gate_span"], 0)[:T]
            got = torch.autograd.grad(case["alpha"] * x + full * rms(y, w), (x, y, w) + ((leaf,) if leaf is not None else ()), grad)
        out.update(zip(("dx", "dy", "dw_post", "dgate"), got))
        return out
    logits = f64(s["logits"])
    if not case["backward"]:
        score = torch.sigmoid(logits) if case["score"] == "sigmoid" else torch.softmax(logits, 1)
        key = score.clone() if s["sel_bias"] is None else score + f64(s["sel_bias"])
        n, E = case["groups"], case["E"]
        if n > 1:
            total = key.view(-1, n, E // n).topk(case["top"], 2)[0].sum(2)
            order = torch.argsort(-total, dim=1, stable=True)
            rank = torch.empty_like(order).scatter_(1, order, torch.arange(n, device=order.device).expand_as(order).contiguous())
            key[(rank >= case["keep"]).repeat_interleave(E // n, 1)] = -math.inf
        idx = torch.argsort(-key, dim=1, stable=True)[:, :case["k"]]
        w = torch.gather(score, 1, idx)
        if s["k_per_token"] is not None:
            pad = torch.arange(case["k"], device=idx.device) >= s["k_per_token"][:, None]
            w[pad], idx[pad] = 0.0, -1
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        return dict(topk_idx=idx.to(torch.int32), topk_w=case["scale"] * w)
    with torch.enable_grad():
        leaf = logits.requires_grad_()
        score = torch.sigmoid(leaf) if case["score"] == "sigmoid" else torch.softmax(leaf, 1)
        live = s["topk_idx"] >= 0
        w = torch.gather(score, 1, s["topk_idx"].clamp(min=0).long()) * live
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        return torch.autograd.grad(case["scale"] * w, leaf, f64(s["dtopk_w"]))[0]
