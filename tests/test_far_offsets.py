"""Tensors of more than 2^31 elements: rows, groups and tokens behind that
border come out as in a call that has them alone, bit for bit."""
import pytest
import torch

from routing_dispatch_expert_sigmoid_b200 import ops

BORDER = 2 ** 31
pytestmark = pytest.mark.gpu


def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    torch.cuda.empty_cache()
    g = torch.Generator(device="cuda")
    g.manual_seed(31)
    return torch.device("cuda:0"), g


def normal(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def test_norm_rows():
    d, gen = dev()
    D, far = 4096, 65
    T = BORDER // D + far
    x, y = normal(gen, T, D), normal(gen, T, D)
    w_post, w_pre, gate = normal(gen, D), normal(gen, D), normal(gen, 1, D)
    last = [v[-far:].clone() for v in (x, y)]
    rs = [torch.empty(T, device=d) for _ in range(2)]
    ops.moe_norm(ops.norm_config(T, D, gate_span=T), x, y=y, w_post=w_post, gate=gate, w_pre=w_pre,
                 z=x, h=y, rstd_post=rs[0], rstd_pre=rs[1])
    z, h, one = torch.empty_like(last[0]), torch.empty_like(last[0]), [torch.empty(far, device=d) for _ in range(2)]
    ops.moe_norm(ops.norm_config(far, D, gate_span=far), last[0], y=last[1], w_post=w_post, gate=gate,
                 w_pre=w_pre, z=z, h=h, rstd_post=one[0], rstd_pre=one[1])
    assert torch.equal(x[-far:], z) and torch.equal(y[-far:], h)
    assert torch.equal(rs[0][-far:], one[0]) and torch.equal(rs[1][-far:], one[1])
    # the gradient, its outputs in the places of dz and dh
    dz, dh = normal(gen, T, D), normal(gen, T, D)
    near = [v[-far:].clone() for v in (dz, dh, x, y)]
    kw = dict(w_post=w_post, gate=gate, w_pre=w_pre)
    ops.moe_norm_backward(ops.norm_config(T, D, gate_span=T), dz=dz, dh=dh, z=x, y=y,
                          rstd_post=rs[0], rstd_pre=rs[1], dx=dz, dy=dh, **kw)
    dx, dy = torch.empty_like(z), torch.empty_like(z)
    ops.moe_norm_backward(ops.norm_config(far, D, gate_span=far), dz=near[0], dh=near[1], z=near[2],
                          y=near[3], rstd_post=one[0], rstd_pre=one[1], dx=dx, dy=dy, **kw)
    assert torch.equal(dz[-far:], dx) and torch.equal(dh[-far:], dy)
    ops.moe_check_errors()


def test_gate_tokens():
    d, gen = dev()
    E, k, far = 512, 8, 9
    T = BORDER // E + far
    l = normal(gen, T, E, dtype=torch.float32)
    b = normal(gen, E, dtype=torch.float32) * 0.05
    for mode in ("softmax", "sigmoid_renorm"):
        res = []
        for rows in (l, l[-far:].clone()):
            n = rows.shape[0]
            cfg = ops.gate_config(n, E, k, mode, 4, 2, 2)
            idx = torch.empty(n, k, dtype=torch.int32, device=d)
            w = torch.empty(n, k, device=d)
            ops.moe_gate(cfg, rows, b, None, idx, w)
            grad = torch.empty(n, E, device=d)
            ops.moe_gate_backward(cfg, rows, idx, w, grad)
            res.append([v[-far:].clone() for v in (idx, w, grad)])
            del idx, w, grad
        assert all(torch.equal(p, q) for p, q in zip(*res))
    ops.moe_check_errors()


def test_int8_rows():
    d, gen = dev()
    K = N = 2048
    far = 5
    rows = BORDER // K + far
    x = normal(gen, rows, K)
    W = torch.randint(-127, 128, (1, N, K), generator=gen, device=d, dtype=torch.int8)
    s = torch.rand((1, N), generator=gen, device=d) + 0.5
    res = []
    for v in (x, x[-far:].clone()):
        lin = ops.int8_linear(v.shape[0], K, N, 1)
        out = torch.empty(v.shape[0], N, device=d, dtype=torch.bfloat16)
        ops.moe_linear_int8(lin, v, None, W, s, None, None, out, ops.int8_workspace(lin))
        res.append(out[-far:].clone())
        del out
    assert torch.equal(*res)
    ops.moe_check_errors()


@pytest.mark.parametrize("each", (0, 1, 200))
def test_int8_groups(each):
    """`each` rows a group: two rows of the last group alone, then groups for the
    engines of few and of many rows."""
    d, gen = dev()
    K = N = 2048
    G = BORDER // (N * K) + 1
    W = torch.randint(-127, 128, (G, N, K), generator=gen, device=d, dtype=torch.int8)
    s = torch.rand((G, N), generator=gen, device=d) + 0.5
    sizes = [each] * (G - 1) + [max(each, 2)]
    rows = sum(sizes)
    x = normal(gen, rows, K)
    off = torch.tensor([0] + sizes, device=d).cumsum(0).to(torch.int32)
    lin = ops.int8_linear(rows, K, N, G)
    out = torch.empty(rows, N, device=d, dtype=torch.bfloat16)
    ops.moe_linear_int8(lin, x, off, W, s, None, None, out, ops.int8_workspace(lin))
    n = sizes[-1]
    one = ops.int8_linear(n, K, N, 1)
    ref = torch.empty(n, N, device=d, dtype=torch.bfloat16)
    ops.moe_linear_int8(one, x[-n:].clone(), None, W[-1:].clone(), s[-1:].clone(), None, None, ref,
                        ops.int8_workspace(one))
    assert torch.equal(out[-n:], ref)
    ops.moe_check_errors()
