"""The norms' values again, every one compared: a NaN is off, whatever it is
compared with, and what is finite in 64 bits has to be finite.

The cases, the fp64 formulas and the tolerances are those of test_norm; where no
gradient arrives at z, none is counted in the tolerances either.
"""
import pytest
import torch

import test_norm
from test_norm import Case, SIZES, check_backward, check_forward, dev, f64


def near(got, ref, tol, what):
    err = (f64(got) - ref).abs()
    off = ~(err <= tol)  # a comparison with NaN is False
    assert not off.any(), f"{what}: {int(off.sum())} off, {int(got.isnan().sum())} of them NaN"
    assert bool((got.isfinite() | ~ref.isfinite()).all()), f"{what}: not finite"


@pytest.fixture(autouse=True)
def every_value_counts(monkeypatch):
    monkeypatch.setattr(test_norm, "near", near)


def run(c, dz=True, codes=False):
    if not dz:
        c.dz.zero_()  # nothing arrives at z, and nothing of it enters a tolerance
    o = c.forward(codes)
    check_forward(c, o)
    check_backward(c, o, c.backward(o, dz), dz)


def test_nan_and_infinity_are_off():
    one = torch.ones(3, dtype=torch.float64)
    near(torch.ones(3), one, one * 1e-6, "ones")
    for v in (float("nan"), float("inf")):
        for got in (torch.full((3,), v), torch.tensor([1.0, v, 1.0])):
            with pytest.raises(AssertionError):
                test_norm.near(got, one, one * 1e-6, "x")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("T,d", SIZES)
@pytest.mark.parametrize("parts,dz", [("both", True), ("both", False), ("post", True),
                                      ("pre", True), ("pre", False)])
def test_forward_and_backward(dtype, T, d, parts, dz):
    run(Case(T, d, dtype, post=parts != "pre", pre=parts != "post", span=3 if parts == "both" else 0,
             device=dev()), dz)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("T,d", [(1, 8), (33, 264), (300, 4096)])
@pytest.mark.parametrize("span", (0, 1, 10, 400))
def test_residual_without_a_post_norm(dtype, T, d, span):
    run(Case(T, d, dtype, pre=False, span=span, normed=False, device=dev()))
    for dz in (True, False):
        run(Case(T, d, dtype, span=span, normed=False, device=dev()), dz)


@pytest.mark.gpu
@pytest.mark.parametrize("d", (7176, 8192, 8200, 12288, 16384))
@pytest.mark.parametrize("dz", (True, False))
def test_long_rows(d, dz):
    run(Case(301, d, "bf16", span=100, device=dev()), dz, codes=True)
    run(Case(37, d // 8 * 4, "f32", span=2, device=dev()), dz, codes=True)


@pytest.mark.gpu
@pytest.mark.parametrize("span", (1, 2, 7, 64, 999, 1000, 1001, 5000, 2 ** 31 - 1))
@pytest.mark.parametrize("d", (128, 4096))
def test_gate_spans(span, d):
    run(Case(1000, d, "bf16", span=span, device=dev()))


@pytest.mark.gpu
@pytest.mark.parametrize("T", (148, 149, 296, 700, 4001))
def test_gate_rows_across_the_ranges_of_ctas(T):
    for span in (T // 3, T // 148 + 1, 5, T - 1):
        run(Case(T, 512, "f32", span=span, pre=False, device=dev()))
        run(Case(T, 512, "f32", span=span, device=dev()), dz=False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("dz", (True, False))
def test_without_weights_and_without_a_post_norm(dtype, dz):
    run(Case(33, 256, dtype, weights=False, device=dev()), dz)
    run(Case(9, 264, dtype, post=False, device=dev()), dz)
    run(Case(9, 264, dtype, post=False, weights=False, device=dev()), dz)
