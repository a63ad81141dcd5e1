"""General gating where 32-bit words of the keys cannot carry the selection.

The selection has to be that of the scores in 64 bits also where keys are -inf
(experts that a bias masks) and groups have fewer experts left than scores that
are summed, where keys lie too far apart for steps of one size, and where a bias
cancels the scores so far that fp32 leaves nothing of their order.
"""
import numpy as np
import pytest

from routing_dispatch_expert_sigmoid_b200 import ops
from test_gate_general import MODES, W_REL, dev, ref_gate, ref_scores, run_gate

# E, k, groups, kept groups: groups of 32, 64 and 128 experts (whole registers of
# a warp) and of other sizes (scanned in shared memory)
GROUPED = [(64, 6, 2, 1), (256, 8, 8, 4), (96, 5, 3, 2), (192, 7, 3, 1), (512, 16, 8, 3),
           (256, 8, 2, 1), (1024, 32, 8, 5), (64, 6, 8, 3), (160, 6, 8, 3), (40, 3, 5, 2),
           (384, 7, 4, 2)]


def check(l, mode, k, b, groups, keep, top):
    T, E = l.shape
    cfg = ops.gate_config(T, E, k, mode, groups, keep, top, 1.5)
    idx, w = run_gate(cfg, l, b, None, dev())
    ridx, rw = ref_gate(l, mode, k, b, None, groups, keep, top, 1.5)
    off = np.argwhere((idx != ridx).any(1))[:, 0]
    assert off.size == 0, f"{off.size} of {T} rows, first {off[:4].tolist()}"
    np.testing.assert_allclose(w, rw, rtol=W_REL, atol=0)
    ops.moe_check_errors()


@pytest.mark.gpu
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("top", (2, 3))
def test_a_group_with_too_few_experts_left_goes_last(mode, top):
    """Two experts of large scores and 30 masked ones against 32 of small scores:
    a sum over three, or over two of one, is -inf."""
    l = np.full((2, 64), -1.0, np.float32)
    l[:, :2] = 6.0
    b = np.zeros(64, np.float32)
    b[top - 1:32] = -np.inf
    if top == 2:
        b[32:] = -0.75  # keys below zero are above -inf too
    check(l, mode, 6, b, 2, 1, top)


@pytest.mark.gpu
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("shape", GROUPED, ids=lambda s: f"E{s[0]}k{s[1]}g{s[2]}")
@pytest.mark.parametrize("masked", (0.3, 0.9, 0.98))
@pytest.mark.parametrize("shift", (0.0, -1.5))
def test_masked_experts_in_groups(mode, shape, masked, shift):
    E, k, groups, keep = shape
    T = 96
    rng = np.random.default_rng(E * 5 + groups)
    for top in (1, 2, 3, min(8, E // groups)):
        l = np.clip(rng.standard_normal((T, E)) * 1.5, -8, 8).astype(np.float32)
        b = (shift + rng.standard_normal(E) * 0.05).astype(np.float32)
        b[rng.random(E) < masked] = -np.inf
        check(l, mode, k, b, groups, keep, top)


@pytest.mark.gpu
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("shape", GROUPED, ids=lambda s: f"E{s[0]}k{s[1]}g{s[2]}")
def test_groups_without_a_finite_sum_tie(mode, shape):
    """One expert left in every group but the last, whatever its key: sums of two
    are -inf, and the groups of the lowest index follow the last one."""
    E, k, groups, keep = shape
    T, gsz = 40, E // groups
    rng = np.random.default_rng(E + keep)
    l = np.clip(rng.standard_normal((T, E)) * 1.5, -8, 8).astype(np.float32)
    b = np.full(E, -np.inf, np.float32)
    b[::gsz] = 0.0
    b[-gsz:] = rng.standard_normal(gsz) * 0.05 - 2.0
    check(l, mode, k, b, groups, keep, 2)


@pytest.mark.gpu
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("shape", GROUPED, ids=lambda s: f"E{s[0]}k{s[1]}g{s[2]}")
@pytest.mark.parametrize("kind", ("spread", "lowest", "two masks"))
def test_groups_of_keys_at_the_end_of_the_range(mode, shape, kind):
    """Biases up to the type's limits: sums of keys that are more than any range
    of fp32 steps below the largest."""
    E, k, groups, keep = shape
    T = 24
    for seed in range(6):
        rng = np.random.default_rng(E * 11 + groups + seed)
        l = np.clip(rng.standard_normal((T, E)) * 1.5, -8, 8).astype(np.float32)
        low = np.finfo(np.float32).min
        if kind == "spread":
            b = (rng.standard_normal(E) * 10.0 ** rng.uniform(30, 37.9, E)).astype(np.float32)
        else:
            b = (rng.standard_normal(E) * 0.05).astype(np.float32)
            b[rng.random(E) < 0.6] = low
            if kind == "two masks":  # the keys of the second are below the range as well
                b[rng.random(E) < 0.4] = low / 16
        for top in (1, 2, 3, min(8, E // groups)):
            check(l, mode, k, b, groups, keep, top)


@pytest.mark.gpu
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("shape", [(128, 8, 1, 1), (64, 6, 1, 1), (80, 9, 1, 1), (1024, 32, 1, 1),
                                   (512, 16, 8, 3)] + GROUPED, ids=lambda s: f"E{s[0]}k{s[1]}g{s[2]}")
@pytest.mark.parametrize("offset", (0.0, 1e-9, 1e-7))
def test_a_bias_that_cancels_the_scores(mode, shape, offset):
    """Keys that are the rounding of the bias, and small offsets: the error of an
    fp32 score is many times the largest of them."""
    E, k, groups, keep = shape
    for seed in range(12):
        rng = np.random.default_rng(E * 3 + groups + seed)
        l = (rng.standard_normal((1, E)) * (1.5, 4.0)[seed % 2]).astype(np.float32)
        s = ref_scores(l.astype(np.float64), mode)[0]
        b = (-s + rng.standard_normal(E) * offset).astype(np.float32)
        # rows of the same logits, and of logits a unit in the last place beside them
        l = np.repeat(l, 8, 0)
        l[4:] = np.nextafter(l[4:], np.float32(99) * rng.choice([-1, 1], (4, E)), dtype=np.float32)
        check(l, mode, k, b, groups, keep, min(2, groups))
