"""Gradients of the combine weights for rows that are not ordinary: logits that are
not finite, rows without a slot, and scores far below the largest.
"""
import numpy as np
import pytest

from routing_dispatch_expert_sigmoid_b200 import ops
from test_gate_general import MODES, dev, ref_gate, run_grad

FIXED = ("topk_softmax", "softmax_topk_renorm", "sigmoid_grouped")


@pytest.mark.gpu
@pytest.mark.parametrize("mode", MODES + FIXED)
@pytest.mark.parametrize("E", (33, 64, 512))
def test_rows_that_are_not_finite(mode, E):
    """The weights of such a row are NaN in the general modes, and so is what its
    loss tells of the logits: NaN must not turn into a gradient of zero."""
    d = dev()
    T, k = 12, 4
    rng = np.random.default_rng(E)
    l = rng.standard_normal((T, E)).astype(np.float32)
    idx, _ = ref_gate(l, "softmax", k)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    cfg = ops.gate_config(T, E, k, mode)
    clean = run_grad(cfg, l, idx, dw, d)
    assert np.isfinite(clean).all()
    bad, slots, grads = l.copy(), idx.copy(), dw.copy()
    bad[1, idx[1, 2]] = np.nan                    # a selected logit
    bad[2, idx[2, 0]] = np.inf
    bad[3, idx[3, 3]] = bad[3, idx[3, 1]] = np.inf
    last = [next(e for e in range(E) if e not in idx[t]) for t in range(T)]
    bad[4, last[4]] = np.nan                      # one that is not selected
    slots[5:8], grads[5:8] = -1, np.nan           # no slot at all
    bad[6, 3], bad[7] = np.nan, np.inf
    slots[8, 1:], grads[8, 1:] = -1, np.nan       # one slot, the others empty
    bad[9, last[9]] = -np.inf                     # masked, not selected
    got = run_grad(cfg, bad, slots, grads, d)
    ops.moe_check_errors()
    dense = mode == "softmax"
    for t in (1, 2, 3):
        hit = np.zeros(E, bool)
        hit[idx[t]] = True
        assert np.isnan(got[t][hit]).all()
        assert np.isnan(got[t][~hit]).all() if dense else (got[t][~hit] == 0).all()
    if dense:
        assert np.isnan(got[4]).all()
    else:
        assert (got[4] == clean[4]).all()
    assert (got[5:8] == 0).all()
    assert np.isfinite(got[8]).all() and (got[8] != 0).any() == (not mode.endswith("renorm") and mode not in FIXED)
    assert np.isfinite(got[9]).all() and (got[9, last[9]] == 0)
    assert (got[[0, 10, 11]] == clean[[0, 10, 11]]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("E", (9, 64))
def test_small_scores_keep_their_digits(E):
    """One expert of logit 0, selected, the others at -20 .. -80: the softmax's sum
    is 1 to the last bit, so an expert's gradient is -g e^l with the error of expf
    (2 units of 2^-23, 4 of 2^-24) and three roundings."""
    d = dev()
    rng = np.random.default_rng(E)
    l = (-rng.uniform(20, 80, (50, E))).astype(np.float32)
    l[:, 5] = 0
    idx = np.full((50, 1), 5, np.int32)
    dw = rng.standard_normal((50, 1)).astype(np.float32)
    got = run_grad(ops.gate_config(50, E, 1, "softmax"), l, idx, dw, d)
    ops.moe_check_errors()
    ref = -dw.astype(np.float64) * np.exp(l.astype(np.float64))
    rest = np.arange(E) != 5
    np.testing.assert_allclose(got[:, rest], ref[:, rest], rtol=7 * 2.0 ** -24, atol=0)
