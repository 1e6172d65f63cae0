"""Pins of the float64 oracle of the operators on vocabulary rows, and the refusals of their entry points
(argument checks on the host: nothing here needs a GPU)."""
import ctypes as C

import numpy as np
import pytest
import torch

from eagle_speculative_decoding_02_gb300 import _lib as L
from eagle_speculative_decoding_02_gb300 import build as B
from oracle import vocab as OV


def test_logprobs_by_hand():
    z = np.log([0.5, 0.125, 0.25, 0.125])
    lp, h, lse, idx, val = OV.token_logprobs(z + 3, 2, 3)
    assert np.isclose(lp, np.log(0.25)) and np.isclose(lse, 3) and np.isclose(h, 1.75 * np.log(2))
    assert idx.tolist() == [0, 2, 1] and np.allclose(val, np.log([0.5, 0.25, 0.125]))
    assert np.isclose(OV.token_logprobs(z, 0, 0, temperature=0.5)[0], np.log(0.25 / (0.25 + 2 / 64 + 1 / 16)))
    masked = np.array([-np.inf, 1.0, -np.inf, 1.0])
    lp, h, lse, idx, val = OV.token_logprobs(masked, 0, 3)
    assert lp == -np.inf and np.isclose(h, np.log(2)) and idx.tolist() == [1, 3, -1] and val[2] == -np.inf
    for bad in (np.full(3, -np.inf), np.array([1, np.nan, 2]), np.array([1, np.inf, 2])):
        lp, h, lse, idx, val = OV.token_logprobs(bad, 1, 2)
        assert np.isnan([lp, h, lse, *val]).all() and idx.tolist() == [-1, -1]


@pytest.mark.parametrize("tail", [True, False])
def test_distill_is_a_divergence_with_its_gradient(tail):
    """Zero exactly at the teacher; the gradient equals central differences of the loss."""
    rng = np.random.default_rng(1)
    V, T = 23, 0.8
    t = np.log(rng.dirichlet(np.ones(V)))
    idx = rng.permutation(V)[:6]
    z0 = t * T if tail else np.where(np.isin(np.arange(V), idx), t * T, -np.inf)
    assert abs(OV.distill(z0, idx, t[idx], T, tail)[0]) < 1e-12
    z = rng.standard_normal(V)
    loss, stats, d = OV.distill(z, idx, t[idx], T, tail, g=1.5)
    assert loss > 0
    eps = 1e-5
    for j in range(V):
        e = np.eye(V)[j] * eps
        num = (OV.distill(z + e, idx, t[idx], T, tail)[0] - OV.distill(z - e, idx, t[idx], T, tail)[0]) / (2 * eps)
        assert abs(1.5 * num - d[j]) < 1e-8
    assert np.isclose(stats[1], np.log(np.exp((z - z.max()) / T).sum()))
    if tail:
        rest = ~np.isin(np.arange(V), idx)
        assert stats[2] == z[rest].max() and np.isclose(stats[3], np.log(np.exp((z - z[rest].max()) / T)[rest].sum()))
    else:
        assert stats[2:].tolist() == [0, 0]


def test_distill_rows_with_little_to_learn_from():
    z = np.array([1.0, 2.0, 3.0])
    assert OV.distill(z, [-1, -1], [0.0, np.nan])[0] == 0.0
    assert OV.distill([np.nan] * 3, [-1], [0.0])[0] == 0.0
    assert np.isnan(OV.distill(z, [3], [-1.0])[0]) and np.isnan(OV.distill(z, [-2], [-1.0])[0])
    assert np.isnan(OV.distill([np.nan, 1, 2], [0], [-1.0])[0])
    a, b = OV.distill(z, [1, 1], [-0.5, -3.0]), OV.distill(z, [1, -1], [-0.5, 0.0])
    assert a[0] == b[0] and (a[2] == b[2]).all()
    # every token listed: no other outcome, however the probabilities are rounded
    assert np.isfinite(OV.distill(z, [0, 1, 2], np.log([0.5, 0.25, 0.2]))[0])


@pytest.fixture(scope="module")
def lib():
    B.build_lib()
    return L.load()


# dummy addresses, never read: every call below is refused (or has no rows) before any CUDA call
P = 1 << 20
GOOD = {"eagle_op_token_logprobs": dict(dtype=0, rows=4, vocab=100, ld=100, z=P, tok=P, T=1.0, k=5, lp=P, ent=P,
                                        lse=P, idx=P, val=P, stream=None),
        "eagle_op_distill_loss": dict(dtype=0, rows=4, vocab=100, ld=100, z=P, k=5, idx=P, lp=P, T=1.0, tail=1,
                                      loss=P, stats=P, stream=None),
        "eagle_op_distill_grad": dict(dtype=0, rows=4, vocab=100, ld=100, z=P, k=5, idx=P, lp=P, T=1.0, tail=1,
                                      stats=P, g=P, ld_out=100, dz=2 * P, stream=None),
        "eagle_op_distill_loss_grad": dict(dtype=0, rows=4, vocab=100, ld=100, z=P, k=5, idx=P, lp=P, T=1.0, tail=1,
                                           g=P, loss=P, stats=P, ld_out=100, dz=2 * P, stream=None)}
BAD_ROWS = [dict(dtype=3), dict(dtype=-1), dict(rows=-1), dict(vocab=0), dict(vocab=-5), dict(ld=99), dict(z=None),
            dict(z=P + 2), dict(dtype=1, z=P + 1), dict(dtype=2, z=P + 1), dict(T=0.0), dict(T=-1.0),
            dict(T=float("nan")), dict(T=float("inf")), dict(T=1e-7), dict(T=2e6), dict(ld=1 << 62)]
BAD_TEACHER = [dict(k=0), dict(k=65), dict(idx=None), dict(lp=None), dict(tail=2), dict(tail=-1)]
# of 4-byte elements: rows of the gradient that reach into rows of the logits
BAD_OUT = [dict(dz=None), dict(dz=P + 4), dict(dz=P - 4), dict(dz=P, ld_out=101), dict(dz=P + 400, ld_out=100),
           dict(ld=150, ld_out=150, dz=P + 4 * 60), dict(ld_out=99), dict(dz=2 * P + 1), dict(g=None),
           dict(ld=150, ld_out=150, dz=P - 4 * 60)]
BAD = {"eagle_op_token_logprobs": BAD_ROWS + [dict(k=-1), dict(k=65), dict(tok=None), dict(lp=None), dict(idx=None),
                                              dict(val=None)],
       "eagle_op_distill_loss": BAD_ROWS + BAD_TEACHER + [dict(loss=None), dict(stats=None)],
       "eagle_op_distill_grad": BAD_ROWS + BAD_TEACHER + BAD_OUT + [dict(stats=None)],
       # the sums may be left out but for rows that take two passes
       "eagle_op_distill_loss_grad": BAD_ROWS + BAD_TEACHER + BAD_OUT + [
           dict(loss=None), dict(stats=None, vocab=196609, ld=196609, ld_out=196609, dz=1 << 40)]}


@pytest.mark.parametrize("fn,over", [(f, o) for f in BAD for o in BAD[f]])
def test_refusals_on_the_host(lib, fn, over):
    assert getattr(lib, fn)(*{**GOOD[fn], **over}.values()) == 1


@pytest.mark.parametrize("fn", list(GOOD))
def test_no_rows_is_no_work(lib, fn):
    kw = dict(GOOD[fn], rows=0)
    kw.update({k: None for k, v in kw.items() if v in (P, 2 * P)})
    assert getattr(lib, fn)(*kw.values()) == 0


def test_binding_refuses_host_tensors_and_types():
    from eagle_speculative_decoding_02_gb300 import op_distill_loss, op_token_logprobs
    with pytest.raises(ValueError):
        op_token_logprobs(torch.zeros(2, 8))
    with pytest.raises(TypeError):
        op_token_logprobs(torch.zeros(2, 8, dtype=torch.float64))
    with pytest.raises(ValueError):
        op_distill_loss(torch.zeros(2, 8), torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1))


# the gradient's rows (of 400 bytes, from 2 P on; with ld_out = 200 every 800 bytes) and another array of the call
MEETS = [(f, o) for f in ("eagle_op_distill_grad", "eagle_op_distill_loss_grad") for o in
         [dict(idx=2 * P), dict(idx=2 * P + 1596), dict(idx=2 * P - 76), dict(lp=2 * P + 400), dict(lp=2 * P - 4, ld_out=200),
          dict(g=2 * P - 12), dict(g=2 * P + 1596), dict(g=2 * P + 1600 + 396, ld_out=200), dict(g=2 * P + 796, ld_out=200),
          dict(stats=2 * P - 60), dict(stats=2 * P + 1200), dict(stats=2 * P + 2400 - 60, ld_out=200),
          dict(k=64, idx=2 * P - 1020), dict(dtype=1, ld_out=101, idx=2 * P + 200 + 204 * 2)]]
MEETS += [("eagle_op_distill_loss_grad", o) for o in [dict(loss=2 * P), dict(loss=2 * P - 12), dict(loss=2 * P + 1596)]]


@pytest.mark.parametrize("fn,over", MEETS)
def test_gradients_over_other_arguments_are_refused(lib, fn, over):
    assert getattr(lib, fn)(*{**GOOD[fn], **over}.values()) == 1


ODD = [("eagle_op_token_logprobs", n) for n in ("tok", "lp", "ent", "lse", "idx", "val")] + \
    [("eagle_op_distill_loss", n) for n in ("idx", "lp", "loss", "stats")] + \
    [("eagle_op_distill_grad", n) for n in ("idx", "lp", "stats", "g")] + \
    [("eagle_op_distill_loss_grad", n) for n in ("idx", "lp", "g", "loss", "stats")]


@pytest.mark.parametrize("fn,name", ODD)
def test_arrays_off_their_elements_size_are_refused(lib, fn, name):
    for off in (1, 2, 3):
        assert getattr(lib, fn)(*{**GOOD[fn], name: P + off}.values()) == 1


def test_teachers_whose_sum_overflows_are_broken():
    """Each exponential fits float32, their sum does not; a twice given token counts once."""
    z = np.zeros(9)
    assert np.isnan(OV.distill(z, [1, 2], [88.5, 88.5])[0]) and np.isnan(OV.distill(z, [1, 2], [88.5, 88.5])[2]).all()
    assert np.isfinite(OV.distill(z, [1, 1], [88.5, 88.5])[0]) and np.isfinite(OV.distill(z, [1, 2], [88.5, 80.0])[0])
    assert np.isfinite(OV.distill(z, [1, 2], [88.5, 88.5], tail=False)[0])
