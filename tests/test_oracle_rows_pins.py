"""Pins of the row operators' oracle (oracle/rows.py) on the CPU: against torch's float64 autograd
on formulas written separately, against differences, and at rows with closed forms."""

import numpy as np
import pytest
import torch

from oracle import rows


def _rng(seed):
    return np.random.default_rng(seed)


@pytest.mark.parametrize("T,H,affine", [(3, 7, True), (5, 64, False), (1, 1, True)])
def test_layer_norm_and_gradient(T, H, affine):
    g = _rng(T + H)
    x = torch.tensor(g.standard_normal((T, H)) + 3.0, requires_grad=True)
    ga = torch.tensor(g.standard_normal(H), requires_grad=True)
    be = torch.tensor(g.standard_normal(H), requires_grad=True)
    dy = g.standard_normal((T, H))
    out = torch.nn.functional.layer_norm(x, (H,), ga if affine else None, be if affine else None,
                                         eps=1e-3)
    y, mean, rstd = rows.layer_norm(x.detach(), *((ga.detach(), be.detach()) if affine else ()),
                                    eps=1e-3)
    np.testing.assert_allclose(y, out.detach(), rtol=1e-12, atol=1e-12)
    out.backward(torch.tensor(dy))
    dx, dg, db = rows.layer_norm_backward(dy, x.detach(), ga.detach() if affine else None, mean,
                                          rstd)
    np.testing.assert_allclose(dx, x.grad, rtol=1e-10, atol=1e-10)
    if affine:
        np.testing.assert_allclose(dg, ga.grad, rtol=1e-10, atol=1e-10)
        np.testing.assert_allclose(db, be.grad, rtol=1e-10, atol=1e-10)


def test_layer_norm_gradient_by_differences():
    g = _rng(1)
    x, ga, dy = g.standard_normal((2, 5)), g.standard_normal(5), g.standard_normal((2, 5))
    f = lambda v: (rows.layer_norm(v, ga, None)[0] * dy).sum()
    _, mean, rstd = rows.layer_norm(x, ga)
    dx, _, _ = rows.layer_norm_backward(dy, x, ga, mean, rstd)
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = 1e-6
        assert abs((f(x + e) - f(x - e)) / 2e-6 - dx[i]) < 1e-7


@pytest.mark.parametrize("tau", [1.0, 0.5, 3.0])
def test_token_logprobs_and_gradient(tau):
    g = _rng(int(10 * tau))
    T, V = 4, 11
    z = torch.tensor(2 * g.standard_normal((T, V)), requires_grad=True)
    y = np.array([0, 10, -100, 5])
    lp = torch.log_softmax(z / tau, 1)
    ent = -(lp.exp() * lp).sum(1)
    got = rows.token_logprobs(z.detach(), y, tau, top=3)
    pick = torch.where(torch.tensor(y) >= 0, lp[torch.arange(T), torch.tensor(y).clamp(min=0)], 0.0)
    np.testing.assert_allclose(got["logprob"], pick.detach(), rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(got["entropy"], ent.detach(), rtol=1e-12)
    v, i = z.detach().topk(3, dim=1)
    np.testing.assert_array_equal(got["top_index"], i)
    np.testing.assert_allclose(got["top_logprob"], lp.detach().gather(1, i), rtol=1e-12)
    a, b = g.standard_normal(T), g.standard_normal(T)
    ((pick * torch.tensor(a)).sum() + (ent * torch.tensor(b)).sum()).backward()
    np.testing.assert_allclose(rows.token_logprobs_backward(z.detach(), y, tau, a, b), z.grad,
                               rtol=1e-10, atol=1e-12)


def test_token_logprobs_rows_with_closed_forms():
    inf = np.inf
    z = np.array([[-inf] * 4, [0.0] * 4, [-inf, 5.0, -inf, -inf], [0, np.nan, 0, 0], [0, inf, 0, 0]])
    r = rows.token_logprobs(z, np.array([1, 1, 1, 1, 1]), 1.0, top=2)
    np.testing.assert_allclose(r["entropy"], [0, np.log(4), 0, np.nan, np.nan])
    np.testing.assert_allclose(r["logprob"], [-inf, -np.log(4), 0, np.nan, np.nan])
    np.testing.assert_array_equal(r["top_index"], [[0, 1], [0, 1], [1, 0], [-1, -1], [-1, -1]])
    d = rows.token_logprobs_backward(z, np.array([1] * 5), 1.0, np.ones(5), np.ones(5))
    np.testing.assert_array_equal(d[0], 0)
    np.testing.assert_allclose(d[1], [-.25, .75, -.25, -.25])
    np.testing.assert_array_equal(d[2], 0)
    assert np.isnan(d[3:]).all()
    z0 = rows.token_logprobs_backward(z, np.array([-1] * 5), 1.0, np.ones(5))
    np.testing.assert_array_equal(z0, 0)


@pytest.mark.parametrize("tau", [1.0, 2.0])
def test_distill_and_gradient(tau):
    g = _rng(int(tau))
    T, V, K = 4, 13, 5
    z = torch.tensor(2 * g.standard_normal((T, V)), requires_grad=True)
    idx = np.stack([g.permutation(V)[:K] for _ in range(T)])
    idx[1, 3:] = -1
    idx[2, 4] = idx[2, 1]  # the same token twice
    idx[3] = -1
    t = g.standard_normal((T, K))
    lp = torch.log_softmax(z / tau, 1)
    total = 0
    d = g.standard_normal(T)
    ref = []
    for r in range(T):
        used = idx[r] >= 0
        if not used.any():
            ref.append(0.0)
            continue
        w = torch.softmax(torch.tensor(t[r, used]) / tau, 0)
        loss = (w * (w.log() - lp[r, torch.tensor(idx[r, used])])).sum()
        ref.append(loss.item())
        total = total + d[r] * loss
    total.backward()
    loss, w = rows.distill_topk(z.detach(), idx, t, tau)
    np.testing.assert_allclose(loss, ref, rtol=1e-12)
    np.testing.assert_allclose(rows.distill_topk_backward(z.detach(), idx, w, d, tau), z.grad,
                               rtol=1e-10, atol=1e-12)


def test_distill_of_a_teacher_that_agrees_is_zero():
    z = np.log(np.array([[0.5, 0.25, 0.125, 0.125]]))
    loss, w = rows.distill_topk(z, np.array([[0, 1, 2, 3]]), z, 1.0)
    np.testing.assert_allclose(loss, 0, atol=1e-15)
    np.testing.assert_allclose(rows.distill_topk_backward(z, np.array([[0, 1, 2, 3]]), w, [1.0]), 0,
                               atol=1e-15)
