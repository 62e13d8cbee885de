"""Pins of the routing and optimizer oracles (CPU): brute force, autograd, differences, grids."""
import itertools

import numpy as np
import pytest
import torch

from oracle import optim_oracle as OO
from oracle import route_oracle as RO


@pytest.mark.parametrize("router,score", [(0, 0), (0, 1), (1, 0), (1, 1)])
def test_selection_by_exhaustion(router, score):
    """Against the definition read as a maximum: of all sets of groups and of all experts in them."""
    rng = np.random.default_rng(3 + router * 2 + score)
    E, G, kg, k = 12, 4, 2, 3
    x, bias = rng.normal(size=(20, E)), (None if router == 0 else rng.normal(size=E) * 0.1)
    idx, _ = RO.select(x, bias, router, k, G, kg, score)
    s = RO.scores(x, router)
    r = s if bias is None else s + bias
    for t in range(20):
        val = [sorted(r[t, g * 3:g * 3 + 3])[::-1] for g in range(G)]
        val = [v[0] if score == RO.GROUP_MAX else v[0] + v[1] for v in val]
        groups = max(itertools.combinations(range(G), kg), key=lambda c: sum(val[g] for g in c))
        pool = [e for e in range(E) if e // 3 in groups]
        best = max(itertools.combinations(pool, k), key=lambda c: sum(r[t, e] for e in c))
        assert set(idx[t]) == set(best)
        assert all(r[t, a] >= r[t, b] for a, b in zip(idx[t], idx[t][1:]))


def test_selection_ties_masks_and_nothing_left():
    x = np.zeros((1, 8))
    assert RO.select(x, None, 1, 3, 4, 2, 1)[0].tolist() == [[0, 1, 2]]
    x[0, :3] = -np.inf
    assert RO.select(x, None, 1, 3, 1, 1, 1)[0].tolist() == [[3, 4, 5]]
    x[:] = -np.inf
    idx, _ = RO.select(x, None, 0, 3, 4, 2, 0)
    assert idx.tolist() == [[0, 1, 2]]
    assert RO.gates(RO.scores(x, 0), idx, True, 2.0).tolist() == [[0.0, 0.0, 0.0]]


@pytest.mark.parametrize("router,renorm,use", list(itertools.product((0, 1), (False, True), ("gates", "prob", "both"))))
def test_backward_by_autograd_and_differences(router, renorm, use):
    rng = np.random.default_rng(11)
    T, E, k, scale = 4, 10, 3, 2.5
    x = rng.normal(size=(T, E))
    idx, _ = RO.select(x, None, router, k, 2, 1, 1)
    dg = rng.normal(size=(T, k)) if use != "prob" else None
    dp = rng.normal(size=E) if use != "gates" else None
    got = RO.backward(x, idx, dg, dp, router, renorm, scale)

    def f(z):
        s = RO.scores(z, router)
        v = 0.0 if dg is None else (dg * RO.gates(s, idx, renorm, scale)).sum()
        return v if dp is None else v + (dp * RO.probabilities(s).sum(axis=0)).sum()

    xt = torch.tensor(x, requires_grad=True)
    s = torch.sigmoid(xt) if router else torch.softmax(xt, 1)
    c = s.gather(1, torch.tensor(idx, dtype=torch.int64))
    loss = 0.0
    if dg is not None:
        loss = loss + (torch.tensor(dg) * scale * (c / c.sum(1, keepdim=True) if renorm else c)).sum()
    if dp is not None:
        loss = loss + (torch.tensor(dp) * s / s.sum(1, keepdim=True)).sum()
    loss.backward()
    assert np.allclose(got, xt.grad.numpy(), rtol=1e-10, atol=1e-13)
    h = 1e-6
    for t, e in itertools.product(range(T), range(E)):
        up, down = x.copy(), x.copy()
        up[t, e] += h
        down[t, e] -= h
        assert abs((f(up) - f(down)) / (2 * h) - got[t, e]) < 1e-7


def test_balance_of_a_uniform_router():
    """Equal scores: every probability 1 / E, and the loss is coef whatever the counts."""
    T, E, k = 6, 5, 2
    s = np.full((T, E), 0.3)
    idx = np.array([[0, 1]] * 5 + [[2, 3]])
    counts, prob, loss, dprob, moved = RO.balance(s, idx, 0.7, np.zeros(E), 0.5)
    assert counts.tolist() == [5, 5, 1, 1, 0] and np.allclose(prob, T / E) and np.isclose(loss, 0.7)
    assert moved.tolist() == [-0.5, -0.5, 0.5, 0.5, 0.5]


def test_adamw_is_torch_adamw():
    rng = np.random.default_rng(0)
    p = rng.normal(size=50)
    t = torch.tensor(p, requires_grad=True)
    opt = torch.optim.AdamW([t], lr=1e-2, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
    m = v = np.zeros(50)
    for step in range(1, 6):
        g = rng.normal(size=50)
        t.grad = torch.tensor(g)
        opt.step()
        p, m, v = OO.adamw(p, g, m, v, lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=step)
        assert np.allclose(p, t.detach().numpy(), rtol=1e-12, atol=1e-14)


def test_mx8_values_are_e4m3_and_their_mean_is_the_input():
    rng = np.random.default_rng(1)
    t = rng.normal(size=320) * np.exp2(rng.integers(-20, 3, 320))
    total = np.zeros(320)
    n = 4000
    for i in range(n):
        q, x = OO.to_mx8(t, rng.integers(0, 2 ** 32, 320, dtype=np.uint64), False)
        total += q * np.exp2(np.repeat(x, 32))
        if i == 0:
            f8 = torch.tensor(q).float().to(torch.float8_e4m3fn).double().numpy()
            assert np.array_equal(f8, q)
            top = np.abs(t).reshape(-1, 32).max(axis=1) / np.exp2(x)
            assert ((top <= 448) & (top > 224)).all()
    spacing = OO.grid(t / np.exp2(np.repeat(x, 32))) * np.exp2(np.repeat(x, 32))
    # a rounding's deviation is at most half a spacing: 6 deviations of the mean over n of them
    assert (np.abs(total / n - t) <= 6 * 0.5 * spacing / np.sqrt(n)).all()


def test_mx8_root_never_becomes_zero_and_zero_stays():
    t = np.zeros(64)
    t[:32] = 1e-12
    t[0] = 1.0
    q, _ = OO.to_mx8(t, np.zeros(64, np.uint64), True)
    assert (q[:32] > 0).all() and not q[32:].any()


def test_rounding_bits_are_uniform():
    """Each of the 32 bits is set in half of the elements, within 6 deviations; groups and steps differ."""
    n = 1 << 16
    b = OO.rounding_bits(n, 64, 7, 3)
    for i in range(32):
        share = ((b >> np.uint64(i)) & np.uint64(1)).mean()
        assert abs(share - 0.5) < 6 * 0.5 / np.sqrt(n), i
    assert (b[8:] == OO.rounding_bits(n - 8, 72, 7, 3)).all()
    assert (b != OO.rounding_bits(n, 64, 7, 4)).mean() > 0.99
    assert (b != OO.rounding_bits(n, 64 + 2 ** 35, 7, 3)).mean() > 0.99
