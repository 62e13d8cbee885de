"""GPU parity of the gradient norm and the AdamW step against the float64 CPU oracle.

Tolerances: f32 arithmetic rounds each term a few times, so m and v are held to 2^-21 of the sum of
their terms' magnitudes (4 roundings of 2^-24 and two constants rounded to f32), and a parameter to
2^-23 of itself plus 2^-19 of the step's magnitude (m, v, a square root and a division of up to 2^-22
each, and three more roundings).  A rounding at random compares y / spacing + u with a whole number;
y / spacing is below 16 with a relative error of 2^-21, so a value falls on the other side with a
probability of 2^-16 at most: 2^-14 of the elements (and 3 more) may differ by one spacing.
"""
import numpy as np
import pytest
import torch

import mixture_experts_layer_table_gb300 as mok
from oracle import optim_oracle as O

pytestmark = pytest.mark.gpu

HYPER = dict(betas=(0.9, 0.95), eps=1e-8)
SIZES = (1, 7, 8, 31, 32, 33, 255, 2047, 2048, 2049, 100003)


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_ok):
    from mixture_experts_layer_table_gb300 import build
    build.build()
    mok.load()


def f64(t):
    return t.detach().double().cpu().numpy().ravel()


def _tensors(sizes, dtype, std, seed, offset=0):
    """Seeded tensors; offset > 0: views that start `offset` elements into their memory."""
    out = []
    for i, n in enumerate(sizes):
        g = torch.Generator().manual_seed(seed * 1000 + i)
        t = torch.randn(n + offset, generator=g) * std * (1 + 9 * torch.rand(n + offset, generator=g) ** 4)
        out.append(t.to(dtype).cuda()[offset:])
    return out


def _f32_states(sizes, seed, offset=0):
    return {"m": _tensors(sizes, torch.float32, 1e-3, seed, offset),
            "v": [t.square() for t in _tensors(sizes, torch.float32, 2e-3, seed + 1)] if not offset else
                 [t.square_() for t in _tensors(sizes, torch.float32, 2e-3, seed + 1, offset)]}


def _mx8_states(sizes, seed):
    rng = np.random.default_rng(seed)
    cast = lambda a: torch.tensor(a, dtype=torch.float32).to(torch.float8_e4m3fn).cuda()  # noqa: E731
    scales = lambda lo: [torch.tensor(rng.integers(lo, lo + 3, -(-n // 32)), dtype=torch.uint8).cuda()  # noqa: E731
                         for n in sizes]
    return {"m": [cast(np.clip(rng.normal(0, 120, n), -448, 448)) for n in sizes],
            "v": [cast(np.clip(np.abs(rng.normal(0, 120, n)), 0, 448)) for n in sizes],
            "m_scale": scales(107), "v_scale": scales(108)}


def _check_f32(got, want, terms, what, rel=2.0 ** -21):
    bad = np.abs(got - want) > rel * terms + 1e-38
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, first at {np.argmax(bad)}"


def _check_step(opt, before, i, scale, lr, wd, step, counter, seed):
    """Tensor i of an optimizer after a step from `before` (float64 copies)."""
    b1, b2 = HYPER["betas"]
    p0, g, m0, v0 = before
    p, m, v = O.adamw(p0, g, m0, v0, lr=lr, beta1=b1, beta2=b2, eps=HYPER["eps"], weight_decay=wd, step=step, scale=scale)
    gs = g * scale
    m_terms, v_terms = b1 * np.abs(m0) + (1 - b1) * np.abs(gs), b2 * v0 + (1 - b2) * gs * gs
    denom = np.sqrt(v / (1 - b2 ** step)) + HYPER["eps"]
    p_tol = 2.0 ** -23 * np.abs(p0) + lr * 2.0 ** -19 * (m_terms / (1 - b1 ** step) / denom + wd * np.abs(p0)) + 1e-38
    bits = O.rounding_bits(p.size, counter, seed, step)
    few = 2.0 ** -14 * p.size + 3
    param, master = opt.params[i], opt.masters[i]
    if param.dtype == torch.float32:
        assert (np.abs(f64(param) - p) <= p_tol).all()
    elif master is not None:
        assert (np.abs(f64(master) - p) <= p_tol).all()
        assert torch.equal(param, master.bfloat16())
    else:
        want = O.to_bf16_random(p, bits).astype(np.float64)
        got = f64(param)
        assert (got != want).sum() <= few
        assert (np.abs(got - p) <= p_tol + np.abs(p) * 2.0 ** -7).all()   # a neighbour on bf16's grid
    if not opt.mx8:
        _check_f32(f64(opt.states["m"][i]), m, m_terms, "m")
        _check_f32(f64(opt.states["v"][i]), v, v_terms, "v")
        return
    for name, value, root in (("m", m, False), ("v", np.sqrt(v), True)):
        q, x = O.to_mx8(value, bits, root)
        got_q, got_x = f64(opt.states[name][i]), opt.states[name + "_scale"][i].cpu().numpy().astype(np.int64) - 127
        same = got_x == x                       # a block maximum next to 448 * 2^x may fall on either side
        assert (~same).sum() <= 1 + 2.0 ** -14 * same.size
        here = np.repeat(same, 32)[:value.size]
        off = got_q[here] != q[here]
        assert off.sum() <= few, f"{name}: {off.sum()} of {value.size}"
        s = np.exp2(np.repeat(got_x, 32)[:value.size].astype(np.float64))
        assert (np.abs(got_q * s - value) <= s * O.grid(value / s) * 1.001).all()
        if root:
            assert (got_q[value > 0] > 0).all()


def _run_and_check(sizes, pk, grad_dtype, state, seed, scale=0.37, step0=41, offset=0, lr=1e-2, wd=0.1):
    pdt = torch.float32 if pk == "f32" else torch.bfloat16
    params, grads = _tensors(sizes, pdt, 0.05, seed, offset), _tensors(sizes, grad_dtype, 2e-3, seed + 7, offset)
    masters = [(p.float() + 1e-5) for p in params] if pk == "master" else None
    states = _f32_states(sizes, seed + 3, offset) if state == "f32" else _mx8_states(sizes, seed)
    opt = mok.AdamW(params, grads, lr=lr, weight_decay=wd, state=state, masters=masters, seed=99, step=step0,
                    states=states, **HYPER)
    values = [opt.state_values(i) for i in range(len(sizes))]
    before = [(f64(masters[i] if masters else params[i]), f64(grads[i]), f64(values[i]["m"]), f64(values[i]["v"]))
              for i in range(len(sizes))]
    s = None if scale is None else torch.tensor([scale], device="cuda")
    opt.step(s)
    torch.cuda.synchronize()
    at = 0
    for i, n in enumerate(sizes):
        _check_step(opt, before[i], i, 1.0 if scale is None else float(np.float32(scale)), float(np.float32(lr)),
                    float(np.float32(wd)), step0 + 1, at, 99)
        at += -(-n // 32) * 32
    return opt


@pytest.mark.parametrize("pk", ["f32", "master", "bf16"])
@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16], ids=["g32", "g16"])
@pytest.mark.parametrize("state", ["f32", "mx8"])
def test_adamw_step(pk, grad, state):
    _run_and_check(SIZES, pk, grad, state, seed=1)


@pytest.mark.parametrize("pk,grad,state", [("f32", torch.float32, "f32"), ("bf16", torch.bfloat16, "f32"),
                                           ("master", torch.float32, "f32"), ("bf16", torch.float32, "mx8")])
def test_adamw_on_tensors_that_start_off_16_bytes(pk, grad, state):
    _run_and_check((1, 37, 4099), pk, grad, state, seed=2, offset=1)


def test_adamw_first_step_from_zero_states_without_a_scale():
    for state in ("f32", "mx8"):
        params, grads = _tensors((1000,), torch.float32, 0.05, 5), _tensors((1000,), torch.float32, 1e-3, 6)
        before = (f64(params[0]), f64(grads[0]), np.zeros(1000), np.zeros(1000))
        opt = mok.AdamW(params, grads, lr=1e-2, weight_decay=0.0, state=state, seed=3, **HYPER)
        opt.step()
        _check_step(opt, before, 0, 1.0, float(np.float32(1e-2)), 0.0, 1, 0, 3)


def test_adamw_on_more_tensors_than_one_launch_takes():
    """300 tensors of both gradient types in one call, each with its own rate and decay."""
    sizes = [1 + 37 * i % 500 for i in range(300)]
    params = _tensors(sizes, torch.float32, 0.05, 11)
    grads = [g.bfloat16() if i % 3 else g for i, g in enumerate(_tensors(sizes, torch.float32, 1e-3, 12))]
    lrs, wds = [1e-3 * (1 + i % 5) for i in range(300)], [0.1 * (i % 2) for i in range(300)]
    before = [(f64(p), f64(g), np.zeros(p.numel()), np.zeros(p.numel())) for p, g in zip(params, grads)]
    opt = mok.AdamW(params, grads, lr=lrs, weight_decay=wds, **HYPER)
    opt.step()
    torch.cuda.synchronize()
    at = 0
    for i, n in enumerate(sizes):
        _check_step(opt, before[i], i, 1.0, float(np.float32(lrs[i])), float(np.float32(wds[i])), 1, at, 0)
        at += -(-n // 32) * 32


def test_adamw_empty_and_zero():
    """Empty tensors are skipped; a gradient that is always zero leaves zero states and only decays."""
    for state in ("f32", "mx8"):
        params = [torch.zeros(0, device="cuda"), torch.full((100,), 0.5, device="cuda")]
        opt = mok.AdamW(params, [torch.zeros_like(p) for p in params], lr=0.1, weight_decay=0.5, state=state, **HYPER)
        for _ in range(2):
            opt.step()
        got = opt.state_values(1)
        assert torch.equal(got["m"], torch.zeros(100, device="cuda")) and torch.equal(got["v"], torch.zeros(100, device="cuda"))
        assert torch.allclose(params[1], torch.full((100,), 0.5 * 0.95 ** 2, device="cuda"), rtol=1e-6)
    mok.AdamW([], []).step()


@pytest.mark.parametrize("state", ["f32", "mx8"])
def test_adamw_leaves_everything_where_the_scale_is_nan(state):
    params, grads = _tensors((4097,), torch.bfloat16, 0.05, 21), _tensors((4097,), torch.float32, 1e-3, 22)
    states = _f32_states((4097,), 23) if state == "f32" else _mx8_states((4097,), 23)
    kept = [params[0].clone(), *[s[0].clone() for s in states.values()]]
    opt = mok.AdamW(params, grads, state=state, states=states, step=3, **HYPER)
    opt.step(torch.full((1,), float("nan"), device="cuda"))
    same = lambda a, b: torch.equal(a.view(torch.uint8), b.view(torch.uint8))  # noqa: E731
    assert all(same(a, b) for a, b in zip(kept, [params[0], *[s[0] for s in opt.states.values()]]))


def test_adamw_infinite_gradient_shows():
    """Without a clip factor an infinite gradient makes its own elements non-finite, and no others."""
    params, grads = _tensors((64,), torch.float32, 0.05, 31), _tensors((64,), torch.float32, 1e-3, 32)
    grads[0][5] = float("inf")
    opt = mok.AdamW(params, grads, **HYPER)
    opt.step()
    bad = ~torch.isfinite(params[0])
    assert bad.nonzero().flatten().tolist() == [5]


KINDS = [(pk, grad, state) for pk in ("f32", "master", "bf16") for grad in (torch.float32, torch.bfloat16)
         for state in ("f32", "mx8")]


def _with_and_without(pk, grad_dtype, state, at, n=2085, **kw):
    """Two optimizers on the same tensors, but for the gradients at `at`, zero in the second's: what the others' rounding
    and scales are held against.  2,085 elements: whole words, and a tail of single ones."""
    made = []
    for clean in (False, True):
        params = _tensors((n,), torch.float32 if pk == "f32" else torch.bfloat16, 0.05, 71)
        grads = _tensors((n,), grad_dtype, 1e-3, 72)
        grads[0][list(at)] = 0.0
        for i, x in at.items():
            if not clean:
                grads[0][i] = x
        made.append(mok.AdamW(params, grads, state=state, masters=True if pk == "master" else None, seed=17, **HYPER, **kw))
    return made


@pytest.mark.parametrize("pk,grad,state", KINDS)
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_adamw_gradients_that_are_not_finite_show_in_every_kind_of_parameter(pk, grad, state, bad):
    """Their own parameters become NaN, whatever random bits round them, and stay so; no others do."""
    at = {i: bad for i in (5, 700, 701, 2080, 2084)}
    opt, _ = _with_and_without(pk, grad, state, at)
    for _ in range(3):
        opt.step()
        assert torch.isnan(opt.params[0]).nonzero().flatten().tolist() == sorted(at)
        assert torch.isfinite(opt.params[0]).sum().item() == 2085 - len(at)
        opt.grads[0][list(at)] = 0.0


def _same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("pk,grad,state", [k for k in KINDS if k[2] == "mx8"])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_adamw_gradients_that_are_not_finite_leave_the_rest_of_a_block_of_8_bit_states(pk, grad, state, bad):
    """The other 31 elements of the block are stepped as if those gradients had been zero, state for state and bit for
    bit, in this step and the ones after it; the elements' own states become NaN."""
    at = {i: bad for i in (5, 700, 701, 2080, 2084)}
    opt, clean = _with_and_without(pk, grad, state, at)
    others = torch.ones(2085, dtype=torch.bool, device="cuda")
    others[list(at)] = False
    for _ in range(3):
        opt.step()
        clean.step()
        assert _same(opt.params[0][others], clean.params[0][others])
        for n in ("m", "v"):
            assert _same(opt.states[n][0].view(torch.uint8)[others], clean.states[n][0].view(torch.uint8)[others])
            assert torch.isnan(opt.states[n][0].float()[~others]).all()
            assert _same(opt.states[n + "_scale"][0], clean.states[n + "_scale"][0])
        opt.grads[0][list(at)] = 0.0


@pytest.mark.parametrize("pk", ["f32", "bf16"])
def test_adamw_gradients_whose_square_overflows_show_in_8_bit_states(pk):
    """sqrt(v) is not finite then: it is kept as a NaN (E4M3 has no infinity), alone of its block, and shows in the
    parameter at the next step.  m is finite, and its block's scale grows with it."""
    at = {700: 1e25, 2084: 1e25}
    opt, clean = _with_and_without(pk, torch.float32, "mx8", at)
    for o in (opt, clean):
        o.step()
    others = torch.ones(2085, dtype=torch.bool, device="cuda")
    others[list(at)] = False
    v = opt.states["v"][0]
    assert torch.isnan(v.float()).nonzero().flatten().tolist() == sorted(at)
    assert _same(v.view(torch.uint8)[others], clean.states["v"][0].view(torch.uint8)[others])
    assert _same(opt.states["v_scale"][0], clean.states["v_scale"][0])
    assert _same(opt.params[0][others], clean.params[0][others])
    assert torch.isfinite(opt.states["m"][0].float()).all()
    opt.grads[0].zero_()
    opt.step()
    assert torch.isnan(opt.params[0]).nonzero().flatten().tolist() == sorted(at)


def test_adamw_a_scale_byte_of_255_is_not_finite():
    """The block under it becomes NaN, states and, a step later at most, parameters; the other blocks do not."""
    opt, clean = _with_and_without("f32", torch.float32, "mx8", {})
    for o in (opt, clean):
        o.step()
    for name in ("m_scale", "v_scale"):
        opt.states[name][0][3] = 255
        opt.states[name][0][65] = 255          # the last block, of 5 elements
    for o in (opt, clean):
        o.step()
        o.step()
    block = torch.arange(2085, device="cuda") // 32
    hit = (block == 3) | (block == 65)
    assert torch.isnan(opt.params[0][hit]).all() and _same(opt.params[0][~hit], clean.params[0][~hit])
    for n in ("m", "v"):
        assert torch.isnan(opt.states[n][0].float()[hit]).all()
        assert _same(opt.states[n][0].view(torch.uint8)[~hit], clean.states[n][0].view(torch.uint8)[~hit])


@pytest.mark.parametrize("state", ["f32", "mx8"])
@pytest.mark.parametrize("pk", ["f32", "master"])
@pytest.mark.parametrize("lr", [1e-30, 1e-37, 2e-38, 1e-39, 1e-44, 0.0])
def test_adamw_rates_down_to_zero(state, pk, lr):
    """The end of a schedule: rates near and below the least normal f32 number move a parameter by no more than its last
    place, and one of zero by as little as themselves (a step's quotient is at most 1 / sqrt(1 - beta2) < 5, doubled for
    the roundings); nothing is divided by a rate that is too small for it."""
    n = 100
    params = [torch.zeros(n, device="cuda"), torch.full((n,), 0.75, device="cuda")]
    if pk == "master":
        params = [p.bfloat16() for p in params]
    grads = [torch.zeros(n, device="cuda") for _ in params]
    for g in grads:
        g[50:] = torch.linspace(-1e-3, 1e-3, 50, device="cuda")
    opt = mok.AdamW(params, grads, lr=lr, weight_decay=0.1, state=state, masters=True if pk == "master" else None, **HYPER)
    for _ in range(3):
        opt.step()
    held = params if pk == "f32" else opt.masters
    assert held[0].abs().max().item() <= 3 * 10 * lr + 1e-37
    assert torch.equal(held[1], torch.full((n,), 0.75, device="cuda"))
    assert all(torch.isfinite(opt.state_values(i)[s]).all() for i in (0, 1) for s in ("m", "v"))


def test_adamw_states_in_8_bits_follow_the_32_bit_ones():
    """With steps far below a grid spacing (beta2 = 0.999) the 8-bit states keep moving with the f32 ones: over
    4096 elements the mean of sqrt(v) and of m stay together.  sqrt(v) wanders by a random rounding of up to
    12% each time it moves, about 20% of itself in the long run, so its mean over 4096 elements is known to
    0.2 / 64 = 0.3%; 3% leaves room for the spread's own curvature (the mean of sqrt(v) against f32's)."""
    n = 4096
    g = torch.Generator().manual_seed(0)
    opts = []
    for state in ("f32", "mx8"):
        opts.append(mok.AdamW([torch.zeros(n, device="cuda")], [torch.zeros(n, device="cuda")], lr=1e-4,
                              betas=(0.9, 0.999), state=state, seed=5))
    for t in range(600):
        grad = torch.randn(n, generator=g) * (1.0 if t < 300 else 0.25) + 0.1
        for o in opts:
            o.grads[0].copy_(grad)
            o.step()
    a, b = (o.state_values(0) for o in opts)
    r = (b["v"].sqrt().mean() / a["v"].sqrt().mean()).item()
    assert abs(r - 1) < 0.03, r
    assert abs((b["m"].mean() - a["m"].mean()).item()) < 0.02
    spread = ((b["v"].sqrt() - a["v"].sqrt()) / a["v"].sqrt()).std().item()
    assert spread < 0.4, spread


def test_adamw_reproducible_and_on_another_stream():
    results = []
    for run in range(3):
        params, grads = _tensors((70001,), torch.bfloat16, 0.05, 41), _tensors((70001,), torch.bfloat16, 1e-3, 42)
        opt = mok.AdamW(params, grads, state="mx8", seed=7, **HYPER)
        norm = mok.GradNorm(grads, 0.5)
        stream = torch.cuda.Stream()
        torch.cuda.synchronize()
        for _ in range(3):
            if run == 2:
                opt.step(norm.compute(stream)[1:], stream)
            else:
                opt.step(norm.compute()[1:])
        torch.cuda.synchronize()
        results.append([params[0].view(torch.int16).clone(), *[s[0].view(torch.uint8).clone() for s in opt.states.values()]])
    for other in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(results[0], other))


def test_adamw_and_norm_past_32_bit_offsets():
    """A tensor of more than 2^31 elements: its last elements are updated as a tensor of their own would be."""
    n, tail = 2 ** 31 + 4096 + 5, 4096 + 5
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    p[-tail:], g[-tail:] = _tensors((tail,), torch.bfloat16, 0.05, 51)[0], _tensors((tail,), torch.bfloat16, 1e-3, 52)[0]
    small_p, small_g = p[-tail:].clone(), g[-tail:].clone()
    norm, small_norm = mok.GradNorm([g], 1e-3), mok.GradNorm([small_g], 1e-3)
    assert torch.allclose(norm.compute(), small_norm.compute(), rtol=1e-6)
    big = mok.AdamW([p], [g], state="mx8", seed=1, counters=[0], **HYPER)
    small = mok.AdamW([small_p], [small_g], state="mx8", seed=1, counters=[2 ** 31], **HYPER)
    big.step(small_norm.result[1:])
    small.step(small_norm.result[1:])
    assert torch.equal(p[-tail:], small_p) and not p[:4096].any()
    assert torch.equal(big.states["m"][0][-tail:].view(torch.uint8), small.states["m"][0].view(torch.uint8))
    assert torch.equal(big.states["v_scale"][0][-129:], small.states["v_scale"][0])


# ------------------------------------------------------------------ gradient norm

@pytest.mark.parametrize("sizes,dtype,offset", [((1,), torch.float32, 0), ((7, 0, 33), torch.bfloat16, 0),
                                                ((2 ** 20 + 3, 5, 16385), torch.float32, 0),
                                                ((4099, 37), torch.float32, 1), ((4099, 37), torch.bfloat16, 1),
                                                (tuple(range(1, 700)), torch.float32, 0)])
@pytest.mark.parametrize("max_norm", [1e-2, 1e6])
def test_grad_norm(sizes, dtype, offset, max_norm):
    """The sums run in f32 over at most a few thousand squares of a thread and in f64 from there on: 2^-20."""
    grads = _tensors(sizes, dtype, 1e-3, 61, offset)
    want = O.grad_norm([f64(g) for g in grads], max_norm)
    norm = mok.GradNorm(grads, max_norm)
    first = norm.compute().clone()
    got = f64(first)
    assert abs(got[0] - want[0]) <= 2.0 ** -20 * want[0]
    assert abs(got[1] - want[1]) <= 2.0 ** -20 * want[1]
    assert torch.equal(norm.compute(), first)      # the workspace is left ready, the order is fixed


def test_grad_norm_of_nothing_and_of_non_finite():
    assert f64(mok.GradNorm([], 1.0).compute()).tolist() == [0.0, 1.0]
    g = torch.zeros(1000, device="cuda")
    assert f64(mok.GradNorm([g], 1.0).compute()).tolist() == [0.0, 1.0]
    assert f64(mok.GradNorm([torch.ones(4, device="cuda")], float("inf")).compute()).tolist() == [2.0, 1.0]
    for bad in (float("inf"), float("nan")):
        g[777] = bad
        got = f64(mok.GradNorm([g], 1.0).compute())
        assert not np.isfinite(got[0]) and np.isnan(got[1])


@pytest.mark.parametrize("size,n", [(1e18, 100003), (5e18, 40), (1e19, 16384 * 3), (3e19, 100003), (1e25, 7), (1e30, 50000),
                                    (3e38, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_grad_norm_of_large_gradients(size, n, dtype):
    """Finite gradients whose squares, or their sum, pass f32's range: the norm is theirs as long as it is below 3.4e38
    itself.  As above within 2^-20: sums in f32 over at most a few thousand squares of a thread, one root rounded to f32."""
    grads = _tensors((1000,), torch.float32, 1e-3, 81) + [torch.full((n,), size, dtype=dtype, device="cuda")]
    grads[1][::3].neg_()
    norm = mok.GradNorm(grads, 1.0)
    want = O.grad_norm([f64(g) for g in grads], 1.0)
    first = norm.compute().clone()
    got = f64(first)
    assert abs(got[0] - want[0]) <= 2.0 ** -20 * want[0]
    assert abs(got[1] - want[1]) <= 2.0 ** -20 * want[1] + 2.0 ** -149
    assert torch.equal(norm.compute(), first)
    grads[1][n // 2] = float("nan")
    assert torch.isnan(norm.compute()).all()
    grads[1][n // 2] = -float("inf")
    got = f64(norm.compute())
    assert np.isposinf(got[0]) and np.isnan(got[1])


def test_grad_norm_past_f32_is_infinite():
    got = f64(mok.GradNorm([torch.full((2,), 3e38, device="cuda")], 1.0).compute())
    assert np.isposinf(got[0]) and np.isnan(got[1])


def test_what_the_constructors_fill_is_ready_on_another_stream():
    """The current stream is busy when the objects are made, in memory that was not zero; their first calls go to another
    stream at once."""
    params, grads = _tensors((5000,), torch.bfloat16, 0.05, 91), _tensors((5000,), torch.float32, 1e-3, 92)
    want_norm = mok.GradNorm(grads, 0.5).compute().clone()
    want = {}
    for state in ("f32", "mx8"):
        p = [params[0].clone()]
        opt = mok.AdamW(p, grads, state=state, masters=True, **HYPER)
        opt.step()
        want[state] = [p[0], opt.masters[0], *[s[0].view(torch.uint8) for s in opt.states.values()]]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for n in (16640, 5000 * 4, 5000, 157):
        torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")
    copies = [params[0].clone() for _ in want]
    torch.cuda._sleep(40_000_000)
    norm = mok.GradNorm(grads, 0.5)
    assert torch.cuda.current_stream().query()
    norm.compute(side)
    side.synchronize()
    assert torch.equal(norm.result, want_norm)
    for (state, w), copy in zip(want.items(), copies):
        torch.cuda._sleep(40_000_000)
        opt = mok.AdamW([copy], grads, state=state, masters=True, **HYPER)
        assert torch.cuda.current_stream().query()
        opt.step(stream=side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(w, [copy, opt.masters[0], *[s[0].view(torch.uint8) for s in opt.states.values()]]))
