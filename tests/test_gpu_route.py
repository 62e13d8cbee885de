"""GPU parity of the group-limited routing and its backward against the float64 CPU oracle.

The selection is compared exactly, on tokens whose deciding values lie at least 1e-5 apart in the
oracle (f32 scores are off by less than 1e-6; tokens that are closer are left out before the run), on
exact ties, and on masks.  Scores go through one exp, one sum of up to 1024 terms and one division in
f32: gates, scores and probability sums are held to 2^-18 of themselves.  A logit gradient is a sum of
terms that may cancel: 2^-18 of the terms' sizes, and half a bf16 spacing for bf16 gradients.
"""
import ctypes

import numpy as np
import pytest
import torch

import mixture_experts_layer_table_gb300 as mok
from mixture_experts_layer_table_gb300 import workloads as W
from oracle import route_oracle as O

pytestmark = pytest.mark.gpu

SOFTMAX, SIGMOID = 0, 1
MAX, TOP2 = 0, 1
REL = 2.0 ** -18


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_ok):
    from mixture_experts_layer_table_gb300 import build
    build.build()
    mok.load()


def f64(t):
    return t.detach().double().cpu().numpy()


# (T, E, k, n_group, topk_group, group score): one expert, odd counts, groups of one, groups that are not
# whole lanes, every experts-per-lane width, the largest
SHAPES = [(1, 1, 1, 1, 1, MAX), (5, 7, 3, 1, 1, TOP2), (33, 20, 4, 20, 6, TOP2), (40, 60, 5, 6, 2, TOP2),
          (17, 64, 6, 8, 3, MAX), (29, 96, 8, 3, 1, TOP2), (65, 128, 8, 4, 2, TOP2), (31, 160, 6, 8, 3, MAX),
          (23, 192, 8, 8, 4, TOP2), (70, 256, 8, 8, 4, TOP2), (19, 300, 12, 12, 5, TOP2), (9, 384, 8, 16, 4, MAX),
          (11, 502, 7, 2, 1, TOP2), (13, 1024, 16, 32, 8, TOP2), (8, 1000, 16, 8, 8, MAX), (3, 31, 16, 31, 16, MAX)]


def _logits(T, E, seed, dtype, router, bias, k, G, kg, score):
    """T tokens that the oracle's margins keep clear of rounding, as (CUDA tensor, float64)."""
    rng = np.random.default_rng(seed)
    x = torch.tensor(rng.normal(size=(6 * T + 40, E)) * 1.5).to(dtype)
    keep = O.select(x.double().numpy(), bias, router, k, G, kg, score)[1] > 1e-5
    x = x[torch.tensor(keep)][:T]
    assert x.shape[0] == T
    return x.contiguous().cuda(), x.double().numpy()


def _bias(E, seed, with_bias):
    return np.random.default_rng(seed).normal(size=E).astype(np.float32) * np.float32(0.1) if with_bias else None


def _cuda(a):
    return None if a is None else torch.tensor(a).cuda()


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "T%d_E%d_k%d_G%d_kg%d_s%d" % s)
@pytest.mark.parametrize("router,with_bias", [(SIGMOID, True), (SIGMOID, False), (SOFTMAX, False), (SOFTMAX, True)])
def test_route(shape, router, with_bias):
    T, E, k, G, kg, score = shape
    bias = _bias(E, 5, with_bias)
    renorm, scale = bool((T + E) % 2) or router == SIGMOID, 2.5
    x, x64 = _logits(T, E, 7, torch.float32, router, bias, k, G, kg, score)
    desc = mok.make_route_desc(T, E, k, router, renorm, route_scale=scale, n_group=G, topk_group=kg, group_score=score,
                               balance_coef=0.3, bias_rate=0.01)
    out = mok.Router(desc, balance=True, scores=True).forward(x, _cuda(bias))
    idx, _ = O.select(x64, bias, router, k, G, kg, score)
    s = O.scores(x64, router)
    assert np.array_equal(out["topk_idx"].cpu().numpy(), idx)
    assert np.allclose(f64(out["gates"]), O.gates(s, idx, renorm, scale), rtol=REL, atol=0)
    assert np.allclose(f64(out["scores"]), s, rtol=REL, atol=0)
    counts, prob_sum, loss, dprob, moved = O.balance(s, idx, 0.3, bias, 0.01)
    assert np.array_equal(out["counts"].cpu().numpy(), counts)
    assert np.allclose(f64(out["prob_sum"]), prob_sum, rtol=REL, atol=0)
    assert np.allclose(f64(out["dprob"]), dprob, rtol=REL, atol=0)
    assert np.allclose(f64(out["loss"]), [loss], rtol=REL, atol=0)
    if bias is not None:
        assert np.allclose(f64(out["bias_next"]), moved, rtol=0, atol=2.0 ** -23 * (np.abs(moved).max() + 0.01))
    # the selection alone gives the same
    plain = mok.Router(desc).forward(x, _cuda(bias))
    assert torch.equal(plain["topk_idx"], out["topk_idx"]) and torch.equal(plain["gates"], out["gates"])


@pytest.mark.parametrize("E,k,G,kg,score", [(256, 8, 8, 4, MAX), (60, 7, 6, 3, MAX), (100, 9, 1, 1, MAX), (16, 5, 16, 7, TOP2)])
@pytest.mark.parametrize("router", [SIGMOID, SOFTMAX])
def test_exact_ties_go_to_the_lower_index(E, k, G, kg, score, router):
    """bf16 logits on a grid of 9 values: most tokens have ties at the cut; and rows of one value."""
    T = 200
    rng = np.random.default_rng(2)
    x = torch.tensor(rng.integers(-4, 5, (T, E)) * 0.25).bfloat16()
    x[:3] = torch.tensor([[0.0], [-1.0], [2.0]]).bfloat16()
    out = mok.Router(mok.make_route_desc(T, E, k, router, True, n_group=G, topk_group=kg, group_score=score),
                     dtype=torch.bfloat16).forward(x.cuda())
    assert np.array_equal(out["topk_idx"].cpu().numpy(), O.select(x.double().numpy(), None, router, k, G, kg, score)[0])


def test_sum_of_two_ties_on_equal_rows():
    out = mok.Router(mok.make_route_desc(4, 64, 6, SIGMOID, True, n_group=8, topk_group=2)).forward(torch.zeros(4, 64).cuda())
    assert out["topk_idx"].cpu().tolist() == [[0, 1, 2, 3, 4, 5]] * 4


def _many(E):
    """Tokens that the kernel for many takes, at E experts."""
    return -(-2 ** 27 // E ** 2)


# shapes that many tokens are routed with two to a warp (4 to 16 experts to a lane, groups of one to 16 lanes, groups
# in segments, all groups in play)
MANY = [(64, 6, 8, 3, MAX), (64, 6, 1, 1, MAX), (60, 5, 1, 1, TOP2), (96, 8, 3, 1, TOP2), (128, 8, 4, 2, TOP2),
        (128, 16, 4, 2, MAX), (160, 6, 8, 3, MAX), (160, 3, 8, 8, TOP2), (256, 8, 8, 4, TOP2), (256, 1, 16, 2, MAX),
        (256, 12, 4, 3, TOP2), (240, 7, 15, 5, TOP2), (252, 9, 9, 4, TOP2), (512, 8, 8, 4, TOP2), (16, 4, 4, 2, TOP2)]


# groups that do not fill their lanes, sizes that are no whole words, tokens on 32 lanes
MANY += [(222, 8, 6, 3, TOP2), (57, 5, 3, 2, TOP2), (33, 3, 3, 1, MAX), (35, 4, 5, 2, MAX), (17, 2, 1, 1, MAX),
         (225, 12, 1, 1, MAX), (144, 6, 1, 1, MAX), (192, 8, 8, 3, TOP2), (320, 16, 5, 3, MAX), (272, 7, 16, 6, TOP2),
         (384, 8, 1, 1, MAX), (384, 8, 8, 4, TOP2), (500, 9, 2, 1, MAX), (511, 8, 1, 1, MAX), (512, 8, 8, 4, TOP2)]


@pytest.mark.parametrize("shape", MANY, ids=lambda s: "E%d_k%d_G%d_kg%d_s%d" % s)
@pytest.mark.parametrize("router,with_bias", [(SIGMOID, True), (SIGMOID, False), (SOFTMAX, False), (SOFTMAX, True)])
def test_route_many_tokens(shape, router, with_bias):
    """40 tokens, over and over to 2,500, then 5,001 and then enough for the kernel for many: every copy is routed as
    the oracle's."""
    E, k, G, kg, score = shape
    bias = _bias(E, 15, with_bias)
    x, x64 = _logits(40, E, 17, torch.bfloat16 if k % 2 else torch.float32, router, bias, k, G, kg, score)
    idx, _ = O.select(x64, bias, router, k, G, kg, score)
    s = O.scores(x64, router)
    gates = O.gates(s, idx, True, 2.5)
    for T in (2500, 5001, _many(E) + 3):
        of = np.arange(T) % 40
        desc = mok.make_route_desc(T, E, k, router, True, route_scale=2.5, n_group=G, topk_group=kg, group_score=score,
                                   balance_coef=0.3, bias_rate=0.01)
        rows = x[torch.tensor(of).cuda()]
        plain = mok.Router(desc, dtype=x.dtype).forward(rows, _cuda(bias))
        full = mok.Router(desc, dtype=x.dtype, balance=True, scores=True).forward(rows, _cuda(bias))
        counts, prob_sum, loss, dprob, _ = O.balance(s[of], idx[of], 0.3, bias, 0.01)
        for out in (plain, full):
            assert np.array_equal(out["topk_idx"].cpu().numpy(), idx[of])
            assert np.allclose(f64(out["gates"]), gates[of], rtol=REL, atol=0)
        assert np.allclose(f64(full["scores"]), s[of], rtol=REL, atol=0)
        assert np.array_equal(full["counts"].cpu().numpy(), counts)
        assert np.allclose(f64(full["prob_sum"]), prob_sum, rtol=REL, atol=0)
        assert np.allclose(f64(full["loss"]), [loss], rtol=REL, atol=0)
        # rows of a wider tensor, not aligned
        wide = torch.zeros((T, E + 3), dtype=x.dtype, device="cuda")
        wide[:, 1:E + 1] = rows
        again = mok.Router(desc, dtype=x.dtype, balance=True).forward(wide[:, 1:E + 1], _cuda(bias))
        assert torch.equal(again["topk_idx"], plain["topk_idx"]) and torch.equal(again["counts"], full["counts"])


@pytest.mark.parametrize("E,k,G,kg,score", [(256, 8, 8, 4, MAX), (64, 6, 1, 1, MAX), (160, 6, 8, 3, MAX), (222, 7, 6, 3, MAX),
                                            (35, 4, 5, 2, MAX), (384, 8, 1, 1, MAX), (500, 9, 2, 1, MAX)])
@pytest.mark.parametrize("router,with_bias", [(SIGMOID, False), (SIGMOID, True), (SOFTMAX, False)])
def test_many_tokens_with_ties_and_masks(E, k, G, kg, score, router, with_bias):
    """Exact ties (with a bias of zeros too), rows of one value, masked experts and groups, rows with too few experts
    left and with none: rank values here are equal or far apart in f32 as in f64."""
    T, times = 3000, -(-_many(E) // 3000)  # over and over
    rng = np.random.default_rng(5)
    x = rng.integers(-4, 5, (T, E)) * 0.25
    x[:3] = [[0.0], [-1.0], [2.0]]
    x[10:700][rng.random((690, E)) < 0.2] = -np.inf
    x[700:900, :E // 2] = -np.inf
    x[900:950] = np.where(np.isin(np.arange(E), (3, E - 2)), x[900:950], -np.inf)
    x[950:1000] = -np.inf
    bias = np.zeros(E, np.float32) if with_bias else None
    desc = mok.make_route_desc(T * times, E, k, router, True, n_group=G, topk_group=kg, group_score=score)
    out = mok.Router(desc).forward(torch.tensor(x).float().cuda().repeat(times, 1), _cuda(bias))
    out = {n: t[-T:] for n, t in out.items()}
    got = out["topk_idx"].cpu().numpy()
    want, _ = O.select(x, bias, router, k, G, kg, score)
    assert np.array_equal(got, want)
    s = O.scores(x, router)
    assert np.allclose(f64(out["gates"]), O.gates(s, got, True, 1.0), rtol=REL, atol=0)


def test_selection_is_that_of_the_f32_scores_however_near():
    """Rank values a few f32 steps apart, with a bias (the many-token kernel forms approximate scores first): the
    order is that of s + b in f32, s = 1 / (1 + e^-x) by steps rounded to f32."""
    T, E, k = 4096, 256, 8
    g = torch.Generator(device="cuda").manual_seed(0)
    x = (torch.randn(T, E, generator=g, device="cuda") * 1e-6 + torch.randn(T, 1, generator=g, device="cuda"))
    bias = torch.randint(-4, 5, (E,), generator=g, device="cuda").float() * 2.0 ** -23
    out = mok.Router(mok.make_route_desc(T, E, k, SIGMOID, True, n_group=8, topk_group=4)).forward(x, bias)
    r = 1.0 / (1.0 + torch.exp(-x)) + bias
    best = r.view(T, 8, 32).sort(dim=2, descending=True, stable=True).values
    chosen = (best[:, :, 0] + best[:, :, 1]).sort(dim=1, descending=True, stable=True).indices[:, :4]
    keep = torch.zeros((T, 8), dtype=torch.bool, device="cuda").scatter_(1, chosen, True).repeat_interleave(32, 1)
    want = torch.where(keep, r, -float("inf")).sort(dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(out["topk_idx"].long(), want)
    one = mok.Router(mok.make_route_desc(100, E, k, SIGMOID, True, n_group=8, topk_group=4)).forward(x[:100], bias)
    assert torch.equal(one["topk_idx"], out["topk_idx"][:100])


@pytest.mark.parametrize("E,G,kg", [(256, 8, 4), (222, 6, 3), (384, 8, 3)])
def test_near_experts_and_groups_among_many_tokens(E, G, kg):
    """A group of each token is another one's copy in another order, off by a few f32 steps or not at all: which of
    them is chosen, and the order of their experts, is that of s + b in f32; calls of few tokens agree in every bit."""
    T, k, size = 6000, 8, E // G
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(T, G, size, generator=g, device="cuda")
    token = torch.arange(T, device="cuda")
    of = torch.randint(0, G, (T,), generator=g, device="cuda")
    to = (of + torch.randint(1, G, (T,), generator=g, device="cuda")) % G
    copy = x[token, of][:, torch.randperm(size, generator=g, device="cuda")]
    x[token, to] = copy + torch.randint(-2, 3, (T, 1), generator=g, device="cuda") * 2.0 ** -22
    x = x.view(T, E)
    bias = torch.randint(-2, 3, (G,), generator=g, device="cuda").float().repeat_interleave(size) * 2.0 ** -23
    desc = lambda n: mok.make_route_desc(n, E, k, SIGMOID, True, n_group=G, topk_group=kg)  # noqa: E731
    out = mok.Router(desc(T)).forward(x, bias)
    r = 1.0 / (1.0 + torch.exp(-x)) + bias
    best = r.view(T, G, size).sort(dim=2, descending=True, stable=True).values
    chosen = (best[:, :, 0] + best[:, :, 1]).sort(dim=1, descending=True, stable=True).indices[:, :kg]
    keep = torch.zeros((T, G), dtype=torch.bool, device="cuda").scatter_(1, chosen, True).repeat_interleave(size, 1)
    want = torch.where(keep, r, -float("inf")).sort(dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(out["topk_idx"].long(), want)
    few = mok.Router(desc(600))
    for at in range(0, T, 600):
        part = few.forward(x[at:at + 600], bias)
        assert all(torch.equal(part[n], out[n][at:at + 600]) for n in part)


@pytest.mark.parametrize("G,kg,score", [(1, 1, MAX), (8, 3, TOP2), (8, 3, MAX), (5, 2, TOP2)])
@pytest.mark.parametrize("router", [SIGMOID, SOFTMAX])
@pytest.mark.parametrize("with_bias", [False, True])
def test_masked_experts(G, kg, score, router, with_bias):
    """-inf logits: here and there, whole groups, all but two experts, all of them."""
    T, E, k = 24, 40, 5
    bias = _bias(E, 6, with_bias)
    x, x64 = _logits(T, E, 8, torch.float32, router, bias, k, G, kg, score)
    rng = np.random.default_rng(9)
    x64 = x64.copy()
    x64[:10][rng.random((10, E)) < 0.3] = -np.inf
    x64[10:16, :E // 2] = -np.inf
    x64[16:20] = np.where(np.isin(np.arange(E), (11, 29)), x64[16:20], -np.inf)
    x64[20:] = -np.inf
    idx, margin = O.select(x64, bias, router, k, G, kg, score)
    clear = margin > 1e-5
    desc = mok.make_route_desc(T, E, k, router, True, n_group=G, topk_group=kg, group_score=score, balance_coef=1.0)
    r = mok.Router(desc, balance=True, scores=True)
    out = r.forward(torch.tensor(x64).float().cuda(), _cuda(bias))
    got = out["topk_idx"].cpu().numpy()
    assert clear[20:].all() and np.array_equal(got[clear], idx[clear])
    s = O.scores(x64, router)
    assert np.allclose(f64(out["gates"]), O.gates(s, got, True, 1.0), rtol=REL, atol=0)
    assert np.allclose(f64(out["prob_sum"]), O.probabilities(s).sum(axis=0), rtol=REL, atol=0)
    dg = np.random.default_rng(1).normal(size=(T, k)).astype(np.float32)
    dp = np.random.default_rng(2).normal(size=E).astype(np.float32)
    dl = f64(r.backward(torch.tensor(x64).float().cuda(), out["topk_idx"], _cuda(dg), _cuda(dp)))
    want = O.backward(x64, got, dg.astype(np.float64), dp.astype(np.float64), router, True, 1.0)
    # sums over the token's terms: at most 8 times its largest score and gradients
    size = (np.abs(dg).max() + np.abs(dp).max()) * 8 / np.maximum(np.take_along_axis(s, got.astype(np.int64), 1).sum(1), 1e-30)
    assert np.isfinite(dl).all()
    assert (np.abs(dl - want) <= REL * np.minimum(size, 1e4)[:, None]).all()
    assert not dl[20:].any() and not dl[np.isneginf(x64)].any()


def test_nan_logits_rank_last():
    """An expert with a NaN logit is taken only when nothing else is left; indices stay valid and distinct."""
    x = torch.randn(16, 24, generator=torch.Generator().manual_seed(0))
    x[:8, 5] = float("nan")
    x[8:, :] = float("nan")
    x[8:, 3] = 1.0
    for router in (SIGMOID, SOFTMAX):
        r = mok.Router(mok.make_route_desc(16, 24, 4, router, True, n_group=4, topk_group=2, balance_coef=1.0), balance=True)
        out = r.forward(x.cuda())
        idx = out["topk_idx"].cpu().numpy()
        assert not (idx[:8] == 5).any()
        assert all(len(set(row)) == 4 and min(row) >= 0 and max(row) < 24 for row in idx.tolist())
        assert (idx[8:, 0] == 3).all()
        assert torch.isnan(out["prob_sum"]).all() and torch.isnan(out["loss"]).all()
        # the next call on finite logits is not touched by it
        again = r.forward(torch.zeros(16, 24).cuda())
        assert torch.allclose(again["prob_sum"], torch.full((24,), 16 / 24).cuda(), rtol=1e-6)


@pytest.mark.parametrize("T,E", [(2500, 64), (40000, 64), (2500, 256), (1500, 384)])
def test_nan_logits_among_many_tokens(T, E):
    """As above where two tokens share a warp; the other tokens are routed as without the NaN."""
    k = 4
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(1)).cuda()
    y = x.clone()
    y[7, 3] = float("nan")
    y[1000] = float("nan")
    y[1000, 40:42] = 1.0
    bias = torch.linspace(-0.1, 0.1, E).cuda()
    others = torch.ones(T, dtype=torch.bool)
    others[[7, 1000]] = False
    for router, b in ((SIGMOID, None), (SIGMOID, bias), (SOFTMAX, None)):
        r = mok.Router(mok.make_route_desc(T, E, k, router, True, n_group=8, topk_group=3, balance_coef=1.0), balance=True)
        want = r.forward(x, b)["topk_idx"].clone()
        out = r.forward(y, b)
        assert torch.equal(out["topk_idx"][others], want[others])
        assert not (out["topk_idx"][7] == 3).any()
        last = out["topk_idx"][1000].cpu().tolist()
        assert set(last[:2]) == {40, 41} and len(set(last)) == k and min(last) >= 0 and max(last) < E
        assert torch.isnan(out["prob_sum"]).all()
        assert torch.isfinite(r.forward(x, b)["prob_sum"]).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("E,offset", [(256, 0), (256, 3), (160, 8), (61, 1)])
def test_rows_of_a_wider_tensor(dtype, E, offset):
    """Rows that are a slice of wider ones (aligned and not): forward and backward as on a copy."""
    T, k = 50, 6
    wide = torch.randn(T, E + 16, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    x = wide[:, offset:offset + E]
    r = mok.Router(mok.make_route_desc(T, E, k, SIGMOID, True), dtype=dtype)
    a = {n: t.clone() for n, t in r.forward(x).items()}
    b = r.forward(x.contiguous())
    assert all(torch.equal(a[n], b[n]) for n in a)
    dg = torch.randn(T, k, generator=torch.Generator().manual_seed(2)).cuda()
    dp = torch.randn(E, generator=torch.Generator().manual_seed(3)).cuda()
    room = torch.full((T, E + 16), 7.0, dtype=dtype, device="cuda")
    r.backward(x, a["topk_idx"], dg, dp, out=room[:, offset:offset + E])
    assert torch.equal(room[:, offset:offset + E], r.backward(x.contiguous(), a["topk_idx"], dg, dp))
    assert (room[:, :offset] == 7).all() and (room[:, offset + E:] == 7).all()


@pytest.mark.parametrize("T", [0, 1, 2, 300, 5000, 20000])
def test_balance_outputs_at_every_length(T):
    E, k = 256, 8
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(T)) + torch.linspace(-1, 1, E)
    bias = torch.linspace(0.02, -0.02, E)
    desc = mok.make_route_desc(T, E, k, SIGMOID, True, n_group=8, topk_group=4, balance_coef=2.0, bias_rate=0.001)
    r = mok.Router(desc, balance=True)
    b = bias.cuda()
    first = {n: t.clone() for n, t in r.forward(x.cuda(), b).items()}
    again = r.forward(x.cuda(), b)
    assert all(torch.equal(first[n], again[n]) for n in first)       # any order of the blocks gives these bits
    idx = first["topk_idx"].cpu().numpy()
    s = O.scores(x.double().numpy(), SIGMOID)
    counts, prob_sum, loss, dprob, moved = O.balance(s, idx, 2.0, bias.double().numpy(), float(np.float32(0.001)))
    assert np.array_equal(first["counts"].cpu().numpy(), counts)
    assert np.allclose(f64(first["prob_sum"]), prob_sum, rtol=REL, atol=0)
    assert np.allclose(f64(first["loss"]), [loss], rtol=REL, atol=0)
    assert np.allclose(f64(first["dprob"]), dprob, rtol=REL, atol=0)
    assert np.allclose(f64(first["bias_next"]), moved, rtol=0, atol=2.0 ** -24)
    r.forward(x.cuda(), b, bias_next=b)                               # the bias moved in place
    assert torch.equal(b, first["bias_next"])


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "T%d_E%d_k%d" % s[:3])
@pytest.mark.parametrize("router", [SIGMOID, SOFTMAX])
@pytest.mark.parametrize("use", ["gates", "prob", "both"])
def test_route_backward(shape, router, use):
    T, E, k, G, kg, score = shape
    rng = np.random.default_rng(13)
    for dtype, renorm in ((torch.float32, True), (torch.bfloat16, False)):
        x = torch.tensor(rng.normal(size=(T, E)) * 1.5).to(dtype)
        x64 = x.double().numpy()
        idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
        dg = rng.normal(size=(T, k)).astype(np.float32) if use != "prob" else None
        dp = rng.normal(size=E).astype(np.float32) if use != "gates" else None
        desc = mok.make_route_desc(T, E, k, router, renorm, route_scale=2.5, n_group=G, topk_group=kg, group_score=score)
        status = torch.zeros(2, dtype=torch.int32, device="cuda")
        got = f64(mok.Router(desc, dtype=dtype).backward(x.cuda(), _cuda(idx), _cuda(dg), _cuda(dp), device_status=status))
        want = O.backward(x64, idx, None if dg is None else dg.astype(np.float64),
                          None if dp is None else dp.astype(np.float64), router, renorm, 2.5)
        s = O.scores(x64, router)
        S = np.take_along_axis(s, idx.astype(np.int64), 1).sum(1, keepdims=True)
        # sizes of the terms that each entry is a sum of
        dsel = np.zeros((T, E))
        if dg is not None:
            np.put_along_axis(dsel, idx.astype(np.int64), 2.5 * (np.abs(dg) + np.abs(dg).max(1, keepdims=True) * renorm) /
                              (S if renorm else 1.0), 1)
        both = dsel if dp is None else dsel + (np.abs(dp) + np.abs(dp).max()) / (s.sum(1, keepdims=True) if router else 1.0)
        size = s * (both + (0 if router else (s * both).sum(1, keepdims=True)))
        tol = REL * size + (np.abs(want) * 2.0 ** -8 if dtype == torch.bfloat16 else 0) + 1e-38
        assert (np.abs(got - want) <= tol).all(), (dtype, np.abs(got - want).max())
        assert status.tolist() == [0, 0]


@pytest.mark.parametrize("router", [SIGMOID, SOFTMAX])
@pytest.mark.parametrize("E", [24, 300, 600])
def test_backward_against_differences_of_the_forward(router, E):
    """Central differences of f = sum dgates * gates + sum dprob * prob_sum, of the forward kernel's scores and sums.  The step
    is 2^-5: f in f32 (a sum of about 30 terms near 1 in f64, each off by 2^-21) is off by 30 * 2^-21, over twice the
    step 2.3e-4; the third derivative, at most 1 for a sigmoid's or softmax's share times gradients of about 3,
    leaves 3 * 2^-10 / 6 = 5e-4."""
    T, k = 3, 4
    rng = np.random.default_rng(3)
    x = torch.tensor(rng.normal(size=(T, E))).float()
    x[:, :k] += 3.0
    dg = torch.tensor(rng.normal(size=(T, k))).float().cuda()
    dp = torch.tensor(rng.normal(size=E)).float().cuda()
    r = mok.Router(mok.make_route_desc(T, E, k, router, True, balance_coef=1.0), balance=True, scores=True)

    def f(z):
        out = r.forward(z.cuda())
        s = out["scores"].double()[:, :k]             # the selection is held fixed
        return ((dg.double() * s / s.sum(1, keepdim=True)).sum() + (dp.double() * out["prob_sum"].double()).sum()).item()

    idx = torch.arange(k, dtype=torch.int32).repeat(T, 1).cuda()
    got = r.backward(x.cuda(), idx, dg, dp).cpu()
    h = 2.0 ** -5
    for t in range(T):
        for e in [0, 1, 2, 3, 4, 7, E - 1]:
            up, down = x.clone(), x.clone()
            up[t, e] += h
            down[t, e] -= h
            assert abs((f(up) - f(down)) / (2 * h) - got[t, e].item()) < 2.3e-4 + 5e-4, (t, e)


def test_backward_leaves_out_and_reports_a_bad_index():
    T, E, k = 4, 32, 3
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(0)).cuda()
    idx = torch.tensor([[0, 1, 2]] * T, dtype=torch.int32)
    bad = idx.clone()
    bad[1, 2], bad[2, 0] = E, -1
    dg = torch.ones(T, k).cuda()
    r = mok.Router(mok.make_route_desc(T, E, k, SIGMOID, False))
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    a = r.backward(x, bad.cuda(), dg, device_status=status).clone()
    assert status[0].item() == 6
    b = r.backward(x, idx.cuda(), dg)
    b[1, 2], b[2, 0] = 0, 0
    assert torch.equal(a, b)


def test_no_tokens():
    r = mok.Router(mok.make_route_desc(0, 16, 2, SIGMOID, True))
    x = torch.empty(0, 16).cuda()
    assert r.forward(x)["topk_idx"].shape == (0, 2)
    assert r.backward(x, torch.empty(0, 2, dtype=torch.int32).cuda(), torch.empty(0, 2).cuda()).shape == (0, 16)


@pytest.mark.parametrize("T,E", [(2 ** 21 + 3, 1024), (2 ** 23 + 3, 256)])
def test_rows_past_32_bit_offsets(T, E):
    """More than 2^31 logits: the last tokens are routed, and their gradients written, as on their own."""
    k, tail = 4, 100
    x = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    x[-tail:] = torch.randn(tail, E, generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    x[-2 * tail:-tail] = x[-tail:]
    big = mok.Router(mok.make_route_desc(T, E, k, SIGMOID, True, n_group=8, topk_group=4), dtype=torch.bfloat16)
    small = mok.Router(mok.make_route_desc(tail, E, k, SIGMOID, True, n_group=8, topk_group=4), dtype=torch.bfloat16)
    a, b = big.forward(x), small.forward(x[-tail:])
    assert torch.equal(a["topk_idx"][-tail:], b["topk_idx"]) and torch.equal(a["gates"][-2 * tail:-tail], b["gates"])
    assert (a["topk_idx"][:1000] == torch.arange(k, device="cuda")).all()
    dg = torch.ones(T, k, device="cuda") + torch.arange(k, device="cuda")
    dl, small_dl = big.backward(x, a["topk_idx"], dg), small.backward(x[-tail:], b["topk_idx"], dg[:tail])
    assert torch.equal(dl[-tail:], small_dl) and torch.equal(dl[-2 * tail:-tail], small_dl)


def test_on_another_stream_and_in_a_graph():
    T, E, k = 300, 256, 8
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(4)).cuda()
    bias = torch.zeros(E, device="cuda")
    r = mok.Router(mok.make_route_desc(T, E, k, SIGMOID, True, n_group=8, topk_group=4, balance_coef=1.0, bias_rate=0.1),
                   balance=True)
    want = {n: t.clone() for n, t in r.forward(x, bias).items()}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for t in r.out.values():
        t.zero_()
    torch.cuda.synchronize()
    out = r.forward(x, bias, stream=side)
    side.synchronize()
    assert all(torch.equal(out[n], want[n]) for n in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.forward(x, bias)
        dl = r.backward(x, r.out["topk_idx"], torch.ones(T, k, device="cuda"), r.out["dprob"], out=torch.empty_like(x))
    for _ in range(2):
        for t in r.out.values():
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[n], want[n]) for n in want)
    assert torch.equal(dl, r.backward(x, r.out["topk_idx"], torch.ones(T, k, device="cuda"), r.out["dprob"]))


# ------------------------------------------------------------------ the layer with groups

GROUPED = W.MoEShape("grouped_T200_H256_E32_I256_top4", T=200, H=256, E=32, I=256, k=4, router=SIGMOID, renorm=True,
                     x_std=1.0, w_std=0.05)


@pytest.mark.parametrize("router,score", [(SIGMOID, TOP2), (SOFTMAX, MAX)])
@pytest.mark.parametrize("mxfp8", [False, True])
def test_layer_routes_within_groups(router, score, mxfp8):
    """The layer's selection, gates and scores with groups are mok_route's on the layer's own logits; the rest
    of the forward is the layer's on that selection, given."""
    shape = GROUPED.scaled(router=router, renorm=router == SIGMOID, mxfp8=mxfp8)
    inp = {n: t.cuda() for n, t in W.make_inputs(shape, seed=3).items() if t is not None}
    bias = _cuda(_bias(32, 4, router == SIGMOID))
    kw = dict(n_group=8, topk_group=3, group_score=score)
    layer, given = mok.MoELayer(mok.desc_from_shape(shape, **kw)), mok.MoELayer(mok.desc_from_shape(shape))
    results = []
    for lay, sel in ((layer, None), (given, "given")):
        sel = None if sel is None else layer.view("topk_idx").clone()
        if mxfp8:
            wq = mok.quantize_weights(lay.desc, inp["w13"], inp["w2"])
            y = torch.empty((shape.T, shape.H), dtype=torch.bfloat16, device="cuda")
            mok.moe_forward_mxfp8(lay.desc, inp["x"], inp["w_router"], bias, sel, wq, y, lay.ctx, lay.ws)
        else:
            y = lay.forward(inp["x"], inp["w_router"], inp["w13"], inp["w2"], router_bias=bias, given_topk=sel)
        assert lay.status() == (0, 0)
        results.append(y)
    assert torch.equal(results[0], results[1])
    desc = mok.make_route_desc(shape.T, 32, 4, router, shape.renorm, **kw)
    out = mok.Router(desc, scores=True).forward(layer.view("logits"), bias)
    for n in ("topk_idx", "gates", "scores"):
        assert torch.equal(out[n], layer.view(n)), n
    idx = out["topk_idx"].cpu().numpy()
    assert max(len(set(row // 4)) for row in idx) <= 3
    if mxfp8:
        return
    # the schedule entry points take the same selection
    outs = {n: torch.empty(s, dtype=torch.int32, device="cuda") for n, s in
            (("topk_idx", (200, 4)), ("counts", (32,)), ("offsets", (33,)), ("row_of", (800,)), ("src_of", (800,)))}
    gates = torch.empty((200, 4), device="cuda")
    rest = (outs["topk_idx"], gates, outs["counts"], outs["offsets"], outs["row_of"], outs["src_of"])
    from mixture_experts_layer_table_gb300 import _native as N
    for call in (lambda: mok.schedule(layer.desc, inp["x"], inp["w_router"], bias, None, *rest, layer.ws),
                 lambda: N.schedule_noalloc(layer.desc, inp["x"], inp["w_router"], bias, None, *rest)):
        outs["topk_idx"].fill_(-1)
        call()
        assert torch.equal(outs["topk_idx"], out["topk_idx"]) and torch.equal(gates, out["gates"])
    # the gate gradients go back through the same Jacobian
    grads = given.backward(inp["dy"], inp["x"], inp["w_router"], inp["w13"], inp["w2"])
    mine = layer.forward(inp["x"], inp["w_router"], inp["w13"], inp["w2"], router_bias=bias)
    assert torch.equal(mine, results[0])
    grouped = layer.backward(inp["dy"], inp["x"], inp["w_router"], inp["w13"], inp["w2"])
    assert all(torch.equal(grads[n], grouped[n]) for n in grads)
    dl = mok.Router(desc).backward(layer.view("logits"), layer.view("topk_idx"), grads["dgates"])
    assert torch.allclose(dl, layer.view("dlogits"), rtol=1e-4, atol=1e-6 * layer.view("dlogits").abs().max().item())


@pytest.mark.parametrize("E", [32, 256])
def test_layer_with_groups_and_many_tokens(E):
    """With 256 experts 2,100 tokens are many: the layer's selection is that kernel's, with the scores it hands out."""
    shape = GROUPED.scaled(T=2100, E=E)
    inp = {n: t.cuda() for n, t in W.make_inputs(shape, seed=3).items() if t is not None}
    bias = _cuda(_bias(E, 4, True))
    layer = mok.MoELayer(mok.desc_from_shape(shape, n_group=8, topk_group=3, group_score=TOP2))
    layer.forward(inp["x"], inp["w_router"], inp["w13"], inp["w2"], router_bias=bias)
    assert layer.status() == (0, 0)
    logits = layer.view("logits")
    out = mok.Router(mok.make_route_desc(2100, E, 4, SIGMOID, True, n_group=8, topk_group=3), scores=True).forward(logits, bias)
    for n in ("topk_idx", "gates", "scores"):
        assert torch.equal(out[n], layer.view(n)), n
    first = mok.Router(mok.make_route_desc(100, E, 4, SIGMOID, True, n_group=8, topk_group=3), scores=True).forward(logits[:100], bias)
    for n in ("topk_idx", "gates", "scores"):
        assert torch.equal(first[n], out[n][:100]), n


def test_layer_refuses_bad_groups():
    for kw in (dict(n_group=-1), dict(n_group=5, topk_group=1), dict(n_group=8, topk_group=0),
               dict(n_group=8, topk_group=9), dict(n_group=32, topk_group=3), dict(n_group=8, topk_group=2, group_score=2)):
        with pytest.raises(mok.MokError):
            mok.get_layout(mok.desc_from_shape(GROUPED, **kw))


def _f32_selection(x, bias, k, G, kg, top2=True):
    """The selection by s + b in f32, s = 1 / (1 + e^-x) by steps rounded to f32, ties to the lower index: -inf ranks
    (masked logits, biases of -inf or NaN) behind all others and in no group's value."""
    T, E = x.shape
    r = 1.0 / (1.0 + torch.exp(-x)) + bias
    r = torch.where((x > -float("inf")) & ~torch.isnan(r), r, -float("inf"))
    first = r.sort(dim=1, descending=True, stable=True).indices
    if G > 1:
        best = r.view(T, G, E // G).sort(dim=2, descending=True, stable=True).values
        value = best[:, :, 0]
        if top2 and E > G:
            value = torch.where(best[:, :, 1] > -float("inf"), value + best[:, :, 1], value)
        chosen = value.sort(dim=1, descending=True, stable=True).indices[:, :kg]
        left_out = torch.ones((T, G), dtype=torch.int32, device=x.device).scatter_(1, chosen, 0).repeat_interleave(E // G, 1)
        first = first.gather(1, left_out.gather(1, first).sort(dim=1, stable=True).indices)   # behind -inf
    return first[:, :k]


LOWEST, LARGEST, INF = torch.finfo(torch.float32).min, torch.finfo(torch.float32).max, float("inf")


def _extreme_bias(kind, E, size, rng):
    b = (rng.normal(size=E) * 0.1).astype(np.float32)
    at = np.arange(E)
    if kind == "lowest":
        b[rng.random(E) < 0.2] = LOWEST
    elif kind == "lowest_groups":                       # whole groups, and all but one expert of another
        b[: size] = LOWEST
        b[E - size + 1:] = LOWEST
    elif kind == "lowest_but_three":
        b[~np.isin(at, (1, E // 2, E - 1))] = LOWEST
    elif kind == "minus_inf":
        b[rng.random(E) < 0.3] = -np.inf
    elif kind == "plus_inf":                            # in every group, and twice in some
        b[at % size == 0] = np.inf
        b[min(3, E - 1)] = np.inf
    elif kind == "plus_inf_one":
        b[E - 1] = np.inf
    elif kind == "mixed":
        for value in (LOWEST, LARGEST, -np.inf, np.nan, 1e30, -1e30, 2.0 ** 26, -2.0 ** 25, 1e5, -1e5, 30.0):
            b[rng.random(E) < 0.03] = value
    elif kind == "all_lowest":
        b[:] = LOWEST
    elif kind == "all_largest":
        b[:] = LARGEST
    return b


@pytest.mark.parametrize("E,k,G,kg,score", [(256, 8, 8, 4, TOP2), (222, 8, 6, 3, TOP2), (222, 8, 6, 3, MAX), (35, 4, 5, 2, MAX),
                                            (57, 5, 3, 2, TOP2), (511, 8, 1, 1, MAX), (384, 8, 8, 3, TOP2), (20, 4, 20, 6, TOP2)])
@pytest.mark.parametrize("kind", ["lowest", "lowest_groups", "lowest_but_three", "minus_inf", "plus_inf", "plus_inf_one",
                                  "mixed", "all_lowest", "all_largest"])
def test_biases_at_the_ends_of_the_type(E, k, G, kg, score, kind):
    """Masks by the type's lowest value or -inf, experts forced by +inf, in calls of many tokens and of few: the selection
    of the f32 rank values, indices in range and distinct."""
    T, rng = max(_many(E) + 3, 2500), np.random.default_rng(43)
    g = torch.Generator(device="cuda").manual_seed(2)
    rows = torch.randn(500, E, generator=g, device="cuda")
    rows[:100][torch.rand(100, E, generator=g, device="cuda") < 0.1] = -INF
    x = rows[torch.arange(T, device="cuda") % 500]
    bias = _cuda(_extreme_bias(kind, E, E // G, rng))
    want = _f32_selection(rows, bias, k, G, kg, score == TOP2)[torch.arange(T, device="cuda") % 500]
    desc = lambda n: mok.make_route_desc(n, E, k, SIGMOID, True, n_group=G, topk_group=kg, group_score=score)  # noqa: E731
    first = mok.Router(desc(500)).forward(rows, bias)
    assert torch.equal(first["topk_idx"].long(), want[:500])
    for kw in (dict(), dict(scores=True), dict(balance=True)):
        out = mok.Router(desc(T), **kw).forward(x, bias)
        assert torch.equal(out["topk_idx"].long(), want), kw
        assert torch.equal(out["gates"][-500:], first["gates"][torch.arange(T - 500, T, device="cuda") % 500])
        if "counts" in out:
            assert torch.equal(out["counts"].long(), torch.bincount(want.flatten(), minlength=E))


@pytest.mark.parametrize("E,k,G,kg", [(256, 8, 8, 4), (222, 8, 6, 3), (35, 4, 5, 2), (384, 8, 8, 3)])
def test_infinite_logits_in_groups_that_are_not_chosen(E, k, G, kg):
    """Groups ranked by their best logit, +inf in more of them than are chosen: ties to the lower groups, and no expert of
    the others."""
    T, size = max(_many(E) + 3, 2500), E // G
    rows = torch.randn(500, E, generator=torch.Generator().manual_seed(3))
    rows[:, 1::size] = INF
    x = rows.cuda()[torch.arange(T, device="cuda") % 500]
    desc = lambda n: mok.make_route_desc(n, E, k, SOFTMAX, True, n_group=G, topk_group=kg, group_score=MAX)  # noqa: E731
    idx, _ = O.select(rows.double().numpy(), None, SOFTMAX, k, G, kg, MAX)
    assert np.array_equal(mok.Router(desc(500)).forward(rows.cuda())["topk_idx"].cpu().numpy(), idx)
    out = mok.Router(desc(T)).forward(x)["topk_idx"]
    assert torch.equal(out, _cuda(idx)[torch.arange(T, device="cuda") % 500])


@pytest.mark.parametrize("size_of_bias", [30.0, 1000.0])
@pytest.mark.parametrize("E,G,kg", [(256, 8, 4), (222, 6, 3), (384, 8, 3)])
def test_near_groups_whose_best_have_large_biases_of_opposite_sign(E, G, kg, size_of_bias):
    """One expert of each group is favoured by a large bias and the others are held back by it: a group's sum of two is
    small, its summands and what the approximate ones are off by are not.  The groups are copies of one another, off by a
    few steps of their rank values' rounding."""
    T, k, size = 6000, 8, E // G
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, 1, size, generator=g, device="cuda").repeat(1, G, 1)
    x = x + torch.randint(-3, 4, (T, G, 1), generator=g, device="cuda") * (size_of_bias * 2.0 ** -25)
    x = x.view(T, E)
    bias = torch.where(torch.arange(E, device="cuda") % size == 0, size_of_bias, -size_of_bias)
    desc = lambda n: mok.make_route_desc(n, E, k, SIGMOID, True, n_group=G, topk_group=kg)  # noqa: E731
    out = mok.Router(desc(T)).forward(x, bias)
    assert torch.equal(out["topk_idx"].long(), _f32_selection(x, bias, k, G, kg))
    few = mok.Router(desc(600))
    for at in range(0, T, 600):
        part = few.forward(x[at:at + 600], bias)
        assert all(torch.equal(part[n], out[n][at:at + 600]) for n in part)


def _spread(T, E, seed, std, offset, router, bias, k, G, kg, score):
    """As _logits, of any spread and place, for the softmax."""
    x = torch.tensor(np.random.default_rng(seed).normal(size=(8 * T + 40, E)) * std + offset).float()
    keep = O.select(x.double().numpy(), bias, router, k, G, kg, score)[1] > 1e-5
    x = x[torch.tensor(keep)][:T]
    assert x.shape[0] == T
    return x.contiguous().cuda(), x.double().numpy()


SPREADS = [(1.5, 0.0), (3.0, 300.0), (8.0, 0.0), (1.5, -1000.0), (1.5, 20000.0)]


@pytest.mark.parametrize("E,k,G,kg,score", [(64, 6, 8, 3, MAX), (160, 6, 8, 3, MAX), (222, 8, 6, 3, MAX), (256, 8, 1, 1, MAX),
                                            (384, 8, 8, 4, MAX), (1024, 12, 8, 4, MAX)])
@pytest.mark.parametrize("std,offset", SPREADS)
@pytest.mark.parametrize("renorm", [False, True])
def test_softmax_gates_of_wide_and_shifted_logits(E, k, G, kg, score, std, offset, renorm):
    """Gates are e^(x - max) over one sum, whatever the largest logit is and however many tokens a call has.  A score's
    exponent (x - max) log2 e is rounded twice on top: 2^-23 of its size."""
    x, x64 = _spread(40, E, 23, std, offset, SOFTMAX, None, k, G, kg, score)
    idx, _ = O.select(x64, None, SOFTMAX, k, G, kg, score)
    s = O.scores(x64, SOFTMAX)
    away = x64.max(axis=1, keepdims=True) - x64
    for T in (40, _many(E) + 3):
        of = np.arange(T) % 40
        desc = mok.make_route_desc(T, E, k, SOFTMAX, renorm, route_scale=2.5, n_group=G, topk_group=kg, group_score=score,
                                   balance_coef=0.3)
        rows = x[torch.tensor(of).cuda()]
        plain = mok.Router(desc).forward(rows)
        full = mok.Router(desc, balance=True, scores=True).forward(rows)
        for out in (plain, full):
            assert np.array_equal(out["topk_idx"].cpu().numpy(), idx[of])
            assert np.allclose(f64(out["gates"]), O.gates(s, idx, renorm, 2.5)[of], rtol=REL, atol=1e-37)
        assert (np.abs(f64(full["scores"]) - s[of]) <= (REL + 2.0 ** -23 * away[of]) * s[of] + 1e-37).all()
        prob = s[of].sum(axis=0)
        assert (np.abs(f64(full["prob_sum"]) - prob) <= REL * prob + (2.0 ** -23 * away * s)[of].sum(axis=0) + T * 1e-37).all()


@pytest.mark.parametrize("E,k,G,kg,score", [(64, 6, 8, 3, MAX), (222, 8, 6, 3, TOP2), (256, 8, 8, 4, TOP2), (384, 8, 8, 4, MAX)])
def test_sigmoid_gates_of_many_tokens_without_renormalisation(E, k, G, kg, score):
    for with_bias in (False, True):
        bias = _bias(E, 15, with_bias)
        x, x64 = _logits(40, E, 19, torch.float32, SIGMOID, bias, k, G, kg, score)
        idx, _ = O.select(x64, bias, SIGMOID, k, G, kg, score)
        T = _many(E) + 3
        of = np.arange(T) % 40
        desc = mok.make_route_desc(T, E, k, SIGMOID, False, route_scale=2.5, n_group=G, topk_group=kg, group_score=score)
        for scores in (False, True):
            out = mok.Router(desc, scores=scores).forward(x[torch.tensor(of).cuda()], _cuda(bias))
            assert np.array_equal(out["topk_idx"].cpu().numpy(), idx[of])
            assert np.allclose(f64(out["gates"]), O.gates(O.scores(x64, SIGMOID), idx, False, 2.5)[of], rtol=REL, atol=0)


@pytest.mark.parametrize("E,k", [(24, 3), (61, 4), (160, 6), (256, 8), (500, 9), (1024, 16)])
@pytest.mark.parametrize("std,offset", SPREADS)
@pytest.mark.parametrize("renorm", [False, True])
def test_softmax_backward_of_wide_and_shifted_logits(E, k, std, offset, renorm):
    """f32 gradients at the selected experts and at the others, to 2^-18 of their terms, and 2^-23 more for each unit
    that a logit lies below the largest."""
    T = 50
    rng = np.random.default_rng(29)
    x = torch.tensor(rng.normal(size=(T, E)) * std + offset).float()
    x64 = x.double().numpy()
    idx = np.argsort(-x64, axis=1, kind="stable")[:, :k].astype(np.int32)
    s, away = O.scores(x64, SOFTMAX), x64.max(axis=1, keepdims=True) - x64
    S = np.take_along_axis(s, idx.astype(np.int64), 1).sum(1, keepdims=True)
    r = mok.Router(mok.make_route_desc(T, E, k, SOFTMAX, renorm, route_scale=2.5))
    for use in ("gates", "both"):
        dg = rng.normal(size=(T, k)).astype(np.float32)
        dp = rng.normal(size=E).astype(np.float32) if use == "both" else None
        got = f64(r.backward(x.cuda(), _cuda(idx), _cuda(dg), _cuda(dp)))
        want = O.backward(x64, idx, dg.astype(np.float64), None if dp is None else dp.astype(np.float64), SOFTMAX, renorm, 2.5)
        both = np.zeros((T, E))
        np.put_along_axis(both, idx.astype(np.int64), 2.5 * (np.abs(dg) + np.abs(dg).max(1, keepdims=True) * renorm) /
                          (S if renorm else 1.0), 1)
        both = both if dp is None else both + np.abs(dp) + np.abs(dp).max()
        more = REL + 2.0 ** -23 * away
        tol = s * (more * both + (s * more * both).sum(1, keepdims=True) + more * (s * both).sum(1, keepdims=True)) + 1e-36
        assert (np.abs(got - want) <= tol).all(), (use, (np.abs(got - want) / tol).max())


@pytest.mark.parametrize("E,k", [(24, 3), (160, 6), (256, 8), (500, 9)])
def test_sigmoid_backward_without_renormalisation(E, k):
    T = 50
    rng = np.random.default_rng(31)
    x = torch.tensor(rng.normal(size=(T, E)) * 1.5).float()
    x64 = x.double().numpy()
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    dg, dp = rng.normal(size=(T, k)).astype(np.float32), rng.normal(size=E).astype(np.float32)
    s = O.scores(x64, SIGMOID)
    for p in (None, dp):
        got = f64(mok.Router(mok.make_route_desc(T, E, k, SIGMOID, False, route_scale=2.5)).backward(
            x.cuda(), _cuda(idx), _cuda(dg), _cuda(p)))
        want = O.backward(x64, idx, dg.astype(np.float64), None if p is None else p.astype(np.float64), SIGMOID, False, 2.5)
        both = np.zeros((T, E))
        np.put_along_axis(both, idx.astype(np.int64), 2.5 * np.abs(dg), 1)
        if p is not None:
            both += (np.abs(p) + np.abs(p).max()) / s.sum(1, keepdims=True)
        assert (np.abs(got - want) <= REL * s * both + 1e-38).all()


def test_a_new_workspace_is_ready_on_another_stream():
    """The current stream is busy when the router is made, in memory that was not zero; its first call goes to another."""
    T, E, k = 300, 64, 4
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(6)).cuda()
    desc = mok.make_route_desc(T, E, k, SIGMOID, True, n_group=8, topk_group=4, balance_coef=1.0)
    want = {n: t.clone() for n, t in mok.Router(desc, balance=True).forward(x).items()}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.full((98560,), 0xff, dtype=torch.uint8, device="cuda")
    torch.cuda._sleep(40_000_000)
    r = mok.Router(desc, balance=True)
    assert torch.cuda.current_stream().query()
    out = r.forward(x, stream=side)
    side.synchronize()
    assert all(torch.equal(out[n], want[n]) for n in want)
