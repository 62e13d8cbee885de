"""GPU parity of the operators for experts outside the layer against the float64 CPU oracle.

Tolerances, from the arithmetic (u = 2^-24, half = half a spacing of the output's type, relative to the value):
  gathered rows are copies, with gates one f32 product: u and half
  merged rows: k products and additions in f32: (k + 1) u of the terms' sizes, and half
  gate gradients: a chain of at most H / 32 + 8 fused additions, 5 over the lanes, 16 over the warps: that many u of the
    terms' sizes
  E4M3 elements are nearest to 448 x / amax: exact for bf16 inputs (the quotient is corrected, ties stay ties); for values
    that were computed in f32 with a relative error d (of their terms), within half an E4M3 step and 2 d: plain f32
    rows d = 2^-22, SwiGLU and its gradient (an exponential, a quotient, up to six roundings) d = 2^-19
  products: a block's 128 terms in the tensor cores' f32 (which may cut where f32 would round: 2 u a step), three
    roundings for its scales, one addition for each block: (128 + 4 + blocks) 2 u of the terms' sizes, and half
"""


import numpy as np
import pytest
import torch

import mixture_experts_layer_table_gb300 as mok
from mixture_experts_layer_table_gb300 import experts as X
from oracle import experts_oracle as O

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_ok):
    from mixture_experts_layer_table_gb300 import build
    build.build()
    mok.load()


def f64(t):
    return t.detach().float().double().cpu().numpy()


def cuda(a, dtype=None):
    return torch.tensor(np.asarray(a), dtype=dtype).cuda()


def values(rng, shape, dtype, spread=0.5):
    """(CUDA tensor, its float64 values): rows of unequal size."""
    x = torch.tensor(rng.normal(size=shape) * np.exp(spread * rng.normal(size=(*shape[:-1], 1)))).to(dtype)
    return x.cuda(), x.double().numpy()


def wide(t, extra, unit=1):
    """The same rows further apart, and behind them what must not be touched."""
    rows, width = t.shape
    ld = -(-(width + extra) // unit) * unit
    big = torch.full((rows, ld), 3.0, device=t.device).to(t.dtype)
    big[:, :width] = t
    return big[:, :width]


def table(rng, T, k, E, dropped=0.0, skew=0.0):
    """expert of each assignment (distinct in a token), src_of, row_of, offsets"""
    w = np.exp(skew * rng.normal(size=E))
    expert = np.concatenate([rng.choice(E, k, replace=False, p=w / w.sum()) for _ in range(T)]) if T else np.zeros(0, int)
    expert = np.where(rng.random(T * k) < dropped, -1, expert)
    return O.table(expert, E)


# (T, k, E, H): one of everything, narrow and odd rows, pieces of 2, 4 and 16 bytes, k of every kernel, wide rows
ROWS = [(1, 1, 1, 1), (3, 2, 5, 7), (50, 3, 8, 36), (33, 4, 16, 126), (20, 6, 48, 1111), (9, 8, 16, 4096),
        (5, 16, 16, 264), (200, 1, 2, 40), (2, 12, 20, 9000), (330, 2, 8, 520), (600, 3, 8, 101), (520, 2, 4, 402)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,k,E,H", ROWS)
def test_rows_by_expert_and_back(T, k, E, H, dtype):
    rng = np.random.default_rng(T * 31 + H)
    src, row, _ = table(rng, T, k, E, dropped=0.3 if T > 2 else 0.0)
    x, x64 = values(rng, (T, H), dtype)
    g = cuda(rng.random((T, k)) + 0.1, F32)
    g64 = f64(g)
    out = mok.gather_rows(x, cuda(src), k)
    assert np.array_equal(f64(out), O.gather(x64, src, k))
    want = O.gather(x64, src, k, g64)
    got = f64(mok.gather_rows(x, cuda(src), k, gates=g))
    assert (np.abs(got - want) <= (U + HALF[dtype]) * np.abs(want)).all()
    o, o64 = values(rng, (T * k, H), dtype)
    for gates, gates64 in ((g, g64), (None, None)):
        y, size = O.merge(o64, row, k, gates64)
        got = f64(mok.merge_rows(o, cuda(row), k, gates))
        assert (np.abs(got - y) <= (k + 1) * U * size + HALF[dtype] * np.abs(y)).all()
    dy, dy64 = values(rng, (T, H), dtype)
    do, dg, size = O.merge_backward(dy64, o64, row, g64)
    buffers = {"do": torch.full((T * k, H), 7.0, dtype=dtype).cuda(), "dgates": torch.full((T, k), 7.0).cuda()}
    out = mok.merge_rows_backward(dy, o, cuda(row), g, out=buffers)
    got = f64(out["do"])
    untouched = np.isnan(do)
    assert (got[untouched] == 7.0).all()
    assert (np.abs(got - do) <= (U + HALF[dtype]) * np.abs(do))[~untouched].all()
    assert (np.abs(f64(out["dgates"]) - dg) <= (H / 32 + 29) * U * size).all()


@pytest.mark.parametrize("dtype,extra", [(BF, 1), (BF, 2), (BF, 8), (F32, 1), (F32, 4)])
def test_rows_further_apart(dtype, extra):
    rng = np.random.default_rng(extra)
    T, k, E, H = 40, 4, 8, 264
    src, row, _ = table(rng, T, k, E)
    x, x64 = values(rng, (T, H), dtype)
    o, o64 = values(rng, (T * k, H), dtype)
    g = cuda(rng.random((T, k)), F32)
    xg = wide(torch.zeros(T * k, H, dtype=dtype).cuda(), extra)
    mok.gather_rows(wide(x, extra), cuda(src), k, out=xg)
    assert torch.equal(xg, mok.gather_rows(x, cuda(src), k))
    y = wide(torch.zeros(T, H, dtype=dtype).cuda(), extra)
    mok.merge_rows(wide(o, extra), cuda(row), k, g, out=y)
    assert torch.equal(y, mok.merge_rows(o, cuda(row), k, g))
    out = {"do": wide(torch.zeros(T * k, H, dtype=dtype).cuda(), extra), "dgates": torch.empty(T, k).cuda()}
    mok.merge_rows_backward(wide(x, extra), wide(o, extra), cuda(row), g, out=out)
    plain = mok.merge_rows_backward(x, o, cuda(row), g)
    assert torch.equal(out["do"], plain["do"])
    # other pieces, another order of the sum
    assert (np.abs(f64(out["dgates"]) - f64(plain["dgates"])) <= 2 * (H / 32 + 29) * U *
            O.merge_backward(x64, o64, row, f64(g))[2]).all()
    for t in (xg, y, out["do"]):
        ld = t.stride(0)
        assert (torch.as_strided(t, (t.shape[0] - 1, ld - H), (ld, 1), H) == 3.0).all()


def test_merge_gradient_of_rows_further_apart_without_buffers():
    rng = np.random.default_rng(8)
    T, k, E, H = 12, 2, 4, 136
    _, row, _ = table(rng, T, k, E)
    dy, _ = values(rng, (T, H), BF)
    o, _ = values(rng, (T * k, H + 24), BF)
    o = o[:, :H]
    g = cuda(rng.random((T, k)), F32)
    got, want = mok.merge_rows_backward(dy, o, cuda(row), g), mok.merge_rows_backward(dy, o.contiguous(), cuda(row), g)
    assert torch.equal(got["do"], want["do"]) and torch.equal(got["dgates"], want["dgates"])


def test_indices_out_of_range_are_reported_and_left_out():
    x, o = torch.ones(4, 16).cuda(), torch.ones(8, 16).cuda()
    good = torch.arange(8, dtype=torch.int32)
    for bad in (-2, 8, 2 ** 31 - 1, -2 ** 31):
        idx = good.clone()
        idx[3] = bad
        status = torch.zeros(2, dtype=torch.int32).cuda()
        xg = mok.gather_rows(x, idx.cuda(), 2, device_status=status)
        assert status.tolist() == [6, 40] and (xg[3] == 0).all() and xg.sum() == 7 * 16
        status.zero_()
        y = mok.merge_rows(o, idx.cuda(), 2, device_status=status)
        assert status.tolist() == [6, 41] and y.sum() == 7 * 16
        status.zero_()
        out = mok.merge_rows_backward(x, o, idx.cuda(), torch.ones(4, 2).cuda(), device_status=status)
        assert status.tolist() == [6, 41] and out["dgates"][1, 1] == 0 and (out["do"][3] == 0).all()
        status.zero_()
        q = mok.fp8_quantize(x, src_of=idx.cuda(), k=2, device_status=status)
        assert status.tolist() == [6, 42] and (q["q"][3].float() == 0).all()
        assert mok.gather_rows(x, idx.cuda(), 2).shape == (8, 16)       # no status word wanted


def test_empty_tables():
    x, none = torch.ones(0, 16).cuda(), torch.empty(0, dtype=torch.int32).cuda()
    assert mok.gather_rows(x, none, 2).shape == (0, 16)
    assert mok.merge_rows(x, none, 2).shape == (0, 16)
    # tokens without rows
    drop = torch.full((6,), -1, dtype=torch.int32).cuda()
    assert (mok.merge_rows(x, drop, 2) == 0).all()
    out = mok.merge_rows_backward(torch.ones(3, 16).cuda(), x, drop, torch.ones(3, 2).cuda())
    assert (out["dgates"] == 0).all()
    # no rows at all, with and without groups, through every call of an expert
    off = torch.zeros(4, dtype=torch.int32).cuda()
    w = mok.Fp8Weights(torch.ones(3, 8, 16).cuda(), transposed=True)
    q = mok.fp8_quantize(x, src_of=none, k=2, offsets=off)
    h = mok.fp8_quantize(w.matmul(q["q"], q["scale"], off), source="swiglu", offsets=off)
    assert h["q"].shape == (0, 4) and w.matmul_transposed(mok.fp8_quantize(torch.ones(0, 8).cuda())["q"],
                                                          torch.ones(1, 0).cuda(), off).shape == (0, 16)
    assert (mok.fp8_weight_grad(h["qt"], h["qt_scale"], q["qt"], q["qt_scale"], off) == 0).all()
    # rows without tokens
    assert (mok.gather_rows(x, drop, 2) == 0).all()
    q = mok.fp8_quantize(x, src_of=drop, k=2)
    assert (q["q"].float() == 0).all() and torch.equal(q["scale"], torch.full((1, 6), 2.0 ** -110 / 448).cuda())


def test_merge_gradient_by_differences():
    """The merge is linear in the rows and in the gates: differences are its derivatives up to f32's rounding."""
    rng = np.random.default_rng(3)
    T, k, E, H = 6, 3, 4, 40
    src, row, _ = table(rng, T, k, E, dropped=0.2)
    o, _ = values(rng, (T * k, H), F32)
    dy, dy64 = values(rng, (T, H), F32)
    g = cuda(rng.random((T, k)), F32)
    out = mok.merge_rows_backward(dy, o, cuda(row), g)
    loss = lambda o, g: (f64(mok.merge_rows(o, cuda(row), k, g)) * dy64).sum()  # noqa: E731
    base, size = loss(o, g), (np.abs(f64(mok.merge_rows(o.abs(), cuda(row), k, g))) * np.abs(dy64)).sum()
    for _ in range(10):
        r, h, t, j = rng.integers(T * k), rng.integers(H), rng.integers(T), rng.integers(k)
        o2, g2 = o.clone(), g.clone()
        o2[r, h] += 4.0
        g2[t, j] += 4.0
        assert abs((loss(o2, g) - base) / 4.0 - float(out["do"][r, h])) <= 8 * (k + 1) * U * (size + 50)
        assert abs((loss(o, g2) - base) / 4.0 - float(out["dgates"][t, j])) <= 8 * (k + 1) * U * (size + 1000)


# ------------------------------------------------------------------ quantisers

def check_elements(got, y, size=None, d=0.0, top=1.0):
    """E4M3 elements against the quotients y (NaN: not looked at).  size: the values' terms in units of y; top: the
    block's largest size over its amax.  A value x is off by at most d size, so a block's amax by d top amax (the maxima of two
    lists differ by no more than their elements do), so 448 x / amax by d (size + |y| top), rounded twice."""
    seen = ~np.isnan(y)
    if d == 0.0:
        assert np.array_equal(got[seen], O.e4m3(y[seen]))
        return
    size = np.abs(y) if size is None else size
    assert (np.abs(got - np.clip(y, -448, 448)) <= O.e4m3_step(y) / 2 + 2 * d * (size + np.abs(y) * top))[seen].all()


def check_scales(got, want, d, top=1.0):
    seen = ~np.isnan(want)
    if d == 0.0:  # amax is exact, the quotient rounded once
        assert np.array_equal(got[seen], want[seen].astype(np.float32).astype(np.float64))
    else:
        assert (np.abs(got - want) <= 2 * d * top * want)[seen].all()


def check_quantized(out, x64, offsets, d=0.0, size=None):
    size = np.abs(x64) if size is None else size
    if "q" in out:
        y, s = O.rows(x64)
        C = y.shape[1]
        top = np.maximum(1.0, O.rows(size)[1] / s)
        each = lambda t: np.repeat(t, 128, 0)[:C].T  # noqa: E731
        check_elements(f64(out["q"]), y, size / each(s), d, each(top))
        check_scales(f64(out["scale"]), s, d, top)
    if "qt" in out:
        y, s = O.columns(x64, offsets)
        top = np.maximum(1.0, O.columns(size, offsets)[1] / s)
        terms = np.zeros(y.shape)
        b = 0
        for e in range(len(offsets) - 1):
            for r in range(offsets[e], offsets[e + 1], 128):
                part = size[r:min(r + 128, offsets[e + 1])]
                terms[:, 128 * b:128 * b + len(part)] = (part / s[b]).T
                b += 1
        check_elements(f64(out["qt"]), y, terms, d, np.repeat(top, 128, 0).T)
        check_scales(f64(out["qt_scale"]), s, d, top)


# (T, k, E, C): a token, odd widths, tails of blocks, many experts with no or few rows, one expert, whole tiles
QUANT = [(1, 1, 1, 1), (3, 2, 5, 7), (50, 3, 8, 130), (33, 4, 300, 264), (20, 6, 48, 1111), (130, 1, 1, 128),
         (257, 2, 2, 384), (5, 8, 1024, 512), (700, 2, 6, 640), (70, 8, 16, 2500)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,k,E,C", QUANT)
def test_quantized_rows_and_columns(T, k, E, C, dtype):
    rng = np.random.default_rng(T + C)
    src, _, offsets = table(rng, T, k, E, skew=1.0)
    x, x64 = values(rng, (T * k, C), dtype)
    d = 0.0 if dtype == BF else 2.0 ** -22
    out = mok.fp8_quantize(x, offsets=cuda(offsets))
    check_quantized(out, x64, offsets, d)
    rows = mok.fp8_quantize(x)                       # the kernel for rows alone
    assert torch.equal(rows["q"].view(torch.uint8), out["q"].view(torch.uint8))
    assert torch.equal(rows["scale"], out["scale"])
    columns = mok.fp8_quantize(x, offsets=cuda(offsets), rows=False)
    assert set(columns) == {"qt", "qt_scale"}
    used = 128 * sum(-(-int(n) // 128) for n in np.diff(offsets))
    assert torch.equal(columns["qt"].view(torch.uint8)[:, :used], out["qt"].view(torch.uint8)[:, :used])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,k,E,C", QUANT[:8])
def test_quantized_gathered_rows(T, k, E, C, gated, dtype):
    rng = np.random.default_rng(T + C)
    src, _, offsets = table(rng, T, k, E, dropped=0.2 if T > 2 else 0.0)
    x, x64 = values(rng, (T, C), dtype)
    g = cuda(rng.random((T, k)) + 0.1, F32) if gated else None
    out = mok.fp8_quantize(x, src_of=cuda(src), k=k, gates=g)
    d = 0.0 if dtype == BF and not gated else 2.0 ** -22
    x64 = O.gather(x64, src, k, None if g is None else f64(g))
    check_quantized(out, x64, offsets, d)
    check_quantized(mok.fp8_quantize(x, src_of=cuda(src), k=k, gates=g, offsets=cuda(offsets), rows=False), x64, offsets, d)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,k,E,C", [s for s in QUANT if s[3] > 1])
def test_quantized_swiglu_and_its_gradient(T, k, E, C, dtype):
    rng = np.random.default_rng(T + C)
    _, _, offsets = table(rng, T, k, E)
    hu, hu64 = values(rng, (T * k, 2 * C), dtype, spread=1.0)
    a, size = O.swiglu(hu64)
    check_quantized(mok.fp8_quantize(hu, source="swiglu", offsets=cuda(offsets)), a, offsets, 2.0 ** -19, size)
    check_quantized(mok.fp8_quantize(hu, source="swiglu"), a, offsets, 2.0 ** -19, size)
    da, da64 = values(rng, (T * k, C), dtype)
    g, size = O.swiglu_grad(hu64, da64)
    out = mok.fp8_quantize(hu, source="swiglu_grad", grad=da, offsets=cuda(offsets))
    check_quantized(out, g, offsets, 2.0 ** -19, size)
    check_quantized(mok.fp8_quantize(hu, source="swiglu_grad", grad=da), g, offsets, 2.0 ** -19, size)


# rows, width of u: pairs of column blocks, aligned rows, odd widths, few rows and as many as take the larger tiles
WIDTHS = [(300, 512), (140, 264), (70, 7), (130, 1111), (5000, 512), (2400, 1111)]


def per_row(rng, R, choices):
    return rng.choice(choices, (R, 1)) * rng.choice([-1.0, 1.0], (R, 1))


def check_swiglu(hu64, da64, dtype, offsets):
    """The SwiGLU and its gradient of these values, along the rows alone and in both layouts."""
    hu, da = torch.tensor(hu64).to(dtype).cuda(), torch.tensor(da64).to(dtype).cuda()
    off = cuda(offsets)
    a, size = O.swiglu(f64(hu))
    g, terms = O.swiglu_grad(f64(hu), f64(da))
    for kw in (dict(), dict(offsets=off)):
        check_quantized(mok.fp8_quantize(hu, source="swiglu", **kw), a, offsets, 2.0 ** -19, size)
        check_quantized(mok.fp8_quantize(hu, source="swiglu_grad", grad=da, **kw), g, offsets, 2.0 ** -19, terms)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("R,C", WIDTHS)
def test_swiglu_far_below_zero(R, C, dtype):
    """h where e^h is smaller than f32's normal values, down to the type's lowest, in rows of nothing else and among others.
    (The part of the sigmoid below e^-40 is an exponential of its own: two more roundings than counted at the top, in 2^-19.)"""
    rng = np.random.default_rng(R + C)
    far = rng.choice([-86.5, -87.5, -88.0, -90.0, -100.0, -104.0, -150.0, -1e4, -1e30, float(torch.finfo(dtype).min)], (R, C))
    often = np.where(np.arange(R)[:, None] % 3 == 0, 1.0, 0.2)
    h = np.where(rng.random((R, C)) < often, far, 2.0 * rng.normal(size=(R, C)))
    u = rng.normal(size=(R, C)) * per_row(rng, R, [1.0, 1e3, 1e6, 1e30])
    da = rng.normal(size=(R, C)) * per_row(rng, R, [1e-3, 1.0, 1e4])
    check_swiglu(np.concatenate([h, u], 1), da, dtype, np.array([0, R // 3, R // 3, R], np.int32))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("R,C", WIDTHS[:4])
def test_swiglu_gradient_whose_parts_leave_the_range(R, C, dtype):
    """da u, da h and da s out of f32's range where the gradient is not; h and u both at the type's lowest."""
    rng = np.random.default_rng(R)
    h = -45 - 30 * rng.random((R, C))
    size = rng.choice([(1e25, 1e25), (1.0, 1e36), (1e-10, 1e36), (1e25, 1e-10)], R)
    u, da = rng.normal(size=(R, C)) * size[:, :1], rng.normal(size=(R, C)) * size[:, 1:]
    h[::5] = u[::5] = float(torch.finfo(dtype).min)
    check_swiglu(np.concatenate([h, u], 1), da, dtype, np.array([0, R // 2, R], np.int32))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_swiglu_of_minus_infinity(dtype):
    """-inf e^-inf has no value: a NaN, out of its block's scale."""
    hu = torch.ones(3, 512, dtype=dtype).cuda()
    hu[1, 3] = float("-inf")
    da = torch.ones(3, 256, dtype=dtype).cuda()
    q, g = mok.fp8_quantize(hu, source="swiglu"), mok.fp8_quantize(hu, source="swiglu_grad", grad=da)
    for out, places in ((q, [3]), (g, [3, 259])):
        nan = torch.isnan(out["q"].float())
        assert nan[1, places].all() and int(nan.sum()) == len(places)
        assert torch.equal(out["scale"][:, 1], out["scale"][:, 0])


def test_the_oracles_swiglu_gradient_by_differences():
    rng = np.random.default_rng(1)
    x, da = rng.normal(size=(3, 10)), rng.normal(size=(3, 5))
    g, _ = O.swiglu_grad(x, da)
    for i in range(3):
        for j in range(10):
            hi, lo = x.copy(), x.copy()
            hi[i, j] += 1e-5
            lo[i, j] -= 1e-5
            d = ((O.swiglu(hi)[0] - O.swiglu(lo)[0]) * da).sum() / 2e-5
            assert abs(d - g[i, j]) < 1e-8


@pytest.mark.parametrize("extra", [1, 3, 8])
def test_quantized_rows_further_apart(extra):
    rng = np.random.default_rng(extra)
    offsets = cuda(np.array([0, 50, 50, 177], np.int32))
    x, _ = values(rng, (177, 264), BF)
    hu, _ = values(rng, (177, 528), BF)
    for kw in (dict(), dict(source="swiglu"), dict(source="swiglu_grad", grad=hu[:, :132].contiguous())):
        t = hu if kw.get("source") == "swiglu" else x
        want = mok.fp8_quantize(t, offsets=offsets, **kw)
        out = {n: wide(v, extra, 16 if n in ("q", "qt") else 1) for n, v in want.items() if n != "qt_scale"}
        before = {n: v.clone() for n, v in out.items()}
        for v in out.values():
            v.view(torch.uint8 if v.element_size() == 1 else torch.int32).zero_()
        out["qt_scale"] = torch.empty_like(want["qt_scale"])
        if "grad" in kw:
            kw = dict(kw, grad=wide(kw["grad"], extra))
        mok.fp8_quantize(wide(t, extra), offsets=offsets, out=out, **kw)
        for n in ("q", "scale"):
            assert torch.equal(out[n].float(), before[n].float()), n
            assert torch.equal(out[n].float(), want[n].float()), n
            ld, (rows, width) = out[n].stride(0), out[n].shape
            assert (torch.as_strided(out[n], (rows - 1, ld - width), (ld, 1), width).float() == 3.0).all()
        assert torch.equal(out["qt"].float()[:, :256], want["qt"].float()[:, :256])   # two blocks of rows


def test_what_is_not_finite_stays_an_element():
    """NaN and infinities become NaN; the rest of the block is as if they were zero."""
    rng = np.random.default_rng(5)
    offsets = cuda(np.array([0, 256], np.int32))
    for dtype in (BF, F32):
        x, _ = values(rng, (256, 256), dtype)
        bad = x.clone()
        places = [(3, 5, float("nan")), (3, 200, float("inf")), (130, 0, float("-inf")), (255, 255, float("nan"))]
        clean = x.clone()
        for r, c, v in places:
            bad[r, c] = v
            clean[r, c] = 0.0
        got, want = mok.fp8_quantize(bad, offsets=offsets), mok.fp8_quantize(clean, offsets=offsets)
        for out in (got, want):   # two of three blocks of rows are used
            out["qt"], out["qt_scale"] = out["qt"][:, :256], out["qt_scale"][:2]
        for n in ("scale", "qt_scale"):
            assert torch.equal(got[n], want[n])
        for n in ("q", "qt"):
            g, w = got[n].float(), want[n].float()
            for r, c, _ in places:
                assert torch.isnan(g[(r, c) if n == "q" else (c, r)])
                g[(r, c) if n == "q" else (c, r)] = 0.0
            assert torch.equal(g, w)
        w = mok.Fp8Weights(bad, transposed=True)
        v = mok.Fp8Weights(clean, transposed=True)
        assert torch.equal(w.scale, v.scale) and int(torch.isnan(w.q.float()).sum()) == 4
        assert torch.equal(torch.nan_to_num(w.q.float()), v.q.float())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("R,C", [(10_000, 384), (10_001, 376)])
def test_what_is_not_finite_in_many_rows(R, C, dtype):
    """As above in as many rows as take the larger tiles: along the rows alone and in both layouts."""
    rng = np.random.default_rng(6)
    x, _ = values(rng, (R, C), dtype)
    bad, clean = x.clone(), x.clone()
    rows = rng.integers(0, R, 500)
    cols = rng.integers(0, C, 500)
    for i, v in enumerate((float("nan"), float("inf"), float("-inf"), -float("nan"))):
        bad[cuda(rows[i::4]), cuda(cols[i::4])] = v
    places = ~torch.isfinite(bad)
    clean[places] = 0.0
    offsets = cuda(np.array([0, 1, 1, 5_000, R], np.int32))
    got, want = mok.fp8_quantize(bad), mok.fp8_quantize(clean)
    both = mok.fp8_quantize(bad, offsets=offsets)
    assert torch.equal(got["scale"], want["scale"]) and torch.equal(both["scale"], want["scale"])
    for q in (got["q"], both["q"]):
        assert torch.equal(torch.isnan(q.float()), places)
        assert torch.equal(torch.nan_to_num(q.float()), want["q"].float())


def test_the_ends_of_the_range():
    """Blocks of zeros, of the type's smallest and largest values."""
    for dtype in (BF, F32):
        for v in (0.0, 2.0 ** -133, 2.0 ** -126, 2.0 ** -111, 2.0 ** -110, 1.0, 2.0 ** 100, float(torch.finfo(dtype).max)):
            x = torch.zeros(2, 128, dtype=dtype).cuda()
            x[1] = v
            x[1, 1] = -v
            x[1, 2] = v / 2
            out = mok.fp8_quantize(x)
            y, s = O.rows(f64(x))
            check_elements(f64(out["q"]), y)
            check_scales(f64(out["scale"]), s, 0.0)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("E,N,K", [(1, 1, 1), (2, 7, 300), (3, 130, 36), (1, 256, 384), (5, 200, 129), (2, 1000, 264)])
def test_quantized_weights(E, N, K, dtype):
    rng = np.random.default_rng(N)
    w, w64 = values(rng, (E, N, K), dtype)
    d = 0.0 if dtype == BF else 2.0 ** -22
    got = mok.Fp8Weights(w, transposed=True)
    y, s = O.weights(w64)
    check_elements(f64(got.q), y, None, d)
    check_scales(f64(got.scale), s, d)
    assert torch.equal(got.qt.float(), got.q.float().transpose(1, 2))
    assert torch.equal(got.qt_scale, got.scale.transpose(1, 2))
    plain = mok.Fp8Weights(w)
    assert plain.qt is None and torch.equal(plain.q.float(), got.q.float()) and torch.equal(plain.scale, got.scale)
    if E == 1:
        flat = mok.Fp8Weights(w[0])
        assert torch.equal(flat.q.float(), got.q.float())


# ------------------------------------------------------------------ products

def random_e4m3(rng, shape):
    t = mok.empty_e4m3(*shape)
    t.view(torch.uint8).copy_(torch.tensor(np.clip(rng.normal(size=shape) * 150, -448, 448)).to(torch.float8_e4m3fn)
                              .view(torch.uint8))
    return t


def scales(rng, shape, size=0.01):
    return cuda(np.exp(rng.normal(size=shape)) * size, F32)


def check_product(got, want, size, K, dtype):
    blocks = -(-K // 128)
    seen = ~np.isnan(want)
    assert (np.abs(got - want) <= (132 + blocks) * 2 * U * size + HALF[dtype] * np.abs(want))[seen].all()


# (rows of each group, N, K): a row, odd sizes, tails of 128 along N and K, empty groups, groups on both sides of every
# rule on sizes, rows behind the last group
PRODUCTS = [([1], 1, 1), ([3], 7, 16), ([1, 0, 2], 130, 300), ([8, 9, 0, 7], 100, 128), ([17, 30, 5], 264, 1111),
            ([40], 513, 640), ([0, 0, 70, 1], 384, 257), ([129], 256, 512), ([300, 0, 5, 64], 500, 384), ([1] * 40, 48, 200),
            ([513, 250], 260, 900), ([0, 0], 16, 16), ([33] * 5, 1024, 128), ([700], 250, 2000), ([5, 0, 90], 64, 4100),
            ([250], 96, 2200), ([100], 1000, 6000)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("counts,N,K", PRODUCTS, ids=lambda v: str(v)[:24])
def test_product(counts, N, K, dtype):
    rng = np.random.default_rng(sum(counts) + N)
    E, behind = len(counts), 5
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    R = int(offsets[-1]) + behind
    x, xs = random_e4m3(rng, (R, K)), scales(rng, (-(-K // 128), R))
    w, ws = random_e4m3(rng, (E, N, K)), scales(rng, (E, -(-N // 128), -(-K // 128)))
    want, size = O.product(f64(x), f64(xs), f64(w), f64(ws), offsets)
    weights = mok.Fp8Weights.of(w, ws)
    out = torch.full((R, N), 7.0, dtype=dtype).cuda()
    got = f64(weights.matmul(x, xs, cuda(offsets), out=out))
    check_product(got, want, size, K, dtype)
    assert (got[R - behind:] == 7.0).all()
    assert weights.status() == (0, 0)
    # rows further apart, and the same bits
    out2 = wide(torch.zeros(R, N, dtype=dtype).cuda(), 3)
    weights.matmul(wide(x, 16, 16), wide(xs, 1), cuda(offsets), out=out2)
    assert torch.equal(out2[:R - behind], out[:R - behind]) and (out2[R - behind:] == 0).all()
    assert (torch.as_strided(out2, (R - 1, 3), (N + 3, 1), N) == 3.0).all()


# counts, N, K: tiles of every width (16 to 256 columns, some of them with splits), f32's packed sums too
SCALED = [([1], 130, 300), ([70, 0, 5], 264, 1111), ([129], 256, 512), ([513, 250], 260, 900), ([33] * 5, 1024, 200),
          ([40], 130, 6000), ([1000], 384, 1500)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("counts,N,K", SCALED, ids=lambda v: str(v)[:24])
def test_product_of_scales_out_of_range(counts, N, K, dtype):
    """A row's scale times a weights' one beyond f32's normal range on either side, beside rows where it is not.  Where the scales
    meet apart, two of the three roundings at the top are of numbers that may be subnormal: off by 2^-150 each and block;
    out's own rounding by half its smallest number."""
    rng = np.random.default_rng(sum(counts) + K)
    E, R = len(counts), sum(counts)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    blocks = -(-K // 128)
    x, w = random_e4m3(rng, (R, K)), random_e4m3(rng, (E, N, K))
    kind = rng.integers(0, 5, R)       # ordinary rows, blocks of nearly nothing, small rows, rows of zeros, smallest elements
    size = np.array([1.0, 2.0 ** -112, 2.0 ** -92, 2.0 ** 115, 2.0 ** 109])[kind]
    kind[0], size[0] = 4, 2.0 ** 109
    each = scales(rng, (blocks, R))
    xs = each * cuda(size, F32)
    zeros, least = cuda(np.nonzero(kind == 3)[0]), cuda(np.nonzero(kind == 4)[0])
    x.view(torch.uint8)[zeros] = 0
    x.view(torch.uint8)[least] &= 0x81  # zeros, and elements of 2^-9
    small = rng.integers(0, 3, (E, -(-N // 128), blocks))
    ws = scales(rng, small.shape) * cuda(np.array([1.0, 2.0 ** -32, 2.0 ** 32])[small], F32)
    # large scales have small elements: below 2^-3
    large = np.repeat(np.repeat(small == 2, 128, 1), 128, 2)[:, :N, :K]
    w.view(torch.uint8)[cuda(large)] &= 0x9f
    want, terms = O.product(f64(x), f64(xs), f64(w), f64(ws), offsets)
    assert (np.abs(want)[kind != 4] < 3e38).all()
    weights = mok.Fp8Weights.of(w, ws)
    got = f64(weights.matmul(x, xs, cuda(offsets), dtype=dtype))
    tiny = (2 * blocks + 1) * 2.0 ** -150 + (2.0 ** -134 if dtype == BF else 2.0 ** -150)
    fits = np.abs(terms) < 3e38
    bound = (132 + blocks) * 2 * U * terms + HALF[dtype] * np.abs(want) + tiny
    assert fits[kind == 4].any() and (np.abs(got - want) <= bound)[fits].all()
    assert weights.status() == (0, 0)
    # an ordinary row has the same bits whatever its neighbours are
    assert np.array_equal(f64(weights.matmul(x, each, cuda(offsets), dtype=dtype))[kind == 0], got[kind == 0])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("counts,N,K", SCALED, ids=lambda v: str(v)[:24])
def test_product_of_least_scales(counts, N, K, dtype):
    """Rows and weights at the quantisers' least scale, or at 0: their factors may be subnormal, off by 2^-150 and a block's sum by
    that times 128 x 448^2 < 2^24.7."""
    rng = np.random.default_rng(sum(counts) + N)
    E, R = len(counts), sum(counts)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    blocks = -(-K // 128)
    least = float(np.float32(2.0 ** -110 / 448))
    pick = lambda t: torch.where(cuda(rng.random(t.shape) < 0.3), cuda(rng.choice([least, 0.0], t.shape), F32), t)  # noqa: E731
    x, xs = random_e4m3(rng, (R, K)), pick(scales(rng, (blocks, R)))
    w, ws = random_e4m3(rng, (E, N, K)), pick(scales(rng, (E, -(-N // 128), blocks)))
    xs[:, -1] = least
    want, terms = O.product(f64(x), f64(xs), f64(w), f64(ws), offsets)
    got = f64(mok.Fp8Weights.of(w, ws).matmul(x, xs, cuda(offsets), dtype=dtype))
    bound = (132 + blocks) * 2 * U * terms + HALF[dtype] * np.abs(want) + blocks * 2.0 ** -125
    assert (np.abs(got - want) <= bound).all()
    zeros = torch.zeros(R, K, device="cuda")
    q = mok.fp8_quantize(zeros)
    assert (q["scale"] == least).all()
    assert (mok.Fp8Weights.of(w, ws).matmul(q["q"], q["scale"], cuda(offsets), dtype=dtype) == 0).all()


@pytest.mark.parametrize("R,N,K", [(1, 64, 256), (5, 1000, 100), (16, 256, 2048), (100, 130, 384), (257, 700, 1300), (1, 520, 7168), (64, 260, 4100),
                                   (200, 96, 3000)])
def test_product_without_groups(R, N, K):
    rng = np.random.default_rng(R)
    w, _ = values(rng, (N, K), BF)
    x, _ = values(rng, (R, K), BF)
    dy, _ = values(rng, (R, N), BF)
    weights = mok.Fp8Weights(w, transposed=True)
    xq, dyq = mok.fp8_quantize(x), mok.fp8_quantize(dy)
    got = weights.matmul(xq["q"], xq["scale"], dtype=F32)
    want, size = O.product(f64(xq["q"]), f64(xq["scale"]), f64(weights.q), f64(weights.scale), [0, R])
    check_product(f64(got), want, size, K, F32)
    got = weights.matmul_transposed(dyq["q"], dyq["scale"], dtype=F32)
    want, size = O.product(f64(dyq["q"]), f64(dyq["scale"]), f64(weights.q).transpose(0, 2, 1),
                           f64(weights.scale).transpose(0, 2, 1), [0, R])
    check_product(f64(got), want, size, N, F32)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("counts,N,H", [([1], 1, 1), ([3, 0, 130], 7, 300), ([128, 256], 129, 64), ([0, 0, 0], 33, 65),
                                        ([1] * 30, 40, 24), ([300, 1, 513], 256, 260), ([700], 513, 640),
                                        ([64] * 8, 520, 256), ([2100], 70, 100), ([1100, 1200], 40, 64)],
                         ids=lambda v: str(v)[:24])
def test_weight_grad(counts, N, H, dtype):
    rng = np.random.default_rng(sum(counts) + N)
    E = len(counts)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    R = int(offsets[-1])
    dy, _ = values(rng, (R + 3, N), BF)
    x, _ = values(rng, (R + 3, H), BF)
    a = mok.fp8_quantize(dy, offsets=cuda(offsets), rows=False)
    b = mok.fp8_quantize(x, offsets=cuda(offsets), rows=False)
    got = mok.fp8_weight_grad(a["qt"], a["qt_scale"], b["qt"], b["qt_scale"], cuda(offsets), dtype=dtype)
    want, size = O.weight_grad(f64(a["qt"]), f64(a["qt_scale"]), f64(b["qt"]), f64(b["qt_scale"]), offsets)
    check_product(f64(got), want, size, max(counts + [1]), dtype)


def test_bad_offsets_stay_in_the_tensors():
    """Offsets out of range or out of order: nothing outside the tensors is touched; ends behind R count as R."""
    rng = np.random.default_rng(8)
    R, N, K, E = 100, 70, 200, 4
    x, xs = random_e4m3(rng, (R, K)), scales(rng, (2, R))
    w, ws = random_e4m3(rng, (E, N, K)), scales(rng, (E, 1, 2))
    weights = mok.Fp8Weights.of(w, ws)
    for bad, good in (([0, 30, 20, 60, 2 ** 31 - 1], None), ([-5, 10, 2 ** 30, 2 ** 30, 100], None),
                      ([-2 ** 31, 0, 0, 0, 500], [0, 0, 0, 0, 100])):
        out = torch.full((R, N), 7.0).cuda()
        weights.matmul(x, xs, cuda(np.array(bad, np.int32)), out=out)
        if good:
            want, size = O.product(f64(x), f64(xs), f64(w), f64(ws), good)
            check_product(f64(out), want, size, K, F32)
        q = mok.fp8_quantize(out, offsets=cuda(np.array(bad, np.int32)))
        mok.fp8_weight_grad(q["qt"], q["qt_scale"], q["qt"], q["qt_scale"], cuda(np.array(bad, np.int32)))
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("counts", [[300], [1000, 40], [60, 0, 129]], ids=str)
def test_weight_grad_of_rows_at_the_types_lowest(counts, dtype):
    """x holds masks' lowest values, dy what gradients are: the products lie within f32."""
    rng = np.random.default_rng(sum(counts))
    N, H = 130, 200
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    R = int(offsets[-1])
    dy, x = values(rng, (R, N), BF)[0] * 2.0 ** -20, values(rng, (R, H), BF)[0]
    x[cuda(rng.integers(0, R, 40)), cuda(rng.integers(0, H, 40))] = float(torch.finfo(BF).min)
    a = mok.fp8_quantize(dy, offsets=cuda(offsets), rows=False)
    b = mok.fp8_quantize(x, offsets=cuda(offsets), rows=False)
    want, size = O.weight_grad(f64(a["qt"]), f64(a["qt_scale"]), f64(b["qt"]), f64(b["qt_scale"]), offsets)
    assert size.max() < 3e38
    got = mok.fp8_weight_grad(a["qt"], a["qt_scale"], b["qt"], b["qt_scale"], cuda(offsets), dtype=dtype)
    check_product(f64(got), want, size, max(counts), dtype)


class Fenced:
    """A [rows][width] tensor inside of a larger buffer: bytes of 0x5a in front, behind and between the rows."""

    def __init__(self, shape, dtype, between=0):
        rows, width = shape
        item = torch.empty(0, dtype=dtype).element_size()
        ld = -(-width * item // 16) * 16 + between if between else width * item
        self.big = torch.full((4096 + rows * ld + 4096,), 0x5a, dtype=torch.uint8).cuda()
        inside = torch.as_strided(self.big, (rows, width * item), (ld, 1), 4096)
        self.t = torch.as_strided(self.big.view(dtype), (rows, width), (ld // item, 1), 4096 // item)
        self.mask = torch.ones_like(self.big, dtype=torch.bool)
        torch.as_strided(self.mask, inside.shape, inside.stride(), 4096).fill_(False)

    def intact(self):
        return bool((self.big[self.mask] == 0x5a).all())


BAD_TABLES = [[0, 30, 20, 60, 2 ** 31 - 1], [-5, 10, 2 ** 30, 2 ** 30, 100], [-2 ** 31, 0, 0, 0, 500], [100, 0, 100, 0, 100],
              [0, 400, 0, 400, 0], [300, 200, 100, 0, -100], [2 ** 31 - 1] * 5, [-1] * 5, [0, 299, 1, 299, 299]]


@pytest.mark.parametrize("bad", BAD_TABLES, ids=str)
def test_bad_offsets_write_nothing_beside_the_outputs(bad):
    """As above for the outputs: what lies in front of them, behind them and between their rows stays as it was."""
    rng = np.random.default_rng(8)
    R, N, K, E = 300, 70, 200, 4
    offsets = cuda(np.array(bad, np.int32))
    x, xs = random_e4m3(rng, (R, K)), scales(rng, (2, R))
    weights = mok.Fp8Weights.of(random_e4m3(rng, (E, N, K)), scales(rng, (E, 1, 2)))
    P = mok.fp8_columns(R, E)
    fences = []

    def fenced(*a, **kw):
        fences.append(Fenced(*a, **kw))
        return fences[-1].t

    for dtype in (BF, F32):
        weights.matmul(x, xs, offsets, out=fenced((R, N), dtype, between=32))
        for source, width in (("plain", N), ("swiglu", 2 * N), ("swiglu_grad", N), ("swiglu_grad", 512)):
            C = width // 2 if source == "swiglu" else width
            src, _ = values(rng, (R, width), dtype)
            grad = values(rng, (R, C // 2), dtype)[0] if source == "swiglu_grad" else None
            out = {"q": fenced((R, C), X.E4M3, between=16), "scale": fenced((-(-C // 128), R), F32, between=16),
                   "qt": fenced((C, P), X.E4M3, between=16), "qt_scale": fenced((P // 128, C), F32)}
            mok.fp8_quantize(src, source=source, grad=grad, offsets=offsets, out=out)
        good = mok.fp8_quantize(src, offsets=cuda(np.array([0, 100, 100, 200, R], np.int32)), rows=False)
        dw = fenced((E * 512, 512), dtype)
        mok.fp8_weight_grad(good["qt"], good["qt_scale"], good["qt"], good["qt_scale"], offsets, out=dw.view(E, 512, 512))
    assert all(f.intact() for f in fences) and weights.status() == (0, 0) == mok.fp8_status()


def test_as_many_groups_as_there_may_be():
    rng = np.random.default_rng(12)
    E, N, K = 1024, 40, 150
    counts = rng.integers(0, 4, E)
    counts[[3, 500, 1023]] = 130, 0, 77
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    R = int(offsets[-1])
    x, _ = values(rng, (R, K), BF)
    dy, _ = values(rng, (R, N), BF)
    w = mok.Fp8Weights(values(rng, (E, N, K), BF)[0])
    q, d = mok.fp8_quantize(x, offsets=cuda(offsets)), mok.fp8_quantize(dy, offsets=cuda(offsets), rows=False)
    got = w.matmul(q["q"], q["scale"], cuda(offsets), dtype=F32)
    want, size = O.product(f64(q["q"]), f64(q["scale"]), f64(w.q), f64(w.scale), offsets)
    check_product(f64(got), want, size, K, F32)
    got = mok.fp8_weight_grad(d["qt"], d["qt_scale"], q["qt"], q["qt_scale"], cuda(offsets))
    want, size = O.weight_grad(f64(d["qt"]), f64(d["qt_scale"]), f64(q["qt"]), f64(q["qt_scale"]), offsets)
    check_product(f64(got), want, size, int(counts.max()), F32)
    with pytest.raises(mok.MokError):
        mok.Fp8Weights.empty(1025, 16, 16).matmul(mok.empty_e4m3(1, 16), torch.zeros(1, 1).cuda(),
                                                  torch.zeros(1026, dtype=torch.int32).cuda())


@pytest.mark.slow
def test_elements_behind_the_reach_of_32_bits():
    """Tensors of more than 2^31 elements: the last rows against calls on those rows alone."""
    R, H, tail = 540_000, 4096, 300
    x = torch.empty(R, H, dtype=BF, device="cuda").normal_()
    back = torch.arange(R - 1, -1, -1, dtype=torch.int32, device="cuda")
    g = mok.gather_rows(x, back, 1)
    assert torch.equal(g[-5:], x[:5].flip(0)) and torch.equal(g[:5], x[-5:].flip(0))
    gates = torch.rand(R, 1, device="cuda")
    y = mok.merge_rows(g, back, 1, gates)
    assert torch.equal(y[-tail:], (x[-tail:].float() * gates[-tail:]).bfloat16())
    out = mok.merge_rows_backward(x, g, back, gates)
    assert torch.equal(out["do"][:tail], (x[-tail:].float() * gates[-tail:]).bfloat16().flip(0))
    dots = (x[-tail:].double() ** 2).sum(1)
    assert ((out["dgates"][-tail:, 0].double() - dots).abs() <= (H / 32 + 29) * U * dots).all()
    del g, y, out
    first = R - tail
    offsets = torch.tensor([0, 100, first, R], dtype=torch.int32, device="cuda")
    q = mok.fp8_quantize(x, offsets=offsets)
    alone = mok.fp8_quantize(x[-tail:], offsets=torch.tensor([0, tail], dtype=torch.int32, device="cuda"))
    assert torch.equal(q["q"][-tail:].view(torch.uint8), alone["q"].view(torch.uint8))
    assert torch.equal(q["scale"][:, -tail:], alone["scale"])
    block = 1 + -(-(first - 100) // 128)
    assert torch.equal(q["qt"][:, 128 * block:128 * (block + 3)].view(torch.uint8), alone["qt"][:, :384].view(torch.uint8))
    assert torch.equal(q["qt_scale"][block:block + 3], alone["qt_scale"][:3])
    del x
    w = mok.Fp8Weights(torch.randn(3, H, 256, device="cuda"))
    few = {n: (t[:, :256] if n == "q" else t[:2]) for n, t in q.items() if n in ("q", "scale")}
    out = w.matmul(few["q"], few["scale"], offsets)
    want, size = O.product(f64(few["q"][-tail:]), f64(few["scale"][:, -tail:]), f64(w.q[2:]), f64(w.scale[2:]), [0, tail])
    check_product(f64(out[-tail:]), want, size, 256, BF)
    del out
    E = 140
    some = (torch.arange(E + 1, device="cuda") * 3).int()
    a = mok.fp8_quantize(torch.randn(3 * E, H, device="cuda"), offsets=some, rows=False)
    out = mok.fp8_weight_grad(a["qt"], a["qt_scale"], a["qt"], a["qt_scale"], some, dtype=BF)
    p = f64(a["qt"][:, 128 * (E - 1):128 * E]) * f64(a["qt_scale"][E - 1])[:, None]
    check_product(f64(out[-1]), p @ p.T, np.abs(p) @ np.abs(p).T, 3, BF)


def test_an_experts_training_step_together():
    """Both products, their gradients and the way of the rows, each against the oracle on the operands that the call
    before it made, the last ones against the unquantised layer too."""
    rng = np.random.default_rng(11)
    T, k, E, H, I = 60, 3, 6, 256, 384
    src, row, offsets = table(rng, T, k, E, skew=0.7)
    x, x64 = values(rng, (T, H), BF)
    dy, dy64 = values(rng, (T, H), BF)
    w13, w13_64 = values(rng, (E, 2 * I, H), BF)
    w2, w2_64 = values(rng, (E, H, I), BF)
    w13, w2 = w13 / 16, w2 / 16
    w13_64, w2_64 = w13_64 / 16, w2_64 / 16
    g = cuda(rng.random((T, k)), F32)
    off, src_of, row_of = cuda(offsets), cuda(src), cuda(row)
    W13, W2 = mok.Fp8Weights(w13, transposed=True), mok.Fp8Weights(w2, transposed=True)
    xq = mok.fp8_quantize(x, src_of=src_of, k=k, offsets=off)
    hu = W13.matmul(xq["q"], xq["scale"], off)
    aq = mok.fp8_quantize(hu, source="swiglu", offsets=off)
    o = W2.matmul(aq["q"], aq["scale"], off)
    y = mok.merge_rows(o, row_of, k, g)
    back = mok.merge_rows_backward(dy, o, row_of, g)
    doq = mok.fp8_quantize(back["do"], offsets=off)
    da = W2.matmul_transposed(doq["q"], doq["scale"], off)
    dhuq = mok.fp8_quantize(hu, source="swiglu_grad", grad=da, offsets=off)
    dx = mok.merge_rows(W13.matmul_transposed(dhuq["q"], dhuq["scale"], off), row_of, k)
    dw2 = mok.fp8_weight_grad(doq["qt"], doq["qt_scale"], aq["qt"], aq["qt_scale"], off)
    dw13 = mok.fp8_weight_grad(dhuq["qt"], dhuq["qt_scale"], xq["qt"], xq["qt_scale"], off)
    # stage by stage
    check_quantized(xq, O.gather(x64, src, k), offsets)
    for got, q, w, ws, K in ((hu, xq, W13.q, W13.scale, H), (o, aq, W2.q, W2.scale, I), (da, doq, W2.qt, W2.qt_scale, H)):
        want, size = O.product(f64(q["q"]), f64(q["scale"]), f64(w), f64(ws), offsets)
        check_product(f64(got), want, size, K, BF)
    a, size = O.swiglu(f64(hu))
    check_quantized(aq, a, offsets, 2.0 ** -19, size)
    check_quantized(doq, f64(back["do"]), offsets)
    grad, size = O.swiglu_grad(f64(hu), f64(da))
    check_quantized(dhuq, grad, offsets, 2.0 ** -19, size)
    for got, p, q in ((dw2, doq, aq), (dw13, dhuq, xq)):
        want, size = O.weight_grad(f64(p["qt"]), f64(p["qt_scale"]), f64(q["qt"]), f64(q["qt_scale"]), offsets)
        check_product(f64(got), want, size, int(np.diff(offsets).max()), F32)
    # the whole of it, unquantised: an E4M3 rounding is off by at most 2^-4 of an element, on average by 2^-5.8; a product
    # of two such operands by about 2^-5.3 of its root of squares, and four of them follow each other here
    x_g = O.gather(x64, src, k)
    hu64, do64 = np.zeros((T * k, 2 * I)), O.gather(dy64, src, k, f64(g))
    o64, dx_g, dw13_64, dw2_64 = np.zeros((T * k, H)), np.zeros((T * k, H)), np.zeros((E, 2 * I, H)), np.zeros((E, H, I))
    for e in range(E):
        c = slice(offsets[e], offsets[e + 1])
        hu64[c] = x_g[c] @ w13_64[e].T
        a64 = O.swiglu(hu64[c])[0]
        o64[c] = a64 @ w2_64[e].T
        dhu64 = O.swiglu_grad(hu64[c], do64[c] @ w2_64[e])[0]
        dx_g[c] = dhu64 @ w13_64[e]
        dw13_64[e], dw2_64[e] = dhu64.T @ x_g[c], do64[c].T @ a64
    for got, want in ((y, O.merge(o64, row, k, f64(g))[0]), (dx, O.merge(dx_g, row, k)[0]), (dw13, dw13_64), (dw2, dw2_64),
                      (back["dgates"], O.merge_backward(dy64, o64, row, f64(g))[1])):
        assert np.linalg.norm(f64(got) - want) <= 4 * 2.0 ** -4 * np.linalg.norm(want)


def test_the_schedule_tables_rows():
    """src_of, row_of and offsets of mok_schedule as they are."""
    from mixture_experts_layer_table_gb300 import _native as N
    T, E, k, H = 64, 8, 2, 256
    desc = mok.make_desc(T, H, 128, E, k, 1, True)
    i32 = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")  # noqa: E731
    x = torch.randn(T, H, device="cuda").bfloat16()
    topk, counts, offsets, row_of, src_of = i32(T, k), i32(E), i32(E + 1), i32(T * k), i32(T * k)
    gates, ws = torch.empty(T, k, device="cuda"), torch.zeros(N.workspace_size(desc)[0], dtype=torch.uint8, device="cuda")
    mok.schedule(desc, x, torch.randn(E, H, device="cuda").bfloat16(), None, None, topk, gates, counts, offsets, row_of,
                 src_of, ws)
    x_g = mok.gather_rows(x, src_of, k)
    assert torch.equal(x_g, x[src_of.long() // k])
    y = mok.merge_rows(x_g, row_of, k)
    assert torch.equal(y.float(), (x.float() * 2))
    w = mok.Fp8Weights(torch.randn(E, 128, H, device="cuda") * 0.05)
    q = mok.fp8_quantize(x, src_of=src_of, k=k)
    out = w.matmul(q["q"], q["scale"], offsets, dtype=F32)
    want, size = O.product(f64(q["q"]), f64(q["scale"]), f64(w.q), f64(w.scale), offsets.tolist())
    check_product(f64(out), want, size, H, F32)


def test_captured_and_on_another_stream():
    """The calls captured into a graph and replayed on new inputs, and on a stream that is not the current one."""
    rng = np.random.default_rng(2)
    T, k, E, H, N = 100, 2, 4, 256, 300
    src, row, offsets = table(rng, T, k, E)
    src_of, row_of, off = cuda(src), cuda(row), cuda(offsets)
    x, _ = values(rng, (T, H), BF)
    w = mok.Fp8Weights(values(rng, (E, N, H), BF)[0], transposed=True)
    g = cuda(rng.random((T, k)), F32)

    def step(x, stream=None):
        q = mok.fp8_quantize(x, src_of=src_of, k=k, offsets=off, stream=stream)
        o = w.matmul(q["q"], q["scale"], off, stream=stream)
        y = mok.merge_rows(o, row_of, k, g, stream=stream)
        b = mok.merge_rows_backward(y, o, row_of, g, stream=stream)
        d = mok.fp8_quantize(b["do"], offsets=off, stream=stream)
        dx = w.matmul_transposed(d["q"], d["scale"], off, stream=stream)
        return y, b["dgates"], dx, mok.fp8_weight_grad(d["qt"], d["qt_scale"], q["qt"], q["qt_scale"], off, stream=stream)

    step(x)
    static = x.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(static)
    for seed in range(3):
        new, _ = values(np.random.default_rng(seed), (T, H), BF)
        static.copy_(new)
        graph.replay()
        for a, b in zip(captured, step(new)):
            assert torch.equal(a, b)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):   # the allocations belong to it, the calls name it
        other = step(x, stream=side)
    side.synchronize()
    for a, b in zip(other, step(x)):
        assert torch.equal(a, b)


def test_buffers_made_for_another_stream():
    """Calls without buffers on a stream that is not the current one, given as such and by its handle, while the current
    stream is busy and has still to write memory that its allocator has taken back."""
    rng = np.random.default_rng(9)
    T, k, E, H, N = 90, 3, 4, 256, 272
    src, row, offsets = table(rng, T, k, E, dropped=0.3)
    src_of, row_of, off = cuda(src), cuda(row), cuda(offsets)
    x, _ = values(rng, (T, H), BF)
    o, _ = values(rng, (T * k, H), BF)
    dn, _ = values(rng, (T * k, N), BF)
    g = cuda(rng.random((T, k)), F32)
    w = mok.Fp8Weights(values(rng, (E, N, H), BF)[0], transposed=True)
    q, d = mok.fp8_quantize(o, offsets=off), mok.fp8_quantize(dn, offsets=off)
    used = 128 * int(sum(-(-n // 128) for n in np.diff(offsets)))

    def calls(stream=None):
        yield mok.gather_rows(x, src_of, k, g, stream=stream)
        yield mok.merge_rows(o, row_of, k, g, stream=stream)
        yield from mok.merge_rows_backward(x, o, row_of, g, stream=stream).values()
        both = mok.fp8_quantize(x, src_of=src_of, k=k, offsets=off, stream=stream)
        rows = int(offsets[-1])
        yield both["q"][:rows].view(torch.uint8)
        yield both["scale"][:, :rows]
        yield both["qt"][:, :used].view(torch.uint8)
        yield both["qt_scale"][:used // 128]
        yield w.matmul(q["q"], q["scale"], off, stream=stream)[:rows]
        yield w.matmul_transposed(d["q"], d["scale"], off, stream=stream)[:rows]
        yield mok.fp8_weight_grad(d["qt"], d["qt_scale"], q["qt"], q["qt_scale"], off, stream=stream)

    want = [t.clone() for t in calls()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for here, stream in ((torch.cuda.current_stream(), side), (torch.cuda.current_stream(), side.cuda_stream),
                         (side, torch.cuda.default_stream()), (side, 0)):
        with torch.cuda.stream(here):
            torch.cuda._sleep(200_000_000)
            for n in (4, 1024, 16_384, 24_000, 70_000, 90_000, 140_000, 200_000, 500_000, 1_200_000):
                for _ in range(3):
                    torch.full((n,), 0x55, dtype=torch.uint8, device="cuda")
            got = list(calls(stream))
        assert not here.query()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), i


def test_new_weights_are_ready_on_another_stream():
    """The current stream is busy when weights are made; their first product goes to another stream at once."""
    rng = np.random.default_rng(10)
    E, N, K, R = 3, 304, 272, 50
    offsets = cuda(np.array([0, 20, 20, R], np.int32))
    w, _ = values(rng, (E, N, K), BF)
    q, d = mok.fp8_quantize(values(rng, (R, K), BF)[0]), mok.fp8_quantize(values(rng, (R, N), BF)[0])
    first = mok.Fp8Weights(w, transposed=True)
    want = first.matmul(q["q"], q["scale"], offsets), first.matmul_transposed(d["q"], d["scale"], offsets)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for make in (lambda: mok.Fp8Weights(w, transposed=True),
                 lambda: mok.Fp8Weights.of(first.q.clone(), first.scale.clone(), first.qt.clone(), first.qt_scale.clone())):
        for n in (8, E * N * 272, E * K * 304, 64, 4096):
            torch.full((n,), 0x55, dtype=torch.uint8, device="cuda")
        torch.cuda._sleep(40_000_000)
        weights = make()
        assert torch.cuda.current_stream().query()
        got = (weights.matmul(q["q"], q["scale"], offsets, stream=side),
               weights.matmul_transposed(d["q"], d["scale"], offsets, stream=side))
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and weights.status() == (0, 0)
    torch.cuda._sleep(40_000_000)
    weights = mok.Fp8Weights.empty(E, N, K)
    assert torch.cuda.current_stream().query()
    got = weights.quantize(w, stream=side).matmul(q["q"], q["scale"], offsets, stream=side)
    side.synchronize()
    assert torch.equal(got, want[0]) and weights.status() == (0, 0)


def test_status_of_work_on_another_stream():
    """What a busy stream reports late (written here by a fill) is read, and cleared for whatever comes next."""
    w = mok.Fp8Weights(torch.ones(16, 16).cuda())
    late = torch.tensor([5, 43], dtype=torch.int32).cuda()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(2):
        with torch.cuda.stream(side):
            torch.cuda._sleep(40_000_000)
            w.device_status.copy_(late)
        assert w.status() == (5, 43)
        assert torch.cuda.current_stream().query()
        assert w.status() == (0, 0)


def test_the_weight_gradient_has_a_status_word(monkeypatch):
    """Its own unless one is given, and the same for every call on a device."""
    rng = np.random.default_rng(13)
    offsets = cuda(np.array([0, 70, 90], np.int32))
    q = mok.fp8_quantize(values(rng, (90, 48), BF)[0], offsets=offsets)
    operands = (q["qt"], q["qt_scale"], q["qt"], q["qt_scale"], offsets)
    mok.fp8_weight_grad(*operands)
    assert mok.fp8_status() == (0, 0) == mok.fp8_status("cuda:0")
    given = torch.zeros(2, dtype=torch.int32).cuda()
    mok.fp8_weight_grad(*operands, device_status=given)
    assert given.tolist() == [0, 0]
    words = []
    monkeypatch.setitem(X._FNS, "mok_fp8_weight_grad", lambda *a: words.append(a[-2]) or 0)
    mok.fp8_weight_grad(*operands)
    mok.fp8_weight_grad(*operands, device_status=given)
    word = X._STATUS[0]
    assert words == [word.data_ptr(), given.data_ptr()]
    side, late = torch.cuda.Stream(), torch.tensor([5, 43], dtype=torch.int32).cuda()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):     # what a kernel would report
        torch.cuda._sleep(40_000_000)
        word.copy_(late)
    assert mok.fp8_status() == (5, 43) and mok.fp8_status() == (0, 0)


def test_threads_share_the_status_word(monkeypatch):
    import threading
    monkeypatch.setattr(X, "_STATUS", {})
    x, start, got = torch.zeros(1, device="cuda"), threading.Barrier(16), []

    def call():
        start.wait()
        got.append(X._status_of(x, 0))

    threads = [threading.Thread(target=call) for _ in range(16)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert got == [X._STATUS[0].data_ptr()] * 16
    with pytest.raises(ValueError):
        mok.fp8_status("cpu")


def test_two_calls_at_once():
    """The same weights on two streams: nothing is shared between calls."""
    rng = np.random.default_rng(4)
    E, N, K, R = 8, 512, 1024, 900
    offsets = cuda((np.arange(E + 1) * R // E).astype(np.int32))
    w = mok.Fp8Weights(values(rng, (E, N, K), BF)[0])
    q = [mok.fp8_quantize(values(rng, (R, K), BF)[0], offsets=offsets) for _ in range(2)]
    want = [w.matmul(a["q"], a["scale"], offsets) for a in q]
    outs = [[torch.empty(R, N, dtype=BF, device="cuda") for _ in range(20)] for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(20):
        for a, o, s in zip(q, outs, streams):
            w.matmul(a["q"], a["scale"], offsets, out=o[i], stream=s)
    torch.cuda.synchronize()
    for o, b in zip(outs, want):
        assert all(torch.equal(t, b) for t in o)
    assert w.status() == (0, 0)


def test_repeated_calls_give_the_same_bits():
    rng = np.random.default_rng(6)
    counts = [300, 0, 5, 64, 1]
    offsets = cuda(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))
    R = sum(counts)
    x, _ = values(rng, (R, 640), BF)
    w = mok.Fp8Weights(values(rng, (5, 500, 640), BF)[0])
    q = mok.fp8_quantize(x, offsets=offsets)
    first = None
    for _ in range(5):
        out = (w.matmul(q["q"], q["scale"], offsets, dtype=F32),
               mok.fp8_weight_grad(q["qt"], q["qt_scale"], q["qt"], q["qt_scale"], offsets))
        if first is None:
            first = out
        assert all(torch.equal(a, b) for a, b in zip(first, out))


def test_merge_gradient_without_gates_and_without_their_gradient():
    rng = np.random.default_rng(21)
    T, k, E, H = 30, 3, 5, 72
    _, row, _ = table(rng, T, k, E, dropped=0.2)
    dy, dy64 = values(rng, (T, H), BF)
    o, o64 = values(rng, (T * k, H), BF)
    ones = torch.ones(T, k).cuda()
    want, got = mok.merge_rows_backward(dy, o, cuda(row), ones), mok.merge_rows_backward(dy, o, cuda(row))
    assert torch.equal(got["do"], want["do"]) and torch.equal(got["dgates"], want["dgates"])
    only = {"do": torch.zeros_like(o)}
    assert mok.merge_rows_backward(dy, o, cuda(row), out=only) is only and set(only) == {"do"}
    assert torch.equal(only["do"], want["do"])
    none = torch.empty(0, dtype=torch.int32).cuda()
    assert mok.merge_rows_backward(dy[:0], o, none)["do"].shape == o.shape


def test_the_binding_refuses_half_of_a_pair():
    c = lambda *s, dt=F32: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    x, e = c(6, 32), mok.empty_e4m3
    for call in (lambda: mok.fp8_quantize(x, out={"q": e(6, 32)}), lambda: mok.fp8_quantize(x, out={"scale": c(1, 6)}),
                 lambda: mok.fp8_quantize(x, offsets=i(2), out={"qt": e(32, 128)}),
                 lambda: mok.fp8_quantize(x, offsets=i(2), out={"q": e(6, 32), "scale": c(1, 6), "qt_scale": c(1, 32)}),
                 lambda: mok.fp8_quantize(x, out={"q": e(6, 32), "scale": c(1, 6)}, rows=False),
                 lambda: mok.merge_rows_backward(c(4, 32), c(8, 32), i(8), c(4, 2), out={"dgates": c(4, 2)}),
                 lambda: mok.merge_rows_backward(c(4, 32), c(8, 32), i(9)), lambda: mok.merge_rows_backward(c(0, 32), c(8, 32), i(9)),
                 lambda: mok.merge_rows_backward(c(4, 32), c(8, 32), None),
                 lambda: mok.Fp8Weights.of(e(48, 32), None), lambda: mok.Fp8Weights.of(e(48, 32), 1.0)):
        with pytest.raises(ValueError):
            call()


def test_the_binding_refuses(cuda_ok):
    c = lambda *s, dt=F32: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    e = lambda *s: mok.empty_e4m3(*s)  # noqa: E731
    x, w = c(6, 32), mok.Fp8Weights(c(2, 48, 32))
    calls = [lambda: mok.gather_rows(x, i(8).long(), 2), lambda: mok.gather_rows(x.t(), i(8), 2),
             lambda: mok.gather_rows(x.half(), i(8), 2), lambda: mok.gather_rows(x, i(8), 2, gates=c(6, 3)),
             lambda: mok.gather_rows(x, i(8), 2, out=c(7, 32)), lambda: mok.gather_rows(x.expand(6, 32)[:, :1].expand(6, 32), i(8), 2),
             lambda: mok.gather_rows(x.cpu(), i(8), 2), lambda: mok.gather_rows(x, i(8), 0),
             lambda: mok.gather_rows(x, i(8), 17), lambda: mok.gather_rows(x, i(8), 2, device_status=i(1)),
             lambda: mok.merge_rows(x, i(7), 2), lambda: mok.merge_rows(x, i(8), 2, gates=c(4, 3)),
             lambda: mok.merge_rows(x, i(16)[::2], 2), lambda: mok.merge_rows_backward(c(4, 32), x, i(8), c(4, 3)),
             lambda: mok.merge_rows_backward(c(4, 32), c(6, 32, dt=BF), i(8), c(4, 2)),
             lambda: mok.merge_rows_backward(c(4, 32), x, i(8), c(4, 2), out={"do": c(6, 40)[:, :32], "dgates": c(4, 2)}),
             lambda: mok.fp8_quantize(x, source="relu"), lambda: mok.fp8_quantize(x.half()),
             lambda: mok.fp8_quantize(c(6, 33), source="swiglu"), lambda: mok.fp8_quantize(x, source="swiglu_grad"),
             lambda: mok.fp8_quantize(x, grad=c(6, 16)), lambda: mok.fp8_quantize(x, source="swiglu", src_of=i(6)),
             lambda: mok.fp8_quantize(x, gates=c(6, 1)), lambda: mok.fp8_quantize(x, rows=False),
             lambda: mok.fp8_quantize(x, offsets=i(1)), lambda: mok.fp8_quantize(x, out={"qt": e(32, 128), "qt_scale": c(1, 32)}),
             lambda: mok.fp8_quantize(x, out={"q": c(6, 33, dt=torch.uint8).view(X.E4M3)[:, :32], "scale": c(1, 6)}),
             lambda: w.matmul(e(6, 32), c(1, 6)), lambda: w.matmul(e(6, 31), c(1, 6), i(3)),
             lambda: w.matmul(e(6, 32), c(1, 5), i(3)), lambda: w.matmul(e(6, 32), c(1, 6), i(2)),
             lambda: w.matmul(e(6, 32), c(1, 6), i(3), out=c(6, 48, dt=torch.float16)),
             lambda: w.matmul(c(6, 32), c(1, 6), i(3)), lambda: w.matmul_transposed(e(6, 48), c(1, 6), i(3)),
             lambda: w.matmul(e(6, 32), c(1, 6), i(3), dtype=torch.float16),
             lambda: w.quantize(c(2, 48, 33)), lambda: w.quantize(c(2, 32, 48).transpose(1, 2)),
             lambda: mok.Fp8Weights.of(e(2, 48, 32), c(2, 1, 2)), lambda: mok.Fp8Weights.of(e(2, 48, 32), c(2, 1, 1), qt=e(2, 32, 48)),
             lambda: mok.Fp8Weights.of(c(2, 48, 33, dt=torch.uint8).view(X.E4M3)[:, :, :32], c(2, 1, 1)),
             lambda: mok.fp8_weight_grad(e(8, 100), c(1, 8), e(9, 100), c(1, 9), i(2)),
             lambda: mok.fp8_weight_grad(e(8, 128), c(1, 8), e(9, 256), c(2, 9), i(2)),
             lambda: mok.fp8_weight_grad(e(8, 128), c(1, 8), e(9, 128), c(1, 9), i(3)),
             lambda: mok.fp8_weight_grad(e(8, 128), c(1, 8), e(9, 128), c(1, 9), i(2), out=c(1, 9, 8))]
    for n, call in enumerate(calls):
        with pytest.raises((ValueError, mok.MokError)):
            call()
            pytest.fail(f"call {n} was taken")
