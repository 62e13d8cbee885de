"""Refusals of the entry points for experts outside the layer (CPU only): the C ABI answers before it touches the
GPU, and the binding refuses what the bare pointers could not carry.  And the oracle's own properties."""
import ctypes

import numpy as np
import pytest
import torch

import mixture_experts_layer_table_gb300 as mok
from mixture_experts_layer_table_gb300 import _native as N
from mixture_experts_layer_table_gb300 import experts as X
from oracle import experts_oracle as O

P = ctypes.c_void_p
OK, INVALID, UNSUPPORTED = 0, 1, 2
A = [0x100000 * (i + 1) for i in range(12)]


@pytest.fixture(scope="module")
def lib():
    from mixture_experts_layer_table_gb300 import build
    build.build()
    if torch.cuda.is_available():
        pytest.skip("placeholder addresses are for hosts without a GPU")
    return N.load()


ROWS = dict(T=10, R=20, H=64, token_stride=0, row_stride=0, k=2, type=1)
ROW_CALLS = [("mok_gather_rows", 5), ("mok_merge_rows", 5), ("mok_merge_rows_backward", 7)]


@pytest.mark.parametrize("name,n", ROW_CALLS)
@pytest.mark.parametrize("kw,code", [(dict(T=-1), 1), (dict(R=-1), 1), (dict(H=0), 1), (dict(k=0), 1), (dict(k=17), 2),
                                     (dict(type=2), 1), (dict(token_stride=63), 1), (dict(row_stride=-1), 1),
                                     (dict(R=1 << 31), 2), (dict(T=1 << 30, k=2), 2), (dict(H=1 << 28), 2)])
def test_rows_refuse_a_bad_descriptor(lib, name, n, kw, code):
    fn = X._fn(name, X.RowsDesc, n)
    assert fn(X.RowsDesc(**{**ROWS, **kw}), *A[:n], None) == code
    assert fn(None, *A[:n], None) == INVALID


@pytest.mark.parametrize("name,n", ROW_CALLS)
def test_rows_refuse_bad_pointers(lib, name, n):
    fn, d = X._fn(name, X.RowsDesc, n), X.RowsDesc(**{**ROWS, "type": 0})
    optional = {"mok_gather_rows": (2, 4), "mok_merge_rows": (2, 4), "mok_merge_rows_backward": (3, 5, 6)}[name]
    for i in range(n):
        a = list(A[:n])
        a[i] = 0x100002
        assert fn(d, *a, None) == INVALID, i
        if i not in optional:
            a[i] = None
            assert fn(d, *a, None) == INVALID, i
    # nothing to do: no pointer is looked at
    empty = X.RowsDesc(**{**ROWS, "T": 0, "R": 0})
    assert fn(empty, *[None] * n, None) == OK


QUANT = dict(R=100, C=256, T=50, x_stride=0, grad_stride=0, q_stride=0, scale_stride=0, qt_stride=0, E=4, k=2, source=0,
             type=1)
QNAMES = ("x", "grad", "src_of", "gates", "offsets", "q", "scale", "qt", "qt_scale", "status")


def quantize(d, **kw):
    a = dict(zip(QNAMES, A), grad=None)
    a.update(kw)
    return X._fn("mok_fp8_quantize", X.Fp8QuantizeDesc, 10)(X.Fp8QuantizeDesc(**{**QUANT, **d}), *[a[n] for n in QNAMES], None)


@pytest.mark.parametrize("d,kw,code", [
    (dict(R=-1), {}, 1), (dict(C=0), {}, 1), (dict(T=-1), {}, 1), (dict(type=2), {}, 1), (dict(source=3), {}, 1),
    (dict(k=0), {}, 1), (dict(k=17), {}, 2), (dict(E=0), {}, 1), (dict(E=1025), {}, 2), (dict(C=1 << 28), {}, 2),
    (dict(R=1 << 31), {}, 2), (dict(x_stride=255), {}, 1), (dict(q_stride=264), {}, 1), (dict(q_stride=240), {}, 1),
    (dict(scale_stride=99), {}, 1), (dict(qt_stride=16), {}, 1), (dict(qt_stride=521), {}, 1),
    (dict(source=1), {}, 1), (dict(source=1), dict(src_of=None), 1), (dict(source=2), dict(src_of=None, gates=None), 1),
    (dict(source=2, C=257), dict(src_of=None, gates=None, grad=A[1]), 1),
    (dict(source=2, grad_stride=100), dict(src_of=None, gates=None, grad=A[1]), 1),
    ({}, dict(grad=A[1]), 1), ({}, dict(src_of=None), 1), ({}, dict(q=None), 1), ({}, dict(scale=None), 1),
    ({}, dict(qt=None), 1), ({}, dict(qt_scale=None), 1), ({}, dict(q=None, scale=None, qt=None, qt_scale=None), 1),
    ({}, dict(offsets=None), 1), ({}, dict(x=None), 1), ({}, dict(x=0x100001), 1), ({}, dict(q=0x100008), 1),
    ({}, dict(qt=0x100004), 1), ({}, dict(scale=0x100002), 1), ({}, dict(offsets=0x100001), 1), ({}, dict(status=0x100002), 1),
    (dict(R=0, T=0), {}, 0), (dict(R=0), dict(x=None, q=None, scale=None, qt=None, qt_scale=None), 0)])
def test_quantize_refuses(lib, d, kw, code):
    assert quantize(d, **kw) == code


def test_quantize_weights_refuses(lib):
    fn = X._fn("mok_fp8_quantize_weights", X.Fp8WeightsDesc, 5)
    ok = dict(N=100, K=200, q_stride=0, qt_stride=0, E=2, type=1)
    for kw, code in ((dict(N=0), 1), (dict(K=0), 1), (dict(E=0), 1), (dict(type=2), 1), (dict(q_stride=100), 1),
                     (dict(q_stride=204), 1), (dict(qt_stride=90), 1), (dict(E=1025), 2), (dict(N=1 << 28), 2)):
        assert fn(X.Fp8WeightsDesc(**{**ok, **kw}), *A[:5], None) == code, kw
    for i in range(5):
        a = list(A[:5])
        a[i] = None
        assert fn(X.Fp8WeightsDesc(**ok), *a, None) == INVALID
        a[i] = 0x100001
        assert fn(X.Fp8WeightsDesc(**ok), *a, None) == INVALID
    assert fn(X.Fp8WeightsDesc(**ok), A[0], None, None, None, None, None) == INVALID


def test_matmul_refuses(lib):
    fn = X._fn("mok_fp8_matmul", X.Fp8MatmulDesc, 7)
    ok = dict(R=100, N=300, K=200, x_stride=0, x_scale_stride=0, w_stride=0, out_stride=0, E=2, out_type=1)
    for kw, code in ((dict(R=-1), 1), (dict(N=0), 1), (dict(K=0), 1), (dict(E=0), 1), (dict(out_type=2), 1),
                     (dict(x_stride=200), 1), (dict(x_stride=192), 1), (dict(w_stride=201), 1), (dict(x_scale_stride=99), 1),
                     (dict(out_stride=299), 1), (dict(E=1025), 2), (dict(R=1 << 31), 2), (dict(K=1 << 28), 2)):
        assert fn(X.Fp8MatmulDesc(**{**ok, **kw}), *A[:7], None) == code, kw
    for i in range(7):
        a = list(A[:7])
        a[i] = 0x100001
        assert fn(X.Fp8MatmulDesc(**ok), *a, None) == INVALID, i
        if i < 6:
            a[i] = None
            assert fn(X.Fp8MatmulDesc(**ok), *a, None) == INVALID, i
    assert fn(X.Fp8MatmulDesc(**{**ok, "R": 0}), *A[:7], None) == OK


def test_weight_grad_refuses(lib):
    fn = X._fn("mok_fp8_weight_grad", X.Fp8WeightGradDesc, 7)
    ok = dict(R=100, N=300, H=200, dy_stride=0, x_stride=0, E=2, out_type=0)
    for kw, code in ((dict(R=-1), 1), (dict(N=0), 1), (dict(H=0), 1), (dict(E=0), 1), (dict(out_type=-1), 1),
                     (dict(dy_stride=240), 1), (dict(x_stride=264), 1), (dict(E=1025), 2), (dict(R=1 << 31), 2)):
        assert fn(X.Fp8WeightGradDesc(**{**ok, **kw}), *A[:7], None) == code, kw
    for i in range(7):
        a = list(A[:7])
        a[i] = 0x100001
        assert fn(X.Fp8WeightGradDesc(**ok), *a, None) == INVALID, i
        if i < 6:
            a[i] = None
            assert fn(X.Fp8WeightGradDesc(**ok), *a, None) == INVALID, i


def test_the_binding_refuses_host_tensors():
    x, i = torch.zeros(4, 32), torch.zeros(8, dtype=torch.int32)
    for call in (lambda: mok.gather_rows(x, i, 2), lambda: mok.merge_rows(x, i, 2),
                 lambda: mok.merge_rows_backward(x, x, i, torch.zeros(4, 2)), lambda: mok.fp8_quantize(x),
                 lambda: mok.Fp8Weights(x), lambda: mok.Fp8Weights.of(x.to(torch.float8_e4m3fn), torch.zeros(1, 1)),
                 lambda: mok.fp8_weight_grad(mok.empty_e4m3(4, 128, device="cpu"), torch.zeros(1, 4),
                                             mok.empty_e4m3(4, 128, device="cpu"), torch.zeros(1, 4), i[:2])):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_e4m3_rows_start_at_multiples_of_16_bytes():
    for width in (1, 15, 16, 17, 128, 1111):
        t = mok.empty_e4m3(3, 5, width, device="cpu")
        assert t.shape == (3, 5, width) and t.stride(1) % 16 == 0 and t.stride(0) == 5 * t.stride(1)


def test_the_oracles_e4m3_is_torchs():
    rng = np.random.default_rng(0)
    y = np.concatenate([rng.normal(size=4000) * 100, rng.normal(size=4000) * 0.01, np.linspace(-448, 448, 7169),
                        np.arange(-64, 65) * 2.0 ** -10]).astype(np.float32)
    y = np.clip(y, -448, 448)
    assert np.array_equal(O.e4m3(y.astype(np.float64)), torch.tensor(y).to(torch.float8_e4m3fn).double().numpy())


def test_the_oracles_products_are_each_others_gradients():
    """<dy, x W^T> = <dy W, x> = <dy^T x, W> with blocks' scales of one."""
    rng = np.random.default_rng(1)
    offsets = [0, 5, 5, 40]
    x, w, dy = rng.normal(size=(40, 36)), rng.normal(size=(3, 20, 36)), rng.normal(size=(40, 20))
    ones = lambda *s: np.ones(s)  # noqa: E731
    y = O.product(x, ones(1, 40), w, ones(3, 1, 1), offsets)[0]
    dx = O.product(dy, ones(1, 40), w.transpose(0, 2, 1), ones(3, 1, 1), offsets)[0]
    cols = lambda t: np.concatenate([np.pad(t[a:b], ((0, -(b - a) % 128), (0, 0))) for a, b in zip(offsets, offsets[1:])]).T  # noqa: E731
    dw = O.weight_grad(cols(dy), ones(3, 20), cols(x), ones(3, 36), offsets)[0]
    assert np.isclose((dy * y).sum(), (dx * x).sum()) and np.isclose((dy * y).sum(), (dw * w).sum())
