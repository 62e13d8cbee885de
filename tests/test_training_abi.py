"""Refusals of the training-step entry points (CPU only): the C ABI answers before it touches the GPU,
and the binding refuses what the bare pointers could not carry."""
import ctypes

import pytest
import torch

import mixture_experts_layer_table_gb300 as mok
from mixture_experts_layer_table_gb300 import _native as N
from mixture_experts_layer_table_gb300 import training as TR

P = ctypes.c_void_p
INVALID, WS_SMALL = 1, 3


@pytest.fixture(scope="module")
def lib():
    from mixture_experts_layer_table_gb300 import build
    build.build()
    if torch.cuda.is_available():
        pytest.skip("placeholder addresses are for hosts without a GPU")
    return N.load()


def _adamw(**kw):
    t = dict(param=0x100000, master=None, grad=0x200000, m=0x300000, v=0x400000, m_scale=None, v_scale=None, n=100,
             counter=0, lr=1e-3, weight_decay=0.1, param_type=0, grad_type=0, state_type=0, reserved=0)
    t.update(kw)
    return TR.AdamWTensor(**t)


@pytest.mark.parametrize("kw", [dict(param=None), dict(grad=None), dict(m=None), dict(v=None), dict(n=-1),
                                dict(param_type=2), dict(grad_type=-1), dict(state_type=2), dict(reserved=1),
                                dict(counter=4), dict(lr=float("nan")), dict(weight_decay=float("inf")),
                                dict(master=0x500000), dict(m_scale=0x500000), dict(state_type=1),
                                dict(param=0x100002), dict(grad=0x200001), dict(m=0x300002),
                                dict(param_type=1, param=0x100001), dict(param_type=1, master=0x500002)])
def test_adamw_refuses_a_bad_tensor(lib, kw):
    call, hyper = TR._adamw_fn(), TR.AdamWHyper(0.9, 0.95, 1e-8, 1, 0, 0)
    arr = (TR.AdamWTensor * 2)(_adamw(n=0, param=None, grad=None, m=None, v=None), _adamw(**kw))
    assert call(arr, 2, ctypes.byref(hyper), None, None) == INVALID


@pytest.mark.parametrize("hyper", [(1.0, 0.95, 1e-8, 1, 0, 0), (0.9, -0.1, 1e-8, 1, 0, 0), (0.9, 0.95, -1.0, 1, 0, 0),
                                   (0.9, 0.95, float("inf"), 1, 0, 0), (0.9, 0.95, 1e-8, 0, 0, 0),
                                   (0.9, 0.95, 1e-8, 1, 0, 1), (float("nan"), 0.95, 1e-8, 1, 0, 0)])
def test_adamw_refuses_bad_hyperparameters(lib, hyper):
    arr = (TR.AdamWTensor * 1)(_adamw())
    call = TR._adamw_fn()
    assert call(arr, 1, ctypes.byref(TR.AdamWHyper(*hyper)), None, None) == INVALID
    assert call(arr, 1, None, None, None) == INVALID
    ok = ctypes.byref(TR.AdamWHyper(0.9, 0.95, 1e-8, 1, 0, 0))
    assert call(None, 1, ok, None, None) == INVALID
    assert call(arr, -1, ok, None, None) == INVALID
    assert call(arr, 1, ok, P(0x100002), None) == INVALID      # misaligned scale


def test_grad_norm_refuses(lib):
    call = TR._grad_norm_fn()
    ok = TR.GradTensor(0x100000, 10, 0, 0)
    arr = lambda t: (TR.GradTensor * 1)(t)  # noqa: E731
    ws, n, out = P(0x200000), TR.GRAD_NORM_WS_BYTES, P(0x300000)
    for bad in (TR.GradTensor(None, 10, 0, 0), TR.GradTensor(0x100000, -1, 0, 0), TR.GradTensor(0x100000, 10, 2, 0),
                TR.GradTensor(0x100002, 10, 0, 0), TR.GradTensor(0x100001, 10, 1, 0), TR.GradTensor(0x100000, 10, 0, 1)):
        assert call(arr(bad), 1, 1.0, out, ws, n, None) == INVALID
    for max_norm in (0.0, -1.0, float("nan")):
        assert call(arr(ok), 1, max_norm, out, ws, n, None) == INVALID
    assert call(None, 1, 1.0, out, ws, n, None) == INVALID
    assert call(arr(ok), -1, 1.0, out, ws, n, None) == INVALID
    assert call(arr(ok), 1, 1.0, None, ws, n, None) == INVALID
    assert call(arr(ok), 1, 1.0, out, None, n, None) == INVALID
    assert call(arr(ok), 1, 1.0, out, P(0x200008), n, None) == INVALID
    assert call(arr(ok), 1, 1.0, out, ws, n - 1, None) == WS_SMALL


def test_the_binding_refuses_host_tensors_and_mismatches(lib):
    t = torch.zeros(8)
    with pytest.raises(ValueError, match="CUDA"):
        mok.GradNorm([t], 1.0)
    with pytest.raises(ValueError, match="CUDA"):
        mok.AdamW([t], [t])
    with pytest.raises(ValueError, match="expected a tensor"):
        mok.AdamW([t.double()], [t])
    with pytest.raises(ValueError, match="1 params and 0 grads"):
        mok.AdamW([t], [])
    with pytest.raises(ValueError, match="state"):
        mok.AdamW([t], [t], state="int8")
    with pytest.raises(ValueError, match="betas"):
        mok.AdamW([t], [t], betas=(0.9, 1.0))
    with pytest.raises(ValueError, match="max_norm"):
        mok.GradNorm([t], 0.0)


def _route_desc(**kw):
    d = mok.make_route_desc(10, 32, 4, 1, True, n_group=8, topk_group=4)
    for n, v in kw.items():
        setattr(d, n, v)
    return d


@pytest.mark.parametrize("kw,code", [(dict(T=-1), 1), (dict(E=0), 1), (dict(k=0), 1), (dict(k=17), 1), (dict(router=2), 1),
                                     (dict(group_score=2), 1), (dict(n_group=0), 1), (dict(n_group=5), 1),
                                     (dict(topk_group=0), 1), (dict(topk_group=9), 1), (dict(logits_type=2), 1),
                                     (dict(logits_stride=31), 1), (dict(route_scale=float("nan")), 1),
                                     (dict(balance_coef=float("inf")), 1), (dict(bias_rate=float("nan")), 1),
                                     (dict(reserved=1), 1), (dict(E=2048), 2), (dict(E=64, n_group=64, topk_group=64), 2),
                                     (dict(E=64, n_group=1, topk_group=1, k=17), 2), (dict(topk_group=1, k=5), 1)])
def test_route_refuses_a_bad_descriptor(lib, kw, code):
    from mixture_experts_layer_table_gb300 import routing as RT
    a = [P(0x100000 * (i + 1)) for i in range(12)]
    d = ctypes.byref(_route_desc(**kw))
    assert RT._route_fn()(d, *a[:10], a[10], RT.ROUTE_WS_BYTES, None) == code
    assert RT._route_backward_fn()(d, *a[:5], 0, a[5], None) == code


def test_route_refuses_bad_pointers_and_workspaces(lib):
    from mixture_experts_layer_table_gb300 import routing as RT
    d = _route_desc()
    names = ("logits", "bias", "topk_idx", "gates", "scores", "counts", "prob_sum", "loss", "dprob", "bias_next")
    ok = {n: 0x100000 * (i + 1) for i, n in enumerate(names)}

    def call(ws=0xF00000, n=RT.ROUTE_WS_BYTES, **kw):
        p = {**ok, **kw}
        return RT._route_fn()(ctypes.byref(d), *[p[n] for n in names], ws, n, None)

    for n in names:
        assert call(n=0, **{n: 0x100002}) == INVALID, n
    assert call(logits=None) == INVALID and call(topk_idx=None) == INVALID
    assert call(bias=None) == INVALID                       # bias_next without a bias
    assert call(ws=None) == INVALID and call(ws=0xF00010) == INVALID
    assert call(n=RT.ROUTE_WS_BYTES - 1) == WS_SMALL
    d.T = 1 << 31
    assert call() == 2
    d.T = 10
    back = RT._route_backward_fn()
    a = [P(0x100000 * (i + 1)) for i in range(6)]

    def call_back(logits=a[0], idx=a[1], dg=a[2], dp=a[3], out=a[4], stride=0, status=a[5]):
        return back(ctypes.byref(d), logits, idx, dg, dp, out, stride, status, None)

    assert call_back(dg=None, dp=None) == INVALID
    assert call_back(idx=None) == INVALID and call_back(logits=None) == INVALID and call_back(out=None) == INVALID
    assert call_back(stride=31) == INVALID and call_back(out=P(0x100002)) == INVALID and call_back(status=P(0x100001)) == INVALID


def test_the_router_binding_refuses_mismatches(lib):
    r = mok.Router(mok.make_route_desc(4, 8, 2, 1, True), device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        r.forward(torch.zeros(4, 8))
    with pytest.raises(ValueError, match="logits"):
        r.forward(torch.zeros(4, 9))
    with pytest.raises(ValueError, match="logits"):
        r.forward(torch.zeros(4, 8).bfloat16())
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        mok.Router(mok.make_route_desc(4, 8, 2, 1, True), dtype=torch.float16, device="cpu")


class _OnGpu:
    """What the binding looks at of a CUDA tensor, with an address that is none."""

    def __init__(self, shape, dtype=torch.float32, index=0):
        self.shape, self.dtype, self.is_cuda, self.device = torch.Size(shape), dtype, True, torch.device("cuda", index)

    def get_device(self):
        return self.device.index

    def is_contiguous(self):
        return True

    def stride(self, i):
        return self.shape[1] if i == 0 else 1

    def data_ptr(self):
        return 0x100000


def test_the_router_binding_refuses_another_device_than_its_buffers(lib, monkeypatch):
    """Buffers on the CPU or on another GPU, logits on this one: their addresses do not go to the kernel."""
    from mixture_experts_layer_table_gb300 import routing as RT
    monkeypatch.setattr(RT, "_stream", lambda s: None)
    r = mok.Router(mok.make_route_desc(4, 8, 2, 1, True), device="cpu")
    monkeypatch.setattr(r, "_call", lambda *a: pytest.fail("called"))
    monkeypatch.setattr(r, "_call_backward", lambda *a: pytest.fail("called"))
    for call in (lambda: r.forward(_OnGpu((4, 8))), lambda: r.backward(_OnGpu((4, 8)), None, None)):
        with pytest.raises(ValueError, match="logits is on cuda:0"):
            call()
    r._device = 1                                            # as of buffers on a second GPU
    with pytest.raises(ValueError, match="logits is on cuda:0"):
        r.forward(_OnGpu((4, 8)))
    with pytest.raises(ValueError, match="out is on cuda:0"):
        r.backward(_OnGpu((4, 8), index=1), None, None, out=_OnGpu((4, 8)))


def test_the_router_binding_refuses_a_moved_bias_that_nothing_would_move(lib, monkeypatch):
    from mixture_experts_layer_table_gb300 import routing as RT
    monkeypatch.setattr(RT, "_stream", lambda s: None)
    b = _OnGpu((8,))
    for balance, bias in ((False, b), (True, None), (False, None)):
        r = mok.Router(mok.make_route_desc(4, 8, 2, 1, True), balance=balance, device="cpu")
        r._device = 0
        monkeypatch.setattr(r, "_call", lambda *a: pytest.fail("called"))
        with pytest.raises(ValueError, match="bias_next"):
            r.forward(_OnGpu((4, 8)), bias, bias_next=b)
