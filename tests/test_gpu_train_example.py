"""The training example: the layer with groups, the balance loss, the clip and AdamW together learn."""
import importlib.util
import os

import pytest
import torch

from mixture_experts_layer_table_gb300 import workloads as W

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("state", ["f32", "mx8"])
def test_the_example_learns(cuda_ok, state):
    from mixture_experts_layer_table_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("train_step", os.path.join(ROOT, "examples", "train_step.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    shape = W.MoEShape("train_T512_H256_E16_I256_top4", T=512, H=256, E=16, I=256, k=4, router=W.ROUTER_SIGMOID,
                       renorm=True, x_std=1.0, w_std=0.05)
    trainer, teacher = ex.Trainer(shape, state=state), ex.Trainer(shape, seed=100)
    x = W.make_inputs(shape, seed=7, device="cuda", with_dy=False)["x"]
    w = teacher.weights
    target = teacher.layer.forward(x, w["w_router"], w["w13"], w["w2"])
    first = trainer.step(x, target)
    assert first["counts"].sum().item() == shape.T * shape.k
    for _ in range(60):
        last = trainer.step(x, target)
    assert trainer.layer.status() == (0, 0) and trainer.opt.steps == 61
    assert torch.isfinite(last["norm"]) and last["mse"].item() < 0.5 * first["mse"].item()


def test_the_balance_loss_reaches_the_router_weights_and_the_input(cuda_ok):
    """A step with the balance loss against one without: the gradients differ by the oracle's gradient of the logits,
    times the input and times the router's weights (dx within its two roundings to bf16, dw_router in f32 sums of 512
    terms)."""
    from mixture_experts_layer_table_gb300 import build
    from oracle import route_oracle as O
    build.build()
    spec = importlib.util.spec_from_file_location("train_step", os.path.join(ROOT, "examples", "train_step.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    shape = W.MoEShape("train_T512_H256_E16_I256_top4", T=512, H=256, E=16, I=256, k=4, router=W.ROUTER_SIGMOID,
                       renorm=True, x_std=1.0, w_std=0.05)
    x = W.make_inputs(shape, seed=7, device="cuda", with_dy=False)["x"]
    target = torch.zeros_like(x)
    without, trainer = ex.Trainer(shape, state="f32", balance_coef=0.0), ex.Trainer(shape, state="f32", balance_coef=3.0)
    w = trainer.weights["w_router"].double().cpu().numpy()
    without.step(x, target)
    trainer.step(x, target)
    logits, idx = (trainer.layer.view(n).cpu().numpy() for n in ("logits", "topk_idx"))
    logits = logits.astype("float64")
    dprob = O.balance(O.scores(logits, O.SIGMOID), idx, 3.0, None, 0.0)[3]
    dl = O.backward(logits, idx, None, dprob, O.SIGMOID, True, 1.0)
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    dx0, dx1 = f64(without.grads["dx"]), f64(trainer.grads["dx"])
    term = dl @ w
    assert abs(term).max() > 20 * 2.0 ** -8 * abs(dx0).mean()
    assert (abs(dx1 - dx0 - term) <= 2.0 ** -8 * abs(dx1) + 2.0 ** -14 * abs(term).max()).all()
    dw = f64(trainer.grads["dw_router"]) - f64(without.grads["dw_router"])
    want = dl.T @ f64(x)
    assert (abs(dw - want) <= 2.0 ** -14 * (abs(dl).T @ abs(f64(x)) + abs(f64(without.grads["dw_router"])))).all()
