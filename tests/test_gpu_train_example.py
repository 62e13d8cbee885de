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
