"""A training loop of one group-limited mixture-of-experts layer on the library's kernels.

    python examples/train_step.py [--steps N] [--state f32|mx8]

Each step: the layer's forward (experts chosen within the best groups, selection moved by a bias), its
backward, the balance loss and its gradient through the router logits, the global gradient norm, and one
AdamW step of all weights on the clipped gradients.  The balance loss is not the layer's: its gradient comes as
that of the logits, and two products of PyTorch's add it to the gradients of the router's weights and of the
layer's input (which a layer below this one would take).  The layer learns to reproduce another layer of the
same shape (random weights); the expert loads are kept together by the balance loss and by the bias that
moves after each step.
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import mixture_experts_layer_table_gb300 as mok  # noqa: E402
from mixture_experts_layer_table_gb300 import workloads as W  # noqa: E402

GROUPS = dict(n_group=4, topk_group=2, group_score=mok.GROUP_TOP2)


class Trainer:
    """The layer, its weights and buffers, and one step on a batch."""

    def __init__(self, shape, state="mx8", lr=2e-3, balance_coef=1e-2, bias_rate=1e-3, max_norm=1.0, seed=0):
        self.shape = shape
        dev = "cuda"
        T, H, E, I, k = shape.T, shape.H, shape.E, shape.I, shape.k
        inp = W.make_inputs(shape, seed=seed, device=dev, with_dy=False)
        self.weights = {n: inp[n] for n in ("w_router", "w13", "w2")}
        self.bias = torch.zeros(E, device=dev)
        self.layer = mok.MoELayer(mok.desc_from_shape(shape, **GROUPS))
        self.grads = {"dx": torch.empty((T, H), dtype=torch.bfloat16, device=dev),
                      "dw_router": torch.empty((E, H), device=dev), "dw13": torch.empty((E, 2 * I, H), device=dev),
                      "dw2": torch.empty((E, H, I), device=dev), "dgates": torch.empty((T, k), device=dev)}
        self.router = mok.Router(mok.make_route_desc(T, E, k, shape.router, shape.renorm, balance_coef=balance_coef,
                                                     bias_rate=bias_rate, **GROUPS), balance=True)
        wgrads = [self.grads[n] for n in ("dw_router", "dw13", "dw2")]
        self.norm = mok.GradNorm(wgrads, max_norm)
        self.opt = mok.AdamW(list(self.weights.values()), wgrads, lr=lr, betas=(0.9, 0.95), weight_decay=0.0,
                             state=state, masters=True if state == "f32" else None, seed=seed)

    def step(self, x, target):
        """One step on rows x; returns {"mse", "balance", "norm", "counts"} as device tensors."""
        w = self.weights
        y = self.layer.forward(x, w["w_router"], w["w13"], w["w2"], router_bias=self.bias)
        diff = y.float() - target.float()
        dy = (diff * (2.0 / diff.numel())).bfloat16()
        self.layer.backward(dy, x, w["w_router"], w["w13"], w["w2"], out=self.grads)
        # balance: loads and probabilities of the layer's own logits; its gradient joins that of the router's weights and
        # that of the input
        logits = self.layer.view("logits")
        stats = self.router.forward(logits, self.bias, bias_next=self.bias)
        dlogits = self.router.backward(logits, None, None, stats["dprob"])
        self.grads["dw_router"] += dlogits.T @ x.float()
        self.grads["dx"].copy_(self.grads["dx"].float() + dlogits @ w["w_router"].float())
        norm = self.norm.compute()
        self.opt.step(norm[1:])
        return {"mse": diff.square().mean(), "balance": stats["loss"][0].clone(), "norm": norm[0].clone(),
                "counts": stats["counts"].clone()}


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--state", choices=("f32", "mx8"), default="mx8")
    a = ap.parse_args()
    shape = W.MoEShape("train_T2048_H512_E16_I512_top4", T=2048, H=512, E=16, I=512, k=4, router=W.ROUTER_SIGMOID,
                       renorm=True, x_std=1.0, w_std=0.04)
    trainer, teacher = Trainer(shape, state=a.state), Trainer(shape, seed=100)
    for i in range(a.steps):
        x = W.make_inputs(shape, seed=1000 + 10 * i, device="cuda", with_dy=False)["x"]
        w = teacher.weights
        target = teacher.layer.forward(x, w["w_router"], w["w13"], w["w2"])
        out = trainer.step(x, target)
        if i % 20 == 0 or i == a.steps - 1:
            c = out["counts"].float()
            print(f"step {i:4d}  mse {out['mse'].item():.5f}  balance {out['balance'].item():.5f}  "
                  f"|g| {out['norm'].item():.3e}  largest load / mean {(c.max() / c.mean()).item():.2f}")
    assert trainer.layer.status() == (0, 0)


if __name__ == "__main__":
    main()
