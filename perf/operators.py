"""Cases, plain forms and 64-bit definitions of the training-step operators around the MoE layer.

Four operators: ``route`` (expert selection limited to groups of experts, with the balance loss and
the moved selection bias), ``route_backward`` (its gradient with respect to the logits),
``grad_norm`` (the 2-norm of many gradients and the clip factor) and ``adamw`` (an AdamW step over
many tensors, states in 32 or 8 bits).

``run`` computes an operator in elementary torch operations in 32 bits, or, with ``own`` set, with
the library's kernels; ``exact`` restates it in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
SOFTMAX, SIGMOID = 0, 1
GROUP_MAX, GROUP_TOP2 = 0, 1
BALANCE_COEF, BIAS_RATE, ROUTE_SCALE = 1e-3, 1e-3, 2.5
BETA1, BETA2, EPS, LR, WD = 0.9, 0.95, 1e-8, 2e-4, 0.1
SEED = 20250
MAX_NORM = 1.0

# Parameters of one layer's share of experts: w13, w2 and the router (H = 7168, I = 2048, 256 experts
# in all, of which a device that holds a 32nd part updates 8).
DSV3_SHARE = "8x4096x7168,8x7168x2048,256x7168"
# The tiny layer (H = 256, I = 512, 8 experts).
TINY = "8x1024x256,8x256x512,8x256"


def listed():
    return [
        # one decoded token, 256 experts in 8 groups: latency
        dict(name="route_token", op="route", T=1, E=256, k=8, router=SIGMOID, n_group=8, topk_group=4,
             group=GROUP_TOP2, bits=32, balance=False),
        # one training micro-batch with the balance loss and the moved bias
        dict(name="route_train_4096", op="route", T=4096, E=256, k=8, router=SIGMOID, n_group=8, topk_group=4,
             group=GROUP_TOP2, bits=32, balance=True),
        # softmax router, groups ranked by their best expert, bf16 logits, an odd number of tokens
        dict(name="route_softmax_12345", op="route", T=12345, E=160, k=6, router=SOFTMAX, n_group=8, topk_group=3,
             group=GROUP_MAX, bits=16, balance=True),
        # a long prefill or a large global batch
        dict(name="route_prefill_65536", op="route", T=65536, E=256, k=8, router=SIGMOID, n_group=8, topk_group=4,
             group=GROUP_TOP2, bits=32, balance=False),
        # backward of the training micro-batch: gate gradients and the balance term
        dict(name="route_bwd_4096", op="route_backward", T=4096, E=256, k=8, router=SIGMOID, n_group=8, topk_group=4,
             group=GROUP_TOP2, bits=32, balance=True),
        # softmax router backward at a large batch
        dict(name="route_bwd_softmax_65536", op="route_backward", T=65536, E=160, k=6, router=SOFTMAX, n_group=8,
             topk_group=3, group=GROUP_MAX, bits=32, balance=True),
        # norms, biases and small matrices of odd sizes
        dict(name="norm_many", op="grad_norm", count=96, smallest=1, largest=30011, grad=32),
        # the gradients of one layer's share of experts
        dict(name="norm_experts", op="grad_norm", shapes=DSV3_SHARE, grad=32),
        # a small layer's step: latency
        dict(name="adamw_tiny", op="adamw", shapes=TINY, param=16, master=True, grad=32, state=32),
        # many small tensors of odd sizes kept in f32
        dict(name="adamw_many", op="adamw", count=96, smallest=1, largest=30011, param=32, master=False, grad=32,
             state=32),
        # one layer's share of experts: bf16 weights with f32 masters, f32 states
        dict(name="adamw_experts", op="adamw", shapes=DSV3_SHARE, param=16, master=True, grad=32, state=32),
        # the same weights with 8-bit states, bf16 gradients and no masters
        dict(name="adamw_experts_8bit", op="adamw", shapes=DSV3_SHARE, param=16, master=False, grad=16, state=8),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_backward", "grad_norm", "adamw"])
    if op in ("route", "route_backward"):
        n_group = rng.choice([1, 2, 4, 6, 8, 16])
        size = _log_uniform(rng, 4, 512 // n_group)
        topk_group = rng.randint(1, n_group)
        # a single renormalised gate is the constant 1: its gradient is zero, and nothing to compare
        k = rng.randint(1 if op == "route" else 2, min(16, topk_group * size))
        E = n_group * size
        T = _log_uniform(rng, 1, 65536)
        T = min(T, 65536 * 256 // E)
        return dict(op=op, T=T, E=E, k=k, router=rng.choice([SOFTMAX, SIGMOID]), n_group=n_group,
                    topk_group=topk_group, group=rng.choice([GROUP_MAX, GROUP_TOP2]), bits=rng.choice([16, 32]),
                    balance=rng.random() < 0.5)
    count = _log_uniform(rng, 1, 200)
    largest = _log_uniform(rng, 100, 120_000_000 // count)
    case = dict(op=op, count=count, smallest=max(1, largest // rng.choice([1, 2, 50])), largest=largest,
                grad=rng.choice([16, 32]))
    if op == "adamw":
        case["param"], case["master"] = rng.choice([(32, False), (16, True), (16, False)])
        case["state"] = rng.choice([8, 32])
    return case


# ------------------------------------------------------------------ inputs

def _sizes(case):
    """Elements of each tensor: from the shapes, or `count` odd sizes from smallest to largest."""
    if "shapes" in case:
        return [math.prod(int(n) for n in s.split("x")) for s in case["shapes"].split(",")]
    lo, hi, count = case["smallest"], case["largest"], case["count"]
    ratio = (hi / lo) ** (1 / max(1, count - 1))
    return [min(hi, int(lo * ratio ** i) | 1) for i in range(count)]


def _spans(case):
    """(start, size) of each tensor in a flat buffer; every tensor starts at a multiple of 32 elements."""
    spans, at = [], 0
    for n in _sizes(case):
        spans.append((at, n))
        at += (n + 31) // 32 * 32
    return spans, at


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(shape, g, std=1.0):
    return torch.empty(shape, dtype=torch.float32, device=DEV).normal_(0.0, std, generator=g)


def _flat(case, fill):
    """A flat float32 buffer of all tensors, `fill`ed, zero between them."""
    spans, total = _spans(case)
    t = fill(total)
    if total != sum(n for _, n in spans):
        keep = torch.zeros(total, dtype=torch.bool, device=DEV)
        for at, n in spans:
            keep[at:at + n] = True
        t = torch.where(keep, t, torch.zeros((), device=DEV))
    return t


def _prepare_route(case, seed):
    g = _generator(seed)
    T, E = case["T"], case["E"]
    # what x W_r^T gives at the layer's widths (std 0.5), and experts of unequal popularity
    logits = _normal((T, E), g, 0.5) + _normal((E,), g, 0.25)
    bias = _normal((E,), g, 0.05) if case["router"] == SIGMOID else None
    s = dict(logits=logits if case["bits"] == 32 else logits.bfloat16(), bias=bias)
    if case["op"] == "route_backward":
        s["idx"] = _select(s["logits"].float(), bias, case)[0].int()
        s["dgates"] = _normal((T, case["k"]), g, 1.0 / T)
        s["dprob"] = torch.rand(E, generator=g, device=DEV) * (2e-3 / T) if case["balance"] else None
    if own:
        import mixture_experts_layer_table_gb300 as mok
        desc = mok.make_route_desc(T, E, case["k"], case["router"], True, route_scale=ROUTE_SCALE,
                                   n_group=case["n_group"], topk_group=case["topk_group"],
                                   group_score=case["group"], balance_coef=BALANCE_COEF, bias_rate=BIAS_RATE)
        s["router"] = mok.Router(desc, dtype=s["logits"].dtype, balance=case["balance"])
    return s


def _gradients(case, g):
    """Gradients after a normalised loss: most small, some rows far larger (a log-normal spread)."""
    def fill(n):
        t = _normal(n, g, 1e-3)
        rows = torch.exp(_normal((n // 32,), g, 1.0))
        t.view(-1, 32).mul_(rows[:, None])
        return t
    t = _flat(case, fill)
    return t if case["grad"] == 32 else t.bfloat16()


def _prepare_norm(case, seed):
    s = dict(grad=_gradients(case, _generator(seed)))
    if own:
        import mixture_experts_layer_table_gb300 as mok
        s["norm"] = mok.GradNorm([s["grad"][a:a + n] for a, n in _spans(case)[0]], MAX_NORM)
    return s


def _prepare_adamw(case, seed):
    g = _generator(seed)
    total = _spans(case)[1]
    s = dict(grad=_gradients(case, g), step=100,
             scale=torch.tensor([0.37], device=DEV))  # the clip factor, on the device
    p = _flat(case, lambda n: _normal(n, g, 0.02))
    s["param"] = p if case["param"] == 32 else p.bfloat16()
    s["master"] = p if case["master"] else None
    if case["state"] == 32:
        s["m"] = _flat(case, lambda n: _normal(n, g, 2e-4))
        s["v"] = _flat(case, lambda n: _normal(n, g, 5e-4).square_())
    else:  # E4M3 elements of each block of 32 and the block's power of two
        s["m"] = _flat(case, lambda n: _normal(n, g, 120.0).clamp_(-448, 448)).to(torch.float8_e4m3fn)
        s["v"] = _flat(case, lambda n: _normal(n, g, 120.0).abs_().clamp_(0, 448)).to(torch.float8_e4m3fn)
        for name, low in (("m_scale", 127 - 20), ("v_scale", 127 - 19)):
            s[name] = torch.randint(low, low + 3, (total // 32,), generator=g, device=DEV, dtype=torch.uint8)
    if own:
        import mixture_experts_layer_table_gb300 as mok

        def cut(name):
            t = s.get(name)
            return None if t is None else [t[a:a + n] for a, n in _spans(case)[0]]

        def cut_scales(name):
            t = s.get(name)
            return None if t is None else [t[a // 32:a // 32 + (n + 31) // 32] for a, n in _spans(case)[0]]
        s["opt"] = mok.AdamW(cut("param"), cut("grad"), lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=WD,
                             state="f32" if case["state"] == 32 else "mx8", masters=cut("master"), seed=SEED,
                             step=s["step"],
                             states=dict(m=cut("m"), v=cut("v"), m_scale=cut_scales("m_scale"),
                                         v_scale=cut_scales("v_scale")),
                             counters=[a for a, _ in _spans(case)[0]])
    return s


def prepare(case, seed):
    make = {"route": _prepare_route, "route_backward": _prepare_route, "grad_norm": _prepare_norm,
            "adamw": _prepare_adamw}[case["op"]]
    return dict(make(case, seed), case=case)


# ------------------------------------------------------------------ plain forms

def _scores(x, router):
    """(scores, exp(x - max) or None): sigmoid, or softmax over the experts."""
    if router == SIGMOID:
        return 1.0 / (1.0 + torch.exp(-x)), None
    e = torch.exp(x - x.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True), e


def _select(x, bias, case):
    """Selected experts [T][k], best first, ties to the lower index, and the scores."""
    T, E, G, k = case["T"], case["E"], case["n_group"], case["k"]
    s, e = _scores(x, case["router"])
    # without a bias the softmax is ranked by its logits: it is increasing
    rank = x if e is not None and bias is None else s if bias is None else s + bias
    if G > 1:
        in_groups = (e if e is not None and bias is None and case["group"] == GROUP_TOP2 else rank).view(T, G, E // G)
        best = in_groups.sort(dim=2, descending=True, stable=True).values
        value = best[:, :, 0] if case["group"] == GROUP_MAX or E == G else best[:, :, 0] + best[:, :, 1]
        chosen = value.sort(dim=1, descending=True, stable=True).indices[:, :case["topk_group"]]
        keep = torch.zeros((T, G), dtype=torch.bool, device=x.device).scatter_(1, chosen, True)
        rank = torch.where(keep.repeat_interleave(E // G, 1), rank, -math.inf)
    return rank.sort(dim=1, descending=True, stable=True).indices[:, :k], s


def _run_route(s, case):
    x, T, E, k = s["logits"].float(), case["T"], case["E"], case["k"]
    idx, score = _select(x, s["bias"], case)
    chosen = score.gather(1, idx)
    out = dict(topk_idx=idx.int(), gates=chosen / chosen.sum(1, keepdim=True) * ROUTE_SCALE)
    if case["balance"]:
        counts = torch.zeros(E, dtype=torch.int32, device=x.device)
        counts.scatter_add_(0, idx.flatten(), torch.ones(T * k, dtype=torch.int32, device=x.device))
        q = score / score.sum(1, keepdim=True) if case["router"] == SIGMOID else score
        prob_sum = q.sum(0)
        dprob = counts.float() * (BALANCE_COEF * E / (k * float(T) * T))
        out |= dict(counts=counts, prob_sum=prob_sum, loss=(dprob * prob_sum).sum().view(1), dprob=dprob)
        if s["bias"] is not None:
            out["bias_next"] = s["bias"] + BIAS_RATE * torch.sign(T * k - E * counts.long()).float()
    return out


def _run_route_backward(s, case):
    x, idx = s["logits"].float(), s["idx"].long()
    p, _ = _scores(x, case["router"])
    chosen = p.gather(1, idx)
    total = chosen.sum(1, keepdim=True)
    ds = ROUTE_SCALE * (s["dgates"] - (s["dgates"] * chosen).sum(1, keepdim=True) / total) / total
    d = torch.zeros_like(p).scatter_(1, idx, ds)
    if case["router"] == SOFTMAX:
        d = d if s["dprob"] is None else d + s["dprob"]
        dl = p * (d - (p * d).sum(1, keepdim=True))
    else:
        if s["dprob"] is not None:
            all_ = p.sum(1, keepdim=True)
            d = d + (s["dprob"] - (p * s["dprob"]).sum(1, keepdim=True) / all_) / all_
        dl = d * p * (1.0 - p)
    return dl.to(s["logits"].dtype)


def _run_norm(s, case):
    norm = s["grad"].float().square().sum().sqrt()
    return torch.stack([norm, torch.clamp(MAX_NORM / (norm + 1e-6), max=1.0)])


def _mix(total, step):
    """32 pseudo-random bits of each element: murmur3's finaliser of its group of 8, times an odd number."""
    seed = (SEED ^ (step * 0x9E3779B1)) & 0xFFFFFFFF
    low = 0xFFFFFFFF
    x = torch.arange(total // 8, dtype=torch.int64, device=DEV) ^ seed
    x = ((x ^ (x >> 16)) * 0x85EBCA6B) & low
    x = ((x ^ (x >> 13)) * 0xC2B2AE35) & low
    x = x ^ (x >> 16)
    odd = torch.tensor([0x9E3779B1, 0x85EBCA77, 0xC2B2AE3D, 0x27D4EB2F, 0x165667B1, 0xD3A2646D, 0xFD7046C5, 0xB55A4F09],
                       dtype=torch.int64, device=DEV)
    return ((x[:, None] * odd) & low).flatten()


def _power_of_two(biased):
    """2^(biased - 127), from the exponent's bits."""
    return (biased.int() << 23).view(torch.float32)


def _to_e4m3(t, u, nonzero):
    """E4M3 elements and powers of two (E8M0 bytes) of blocks of 32; u in [0, 1) decides each rounding."""
    t, u = t.view(-1, 32), u.view(-1, 32)
    exponent = (((t.abs().amax(1).view(torch.int32) + 0x1FFFFF) >> 23) - 8).clamp(1, 254)
    y = t * _power_of_two(254 - exponent)[:, None]
    ulp = _power_of_two((y.view(torch.int32) >> 23 & 0xFF).clamp(min=121) - 3)  # 3 bits; 2^-9 below 2^-6
    q = torch.floor(y / ulp + u) * ulp
    if nonzero:
        q = torch.where(y > 0, q.clamp(min=2.0 ** -9), q)
    return q.clamp(-448, 448).to(torch.float8_e4m3fn).flatten(), exponent.to(torch.uint8)


def _from_e4m3(q, exponent):
    return (q.float().view(-1, 32) * _power_of_two(exponent)[:, None]).flatten()


def _run_adamw(s, case):
    s["step"] += 1
    bc1, bc2 = 1 - BETA1 ** s["step"], 1 - BETA2 ** s["step"]
    g = s["grad"].float() * s["scale"]
    eight = case["state"] == 8
    m = _from_e4m3(s["m"], s["m_scale"]) if eight else s["m"]
    v = _from_e4m3(s["v"], s["v_scale"]).square() if eight else s["v"]
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    p = s["master"] if case["master"] else s["param"].float()
    p = p - LR * ((m / bc1) / (torch.sqrt(v / bc2) + EPS) + WD * p)
    random = _mix(p.numel(), s["step"]) if eight or (case["param"] == 16 and not case["master"]) else None
    if eight:
        s["m"], s["m_scale"] = _to_e4m3(m, (random >> 9).float() * 2.0 ** -23, False)
        s["v"], s["v_scale"] = _to_e4m3(torch.sqrt(v), (random & 0x7FFFFF).float() * 2.0 ** -23, True)
    else:
        s["m"], s["v"] = m, v
    if case["master"]:
        s["master"], s["param"] = p, p.bfloat16()
    elif case["param"] == 16:  # the bits below bf16 decide, against 16 random ones, whether it is rounded up
        bits = (p.view(torch.int32).long() & 0xFFFFFFFF) + (random & 0xFFFF)
        s["param"] = (bits >> 16).to(torch.int16).view(torch.bfloat16)
    else:
        s["param"] = p
    return _adamw_outputs(s, case)


def _adamw_outputs(s, case):
    out = {n: s[n] for n in ("param", "m", "v")}
    if case["master"]:
        out["master"] = s["master"]
    if case["state"] == 8:  # the scales as the powers of two that they stand for
        out["m_scale"], out["v_scale"] = (s[n].view(torch.float8_e8m0fnu) for n in ("m_scale", "v_scale"))
    return out


def _run_own(s, case):
    if case["op"] == "route":
        r = s["router"].forward(s["logits"], s["bias"])
        names = ["topk_idx", "gates"]
        if case["balance"]:
            names += ["counts", "prob_sum", "loss", "dprob"] + (["bias_next"] if s["bias"] is not None else [])
        return {n: r[n] for n in names}
    if case["op"] == "route_backward":
        return s["router"].backward(s["logits"], s["idx"], s["dgates"], s["dprob"])
    if case["op"] == "grad_norm":
        return s["norm"].compute()
    s["opt"].step(s["scale"])
    return _adamw_outputs(s, case)


def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    return {"route": _run_route, "route_backward": _run_route_backward, "grad_norm": _run_norm,
            "adamw": _run_adamw}[case["op"]](state, case)


def work(case):
    if case["op"] in ("route", "route_backward"):
        n, sel, item = case["T"] * case["E"], case["T"] * case["k"], case["bits"] // 8
        if case["op"] == "route":
            return {"bytes": n * item + sel * 8 + case["E"] * (24 if case["balance"] else 4), "flops": 8 * n}
        return {"bytes": 2 * n * item + sel * 8 + case["E"] * 4, "flops": 10 * n}
    n = sum(_sizes(case))
    if case["op"] == "grad_norm":
        return {"bytes": n * case["grad"] // 8, "flops": 2 * n}
    each = case["grad"] / 8 + (10 if case["master"] else case["param"] / 4)
    each += 16 if case["state"] == 32 else 4 + 4 / 32
    return {"bytes": n * each, "flops": 16 * n}


# ------------------------------------------------------------------ 64 bits

def _exact_scores(x, router):
    if router == SIGMOID:
        return torch.where(x >= 0, 1 / (1 + torch.exp(-x.abs())), torch.exp(-x.abs()) / (1 + torch.exp(-x.abs())))
    return torch.exp(x - torch.logsumexp(x, 1, keepdim=True))


def _exact_route(s, case):
    x, E, k, T, G = s["logits"].double(), case["E"], case["k"], case["T"], case["n_group"]
    score = _exact_scores(x, case["router"])
    rank = score if s["bias"] is None else score + s["bias"].double()
    if G > 1:
        parts = rank.view(T, G, -1)
        value = parts.topk(2 if case["group"] == GROUP_TOP2 and E > G else 1, dim=2).values.sum(2)
        keep = torch.zeros_like(value).scatter_(1, value.topk(case["topk_group"], dim=1).indices, 1.0) > 0
        rank = parts.masked_fill(~keep[:, :, None], -math.inf).view(T, E)
    idx = torch.argsort(rank, dim=1, descending=True, stable=True)[:, :k]
    chosen = torch.take_along_dim(score, idx, 1)
    out = dict(topk_idx=None, gates=ROUTE_SCALE * chosen / chosen.sum(1, keepdim=True))
    if case["balance"]:
        counts = torch.bincount(idx.flatten(), minlength=E).double()
        prob = (score / score.sum(1, keepdim=True)).sum(0)
        dprob = BALANCE_COEF * E * counts / (k * T * T)
        out |= dict(counts=None, prob_sum=prob, loss=(dprob @ prob).view(1), dprob=dprob)
        if s["bias"] is not None:
            out["bias_next"] = s["bias"].double() + BIAS_RATE * torch.sign(k * T / E - counts)
    return out


def _exact_route_backward(s, case):
    """By the derivative of the gates and of the probabilities: torch's own, of the definition."""
    x = s["logits"].double().requires_grad_(True)
    with torch.enable_grad():
        score = torch.sigmoid(x) if case["router"] == SIGMOID else torch.softmax(x, 1)
        chosen = score.gather(1, s["idx"].long())
        f = (s["dgates"].double() * ROUTE_SCALE * chosen / chosen.sum(1, keepdim=True)).sum()
        if s["dprob"] is not None:
            f = f + (s["dprob"].double() * score / score.sum(1, keepdim=True)).sum()
    return torch.autograd.grad(f, x)[0]


def _exact_norm(s, case):
    n = torch.linalg.vector_norm(s["grad"].double())
    return torch.stack([n, torch.minimum(MAX_NORM / (n + 1e-6), torch.ones_like(n))])


def _exact_adamw(s, case):
    t = s["step"] + 1
    g = s["scale"].double() * s["grad"].double()
    if case["state"] == 8:
        two = {n: torch.exp2(s[n].double() - 127) for n in ("m_scale", "v_scale")}
        m0 = (s["m"].double().view(-1, 32) * two["m_scale"][:, None]).view(-1)
        v0 = (s["v"].double().view(-1, 32) * two["v_scale"][:, None]).view(-1) ** 2
    else:
        m0, v0 = s["m"].double(), s["v"].double()
    m = torch.lerp(g, m0, BETA1)
    v = torch.lerp(g * g, v0, BETA2)
    p0 = (s["master"] if case["master"] else s["param"]).double()
    p = p0 * (1 - LR * WD) - LR * (m / (1 - BETA1 ** t)) / (torch.sqrt(v / (1 - BETA2 ** t)) + EPS)
    out = dict(param=p, m=m, v=v)
    if case["param"] == 16 and not case["master"]:
        out["param"] = None  # rounded by random bits
    if case["master"]:
        out["master"] = p
    if case["state"] == 8:
        # elements are rounded by random bits; the scales are the least powers of two that reach 448 / amax
        out["m"] = out["v"] = None
        for name, w in (("m_scale", m), ("v_scale", v.sqrt())):
            top = w.abs().view(-1, 32).amax(1) / 448
            out[name] = torch.where(top > 0, torch.exp2(torch.ceil(torch.log2(top))), torch.full_like(top, 2.0 ** -126))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "route_backward": _exact_route_backward, "grad_norm": _exact_norm,
            "adamw": _exact_adamw}[case["op"]](s, case)
