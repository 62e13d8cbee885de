"""Cases, plain forms and 64-bit definitions of the operators around experts in 8-bit floating point.

Four operators:
  rows       tokens sorted by expert (``gather_rows``), back with their weights (``merge_rows``) and the
             gradient of that (``merge_rows_backward``)
  quantize   rows, or the SwiGLU of rows, or its gradient, as E4M3 with a scale for each 128 elements along the
             row and for each 128 rows of an expert (``fp8_quantize``), and weights with one for each
             128 x 128 (``Fp8Weights``)
  product    each expert's rows with its weights, x W^T or dy W (``Fp8Weights.matmul`` and
             ``matmul_transposed``); without groups it is a plain matrix product
  weight_grad  dW = dy^T x over each expert's rows (``fp8_weight_grad``)

``run`` computes an operator in elementary torch operations in 32 bits, or, with ``own`` set, with
the library's kernels; ``exact`` restates it in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
TOP = 448.0            # E4M3's largest value
LEAST = 2.0 ** -110    # a block's largest magnitude counts as at least this


def listed():
    return [
        # a batch with capacity: some assignments dropped, f32 rows of an odd width, zero rows behind the last
        dict(name="sort_odd", op="sort", T=1000, k=6, E=48, H=1111, bits=32, dropped=100),
        # one decoded token comes back from its 8 experts: latency
        dict(name="merge_token", op="merge", T=1, k=8, E=256, H=7168, bits=16, dropped=0),
        # the weighted merge of a training micro-batch
        dict(name="merge_train", op="merge", T=4096, k=8, E=256, H=7168, bits=16, dropped=0),
        # its gradient: the experts' rows and the gates
        dict(name="merge_grad_train", op="merge_grad", T=4096, k=8, E=256, H=7168, bits=16, dropped=0),
        # a few decoded tokens on their way to the first product
        dict(name="quantize_decode", op="quantize", source="plain", T=16, k=8, E=256, C=7168, bits=16, gathered=True,
             gated=False, columns=False),
        # the SwiGLU's gradient for the first product's two gradients: along the rows and along the tokens
        dict(name="quantize_swiglu_grad", op="quantize", source="swiglu_grad", T=2048, k=8, E=128, C=4096, bits=16,
             gathered=False, gated=False, columns=True),
        # 16 experts' first weights after an optimizer step, both orientations
        dict(name="quantize_weights", op="weights", E=16, N=4096, K=7168, bits=16),
        # 4 decoded tokens, second weights: each expert has a row or two
        dict(name="product_decode", op="product", T=4, k=8, E=64, N=7168, K=2048, bits=16, back=False),
        # a dense matrix of odd sizes (a shared expert's, say), no groups
        dict(name="product_dense_odd", op="product", T=1000, k=1, E=0, N=2050, K=2500, bits=32, back=False),
        # first weights of a training micro-batch, about 128 rows an expert
        dict(name="product_train", op="product", T=2048, k=8, E=128, N=4096, K=7168, bits=16, back=False),
        # the tiny layer's first weights: latency
        dict(name="weight_grad_tiny", op="weight_grad", T=256, k=2, E=8, N=1024, H=256, bits=32),
        # the same for a share of the experts of a training micro-batch
        dict(name="weight_grad_train", op="weight_grad", T=4096, k=8, E=32, N=4096, H=7168, bits=16),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sort", "merge", "merge_grad", "quantize", "weights", "product", "product", "product",
                     "weight_grad", "weight_grad"])
    E = _log_uniform(rng, 1, 256)
    k = rng.randint(1, min(16, E))
    bits = rng.choice([16, 32])
    width = lambda lo, hi: _log_uniform(rng, lo, hi) if rng.random() < 0.5 else 64 * _log_uniform(rng, 1, hi // 64)  # noqa: E731
    if op in ("sort", "merge", "merge_grad"):
        H = width(8, 7168)
        T = _log_uniform(rng, 1, min(65536, 200_000_000 // (k * H)))
        return dict(op=op, T=T, k=k, E=E, H=H, bits=bits, dropped=rng.choice([0, 0, 50, 500]))
    if op == "quantize":
        source = rng.choice(["plain", "swiglu", "swiglu_grad"])
        C = 2 * width(8, 2048) if source == "swiglu_grad" else width(8, 7168)
        T = _log_uniform(rng, 1, min(32768, 60_000_000 // (k * C)))
        gathered = source == "plain" and rng.random() < 0.5
        return dict(op=op, source=source, T=T, k=k, E=E, C=C, bits=bits, gathered=gathered,
                    gated=gathered and rng.random() < 0.5, columns=rng.random() < 0.5)
    if op == "weights":
        N, K = width(8, 7168), width(8, 7168)
        return dict(op=op, E=min(E, 400_000_000 // (N * K)), N=N, K=K, bits=bits)
    if op == "weight_grad":
        N, H = width(8, 4096), width(8, 4096)
        E = min(E, 400_000_000 // (N * H))
        k = min(k, E)
        T = _log_uniform(rng, 1, min(8192, 16384 // k, 150_000_000_000 // (k * N * H)))
        return dict(op=op, T=T, k=k, E=E, N=N, H=H, bits=bits)
    N, K = width(8, 7168), width(8, 7168)
    if rng.random() < 0.3:
        E, k = 0, 1
    E = min(E, 1_000_000_000 // (N * K))
    k = min(k, max(1, E))
    T = _log_uniform(rng, 1, min(8192, 16384 // k, 400_000_000_000 // (k * N * K)))
    return dict(op=op, T=T, k=k, E=E, N=N, K=K, bits=bits, back=rng.random() < 0.4)


# ------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(shape, g, std=1.0):
    return torch.empty(shape, dtype=torch.float32, device=DEV).normal_(0.0, std, generator=g)


def _type(bits):
    return torch.bfloat16 if bits == 16 else torch.float32


def _tokens(shape, g, dtype):
    """Activations: rows of unequal size."""
    return (_normal(shape, g) * torch.exp(_normal((shape[0], 1), g, 0.5))).to(dtype)


def _assignments(case, g):
    """(expert of each assignment [T][k], distinct in a token): experts of unequal popularity."""
    T, k, E = case["T"], case["k"], case["E"]
    if E < 2:
        return torch.zeros((T, k), dtype=torch.int64, device=DEV)
    noise = -torch.log(-torch.log(torch.rand((T, E), generator=g, device=DEV).clamp(1e-9, 1 - 1e-7)))
    return (noise + _normal((E,), g, 0.3)).topk(k, dim=1).indices


def _sorted_rows(case, g):
    """src_of, row_of and offsets of the stable order by expert.  Dropped assignments (per mille) have row -1; the
    rows behind the last one have source -1."""
    expert = _assignments(case, g).flatten()
    n = expert.numel()
    E = max(1, case["E"])
    dropped = torch.rand(n, generator=g, device=DEV) * 1000 < case.get("dropped", 0)
    key = torch.where(dropped, E, expert)
    src = key.sort(stable=True).indices
    row_of = torch.empty_like(src)
    row_of[src] = torch.arange(n, device=DEV)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=DEV).scatter_add_(0, key, torch.ones_like(key))[:E]
    kept = int(counts.sum())
    src[kept:] = -1
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = counts.cumsum(0).int()
    return src.int(), torch.where(dropped, -1, row_of).int(), offsets


def _gates(case, g):
    w = torch.rand((case["T"], case["k"]), generator=g, device=DEV) + 0.1
    return w / w.sum(1, keepdim=True)


def _blocks(n):
    return (n + 127) // 128


def _padded(n):
    """Bytes between rows of E4M3 elements: a multiple of 16."""
    return (n + 15) // 16 * 16


def _e4m3(shape):
    """An E4M3 buffer whose rows start at multiples of 16 bytes, zero-filled."""
    return torch.zeros((*shape[:-1], _padded(shape[-1])), dtype=torch.uint8, device=DEV).view(E4M3)[..., :shape[-1]]


def _stored(values):
    """Values as E4M3 in such a buffer."""
    t = _e4m3(values.shape)
    t.view(torch.uint8).copy_(values.to(E4M3).view(torch.uint8))
    return t


def _prepare_rows(case, g):
    s = dict(zip(("src_of", "row_of", "offsets"), _sorted_rows(case, g)))
    T, n, H, dtype = case["T"], case["T"] * case["k"], case["H"], _type(case["bits"])
    if case["op"] == "sort":
        s["x"] = _tokens((T, H), g, dtype)
        s["out"] = torch.empty((n, H), dtype=dtype, device=DEV)
        return s
    s["o"], s["gates"] = _tokens((n, H), g, dtype), _gates(case, g)
    if case["op"] == "merge":
        s["out"] = torch.empty((T, H), dtype=dtype, device=DEV)
        return s
    s["dy"] = _normal((T, H), g, 1.0 / T).to(dtype)
    # the rows behind the last one stay as they are
    s["out"] = dict(do=torch.zeros((n, H), dtype=dtype, device=DEV),
                    dgates=torch.empty((T, case["k"]), dtype=torch.float32, device=DEV))
    return s


def _prepare_quantize(case, g):
    s = dict(zip(("src_of", "row_of", "offsets"), _sorted_rows(case, g)))
    T, n, C, dtype = case["T"], case["T"] * case["k"], case["C"], _type(case["bits"])
    width = {"plain": C, "swiglu": 2 * C, "swiglu_grad": C}[case["source"]]
    s["x"] = _tokens((T if case["gathered"] else n, width), g, dtype)
    if case["source"] == "swiglu_grad":
        s["grad"] = _normal((n, C // 2), g, 1.0 / T).to(dtype)
    s["gates"] = _gates(case, g) if case["gated"] else None
    s["counts"] = (s["offsets"][1:] - s["offsets"][:-1]).tolist()
    s["out"] = dict(q=_e4m3((n, C)), scale=torch.zeros((_blocks(C), n), device=DEV))
    if case["columns"]:
        blocks = n // 128 + max(1, case["E"])
        s["out"] |= dict(qt=_e4m3((C, 128 * blocks)), qt_scale=torch.zeros((blocks, C), device=DEV))
    return s


def _prepare_weights(case, g):
    E, N, K = case["E"], case["N"], case["K"]
    w = torch.empty((E, N, K), dtype=_type(case["bits"]), device=DEV)
    for e in range(E):
        w[e] = _normal((N, K), g, 0.02)
    s = dict(w=w)
    if own:
        import mixture_experts_layer_table_gb300 as mok
        s["weights"] = mok.Fp8Weights.empty(E, N, K, transposed=True, device=DEV)
    else:
        s["out"] = dict(q=_e4m3((E, N, K)), scale=torch.empty((E, _blocks(N), _blocks(K)), device=DEV),
                        qt=_e4m3((E, K, N)), qt_scale=torch.empty((E, _blocks(K), _blocks(N)), device=DEV))
    return s


def _random_e4m3(shape, g):
    """What a block scaled to its largest magnitude holds: a normal spread of which few reach the top."""
    return _stored(_normal(shape, g, 150.0).clamp_(-TOP, TOP))


def _prepare_product(case, g):
    offsets = _sorted_rows(case, g)[2]
    n, E, N, K = case["T"] * case["k"], max(1, case["E"]), case["N"], case["K"]
    s = dict(offsets=offsets if case["E"] else None, counts=(offsets[1:] - offsets[:-1]).tolist())
    s["x"] = _random_e4m3((n, K), g)
    s["x_scale"] = torch.exp(_normal((_blocks(K), n), g, 0.3)) * 0.006
    # the weights as they are stored, [E][N][K], and the transposed ones for the way back, [E][K][N]
    a, b = (K, N) if case["back"] else (N, K)
    w = _e4m3((E, a, b))
    for e in range(E):
        w.view(torch.uint8)[e] = _normal((a, b), g, 150.0).clamp_(-TOP, TOP).to(E4M3).view(torch.uint8)
    w_scale = torch.exp(_normal((E, _blocks(a), _blocks(b)), g, 0.3)) * 1e-4
    if case["back"]:  # rows of width K meet W [K][N]
        s["wt"], s["wt_scale"] = _transposed(w), w_scale.transpose(1, 2).contiguous()
    else:
        s["wt"], s["wt_scale"] = w, w_scale
    s["out"] = torch.empty((n, N), dtype=_type(case["bits"]), device=DEV)
    if own:
        import mixture_experts_layer_table_gb300 as mok
        if case["back"]:
            s["weights"] = mok.Fp8Weights.of(w, w_scale, s["wt"], s["wt_scale"])
        else:
            s["weights"] = mok.Fp8Weights.of(w, w_scale)
    return s


def _transposed(w):
    t = _e4m3((w.shape[0], w.shape[2], w.shape[1]))
    t.view(torch.uint8).copy_(w.view(torch.uint8).transpose(1, 2))
    return t


def _prepare_weight_grad(case, g):
    offsets = _sorted_rows(case, g)[2]
    n, E, N, H = case["T"] * case["k"], case["E"], case["N"], case["H"]
    blocks = n // 128 + E
    s = dict(offsets=offsets, counts=(offsets[1:] - offsets[:-1]).tolist())
    # each expert's rows from a multiple of 128 on, zeros behind its last
    valid = torch.zeros(128 * blocks, dtype=torch.bool, device=DEV)
    at = 0
    for c in s["counts"]:
        valid[at:at + c] = True
        at += 128 * _blocks(c)
    for name, width, size in (("dy", N, 1e-6), ("x", H, 0.006)):
        t = _random_e4m3((width, 128 * blocks), g)
        t.view(torch.uint8).mul_(valid)
        s[name], s[name + "_scale"] = t, torch.exp(_normal((blocks, width), g, 0.3)) * size
    s["out"] = torch.empty((E, N, H), dtype=_type(case["bits"]), device=DEV)
    return s


def prepare(case, seed):
    make = {"sort": _prepare_rows, "merge": _prepare_rows, "merge_grad": _prepare_rows, "quantize": _prepare_quantize,
            "weights": _prepare_weights, "product": _prepare_product, "weight_grad": _prepare_weight_grad}[case["op"]]
    return dict(make(case, _generator(seed)), case=case)


# ------------------------------------------------------------------ plain forms

def _gathered(x, src_of, k, gates):
    """Rows x[src_of / k] in 32 bits, times their gates; zero where there is no source."""
    src = src_of.long()
    rows = x[src.clamp(min=0) // k].float()
    if gates is not None:
        rows = rows * gates.flatten()[src.clamp(min=0)][:, None]
    return torch.where((src >= 0)[:, None], rows, 0.0)


def _run_sort(s, case):
    s["out"].copy_(_gathered(s["x"], s["src_of"], case["k"], None))
    return s["out"]


def _run_merge(s, case):
    T, k = case["T"], case["k"]
    row = s["row_of"].long().view(T, k)
    acc = torch.zeros((T, case["H"]), device=DEV)
    for j in range(k):
        w = torch.where(row[:, j] >= 0, s["gates"][:, j], 0.0)
        acc += w[:, None] * s["o"][row[:, j].clamp(min=0)].float()
    s["out"].copy_(acc)
    return s["out"]


def _run_merge_grad(s, case):
    T, k = case["T"], case["k"]
    row = s["row_of"].long().view(T, k)
    dy = s["dy"].float()
    for j in range(k):
        has = row[:, j] >= 0
        dot = (dy * s["o"][row[:, j].clamp(min=0)].float()).sum(1)
        s["out"]["dgates"][:, j] = torch.where(has, dot, 0.0)
        s["out"]["do"][row[has, j]] = (s["gates"][:, j:j + 1] * dy)[has].to(s["dy"].dtype)
    return s["out"]


def _to_e4m3(x, dims):
    """x [..., 128-blocks cut out along `dims`] as E4M3 and the blocks' scales amax / 448.  448 x / amax is formed as
    (448 x / 512) / (amax / 512), both exact for bf16: a quotient on a border of the rounding stays on it."""
    amax = x.abs().amax(dims, keepdim=True).clamp(min=LEAST)
    return ((x * (TOP / 512)) / (amax / 512)).clamp(-TOP, TOP).to(E4M3), amax / TOP


def _padded_to(x, rows, cols):
    if x.shape[-2:] == (rows, cols):
        return x
    t = torch.zeros((*x.shape[:-2], rows, cols), dtype=x.dtype, device=x.device)
    t[..., :x.shape[-2], :x.shape[-1]] = x
    return t


def _source(s, case):
    """The values to quantise, in 32 bits."""
    if case["source"] == "plain":
        if case["gathered"]:
            return _gathered(s["x"], s["src_of"], case["k"], s["gates"])
        return s["x"].float()
    half = s["x"].shape[1] // 2
    h, u = s["x"][:, :half].float(), s["x"][:, half:].float()
    sg = 1.0 / (1.0 + torch.exp(-h))
    if case["source"] == "swiglu":
        return h * sg * u
    da = s["grad"].float()
    return torch.cat([da * u * sg * (1.0 + h * (1.0 - sg)), da * h * sg], 1)


def _run_quantize(s, case):
    x, out, C = _source(s, case), s["out"], case["C"]
    n, B = x.shape[0], _blocks(C)
    q, scale = _to_e4m3(_padded_to(x, n, 128 * B).view(n, B, 128), (2,))
    out["q"].view(torch.uint8).copy_(q.view(torch.uint8).view(n, 128 * B)[:, :C])
    out["scale"].copy_(scale.view(n, B).T)
    if case["columns"]:
        row = at = 0
        for c in s["counts"]:
            if c:
                m = _blocks(c)
                q, scale = _to_e4m3(_padded_to(x[row:row + c], 128 * m, C).view(m, 128, C), (1,))
                out["qt"].view(torch.uint8)[:, at:at + 128 * m] = q.view(torch.uint8).view(128 * m, C).T
                out["qt_scale"][at // 128:at // 128 + m] = scale.view(m, C)
                row, at = row + c, at + 128 * m
    return out


def _run_weights(s, case):
    E, N, K = case["E"], case["N"], case["K"]
    n, m, out = _blocks(N), _blocks(K), s["out"]
    for e in range(E):
        q, scale = _to_e4m3(_padded_to(s["w"][e].float(), 128 * n, 128 * m).view(n, 128, m, 128), (1, 3))
        q = q.view(torch.uint8).view(128 * n, 128 * m)[:N, :K]
        out["q"].view(torch.uint8)[e] = q
        out["qt"].view(torch.uint8)[e] = q.T
        out["scale"][e] = scale.view(n, m)
        out["qt_scale"][e] = scale.view(n, m).T
    return out


def _run_product(s, case):
    out, row = s["out"], 0
    n, K, N = case["T"] * case["k"], case["K"], case["N"]
    x = s["x"].float() * s["x_scale"].T.repeat_interleave(128, 1)[:, :K]
    for e, c in enumerate(s["counts"]):
        if c:
            scale = s["wt_scale"][e].repeat_interleave(128, 0).repeat_interleave(128, 1)[:N, :K]
            out[row:row + c] = x[row:row + c] @ (s["wt"][e].float() * scale).T
            row += c
    return out


def _run_weight_grad(s, case):
    at = 0
    dy = s["dy"].float() * s["dy_scale"].T.repeat_interleave(128, 1)
    x = s["x"].float() * s["x_scale"].T.repeat_interleave(128, 1)
    for e, c in enumerate(s["counts"]):
        p = 128 * _blocks(c)
        s["out"][e] = dy[:, at:at + p] @ x[:, at:at + p].T
        at += p
    return s["out"]


def _run_own(s, case):
    import mixture_experts_layer_table_gb300 as mok
    op = case["op"]
    if op == "sort":
        return mok.gather_rows(s["x"], s["src_of"], case["k"], out=s["out"])
    if op == "merge":
        return mok.merge_rows(s["o"], s["row_of"], case["k"], s["gates"], out=s["out"])
    if op == "merge_grad":
        return mok.merge_rows_backward(s["dy"], s["o"], s["row_of"], s["gates"], out=s["out"])
    if op == "quantize":
        return mok.fp8_quantize(s["x"], source=case["source"], grad=s.get("grad"),
                                src_of=s["src_of"] if case["gathered"] else None, k=case["k"], gates=s["gates"],
                                offsets=s["offsets"] if case["columns"] else None, out=s["out"])
    if op == "weights":
        w = s["weights"].quantize(s["w"])
        return dict(q=w.q, scale=w.scale, qt=w.qt, qt_scale=w.qt_scale)
    if op == "product":
        call = s["weights"].matmul_transposed if case["back"] else s["weights"].matmul
        return call(s["x"], s["x_scale"], s["offsets"], out=s["out"])
    return mok.fp8_weight_grad(s["dy"], s["dy_scale"], s["x"], s["x_scale"], s["offsets"], out=s["out"])


def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    return {"sort": _run_sort, "merge": _run_merge, "merge_grad": _run_merge_grad, "quantize": _run_quantize,
            "weights": _run_weights, "product": _run_product, "weight_grad": _run_weight_grad}[case["op"]](state, case)


def work(case):
    op, item = case["op"], case["bits"] // 8
    if op == "weights":
        n = case["E"] * case["N"] * case["K"]
        return {"bytes": n * (item + 2) + 8 * case["E"] * _blocks(case["N"]) * _blocks(case["K"]), "flops": 2 * n}
    T, n = case["T"], case["T"] * case["k"]
    if op in ("sort", "merge", "merge_grad"):
        H, kept = case["H"], n * (1000 - case["dropped"]) // 1000
        rows, tokens = kept * H * item, T * H * item
        if op == "sort":
            return {"bytes": n * H * item + tokens + 4 * n, "flops": n * H}
        if op == "merge":
            return {"bytes": rows + tokens + 8 * n, "flops": 2 * n * H}
        return {"bytes": 2 * rows + tokens + 12 * n, "flops": 3 * n * H}
    if op == "quantize":
        C = case["C"]
        read = {"plain": (T if case["gathered"] else n) * C, "swiglu": 2 * n * C, "swiglu_grad": n * C * 3 // 2}
        wrote = (2 if case["columns"] else 1) * (n * C + 4 * n * _blocks(C))
        return {"bytes": read[case["source"]] * item + wrote, "flops": 4 * n * C}
    N, E = case["N"], max(1, case["E"])
    if op == "product":
        K = case["K"]
        touched = E * (1 - (1 - 1 / E) ** n) if E > 1 else 1  # experts that have rows
        return {"bytes": n * K + touched * N * K + n * N * item + 4 * n * _blocks(K), "flops": 2 * n * N * K}
    H = case["H"]
    return {"bytes": n * (N + H) + E * N * H * item + 4 * _blocks(n) * (N + H), "flops": 2 * n * N * H}


# ------------------------------------------------------------------ 64 bits

def _exact_rows(s, case):
    T, k, H, n = case["T"], case["k"], case["H"], case["T"] * case["k"]
    if case["op"] == "sort":
        out = torch.zeros((n, H), dtype=torch.float64, device=DEV)
        a = torch.arange(n, device=DEV)[s["row_of"] >= 0]
        out[s["row_of"].long()[a]] = s["x"].double()[a // k]
        return out
    row, gates = s["row_of"].long(), s["gates"].double().flatten()
    a = torch.arange(n, device=DEV)[row >= 0]
    if case["op"] == "merge":
        out = torch.zeros((T, H), dtype=torch.float64, device=DEV)
        for lo in range(0, a.numel(), 4096):  # one assignment after the other into its token
            part = a[lo:lo + 4096]
            out.index_add_(0, part // k, gates[part][:, None] * s["o"][row[part]].double())
        return out
    do = torch.zeros((n, H), dtype=torch.float64, device=DEV)
    dgates = torch.zeros(n, dtype=torch.float64, device=DEV)
    for lo in range(0, a.numel(), 4096):
        part = a[lo:lo + 4096]
        dy = s["dy"].double()[part // k]
        do[row[part]] = gates[part][:, None] * dy
        dgates[part] = torch.einsum("ah,ah->a", dy, s["o"][row[part]].double())
    return dict(do=do, dgates=dgates.view(T, k))


def _round_e4m3(y):
    """The E4M3 value nearest to y, ties to even: 3 bits after the leading one, multiples of 2^-9 below 2^-6."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.clamp(torch.round(y / step) * step, -TOP, TOP)


def _exact_source(s, case):
    x = s["x"].double()
    if case["source"] == "plain":
        if not case["gathered"]:
            return x
        src = s["src_of"].long()
        rows = x[torch.div(src, case["k"], rounding_mode="floor").clamp(min=0)]
        if s["gates"] is not None:
            rows = rows * s["gates"].double().view(-1, 1)[src.clamp(min=0)]
        return rows * (src >= 0).double()[:, None]
    h, u = x.chunk(2, 1)
    if case["source"] == "swiglu":
        return torch.nn.functional.silu(h) * u
    da, sg = s["grad"].double(), torch.sigmoid(h)
    return torch.cat([da * u * (sg + h * sg * torch.sigmoid(-h)), da * (h * sg)], 1)


def _exact_quantize(s, case):
    x, C, n = _exact_source(s, case), case["C"], case["T"] * case["k"]
    out = dict(q=torch.empty((n, C), dtype=torch.float64, device=DEV),
               scale=torch.empty((_blocks(C), n), dtype=torch.float64, device=DEV))
    for b in range(_blocks(C)):
        part = x[:, 128 * b:128 * (b + 1)]
        amax = part.abs().max(1).values.clamp(min=LEAST)
        out["q"][:, 128 * b:128 * (b + 1)] = _round_e4m3(part * TOP / amax[:, None])
        out["scale"][b] = amax / TOP
    if case["columns"]:
        blocks = n // 128 + max(1, case["E"])
        qt = torch.zeros((C, 128 * blocks), dtype=torch.float64, device=DEV)
        qt_scale = torch.zeros((blocks, C), dtype=torch.float64, device=DEV)
        block = 0
        for e in range(max(1, case["E"])):
            lo, hi = int(s["offsets"][e]), int(s["offsets"][e + 1])
            for r in range(lo, hi, 128):
                part = x[r:min(r + 128, hi)].T
                amax = part.abs().max(1).values.clamp(min=LEAST)
                qt[:, 128 * block:128 * block + part.shape[1]] = _round_e4m3(part * TOP / amax[:, None])
                qt_scale[block] = amax / TOP
                block += 1
        out |= dict(qt=qt, qt_scale=qt_scale)
    return out


def _exact_weights(s, case):
    E, N, K = case["E"], case["N"], case["K"]
    out = dict(q=torch.empty((E, N, K), dtype=torch.float64, device=DEV),
               scale=torch.empty((E, _blocks(N), _blocks(K)), dtype=torch.float64, device=DEV))
    for i in range(_blocks(N)):
        for j in range(_blocks(K)):
            part = s["w"][:, 128 * i:128 * i + 128, 128 * j:128 * j + 128].double()
            amax = part.abs().flatten(1).max(1).values.clamp(min=LEAST)
            out["q"][:, 128 * i:128 * i + 128, 128 * j:128 * j + 128] = _round_e4m3(part * TOP / amax[:, None, None])
            out["scale"][:, i, j] = amax / TOP
    return dict(out, qt=out["q"].transpose(1, 2), qt_scale=out["scale"].transpose(1, 2))


def _exact_product(s, case):
    """The sum over the blocks of 128 of (scale of the row) (scale of the weights) (elements' product)."""
    n, K, N = case["T"] * case["k"], case["K"], case["N"]
    out = torch.zeros((n, N), dtype=torch.float64, device=DEV)
    row = 0
    for e, c in enumerate(s["counts"]):
        for b in range(_blocks(K)) if c else ():
            cut = slice(128 * b, min(K, 128 * b + 128))
            xs = s["x_scale"][b, row:row + c].double()
            ws = s["wt_scale"][e, :, b].double().repeat_interleave(128)[:N]
            out[row:row + c] += torch.outer(xs, ws) * (s["x"][row:row + c, cut].double() @ s["wt"][e][:, cut].double().T)
        row += c
    return out


def _exact_weight_grad(s, case):
    out = torch.zeros((case["E"], case["N"], case["H"]), dtype=torch.float64, device=DEV)
    block = 0
    for e, c in enumerate(s["counts"]):
        for _ in range(_blocks(c)):
            cut = slice(128 * block, 128 * block + 128)
            scales = torch.outer(s["dy_scale"][block].double(), s["x_scale"][block].double())
            out[e] += scales * (s["dy"][:, cut].double() @ s["x"][:, cut].double().T)
            block += 1
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"sort": _exact_rows, "merge": _exact_rows, "merge_grad": _exact_rows, "quantize": _exact_quantize,
            "weights": _exact_weights, "product": _exact_product, "weight_grad": _exact_weight_grad}[case["op"]](s, case)
