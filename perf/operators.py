"""The training-side operators around a DeepSeekMoE layer, as cases that can be timed and checked.

Three families: products grouped by expert over ragged rows (``mm``, ``dgrad``, ``wgrad``), the
norms before and after a block fused with its gate and residual scale (``norm``, ``norm_bwd``),
and the global gradient norm with clipping (``gnorm``, ``clip``).  ``own`` chooses between the
plain torch form (False) and the library's calls (True).  Sizes are those of the layer
configurations in ``workloads.CONFIGS`` or generic ones.
"""
import math

import torch

own = False

EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # ------------------------------------------------ products grouped by expert
        # the fp32 "tiny" layer's gate projection: 15 experts, three choices of 128 tokens
        {"name": "mm_tiny_fp32", "op": "mm", "dtype": "fp32", "groups": 15, "rows": 384, "tail": 0,
         "n": 128, "k": 256, "load": "routed"},
        # one decode step of the 16B layer's gate and up projections: 64 tokens, six experts each
        {"name": "mm_decode", "op": "mm", "dtype": "bf16", "groups": 64, "rows": 384, "tail": 0,
         "n": 2816, "k": 2048, "load": "routed"},
        # the 16B layer's gate and up projections over a prompt of 16384 tokens
        {"name": "mm_prefill", "op": "mm", "dtype": "bf16", "groups": 64, "rows": 98304, "tail": 0,
         "n": 2816, "k": 2048, "load": "routed"},
        # the 2B layer's gate projection, gradient of its input; a receive buffer that is not full
        {"name": "dgrad_2b", "op": "dgrad", "dtype": "bf16", "groups": 63, "rows": 57344, "tail": 1001,
         "n": 896, "k": 1280, "load": "routed"},
        # the 16B layer's gate projection, gradient of its weights, experts loaded unevenly
        {"name": "wgrad_16b", "op": "wgrad", "dtype": "bf16", "groups": 64, "rows": 49152, "tail": 0,
         "n": 1408, "k": 2048, "load": "skewed"},
        # ------------------------------------------------ norms around a block
        # one decode step of the 16B layer's block
        {"name": "norm_decode", "op": "norm", "dtype": "bf16", "rows": 64, "d": 2048,
         "gate": "channel", "post": True, "pre": True},
        # a long prompt through the 145B layer's block
        {"name": "norm_prefill", "op": "norm", "dtype": "bf16", "rows": 32768, "d": 4096,
         "gate": "channel", "post": True, "pre": True},
        # training step of the 2B layer's block, one gate value per token
        {"name": "norm_bwd_2b", "op": "norm_bwd", "dtype": "bf16", "rows": 8192, "d": 1280,
         "gate": "token", "post": True, "pre": True},
        # an fp32 block of an odd width and length, no norm after it
        {"name": "norm_bwd_odd", "op": "norm_bwd", "dtype": "fp32", "rows": 1001, "d": 333,
         "gate": "channel", "post": False, "pre": True},
        # ------------------------------------------------ gradient norm and clipping
        # many small tensors of both types (norms, gates, biases, adapters): launches count
        {"name": "clip_many", "op": "clip", "dtype": "mixed", "layout": "many", "tensors": 600,
         "least": 1, "most": 9000, "over": True},
        # the norm alone of the 2B layer's fp32 gradients (logging, or a step that is not clipped)
        {"name": "gnorm_2b", "op": "gnorm", "dtype": "fp32", "layout": "layer", "experts": 64,
         "inter": 896, "d": 1280, "routed": 63, "over": False},
        # the 16B layer's fp32 gradients, clipped
        {"name": "clip_16b", "op": "clip", "dtype": "fp32", "layout": "layer", "experts": 66,
         "inter": 1408, "d": 2048, "routed": 64, "over": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    family = rng.choice(["grouped", "grouped", "norm", "clip"])
    if family == "grouped":
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        most = 1e12 if dtype == "bf16" else 4e9
        side = 4096 if dtype == "bf16" else 1024
        case = {"op": rng.choice(["mm", "dgrad", "wgrad"]), "dtype": dtype, "groups": _log_int(rng, 1, 128),
                "n": _log_int(rng, 33, side), "k": _log_int(rng, 33, side),
                "load": rng.choice(["routed", "skewed", "sparse"])}
        if rng.random() < 0.75:   # the usual widths are multiples of 8
            case["n"], case["k"] = (case["n"] + 7) // 8 * 8, (case["k"] + 7) // 8 * 8
        else:                     # other widths take a slower road: a share of the work
            most = min(most, 4e10)
        while case["groups"] * case["n"] * case["k"] > 3e8:
            case["groups"] = max(1, case["groups"] // 2)
        top = max(2, min(131072, int(most / (2 * case["n"] * case["k"]))))
        case["rows"] = _log_int(rng, 1, top)
        case["tail"] = rng.choice([0, 0, _log_int(rng, 1, 500)])
        return case
    if family == "norm":
        d = _log_int(rng, 17, 8192)
        if rng.random() < 0.7:
            d = (d + 7) // 8 * 8
        pre = rng.random() < 0.8
        return {"op": rng.choice(["norm", "norm_bwd"]), "dtype": rng.choice(["bf16", "bf16", "fp32"]),
                "rows": _log_int(rng, 1, min(65536, int(6e7 / d))), "d": d,
                "gate": rng.choice(["none", "channel", "token"]), "post": rng.random() < 0.7, "pre": pre}
    case = {"op": rng.choice(["clip", "clip", "gnorm"]), "dtype": rng.choice(["fp32", "bf16", "mixed"]),
            "over": rng.random() < 0.7}
    if rng.random() < 0.5:
        case.update(layout="many", tensors=_log_int(rng, 1, 2500), least=1, most=_log_int(rng, 100, 60000))
    else:
        case.update(layout="layer", experts=_log_int(rng, 2, 64), inter=_log_int(rng, 64, 1500),
                    d=_log_int(rng, 64, 2048), routed=_log_int(rng, 2, 64))
    return case


# ------------------------------------------------------------------------------ inputs
def _counts(case, gen):
    """Rows of each expert, summing to `rows`: a router's mild spread, a skewed one, or one
    that leaves most experts without any."""
    g = case["groups"]
    if case["load"] == "routed":
        p = torch.softmax(0.3 * torch.randn(g, generator=gen), 0)
    elif case["load"] == "skewed":
        p = (1.0 / torch.arange(1, g + 1).float() ** 1.1)[torch.randperm(g, generator=gen)]
    else:
        p = torch.zeros(g)
        p[torch.randperm(g, generator=gen)[:max(1, g // 8)]] = 1.0
    ids = torch.multinomial(p, case["rows"], replacement=True, generator=gen)
    return torch.bincount(ids, minlength=g)


def _tensors(case):
    """Shapes and types of the gradients: a model's do not change from step to step."""
    gen = torch.Generator().manual_seed(17)
    if case["layout"] == "layer":   # the outputs of the layer's backward
        e, i, d, r = case["experts"], case["inter"], case["d"], case["routed"]
        sizes = [(e, i, d), (e, i, d), (e, d, i), (r, d), (r,)]
    else:   # lengths spread evenly over their logarithm
        lo, hi = math.log(case["least"]), math.log(case["most"])
        u = torch.rand(case["tensors"], generator=gen)
        sizes = [(int(round(math.exp(lo + float(x) * (hi - lo)))),) for x in u]
    p = torch.rand(len(sizes), generator=gen)
    half = {"bf16": 1.0, "fp32": 0.0, "mixed": 0.5}[case["dtype"]]
    return sizes, [torch.bfloat16 if float(x) < half else torch.float32 for x in p]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator().manual_seed(seed)
    gpu = torch.Generator(device=dev).manual_seed(seed)
    op = case["op"]

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=gpu, device=dev) * std).to(dtype)

    st = dict(case)
    if op in ("mm", "dgrad", "wgrad"):
        dt, g, n, k = TYPES[case["dtype"]], case["groups"], case["n"], case["k"]
        cap = case["rows"] + case["tail"]
        counts = _counts(case, gen)
        st["splits"] = counts.tolist()
        st["counts"] = counts.to(dev, torch.int32)
        if op != "dgrad":
            st["x"] = normal(cap, k, dtype=dt)
        if op != "mm":
            st["dy"] = normal(cap, n, std=0.05, dtype=dt)
        if op != "wgrad":
            st["w"] = normal(g, n, k, std=0.02, dtype=dt)
        if op == "wgrad":
            st["out"] = torch.empty(g, n, k, device=dev)
        else:   # rows behind the last expert's keep what they hold
            st["out"] = torch.zeros(cap, n if op == "mm" else k, dtype=dt, device=dev)
    elif op in ("norm", "norm_bwd"):
        dt, t, d = TYPES[case["dtype"]], case["rows"], case["d"]
        st["x"] = normal(t, d, std=3.0, dtype=dt)
        st["y"] = normal(t, d, std=0.7, dtype=dt)
        st["gate_t"] = {"none": None, "channel": lambda: 0.1 + normal(d, std=0.05),
                        "token": lambda: torch.sigmoid(normal(t, 1))}[case["gate"]]
        st["gate_t"] = st["gate_t"]() if st["gate_t"] else None
        st["post_w"] = 1.0 + normal(d, std=0.1) if case["post"] else None
        st["pre_w"] = 1.0 + normal(d, std=0.1) if case["pre"] else None
        st["beta"] = 1.5
        if op == "norm_bwd":   # what the forward leaves: its residual stream and statistics
            r, _, st["post_rstd"], st["pre_rstd"] = _plain_norm(st)
            st["r"] = r
            st["dr"] = normal(t, d, std=0.1, dtype=dt)
            st["du"] = normal(t, d, std=0.1, dtype=dt) if case["pre"] else None
    else:
        sizes, dts = _tensors(case)
        total = sum(math.prod(s) for s in sizes)
        std = 1e-3
        st["max_norm"] = std * math.sqrt(total) * (0.37 if case["over"] else 3.0)
        if case["layout"] == "many":   # parts of one buffer per type, as a bucketed optimiser keeps them
            flat = {dt: normal(sum(math.prod(s) for s, q in zip(sizes, dts) if q == dt), std=std, dtype=dt)
                    for dt in sorted(set(dts), key=str)}
            st["flat_out"] = {dt: torch.zeros_like(f) for dt, f in flat.items()}

            def parts(bufs):
                at = {dt: 0 for dt in bufs}
                got = []
                for s, dt in zip(sizes, dts):
                    m = math.prod(s)
                    got.append(bufs[dt][at[dt]:at[dt] + m])
                    at[dt] += m
                return got

            st["grads"], st["outs"] = parts(flat), parts(st["flat_out"])
        else:
            st["grads"] = [normal(*s, std=std, dtype=dt) for s, dt in zip(sizes, dts)]
            st["outs"] = [torch.empty_like(g) for g in st["grads"]] if op == "clip" else None
    return st


# ------------------------------------------------------------------------------ plain forms
def _plain_grouped(st):
    splits, op, out = st["splits"], st["op"], st["out"]
    rows = st["rows"]
    if op == "mm":
        parts = [x.float() @ w.float().t() for x, w in zip(st["x"][:rows].split(splits), st["w"])]
    elif op == "dgrad":
        parts = [dy.float() @ w.float() for dy, w in zip(st["dy"][:rows].split(splits), st["w"])]
    else:
        return torch.stack([dy.float().t() @ x.float()
                            for dy, x in zip(st["dy"][:rows].split(splits), st["x"][:rows].split(splits))], out=out)
    out[:rows] = torch.cat(parts).to(out.dtype)
    return out


def _plain_norm(st):
    """r = beta x + gate * norm(y) and u = norm(r), with 1 / rms of y and of r."""
    x, y = st["x"].float(), st["y"].float()
    post_rstd = pre_rstd = u = None
    if st["post_w"] is not None:
        post_rstd = torch.rsqrt(y.square().mean(1) + EPS)
        y = y * post_rstd[:, None] * st["post_w"]
    if st["gate_t"] is not None:
        y = y * st["gate_t"]
    r = st["beta"] * x + y
    if st["pre_w"] is not None:
        pre_rstd = torch.rsqrt(r.square().mean(1) + EPS)
        u = (r * pre_rstd[:, None] * st["pre_w"]).to(st["x"].dtype)
    return r.to(st["x"].dtype), u, post_rstd, pre_rstd


def _plain_norm_bwd(st):
    dt = st["x"].dtype
    g, y = st["dr"].float(), st["y"].float()
    d_pre = d_post = d_gate = None
    if st["pre_w"] is not None:
        xhat = st["r"].float() * st["pre_rstd"][:, None]
        du = st["du"].float()
        d_pre = (du * xhat).sum(0)
        dh = du * st["pre_w"]
        g = g + st["pre_rstd"][:, None] * (dh - xhat * (dh * xhat).mean(1, keepdim=True))
    dx = (st["beta"] * g).to(dt)
    yhat = y * st["post_rstd"][:, None] if st["post_w"] is not None else y
    b = yhat * st["post_w"] if st["post_w"] is not None else yhat
    db = g
    if st["gate_t"] is not None:
        db = g * st["gate_t"]
        d_gate = (g * b).sum(0) if st["gate"] == "channel" else (g * b).sum(1, keepdim=True)
    if st["post_w"] is not None:
        d_post = (db * yhat).sum(0)
        dh = db * st["post_w"]
        db = st["post_rstd"][:, None] * (dh - yhat * (dh * yhat).mean(1, keepdim=True))
    return dx, db.to(dt), d_gate, d_post, d_pre


def _plain_clip(st):
    total = torch.stack([g.double().square().sum() for g in st["grads"]]).sum()
    norm = total.sqrt()
    if st["op"] == "clip":
        coef = torch.clamp(st["max_norm"] / norm, max=1.0).float()
        [o.copy_(g.float() * coef) for o, g in zip(st["outs"], st["grads"])]
    return norm.float().reshape(1)


def run(state):
    st, op = state, state["op"]
    if op in ("mm", "dgrad", "wgrad"):
        if own:
            from mixture_experts_layer_65_b200 import grouped
            if op == "mm":
                return grouped.grouped_mm(st["x"], st["w"], st["counts"], out=st["out"])
            if op == "dgrad":
                return grouped.grouped_mm_dgrad(st["dy"], st["w"], st["counts"], out=st["out"])
            return grouped.grouped_mm_wgrad(st["dy"], st["x"], st["counts"], out=st["out"])
        return _plain_grouped(st)
    if op == "norm":
        if own:
            from mixture_experts_layer_65_b200 import block
            return tuple(block.block_norm(st["x"], st["y"], gate=st["gate_t"], post_weight=st["post_w"],
                                          pre_weight=st["pre_w"], beta=st["beta"], eps=EPS))
        return _plain_norm(st)
    if op == "norm_bwd":
        if own:
            from mixture_experts_layer_65_b200 import block
            fwd = block.BlockNorm(st["r"], None, st["post_rstd"], st["pre_rstd"])
            return tuple(block.block_norm_backward(
                fwd, st["y"], dr=st["dr"], du=st["du"], gate=st["gate_t"], post_weight=st["post_w"],
                pre_weight=st["pre_w"], beta=st["beta"]))
        return _plain_norm_bwd(st)
    if own:
        from mixture_experts_layer_65_b200 import clip
        if op == "gnorm":
            return clip.grad_norm(st["grads"])
        norm = clip.clip_grad_norm(st["grads"], st["max_norm"], out=st["outs"])
    else:
        norm = _plain_clip(st)
    if op == "gnorm":
        return norm
    return (norm, st["flat_out"][torch.bfloat16] if torch.bfloat16 in st["flat_out"] else None,
            st["flat_out"][torch.float32] if torch.float32 in st["flat_out"] else None) \
        if st["layout"] == "many" else (norm, *st["outs"])


# ------------------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    if op in ("mm", "dgrad", "wgrad"):
        es = 2 if case["dtype"] == "bf16" else 4
        r, n, k, g = case["rows"], case["n"], case["k"], case["groups"]
        # experts that get rows, on average, of an evenly loaded router (an expert without any
        # needs no weights)
        p = g if case["load"] != "sparse" else max(1, g // 8)
        hit = p * (1.0 - (1.0 - 1.0 / p) ** r)
        rows = r * (n + k) * es
        return {"bytes": rows + (g * n * k * 4 if op == "wgrad" else hit * n * k * es) + 4 * g,
                "flops": 2.0 * r * n * k}
    if op in ("norm", "norm_bwd"):
        es = 2 if case["dtype"] == "bf16" else 4
        t, d = case["rows"], case["d"]
        if op == "norm":
            streams = 3 + (1 if case["pre"] else 0)      # x, y, r (and u)
        else:
            streams = 4 + (2 if case["pre"] else 0)      # y, dr, dx, dy (and r, du)
        small = 4 * (t * (case["post"] + case["pre"] + (case["gate"] == "token")) +
                     d * (case["post"] + case["pre"] + (case["gate"] == "channel")))
        return {"bytes": streams * t * d * es + small * (2 if op == "norm_bwd" else 1),
                "flops": t * d * (10.0 if op == "norm" else 24.0)}
    sizes, dts = _tensors(case)
    n = sum(math.prod(s) for s in sizes)
    size = sum(math.prod(s) * (2 if dt == torch.bfloat16 else 4) for s, dt in zip(sizes, dts))
    return {"bytes": size * (2 if op == "clip" else 1), "flops": n * (3.0 if op == "clip" else 2.0)}


# ------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The same outputs from the definitions in 64 bits."""
    st = prepare(case, seed)
    op = case["op"]

    def wide(t):
        return None if t is None else t.to(torch.float64)

    if op in ("mm", "dgrad", "wgrad"):
        bounds = [0]
        for c in st["splits"]:
            bounds.append(bounds[-1] + c)
        out = torch.zeros(st["out"].shape, dtype=torch.float64, device=st["out"].device)
        for e in range(case["groups"]):
            lo, hi = bounds[e], bounds[e + 1]
            if op == "mm":
                out[lo:hi] = torch.einsum("rk,nk->rn", wide(st["x"][lo:hi]), wide(st["w"][e]))
            elif op == "dgrad":
                out[lo:hi] = torch.einsum("rn,nk->rk", wide(st["dy"][lo:hi]), wide(st["w"][e]))
            else:
                out[e] = torch.einsum("rn,rk->nk", wide(st["dy"][lo:hi]), wide(st["x"][lo:hi]))
        return out
    if op in ("norm", "norm_bwd"):
        d = case["d"]
        x, y, gate, wq, wp = (wide(st[n]) for n in ("x", "y", "gate_t", "post_w", "pre_w"))
        one = torch.ones(1, dtype=torch.float64, device=x.device)
        gate1, wq1 = one if gate is None else gate, one if wq is None else wq
        if op == "norm":
            sy = torch.pow((y * y).sum(1) / d + EPS, -0.5) if wq is not None else None
            r = st["beta"] * x + gate1 * ((y if sy is None else torch.einsum("td,t->td", y, sy)) * wq1)
            sr = torch.pow((r * r).sum(1) / d + EPS, -0.5) if wp is not None else None
            return r, None if sr is None else torch.einsum("td,t,d->td", r, sr, wp), sy, sr
        g, r, du, sy, sr = (wide(st.get(n)) for n in ("dr", "r", "du", "post_rstd", "pre_rstd"))
        d_pre = None
        if wp is not None:
            a = torch.einsum("td,d,t->td", du, wp, sr)
            d_pre = torch.einsum("td,td,t->d", du, r, sr)
            g = g + a - torch.einsum("td,t->td", r, (a * r).sum(1) * sr * sr / d)
        yh = y if sy is None else torch.einsum("td,t->td", y, sy)
        gb = g * yh * wq1
        d_gate = None if gate is None else (gb.sum(0) if case["gate"] == "channel" else gb.sum(1)[:, None])
        d_post, dy = None, g * gate1
        if wq is not None:
            d_post = (dy * yh).sum(0)
            a = torch.einsum("td,d,t->td", dy, wq, sy)
            dy = a - torch.einsum("td,t->td", y, (a * y).sum(1) * sy * sy / d)
        return st["beta"] * g, dy, d_gate, d_post, d_pre
    sq = sum(float((wide(g) ** 2).sum()) for g in st["grads"])
    norm = math.sqrt(sq)
    out_norm = torch.tensor([norm], dtype=torch.float64, device="cuda")
    if op == "gnorm":
        return out_norm
    c = st["max_norm"] / norm if norm > st["max_norm"] else 1.0
    if case["layout"] == "layer":
        return (out_norm, *[wide(g) * c for g in st["grads"]])
    flat = {dt: torch.cat([wide(g) * c for g in st["grads"] if g.dtype == dt]) for dt in st["flat_out"]}
    return out_norm, flat.get(torch.bfloat16), flat.get(torch.float32)
