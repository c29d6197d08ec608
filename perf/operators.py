"""Cases of the layer operators: a layer's product with its epilogue, the
same product over the experts of an expert tensor, tokens sorted by expert and
back, and the gate that routes them.

Each case is one pass through one operator in one direction.  ``run`` computes
it with the library's operators where ``own`` is true, and otherwise in plain
form: elementary torch operations in 32 bits, rounded once at the end.
``exact`` gives the same outputs from the definitions in 64 bits.

Sizes are those of the benchmark configurations (the dense h = 4096 layers
[4096, 12288] and [4096, 16384], the expert tensor [64, 2048, 7168]) and
generic odd ones.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _linear(**kw):
    return {"op": "linear", "grad": False, "dtype": "bf16", "act": "none", "bias": True, "residual": False,
            "keep": False, "w_out_in": False, **kw}


def _experts(**kw):
    return {"op": "experts", "grad": False, "dtype": "bf16", "act": "none", "bias": False, "keep": False,
            "w_out_in": False, "skew": 0.0, **kw}


def _sort(**kw):
    return {"op": "sort", "grad": False, "dtype": "bf16", "drop": 0.0, "residual": False, **kw}


def _gate(**kw):
    return {"op": "gate", "grad": False, "dtype": "fp32", "renormalize": True, "masked": 0.0, **kw}


def listed():
    return [
        # serving, one new token through the dense model's fused qkv matrix: the weights are read once
        _linear(name="linear_token", tokens=1, n_in=4096, n_out=12288),
        # training, a micro-batch through the dense model's first feed-forward matrix, its
        # pre-activation kept for the way back
        _linear(name="linear_up", tokens=4096, n_in=4096, n_out=16384, act="gelu_tanh", keep=True),
        # the same layer's way back: input, weight and bias gradients through the activation
        _linear(name="linear_up_grad", tokens=4096, n_in=4096, n_out=16384, act="gelu_tanh", grad=True),
        # a small fp32 head of odd sizes, weights stored [out, in], with a residual
        _linear(name="linear_odd_fp32", tokens=515, n_in=1001, n_out=777, dtype="fp32", act="silu", residual=True,
                w_out_in=True),
        # serving, four tokens with eight experts each: at most 32 of 64 experts are read
        _experts(name="experts_tokens", tokens=4, top_k=8, experts=64, n_in=7168, n_out=2048, dtype="fp16",
                 act="silu"),
        # training, 4096 tokens with eight experts each through the experts' first matrix
        _experts(name="experts_up", tokens=4096, top_k=8, experts=64, n_in=7168, n_out=2048, act="silu", keep=True),
        # the way back through the experts' second matrix, popular and empty experts among them
        _experts(name="experts_down_grad", tokens=2053, top_k=8, experts=64, n_in=2048, n_out=7168, skew=1.0,
                 bias=True, grad=True),
        # serving, one token to its eight experts and back
        _sort(name="sort_token", tokens=1, top_k=8, experts=64, hidden=7168, residual=True),
        # training, 8192 tokens to their experts and back
        _sort(name="sort_batch", tokens=8192, top_k=8, experts=64, hidden=7168),
        # the way back of a ragged batch with assignments dropped by a capacity limit
        _sort(name="sort_grad", tokens=4099, top_k=6, experts=48, hidden=2048, dtype="fp16", drop=0.05, grad=True),
        # routing a training batch: the top 8 of 64 experts
        _gate(name="gate_batch", tokens=16384, experts=64, top_k=8),
        # the way back of a router over many experts, 16-bit logits, some experts masked out
        _gate(name="gate_grad", tokens=8192, experts=256, top_k=8, dtype="bf16", masked=0.1, renormalize=False,
              grad=True),
    ]


def draw(rng):
    def log_int(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    def width(lo, hi):  # two of three are multiples of 64, the others any number
        n = log_int(lo, hi)
        return n if rng.random() < 1 / 3 else max(64, n // 64 * 64)

    op = rng.choice(("linear", "experts", "sort", "gate"))
    grad = rng.random() < 0.5
    acts = ("none", "relu", "silu", "gelu", "gelu_tanh")
    if op == "linear":
        dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
        c = _linear(tokens=log_int(1, 4096), n_in=width(64, 4096 if dtype == "fp32" else 12288),
                    n_out=width(64, 4096 if dtype == "fp32" else 12288), dtype=dtype, act=rng.choice(acts),
                    bias=rng.random() < 0.5, w_out_in=rng.random() < 0.5, grad=grad)
        if not grad:
            c["residual"], c["keep"] = rng.random() < 0.5, rng.random() < 0.5
        return c
    if op == "experts":
        c = _experts(tokens=log_int(1, 4096), top_k=rng.choice((1, 2, 4, 8)), experts=log_int(8, 128),
                     n_in=width(64, 4096), n_out=width(64, 4096), dtype=rng.choice(("bf16", "bf16", "fp16")),
                     act=rng.choice(acts), bias=rng.random() < 0.5, w_out_in=rng.random() < 0.5,
                     skew=rng.choice((0.0, 0.0, 1.0)), grad=grad)
        if not grad:
            c["keep"] = rng.random() < 0.5
        return c
    if op == "sort":
        c = _sort(tokens=log_int(1, 8192), top_k=rng.choice((1, 2, 4, 6, 8)), experts=log_int(8, 256),
                  hidden=width(64, 7168), dtype=rng.choice(("bf16", "bf16", "fp16", "fp32")),
                  drop=rng.choice((0.0, 0.1)), grad=grad)
        if not grad:
            c["residual"] = rng.random() < 0.5
        return c
    experts = log_int(8, 512)
    return _gate(tokens=log_int(1, 16384), experts=experts, top_k=rng.choice((1, 2, 4, 8)),
                 dtype=rng.choice(("fp32", "fp32", "bf16", "fp16")), renormalize=rng.random() < 0.5,
                 masked=rng.choice((0.0, 0.2)), grad=grad)


# ---- inputs ----


def _indices(c, g):
    """[tokens, top_k] int32: each token's experts, distinct within a token.
    skew > 0 makes low-numbered experts popular and leaves every 16th empty."""
    score = torch.rand(c["tokens"], c["experts"], generator=g, device="cuda")
    score = -torch.log(-torch.log(score.clamp(1e-9, 1 - 1e-7)))  # Gumbel draws: top_k without replacement
    if c.get("skew"):
        score -= 0.1 * c["skew"] * torch.arange(c["experts"], device="cuda")
        score[:, 15::16] = -math.inf
    return score.argsort(1, descending=True)[:, :c["top_k"]].int().contiguous()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DTYPES[c["dtype"]]

    def normal(*shape, std=1.0, dtype=dt):
        return torch.randn(*shape, generator=g, device="cuda").mul_(std).to(dtype)

    s = {"case": c}
    if c["op"] in ("linear", "experts"):
        k, n = c["n_in"], c["n_out"]
        lead = () if c["op"] == "linear" else (c["experts"],)
        if c["w_out_in"]:  # stored [.., out, in], handed over as its transposed view
            s["w"] = normal(*lead, n, k, std=k ** -0.5).transpose(-1, -2)
        else:
            s["w"] = normal(*lead, k, n, std=k ** -0.5)
        rows = c["tokens"]
        if c["op"] == "experts":
            flat = _indices(c, g).reshape(-1).long()
            rows = flat.numel()
            s["offsets"] = torch.searchsorted(flat.sort()[0], torch.arange(c["experts"] + 1, device="cuda")).int()
            s["cap"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
        s["x"] = normal(rows, k)
        s["b"] = normal(*lead, n, std=0.1) if c["bias"] else None
        if c["grad"]:
            s["dy"] = normal(rows, n, std=0.1)
            s["z"] = normal(rows, n) if c["act"] != "none" else None
        else:
            s["r"] = normal(rows, n) if c.get("residual") else None
        return s
    if c["op"] == "sort":
        t, k, e, h = c["tokens"], c["top_k"], c["experts"], c["hidden"]
        k = min(k, e)
        idx = _indices({**c, "top_k": k}, g)
        if c["drop"]:
            idx.masked_fill_(torch.rand(t, k, generator=g, device="cuda") < c["drop"], -1)
        wts = torch.rand(t, k, generator=g, device="cuda") + 0.05
        s["wts"] = wts / wts.sum(1, keepdim=True)
        s["ys"] = normal(t * k, h)
        if c["grad"]:
            s["slot"], s["offsets"], _ = _plain_order(idx, e)
            s["dy"] = normal(t, h, std=0.1)
            s["dxs"] = normal(t * k, h, std=0.1)
        else:
            s["idx"], s["x"] = idx, normal(t, h)
            s["r"] = normal(t, h) if c["residual"] else None
        return s
    t, e = c["tokens"], c["experts"]
    k = min(c["top_k"], e)
    s["k"] = k
    s["logits"] = normal(t, e)
    if c["masked"]:
        s["logits"].masked_fill_(torch.rand(t, e, generator=g, device="cuda") < c["masked"], -math.inf)
        s["logits"][::17] = -math.inf  # tokens with no expert left
    if c["grad"]:
        s["idx"] = _plain_gate(s["logits"], k, c["renormalize"])[0]
        s["dwts"] = normal(t, k, dtype=torch.float32)
    return s


# ---- plain forms ----


def _act(z, kind):
    if kind == "relu":
        return z.clamp(min=0)
    if kind == "silu":
        return z / (1 + torch.exp(-z))
    if kind == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if kind == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_slope(z, kind):
    if kind == "relu":
        return (z > 0).to(z.dtype)
    if kind == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if kind == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)


def _like_w(dw, w):
    """dw in w's type and memory order."""
    if w.stride(-1) == 1:
        return dw.to(w.dtype)
    return dw.transpose(-1, -2).to(w.dtype).contiguous().transpose(-1, -2)


def _plain_linear(s):
    c, x, w = s["case"], s["x"], s["w"]
    if not c["grad"]:
        z = x.float() @ w.float()
        if s["b"] is not None:
            z = z + s["b"].float()
        y = _act(z, c["act"])
        if s["r"] is not None:
            y = y + s["r"].float()
        return (y.to(x.dtype), z.to(x.dtype)) if c["keep"] else (y.to(x.dtype),)
    dz = s["dy"].float()
    if s["z"] is not None:
        dz = dz * _act_slope(s["z"].float(), c["act"])
    dx = dz @ w.float().transpose(0, 1)
    dw = x.float().transpose(0, 1) @ dz
    out = (dx.to(x.dtype), _like_w(dw, w))
    return out + (dz.sum(0).to(x.dtype),) if c["bias"] else out


def _pad_rows(off, cap):
    """[experts, cap]: the row each place of a padded expert block holds, and whether it holds one."""
    at = off[:-1, None].long() + torch.arange(cap, device=off.device)
    there = at < off[1:, None]
    return at.masked_fill(~there, 0), there


def _plain_experts(s):
    c, x, w = s["case"], s["x"], s["w"]
    at, there = _pad_rows(s["offsets"], s["cap"])
    rows = at[there]  # in order: every row has one place
    xp = x.float()[at] * there[..., None]
    if not c["grad"]:
        z = torch.bmm(xp, w.float())
        if s["b"] is not None:
            z = z + s["b"].float()[:, None]
        z = z[there][rows.argsort()]
        y = _act(z, c["act"]).to(x.dtype)
        return (y, z.to(x.dtype)) if c["keep"] else (y,)
    dz = s["dy"].float()
    if s["z"] is not None:
        dz = dz * _act_slope(s["z"].float(), c["act"])
    dp = dz[at] * there[..., None]
    dx = torch.bmm(dp, w.float().transpose(1, 2))[there][rows.argsort()]
    dw = torch.bmm(xp.transpose(1, 2), dp)
    out = (dx.to(x.dtype), _like_w(dw, w))
    return out + (dp.sum(1).to(x.dtype),) if c["bias"] else out


def _plain_order(idx, experts):
    """(slot [tokens, top_k] int32, -1 where dropped; offsets [experts + 1] int32; the flat assignment of each sorted row)."""
    flat = idx.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    sorted_key, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(sorted_key, torch.arange(experts + 1, device=idx.device)).int()
    slot = torch.empty_like(flat)
    slot[order] = torch.arange(flat.numel(), device=idx.device)
    slot = slot.masked_fill(key == experts, -1)
    return slot.view(idx.shape).int(), offsets, order


def _plain_sort(s):
    c = s["case"]
    if not c["grad"]:
        x, k = s["x"], s["idx"].shape[1]
        slot, offsets, order = _plain_order(s["idx"], c["experts"])
        live = torch.arange(order.numel(), device=x.device) < offsets[-1]
        xs = x[order // k].masked_fill(~live[:, None], 0)
        took = s["ys"].float()[slot.clamp(min=0).long()].masked_fill((slot < 0)[..., None], 0)
        y = (took * s["wts"][..., None]).sum(1)
        if s["r"] is not None:
            y = y + s["r"].float()
        return xs, slot, offsets, y.to(x.dtype)
    slot, dt = s["slot"], s["ys"].dtype
    at, there = slot.clamp(min=0).long(), (slot >= 0)[..., None]
    dx = s["dxs"].float()[at].masked_fill(~there, 0).sum(1)
    dy = s["dy"].float()[:, None]
    dys = torch.zeros(s["ys"].shape, device=dy.device)
    dys[slot[slot >= 0].long()] = (dy * s["wts"][..., None])[slot >= 0]
    dwts = (s["ys"].float()[at].masked_fill(~there, 0) * dy).sum(2)
    return dx.to(dt), dys.to(dt), dwts


def _plain_gate(logits, k, renormalize):
    """The k largest logits of each token (ties: the lower index), -1 and weight 0 where only masked ones (-inf) are left."""
    lf = logits.float()
    top, idx = (v[:, :k] for v in torch.sort(lf, dim=1, descending=True, stable=True))
    there = top > -math.inf
    high = top[:, :1].masked_fill(~there[:, :1], 0)
    p = torch.exp(top - high)
    total = p.sum(1, keepdim=True) if renormalize else torch.exp(lf - high).sum(1, keepdim=True)
    wts = torch.where(there, p / total.masked_fill(~there[:, :1], 1), 0.0)
    return torch.where(there, idx, -1).int(), wts


def _plain_gate_grad(s):
    lf, idx, dwts = s["logits"].float(), s["idx"].long(), s["dwts"]
    there = idx >= 0
    g = torch.zeros_like(lf).scatter_add_(1, idx.clamp(min=0), dwts.masked_fill(~there, 0))
    if s["case"]["renormalize"]:
        kept = torch.zeros_like(lf).scatter_add_(1, idx.clamp(min=0), there.float()) > 0
        lf = lf.masked_fill(~kept, -math.inf)
    high = lf.amax(1, keepdim=True)
    p = torch.exp(lf - high.masked_fill(high == -math.inf, 0))
    total = p.sum(1, keepdim=True)
    p = p / total.masked_fill(total == 0, 1)
    return (p * (g - (p * g).sum(1, keepdim=True))).to(s["logits"].dtype)


# ---- one pass ----


def run(state):
    s, c = state, state["case"]
    if not own:
        if c["op"] == "linear":
            return _plain_linear(s)
        if c["op"] == "experts":
            return _plain_experts(s)
        if c["op"] == "sort":
            return _plain_sort(s)
        return (_plain_gate_grad(s),) if c["grad"] else _plain_gate(s["logits"], s["k"], c["renormalize"])
    import newton_schulz_bucket_gb300 as muon
    if c["op"] == "linear":
        if c["grad"]:
            dx, dw, db = muon.linear_backward(s["dy"], s["x"], s["w"], preact=s["z"], activation=c["act"],
                                              bias=c["bias"])
            return (dx, dw, db) if c["bias"] else (dx, dw)
        y = muon.linear(s["x"], s["w"], bias=s["b"], activation=c["act"], residual=s["r"], keep_preact=c["keep"])
        return y if c["keep"] else (y,)
    if c["op"] == "experts":
        if c["grad"]:
            dx, dw, db = muon.expert_linear_backward(s["dy"], s["x"], s["offsets"], s["w"], preact=s["z"],
                                                     activation=c["act"], bias=c["bias"])
            return (dx, dw, db) if c["bias"] else (dx, dw)
        y = muon.expert_linear(s["x"], s["offsets"], s["w"], bias=s["b"], activation=c["act"], keep_preact=c["keep"])
        return y if c["keep"] else (y,)
    if c["op"] == "sort":
        if c["grad"]:
            dx = muon.dispatch_backward(s["dxs"], s["slot"])
            dys, dwts = muon.combine_backward(s["dy"], s["ys"], s["slot"], s["offsets"], s["wts"])
            return dx, dys, dwts
        xs, slot, offsets = muon.dispatch(s["x"], s["idx"], c["experts"])
        return xs, slot, offsets, muon.combine(s["ys"], slot, s["wts"], residual=s["r"])
    if c["grad"]:
        return (muon.gate_backward(s["dwts"], s["logits"], s["idx"], renormalize=c["renormalize"]),)
    return muon.gate(s["logits"], s["k"], renormalize=c["renormalize"])


# ---- what a pass cannot do without ----


def work(case):
    c = case
    b = 4 if c["dtype"] == "fp32" else 2
    if c["op"] in ("linear", "experts"):
        t, k, n = c["tokens"], c["n_in"], c["n_out"]
        mats = 1
        if c["op"] == "experts":
            t *= c["top_k"]
            mats = c["experts"]
        read = min(mats, t)  # experts that any row reaches, at most
        if c["grad"]:
            act = 1 if c["act"] != "none" else 0
            nbytes = b * (t * n * (1 + act) + t * k * 2 + read * k * n + mats * k * n + (mats * n if c["bias"] else 0))
            return {"bytes": nbytes, "flops": 4 * t * k * n}
        nbytes = b * (t * k + read * k * n + t * n * (1 + bool(c["keep"]) + bool(c.get("residual"))))
        return {"bytes": nbytes + (b * mats * n if c["bias"] else 0), "flops": 2 * t * k * n}
    if c["op"] == "sort":
        t, k, h = c["tokens"], min(c["top_k"], c["experts"]), c["hidden"]
        if c["grad"]:  # dxs, ys, dy read, dys, dx written, slots and weights read, weight gradients written
            return {"bytes": b * h * (3 * t * k + 2 * t) + 12 * t * k, "flops": 4 * t * k * h}
        return {"bytes": b * h * (2 * t * k + 2 * t + (t if c["residual"] else 0)) + 12 * t * k, "flops": 2 * t * k * h}
    t, e, k = c["tokens"], c["experts"], min(c["top_k"], c["experts"])
    if c["grad"]:
        return {"bytes": 2 * b * t * e + 8 * t * k, "flops": 6 * t * e}
    return {"bytes": b * t * e + 8 * t * k, "flops": 4 * t * e}


# ---- the definitions in 64 bits ----


def _d_act(z, kind):
    """(act(z), act'(z)) in 64 bits."""
    one = torch.ones_like(z)
    if kind == "none":
        return z, one
    if kind == "relu":
        return torch.where(z > 0, z, 0.0), torch.where(z > 0, 1.0, 0.0).double()
    if kind == "silu":
        sig = torch.special.expit(z)
        return z * sig, sig + z * sig * torch.special.expit(-z)
    if kind == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z * z / 2) * (2 * math.pi) ** -0.5
    u = (2 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3)
    du = (2 / math.pi) ** 0.5 * (1 + 0.134145 * z ** 2)
    sig = torch.special.expit(2 * u)  # (1 + tanh u) / 2
    return z * sig, sig + 2 * z * sig * torch.special.expit(-2 * u) * du


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] in ("linear", "experts"):
        x, w = s["x"].double(), s["w"]
        rows, n, k = x.shape[0], c["n_out"], c["n_in"]
        ends = s["offsets"].tolist() if c["op"] == "experts" else [0, rows]
        new = lambda *d: torch.zeros(*d, dtype=torch.float64, device="cuda")  # noqa: E731
        first, second = new(rows, k if c["grad"] else n), new(rows, n)
        dw, db = (torch.zeros(s["w"].shape, dtype=torch.float64, device="cuda"), new(len(ends) - 1, n)) if c["grad"] else (None, None)
        for e, (lo, hi) in enumerate(zip(ends, ends[1:])):
            we = (w if c["op"] == "linear" else w[e]).double()
            if c["grad"]:
                d = s["dy"][lo:hi].double()
                if s["z"] is not None:
                    d = d * _d_act(s["z"][lo:hi].double(), c["act"])[1]
                first[lo:hi] = d @ we.T
                (dw if c["op"] == "linear" else dw[e]).copy_(x[lo:hi].T @ d)
                db[e] = d.sum(0)
                continue
            z = x[lo:hi] @ we
            if s["b"] is not None:
                z = z + (s["b"] if c["op"] == "linear" else s["b"][e]).double()
            second[lo:hi] = z
            first[lo:hi] = _d_act(z, c["act"])[0]
        if c["grad"]:
            return (first, dw, db[0] if c["op"] == "linear" else db) if c["bias"] else (first, dw)
        if s.get("r") is not None:
            first = first + s["r"].double()
        return (first, second) if c["keep"] else (first,)
    if c["op"] == "sort":
        h = s["ys"].shape[1]
        if c["grad"]:
            t, k = s["slot"].shape
            row = s["slot"].reshape(-1).long()
            flat = torch.nonzero(row >= 0)[:, 0]
            row, tok = row[flat], flat // k
            wts = s["wts"].double().reshape(-1)
            dx = torch.zeros(t, h, dtype=torch.float64, device="cuda").index_add_(0, tok, s["dxs"].double()[row])
            dys = torch.zeros(t * k, h, dtype=torch.float64, device="cuda")
            dys[row] = s["dy"].double()[tok] * wts[flat, None]
            dwts = torch.zeros(t * k, dtype=torch.float64, device="cuda")
            dwts[flat] = (s["ys"].double()[row] * s["dy"].double()[tok]).sum(1)
            return dx, dys, dwts.view(t, k)
        t, k = s["idx"].shape
        of = s["idx"].reshape(-1)
        order = [torch.nonzero(of == e)[:, 0] for e in range(c["experts"])]  # each expert's assignments in turn
        offsets = torch.tensor([0] + [o.numel() for o in order], device="cuda").cumsum(0).int()
        order = torch.cat(order)
        slot = torch.full_like(of, -1)
        slot[order] = torch.arange(order.numel(), device="cuda", dtype=torch.int32)
        row, slot = slot.long(), slot.view(t, k)
        flat = torch.nonzero(row >= 0)[:, 0]
        xs = torch.zeros(t * k, h, dtype=torch.float64, device="cuda")
        xs[row[flat]] = s["x"].double()[flat // k]
        y = torch.zeros(t, h, dtype=torch.float64, device="cuda") if s["r"] is None else s["r"].double()
        for j in range(k):
            there = torch.nonzero(slot[:, j] >= 0)[:, 0]
            y[there] += s["ys"][slot[there, j].long()].double() * s["wts"][there, j, None].double()
        return xs, slot, offsets, y
    d = s["logits"].double()
    if c["grad"]:
        d = d.requires_grad_()
        live = torch.isfinite(d.detach())
        idx = s["idx"].long()
        there = idx >= 0
        chosen = torch.zeros_like(live).scatter_(1, idx.clamp(min=0), True) & live & there.any(1, keepdim=True)
        over = chosen if c["renormalize"] else live
        m = torch.where(over, d, -1e300)
        rows = over.any(1)
        logp = m[rows] - torch.logsumexp(m[rows], 1, keepdim=True)
        picked = torch.gather(logp.exp(), 1, idx[rows].clamp(min=0))
        (picked * s["dwts"][rows].double())[there[rows]].sum().backward()
        return (d.grad,)
    idx, wts = s["logits"].new_full((c["tokens"], s["k"]), -1, dtype=torch.int32), None
    left, picked = d.clone(), []
    for j in range(s["k"]):
        best = left.amax(1, keepdim=True)
        first = (left == best).int().argmax(1)  # the lowest index of the largest
        idx[:, j] = torch.where(best[:, 0] > -math.inf, first.int(), -1)
        picked.append(best[:, 0])
        left.scatter_(1, first[:, None], -math.inf)
    top = torch.stack(picked, 1)
    total = torch.logsumexp(top if c["renormalize"] else d, 1, keepdim=True)
    wts = torch.where(idx >= 0, torch.exp(top - total.masked_fill(total == -math.inf, 0)), 0.0)
    return idx, wts
