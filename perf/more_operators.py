"""Projections with bias, activation and residual in their epilogue, and the
norms before and after a block fused with its gate and scales: what stands
between the gated projections and the residual stream.  Forward, for training
and for few tokens, and backward.

``own`` False: elementary torch operations in 32 bits.  ``own`` True: the
calls a user makes of layout_folding_gb300.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}


# ---------------------------------------------------------------- cases
def _linear(name, m, k, n, dtype="bf16", act="none", bias="none", residual=False, save=False):
    return {"name": name, "op": "linear", "m": m, "k": k, "n": n, "dtype": dtype, "act": act, "bias": bias,
            "residual": residual, "save": save}


def _linear_bwd(name, m, k, n, act="none", bias="none"):
    return {"name": name, "op": "linear_backward", "m": m, "k": k, "n": n, "act": act, "bias": bias}


def _norms(name, m, d, dtype="bf16", wdtype="bf16", post=True, pre=True, gates=0, branch_scale=1.0,
           residual_scale=1.0, fp8=False):
    """gates: 0 no gate, G >= 1 gate rows, each for m / G consecutive tokens."""
    return {"name": name, "op": "norms", "m": m, "d": d, "dtype": dtype, "wdtype": wdtype, "post": post, "pre": pre,
            "gates": gates, "branch_scale": branch_scale, "residual_scale": residual_scale, "fp8": fp8}


def _norms_bwd(name, m, d, dtype="bf16", wdtype="bf16", post=True, pre=True, gates=0, branch_scale=1.0,
               residual_scale=1.0, dh=True):
    return {"name": name, "op": "norms_backward", "m": m, "d": d, "dtype": dtype, "wdtype": wdtype, "post": post,
            "pre": pre, "gates": gates, "branch_scale": branch_scale, "residual_scale": residual_scale, "dh": dh}


def listed():
    return [
        # one token being generated: the down projection, added to the stream
        _linear("linear_token", 1, 13824, 5120, residual=True),
        # a batch of tokens being generated, e4m3 weights and activations, the down projection with its bias
        _linear("linear_decode_e4m3", 48, 13824, 5120, dtype="e4m3", bias="bf16", residual=True),
        # a small model's ragged batch: the first projection of an ungated feed-forward part
        _linear("linear_small_gelu", 200, 520, 1416, act="gelu", bias="fp32"),
        # a training step: the first projection of a wide ungated feed-forward part, kept for the backward pass
        _linear("linear_train", 4096, 5120, 13824, act="gelu_tanh", bias="bf16", save=True),
        # ... and its gradient
        _linear_bwd("linear_backward_train", 4096, 5120, 13824, act="gelu_tanh", bias="bf16"),
        # a ragged fine-tuning batch of a smaller model: the biased output projection
        _linear_bwd("linear_backward_ragged", 333, 2048, 5632, bias="fp32"),
        # one token being generated: the norm after a block, its scale, and the next block's norm in e4m3
        _norms("norms_token_e4m3", 1, 5120, branch_scale=0.22, fp8=True),
        # a ragged batch in half precision, odd rows, fp32 weights, a learned gate for each channel
        _norms("norms_ragged_fp16", 1333, 1027, dtype="fp16", wdtype="fp32", gates=1, residual_scale=0.7071),
        # a batch of four prompts, each with its own gate
        _norms("norms_prompts", 8192, 5120, gates=4),
        # a training step with sandwich norms
        _norms_bwd("norms_backward_train", 8192, 4096, gates=1),
        # a fine-tuning batch of seven sequences in fp32, gated by sequence, no norm after the block
        _norms_bwd("norms_backward_gates_fp32", 777, 1536, dtype="fp32", wdtype="fp32", post=False, gates=7),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_backward", "norms", "norms_backward"])
    if op in ("norms", "norms_backward"):
        d = _log(rng, 64, 16384)
        if rng.random() < 0.6:
            d = (d + 7) // 8 * 8
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        cap = (8192 * 4096) // (2 if dtype == "fp32" else 1)
        m = max(1, min(_log(rng, 1, 16384), cap // d))
        gates = rng.choice([0, 1, _log(rng, 1, 64)])
        if gates > 1:
            m = max(1, m // gates) * gates
            if m * d > cap:
                gates, m = 1, cap // d
        case = {"op": op, "m": m, "d": d, "dtype": dtype, "wdtype": rng.choice([dtype, "fp32"]),
                "post": rng.random() < 0.8, "pre": rng.random() < 0.9, "gates": gates,
                "branch_scale": rng.choice([1.0, 0.25]), "residual_scale": rng.choice([1.0, 0.7071])}
        if op == "norms":
            case["fp8"] = case["pre"] and rng.random() < 0.4
        else:
            case["dh"] = not case["pre"] or rng.random() < 0.7
        return case
    m = _log(rng, 1, 4096)
    k = max(16, _log(rng, 128, 16384) // 16 * 16)
    n = max(8, _log(rng, 128, 16384) // 8 * 8)
    n = max(8, min(n, (4096 * 5120 * 13824) // (m * k) // 8 * 8))
    act = rng.choice(["none", "none", "silu", "gelu", "gelu_tanh"])
    bias = rng.choice(["none", "bf16", "fp32"])
    if op == "linear_backward":
        return {"op": op, "m": m, "k": k, "n": n, "act": act, "bias": bias}
    dtype = rng.choice(["bf16", "bf16", "e4m3"])
    return {"op": op, "m": m, "k": k, "n": n, "dtype": dtype, "act": act, "bias": bias, "residual": rng.random() < 0.5,
            "save": dtype == "bf16" and act != "none" and rng.random() < 0.5}


# ---------------------------------------------------------------- inputs
def _rows_to_e4m3(t):
    """Rows of fp32 t as e4m3 with one scale each: what the norm and a weight loader hand over."""
    s = t.abs().amax(1) / E4M3_MAX
    s = torch.where(s == 0, torch.ones_like(s), s)
    return (t / s[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(2000 + seed)

    def normal(*shape, std=1.0):
        return torch.empty(*shape, device=DEV).normal_(0.0, std, generator=g)

    s = dict(case)
    m = case["m"]
    if case["op"] in ("norms", "norms_backward"):
        t, wt, d = DTYPES[case["dtype"]], DTYPES[case["wdtype"]], case["d"]
        size = torch.exp(normal(d, std=0.7))  # a stream's channels differ in size
        s["post_weight"] = (1.0 + normal(d, std=0.2)).to(wt) if case["post"] else None
        s["pre_weight"] = (1.0 + normal(d, std=0.2)).to(wt) if case["pre"] else None
        s["gate"] = None
        if case["gates"]:
            # learned for each channel, or made from each sequence's condition
            s["gate"] = normal(case["gates"], d, std=0.5).to(t if case["gates"] > 1 else wt)
            if case["gates"] == 1:
                s["gate"] = s["gate"][0]
        s["x"] = (normal(m, d) * size).to(t)
        s["res"] = (normal(m, d, std=2.0) * size).to(t)
        if case["op"] == "norms_backward":
            s["h"] = _branch_and_stream(s)[1]
            s["dy"] = normal(m, d, std=0.1).to(t) if case["pre"] else None
            s["dh"] = normal(m, d, std=0.1).to(t) if case["dh"] else None
            del s["res"]
        return s
    k, n = case["k"], case["n"]
    x = normal(m, k)
    w = normal(n, k, std=1.0 / math.sqrt(k))
    s["b"] = normal(n, std=0.5).to(DTYPES[case["bias"]]) if case["bias"] != "none" else None
    if case["op"] == "linear":
        s["res"] = normal(m, n, std=2.0).to(torch.bfloat16) if case["residual"] else None
    if case.get("dtype") == "e4m3":
        s["x"], s["x_scale"] = _rows_to_e4m3(x)
        s["w"], s["w_scale"] = _rows_to_e4m3(w)
        return s
    s["x"], s["w"] = x.to(torch.bfloat16), w.to(torch.bfloat16)
    if case["op"] == "linear_backward":
        s["pre"] = None
        if case["act"] != "none":
            z = s["x"].float() @ s["w"].float().t()
            s["pre"] = (z if s["b"] is None else z + s["b"].float()).to(torch.bfloat16)
        s["dout"] = normal(m, n, std=0.1).to(torch.bfloat16)
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    if own:
        return _run_own(s)
    return {"linear": _plain_linear, "linear_backward": _plain_linear_backward, "norms": _plain_norms,
            "norms_backward": _plain_norms_backward}[s["op"]](s)


def _run_own(s):
    import layout_folding_gb300 as lf
    if s["op"] == "linear":
        act = None if s["act"] == "none" else s["act"]
        if s["dtype"] == "e4m3":
            out, pre = lf.linear(s["x"], s["w"], bias=s["b"], act=act, residual=s["res"], x_scale=s["x_scale"],
                                 w_scale=s["w_scale"])
        else:
            out, pre = lf.linear(s["x"], s["w"], bias=s["b"], act=act, residual=s["res"], want_pre=s["save"])
        return {"out": out, "pre": pre}
    if s["op"] == "linear_backward":
        act = None if s["act"] == "none" else s["act"]
        dx, dw, db = lf.linear_backward(s["dout"], s["x"], s["w"], pre=s["pre"], act=act, bias=s["b"])
        return {"dx": dx, "dw": dw, "db": db}
    kw = dict(gate=s["gate"], branch_scale=s["branch_scale"], residual_scale=s["residual_scale"], eps=EPS)
    if s["op"] == "norms":
        y, h, scale = lf.block_norm(s["x"], s["res"], s["post_weight"], s["pre_weight"], fp8=s["fp8"], **kw)
        return {"y": y, "h": h, "scale": scale}
    dx, dres, dpost, dpre, dgate = lf.block_norm_backward(s["dy"], s["x"], s["h"], s["post_weight"], s["pre_weight"],
                                                          dh=s["dh"], **kw)
    return {"dx": dx, "dres": dres, "dpost": dpost, "dpre": dpre, "dgate": dgate}


def _act(v, act):
    if act == "none":
        return v
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))


def _act_slope(v, act):
    if act == "silu":
        sig = 1 / (1 + torch.exp(-v))
        return sig * (1 + v * (1 - sig))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(v * math.sqrt(0.5))) + v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    th = torch.tanh(c * (v + 0.044715 * v ** 3))
    return 0.5 * (1 + th) + 0.5 * v * (1 - th * th) * c * (1 + 3 * 0.044715 * v * v)


def _plain_linear(s):
    z = s["x"].float() @ s["w"].float().t()
    if s["dtype"] == "e4m3":
        z = z * s["x_scale"][:, None] * s["w_scale"][None, :]
    if s["b"] is not None:
        z = z + s["b"].float()
    out = _act(z, s["act"])
    if s["res"] is not None:
        out = out + s["res"].float()
    return {"out": out.to(torch.bfloat16), "pre": z.to(torch.bfloat16) if s["save"] else None}


def _plain_linear_backward(s):
    dz = s["dout"].float()
    if s["act"] != "none":
        dz = dz * _act_slope(s["pre"].float(), s["act"])
    dx = dz @ s["w"].float()
    dw = dz.t() @ s["x"].float()
    db = None if s["b"] is None else dz.sum(0).to(s["b"].dtype)
    return {"dx": dx.to(torch.bfloat16), "dw": dw.to(torch.bfloat16), "db": db}


def _gate_rows(s, t):
    """The gate of every token in 32 bits, or None."""
    if s["gate"] is None:
        return None
    g = s["gate"].float()
    return g if g.dim() == 1 else g.repeat_interleave(s["m"] // g.shape[0], 0)


def _branch_and_stream(s):
    """What the block adds before gate and scale, and the stream after it, kept in its type."""
    x = s["x"].float()
    p = x
    if s["post_weight"] is not None:
        p = x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * s["post_weight"].float()
    add = p
    gate = _gate_rows(s, p)
    if gate is not None:
        add = add * gate
    return p, (s["res"].float() * s["residual_scale"] + add * s["branch_scale"]).to(s["x"].dtype)


def _plain_norms(s):
    h = _branch_and_stream(s)[1]
    if s["pre_weight"] is None:
        return {"y": None, "h": h, "scale": None}
    hf = h.float()
    y = hf * torch.rsqrt(hf.square().mean(1, keepdim=True) + EPS) * s["pre_weight"].float()
    if not s["fp8"]:
        return {"y": y.to(h.dtype), "h": h, "scale": None}
    scale = y.abs().amax(1) / E4M3_MAX
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    q = (y / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return {"y": q, "h": h, "scale": scale}


def _plain_norms_backward(s):
    x, h = s["x"].float(), s["h"].float()
    t = s["x"].dtype
    dpre = None
    total = None if s["dh"] is None else s["dh"].float()
    if s["pre_weight"] is not None:
        dy, w = s["dy"].float(), s["pre_weight"].float()
        r = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
        hh = h * r
        dpre = (dy * hh).sum(0).to(s["pre_weight"].dtype)
        g = dy * w
        g = r * (g - hh * (g * hh).mean(1, keepdim=True))
        total = g if total is None else total + g
    dres = total * s["residual_scale"]
    total = total * s["branch_scale"]
    gate = _gate_rows(s, x)
    if s["post_weight"] is not None:
        r = torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
        xh = x * r
        p = xh * s["post_weight"].float()
    else:
        p = x
    dgate = None
    if gate is not None:
        dgate = total * p
        dgate = (dgate.sum(0) if s["gate"].dim() == 1 else
                 dgate.view(s["gate"].shape[0], -1, s["d"]).sum(1)).to(s["gate"].dtype)
        total = total * gate
    dpost = None
    dx = total
    if s["post_weight"] is not None:
        dpost = (total * xh).sum(0).to(s["post_weight"].dtype)
        g = total * s["post_weight"].float()
        dx = r * (g - xh * (g * xh).mean(1, keepdim=True))
    return {"dx": dx.to(t), "dres": dres.to(t), "dpost": dpost, "dpre": dpre, "dgate": dgate}


# ---------------------------------------------------------------- work
def work(case):
    m = case["m"]
    if case["op"] in ("norms", "norms_backward"):
        d, b, wb = case["d"], BYTES[case["dtype"]], BYTES[case["wdtype"]]
        n = m * d
        params = d * wb * (case["post"] + case["pre"]) + case["gates"] * d * (b if case["gates"] > 1 else wb)
        if case["op"] == "norms":
            bytes_ = 3 * n * b + params
            if case["pre"]:
                bytes_ += n + 4 * m if case["fp8"] else n * b
            return {"bytes": bytes_, "flops": 14 * n}
        # x is needed for its own norm's or the gate's gradient, h and dy for the next norm's
        reads = (1 if case["post"] or case["gates"] else 0) + (2 if case["pre"] else 0) + (1 if case["dh"] else 0)
        return {"bytes": n * b * (reads + 2) + 2 * params, "flops": 26 * n}
    k, n = case["k"], case["n"]
    bias = 0 if case["bias"] == "none" else n * BYTES[case["bias"]]
    if case["op"] == "linear":
        b = BYTES[case["dtype"]]
        bytes_ = b * (m * k + n * k) + bias + 2 * m * n * (1 + case["residual"] + case["save"])
        if case["dtype"] == "e4m3":
            bytes_ += 4 * (m + n)
        return {"bytes": bytes_, "flops": 2 * m * n * k}
    return {"bytes": 2 * (2 * m * k + 2 * n * k + m * n * (2 if case["act"] != "none" else 1)) + bias,
            "flops": 4 * m * n * k}


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The definitions, evaluated in 64 bits on prepare's inputs."""
    s = prepare(case, seed)
    return _exact_norms(case, s) if case["op"] in ("norms", "norms_backward") else _exact_linear(case, s)


def _exact_linear(case, s):
    act = case["act"]
    x, w = s["x"].double(), s["w"].double()

    def phi(v):  # act(v) = v * phi(v)
        if act == "none":
            return torch.ones_like(v)
        if act == "silu":
            return torch.special.expit(v)
        if act == "gelu":
            return torch.special.ndtr(v)
        return torch.special.expit(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))

    if case["op"] == "linear":
        if case["dtype"] == "e4m3":
            x, w = x * s["x_scale"].double()[:, None], w * s["w_scale"].double()[:, None]
        z = x @ w.t()
        if s["b"] is not None:
            z = z + s["b"].double()
        out = z * phi(z)
        if s["res"] is not None:
            out = out + s["res"].double()
        return {"out": out, "pre": z if case["save"] else None}
    dz = s["dout"].double()
    if act != "none":
        z = s["pre"].double()
        p = phi(z)
        if act == "silu":
            dphi = p * (1 - p)
        elif act == "gelu":
            dphi = torch.exp(-z ** 2 / 2) / math.sqrt(2 * math.pi)
        else:
            dphi = p * (1 - p) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z ** 2)
        dz = dz * (p + z * dphi)
    return {"dx": dz @ w, "dw": dz.t() @ x, "db": None if s["b"] is None else dz.sum(0)}


def _exact_norms(case, s):
    d, m = case["d"], case["m"]
    x = s["x"].double()
    branch, stream = case["branch_scale"], case["residual_scale"]
    rms1 = ((x ** 2).sum(1, keepdim=True) / d + EPS) ** 0.5
    gate = torch.ones(1, 1, d, dtype=torch.float64, device=DEV)  # [gate row, its tokens, channel]
    if s["gate"] is not None:
        gate = s["gate"].double().view(-1, 1, d)
    groups = gate.shape[0]
    post = s["post_weight"].double() if case["post"] else None
    p = x / rms1 * post if case["post"] else x
    if case["op"] == "norms":
        add = (p.view(groups, m // groups, d) * gate).view(m, d)
        total = stream * s["res"].double() + branch * add
        if not case["pre"]:
            return {"y": None, "h": total, "scale": None}
        kept = total.to(s["x"].dtype).double()
        y = kept / ((kept ** 2).sum(1, keepdim=True) / d + EPS) ** 0.5 * s["pre_weight"].double()
        scale = None
        if case["fp8"]:
            scale = y.abs().max(1).values / E4M3_MAX
            scale = torch.where(scale == 0, torch.ones_like(scale), scale)
            y = y / scale[:, None]
        return {"y": y, "h": total, "scale": scale}
    at_h = torch.zeros_like(x) if s["dh"] is None else s["dh"].double()
    dpre = None
    if case["pre"]:
        h, dy, w = s["h"].double(), s["dy"].double(), s["pre_weight"].double()
        rms2 = ((h ** 2).sum(1, keepdim=True) / d + EPS) ** 0.5
        # y_i = h_i w_i / rms, d rms / d h_j = h_j / (d rms)
        at_h = at_h + dy * w / rms2 - h * (dy * w * h).sum(1, keepdim=True) / (d * rms2 ** 3)
        dpre = (dy * h / rms2).sum(0)
    at_add = branch * at_h
    at_p = (at_add.view(groups, -1, d) * gate).view(m, d)
    dgate = None
    if s["gate"] is not None:
        dgate = (at_add * p).view(groups, -1, d).sum(1).view(s["gate"].shape)
    if not case["post"]:
        return {"dx": at_p, "dres": stream * at_h, "dpost": None, "dpre": dpre, "dgate": dgate}
    dx = at_p * post / rms1 - x * (at_p * post * x).sum(1, keepdim=True) / (d * rms1 ** 3)
    return {"dx": dx, "dres": stream * at_h, "dpost": (at_p * x / rms1).sum(0), "dpre": dpre, "dgate": dgate}
