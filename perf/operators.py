"""The feed-forward half of a transformer block, operator by operator: the
residual addition with its root-mean-square norm (in the stream's type, or in
e4m3 with a scale for each token), the gated projections with their activation
and product, and the backward pass of both.

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
def _norm(name, m, d, dtype="bf16", wdtype="bf16", residual=True, fp8=False):
    return {"name": name, "op": "norm", "m": m, "d": d, "dtype": dtype, "wdtype": wdtype, "residual": residual,
            "fp8": fp8}


def _norm_bwd(name, m, d, dtype="bf16", wdtype="bf16", residual=True):
    return {"name": name, "op": "norm_backward", "m": m, "d": d, "dtype": dtype, "wdtype": wdtype,
            "residual": residual}


def _ffn(name, m, k, f, dtype="bf16", act="silu", save=False):
    return {"name": name, "op": "ffn", "m": m, "k": k, "f": f, "dtype": dtype, "act": act, "save": save}


def _ffn_bwd(name, m, k, f, act="silu"):
    return {"name": name, "op": "ffn_backward", "m": m, "k": k, "f": f, "act": act}


def listed():
    return [
        # one token being generated: the norm of its hidden state, quantised for an e4m3 projection
        _norm("norm_token_e4m3", 1, 5120, fp8=True),
        # a ragged batch of prompts in half precision with an odd row length and fp32 norm weights, first
        # norm of a network (nothing to add yet)
        _norm("norm_ragged_fp16", 1333, 1027, dtype="fp16", wdtype="fp32", residual=False),
        # a long prompt, stream in bf16, the next projection in e4m3
        _norm("norm_prompt_e4m3", 8192, 5120, fp8=True),
        # the same norm in a training step: bf16 in and out, and its gradient
        _norm("norm_train", 8192, 4096),
        _norm_bwd("norm_backward_train", 8192, 4096),
        # a small fine-tuning batch with the stream and the weights in fp32, odd sizes
        _norm_bwd("norm_backward_ragged_fp32", 777, 1530, dtype="fp32", wdtype="fp32", residual=False),
        # one token through the gated projections: the weights' bytes
        _ffn("ffn_token", 1, 5120, 13824),
        # a batch of tokens being generated, e4m3 weights and activations
        _ffn("ffn_decode_e4m3", 48, 5120, 13824, dtype="e4m3"),
        # a small model's ragged batch, gelu
        _ffn("ffn_small_gelu", 200, 520, 1416, act="gelu"),
        # a training step: forward with the pre-activations kept, and the backward pass
        _ffn("ffn_train", 4096, 5120, 13824, save=True),
        _ffn_bwd("ffn_backward_train", 4096, 5120, 13824),
        # a ragged fine-tuning batch of a smaller model
        _ffn_bwd("ffn_backward_ragged", 333, 2048, 5632, act="gelu_tanh"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "ffn", "ffn", "ffn_backward"])
    if op in ("norm", "norm_backward"):
        d = _log(rng, 64, 16384)
        if rng.random() < 0.5:
            d = (d + 7) // 8 * 8
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        wdtype = rng.choice([dtype, "fp32"])
        cap = (8192 * 4096) // (2 if dtype == "fp32" else 1)
        m = max(1, min(_log(rng, 1, 16384), cap // d))
        case = {"op": op, "m": m, "d": d, "dtype": dtype, "wdtype": wdtype, "residual": rng.random() < 0.7}
        if op == "norm":
            case["fp8"] = rng.random() < 0.5
        return case
    m = _log(rng, 1, 4096)
    k = max(16, _log(rng, 128, 8192) // 16 * 16)
    f = max(8, _log(rng, 128, 16384) // 8 * 8)
    f = min(f, (4096 * 5120 * 13824) // (m * k) // 8 * 8)
    act = rng.choice(["silu", "silu", "gelu", "gelu_tanh"])
    if op == "ffn_backward":
        return {"op": op, "m": m, "k": k, "f": f, "act": act}
    dtype = rng.choice(["bf16", "e4m3"])
    return {"op": op, "m": m, "k": k, "f": f, "dtype": dtype, "act": act,
            "save": dtype == "bf16" and rng.random() < 0.4}


# ---------------------------------------------------------------- inputs
def _rows_to_e4m3(t):
    """Rows of fp32 t as e4m3 with one scale each: what the norm and a weight loader hand over."""
    s = t.abs().amax(1) / E4M3_MAX
    s = torch.where(s == 0, torch.ones_like(s), s)
    return (t / s[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(1000 + seed)

    def normal(*shape, std=1.0):
        return torch.empty(*shape, device=DEV).normal_(0.0, std, generator=g)

    s = dict(case)
    m = case["m"]
    if case["op"] in ("norm", "norm_backward"):
        t, wt, d = DTYPES[case["dtype"]], DTYPES[case["wdtype"]], case["d"]
        # a stream's channels differ in size: a few are much larger than the rest
        size = torch.exp(normal(d, std=0.7))
        s["weight"] = (1.0 + normal(d, std=0.2)).to(wt)
        if case["op"] == "norm":
            s["x"] = (normal(m, d) * size).to(t)
            s["res"] = (normal(m, d, std=2.0) * size).to(t) if case["residual"] else None
        else:
            s["h"] = (normal(m, d, std=2.0) * size).to(t)
            s["dy"] = normal(m, d, std=0.1).to(t)
            s["dh"] = normal(m, d, std=0.1).to(t) if case["residual"] else None
        return s
    k, f = case["k"], case["f"]
    x = normal(m, k)
    w = normal(2 * f, k, std=1.0 / math.sqrt(k))
    if case.get("dtype") == "e4m3":
        s["x"], s["x_scale"] = _rows_to_e4m3(x)
        s["w"], s["w_scale"] = _rows_to_e4m3(w)
        return s
    s["x"], s["w"] = x.to(torch.bfloat16), w.to(torch.bfloat16)
    if case["op"] == "ffn_backward":
        s["gu"] = (s["x"].float() @ s["w"].float().t()).to(torch.bfloat16)
        s["dout"] = normal(m, f, std=0.1).to(torch.bfloat16)
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    if own:
        return _run_own(s)
    return {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "ffn": _plain_ffn,
            "ffn_backward": _plain_ffn_backward}[s["op"]](s)


def _run_own(s):
    import layout_folding_gb300 as lf
    if s["op"] == "norm":
        y, h, scale = lf.add_rms_norm(s["x"], s["weight"], residual=s["res"], eps=EPS, fp8=s["fp8"])
        return {"y": y, "h": h if s["residual"] else None, "scale": scale}
    if s["op"] == "norm_backward":
        dx, dw = lf.add_rms_norm_backward(s["dy"], s["h"], s["weight"], dh=s["dh"], eps=EPS)
        return {"dx": dx, "dw": dw}
    if s["op"] == "ffn":
        if s["dtype"] == "e4m3":
            out, gu = lf.gated_ffn(s["x"], s["w"], act=s["act"], x_scale=s["x_scale"], w_scale=s["w_scale"])
        else:
            out, gu = lf.gated_ffn(s["x"], s["w"], act=s["act"], want_gu=s["save"])
        return {"out": out, "gu": gu}
    dx, dw = lf.gated_ffn_backward(s["dout"], s["x"], s["w"], s["gu"], act=s["act"])
    return {"dx": dx, "dw": dw}


def _plain_norm(s):
    t = s["x"].dtype
    h = s["x"]
    if s["res"] is not None:
        h = (s["x"].float() + s["res"].float()).to(t)  # the stream is kept in its type; the norm reads what is kept
    hf = h.float()
    y = hf * torch.rsqrt(hf.square().mean(1, keepdim=True) + EPS) * s["weight"].float()
    h = h if s["residual"] else None
    if not s["fp8"]:
        return {"y": y.to(t), "h": h, "scale": None}
    scale = y.abs().amax(1) / E4M3_MAX
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    q = (y / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return {"y": q, "h": h, "scale": scale}


def _plain_norm_backward(s):
    h, w = s["h"].float(), s["weight"].float()
    dy = s["dy"].float()
    r = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
    xh = h * r
    g = dy * w
    dx = r * (g - xh * (g * xh).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    dw = (dy * xh).sum(0)
    return {"dx": dx.to(s["h"].dtype), "dw": dw.to(s["weight"].dtype)}


def _act(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    if act == "gelu":
        return 0.5 * g * (1 + torch.erf(g * math.sqrt(0.5)))
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))


def _act_slope(g, act):
    if act == "silu":
        sig = 1 / (1 + torch.exp(-g))
        return sig * (1 + g * (1 - sig))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(g * math.sqrt(0.5))) + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    th = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * (1 + th) + 0.5 * g * (1 - th * th) * c * (1 + 3 * 0.044715 * g * g)


def _plain_ffn(s):
    f = s["f"]
    gu = s["x"].float() @ s["w"].float().t()
    if s["dtype"] == "e4m3":
        gu = gu * s["x_scale"][:, None] * s["w_scale"][None, :]
    out = _act(gu[:, :f], s["act"]) * gu[:, f:]
    return {"out": out.to(torch.bfloat16), "gu": gu.to(torch.bfloat16) if s["save"] else None}


def _plain_ffn_backward(s):
    f = s["f"]
    g, u = s["gu"][:, :f].float(), s["gu"][:, f:].float()
    da = s["dout"].float()
    dgu = torch.cat([da * u * _act_slope(g, s["act"]), da * _act(g, s["act"])], 1)
    dx = dgu @ s["w"].float()
    dw = dgu.t() @ s["x"].float()
    return {"dx": dx.to(torch.bfloat16), "dw": dw.to(torch.bfloat16)}


# ---------------------------------------------------------------- work
def work(case):
    m = case["m"]
    if case["op"] in ("norm", "norm_backward"):
        d, b, wb = case["d"], BYTES[case["dtype"]], BYTES[case["wdtype"]]
        n = m * d
        if case["op"] == "norm":
            bytes_ = n * b + (2 * n * b if case["residual"] else 0) + d * wb
            bytes_ += n + 4 * m if case["fp8"] else n * b
            return {"bytes": bytes_, "flops": 6 * n}
        return {"bytes": n * b * (4 if case["residual"] else 3) + 2 * d * wb, "flops": 12 * n}
    k, f = case["k"], case["f"]
    if case["op"] == "ffn":
        if case["dtype"] == "e4m3":
            bytes_ = m * k + 2 * f * k + 4 * (m + 2 * f) + 2 * m * f
        else:
            bytes_ = 2 * (m * k + 2 * f * k + m * f * (3 if case["save"] else 1))
        return {"bytes": bytes_, "flops": 4 * m * f * k}
    return {"bytes": 2 * (2 * m * k + 4 * f * k + 3 * m * f), "flops": 8 * m * f * k}


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The definitions, evaluated in 64 bits on prepare's inputs."""
    s = prepare(case, seed)
    one = torch.ones((), dtype=torch.float64, device=DEV)
    if case["op"] == "norm":
        total = s["x"].double()
        if s["res"] is not None:
            total = total + s["res"].double()
        kept = total.to(s["x"].dtype).double()
        rms = ((kept ** 2).sum(1, keepdim=True) / case["d"] + EPS) ** 0.5
        y = kept / rms * s["weight"].double()
        scale = None
        if case["fp8"]:
            scale = y.abs().max(1).values / E4M3_MAX
            scale = torch.where(scale == 0, one, scale)
            y = y / scale[:, None]
        return {"y": y, "h": total if case["residual"] else None, "scale": scale}
    if case["op"] == "norm_backward":
        h, w, dy = s["h"].double(), s["weight"].double(), s["dy"].double()
        d = case["d"]
        rms = ((h ** 2).sum(1, keepdim=True) / d + EPS) ** 0.5
        # y_i = h_i w_i / rms, d rms / d h_j = h_j / (d rms)
        dot = (dy * w * h).sum(1, keepdim=True)
        dx = dy * w / rms - h * dot / (d * rms ** 3)
        if s["dh"] is not None:
            dx = dx + s["dh"].double()
        return {"dx": dx, "dw": (dy * h / rms).sum(0)}
    f, act = case["f"], case["act"]

    def phi(v):  # act(v) = v * phi(v)
        if act == "silu":
            return torch.special.expit(v)
        if act == "gelu":
            return torch.special.ndtr(v)
        return torch.special.expit(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))

    if case["op"] == "ffn":
        x, w = s["x"].double(), s["w"].double()
        if case["dtype"] == "e4m3":
            x, w = x * s["x_scale"].double()[:, None], w * s["w_scale"].double()[:, None]
        gate, up = x @ w[:f].t(), x @ w[f:].t()
        return {"out": gate * phi(gate) * up, "gu": torch.cat([gate, up], 1) if case["save"] else None}
    gate, up = s["gu"][:, :f].double(), s["gu"][:, f:].double()
    dout, x, w = s["dout"].double(), s["x"].double(), s["w"].double()
    p = phi(gate)
    if act == "silu":
        dphi = p * (1 - p)
    elif act == "gelu":
        dphi = torch.exp(-gate ** 2 / 2) / math.sqrt(2 * math.pi)
    else:
        dphi = p * (1 - p) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * gate ** 2)
    dgate, dup = dout * up * (p + gate * dphi), dout * gate * p
    return {"dx": dgate @ w[:f] + dup @ w[f:], "dw": torch.cat([dgate.t() @ x, dup.t() @ x])}
