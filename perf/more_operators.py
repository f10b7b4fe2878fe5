"""What stands around the products of a quantized feed-forward block, serving and training: what is timed, and its plain forms.

Six groups of calls on four operators:

  norm          h = x + residual kept in bf16, and y = h / rms(h) * weight as E4M3 codes with a scale for each token (the
                operand of the products on 8-bit activations);
  norm_grad     the gradients of y = h / rms(h) * weight for h (the gradient that reaches h on its own path added) and weight;
  product       C = A W^T from 8-bit integers: activations quantized with a scale for each token, weights with one for each
                channel;
  norm_product  a norm that writes 8-bit integers, and the product that reads them;
  balance       a router's balance loss, the tokens that each expert received, and the gradient for the router's logits;
  clip          the norm over all gradients of a step, and the gradients scaled down to a largest norm.
"""
import math
import random

import torch

own = False

F32, F64, BF16, I32, E4M3 = torch.float32, torch.float64, torch.bfloat16, torch.int32, torch.float8_e4m3fn
EPS = 1e-6


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one token of a serving step: launches and latency
        {"name": "norm_token", "op": "norm", "T": 1, "K": 8192, "w": "bf16"},
        # a prefill batch with an odd number of tokens
        {"name": "norm_batch", "op": "norm", "T": 16385, "K": 8192, "w": "bf16"},
        # a small micro-batch's gradient
        {"name": "norm_grad_small", "op": "norm_grad", "T": 77, "K": 7168, "w": "fp32"},
        # and that of a training batch
        {"name": "norm_grad_batch", "op": "norm_grad", "T": 16384, "K": 8192, "w": "bf16"},
        # decoding one token through the widest layer: the weight's bytes
        {"name": "product_token", "op": "product", "T": 1, "N": 28672, "K": 8192},
        # a few requests together through a down projection, ragged in both directions
        {"name": "product_ragged", "op": "product", "T": 205, "N": 7160, "K": 2048},
        # a prefill
        {"name": "product_prefill", "op": "product", "T": 4096, "N": 8192, "K": 8192},
        # a serving step of some requests: the norm and the product that reads it
        {"name": "norm_product", "op": "norm_product", "T": 33, "N": 8192, "K": 8192, "w": "bf16"},
        # a handful of tokens' router
        {"name": "balance_small", "op": "balance", "T": 16, "E": 64, "k": 8, "off": 0.0},
        # a training batch's, padded tokens left out
        {"name": "balance_batch", "op": "balance", "T": 65537, "E": 256, "k": 8, "off": 0.125},
        # norms, biases and small matrices of odd sizes
        {"name": "clip_small", "op": "clip", "big": 0, "n": 24, "lo": 1, "hi": 4096, "pick": 3, "shift": 1, "most": 0.1},
        # the up projections of one layer's 64 experts (2048 x 7168 each) and what else the layer trains
        {"name": "clip_layer", "op": "clip", "big": 64 * 2048 * 7168, "n": 20, "lo": 64, "hi": 1 << 24, "pick": 5, "shift": 0,
         "most": 1.0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "norm_grad", "product", "product", "norm_product", "balance", "clip"))
    if op in ("norm", "norm_grad"):
        return {"op": op, "T": _log_int(rng, 1, 16384), "K": 16 * _log_int(rng, 4, 512), "w": rng.choice(("bf16", "fp32"))}
    if op == "product":
        return {"op": op, "T": _log_int(rng, 1, 4096), "N": 8 * _log_int(rng, 8, 1024), "K": 128 * _log_int(rng, 1, 64)}
    if op == "norm_product":
        return {"op": op, "T": _log_int(rng, 1, 1024), "N": 8 * _log_int(rng, 8, 1024), "K": 128 * _log_int(rng, 1, 64),
                "w": rng.choice(("bf16", "fp32"))}
    if op == "balance":
        return {"op": op, "T": _log_int(rng, 1, 65536), "E": rng.choice((8, 16, 37, 64, 128, 250, 256)), "k": rng.randint(1, 8),
                "off": rng.choice((0.0, 0.125, 0.5))}
    hi = _log_int(rng, 64, 1 << 24)
    return {"op": op, "big": rng.choice((0, 0, 33554433)), "n": _log_int(rng, 1, 48), "lo": 1, "hi": hi, "pick": rng.randrange(1 << 20),
            "shift": rng.randint(0, 3), "most": rng.choice((0.01, 1.0, 1e6))}


# --------------------------------------------------------------- the inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, std=1.0, dtype=BF16):
    return (torch.randn(*shape, device="cuda", generator=g) * std).to(dtype)


def _tokens(g, T, K):
    """Activations: normal, some channels ten times the others."""
    x = torch.randn(T, K, device="cuda", generator=g)
    x[:, torch.randint(0, K, (max(1, K // 100),), device="cuda", generator=g)] *= 10
    return x.to(BF16)


def _norm_weight(g, K, w):
    return (1 + 0.1 * torch.randn(K, device="cuda", generator=g)).to(BF16 if w == "bf16" else F32)


def _weight8(g, N, K):
    """Codes and scales of a normally distributed weight in 8-bit integers, one scale for each of its N channels."""
    codes = torch.empty(N, K, dtype=torch.int8, device="cuda")
    for part in codes.split(max(1, (1 << 27) // K)):
        part.copy_(torch.clamp(torch.round(torch.randn(part.shape, device="cuda", generator=g) * 30), -127, 127))
    return {"codes": codes, "scales": 0.02 / 30 * (1 + 0.2 * torch.rand(N, device="cuda", generator=g))}


def _sizes(case):
    r = random.Random(case["pick"])
    return ([case["big"]] if case["big"] else []) + [_log_int(r, case["lo"], case["hi"]) for _ in range(case["n"])]


def prepare(case, seed):
    g, c = _gen(seed), dict(case)
    op, st = c["op"], {"case": c}
    if op in ("norm", "norm_product"):
        st |= {"x": _normal(g, c["T"], c["K"], std=0.3), "residual": _tokens(g, c["T"], c["K"]), "weight": _norm_weight(g, c["K"], c["w"])}
    elif op == "norm_grad":
        st |= {"h": _tokens(g, c["T"], c["K"]), "weight": _norm_weight(g, c["K"], c["w"]),
               "dy": _normal(g, c["T"], c["K"], std=0.01), "dh": _normal(g, c["T"], c["K"], std=0.01)}
    elif op == "product":
        st["x"] = _tokens(g, c["T"], c["K"])
    elif op == "balance":
        T, E, k = c["T"], c["E"], min(c["k"], c["E"])
        st["logits"] = torch.randn(T, E, device="cuda", generator=g) + 0.5 * torch.randn(E, device="cuda", generator=g)
        st["ids"] = torch.topk(st["logits"], k, dim=1).indices.to(I32).contiguous()
        st["mask"] = torch.rand(T, device="cuda", generator=g) >= c["off"] if c["off"] else None
    else:
        st["grads"], st["out"] = [], []
        for i, n in enumerate(_sizes(c)):
            # the gradients of a step lie one behind the other in a buffer: not every one begins at a multiple of 16 bytes
            kind, std = (BF16, 0.01) if i % 3 == 2 else (F32, 0.001 * (1 + i % 5))
            st["grads"].append(torch.randn(n + c["shift"], device="cuda", generator=g).mul_(std).to(kind)[c["shift"]:])
            st["out"].append(torch.zeros(n + c["shift"], device="cuda", dtype=kind)[c["shift"]:])
    if op in ("product", "norm_product"):
        st["w"] = _weight8(g, c["N"], c["K"])
    return st


# ---------------------------------------------------------- the plain forms

def _normed(h, weight):
    v = h.float()
    return v / torch.sqrt((v * v).mean(1, keepdim=True) + EPS) * weight.float()


def _rows8(v):
    """(codes as whole numbers, scales) of rows of 32-bit values in 8-bit integers: each value times the 32-bit 127 / amax,
    rounded to nearest, ties to even (a product of 24 bits by 24 has its place in 64)."""
    most = torch.clamp_min(v.abs().amax(1), 1e-12)
    return torch.round(v.double() * (127 / most).double()[:, None]).float(), most / 127


def _pow2(e):
    """2^e for whole e in -126 .. 127, by its exponent bits: a library's exp2 need not be exact."""
    return ((e.to(I32) + 127) << 23).view(F32)


def _rows_e4m3(v):
    s = torch.clamp_min(v.abs().amax(1), 1e-12) / 448
    q = v / s[:, None]
    step = _pow2(torch.clamp_min(torch.frexp(q).exponent - 1, -6) - 3)
    return torch.clamp(torch.round(q / step) * step, -448, 448).to(E4M3), s


def _probabilities(logits):
    most = logits.amax(1, keepdim=True)
    p = torch.exp(logits - torch.where(most == -math.inf, torch.zeros_like(most), most))
    total = p.sum(1, keepdim=True)
    return torch.where(total == 0, torch.zeros_like(p), p / total)


def _plain(st):
    c = st["case"]
    op = c["op"]
    if op == "norm":
        h = (st["x"].float() + st["residual"].float()).to(BF16)
        return (h, *_rows_e4m3(_normed(h, st["weight"])))
    if op == "norm_grad":
        v, dy, w = st["h"].float(), st["dy"].float(), st["weight"].float()
        r = 1 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)
        n, dn = v * r, dy * w
        dx = st["dh"].float() + r * (dn - n * (dn * n).mean(1, keepdim=True))
        return dx.to(BF16), (dy * n).sum(0)
    if op in ("product", "norm_product"):
        if op == "product":
            h, v = None, st["x"].float()
        else:
            h = (st["x"].float() + st["residual"].float()).to(BF16)
            v = _normed(h, st["weight"])
        a, s = _rows8(v)
        y = (a @ st["w"]["codes"].float().t()) * s[:, None] * st["w"]["scales"]
        return y.to(BF16) if h is None else (h, y.to(BF16))
    if op == "balance":
        logits, ids = st["logits"], st["ids"].long()
        T, E = logits.shape
        here = st["mask"] if st["mask"] is not None else torch.ones(T, dtype=torch.bool, device=logits.device)
        n = here.sum().clamp_min(1).double()
        counts = torch.zeros(E, dtype=I32, device=logits.device)
        counts.index_add_(0, ids.reshape(-1), here[:, None].expand_as(ids).reshape(-1).to(I32))
        p = _probabilities(logits) * here[:, None]
        slope = E * counts.double() / (ids.shape[1] * n * n)
        loss = (slope * p.double().sum(0)).sum()
        slope = slope.float()
        return loss.float(), counts, p * (slope - (p * slope).sum(1, keepdim=True))
    square = torch.stack([g.double().square().sum() for g in st["grads"]]).sum()
    norm = torch.sqrt(square)
    by = torch.clamp_max(c["most"] / (norm + EPS), 1.0).float()
    return norm.float(), [(g.float() * by).to(g.dtype) for g in st["grads"]]


# ------------------------------------------------------ the framework's calls

def _own(st):
    import w4_gemm_amd as q4
    c = st["case"]
    op = c["op"]
    if op == "norm":
        y = q4.empty_q4("fp8_row", c["T"], c["K"])
        h, _, _ = q4.q4_rmsnorm(st["x"], st["weight"], EPS, residual=st["residual"], y_q=y)
        return h, y.codes.view(E4M3), y.scales
    if op == "norm_grad":
        return q4.q4_rmsnorm_backward(st["dy"], st["h"], st["weight"], EPS, dh=st["dh"])
    if op in ("product", "norm_product"):
        w = st["w"]
        W = q4.Q4Tensor(q4.INT8_ROW, c["N"], c["K"], w["codes"], w["scales"])
        y = torch.empty(c["T"], c["N"], dtype=BF16, device="cuda")
        if op == "product":
            return q4.q4_gemm(q4.quantize(st["x"], "int8_row"), W, y)
        a = q4.empty_q4("int8_row", c["T"], c["K"])
        h, _, _ = q4.q4_rmsnorm(st["x"], st["weight"], EPS, residual=st["residual"], y_q=a)
        return h, q4.q4_gemm(a, W, y)
    if op == "balance":
        loss, counts, slopes = q4.q4_moe_balance(st["logits"], st["ids"], mask=st["mask"])
        return loss, counts, q4.q4_moe_balance_backward(st["logits"], slopes, mask=st["mask"])
    norm = q4.q4_grad_clip(st["grads"], c["most"], out=st["out"])
    return norm, st["out"]


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------- the work

def work(case):
    c = case
    op = c["op"]
    if op == "clip":
        kinds = [(2 if i % 3 == 2 else 4, n) for i, n in enumerate(_sizes(c))]
        return {"bytes": sum(2 * b * n for b, n in kinds), "flops": sum(3 * n for _, n in kinds)}
    if op == "balance":
        n = c["T"] * c["E"]
        return {"bytes": 8 * n + 4 * c["T"] * min(c["k"], c["E"]), "flops": 12 * n}
    n = c["T"] * c["K"]
    if op == "norm":
        return {"bytes": 7 * n + 4 * c["T"], "flops": 6 * n}
    if op == "norm_grad":
        return {"bytes": 8 * n + 8 * c["K"], "flops": 12 * n}
    # the activations in bf16 come in (with a residual's sum: two in, one out), the weight's bytes, the products
    return {"bytes": (2 if op == "product" else 6) * n + c["N"] * c["K"] + 2 * c["T"] * c["N"], "flops": 2 * n * c["N"]}


# ------------------------------------------------------- in 64 bits, apart

def _exact_rows8(v):
    most = v.abs().amax(1).clamp(min=1e-12)
    return torch.clamp((v * (127 / most)[:, None]).round(), -127, 127), most / 127


def _exact_norm(st):
    total = st["x"].to(F64) + st["residual"].to(F64)
    h = total.to(BF16).to(F64)
    return total, torch.nn.functional.rms_norm(h, h.shape[1:], st["weight"].to(F64), EPS)


def exact(case, seed):
    st, c = prepare(case, seed), case
    op = c["op"]
    if op == "norm":
        h, y = _exact_norm(st)
        s = y.abs().amax(1).clamp(min=1e-12) / 448
        return h, y / s[:, None], s           # the values that the codes round
    if op == "norm_grad":
        h, w = (st[n].to(F64).requires_grad_() for n in ("h", "weight"))
        y = h * torch.rsqrt(h.pow(2).mean(1, keepdim=True) + EPS) * w
        return torch.autograd.grad((y * st["dy"].to(F64)).sum() + (h * st["dh"].to(F64)).sum(), (h, w))
    if op in ("product", "norm_product"):
        h, y = (None, st["x"].to(F64)) if op == "product" else _exact_norm(st)
        a, s = _exact_rows8(y)
        w = st["w"]["codes"].to(F64) * st["w"]["scales"].to(F64)[:, None]
        out = (a * s[:, None]) @ w.t()
        return out if h is None else (h, out)
    if op == "balance":
        logits = st["logits"].to(F64).requires_grad_()
        here = torch.arange(c["T"], device="cuda") if st["mask"] is None else st["mask"].nonzero()[:, 0]
        if not here.numel():
            return torch.zeros((), dtype=F64, device="cuda"), None, torch.zeros_like(logits).detach()
        ids = st["ids"][here].long()
        share = torch.bincount(ids.reshape(-1), minlength=c["E"]).to(F64) / ids.numel()
        loss = c["E"] * torch.dot(share, torch.softmax(logits[here], 1).mean(0))
        grad, = torch.autograd.grad(loss, logits)
        return loss.detach(), None, grad
    norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(g.to(F64)) for g in st["grads"]]))
    by = min(1.0, c["most"] / (norm.item() + EPS))
    return norm, [g.to(F64) * by for g in st["grads"]]
