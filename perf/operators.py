"""The backward pass of a mixture-of-experts layer on 4-bit weights: what is timed, and its plain forms.

Five groups of calls, in the order in which a training step meets them:

  dispatch      each token's chosen experts -> expert-major row order (stable), and the tokens' rows copied into it;
  swiglu        h = silu(g) u with [g u] kept in 8 bits for later, and later the gradient of [g u] from what was kept;
  wgrad         an activation kept in 8 bits, and the weight gradient dW = dC^T A from it, dense or per expert;
  dgrad         the gradient of a W4 product for its activations, dA = dC W', dense or per expert;
  combine_grad  the gradients of the gated combine (expert outputs and gates), of the softmax gates (router logits) and of
                the copy of the tokens into expert order.

The 8-bit formats hold blocks of 32 values with one power-of-two scale, the least s with max|x| <= top s: integers
(top 127) or E4M3 (top 448), rounded to nearest, ties to even.
"""
import math

import torch

own = False

F32, F64, BF16, I32 = torch.float32, torch.float64, torch.bfloat16, torch.int32
LEAST_EXPONENT = -111
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one token of a serving step: launches and latency
        {"name": "dispatch_token", "op": "dispatch", "T": 1, "k": 8, "E": 64, "K": 7168, "dropped": 0.0},
        # a training batch with an odd number of tokens, where an eighth of the choices belongs to another rank
        {"name": "dispatch_batch", "op": "dispatch", "T": 16385, "k": 8, "E": 64, "K": 7168, "dropped": 0.125},
        # a small micro-batch through the SwiGLU of its experts, E4M3
        {"name": "swiglu_small", "op": "swiglu", "P": 33, "I": 2048, "fmt": "mxfp8"},
        # all routed rows of a training batch, integers
        {"name": "swiglu_batch", "op": "swiglu", "P": 32768, "I": 2048, "fmt": "mxint8"},
        # a small layer's weight gradient over a few tokens
        {"name": "wgrad_small", "op": "wgrad", "E": 0, "T": 77, "k": 1, "N": 512, "K": 512, "fmt": "mxint8"},
        # a dense layer of the prefill and W4A4 sizes
        {"name": "wgrad_dense", "op": "wgrad", "E": 0, "T": 8192, "k": 1, "N": 8192, "K": 8192, "fmt": "mxint8"},
        # the up projection of all experts, the tokens' rows read through the routing, ragged groups
        {"name": "wgrad_experts", "op": "wgrad", "E": 64, "T": 4096, "k": 8, "N": 2048, "K": 7168, "fmt": "mxfp8"},
        # a small layer, few tokens
        {"name": "dgrad_small", "op": "dgrad", "E": 0, "T": 77, "k": 1, "N": 512, "K": 512, "fmt": "nvfp4"},
        # a dense layer of the prefill size
        {"name": "dgrad_dense", "op": "dgrad", "E": 0, "T": 4096, "k": 1, "N": 8192, "K": 8192, "fmt": "int4"},
        # the up projection of all experts, ragged groups
        {"name": "dgrad_experts", "op": "dgrad", "E": 64, "T": 4096, "k": 8, "N": 2048, "K": 7168, "fmt": "mxfp4"},
        # the combine's gradient for a handful of tokens
        {"name": "combine_grad_small", "op": "combine_grad", "T": 16, "k": 8, "E": 64, "K": 7168, "dropped": 0.0},
        # and for a training batch
        {"name": "combine_grad_batch", "op": "combine_grad", "T": 8192, "k": 8, "E": 64, "K": 7168, "dropped": 0.0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("dispatch", "swiglu", "wgrad", "wgrad", "dgrad", "dgrad", "combine_grad"))
    if op in ("dispatch", "combine_grad"):
        k = rng.randint(1, 8)
        return {"op": op, "T": _log_int(rng, 1, 16384 if op == "dispatch" else 8192), "k": k,
                "E": rng.choice((8, 16, 37, 64, 128, 256)), "K": 8 * _log_int(rng, 8, 896),
                "dropped": rng.choice((0.0, 0.125, 0.5))}
    if op == "swiglu":
        return {"op": op, "P": _log_int(rng, 1, 32768), "I": 32 * _log_int(rng, 1, 64), "fmt": rng.choice(("mxint8", "mxfp8"))}
    if rng.random() < 0.5:      # dense
        c = {"op": op, "E": 0, "T": _log_int(rng, 1, 8192 if op == "wgrad" else 4096), "k": 1}
        c["N"] = 16 * _log_int(rng, 8, 512)
        c["K"] = 32 * _log_int(rng, 4, 256) if op == "wgrad" else 512 * _log_int(rng, 1, 16)
    else:
        c = {"op": op, "E": rng.choice((4, 8, 16, 32, 64)), "T": _log_int(rng, 1, 4096), "k": rng.randint(1, 4)}
        c["N"] = 16 * _log_int(rng, 8, 128)
        c["K"] = 32 * _log_int(rng, 8, 224) if op == "wgrad" else 512 * _log_int(rng, 1, 14)
    c["fmt"] = rng.choice(("mxint8", "mxfp8")) if op == "wgrad" else rng.choice(("int4", "mxfp4", "nvfp4"))
    return c


# --------------------------------------------------------------- the inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, std=1.0):
    return (torch.randn(*shape, device="cuda", generator=g) * std).to(BF16)


def _choices(g, T, k, E, dropped):
    """Router logits (some experts are liked better), the chosen experts, -1 where a choice is not this program's to run."""
    logits = torch.randn(T, E, device="cuda", generator=g) + 0.5 * torch.randn(E, device="cuda", generator=g)
    ids = torch.topk(logits, k, dim=1).indices.to(I32)
    if dropped:
        ids = torch.where(torch.rand(T, k, device="cuda", generator=g) < dropped, -1, ids)
    return logits, ids.to(I32).contiguous()


def _weight_tiled(g, fmt, rows, cols):
    """Codes and scales of a normally distributed weight in the tiled layout: codes 16-row x 128-column tiles of 1 KB, scales
    of four tiles together."""
    rt, q = (rows + 15) // 16, cols // 512
    codes = torch.empty(rt * q * 4096, dtype=torch.uint8, device="cuda")
    for part in codes.split(1 << 27):
        z = torch.randn(2, part.numel(), device="cuda", generator=g)
        if fmt == "int4":
            n = torch.clamp(torch.round(z * 2.6), -8, 7).to(torch.int16) & 15
        else:
            mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
            n = torch.bucketize(torch.abs(z) * 2.2, mid).to(torch.int16) + 8 * (z < 0)
        part.copy_((n[0] + 16 * n[1]).to(torch.uint8))
    gs = None
    if fmt == "int4":
        s = 0.02 / 2.6 * (1 + 0.2 * torch.rand(rt * q * 64, device="cuda", generator=g))
        scales = s.to(torch.float16).view(torch.int16)
    elif fmt == "mxfp4":
        scales = torch.randint(118, 120, (rt * q * 256,), device="cuda", generator=g).to(torch.uint8)
    else:
        scales = torch.randint(0x60, 0x78, (rt * q * 512,), device="cuda", generator=g).to(torch.uint8)  # 32 .. 240
        gs = torch.full((1,), 0.02 / 2.2 / 100, device="cuda")
    return {"codes": codes, "scales": scales, "gs": gs}


def prepare(case, seed):
    g, c = _gen(seed), dict(case)
    st = {"case": c}
    op = c["op"]
    if op in ("dispatch", "combine_grad"):
        T, k, E, K = c["T"], min(c["k"], c["E"]), c["E"], c["K"]
        logits, ids = _choices(g, T, k, E, c["dropped"])
        P = T * k
        if op == "dispatch":
            st |= {"ids": ids, "x": _normal(g, T, K), "gather": torch.zeros(P, dtype=I32, device="cuda"),
                   "xs": torch.zeros(P, K, dtype=BF16, device="cuda")}
        else:
            offsets, _, inv = _sort(ids, E)
            w = torch.softmax(logits, 1).gather(1, ids.clamp_min(0).long())
            st |= {"logits": logits, "ids": ids, "inv": inv, "weights": w.contiguous(), "dout": _normal(g, T, K, std=0.01),
                   "y": _normal(g, P, K), "dxs": _normal(g, P, K, std=0.01), "dy": torch.zeros(P, K, dtype=BF16, device="cuda")}
    elif op == "swiglu":
        P, I = c["P"], c["I"]
        st |= {"gu": _normal(g, P, 2 * I, std=1.5), "dh": _normal(g, P, I, std=0.01)}
    else:
        T, N, K, E = c["T"], c["N"], c["K"], c["E"]
        if E:
            k = min(c["k"], E)
            _, ids = _choices(g, T, k, E, 0.0)
            offsets, gather, _ = _sort(ids, E)
            st |= {"offsets": offsets, "gather": gather, "most": int((offsets[1:] - offsets[:-1]).max())}
            P = T * k
        else:
            P = T
        st["dc"] = _normal(g, P, N, std=0.01)
        if op == "wgrad":
            x = torch.randn(T, K, device="cuda", generator=g)
            x[:, torch.randint(0, K, (max(1, K // 100),), device="cuda", generator=g)] *= 10     # outlier channels
            st["x"] = x.to(BF16)
        else:
            st["w"] = _weight_tiled(g, c["fmt"], max(E, 1) * N, K)
    return st


# ---------------------------------------------------------- the plain forms

def _sort(ids, E):
    """(offsets [E + 1], gather [P], inv [T, k]); gather is whole here, its rows behind offsets[E] without meaning."""
    T, k = ids.shape
    flat = torch.where((ids >= 0) & (ids < E), ids, E).reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=ids.device).index_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat((counts.new_zeros(1), torch.cumsum(counts[:E], 0)))
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel(), device=ids.device)
    inv = torch.where(flat < E, pos, -1).reshape(T, k)
    return offsets.to(I32), (order // k).to(I32), inv.to(I32)


def _pow2(e):
    """2^e for whole e in -126 .. 127, by its exponent bits: a library's pow need not be exact."""
    return ((e.to(I32) + 127) << 23).view(F32)


def _kept8(x, fmt):
    """The values that the 8-bit form of x stands for (32 bits)."""
    v = x.float().reshape(x.shape[0], -1, 32)
    m, e = torch.frexp(v.abs().amax(2, keepdim=True))
    top_m, top_e = (0.9921875, 7) if fmt == "mxint8" else (0.875, 9)      # 127 and 448
    s = _pow2(torch.clamp_min(e - top_e + (m > top_m).to(e.dtype), LEAST_EXPONENT))
    q = v / s
    if fmt == "mxint8":
        q = torch.round(q)
    else:
        step = _pow2(torch.clamp_min(torch.frexp(q).exponent - 1, -6) - 3)
        q = torch.round(q / step) * step
    return (q * s).reshape(x.shape)


def _weight(w, fmt, rows, cols):
    """A tiled weight's values [rows, cols] (32 bits)."""
    rt, s = (rows + 15) // 16, cols // 128
    q = s // 4
    c = w["codes"].view(rt, s, 4, 16, 16).permute(0, 3, 1, 2, 4).reshape(rt * 16, s * 64)
    c = torch.stack((c & 15, c >> 4), dim=2).reshape(rt * 16, cols).to(I32)
    if fmt == "int4":
        v = (c - 16 * (c >= 8)).float()
        sc = w["scales"].view(torch.float16).float().view(rt, q, 16, 4).permute(0, 2, 1, 3).reshape(rt * 16, -1)
    else:
        v = torch.tensor(E2M1 + tuple(-m for m in E2M1), device=c.device)[c]
        if fmt == "mxfp4":
            sc = _pow2(w["scales"].view(rt, q, 4, 16, 4).permute(0, 3, 1, 4, 2).reshape(rt * 16, -1).to(I32) - 127)
        else:
            b = w["scales"].view(rt, q, 4, 16, 4, 2).permute(0, 3, 1, 4, 2, 5).reshape(rt * 16, -1).to(I32)
            e, m = b >> 3, (b & 7).float()
            sc = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * _pow2(e - 7)) * w["gs"]
    return (v.view(rt * 16, sc.shape[1], -1) * sc[:, :, None]).reshape(rt * 16, cols)[:rows]


def _slots(offsets, P, most):
    """Row of each routed row in a table of `most` rows per expert."""
    p = torch.arange(P, device=offsets.device)
    e = (p[:, None] >= offsets[None, 1:]).sum(1)
    return e * most + p - offsets[:-1].long()[e]


def _table(rows, slots, n):
    return torch.zeros(n, rows.shape[1], dtype=rows.dtype, device=rows.device).index_copy_(0, slots, rows)


def _plain(st):
    c = st["case"]
    op = c["op"]
    if op == "dispatch":
        offsets, gather, inv = _sort(st["ids"], c["E"])
        here = torch.arange(gather.numel(), device=gather.device) < offsets[-1]
        gather = torch.where(here, gather, st["gather"])
        return offsets, gather, inv, torch.where(here[:, None], st["x"][gather.long()], st["xs"])
    if op == "combine_grad":
        inv, w, ids, P = st["inv"], st["weights"], st["ids"], st["y"].shape[0]
        has = (inv >= 0)
        row = inv.clamp_min(0).long()
        dout = st["dout"].float()
        dw = (dout[:, None, :] * st["y"].float()[row]).sum(2) * has
        to = torch.where(has, inv, P).reshape(-1).long()      # one row more takes what was dropped
        dy = torch.cat((st["dy"].float(), dout.new_zeros(1, dout.shape[1])))
        dy = dy.index_copy_(0, to, (w[:, :, None] * dout[:, None, :]).reshape(-1, dout.shape[1]))[:P]
        p = torch.exp(st["logits"] - st["logits"].amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
        to_e = torch.zeros(p.shape[0], c["E"] + 1, device=p.device)
        to_e = to_e.scatter_add_(1, torch.where(ids >= 0, ids, c["E"]).long(), dw)[:, :c["E"]]
        dl = p * (to_e - (to_e * p).sum(1, keepdim=True))
        dx = (st["dxs"].float()[row] * has[:, :, None]).sum(1)
        return dy.to(BF16), dw, dl, dx.to(BF16)
    if op == "swiglu":
        gu, I = st["gu"], c["I"]
        g, u = gu[:, :I].float(), gu[:, I:].float()
        h = g / (1 + torch.exp(-g)) * u
        kept = _kept8(gu, c["fmt"])
        g, u, dh = kept[:, :I], kept[:, I:], st["dh"].float()
        sg = 1 / (1 + torch.exp(-g))
        dgu = torch.cat((dh * u * sg * (1 + g * (1 - sg)), dh * g * sg), 1)
        return h.to(BF16), dgu.to(BF16)
    N, K, E, dc = c["N"], c["K"], c["E"], st["dc"]
    if E:
        slots = _slots(st["offsets"], dc.shape[0], st["most"])
        dct = _table(dc.float(), slots, E * st["most"]).view(E, st["most"], N)
    if op == "wgrad":
        x = _kept8(st["x"], c["fmt"])
        if not E:
            return dc.float().t() @ x
        xt = _table(x[st["gather"].long()], slots, E * st["most"]).view(E, st["most"], K)
        return (dct.transpose(1, 2) @ xt).view(E * N, K)
    w = _weight(st["w"], c["fmt"], max(E, 1) * N, K)
    if not E:
        return (dc.float() @ w).to(BF16)
    return (dct @ w.view(E, N, K)).view(-1, K)[slots].to(BF16)


# ------------------------------------------------------ the framework's calls

def _own(st):
    import w4_gemm_amd as q4
    c = st["case"]
    op = c["op"]
    if op == "dispatch":
        offsets, gather, inv = q4.q4_moe_sort(st["ids"], c["E"], gather=st["gather"])
        return offsets, gather, inv, q4.q4_moe_permute(st["x"], inv, st["xs"])
    if op == "combine_grad":
        dy, dw = q4.q4_moe_combine_backward(st["dout"], st["y"], st["inv"], st["weights"], dy=st["dy"])
        dl = q4.q4_moe_topk_backward(st["logits"], st["ids"], dw)
        return dy, dw, dl, q4.q4_moe_permute_backward(st["dxs"], st["inv"])
    if op == "swiglu":
        kept = q4.empty_q4(c["fmt"], c["P"], 2 * c["I"])
        h = q4.q4_swiglu_save(st["gu"], c["I"], kept)
        return h, q4.q4_swiglu_backward(kept, st["dh"])
    if op == "wgrad":
        kept = q4.quantize(st["x"], c["fmt"])
        if c["E"]:
            return q4.q4_grouped_gemm_wgrad(st["dc"], kept, st["gather"], st["offsets"])
        return q4.q4_gemm_wgrad(st["dc"], kept)
    w = st["w"]
    W = q4.Q4Tensor(q4.FORMAT_NAMES[c["fmt"]], max(c["E"], 1) * c["N"], c["K"], w["codes"], w["scales"], w["gs"], q4.LAYOUT_TILED)
    if c["E"]:
        return q4.q4_grouped_gemm_dgrad(st["dc"], st["offsets"], W, c["N"])
    return q4.q4_gemm_dgrad(st["dc"], W)


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------- the work

def work(case):
    c = case
    op = c["op"]
    if op in ("dispatch", "combine_grad"):
        T, E, K = c["T"], c["E"], c["K"]
        P = T * min(c["k"], E)
        kept = round(P * (1 - c["dropped"]))
        if op == "dispatch":
            return {"bytes": 4 * P + 4 * (E + 1) + 4 * kept + 4 * P + 2 * T * K + 2 * kept * K, "flops": 0}
        return {"bytes": 4 * T * K + 6 * kept * K + 16 * P + 8 * T * E, "flops": 4 * kept * K}
    if op == "swiglu":
        n = c["P"] * c["I"]
        return {"bytes": 6 * n + 8 * n + 2 * (2 * n * 33 // 32), "flops": 20 * n}
    E, T, N, K = c["E"], c["T"], c["N"], c["K"]
    M = T * min(c["k"], E) if E else T
    if op == "wgrad":
        return {"bytes": 2 * M * N + 2 * T * K + 4 * max(E, 1) * N * K, "flops": 2 * M * N * K}
    bits = {"int4": 4.125, "mxfp4": 4.25, "nvfp4": 4.5}[c["fmt"]]
    return {"bytes": int(2 * M * N + 2 * M * K + max(E, 1) * N * K * bits / 8), "flops": 2 * M * N * K}


# ------------------------------------------------------- in 64 bits, apart

def _exact_kept8(x, fmt):
    v = x.to(F64).unflatten(1, (-1, 32))
    powers = torch.tensor([2.0 ** e for e in range(LEAST_EXPONENT, 122)], dtype=F64, device=x.device)
    top = 127.0 if fmt == "mxint8" else 448.0
    s = powers[torch.searchsorted(top * powers, v.abs().amax(-1, keepdim=True))]    # the first with amax <= top s
    q = (v / s).round() if fmt == "mxint8" else (v / s).float().to(torch.float8_e4m3fn).to(F64)
    return (q * s).flatten(1)


def _exact_weight(w, fmt, rows, cols):
    dev = w["codes"].device
    k = torch.arange(cols, device=dev)
    r = torch.arange(rows, device=dev)[:, None]
    s, q, i, gk, n = k // 128, k // 512, (k // 128) % 4, (k // 32) % 4, r % 16
    S, Q = cols // 128, cols // 512
    lane = 16 * gk + n
    byte = w["codes"][((r // 16) * S + s) * 1024 + 16 * lane + (k % 32) // 2]
    code = (byte >> (4 * (k % 2)).to(torch.uint8)) & 15
    if fmt == "int4":
        v = torch.tensor([float(j if j < 8 else j - 16) for j in range(16)], dtype=F64, device=dev)[code.int()]
        return v * w["scales"].view(torch.float16)[(((r // 16) * Q + q) * 16 + n) * 4 + i].to(F64)
    v = torch.tensor([(-1.0) ** (j // 8) * E2M1[j % 8] for j in range(16)], dtype=F64, device=dev)[code.int()]
    if fmt == "mxfp4":
        powers = torch.tensor([2.0 ** (j - 127) for j in range(255)], dtype=F64, device=dev)
        return v * powers[w["scales"][(((r // 16) * Q + q) * 64 + lane) * 4 + i].int()]
    b = w["scales"][(((r // 16) * Q + q) * 64 + lane) * 8 + 2 * i + (k // 16) % 2]
    return v * b.view(torch.float8_e4m3fn).to(F64) * w["gs"].to(F64)


def exact(case, seed):
    st, c = prepare(case, seed), case
    op = c["op"]
    if op == "dispatch":
        offsets, gather, inv = _sort(st["ids"], c["E"])
        xs = torch.zeros(st["xs"].shape, dtype=F64, device="cuda")
        n = int(offsets[-1])
        xs[:n] = st["x"][gather[:n].long()].to(F64)
        return None, None, None, xs
    if op == "combine_grad":
        keep = st["inv"] >= 0
        t, j = keep.nonzero(as_tuple=True)
        p = st["inv"][t, j].long()
        dout, y = st["dout"].to(F64), st["y"].to(F64)
        dy, dw = torch.zeros_like(y), torch.zeros(keep.shape, dtype=F64, device="cuda")
        dy[p] = st["weights"][t, j].to(F64)[:, None] * dout[t]
        dw[t, j] = torch.linalg.vecdot(dout[t], y[p])
        lg = st["logits"].to(F64).requires_grad_()
        grad, = torch.autograd.grad((torch.softmax(lg, 1)[t, st["ids"][t, j].long()] * dw[t, j]).sum(), lg)
        dx = torch.zeros_like(dout).index_add_(0, t, st["dxs"].to(F64)[p])
        return dy, dw, grad, dx
    if op == "swiglu":
        g, u = st["gu"].to(F64).chunk(2, 1)
        h = g * torch.sigmoid(g) * u
        g, u = (v.clone().requires_grad_() for v in _exact_kept8(st["gu"], c["fmt"]).chunk(2, 1))
        grads = torch.autograd.grad(g * torch.sigmoid(g) * u, (g, u), st["dh"].to(F64))
        return h, torch.cat(grads, 1)
    N, K, E = c["N"], c["K"], c["E"]
    ends = st["offsets"].tolist() if E else [0, c["T"]]
    pairs = list(zip(ends[:-1], ends[1:]))
    if op == "wgrad":
        x = _exact_kept8(st["x"], c["fmt"])
        dw = torch.empty(len(pairs) * N, K, dtype=F64, device="cuda")
        for e, (a, b) in enumerate(pairs):
            rows = x[st["gather"][a:b].long()] if E else x
            dw[e * N:(e + 1) * N] = st["dc"][a:b].to(F64).t() @ rows
        return dw
    da = torch.empty(st["dc"].shape[0], K, dtype=F64, device="cuda")
    cb, sb = st["w"]["codes"].numel() // len(pairs), st["w"]["scales"].numel() // len(pairs)
    for e, (a, b) in enumerate(pairs):
        w = {"codes": st["w"]["codes"][e * cb:(e + 1) * cb], "scales": st["w"]["scales"][e * sb:(e + 1) * sb], "gs": st["w"]["gs"]}
        da[a:b] = st["dc"][a:b].to(F64) @ _exact_weight(w, c["fmt"], N, K)
    return da
