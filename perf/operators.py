"""The operators of a mixture-of-experts feed-forward layer around the grouped FP8 GEMMs, as cases to be measured.

Four operators, each with its backward pass where training needs one:

  route      experts of each token from the router's logits, and the gradient of the logits
  dispatch   tokens quantized 1x128 into the rows that the grouped GEMMs read (contiguous: training and prefill,
             masked: decode), the weighted sum that brings the rows back, and that sum's backward pass
  swiglu     the gate between an expert's two products, quantized for the second one, with the 8-bit checkpoint that its
             backward pass starts from
  wgrad      the experts' weight gradients from operands held in 8 bits

`run` computes them in plain torch operations, or through the library where `own` is true.  FP8 outputs are returned as
float8 tensors (views of the codes) beside their FP32 scales.
"""
import math
import random

import numpy as np
import torch

own = False
DEV = "cuda"
F8 = torch.float8_e4m3fn
SOFTMAX, SIGMOID = 0, 1


# ----------------------------------------------------------------------------------------------------------------------
# cases

def listed():
    return [
        # one decode step of 64 sequences through a 256-expert router: launch latency
        dict(name="route_decode", op="route", T=64, E=256, topk=8, groups=8, topk_groups=4, group_top=2, score=SIGMOID,
             bias=True, renorm=True, scale=2.5, bf16=False, pad=0),
        # a training micro-batch through the same router, its last tokens padding
        dict(name="route_train", op="route", T=8192, E=256, topk=8, groups=8, topk_groups=4, group_top=2, score=SIGMOID,
             bias=True, renorm=True, scale=2.5, bf16=False, pad=100),
        # the router's backward pass, softmax scores without renormalisation (every logit has a gradient), BF16 logits
        dict(name="route_bwd_softmax", op="route_bwd", T=8192, E=64, topk=6, groups=1, topk_groups=1, group_top=1,
             score=SOFTMAX, bias=False, renorm=False, scale=1.0, bf16=True, pad=0),
        # one GPU's 32 experts, 8192 tokens x top-8 with Zipf-skewed experts, BF16 activations: the contiguous layout
        dict(name="dispatch_train", op="dispatch", T=8192, H=7168, E=32, topk=8, first=0, G=32, zipf=1.1, bf16=True),
        # decode: 128 tokens of all GPUs, of which 32 of the 256 experts are here, into 128-row buffers
        dict(name="dispatch_decode", op="dispatch_masked", T=128, H=7168, E=256, topk=8, first=64, G=32, zipf=0.3, M_max=128,
             bf16=True),
        # the experts' outputs of the training batch back to their tokens
        dict(name="combine_train", op="combine", T=8192, H=7168, E=32, topk=8, first=0, G=32, zipf=1.1, bf16=True),
        # its backward pass at an odd number of tokens
        dict(name="combine_bwd", op="combine_bwd", T=3001, H=7168, E=32, topk=8, first=0, G=32, zipf=1.1, bf16=True),
        # the gate of the training batch's 67,456 expert rows, with the checkpoint
        dict(name="swiglu_train", op="swiglu", R=67456, used=66900, inner=2048, bf16=True, ckpt=True),
        # the gate in decode, on the masked layout
        dict(name="swiglu_decode", op="swiglu_masked", G=32, M_max=128, hi=64, inner=2048, bf16=True),
        # the gate's backward pass from the checkpoint
        dict(name="swiglu_bwd_train", op="swiglu_bwd", R=67456, used=67456, inner=2048, bf16=True),
        # a few small experts' weight gradients, one of them without rows
        dict(name="wgrad_small", op="wgrad", G=5, rows=1111, M=512, N=768, zipf=0.7),
        # the down projections' weight gradients of the training batch
        dict(name="wgrad_train", op="wgrad", G=32, rows=65536, M=7168, N=2048, zipf=1.1),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(round(v / step)) * step)


def draw(rng):
    """One more case: an operator, and sizes spread over its range."""
    op = rng.choice(("route", "route_bwd", "dispatch", "dispatch_masked", "combine", "combine_bwd", "swiglu",
                     "swiglu_masked", "swiglu_bwd", "wgrad"))
    bf16 = rng.random() < 0.7
    if op in ("route", "route_bwd"):
        groups = rng.choice((1, 1, 2, 4, 8))
        per = _log(rng, 8, 384 // groups)
        E = groups * per
        topk_groups = rng.randint(1, groups)
        renorm = rng.random() < 0.6
        topk = rng.randint(2 if renorm else 1, min(8, topk_groups * per))     # one renormalised weight has no gradient
        T = _log(rng, 1, 16384)
        return dict(op=op, T=T, E=E, topk=topk, groups=groups, topk_groups=topk_groups, group_top=rng.choice((1, 2)),
                    score=rng.choice((SOFTMAX, SIGMOID)), bias=rng.random() < 0.5, renorm=renorm,
                    scale=rng.choice((1.0, 2.5)), bf16=bf16, pad=rng.choice((0, T // 10)))
    if op in ("dispatch", "dispatch_masked", "combine", "combine_bwd"):
        H = _log(rng, 256, 7168, 16)
        E = rng.choice((8, 16, 32, 60, 128, 256))
        G = rng.choice((E, E, max(1, E // 4)))
        topk = rng.randint(1, min(8, E))
        T = _log(rng, 1, 128 if op == "dispatch_masked" else 6000)
        first = rng.choice((0, E - G))
        c = dict(op=op, T=T, H=H, E=E, topk=topk, first=first, G=G, zipf=rng.choice((0.0, 0.5, 1.1)), bf16=bf16)
        if op == "dispatch_masked":
            c["M_max"] = 128
        return c
    if op == "swiglu_masked":
        return dict(op=op, G=rng.choice((4, 8, 32)), M_max=128, hi=rng.randint(1, 128), inner=_log(rng, 256, 2048, 128), bf16=bf16)
    if op in ("swiglu", "swiglu_bwd"):
        R = _log(rng, 128, 40000, 128)
        c = dict(op=op, R=R, used=max(1, R - rng.choice((0, 0, 5, 128))), inner=_log(rng, 256, 2048, 128), bf16=bf16)
        if op == "swiglu":
            c["ckpt"] = rng.random() < 0.7
        else:
            c["used"] = max(128, c["used"] // 128 * 128)
        return c
    return dict(op="wgrad", G=rng.choice((1, 3, 8, 16)), rows=_log(rng, 64, 16384), M=_log(rng, 128, 4096, 16),
                N=_log(rng, 256, 4096, 256) if rng.random() < 0.7 else _log(rng, 64, 2048, 16), zipf=rng.choice((0.0, 1.1)))


# ----------------------------------------------------------------------------------------------------------------------
# inputs

def _up(n, m=128):
    return (n + m - 1) // m * m


def _rows_bound(T, topk, G):
    """Rows that hold any routing of T tokens, every expert's padded to whole 128-row tiles."""
    n = T * topk
    return (n + 127 * min(G, n)) // 128 * 128


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 13)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _type(case):
    return torch.bfloat16 if case["bf16"] else torch.float32


def _outliers(g, x, frac=0.001, times=100.0):
    """The same few channels large in every row, as in the activations of a language model."""
    n = max(1, round(frac * x.shape[-1]))
    at = torch.randperm(x.shape[-1], generator=g, device=DEV)[:n]
    x[..., at] *= times
    return x


def _choices(x, bias, case):
    """The chosen experts (float64, -1 where none is left), and whether the choice hangs on the last bits of a score."""
    T, E = x.shape
    per = E // case["groups"]
    x = x.double()
    dead = torch.isinf(x)
    if case["score"] == SIGMOID:
        s = torch.sigmoid(x)
    else:
        s = torch.nan_to_num(torch.softmax(x, -1))
    c = s + (bias.double() if bias is not None else 0.0)
    c = torch.where(dead, -math.inf, c)
    best = c.view(T, case["groups"], per).sort(-1, descending=True).values[..., : case["group_top"]]
    gs = torch.where(torch.isinf(best), 0.0, best).sum(-1)
    gs = torch.where(torch.isinf(best[..., 0]), -math.inf, gs)
    gv, gi = gs.sort(dim=-1, descending=True, stable=True)
    k = case["topk_groups"]
    close = torch.zeros(T, dtype=torch.bool, device=x.device)
    if k < case["groups"]:
        gap = (gv[:, k - 1] - gv[:, k]) / gv[:, k - 1].abs()
        close |= (gap < 1e-5) & torch.isfinite(gv[:, k])
        keep = torch.zeros_like(gs, dtype=torch.bool).scatter_(1, gi[:, :k], True)
        c = torch.where(keep.repeat_interleave(per, 1), c, -math.inf)
    cv, ci = c.sort(dim=-1, descending=True, stable=True)
    n = min(case["topk"] + 1, E)
    gap = (cv[:, : n - 1] - cv[:, 1:n]) / cv[:, : n - 1].abs()
    same = (x.gather(1, ci[:, : n - 1]) == x.gather(1, ci[:, 1:n])) & (bias is None)   # equal inputs: an exact tie
    close |= ((gap < 1e-5) & torch.isfinite(cv[:, 1:n]) & ~same).any(-1)
    k = case["topk"]
    idx = torch.where(torch.isinf(cv[:, :k]), -1, ci[:, :k])
    return idx.to(torch.int32), close


def _router_inputs(case, g):
    T, E = case["T"], case["E"]
    bias = _randn(g, E) * 0.05 if case["bias"] else None
    liked = _randn(g, E) * 0.3

    def logits():
        x = (_randn(g, T, E) + liked).to(_type(case))
        if case["pad"]:
            x[T - case["pad"]:] = -math.inf
        return x

    x = logits()
    for _ in range(4):          # a token whose choice hangs on rounding is drawn again, so that every right answer is one
        again = _choices(x, bias, case)[1]
        x = torch.where(again[:, None], logits(), x)
    return x, bias


def _expert_ids(case, g):
    """Distinct experts of each token, some experts more popular than others."""
    E = case["E"]
    rank = torch.randperm(E, generator=g, device=DEV).float() + 1
    noise = -torch.log(-torch.log(torch.rand(case["T"], E, generator=g, device=DEV).clamp(1e-7, 1 - 1e-6)))
    return (noise - case["zipf"] * torch.log(rank)).topk(case["topk"], dim=1).indices.to(torch.int32)


def _zipf_offsets(case, seed):
    r = np.random.default_rng(seed)
    p = (r.permutation(case["G"]) + 1.0) ** -case["zipf"]
    n = r.multinomial(case["rows"], p / p.sum())
    if case["G"] >= 4:
        n[int(r.integers(case["G"]))] = 0          # an expert that no token chose
    return [0] + [int(v) for v in np.cumsum((n + 127) // 128 * 128)], [int(v) for v in n]


def _quant_rows(x):
    """1x128 quantization along the last axis: codes (float8 [R][K]) and scales [K/128][R]."""
    R, K = x.shape
    x = x.float()
    if K % 128:
        x = torch.nn.functional.pad(x, (0, _up(K) - K))
    x = x.view(R, -1, 128)
    s = x.abs().amax(-1, keepdim=True) / 448.0
    q = torch.where(s == 0, x, x / s).to(F8)
    return q.view(R, -1)[:, :K].contiguous(), s[..., 0].t().contiguous()


def _values(q, s):
    """The FP32 values of 1x128 codes [R][K] with scales [K/128][R]."""
    K = q.shape[1]
    return q.to(torch.float32) * s.t().repeat_interleave(128, 1)[:, :K]


def _zeros(shape, dtype):
    return torch.zeros(shape, dtype=dtype, device=DEV)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"case": dict(case)}
    if op in ("route", "route_bwd"):
        st["x"], st["bias"] = _router_inputs(case, g)
        if op == "route_bwd":
            st["idx"] = _choices(st["x"], st["bias"], case)[0]
            st["dw"] = _randn(g, case["T"], case["topk"])
        return st
    if op in ("dispatch", "dispatch_masked", "combine", "combine_bwd"):
        T, H, G = case["T"], case["H"], case["G"]
        st["idx"] = _expert_ids(case, g)
        R = G * case["M_max"] if op == "dispatch_masked" else _rows_bound(T, case["topk"], G)
        st["R"] = R
        if op in ("dispatch", "dispatch_masked"):
            st["x"] = _outliers(g, _randn(g, T, H, dtype=_type(case)))
        else:
            w = torch.rand(T, case["topk"], generator=g, device=DEV) + 0.05
            st["w"] = w / w.sum(1, keepdim=True)
            st["y"] = _randn(g, R, H, dtype=_type(case))
            st["row_of"], st["offsets"], st["counts"] = _plain_rows(st["idx"], case["first"], G)
        if op == "combine_bwd":
            st["dout"] = _randn(g, T, H, dtype=_type(case)) * 1e-3
        if op != "combine":         # rows that no expert owns are not written: the buffers a training loop keeps
            shape = (G, case["M_max"]) if op == "dispatch_masked" else (R,)
            lead = (G,) if op == "dispatch_masked" else ()
            st["q"] = _zeros(shape + (H,), torch.uint8)
            st["s"] = _zeros(lead + (_up(H) // 128, shape[-1]), torch.float32)
        return st
    if op in ("swiglu", "swiglu_masked"):
        lead = (case["G"], case["M_max"]) if op == "swiglu_masked" else (case["R"],)
        I = case["inner"]
        st["gu"] = _randn(g, *lead, 2 * I, dtype=_type(case)) * 2
        if op == "swiglu_masked":
            st["rows"] = torch.randint(0, case["hi"] + 1, (case["G"],), generator=g, device=DEV, dtype=torch.int32)
        else:
            st["rows"] = torch.tensor([case["used"]], dtype=torch.int32, device=DEV)
        st["q"] = _zeros(lead + (I,), torch.uint8)
        st["s"] = _zeros(lead[:-1] + (_up(I) // 128, lead[-1]), torch.float32)
        if case.get("ckpt"):
            st["qc"] = _zeros(lead + (2 * I,), torch.uint8)
            st["sc"] = _zeros(lead[:-1] + (2 * (_up(I) // 128), lead[-1]), torch.float32)
        return st
    if op == "swiglu_bwd":
        R, I = case["R"], case["inner"]
        halves = [_quant_rows(_randn(g, R, I) * 2) for _ in range(2)]
        st["qc"] = torch.cat([h[0].view(torch.uint8) for h in halves], 1).contiguous()
        st["sc"] = torch.cat([h[1] for h in halves], 0).contiguous()
        st["dh"] = _randn(g, R, I, dtype=_type(case)) * 1e-3
        st["rows"] = torch.tensor([case["used"]], dtype=torch.int32, device=DEV)
        st["out"] = (_zeros((R, 2 * I), torch.uint8), _zeros((2 * (_up(I) // 128), R), torch.float32),
                     _zeros((2 * I, R), torch.uint8), _zeros((R // 128, 2 * I), torch.float32),
                     _zeros((I, R), torch.uint8), _zeros((R // 128, I), torch.float32))
        return st
    off, counts = _zipf_offsets(case, seed)
    R = max(off[-1], 128)

    def operand(n, sigma):
        x = _randn(g, n, R) * sigma
        pos = torch.arange(R, device=DEV)
        start = torch.tensor(off, device=DEV)
        at = torch.searchsorted(start[1:].contiguous(), pos, right=True).clamp(max=case["G"] - 1)
        fill = torch.tensor(counts, device=DEV)[at]
        x *= (pos - start[at] < fill)                       # padding rows are zero
        q, s = _quant_rows(x)
        return q.view(torch.uint8), s

    st["a"], st["sa"] = operand(case["M"], 1e-3)
    st["b"], st["sb"] = operand(case["N"], 1.0)
    st["off"] = off
    st["offsets"] = torch.tensor(off, dtype=torch.int32, device=DEV)
    return st


# ----------------------------------------------------------------------------------------------------------------------
# the plain forms

def _plain_route(x, bias, c):
    T, E = x.shape
    groups, per, k = c["groups"], E // c["groups"], c["topk"]
    x = x.float()
    dead = torch.isinf(x)
    if c["score"] == SIGMOID:
        s = 1.0 / (1.0 + torch.exp(-x))
    else:
        m = x.amax(1, keepdim=True)
        e = torch.exp(x - torch.where(torch.isinf(m), 0.0, m))
        s = e / e.sum(1, keepdim=True).clamp(min=1e-30)
    choice = s + bias if bias is not None else s
    choice = torch.where(dead, -math.inf, choice)
    if c["topk_groups"] < groups:
        best = choice.view(T, groups, per).sort(2, descending=True).values[..., : c["group_top"]]
        gs = torch.where(torch.isinf(best), 0.0, best).sum(2)
        gs = torch.where(torch.isinf(best[..., 0]), -math.inf, gs)
        gi = gs.sort(dim=1, descending=True, stable=True).indices[:, : c["topk_groups"]]
        keep = torch.zeros_like(gs, dtype=torch.bool).scatter_(1, gi, True)
        choice = torch.where(keep[..., None].expand(T, groups, per).reshape(T, E), choice, -math.inf)
    v, i = choice.sort(dim=1, descending=True, stable=True)
    none = torch.isinf(v[:, :k])
    w = torch.where(none, 0.0, s.gather(1, i[:, :k]))
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total == 0, 0.0, w / total)
    return torch.where(none, -1, i[:, :k]).to(torch.int32), w * c["scale"]


def _plain_route_bwd(x, idx, dw, c):
    dtype = x.dtype
    x = x.float()
    if c["score"] == SIGMOID:
        s = 1.0 / (1.0 + torch.exp(-x))
    else:
        m = x.amax(1, keepdim=True)
        e = torch.exp(x - torch.where(torch.isinf(m), 0.0, m))
        s = e / e.sum(1, keepdim=True).clamp(min=1e-30)
    none = idx < 0
    at = idx.clamp(min=0).long()
    si = torch.where(none, 0.0, s.gather(1, at))
    g = torch.where(none, 0.0, dw) * c["scale"]
    if c["renorm"]:
        v = si.sum(1, keepdim=True).clamp(min=1e-30)
        g = (g - (g * si).sum(1, keepdim=True) / v) / v
        g = torch.where(none, 0.0, g)
    ds = torch.zeros_like(s).scatter_add_(1, at, g)
    if c["score"] == SIGMOID:
        return (ds * s * (1.0 - s)).to(dtype)
    return (s * (ds - (g * si).sum(1, keepdim=True))).to(dtype)


def _plain_rows(idx, first, G):
    """Contiguous layout: each (token, choice)'s row (-1: not an expert of this range), offsets and counts."""
    e = idx.reshape(-1).long() - first
    here = (e >= 0) & (e < G)
    e = torch.where(here, e, G)
    seen = torch.zeros(e.numel(), G + 1, dtype=torch.int32, device=idx.device).scatter_(1, e[:, None], 1).cumsum(0)
    rank = seen.gather(1, e[:, None])[:, 0] - 1
    counts = seen[-1, :G]
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=idx.device), ((counts + 127) // 128 * 128).cumsum(0)])
    row = torch.where(here, offsets[e.clamp(max=G)] + rank, -1)
    return row.view(idx.shape).to(torch.int32), offsets.to(torch.int32), counts.to(torch.int32)


def _spread(q, s, row_of, R, w=None):
    """Token rows q [T][H], s [H/128][T] copied to the rows of `row_of`; the others zero."""
    T, k = row_of.shape
    row = row_of.reshape(-1).long()
    row = torch.where(row < 0, R, row)
    src = torch.arange(T, device=q.device).repeat_interleave(k)
    codes = q.view(torch.uint8)[src]
    scale = s[:, src]
    if w is not None:
        scale = scale * w.reshape(-1).abs()
        codes = torch.where(w.reshape(-1, 1) < 0, codes ^ 128, codes)
    qo = torch.zeros(R + 1, q.shape[1], dtype=torch.uint8, device=q.device)
    so = torch.zeros(s.shape[0], R + 1, device=q.device)
    qo[row] = codes
    so[:, row] = scale
    return qo[:R].view(F8), so[:, :R]


def _gate(gu, inner):
    g, u = gu[..., :inner].float(), gu[..., inner:].float()
    return g / (1.0 + torch.exp(-g)) * u


def _plain(st):
    c, op = st["case"], st["case"]["op"]
    if op == "route":
        return _plain_route(st["x"], st["bias"], c)
    if op == "route_bwd":
        return _plain_route_bwd(st["x"], st["idx"], st["dw"], c)
    if op == "dispatch":
        row_of, offsets, counts = _plain_rows(st["idx"], c["first"], c["G"])
        q, s = _spread(*_quant_rows(st["x"]), row_of, st["R"])
        return q, s, row_of, offsets, counts
    if op == "dispatch_masked":
        row_of, offsets, counts = _plain_rows(st["idx"], c["first"], c["G"])
        e = (st["idx"].long() - c["first"]).clamp(0, c["G"] - 1)
        rank = row_of - offsets[e]
        row_of = torch.where((row_of < 0) | (rank >= c["M_max"]), -1, e * c["M_max"] + rank).to(torch.int32)
        q, s = _spread(*_quant_rows(st["x"]), row_of, st["R"])
        return (q.view(c["G"], c["M_max"], -1), s.view(-1, c["G"], c["M_max"]).transpose(0, 1).contiguous(), row_of,
                counts.clamp(max=c["M_max"]))
    if op == "combine":
        w = torch.where(st["row_of"] < 0, 0.0, st["w"])
        rows = st["y"][st["row_of"].clamp(min=0).long()].float()
        return (rows * w[..., None]).sum(1).to(st["y"].dtype)
    if op == "combine_bwd":
        here = st["row_of"] >= 0
        rows = st["y"][st["row_of"].clamp(min=0).long()].float()
        dw = torch.where(here, (rows * st["dout"].float()[:, None]).sum(2), 0.0)
        return (*_spread(*_quant_rows(st["dout"]), st["row_of"], st["R"], st["w"]), dw)
    if op in ("swiglu", "swiglu_masked"):
        gu, I = st["gu"], c["inner"]
        lead = gu.shape[:-1]
        at = torch.arange(lead[-1], device=gu.device)
        live = at < (st["rows"][:, None] if op == "swiglu_masked" else st["rows"])
        h = torch.where(live[..., None], _gate(gu, I), 0.0)
        q, s = _quant_rows(h.view(-1, I))
        out = [q.view(*lead, I), s if op == "swiglu" else s.view(-1, *lead).transpose(0, 1).contiguous()]
        if c.get("ckpt"):
            x = torch.where(live[..., None], gu, 0.0)
            g, u = _quant_rows(x[:, :I]), _quant_rows(x[:, I:])
            out += [torch.cat([g[0].view(torch.uint8), u[0].view(torch.uint8)], 1).view(F8), torch.cat([g[1], u[1]], 0)]
        return out
    if op == "swiglu_bwd":
        I, nb = c["inner"], st["sc"].shape[0] // 2
        live = (torch.arange(c["R"], device=st["dh"].device) < st["rows"])[:, None]
        qc = st["qc"].view(F8)
        g, u = _values(qc[:, :I], st["sc"][:nb]), _values(qc[:, I:], st["sc"][nb:])
        dh = st["dh"].float()
        sig = 1.0 / (1.0 + torch.exp(-g))
        dg = torch.where(live, dh * u * (sig * (1.0 + g * (1.0 - sig))), 0.0)
        du = torch.where(live, dh * (g * sig), 0.0)
        h = torch.where(live, g * sig * u, 0.0)
        qg, sg = _quant_rows(dg)
        qu, su = _quant_rows(du)
        qgt, sgt = _quant_rows(dg.t())
        qut, sut = _quant_rows(du.t())
        qht, sht = _quant_rows(h.t())
        cat = lambda p, q, d: torch.cat([p.view(torch.uint8), q.view(torch.uint8)], d).view(F8)  # noqa: E731
        return cat(qg, qu, 1), torch.cat([sg, su], 0), cat(qgt, qut, 0), torch.cat([sgt, sut], 1), qht, sht
    a, b = _values(st["a"].view(F8), st["sa"]), _values(st["b"].view(F8), st["sb"])
    out = torch.empty(c["G"], c["M"], c["N"], device=a.device)
    for e in range(c["G"]):
        torch.matmul(a[:, st["off"][e]: st["off"][e + 1]], b[:, st["off"][e]: st["off"][e + 1]].t(), out=out[e])
    return out


# ----------------------------------------------------------------------------------------------------------------------
# the library's calls

def _library(st):
    import fp8_fine_grained_amd as fp8
    c, op = st["case"], st["case"]["op"]
    if op == "route":
        return fp8.moe_route(st["x"], c["topk"], st["bias"], c["groups"], c["topk_groups"], c["group_top"], c["score"],
                             c["renorm"], c["scale"])
    if op == "route_bwd":
        return fp8.moe_route_backward(st["x"], st["idx"], st["dw"], c["score"], c["renorm"], c["scale"])
    if op == "dispatch":
        q, s, row_of, offsets, counts = fp8.fp8_moe_dispatch_contiguous(st["x"], st["idx"], c["G"], c["first"], q=st["q"],
                                                                        s=st["s"])
        return q.view(F8), s, row_of, offsets, counts
    if op == "dispatch_masked":
        q, s, row_of, masked_m = fp8.fp8_moe_dispatch_masked(st["x"], st["idx"], c["G"], c["M_max"], c["first"], q=st["q"],
                                                             s=st["s"])
        return q.view(F8), s, row_of, masked_m
    if op == "combine":
        return fp8.moe_combine(st["y"], st["row_of"], st["w"], out_dtype=st["y"].dtype)
    if op == "combine_bwd":
        q, s, dw = fp8.fp8_moe_combine_backward(st["dout"], st["y"], st["row_of"], st["w"], st["offsets"], st["counts"],
                                                q=st["q"], s=st["s"])
        return q.view(F8), s, dw
    if op in ("swiglu", "swiglu_masked"):
        if c.get("ckpt"):
            q, s, qc, sc = fp8.fp8_swiglu(st["gu"], st["rows"], checkpoint=True, q=st["q"], s=st["s"], qc=st["qc"],
                                          sc=st["sc"])
            return q.view(F8), s, qc.view(F8), sc
        q, s = fp8.fp8_swiglu(st["gu"], st["rows"], q=st["q"], s=st["s"])
        return q.view(F8), s
    if op == "swiglu_bwd":
        q, s, qt, tt, qh, sh = fp8.fp8_swiglu_backward(st["qc"], st["sc"], st["dh"], st["rows"], out=st["out"])
        return q.view(F8), s, qt.view(F8), tt, qh.view(F8), sh
    return fp8.fp8_grouped_gemm_wgrad(st["a"], st["sa"], st["b"], st["sb"], st["offsets"])


def run(state):
    return _library(state) if own else _plain(state)


# ----------------------------------------------------------------------------------------------------------------------
# the work that cannot be done without

def work(case):
    op, el = case["op"], 2 if case.get("bf16") else 4
    if op == "route":
        return {"bytes": case["T"] * (case["E"] * el + 8 * case["topk"]), "flops": case["T"] * case["E"] * 4}
    if op == "route_bwd":
        return {"bytes": case["T"] * (2 * case["E"] * el + 8 * case["topk"]), "flops": case["T"] * case["E"] * 4}
    if op in ("dispatch", "dispatch_masked", "combine", "combine_bwd"):
        T, H = case["T"], case["H"]
        n = T * case["topk"] * case["G"] / case["E"]          # rows of this range's experts
        fp8_rows = n * (H + 4 * (_up(H) // 128) + 4)
        if op == "combine":
            return {"bytes": n * (H * el + 8) + T * H * el, "flops": 2 * n * H}
        if op == "combine_bwd":
            return {"bytes": T * H * el + n * (H * el + 12) + fp8_rows, "flops": 2 * n * H + 2 * T * H}
        return {"bytes": T * H * el + fp8_rows, "flops": 2 * T * H}
    if op in ("swiglu", "swiglu_masked"):
        I = case["inner"]
        n = case["G"] * case["hi"] / 2 if op == "swiglu_masked" else case["used"]
        return {"bytes": n * I * (2 * el + 1 + 4 / 128 + (2 + 8 / 128 if case.get("ckpt") else 0)), "flops": 6 * n * I}
    if op == "swiglu_bwd":
        return {"bytes": case["used"] * case["inner"] * (el + 2 + 5 + 4 * 7 / 128), "flops": 16 * case["used"] * case["inner"]}
    r, M, N = case["rows"], case["M"], case["N"]
    return {"bytes": r * (M + N) * (1 + 4 / 128) + 4 * case["G"] * M * N, "flops": 2 * r * M * N}


# ----------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits

def _exact_quant(x):
    """Values of the codes [.., K] and scales [.., K/128] of float64 rows, from the definition of the 1x128 groups."""
    K = x.shape[-1]
    nb = (K + 127) // 128
    codes, scales = torch.empty_like(x), x.new_empty(*x.shape[:-1], nb)
    for b in range(nb):
        part = x[..., 128 * b: 128 * b + 128]
        s = part.abs().max(-1, keepdim=True)[0] / 448.0
        v = part / torch.where(s > 0, s, 1.0)
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)      # E4M3: three mantissa bits
        codes[..., 128 * b: 128 * b + 128] = (torch.round(v / step) * step).clamp(-448, 448)
        scales[..., b] = s[..., 0]
    return codes, scales


def _exact_scores(x, score):
    x = x.double()
    if score == SIGMOID:
        return torch.sigmoid(x)
    return torch.exp(x - torch.logsumexp(x.nan_to_num(neginf=-1e300), 1, keepdim=True))


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("route", "route_bwd"):
        idx = st["idx"] if op == "route_bwd" else _choices(st["x"], st["bias"], case)[0]
        s = _exact_scores(st["x"], case["score"])
        chosen = torch.zeros_like(s)
        for j in range(case["topk"]):
            col = idx[:, j].long()
            r = torch.nonzero(col >= 0)[:, 0]
            chosen[r, col[r]] = 1.0
        total = (s * chosen).sum(1, keepdim=True)
        total = torch.where(total > 0, total, 1.0)
        if op == "route":
            w = s * chosen / total if case["renorm"] else s * chosen
            w = torch.where(idx >= 0, torch.gather(w, 1, idx.clamp(min=0).long()), 0.0) * case["scale"]
            return None, w
        grad = torch.zeros_like(s)
        for j in range(case["topk"]):
            col = idx[:, j].long()
            r = torch.nonzero(col >= 0)[:, 0]
            grad[r, col[r]] += st["dw"][r, j].double() * case["scale"]
        if case["renorm"]:
            w = s * chosen / total
            grad = chosen * (grad - (grad * w).sum(1, keepdim=True)) / total
        if case["score"] == SIGMOID:
            return grad * s * (1 - s)
        return s * grad - s * (s * grad).sum(1, keepdim=True)
    if op in ("dispatch", "dispatch_masked", "combine_bwd"):
        T, R, G = case["T"], st["R"], case["G"]
        codes, scales = _exact_quant((st["dout"] if op == "combine_bwd" else st["x"]).double())
        q = torch.zeros(R, case["H"], dtype=torch.float64, device=DEV)
        s = torch.zeros(R, scales.shape[1], dtype=torch.float64, device=DEV)
        if op == "dispatch_masked":
            for e in range(G):
                t = torch.nonzero((st["idx"] == case["first"] + e).any(1))[: case["M_max"], 0]
                q[e * case["M_max"] + torch.arange(len(t), device=DEV)] = codes[t]
                s[e * case["M_max"] + torch.arange(len(t), device=DEV)] = scales[t]
            return q.view(G, case["M_max"], -1), s.view(G, case["M_max"], -1).transpose(1, 2).contiguous(), None, None
        at = 0
        for e in range(G):                       # an expert's rows: its tokens in their order
            t, j = torch.nonzero(st["idx"] == case["first"] + e, as_tuple=True)
            q[at: at + len(t)] = codes[t]
            s[at: at + len(t)] = scales[t]
            if op == "combine_bwd":
                s[at: at + len(t)] *= st["w"][t, j].double()[:, None]
            at += (len(t) + 127) // 128 * 128
        if op == "dispatch":
            return q, s.t().contiguous(), None, None, None
        dw = torch.zeros(T, case["topk"], dtype=torch.float64, device=DEV)
        for j in range(case["topk"]):
            r = torch.nonzero(st["row_of"][:, j] >= 0)[:, 0]
            dw[r, j] = torch.einsum("th,th->t", st["dout"][r].double(), st["y"][st["row_of"][r, j].long()].double())
        return q, s.t().contiguous(), dw
    if op == "combine":
        out = torch.zeros(case["T"], case["H"], dtype=torch.float64, device=DEV)
        for j in range(case["topk"]):
            r = torch.nonzero(st["row_of"][:, j] >= 0)[:, 0]
            out[r] += st["w"][r, j].double()[:, None] * st["y"][st["row_of"][r, j].long()].double()
        return out
    if op in ("swiglu", "swiglu_masked"):
        I = case["inner"]
        gu = st["gu"].double().clone()
        if op == "swiglu":
            gu[case["used"]:] = 0
        else:
            for e, n in enumerate(st["rows"].tolist()):
                gu[e, n:] = 0
        g, u = gu[..., :I], gu[..., I:]
        q, s = _exact_quant(torch.nn.functional.silu(g) * u)
        out = [q, s.transpose(-1, -2).contiguous()]
        if case.get("ckpt"):
            (qg, sg), (qu, su) = _exact_quant(g), _exact_quant(u)
            out += [torch.cat([qg, qu], 1), torch.cat([sg, su], 1).t().contiguous()]
        return out
    if op == "swiglu_bwd":
        I, n = case["inner"], case["used"]
        sc = st["sc"].double().t().repeat_interleave(128, 1)
        half = sc.shape[1] // 2
        v = st["qc"].view(F8).to(torch.float64)
        g, u, dh = v[:, :I] * sc[:, :I], v[:, I:] * sc[:, half: half + I], st["dh"].double()
        dh[n:] = 0
        g[n:] = 0
        u[n:] = 0
        slope = torch.sigmoid(g) * (1 + g * torch.sigmoid(-g))
        dg, du, h = dh * u * slope, dh * torch.nn.functional.silu(g), torch.nn.functional.silu(g) * u
        out = []
        for p in ((dg, du), (dg.t(), du.t())):
            (q0, s0), (q1, s1) = _exact_quant(p[0]), _exact_quant(p[1])
            if not out:
                out += [torch.cat([q0, q1], 1), torch.cat([s0, s1], 1).t().contiguous()]
            else:
                out += [torch.cat([q0, q1], 0), torch.cat([s0, s1], 0).t().contiguous()]
        q, s = _exact_quant(h.t())
        return out + [q, s.t().contiguous()]
    out = torch.zeros(case["G"], case["M"], case["N"], dtype=torch.float64, device=DEV)
    for e in range(case["G"]):
        for lo in range(st["off"][e], st["off"][e + 1], 128):        # one 128-row group at a time
            a = st["a"][:, lo: lo + 128].view(F8).double() * st["sa"][lo // 128].double()[:, None]
            b = st["b"][:, lo: lo + 128].view(F8).double() * st["sb"][lo // 128].double()[:, None]
            out[e] += a @ b.t()
    return out
