"""Cases that measure the 8-bit Linear layers, the query/key norm with the
position rotation, and the append to a paged cache.

`run` computes a case with elementary torch operations in 32 bits (64 for the
quotients that are rounded to whole numbers), or, with `own`, through this
package's entry points.  `exact` computes it in 64 bits from the definition.

The layouts are the package's: X [M, K], W [N, K], shard i of a column layer
the rows [i N/P, (i+1) N/P), of a row layer the columns [i K/P, (i+1) K/P);
of a fused QKV layer shard i's columns hold its q heads, its k heads and its v
heads; of a fused gate+up layer its gate rows, then its up rows.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


def listed():
    return [
        # A decode step's input to a column layer: 16 tokens, hidden 8192; latency.
        dict(name="quantize decode", op="quantize", M=16, K=8192, G=1, dtype="bf16"),
        # The gated unit's output of a 4096-token prompt, a scale for each token and shard.
        dict(name="quantize prefill", op="quantize", M=4096, K=14336, G=8, dtype="bf16"),
        # Column layer of a decode step: the weights' bytes bound it.
        dict(name="column decode", op="column", M=16, K=8192, N=28672, P=8, act=0, bias=False, shards=False, dtype="bf16"),
        # Gate+up layer with bias and gated unit over a 4096-token prompt.
        dict(name="column gate+up", op="column", M=4096, K=4096, N=28672, P=8, act=1, bias=True, shards=False, dtype="bf16"),
        # A short ragged prompt through a layer of odd sizes, fp32 outputs in shard blocks.
        dict(name="column ragged", op="column", M=333, K=2000, N=3336, P=3, act=0, bias=True, shards=True, dtype="f32"),
        # Row layer of a decode step, one scale for each token and shard.
        dict(name="row decode", op="row", M=16, K=28672, N=8192, P=8, G=8, bias=False, dtype="bf16"),
        # Down projection of a 4096-token prompt with its bias.
        dict(name="row prefill", op="row", M=4096, K=14336, N=4096, P=8, G=8, bias=True, dtype="bf16"),
        # Queries and keys of an 8192-token prompt, 64 + 8 heads of 128.
        dict(name="qk prefill", op="qk", T=8192, Hq=64, Hkv=8, D=128, R=128, P=8, pairs=False, norm=True, shards=False, pad=0, dtype="bf16"),
        # Part of each head rotated, neighbouring elements paired, a padded tail; fp32.
        dict(name="qk partial f32", op="qk", T=1013, Hq=12, Hkv=4, D=80, R=64, P=2, pairs=True, norm=True, shards=True, pad=13, dtype="f32"),
        # Gradients of a 4096-token training step, 32 + 8 heads of 128.
        dict(name="qk backward", op="qk_backward", T=4096, Hq=32, Hkv=8, D=128, R=128, P=8, pairs=False, norm=True, shards=False, pad=0, dtype="bf16"),
        # One new token of 64 sequences with long pasts; latency.
        dict(name="append decode", op="append", B=64, longest=1, past=8000, Hq=64, Hkv=8, D=128, R=128, P=8, page=16, pairs=False, norm=True, shards=False, dtype="bf16"),
        # Prompts of different lengths written in one call.
        dict(name="append prefill", op="append", B=12, longest=1500, past=700, Hq=64, Hkv=8, D=128, R=128, P=8, page=64, pairs=False, norm=True, shards=False, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _k(rng, lo, hi):
    """A product's length: a multiple of 128, of 16, or any."""
    k, step = _log(rng, lo, hi), rng.choice((128, 128, 16, 1))
    return max(step, k // step * step)


def draw(rng):
    op = rng.choice(("quantize", "column", "row", "qk", "qk_backward", "append"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    P = rng.choice((1, 2, 3, 4, 8))
    if op == "quantize":
        G = rng.choice((1, P))
        K = _k(rng, 16, 2048) * G
        return dict(op=op, M=_log(rng, 1, 4096), K=K, G=G, dtype=dtype)
    if op == "column":
        act = rng.choice((0, 1))
        K, On = _k(rng, 64, 8192), _log(rng, 8, 1792)
        N = On * P * (2 if act else 1)
        M = max(1, min(_log(rng, 1, 4096), int(4.5e11 / N / K)))
        return dict(op=op, M=M, K=K, N=N, P=P, act=act, bias=rng.random() < 0.5, shards=rng.random() < 0.3, dtype=dtype)
    if op == "row":
        K, N = _k(rng, 32, 3584) * P, _log(rng, 16, 8192)
        M = max(1, min(_log(rng, 1, 4096), int(4.5e11 / N / K)))
        return dict(op=op, M=M, K=K, N=N, P=P, G=rng.choice((1, P)), bias=rng.random() < 0.5, dtype=dtype)
    hkv = rng.choice((1, 1, 2, 4))
    Hkv, Hq = hkv * P, hkv * P * rng.choice((1, 3, 4, 8))
    D = rng.choice((64, 80, 96, 128, 128, 128, 256))
    R = D if rng.random() < 0.7 else D // 2
    heads = dict(Hq=Hq, Hkv=Hkv, D=D, R=R, P=P, pairs=rng.random() < 0.3, norm=rng.random() < 0.7, shards=rng.random() < 0.3, dtype=dtype)
    most = max(2, min(8192, 100_000_000 // (BYTES[dtype] * (Hq + 2 * Hkv) * D)))
    if op == "append":
        B = _log(rng, 1, 256)
        return dict(op=op, B=B, longest=max(1, min(_log(rng, 1, 4096), most // B)), past=_log(rng, 1, 8000), page=rng.choice((16, 32, 64)), **heads)
    T = _log(rng, 1, most)
    return dict(op=op, T=T, pad=rng.choice((0, 0, min(T - 1, 5))), **heads)


# ---- inputs -----------------------------------------------------------------

def _ints(g, shape):
    """What a quantized tensor holds: normal values at about 4 sigma full scale."""
    return torch.randn(shape, generator=g, device=DEV).mul_(32.0).round_().clamp_(-127, 127).to(torch.int8)


def _scales(g, shape, about):
    return torch.rand(shape, generator=g, device=DEV).add_(0.5).mul_(about)


def _tables(n, R):
    """cos and sin of the positions 0 .. n-1, angles in 64 bits."""
    inv = 10000.0 ** (-torch.arange(0, R, 2, device=DEV, dtype=torch.float64) / R)
    a = torch.arange(n, device=DEV, dtype=torch.float64)[:, None] * inv
    return a.cos().float(), a.sin().float()


def _lengths(c):
    """New tokens and past lengths of the sequences: part of the case, so that every seed has the same sizes."""
    r = torch.Generator()
    r.manual_seed(c["B"] * 65536 + c["longest"])
    lens = torch.randint(1, c["longest"] + 1, (c["B"],), generator=r)
    return lens, torch.randint(0, c["past"] + 1, (c["B"],), generator=r)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    t = TYPES[c["dtype"]]
    rn = lambda *shape, s=1.0: torch.randn(shape, generator=g, device=DEV).mul_(s).to(t)  # noqa: E731
    st = dict(case=c)
    if c["op"] == "quantize":
        M, K, G = c["M"], c["K"], c["G"]
        st["X"] = rn(M, K)
        st["Q"] = torch.empty((M, K), dtype=torch.int8, device=DEV)
        st["scale"] = torch.empty((M, G), dtype=torch.float32, device=DEV)
        return st
    if c["op"] in ("column", "row"):
        M, K, N, P = c["M"], c["K"], c["N"], c["P"]
        G = c.get("G", 1)
        st["X"], st["sx"] = _ints(g, (M, K)), _scales(g, (M, G), 1 / 32)
        st["W"], st["sw"] = _ints(g, (N, K)), _scales(g, (N,), 0.02 / 32)
        st["bias"] = rn(N, s=0.1) if c["bias"] else None
        if c["op"] == "row":
            st["Y"] = torch.empty((M, N), dtype=t, device=DEV)
            # room for one 32-bit partial of each shard, as a row layer keeps it
            st["ws"] = torch.empty(4 * P * M * N + 255 & -256, dtype=torch.uint8, device=DEV)
        else:
            On = N // P // (2 if c["act"] else 1)
            st["Y"] = torch.empty((P, M, On) if c["shards"] else (M, P * On), dtype=t, device=DEV)
        return st
    Hq, Hkv, D, R, P = c["Hq"], c["Hkv"], c["D"], c["R"], c["P"]
    if c["op"] == "append":
        lens, past = _lengths(c)
        T = int(lens.sum())
        r = torch.Generator()
        r.manual_seed(seed)
        most = (c["longest"] + c["past"] + c["page"] - 1) // c["page"]
        # only the pages that the call writes to are given places of their own
        first, last = past // c["page"], (past + lens - 1) // c["page"]
        used = (last - first + 1).cumsum(0)
        pages = int(used[-1]) + 3
        order = torch.randperm(pages, generator=r).to(torch.int32)
        at = torch.arange(most)[None, :] - first[:, None]
        mine = (at >= 0) & (at <= (last - first)[:, None])
        st["table"] = torch.where(mine, order[((used - (last - first + 1))[:, None] + at).clamp(0, pages - 1)], 0).to(torch.int32).to(DEV)
        st["cu"] = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)]).to(torch.int32).to(DEV)
        st["past"] = past.to(torch.int32).to(DEV)
        st["kc"], st["vc"] = (rn(pages, c["page"], Hkv, D) for _ in "kv")
        n = c["longest"] + c["past"] + 1
    else:
        T, n = c["T"], 2 * c["T"] + 64
        pos = torch.arange(T, device=DEV) + int(torch.randint(0, T + 1, (1,), generator=g, device=DEV))
        pos[T - c["pad"]:] = -1
        st["pos"] = pos
    per = (Hq + 2 * Hkv) // P * D
    st["qkv"] = rn(P, T, per) if c["shards"] else rn(T, P * per)
    st["cos"], st["sin"] = _tables(n, R)
    st["wq"], st["wk"] = ((1 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(t) if c["norm"] else None for _ in "qk")
    st["Q"] = torch.empty((T, Hq * D), dtype=t, device=DEV)
    st["K"] = torch.empty((T, Hkv * D), dtype=t, device=DEV)
    if c["op"] == "qk_backward":
        st["dQ"], st["dK"], st["dV"] = rn(T, Hq * D), rn(T, Hkv * D), rn(T, Hkv * D)
        st["dqkv"] = torch.empty_like(st["qkv"])
        st["dwq"], st["dwk"] = (torch.empty(D, dtype=torch.float32, device=DEV) if c["norm"] else None for _ in "qk")
        # room for the gradient sums of the weights: 2 D values of 2048 workgroups at most
        st["ws"] = torch.empty(2048 * 2 * D * 4, dtype=torch.uint8, device=DEV)
    return st


# ---- one pass ---------------------------------------------------------------

def run(st):
    c = st["case"]
    return (_own if own else _plain)(st, c, c["op"])


def _own(st, c, op):
    import tensor_linear_amd as tl
    if op == "quantize":
        tl.tp_quantize_rows(st["X"], st["Q"], st["scale"])
        return _stands_for(st["Q"], st["scale"]), st["scale"]
    if op == "column":
        tl.tp_linear_column_quant(st["X"], st["sx"], st["W"], st["sw"], st["Y"], c["P"],
                                  tl.TP_Y_SHARDS if c["shards"] else tl.TP_Y_CONCAT, bias=st["bias"],
                                  act=tl.TP_ACT_SWIGLU if c["act"] else tl.TP_ACT_NONE)
        return st["Y"]
    if op == "row":
        tl.tp_linear_row_quant(st["X"], st["sx"], st["W"], st["sw"], st["Y"], c["P"], tl.TP_ROW_FUSED, st["ws"], bias=st["bias"])
        return st["Y"]
    how = dict(q_weight=st["wq"], k_weight=st["wk"], eps=1e-6, style=tl.TP_ROPE_PAIRS if c["pairs"] else tl.TP_ROPE_HALVES,
               x_mode=tl.TP_Y_SHARDS if c["shards"] else tl.TP_Y_CONCAT)
    if op == "qk":
        tl.tp_qk_norm_rope(st["qkv"], st["pos"], st["cos"], st["sin"], st["Q"], st["K"], c["P"], c["Hq"], c["Hkv"], **how)
        return st["Q"], st["K"]
    if op == "qk_backward":
        tl.tp_qk_norm_rope_backward(st["qkv"], st["pos"], st["cos"], st["sin"], st["dQ"], st["dK"], st["dqkv"], c["P"], c["Hq"], c["Hkv"],
                                    dV=st["dV"], dq_weight=st["dwq"], dk_weight=st["dwk"], workspace=st["ws"], **how)
        return st["dqkv"], st["dwq"], st["dwk"]
    tl.tp_kv_append(st["qkv"], st["cos"], st["sin"], st["past"], st["cu"], st["table"], st["kc"], st["vc"], c["P"], c["Hq"], c["Hkv"], Q=st["Q"], **how)
    return st["Q"], st["kc"], st["vc"]


def _stands_for(q, scale):
    """The values that whole numbers and the scale of each row and group stand for."""
    M, K = q.shape
    G = scale.shape[1]
    return (q.view(M, G, K // G) * scale[:, :, None]).view(M, K)


def _plain(st, c, op):
    t = TYPES[c["dtype"]]
    if op == "quantize":
        M, K, G = c["M"], c["K"], c["G"]
        x = st["X"].float().view(M, G, K // G)
        # the quotients in 64 bits: values next to a border between two whole numbers,
        # and a scale one step away would move them all
        scale = (x.abs().amax(2).double() / 127.0).float()
        q = torch.where(scale[:, :, None] > 0, x.double() / scale.double()[:, :, None], 0.0).round().clamp(-127, 127)
        st["Q"].copy_(q.view(M, K))
        st["scale"].copy_(scale)
        return _stands_for(st["Q"], scale), st["scale"]
    if op == "column":
        M, N, P = c["M"], c["N"], c["P"]
        y = (st["X"].float() @ st["W"].float().t()) * st["sx"] * st["sw"]
        if c["bias"]:
            y = y + st["bias"].float()
        y = y.view(M, P, N // P)
        if c["act"]:
            h = N // P // 2
            y = y[:, :, :h] / (1 + torch.exp(-y[:, :, :h])) * y[:, :, h:]
        st["Y"].copy_(y.transpose(0, 1) if c["shards"] else y.reshape(M, -1))
        return st["Y"]
    if op == "row":
        y = (_stands_for(st["X"], st["sx"]) @ st["W"].float().t()) * st["sw"]
        if c["bias"]:
            y = y + st["bias"].float()
        st["Y"].copy_(y)
        return st["Y"]
    cos, sin, pos, ok = _angles(st, c, torch.float32)
    q, k, v = _heads(st["qkv"], c, torch.float32)
    if op == "qk_backward":
        dq, dwq = _backward(q, st["dQ"], st["wq"], cos, sin, ok, c, torch.float32)
        dk, dwk = _backward(k, st["dK"], st["wk"], cos, sin, ok, c, torch.float32)
        st["dqkv"].copy_(_join(dq, dk, st["dV"].float().view(v.shape), c))
        if c["norm"]:
            st["dwq"].copy_(dwq)
            st["dwk"].copy_(dwk)
        return st["dqkv"], st["dwq"], st["dwk"]
    st["Q"].copy_(_forward(q, st["wq"], cos, sin, ok, c).view(st["Q"].shape))
    k = _forward(k, st["wk"], cos, sin, ok, c)
    if op == "qk":
        st["K"].copy_(k.view(st["K"].shape))
        return st["Q"], st["K"]
    page, slot = _places(st, c, pos)
    st["kc"].index_put_((page, slot), k.to(t))
    st["vc"].index_put_((page, slot), v.to(t))
    return st["Q"], st["kc"], st["vc"]


def _angles(st, c, t):
    """cos and sin of each token's position, the positions, and which are in the table."""
    if c["op"] == "append":
        T = st["Q"].shape[0]
        s = _sequence(st, T)
        pos = (st["past"][s] - st["cu"][s]).long() + torch.arange(T, device=DEV)
    else:
        pos = st["pos"]
    ok = (pos >= 0) & (pos < st["cos"].shape[0])
    at = torch.where(ok, pos, 0)
    return st["cos"].to(t)[at][:, None], st["sin"].to(t)[at][:, None], pos, ok[:, None, None]


def _sequence(st, T):
    return torch.searchsorted(st["cu"][1:].long(), torch.arange(T, device=DEV), right=True)


def _places(st, c, pos):
    s = _sequence(st, pos.shape[0])
    return st["table"][s, pos // c["page"]].long(), pos % c["page"]


def _heads(qkv, c, t):
    """q, k and v as [T, heads, D], the shards' heads one after another."""
    P, D, hq, hk = c["P"], c["D"], c["Hq"] // c["P"], c["Hkv"] // c["P"]
    x = qkv.to(t)
    x = x.transpose(0, 1) if c["shards"] else x
    x = x.reshape(x.shape[0], P, hq + 2 * hk, D)
    return x[:, :, :hq].flatten(1, 2), x[:, :, hq:hq + hk].flatten(1, 2), x[:, :, hq + hk:].flatten(1, 2)


def _join(q, k, v, c):
    T, P, D = q.shape[0], c["P"], c["D"]
    x = torch.cat([a.view(T, P, -1, D) for a in (q, k, v)], 2).flatten(2)
    return x.transpose(0, 1) if c["shards"] else x.flatten(1)


def _turn(x, cos, sin, c):
    """The rotation of each pair by its angle."""
    R = c["R"]
    y, rest = x[..., :R], x[..., R:]
    if c["pairs"]:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = y[..., :R // 2], y[..., R // 2:]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, rest), -1)


def _forward(x, w, cos, sin, ok, c):
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.to(x.dtype)
    return torch.where(ok, _turn(x, cos, sin, c), 0)


def _backward(x, dy, w, cos, sin, ok, c, t):
    g = torch.where(ok, _turn(dy.to(t).view(x.shape), cos, -sin, c), 0)
    if w is None:
        return g, None
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    h, n = g * w.to(t), x * r
    return r * (h - n * (h * n).mean(-1, keepdim=True)), (g * n).sum((0, 1))


# ---- what a pass must not do without ----------------------------------------

def work(case):
    c = case
    e = BYTES[c["dtype"]]
    if c["op"] == "quantize":
        n = c["M"] * c["K"]
        return {"bytes": n * (e + 1) + 4 * c["M"] * c["G"], "flops": 4 * n}
    if c["op"] in ("column", "row"):
        M, K, N = c["M"], c["K"], c["N"]
        out = N // 2 if c.get("act") else N
        return {"bytes": M * K + N * K + 4 * (M * c.get("G", 1) + N) + M * out * e + (N * e if c["bias"] else 0), "flops": 2 * M * N * K}
    T = int(_lengths(c)[0].sum()) if c["op"] == "append" else c["T"]
    qk, v = T * (c["Hq"] + c["Hkv"]) * c["D"], T * c["Hkv"] * c["D"]
    table = T * c["R"] * 4
    if c["op"] == "qk":
        return {"bytes": 2 * qk * e + table + 8 * T, "flops": 8 * qk}
    if c["op"] == "append":
        return {"bytes": 2 * (qk + v) * e + table, "flops": 8 * qk}
    read = 2 if c["norm"] else 1
    return {"bytes": (read + 1) * qk * e + 2 * v * e + table + 8 * T, "flops": 16 * qk}


# ---- the same from the definition, in 64 bits -------------------------------

def exact(case, seed):
    c, st = case, prepare(case, seed)
    f = torch.float64
    if c["op"] == "quantize":
        x = st["X"].to(f).unflatten(1, (c["G"], -1))
        held = (x.abs().max(dim=2).values / 127).float().to(f)          # a scale is held in 32 bits
        whole = torch.round(x / held.clamp(min=1e-300).unsqueeze(2))
        return (whole.clamp(-127, 127) * held.unsqueeze(2)).flatten(1), held
    if c["op"] in ("column", "row"):
        P, K, N = c["P"], c["K"], c["N"]
        sx = st["sx"].to(f).repeat_interleave(K // st["sx"].shape[1], 1)
        y = torch.mm(st["X"].to(f) * sx, (st["W"].to(f) * st["sw"].to(f)[:, None]).t().contiguous())
        if c["bias"]:
            y += st["bias"].to(f)
        if c["op"] == "row":
            return y
        parts = list(y.chunk(P, 1))
        if c["act"]:
            parts = [p[:, :N // P // 2] * torch.sigmoid(p[:, :N // P // 2]) * p[:, N // P // 2:] for p in parts]
        return torch.stack(parts) if c["shards"] else torch.cat(parts, 1)
    # the rotation of a pair as a product of complex numbers
    P, D, R, Hq, Hkv = c["P"], c["D"], c["R"], c["Hq"], c["Hkv"]
    blocks = list(st["qkv"]) if c["shards"] else st["qkv"].chunk(P, 1)
    cut = lambda lo, hi: torch.cat([b[:, lo // P * D:hi // P * D] for b in blocks], 1).to(f).unflatten(1, (-1, D))  # noqa: E731
    q, k, v = cut(0, Hq), cut(Hq, Hq + Hkv), cut(Hq + Hkv, Hq + 2 * Hkv)
    if c["op"] == "append":
        own_seq = torch.repeat_interleave(torch.arange(c["B"], device=DEV), (st["cu"][1:] - st["cu"][:-1]).long())
        pos = st["past"].long()[own_seq] + torch.arange(q.shape[0], device=DEV) - st["cu"].long()[own_seq]
    else:
        pos = st["pos"]
    there = (pos >= 0).to(f).view(-1, 1, 1)
    z = torch.complex(st["cos"].to(f), st["sin"].to(f))[pos.clamp(min=0)].unsqueeze(1)

    def turn(x, by):
        p = x[..., :R].unflatten(-1, (R // 2, 2)) if c["pairs"] else x[..., :R].unflatten(-1, (2, R // 2)).transpose(-1, -2)
        p = torch.view_as_real(torch.view_as_complex(p.contiguous()) * by)
        p = p if c["pairs"] else p.transpose(-1, -2)
        return torch.cat((p.flatten(-2), x[..., R:]), -1) * there

    def unit(x, w):
        return x if w is None else x / (x.pow(2).sum(-1, keepdim=True) / D + 1e-6).sqrt() * w.to(f)

    if c["op"] == "qk_backward":
        def back(x, w, dy):
            with torch.enable_grad():
                x = x.clone().requires_grad_()
                w = None if w is None else w.to(f).requires_grad_()
                y = turn(unit(x, w), z)
                got = torch.autograd.grad(y, [x] if w is None else [x, w], dy.to(f).view(y.shape))
            return got[0], None if w is None else got[1]
        (dq, dwq), (dk, dwk) = back(q, st["wq"], st["dQ"]), back(k, st["wk"], st["dK"])
        dv = st["dV"].to(f).unflatten(1, (-1, D))
        parts = [torch.cat([x.chunk(P, 1)[i].flatten(1) for x in (dq, dk, dv)], 1) for i in range(P)]
        return torch.stack(parts) if c["shards"] else torch.cat(parts, 1), dwq, dwk
    q, k = turn(unit(q, st["wq"]), z).flatten(1), turn(unit(k, st["wk"]), z)
    if c["op"] == "qk":
        return q, k.flatten(1)
    kc, vc = st["kc"].to(f), st["vc"].to(f)
    row = st["table"].long()[own_seq, pos // c["page"]] * c["page"] + pos % c["page"]
    kc.view(-1, Hkv, D)[row] = k
    vc.view(-1, Hkv, D)[row] = v
    return q, kc, vc
