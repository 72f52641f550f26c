"""Cases that measure attention of new tokens over a paged cache, the cache in
8 bits (its append and reading it back), and the norms around a block with its
gate and residual.

`run` computes a case with elementary torch operations in 32 bits (64 for what
is rounded to whole numbers), or, with `own`, through this package's entry
points.  `exact` computes it in 64 bits from the definition.

Sequence s of a call has the new tokens cu[s] .. cu[s + 1] - 1 at the positions
past[s], past[s] + 1, ...; position p lies in slot p % page of cache page
table[s, p // page].  Caches are [pages, page, key heads, D]; an 8-bit cache has
a scale for each token and head, [pages, page, key heads].
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
EPS = 1e-6


def listed():
    return [
        # One new token of 4 sequences just begun: latency.
        dict(name="attention decode short", op="attention", B=4, longest=1, past=300, page=16, Hq=32, Hkv=8, D=128, window=0, int8=False, lse=False, even=False, dtype="bf16"),
        # One new token of 64 sequences with pasts of any length up to 8000: the cache's bytes bound it.
        dict(name="attention decode", op="attention", B=64, longest=1, past=8000, page=16, Hq=64, Hkv=8, D=128, window=0, int8=False, lse=False, even=False, dtype="bf16"),
        # The same over a cache in 8 bits, as a server keeps it that wants twice the tokens.
        dict(name="attention decode int8", op="attention", B=64, longest=1, past=16000, page=32, Hq=32, Hkv=8, D=128, window=0, int8=True, lse=False, even=False, dtype="bf16"),
        # A prompt of 4096 tokens, none before it: the matrix products bound it.
        dict(name="attention prompt", op="attention", B=1, longest=4096, past=0, page=16, Hq=64, Hkv=8, D=128, window=0, int8=False, lse=False, even=True, dtype="bf16"),
        # Chunks of several prompts over an 8-bit cache, heads of 96, a sliding window.
        dict(name="attention chunks", op="attention", B=12, longest=600, past=3000, page=64, Hq=24, Hkv=8, D=96, window=1024, int8=True, lse=True, even=False, dtype="bf16"),
        # fp32 heads of 80, a few ragged chunks, with the logarithms of the sums.
        dict(name="attention f32", op="attention", B=5, longest=130, past=700, page=16, Hq=12, Hkv=4, D=80, window=0, int8=False, lse=True, even=False, dtype="f32"),
        # The decode step's keys and values into the 8-bit cache, normed and rotated; latency.
        dict(name="append int8 decode", op="append", B=64, longest=1, past=8000, page=16, Hq=64, Hkv=8, D=128, R=128, P=8, pairs=False, norm=True, shards=False, dtype="bf16"),
        # Prompts of different lengths into the 8-bit cache in one call.
        dict(name="append int8 prompts", op="append", B=12, longest=1500, past=700, page=64, Hq=64, Hkv=8, D=128, R=128, P=8, pairs=False, norm=True, shards=False, dtype="bf16"),
        # The first 4000 tokens or fewer of 12 sequences read back as bf16 rows.
        dict(name="read back int8", op="read", B=12, longest=4000, past=0, page=16, Hkv=8, D=128, int8=True, dtype="bf16"),
        # Between two blocks of a decode step: 16 tokens of 8192, the next layer's input in 8 bits; latency.
        dict(name="norm decode", op="norm", T=16, F=8192, gate="none", post=False, pre=True, int8=True, dtype="bf16"),
        # The same steps over a 4096-token prompt, a norm on either side and a learned gate.
        dict(name="norm prompt", op="norm", T=4096, F=8192, gate="feature", post=True, pre=True, int8=False, dtype="bf16"),
        # Their gradients in a training step of 4096 tokens.
        dict(name="norm backward", op="norm_backward", T=4096, F=4096, gate="feature", post=True, pre=True, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("attention", "attention", "attention", "append", "read", "norm", "norm_backward"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    if op in ("norm", "norm_backward"):
        F = _log(rng, 128, 16384)
        F -= F % rng.choice((1, 8, 128)) if F > 256 else 0
        gate = rng.choice(("none", "feature", "token"))
        most = (1 << 26 if op == "norm" else 1 << 25) // BYTES[dtype] // (2 if gate == "token" else 1)
        c = dict(op=op, T=_log(rng, 1, max(2, min(8192, most // F))), F=F, gate=gate, post=rng.random() < 0.5, pre=True, dtype=dtype)
        if op == "norm":
            c["int8"] = rng.random() < 0.4
        return c
    D = rng.choice((64, 80, 96, 128, 128, 128, 256))
    page = rng.choice((16, 32, 64))
    if op == "read":
        B, Hkv = _log(rng, 1, 64), rng.choice((1, 2, 4, 8))
        longest = max(1, min(_log(rng, 1, 4000), 48_000_000 // (B * Hkv * D)))
        return dict(op=op, B=B, longest=longest, past=_log(rng, 1, 2000), page=page, Hkv=Hkv, D=D, int8=rng.random() < 0.7, dtype=dtype)
    if op == "append":
        P = rng.choice((1, 2, 4, 8))
        hkv = rng.choice((1, 1, 2))
        Hkv, Hq = hkv * P, hkv * P * rng.choice((1, 3, 4, 8))
        B = _log(rng, 1, 256)
        most = max(2, min(8192, 90_000_000 // (BYTES[dtype] * (Hq + 2 * Hkv) * D)))
        return dict(op=op, B=B, longest=max(1, min(_log(rng, 1, 4096), most // B)), past=_log(rng, 1, 8000), page=page, Hq=Hq, Hkv=Hkv, D=D,
                    R=D if rng.random() < 0.7 else D // 2, P=P, pairs=rng.random() < 0.3, norm=rng.random() < 0.7, shards=rng.random() < 0.3, dtype=dtype)
    # attention: one token a sequence half the time, else chunks and prompts
    Hkv, G = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 8))
    Hq = Hkv * G
    window = rng.choice((0, 0, 0, _log(rng, 16, 4096)))
    c = dict(op=op, page=page, Hq=Hq, Hkv=Hkv, D=D, window=window, int8=rng.random() < 0.4, lse=rng.random() < 0.4, even=rng.random() < 0.2, dtype=dtype)
    if rng.random() < 0.5:
        B = _log(rng, 1, 128)
        most = int(1e9 / (BYTES[dtype] * B * Hkv * D))        # keys of a sequence
        return dict(c, B=B, longest=1, past=max(1, min(_log(rng, 16, 16000), most)))
    B = _log(rng, 1, 16)
    longest = _log(rng, 2, 4096)
    past = rng.choice((0, _log(rng, 1, 8000)))
    # at most 5.4e8 pairs of a query head's token and a key, 1.2e8 in fp32
    while B * Hq * longest * (longest / 2 + past) * max(1.0, D / 128) > (5.4e8 if dtype == "bf16" else 1.2e8):
        longest, past = longest // 2 + 1, past // 2
        B = max(1, B - 1)
    return dict(c, B=B, longest=longest, past=past)


# ---- inputs -----------------------------------------------------------------

def _lengths(c):
    """New tokens and past lengths of the sequences: part of the case, so that every seed has the same sizes."""
    B = c["B"]
    if c.get("even"):
        return torch.full((B,), c["longest"]), torch.full((B,), c["past"])
    r = torch.Generator()
    r.manual_seed(B * 65536 + c["longest"])
    return torch.randint(1, c["longest"] + 1, (B,), generator=r), torch.randint(0, c["past"] + 1, (B,), generator=r)


def _tables(n, R):
    """cos and sin of the positions 0 .. n-1, angles in 64 bits."""
    inv = 10000.0 ** (-torch.arange(0, R, 2, device=DEV, dtype=torch.float64) / R)
    a = torch.arange(n, device=DEV, dtype=torch.float64)[:, None] * inv
    return a.cos().float(), a.sin().float()


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    t = TYPES[c["dtype"]]
    rn = lambda *shape, s=1.0, mean=0.0: torch.randn(shape, generator=g, device=DEV).mul_(s).add_(mean).to(t)  # noqa: E731
    st = dict(case=c)
    empty = lambda *shape, t=t: torch.empty(shape, dtype=t, device=DEV)  # noqa: E731
    if c["op"] in ("norm", "norm_backward"):
        T, F = c["T"], c["F"]
        # a block's output, and the residual stream, which grows over the layers
        st["Y"], st["R"] = rn(T, F), rn(T, F, s=2.0)
        # per feature: learned gates that begin small; per token: what a condition's layer gives
        st["gate"] = dict(none=lambda: None, feature=lambda: rn(F, s=0.1, mean=0.3), token=lambda: rn(T, F, s=0.5))[c["gate"]]()
        st["post"], st["pre"] = (rn(F, s=0.1, mean=1.0) if c[k] else None for k in ("post", "pre"))
        if c["op"] == "norm":
            st["H"] = empty(T, F)
            st["N"] = empty(T, F, t=torch.int8 if c["int8"] else t)
            if c["int8"]:
                st["scale"], st["values"] = empty(T, t=torch.float32), empty(T, F, t=torch.bfloat16)
            return st
        st["dH"], st["dN"] = rn(T, F), rn(T, F)
        st["dY"], st["dR"] = empty(T, F), empty(T, F)
        st["dgate"] = dict(none=lambda: None, feature=lambda: empty(F, t=torch.float32), token=lambda: empty(T, F))[c["gate"]]()
        st["dpost"], st["dpre"] = (empty(F, t=torch.float32) if c[k] else None for k in ("post", "pre"))
        # room for the sums of 1024 workgroups
        st["ws"] = empty(3 * 1024 * F * 4, t=torch.uint8)
        return st
    Hkv, D, B, page = c["Hkv"], c["D"], c["B"], c["page"]
    lens, past = _lengths(c)
    T = int(lens.sum())
    r = torch.Generator()
    r.manual_seed(seed)
    most = -(-int((lens + past).max()) // page)
    # pages in any order; only those that the call reads or writes have places of their own
    first = (past if c["op"] in ("append", "read") else 0 * past) // page
    last = (past + lens - 1) // page
    ends = (last - first + 1).cumsum(0)
    pages = int(ends[-1]) + 3
    order = torch.randperm(pages, generator=r).to(torch.int32)
    at = torch.arange(most)[None, :] - first[:, None]
    mine = (at >= 0) & (at <= (last - first)[:, None])
    st["table"] = torch.where(mine, order[((ends - (last - first + 1))[:, None] + at).clamp(0, pages - 1)], 0).to(torch.int32).to(DEV)
    st["cu"] = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)]).to(torch.int32).to(DEV)
    st["past"] = past.to(torch.int32).to(DEV)
    if c.get("int8", True):     # normal values at about 4 sigma full scale
        ints = lambda: torch.randn((pages, page, Hkv, D), generator=g, device=DEV).mul_(32.0).round_().clamp_(-127, 127).to(torch.int8)  # noqa: E731
        st["kc"], st["vc"] = ints(), ints()
        st["ks"], st["vs"] = (torch.rand((pages, page, Hkv), generator=g, device=DEV).add_(0.5).div_(32.0) for _ in "kv")
    else:
        st["kc"], st["vc"] = rn(pages, page, Hkv, D), rn(pages, page, Hkv, D)
        st["ks"] = st["vs"] = None
    if c["op"] == "read":
        st["K"], st["V"] = empty(T, Hkv * D), empty(T, Hkv * D)
        return st
    Hq = c["Hq"]
    if c["op"] == "attention":
        # scores of a standard deviation of 2
        st["Q"] = rn(T, Hq * D, s=2.0)
        st["O"] = empty(T, Hq * D)
        st["lse"] = empty(T, Hq, t=torch.float32) if c["lse"] else None
        st["ws"] = empty(256 << 20, t=torch.uint8)
        return st
    P, R = c["P"], c["R"]
    per = (Hq + 2 * Hkv) // P * D
    st["qkv"] = rn(P, T, per) if c["shards"] else rn(T, P * per)
    st["cos"], st["sin"] = _tables(c["longest"] + c["past"] + 1, R)
    st["wq"], st["wk"] = (rn(D, s=0.1, mean=1.0) if c["norm"] else None for _ in "qk")
    st["Q"] = empty(T, Hq * D)
    # all pages in their order as one sequence, which is read back after the append
    st["whole"] = dict(past=torch.zeros(1, dtype=torch.int32, device=DEV), table=torch.arange(pages, dtype=torch.int32, device=DEV)[None],
                       cu=torch.tensor([0, pages * page], dtype=torch.int32, device=DEV))
    st["K"], st["V"] = (empty(pages * page, Hkv * D, t=torch.bfloat16) for _ in "kv")
    return st


# ---- one pass ---------------------------------------------------------------

def run(st):
    c = st["case"]
    if own:
        return _own(st, c, c["op"])
    return dict(attention=_attention, append=_append, read=_read, norm=_norm, norm_backward=_norm_backward)[c["op"]](st, c)


def _own(st, c, op):
    import tensor_linear_amd as tl
    if op == "attention":
        tl.tp_kv_attention(st["Q"], st["past"], st["cu"], st["table"], st["kc"], st["vc"], st["O"], st["ws"], k_scale=st["ks"], v_scale=st["vs"],
                           window=c["window"], lse=st["lse"])
        return st["O"], st["lse"]
    if op == "append":
        tl.tp_kv_append_quant(st["qkv"], st["cos"], st["sin"], st["past"], st["cu"], st["table"], st["kc"], st["vc"], st["ks"], st["vs"],
                              c["P"], c["Hq"], c["Hkv"], Q=st["Q"], q_weight=st["wq"], k_weight=st["wk"], eps=EPS,
                              style=tl.TP_ROPE_PAIRS if c["pairs"] else tl.TP_ROPE_HALVES,
                              x_mode=tl.TP_Y_SHARDS if c["shards"] else tl.TP_Y_CONCAT)
        w = st["whole"]
        tl.tp_kv_read(w["past"], w["cu"], w["table"], st["kc"], st["vc"], st["K"], st["V"], k_scale=st["ks"], v_scale=st["vs"])
        return st["Q"], st["K"], st["ks"], st["V"], st["vs"]
    if op == "read":
        tl.tp_kv_read(st["past"], st["cu"], st["table"], st["kc"], st["vc"], st["K"], st["V"], k_scale=st["ks"], v_scale=st["vs"])
        return st["K"], st["V"]
    if op == "norm":
        tl.tp_residual_norm(st["Y"], st["H"], st["N"], residual=st["R"], gate=st["gate"], post_weight=st["post"], pre_weight=st["pre"],
                            residual_scale=0.75, branch_scale=0.5, eps=EPS, scale=st.get("scale"))
        return (st["H"], _stands_for(st["N"], st["scale"], st["values"]), st["scale"]) if c["int8"] else (st["H"], st["N"])
    tl.tp_residual_norm_backward(st["Y"], st["dH"], st["dN"], st["dY"], st["dR"], residual=st["R"], gate=st["gate"], post_weight=st["post"],
                                 pre_weight=st["pre"], dgate=st["dgate"], dpost_weight=st["dpost"], dpre_weight=st["dpre"], workspace=st["ws"],
                                 residual_scale=0.75, branch_scale=0.5, eps=EPS)
    return st["dY"], st["dR"], st["dgate"], st["dpost"], st["dpre"]


def _stands_for(q, scale, out):
    """The values that whole numbers and their scales stand for, rounded once to the type that matrix products take."""
    return torch.mul(q, scale.unsqueeze(-1), out=out)


def _to_ints(x):
    """Rows of x in 64 bits to whole numbers and scales max |x| / 127, held in 32 bits."""
    s = (x.abs().amax(-1) / 127.0).float()
    d = s.double().unsqueeze(-1)
    return torch.where(d > 0, x / d, 0.0).round().clamp(-127, 127).to(torch.int8), s


def _sequence(st, T):
    """The sequence of each token and its position."""
    i = torch.arange(T, device=DEV)
    s = torch.searchsorted(st["cu"][1:].long(), i, right=True)
    return s, (st["past"][s] - st["cu"][s]).long() + i


def _gather(st, c, name, rows):
    """Rows of a cache as 32-bit values."""
    x = st[name + "c"].flatten(0, 1)[rows].float()
    return x if st[name + "s"] is None else x * st[name + "s"].flatten(0, 1)[rows].unsqueeze(-1)


def _attention(st, c):
    Hq, Hkv, D, B, page = c["Hq"], c["Hkv"], c["D"], c["B"], c["page"]
    lens, past = _lengths(c)
    n, keys = int(lens.max()), int((lens + past).max())
    j = torch.arange(keys, device=DEV)
    rows = st["table"][:, j // page].long() * page + j % page                              # [B, keys]
    there = j < (st["past"] + st["cu"][1:] - st["cu"][:-1])[:, None]
    k, v = (_gather(st, c, x, torch.where(there, rows, 0)).permute(0, 2, 1, 3).contiguous() for x in "kv")     # [B, Hkv, keys, D]
    T = st["Q"].shape[0]
    i = torch.arange(n, device=DEV)
    tok = (st["cu"][:-1, None] + i).clamp(max=T - 1)
    q = st["Q"].float()[tok].view(B, n, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    s = q @ k.transpose(2, 3).contiguous() * D ** -0.5                                      # [B, Hkv, heads * n, keys]
    pos = (st["past"][:, None] + i)[:, None, None, :, None]
    seen = j <= pos
    if c["window"]:
        seen &= j > pos - c["window"]
    s = s.view(B, Hkv, -1, n, keys).masked_fill_(~seen, float("-inf"))
    m = s.amax(-1, keepdim=True)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, Hkv, -1, keys) @ v).view(B, Hkv, -1, n, D) / total
    seq, at = _sequence(st, T)
    at = at - st["past"][seq]
    st["O"].copy_(o.permute(0, 3, 1, 2, 4)[seq, at].reshape(T, -1))
    if c["lse"]:
        st["lse"].copy_((m + total.log()).squeeze(-1).permute(0, 3, 1, 2)[seq, at].reshape(T, -1))
    return st["O"], st["lse"]


def _read(st, c):
    s, pos = _sequence(st, st["K"].shape[0])
    rows = st["table"][s, pos // c["page"]].long() * c["page"] + pos % c["page"]
    st["K"].copy_(_gather(st, c, "k", rows).flatten(1))
    st["V"].copy_(_gather(st, c, "v", rows).flatten(1))
    return st["K"], st["V"]


def _append(st, c):
    # in 64 bits: values next to a border between two whole numbers
    f = torch.float64
    P, D, R, hq, hk = c["P"], c["D"], c["R"], c["Hq"] // c["P"], c["Hkv"] // c["P"]
    T = st["Q"].shape[0]
    x = (st["qkv"].transpose(0, 1) if c["shards"] else st["qkv"]).reshape(T, P, hq + 2 * hk, D).to(f)
    s, pos = _sequence(st, T)
    cos, sin = st["cos"].to(f)[pos][:, None, None], st["sin"].to(f)[pos][:, None, None]

    def turned(y, w):
        if w is not None:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w.to(f)
        a, b = (y[..., 0:R:2], y[..., 1:R:2]) if c["pairs"] else (y[..., :R // 2], y[..., R // 2:R])
        a, b = a * cos - b * sin, b * cos + a * sin
        return torch.cat((torch.stack((a, b), -1).flatten(-2) if c["pairs"] else torch.cat((a, b), -1), y[..., R:]), -1)

    st["Q"].copy_(turned(x[:, :, :hq], st["wq"]).reshape(T, -1))
    rows = st["table"][s, pos // c["page"]].long() * c["page"] + pos % c["page"]
    for name, y in (("k", turned(x[:, :, hq:hq + hk], st["wk"])), ("v", x[:, :, hq + hk:])):
        q, scale = _to_ints(y.reshape(T, -1, D))
        st[name + "c"].flatten(0, 1)[rows] = q
        st[name + "s"].flatten(0, 1)[rows] = scale
        _stands_for(st[name + "c"].flatten(0, 1), st[name + "s"].flatten(0, 1), st[name.upper()].view(-1, c["Hkv"], D))
    return st["Q"], st["K"], st["ks"], st["V"], st["vs"]


def _wide(st, name, f):
    return None if st[name] is None else st[name].to(f)


def _normed(x, w):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w


def _norm(st, c):
    f = torch.float64 if c["int8"] else torch.float32
    y, post, gate = st["Y"].to(f), _wide(st, "post", f), _wide(st, "gate", f)
    u = y if post is None else _normed(y, post)
    h = 0.75 * st["R"].to(f) + 0.5 * (u if gate is None else u * gate)
    n = _normed(h, st["pre"].to(f))
    st["H"].copy_(h)
    if not c["int8"]:
        st["N"].copy_(n)
        return st["H"], st["N"]
    q, scale = _to_ints(n)
    st["N"].copy_(q)
    st["scale"].copy_(scale)
    return st["H"], _stands_for(st["N"], st["scale"], st["values"]), st["scale"]


def _norm_backward(st, c):
    f = torch.float32
    y, r, post, pre, gate = st["Y"].to(f), st["R"].to(f), _wide(st, "post", f), _wide(st, "pre", f), _wide(st, "gate", f)

    def back(x, w, dy):
        """The gradients of a norm's input and weight."""
        rr = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        z, xn = dy * w, x * rr
        return rr * (z - xn * (z * xn).mean(-1, keepdim=True)), (dy * xn).sum(0)

    u = y if post is None else _normed(y, post)
    h = 0.75 * r + 0.5 * (u if gate is None else u * gate)
    dx, dpre = back(h, pre, st["dN"].to(f))
    dh = st["dH"].to(f) + dx
    st["dpre"].copy_(dpre)
    st["dR"].copy_(0.75 * dh)
    du = 0.5 * dh if gate is None else 0.5 * dh * gate
    if gate is not None:
        dg = 0.5 * dh * u
        st["dgate"].copy_(dg if c["gate"] == "token" else dg.sum(0))
    if post is not None:
        du, dpost = back(y, post, du)
        st["dpost"].copy_(dpost)
    st["dY"].copy_(du)
    return st["dY"], st["dR"], st["dgate"], st["dpost"], st["dpre"]


# ---- what a pass must not do without ----------------------------------------

def work(case):
    c = case
    e = BYTES[c["dtype"]]
    if c["op"] in ("norm", "norm_backward"):
        n = c["T"] * c["F"]
        gate = n * e if c["gate"] == "token" else 0
        if c["op"] == "norm":
            return {"bytes": 3 * n * e + gate + n * (1 if c["int8"] else e), "flops": 10 * n}
        return {"bytes": 6 * n * e + 2 * gate, "flops": 30 * n}
    lens, past = _lengths(c)
    T = int(lens.sum())
    row = c["Hkv"] * c["D"]                                   # values of a token's keys
    held = row + 4 * c["Hkv"] if c.get("int8", True) else row * e
    if c["op"] == "read":
        return {"bytes": 2 * T * (held + row * e), "flops": 2 * T * row}
    if c["op"] == "append":
        # with the caches' values read back
        pages = int(((past + lens - 1) // c["page"] - past // c["page"] + 1).sum()) + 3
        back = 2 * pages * c["page"] * (held + 2 * row)
        return {"bytes": 2 * T * (held + row * e + c["Hq"] * c["D"] * e) + 4 * T * c["R"] + back, "flops": 10 * T * (row + c["Hq"] * c["D"])}
    w = c["window"]
    # keys that some token sees, and pairs of a token and a key that it sees
    first = (past - w + 1).clamp(min=0) if w else 0 * past
    keys = int((past + lens - first).sum())
    pairs = 0
    for n, p in zip(lens.tolist(), past.tolist()):
        full = max(0, min(n, w - p)) if w else n              # tokens that see all before them
        pairs += full * p + full * (full + 1) // 2 + (n - full) * w
    return {"bytes": 2 * keys * held + 2 * T * c["Hq"] * c["D"] * e + (4 * T * c["Hq"] if c["lse"] else 0), "flops": 4 * pairs * c["Hq"] * c["D"]}


# ---- the same from the definition, in 64 bits -------------------------------

def exact(case, seed):
    c, st = case, prepare(case, seed)
    f = torch.float64
    if c["op"] in ("norm", "norm_backward"):
        leaf = {k: st[k].to(f).requires_grad_() for k in ("Y", "R", "gate", "post", "pre") if st[k] is not None}
        unit = lambda x, w: x / (x.pow(2).sum(1, keepdim=True) / c["F"] + EPS).sqrt() * w  # noqa: E731
        with torch.enable_grad():
            u = unit(leaf["Y"], leaf["post"]) if c["post"] else leaf["Y"]
            h = leaf["R"] * 3 / 4 + u * leaf.get("gate", 1) / 2
            n = unit(h, leaf["pre"])
            if c["op"] == "norm_backward":
                grads = dict(zip(leaf, torch.autograd.grad([h, n], list(leaf.values()), [st["dH"].to(f), st["dN"].to(f)])))
                return grads["Y"], grads["R"], grads.get("gate"), grads.get("post"), grads["pre"]
        h, n = h.detach(), n.detach()
        return (h, *_as_ints(n)) if c["int8"] else (h, n)
    page, D, Hkv = c["page"], c["D"], c["Hkv"]
    lens, past = _lengths(c)
    begin = lens.cumsum(0) - lens
    wide = lambda x, s: x.to(f) if s is None else torch.mul(x.to(f), s.to(f)[..., None])  # noqa: E731

    def place(s, p):
        """Cache page and slot of the positions p of sequence s."""
        return st["table"][s].long()[torch.div(p, page, rounding_mode="floor")], p.remainder(page)

    def span(s, lo=None):
        return torch.arange(int(past[s]) if lo is None else lo, int(past[s] + lens[s]), device=DEV)

    if c["op"] == "read":
        k, v = wide(st["kc"], st["ks"]), wide(st["vc"], st["vs"])
        return tuple(torch.cat([x[place(s, span(s))] for s in range(c["B"])]).flatten(1) for x in (k, v))
    if c["op"] == "append":
        return _exact_append(st, c, place, span)
    Hq, w = c["Hq"], c["window"]
    out, lse = [], []
    step = max(1, 400_000_000 // (Hq * int((lens + past).max())))            # tokens at a time
    for s in range(c["B"]):
        at = place(s, span(s, 0))
        k, v = (wide(st[x + "c"][at], None if st[x + "s"] is None else st[x + "s"][at]).transpose(0, 1) for x in "kv")
        k, v = (x.repeat_interleave(Hq // Hkv, 0) for x in (k, v))           # [Hq, keys, D]
        kt = k.transpose(1, 2).contiguous()
        for lo in range(0, int(lens[s]), step):
            hi = min(int(lens[s]), lo + step)
            q = st["Q"][int(begin[s]) + lo:int(begin[s]) + hi].to(f).unflatten(1, (Hq, D)).transpose(0, 1)
            score = torch.bmm(q, kt) / math.sqrt(D)
            back = (int(past[s]) + torch.arange(lo, hi, device=DEV))[:, None] - torch.arange(kt.shape[2], device=DEV)
            score[:, (back < 0) | (back >= (w or 1 << 40))] = -math.inf
            lse.append(score.logsumexp(2).t())
            out.append(torch.bmm(score.softmax(2), v).transpose(0, 1).flatten(1))
    return torch.cat(out), torch.cat(lse) if c["lse"] else None


def _as_ints(x):
    """What 8 bits hold of each row of x, and the scales."""
    held = (x.abs().max(dim=-1).values / 127).float().to(x.dtype)            # a scale is held in 32 bits
    whole = torch.round(x / held.clamp(min=1e-300)[..., None])
    return whole.clamp(-127, 127) * held[..., None], held


def _exact_append(st, c, place, span):
    f = torch.float64
    D, R, Hq, Hkv, P = c["D"], c["R"], c["Hq"], c["Hkv"], c["P"]
    blocks = list(st["qkv"]) if c["shards"] else st["qkv"].chunk(P, 1)
    cut = lambda lo, hi: torch.cat([b[:, lo // P * D:hi // P * D] for b in blocks], 1).to(f).unflatten(1, (-1, D))  # noqa: E731
    pos = torch.cat([span(s) for s in range(c["B"])])
    z = torch.complex(st["cos"].to(f), st["sin"].to(f))[pos].unsqueeze(1)

    def turn(x, w):
        """The rotation of a pair as a product of complex numbers."""
        x = x if w is None else x / (x.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * w.to(f)
        p = x[..., :R].unflatten(-1, (R // 2, 2)) if c["pairs"] else x[..., :R].unflatten(-1, (2, R // 2)).transpose(-1, -2)
        p = torch.view_as_real(torch.view_as_complex(p.contiguous()) * z)
        p = p if c["pairs"] else p.transpose(-1, -2)
        return torch.cat((p.flatten(-2), x[..., R:]), -1)

    q, k, v = turn(cut(0, Hq), st["wq"]), turn(cut(Hq, Hq + Hkv), st["wk"]), cut(Hq + Hkv, Hq + 2 * Hkv)
    at = [place(s, span(s)) for s in range(c["B"])]
    at = tuple(torch.cat([a[i] for a in at]) for i in (0, 1))
    found = [q.flatten(1)]
    for name, x in (("k", k), ("v", v)):
        values, held = _as_ints(x)
        cache = torch.mul(st[name + "c"].to(f), st[name + "s"].to(f)[..., None])
        scales = st[name + "s"].to(f)
        cache[at], scales[at] = values, held
        found += [cache.flatten(0, 1).flatten(1), scales]
    return tuple(found)
