"""The append to a cache in 8 bits and the cache's rows as matrices, against plain
computations in 64 bits on the CPU, and the steps of an attention block in a row.

Tolerances.  Without norm and rotation the values are the data's: scales and whole
numbers are the quantizer's, bit for bit.  With them a key is off by e = (D / 2 + 12) u
times its magnitude (a norm's sum of D squares has D + 6 roundings before the root
halves them; u = 2^-24; the magnitude of a rotated pair is |a cos| + |b sin|), so a
scale by e / 127 of the largest magnitude plus its own rounding, and a whole number is
one of those that the quotients within e of the value round to: the value that it
stands for is at most scale / 2 plus e and the scale's error (times 127) away."""
import pytest
import torch

import tensor_linear_amd as tl
from gpu_util import DEV
from test_gpu_heads import TYPES, dev, forward, make, split

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


class Pages:
    """A paged cache in 8 bits for sequences of the lengths `lens` behind `past`, in any order of memory."""

    def __init__(self, lens, past, Hkv, D, page, order="slot", pad=0, seed=0, lead=0):
        g = torch.Generator().manual_seed(seed)
        self.cu = torch.tensor([lead] + [lead + sum(lens[:i + 1]) for i in range(len(lens))], dtype=torch.int32, device=DEV)
        self.past = torch.tensor(past, dtype=torch.int32, device=DEV)
        need = [-(-max(1, n + p) // page) for n, p in zip(lens, past)]
        self.n, self.page = sum(need) + 2, page
        ids = torch.randperm(self.n, generator=g).tolist()
        table = torch.zeros((len(lens), max(need)), dtype=torch.int32)
        for s, k in enumerate(need):
            table[s, :k] = torch.tensor(ids[:k])
            ids = ids[k:]
        self.table = table.to(DEV)
        mem = [self.n, Hkv, page] if order == "head" else [self.n, page, Hkv]
        view = (lambda x: x.transpose(1, 2)) if order == "head" else (lambda x: x)
        self.kc, self.vc = (view(torch.full(mem + [D + pad], 77, dtype=torch.int8, device=DEV)[..., :D]) for _ in "kv")
        self.ks, self.vs = (view(torch.full(mem, 5.0, device=DEV)) for _ in "kv")
        self.rows = [(s, lead + sum(lens[:s]) + i, past[s] + i) for s in range(len(lens)) for i in range(lens[s])]

    def place(self, s, p):
        return int(self.table[s, p // self.page]), p % self.page


def lengths(T):
    """Lengths of sequences that own T rows but one before the first and one behind the last."""
    lens, left = [], max(0, T - 2)
    while left > 0:
        n = min(left, len(lens) % 4)
        lens.append(n)
        left -= n
    return lens or [0]


CASES = [  # T, Hq, Hkv, D, R, P, pairs, norms, shards, extra
    (3, 1, 1, 16, 16, 1, False, "qk", False, 0), (7, 8, 2, 128, 128, 2, False, "qk", False, 0), (9, 8, 2, 128, 128, 2, True, "qk", True, 8),
    (6, 6, 3, 64, 32, 3, False, "", False, 0), (9, 4, 4, 80, 80, 2, True, "q", True, 0), (5, 12, 4, 96, 32, 4, False, "k", False, 16),
    (4, 16, 8, 256, 256, 8, False, "qk", False, 0), (9, 4, 2, 40, 20, 2, False, "qk", True, 0), (8, 3, 1, 7, 6, 1, True, "qk", False, 1),
    (6, 4, 2, 128, 128, 2, False, "qk", True, 1), (4, 2, 2, 512, 64, 1, False, "qk", False, 0), (5, 2, 1, 600, 600, 1, True, "qk", False, 0),
    (300, 8, 1, 128, 128, 1, False, "qk", False, 0), (9001, 2, 1, 32, 32, 1, False, "qk", False, 0), (7, 4, 2, 80, 40, 2, False, "qk", True, 0),
    (8, 6, 3, 80, 40, 3, True, "qk", False, 1), (5, 4, 2, 16, 8, 2, False, "q", False, 0), (200, 4, 4, 128, 120, 4, False, "", True, 0)]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("order,pad", [("slot", 0), ("head", 5)])
def test_append_quant(case, order, pad, t):
    print("append quant", case, order, t, flush=True)
    T, Hq, Hkv, D, R, P, pairs, norms, shards, extra = case
    x, X, _, _, _, _, wq, wk = make(case, t)
    lens = lengths(T)
    past = [(7 * s + 3) % 40 for s in range(len(lens))]
    pg = Pages(lens, past, Hkv, D, 16, order, pad, lead=1)
    n = 60 + max(lens)
    inv = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / max(R, 1))
    angle = torch.arange(n, dtype=torch.float64)[:, None] * inv
    cos, sin = angle.cos().float(), angle.sin().float()
    Q = torch.full((T, Hq * D), 9.0, dtype=t, device=DEV)
    bad = torch.zeros(1, dtype=torch.int32, device=DEV)
    args = dict(q_weight=dev(wq), k_weight=dev(wk), style=tl.TP_ROPE_PAIRS if pairs else tl.TP_ROPE_HALVES,
                x_mode=tl.TP_Y_SHARDS if shards else tl.TP_Y_CONCAT, eps=1e-5)
    tl.tp_kv_append_quant(X, dev(cos), dev(sin), pg.past, pg.cu, pg.table, pg.kc, pg.vc, pg.ks, pg.vs, P, Hq, Hkv, Q=Q, bad=bad, **args)
    torch.cuda.synchronize()
    assert bad.item() == 0
    q, k, v = split(x, P, Hq, Hkv, shards)
    at = torch.zeros(T, dtype=torch.long)
    for s, row, p in pg.rows:
        at[row] = p
    c, s_ = cos.double()[at][:, None], sin.double()[at][:, None]
    ok = torch.ones(T, 1, 1, dtype=torch.bool)
    eps = (D / 2 + 12) * U * 1.01
    kk, kmag = forward(k, wk, c, s_, R, pairs, ok, 1e-5)
    kc, vc, ks, vs = (y.cpu() for y in (pg.kc, pg.vc, pg.ks, pg.vs))
    mine = [r for _, r, _ in pg.rows]
    place = [pg.place(s, p) for s, _, p in pg.rows]
    if mine:
        pi, si = (torch.tensor(z) for z in zip(*place))
        for cache, scale, want, mag in ((kc, ks, kk, kmag), (vc, vs, v, v.abs())):
            want, mag = want[mine], mag[mine]
            got_q, got_s = cache[pi, si].double(), scale[pi, si].double()
            big = want.abs().amax(-1)
            es = eps * mag.amax(-1) / 127 + U * big / 127 * 2
            assert ((got_s - big / 127).abs() <= es).all()
            off = (got_q * got_s[..., None] - want).abs()
            bound = (got_s / 2 + 127 * es)[..., None] + eps * mag
            assert (off <= bound * (1 + 1e-9)).all(), (off - bound).max()
            assert (got_q.abs() <= 127).all() and (got_q.abs().amax(-1) == 127).logical_or(big == 0).all()
            # the quantizer's numbers for the values, bit for bit (and for keys that nothing touches)
            if want is not kk[mine] and (mag == want.abs()).all() and scale is vs:
                e = (big / 127).float()
                whole = torch.where(e[..., None] > 0, want / e.double()[..., None], 0.0).round().clamp(-127, 127)
                assert torch.equal(got_s.float(), e) and torch.equal(got_q, whole)
    # nothing else was written
    touched = torch.zeros(kc.shape[:2], dtype=torch.bool)
    for p, s in place:
        touched[p, s] = True
    assert (kc[~touched] == 77).all() and (vc[~touched] == 77).all() and (ks[~touched] == 5.0).all() and (vs[~touched] == 5.0).all()
    own = torch.zeros(T, dtype=torch.bool)
    own[mine] = True
    assert (Q.cpu()[~own] == 9.0).all()
    # queries: those of the append to a cache of the data's type
    Q2 = torch.full((T, Hq * D), 9.0, dtype=t, device=DEV)
    k2, v2 = (torch.zeros((pg.n, 16, Hkv, D), dtype=t, device=DEV) for _ in "kv")
    tl.tp_kv_append(X, dev(cos), dev(sin), pg.past, pg.cu, pg.table, k2, v2, P, Hq, Hkv, Q=Q2, **args)
    assert torch.equal(Q, Q2)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("D", [16, 64, 128, 40, 9])
def test_plain_values_are_the_quantizers(D, t):
    """Without norm and rotation: tp_quantize_rows' scales and whole numbers, halves, zeros, tiny and huge values, NaN."""
    T, Hq, Hkv = 40, 2, 2
    g = torch.Generator().manual_seed(D)
    x = torch.randn((T, 6 * D), generator=g)
    x[1] = 0.0
    x[2, 2 * D:] *= 1e-30
    x[3] *= 1e30
    x[4, 2 * D + 1] = float("nan")
    x[5, 5 * D] = float("inf")
    x[6, 2 * D:] = torch.arange(4 * D).float() % 255 - 127           # quotients of whole numbers and halves
    x[7, 2 * D:] = (torch.arange(4 * D).float() % 127 + 0.5)
    x[7, 2 * D], x[7, 3 * D], x[7, 4 * D], x[7, 5 * D] = 127, 127, 127, 127
    x[8, 2 * D:] = 1e-44
    X = x.to(t).to(DEV)
    pg = Pages([T], [3], Hkv, D, 16)
    tl.tp_kv_append_quant(X, None, None, pg.past, pg.cu, pg.table, pg.kc, pg.vc, pg.ks, pg.vs, 1, Hq, Hkv)
    q = torch.empty((T, 4 * D), dtype=torch.int8, device=DEV)
    s = torch.empty((T, 4), device=DEV)
    tl.tp_quantize_rows(X[:, 2 * D:], q, s)
    at = torch.tensor([pg.place(0, 3 + i) for i in range(T)], device=DEV)
    got = torch.cat((pg.kc[at[:, 0], at[:, 1]], pg.vc[at[:, 0], at[:, 1]]), 1).view(T, 4 * D)
    gs = torch.cat((pg.ks[at[:, 0], at[:, 1]], pg.vs[at[:, 0], at[:, 1]]), 1)
    assert torch.equal(got, q) and torch.equal(gs.nan_to_num(-1.0), s.nan_to_num(-1.0))


@pytest.mark.parametrize("t", TYPES)
def test_append_quant_outside(t):
    """Pages and positions outside the cache: not appended, a zero query row, the flag."""
    T, Hq, Hkv, D = 6, 2, 1, 32
    X = torch.randn((T, 4 * D), generator=torch.Generator().manual_seed(1)).to(t).to(DEV)
    pg = Pages([1] * 6, [0, 5, 17, 33, 40, 2], Hkv, D, 16)
    pg.table[0, 0], pg.table[1, 0], pg.table[2, 1] = -1, pg.n, 2 ** 31 - 1
    pg.past[3], pg.past[4] = -1, 10 ** 6
    bad = torch.zeros(1, dtype=torch.int32, device=DEV)
    Q = torch.full((T, Hq * D), 9.0, dtype=t, device=DEV)
    tl.tp_kv_append_quant(X, None, None, pg.past, pg.cu, pg.table, pg.kc, pg.vc, pg.ks, pg.vs, 1, Hq, Hkv, Q=Q, bad=bad)
    assert bad.item() == 1 and (Q[:5] == 0).all() and torch.equal(Q[5], X[5, :Hq * D])
    assert (pg.ks != 5.0).sum() == 1


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("Hkv,D,order,pad,extra", [(2, 128, "slot", 0, 0), (8, 64, "head", 0, 8), (1, 80, "slot", 3, 1), (3, 7, "head", 2, 3), (5, 40, "slot", 0, 0),
                                                  (2, 1024, "slot", 0, 0)])
def test_read(Hkv, D, order, pad, extra, int8, t):
    lens, past = [3, 0, 20, 1], [0, 5, 9, 31]
    pg = Pages(lens, past, Hkv, D, 16, order, pad, lead=2)
    g = torch.Generator().manual_seed(3)
    T = 2 + sum(lens) + 3
    if int8:
        for c, s in ((pg.kc, pg.ks), (pg.vc, pg.vs)):
            c.copy_(torch.randint(-127, 128, c.shape, generator=g))
            s.copy_(torch.rand(s.shape, generator=g) + 0.1)
        kc, vc, sc = pg.kc, pg.vc, dict(k_scale=pg.ks, v_scale=pg.vs)
        wide = [c.cpu().double() * s.cpu().double()[..., None] for c, s in ((kc, pg.ks), (vc, pg.vs))]
    else:
        mem = (pg.n, Hkv, 16, D + pad) if order == "head" else (pg.n, 16, Hkv, D + pad)
        kc, vc = (torch.randn(mem, generator=g).to(t).to(DEV)[..., :D] for _ in "kv")
        if order == "head":
            kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
        sc, wide = {}, [kc.cpu().double(), vc.cpu().double()]
    pg.table[2, 1] = pg.n                    # a page outside
    bad = torch.zeros(1, dtype=torch.int32, device=DEV)
    Kb, Vb = (torch.full((T, Hkv * D + extra), 9.0, dtype=t, device=DEV) for _ in "kv")
    K, V = Kb[:, :Hkv * D], Vb[:, :Hkv * D]
    tl.tp_kv_read(pg.past, pg.cu, pg.table, kc, vc, K, V, bad=bad, **sc)
    torch.cuda.synchronize()
    assert bad.item() == 1
    own = torch.zeros(T, dtype=torch.bool)
    for got, w in ((K.cpu(), wide[0]), (V.cpu(), wide[1])):
        for s, row, p in pg.rows:
            own[row] = True
            page, slot = pg.place(s, p)
            # one product in fp32 and one rounding
            want = w[page, slot].flatten().float().to(t) if page < pg.n else torch.zeros(Hkv * D, dtype=t)
            assert torch.equal(got[row], want), (s, row, p)
        assert (got[~own] == 9.0).all()
    assert (Kb[:, Hkv * D:] == 9.0).all() and (Vb[:, Hkv * D:] == 9.0).all()
    only = torch.full((T, Hkv * D), 9.0, dtype=t, device=DEV)
    tl.tp_kv_read(pg.past, pg.cu, pg.table, kc, vc, None, only, **sc)
    assert torch.equal(only, V)
    only.fill_(9.0)
    tl.tp_kv_read(pg.past, pg.cu, pg.table, kc, vc, only, None, **sc)
    assert torch.equal(only, K)


def test_read_more_than_a_launch_holds():
    """More rows than the wavefronts of one launch (2^25)."""
    T, page = (1 << 25) + 100, 1 << 20
    kc = torch.randint(-127, 128, (33, page, 1, 8), dtype=torch.int8, device=DEV)
    ks = torch.rand((33, page, 1), device=DEV)
    cu, past = torch.tensor([0, T], dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    table = torch.arange(32, -1, -1, dtype=torch.int32, device=DEV)[None]
    K = torch.empty((T, 8), dtype=torch.bfloat16, device=DEV)
    tl.tp_kv_read(past, cu, table, kc, kc, K, None, k_scale=ks, v_scale=ks)
    wide = (kc.float() * ks[..., None]).bfloat16().flip(0).view(-1, 8)[:T]
    assert torch.equal(K, wide)


def test_block_in_a_row():
    """QKV layer in 8 bits, append in 8 bits, attention over it, row layer, norm: a decode step and a chunk through a captured
    graph, against the same steps in 64 bits from the cache's own contents."""
    P, Hq, Hkv, D, M = 2, 8, 2, 64, 7
    Hd = 256
    g = torch.Generator().manual_seed(4)
    N = (Hq + 2 * Hkv) * D
    x = torch.randn((M, Hd), generator=g).bfloat16().to(DEV)
    Wqkv, Wo = (torch.randn(s, generator=g).mul_(0.05).to(DEV) for s in ((N, Hd), (Hd, Hq * D)))
    e8 = lambda *s: torch.empty(s, dtype=torch.int8, device=DEV)  # noqa: E731
    ef = lambda *s: torch.empty(s, device=DEV)  # noqa: E731
    eb = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    wq, sw, wo, so = e8(N, Hd), ef(N), e8(Hd, Hq * D), ef(Hd)
    tl.tp_quantize_rows(Wqkv, wq, sw)
    tl.tp_quantize_rows(Wo, wo, so)
    pg = Pages([1, 5, 1], [40, 0, 90], Hkv, D, 16)
    pg.kc.zero_(), pg.vc.zero_(), pg.ks.fill_(0.01), pg.vs.fill_(0.01)
    pg.kc.copy_(torch.randint(-127, 128, pg.kc.shape, generator=g))
    pg.vc.copy_(torch.randint(-127, 128, pg.vc.shape, generator=g))
    ang = torch.arange(128, dtype=torch.float64)[:, None] * 1e4 ** (-torch.arange(32, dtype=torch.float64) / 32)
    cos, sin = ang.cos().float().to(DEV), ang.sin().float().to(DEV)
    xq, sx, qkv, q, o, oq, os_, y = e8(M, Hd), ef(M), eb(M, N), eb(M, Hq * D), eb(M, Hq * D), e8(M, Hq * D), ef(M, P), eb(M, Hd)
    h, n8, ns = eb(M, Hd), e8(M, Hd), ef(M)
    pre = torch.ones(Hd, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(max(256, tl.tp_kv_attention_workspace_bytes(M, 3, Hq, Hkv, D)), dtype=torch.uint8, device=DEV)
    wr = torch.empty(tl.tp_row_workspace_bytes(tl.TP_ROW_FUSED, M, Hd, P), dtype=torch.uint8, device=DEV)

    def block():
        tl.tp_quantize_rows(x, xq, sx)
        tl.tp_linear_column_quant(xq, sx, wq, sw, qkv, P)
        tl.tp_kv_append_quant(qkv, cos, sin, pg.past, pg.cu, pg.table, pg.kc, pg.vc, pg.ks, pg.vs, P, Hq, Hkv, Q=q)
        tl.tp_kv_attention(q, pg.past, pg.cu, pg.table, pg.kc, pg.vc, o, ws, k_scale=pg.ks, v_scale=pg.vs)
        tl.tp_quantize_rows(o, oq, os_)
        tl.tp_linear_row_quant(oq, os_, wo, so, y, P, tl.TP_ROW_FUSED, wr)
        tl.tp_residual_norm(y, h, n8, residual=x, pre_weight=pre, scale=ns)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block()
    for step in range(3):
        x.copy_(torch.randn((M, Hd), generator=g))
        block()
        torch.cuda.synchronize()
        eager = [t.clone() for t in (q, o, y, h, n8, ns, pg.kc, pg.ks)]
        for t in (q, o, y, h, n8, ns):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, (q, o, y, h, n8, ns, pg.kc, pg.ks)):
            assert torch.equal(a, b)
        # attention and norm from what the steps before them left
        kk, vv = ((c.cpu().double() * s.cpu().double()[..., None]) for c, s in ((pg.kc, pg.ks), (pg.vc, pg.vs)))
        got = o.cpu().double().view(M, Hq, D)
        for s, row, p in pg.rows:
            pl = [pg.place(s, j) for j in range(p + 1)]
            k = torch.stack([kk[a, b] for a, b in pl]).repeat_interleave(Hq // Hkv, 1)
            v = torch.stack([vv[a, b] for a, b in pl]).repeat_interleave(Hq // Hkv, 1)
            w = ((q[row].cpu().double().view(Hq, D) * k).sum(-1) * D ** -0.5).softmax(0)
            want = (w[..., None] * v).sum(0)
            A = (w[..., None] * v.abs()).sum(0)
            assert ((got[row] - want).abs() <= A * (2.0 ** -8 + 1e-3) + 2.0 ** -8 * want.abs()).all()
        hd = x.cpu().double() + y.cpu().double()
        nd = hd * torch.rsqrt(hd.square().mean(-1, keepdim=True) + 1e-6)
        assert ((h.cpu().double() - hd).abs() <= 2.0 ** -8 * hd.abs() + 1e-6).all()
        assert ((n8.cpu().double() * ns.cpu().double()[:, None] - nd).abs() <= ns.cpu().double()[:, None] * 0.5 + 1e-4).all()
