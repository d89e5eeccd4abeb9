"""Attention, its gradient, the 8-bit cache and attention over it on the GPU
against the fp64 oracle, and together with what prepares q and k."""

import numpy as np
import pytest
import torch

from linear_attention_rnn_gated_amd import binding as B
from oracle import attn_oracle as A
from oracle.qk_oracle import qk_bwd, qk_fwd

pytestmark = pytest.mark.gpu

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
DT = {"f32": F32, "bf16": BF16}
UNIT = {"f32": 2.0 ** -22, "bf16": 2.0 ** -8}  # of what goes into a product: see the oracle
NAN, INF = float("nan"), float("inf")


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()


def np64(t):
    return t.detach().double().cpu().numpy()


def half(t):
    return torch.finfo(DT[t]).eps / 2


def check(got, want, bound, what):
    """got within bound of want, and its own rounding on top; infinities and NaN in the same places."""
    h = torch.finfo(got.dtype).eps / 2
    got = np64(got)
    assert got.shape == want.shape, what
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine], want[~fine], equal_nan=True), what
    tol = bound[fine] + h * (np.abs(want[fine]) + bound[fine]) + 2.0 ** -126
    off = np.abs(got[fine] - want[fine])
    bad = ~(off <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.nanmax(off / tol):.3g} of the bound"


def cu_of(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)


def make(lens, Hq, Hkv, d, t, seed=0, lens_k=None, sliced=False, scale=None, extra=0, size=1.0):
    """Inputs on the GPU; `extra` rows behind the last sequence."""
    gen = torch.Generator().manual_seed(seed)
    T = sum(lens) + extra
    Tk = T if lens_k is None else sum(lens_k) + extra

    def rows(n, *heads):
        x = size * torch.randn(n, sum(heads) * d, generator=gen)
        if sliced:
            x = torch.cat([x, torch.full((n, 24), NAN)], 1)
        x = x.to(DT[t]).cuda()
        parts, at = [], 0
        for h in heads:
            y = x[:, at:at + h * d].unflatten(1, (h, d))
            parts.append(y if sliced else y.contiguous())
            at += h * d
        return parts
    p = {"lens": lens, "lens_k": lens if lens_k is None else lens_k, "t": t}
    if lens_k is None:
        p["q"], p["k"], p["v"] = rows(T, Hq, Hkv, Hkv)
        p["cu_k"] = None
    else:
        (p["q"],), (p["k"], p["v"]) = rows(T, Hq), rows(Tk, Hkv, Hkv)
        p["cu_k"] = cu_of(lens_k).cuda()
    p["do"], = rows(T, Hq)
    p["cu"] = cu_of(lens).cuda()
    p["shape"] = B.make_attn_shape(Hq, Hkv, d, DT[t], scale)
    p["scale"] = float(p["shape"].scale)
    return p


def forward(p, **kw):
    return B.gdn_attn_prefill(p["shape"], p["q"], p["k"], p["v"], p["cu"], cu_seqlens_k=p["cu_k"], **kw)


def backward(p, o, lse, **kw):
    return B.gdn_attn_bwd(p["shape"], p["q"], p["k"], p["v"], p["cu"], o, lse, p["do"], cu_seqlens_k=p["cu_k"], **kw)


def spans(p):
    a = b = 0
    for n, m in zip(p["lens"], p["lens_k"]):
        yield slice(a, a + n), slice(b, b + m)
        a, b = a + n, b + m


def check_all(p, o, lse, g=None):
    t = p["t"]
    for i, (rq, rk) in enumerate(spans(p)):
        q, k, v = np64(p["q"][rq]), np64(p["k"][rk]), np64(p["v"][rk])
        wo, wl, bo, bl = A.attn_fwd(q, k, v, p["scale"], UNIT[t])
        check(o[rq], wo, bo, f"o of {i}")
        check(lse[rq], wl, bl, f"lse of {i}")
        if g is None:
            continue
        want = A.attn_bwd(q, k, v, np64(p["do"][rq]), p["scale"], UNIT[t], half(t))
        for name, r in (("dq", rq), ("dk", rk), ("dv", rk)):
            check(g[name][r], *want[name], f"{name} of {i}")


CASES = [
    # lens, Hq, Hkv, d, type, sliced
    ([1], 1, 1, 64, "bf16", False),
    ([0, 1, 2, 0, 31, 32, 33], 2, 1, 64, "bf16", True),
    ([127, 128, 129], 4, 2, 64, "bf16", False),
    ([300, 5], 3, 3, 64, "f32", True),
    ([65, 1, 0, 97], 6, 2, 128, "bf16", True),
    ([257], 8, 1, 128, "bf16", False),
    ([160, 33], 4, 2, 128, "f32", False),
    ([200, 64, 1], 16, 2, 256, "bf16", True),
    ([95, 130], 2, 2, 256, "bf16", False),
    ([70, 129], 3, 1, 256, "f32", True),
    ([4] * 40, 2, 1, 64, "bf16", False),
    ([700], 5, 1, 64, "bf16", False),
]


@pytest.mark.parametrize("lens,Hq,Hkv,d,t,sliced", CASES)
def test_forward_and_gradient(lens, Hq, Hkv, d, t, sliced):
    p = make(lens, Hq, Hkv, d, t, seed=d + len(lens), sliced=sliced)
    o, lse = forward(p)
    assert o.dtype == DT[t] and lse.dtype == F32
    g = backward(p, o, lse)
    check_all(p, o, lse, g)
    again = backward(p, *forward(p))
    assert all(torch.equal(g[k], again[k]) for k in g)


@pytest.mark.parametrize("t,d", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 64), ("f32", 128), ("f32", 256)])
def test_keys_and_queries_of_different_lengths(t, d):
    """More keys than queries, fewer (rows that see nothing), none on either side."""
    p = make([3, 40, 100, 0, 17, 33], 4, 2, d, t, seed=3, lens_k=[200, 40, 35, 9, 0, 161])
    o, lse = forward(p)
    assert not o[43:43 + 65].any() and torch.isneginf(lse[43:43 + 65]).all()
    g = backward(p, o, lse)
    check_all(p, o, lse, g)
    assert not g["dk"][275:284].any() and not g["dv"][275:284].any()  # keys that no query sees


@pytest.mark.parametrize("t,d,Hq,Hkv", [("bf16", 64, 2, 1), ("bf16", 128, 2, 2), ("bf16", 256, 3, 1), ("f32", 64, 4, 2),
                                        ("f32", 128, 1, 1), ("f32", 256, 2, 1)])
def test_gradient_in_parts(t, d, Hq, Hkv):
    """Few heads of many tokens: the tiles of a head are cut into parts, some of them
    empty, and rows behind the last sequence stay as they were."""
    p = make([1030, 0, 3, 391], Hq, Hkv, d, t, seed=23, sliced=True, lens_k=[700, 5, 33, 800])
    T, Tk = 1424, 1538
    assert B.attn_workspace_bytes(p["shape"], T, Tk) >= 4 * d * (2 * T * Hq + 2 * 2 * Tk * Hkv)
    o, lse = forward(p)
    g = backward(p, o, lse)
    check_all(p, o, lse, g)
    again = backward(p, o, lse)
    assert all(torch.equal(g[k], again[k]) for k in g)
    less = dict(p, cu=cu_of(p["lens"][:3]).cuda(), cu_k=cu_of(p["lens_k"][:3]).cuda())
    out = {k: torch.full_like(g[k], 5.0) for k in g}
    backward(less, o, lse, out=out)
    for key, end in (("dq", 1033), ("dk", 738), ("dv", 738)):
        assert torch.equal(out[key][:end], g[key][:end]) and (out[key][end:] == 5).all(), key


@pytest.mark.parametrize("size", [1e-3, 30.0])
def test_flat_and_peaked_rows(size):
    for t in ("bf16", "f32"):
        p = make([150, 40], 4, 2, 128, t, seed=5, size=size, scale=0.125)
        o, lse = forward(p)
        check_all(p, o, lse, backward(p, o, lse))


def test_gradient_by_differences():
    p = make([37], 2, 1, 64, "f32", seed=9)
    o, lse = forward(p)
    g = backward(p, o, lse)
    for name, key in (("dq", "q"), ("dk", "k"), ("dv", "v")):
        u = torch.randn(p[key].shape, generator=torch.Generator().manual_seed(1)).cuda()
        at, f = p[key], []
        for h in (1e-2, -1e-2):
            p[key] = at + h * u
            f.append(float((forward(p)[0].double() * p["do"].double()).sum()))
        p[key] = at
        want = float((g[name].double() * u.double()).sum())
        # fp32 differences of a sum of 4736 terms near 1: 2e-7 sqrt(4736) / 2e-2, and the third derivative 1e-4
        assert abs((f[0] - f[1]) / 2e-2 - want) < 3e-3 * (1 + abs(want)), name


@pytest.mark.parametrize("t,d", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 64)])
def test_bits_do_not_depend_on_the_batch(t, d):
    p = make([100, 33, 290, 1], 4, 2, d, t, seed=7)
    o, lse = forward(p)
    for rq, rk in spans(p):
        alone = dict(p, q=p["q"][rq], k=p["k"][rk], v=p["v"][rk], cu=cu_of([rq.stop - rq.start]).cuda())
        oa, la = forward(alone)
        assert torch.equal(oa, o[rq]) and torch.equal(la, lse[rq])


@pytest.mark.parametrize("t,d", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 64), ("f32", 256)])
def test_infinities_and_nan_stay_where_they_are_seen(t, d):
    lens = [70, 140, 90]
    p = make(lens, 4, 2, d, t, seed=11, extra=9)
    o, lse = forward(p)
    bad = dict(p)
    for key in ("q", "k", "v"):
        bad[key] = p[key].clone()
        bad[key][219 + 81:] = NAN  # behind the last sequence
    bad["v"][70 + 45, 0, 3] = NAN
    bad["v"][70 + 130, 1, 7] = INF
    bad["k"][219 + 40, 1] = NAN
    out = torch.full_like(p["q"].contiguous(), 7.0)
    o2, lse2 = forward(bad, out=out)
    assert (out[300:] == 7).all()
    same = torch.ones_like(o, dtype=torch.bool)
    same[70 + 45:210, :2, 3] = False   # rows that see the NaN, heads of its group, its element
    same[70 + 130:210, 2:, 7] = False
    same[219 + 40:, 2:] = False
    same[300:] = False
    assert torch.equal(o2[same], o[same])
    assert torch.isnan(o2[70 + 45:210, :2, 3]).all() and not torch.isfinite(o2[70 + 130:210, 2:, 7]).any()
    assert torch.isnan(o2[219 + 40:300, 2:]).all()
    assert torch.equal(lse2[:219 + 40], lse[:219 + 40])
    g, g2 = backward(p, o, lse), backward(bad, o2, lse2)
    for key in g:  # other sequences' gradients are untouched
        assert torch.equal(g[key][:70], g2[key][:70]), key


def test_rows_behind_the_last_sequence_are_left():
    p = make([20, 50], 4, 2, 128, "bf16", seed=13, extra=30)
    for key in ("q", "k", "v", "do"):
        p[key] = p[key].clone()
        p[key][70:] = NAN
    o, lse = forward(p, out=torch.full((100, 4, 128), 5.0, dtype=BF16, device="cuda"))
    out = {k: torch.full((100, h, 128), 5.0, dtype=BF16, device="cuda") for k, h in (("dq", 4), ("dk", 2), ("dv", 2))}
    g = backward(p, o, lse, out=out)
    assert all((x[70:] == 5).all() for x in (o, *g.values()))
    check_all(p, o, lse, g)


def test_rows_far_apart():
    """Offsets past 2^32 bytes."""
    T, ld = 600, 1 << 22
    p = make([T], 2, 1, 64, "bf16", seed=17)
    wide = torch.empty(T, ld, dtype=BF16, device="cuda")
    far = dict(p)
    for key, at, h in (("q", 0, 2), ("k", 1024, 1), ("v", ld - 64, 1), ("do", 4096, 2)):
        far[key] = wide[:, at:at + h * 64].unflatten(1, (h, 64))
        far[key].copy_(p[key])
    o, lse = forward(p)
    out = wide[:, 8192:8192 + 128].unflatten(1, (2, 64))
    o2, lse2 = forward(far, out=out)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    g = backward(p, o, lse)
    g2 = backward(far, out, lse2, out={"dk": wide[:, 9000:9064].unflatten(1, (1, 64))})
    assert all(torch.equal(g[k], g2[k]) for k in g)


def test_two_streams_and_a_graph():
    p = make([120, 300, 7], 8, 2, 128, "bf16", seed=19)
    ws = [torch.empty(B.attn_workspace_bytes(p["shape"], 427), dtype=torch.uint8, device="cuda") for _ in range(2)]

    def step(w):
        o, lse = forward(p)
        g = backward(p, o, lse, ws=w)
        return [o, lse, *[g[k] for k in sorted(g)]]
    want = step(ws[0])
    sides = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s, w in zip(sides, ws):  # side by side, each with a workspace of its own
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(step(w))
    for s in sides:
        torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for x in got for a, b in zip(x, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(ws[0])
    for k in range(4):
        p["q"].copy_(torch.randn(427, 8, 128, generator=torch.Generator().manual_seed(k)).cuda())
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        want = step(ws[1])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), k


def test_the_binding_refuses():
    p = make([5], 4, 2, 64, "bf16")
    with pytest.raises(ValueError, match="k: expected"):
        B.gdn_attn_prefill(p["shape"], p["q"], p["q"], p["v"], p["cu"])
    with pytest.raises(ValueError, match="cu_seqlens"):
        B.gdn_attn_prefill(p["shape"], p["q"], p["k"], p["v"], p["cu"].long())
    with pytest.raises(ValueError, match="cu_seqlens_k"):
        B.gdn_attn_prefill(p["shape"], p["q"], p["k"][:3], p["v"][:3], p["cu"])
    o, lse = forward(p)
    with pytest.raises(ValueError, match="lse"):
        B.gdn_attn_bwd(p["shape"], p["q"], p["k"], p["v"], p["cu"], o, lse.double(), p["do"])
    with pytest.raises(ValueError, match="out"):
        backward(p, o, lse, out={"dx": o})
    with pytest.raises(B.GdnError):
        backward(p, o, lse, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    c = B.KvCache(p["shape"], 2, 64, "cuda")
    with pytest.raises(ValueError, match="cache"):
        B.gdn_kv_write(B.make_attn_shape(4, 4, 64, BF16), p["q"], p["q"], c,
                       torch.zeros(1, 1, dtype=torch.int32, device="cuda"), cu_seqlens=p["cu"])
    with pytest.raises(ValueError, match="cu_seqlens"):
        B.gdn_kv_write(p["shape"], p["k"], p["v"], c, torch.zeros(1, 1, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="block_table"):
        B.gdn_kv_write(p["shape"], p["k"], p["v"], c, torch.zeros(1, 1, dtype=torch.int64, device="cuda"),
                       cu_seqlens=p["cu"])


# ---- the cache ------------------------------------------------------------------


class Pool:
    """A cache on the GPU with stale contents, and the oracle's copies of it."""

    def __init__(self, Hq, Hkv, d, t, P, lens, seed=0, spare=2, stale=True):
        self.gen = torch.Generator().manual_seed(seed)
        self.t, self.d, self.Hkv, self.Hq = t, d, Hkv, Hq
        self.shape = B.make_attn_shape(Hq, Hkv, d, DT[t])
        per = [-(-n // P) for n in lens]
        pages = sum(per) + spare
        self.cache = B.KvCache(self.shape, pages, P, "cuda")
        for x in (self.cache.k, self.cache.v):
            codes = torch.randint(0, 256, x.shape, generator=self.gen, dtype=torch.uint8)
            x.view(torch.uint8).copy_(codes if stale else torch.zeros_like(codes))
        self.cache.k_scale.fill_(0.25)
        self.cache.v_scale.fill_(2.0)
        ids = torch.randperm(pages, generator=self.gen)[:sum(per)].tolist()
        table = torch.full((len(lens), max(max(per), 1)), -1, dtype=torch.int32)
        for n, m in enumerate(per):
            for i in range(m):
                table[n, i] = ids.pop()
        self.table, self.dev_table = table.numpy(), table.cuda()
        c = self.cache
        self.k = A.OracleCache(c.k.view(torch.uint8).cpu().numpy(), c.k_scale.cpu().numpy())
        self.v = A.OracleCache(c.v.view(torch.uint8).cpu().numpy(), c.v_scale.cpu().numpy())

    def rows(self, n, size=1.0):
        return (size * torch.randn(n, self.Hkv, self.d, generator=self.gen)).to(DT[self.t]).cuda()

    def queries(self, n):
        return torch.randn(n, self.Hq, self.d, generator=self.gen).to(DT[self.t]).cuda()

    def write(self, k, v, lens, start, one=False):
        first = torch.tensor(start, dtype=torch.int32, device="cuda")
        B.gdn_kv_write(self.shape, k, v, self.cache, self.dev_table, cu_seqlens=None if one else cu_of(lens).cuda(),
                       start=first)
        at = 0
        for n, (m, s) in enumerate(zip(lens, start)):
            self.k.write(np64(k[at:at + m]), self.table[n], s)
            self.v.write(np64(v[at:at + m]), self.table[n], s)
            at += m

    def check(self):
        c = self.cache
        for x, s, o in ((c.k, c.k_scale, self.k), (c.v, c.v_scale, self.v)):
            got = x.view(torch.uint8).cpu().numpy()
            same = (got == o.codes) | (((got & 127) == 127) & ((o.codes & 127) == 127))
            assert same.all(), f"{(~same).sum()} codes of {same.size}"
            assert np.array_equal(s.cpu().numpy().astype(np.float64), o.scales)


@pytest.mark.parametrize("t,d,Hkv,P", [("bf16", 64, 3, 32), ("bf16", 128, 2, 64), ("bf16", 256, 1, 96),
                                       ("f32", 64, 1, 64), ("f32", 128, 3, 96), ("f32", 256, 2, 32)])
def test_cache_write_and_read(t, d, Hkv, P):
    """Prompts of all sorts of lengths, then tokens that end, open and straddle blocks, with larger and smaller values."""
    lens = [0, 1, 31, 32, 33, 95, 200]
    pool = Pool(2 * Hkv, Hkv, d, t, P, [n + 140 for n in lens], seed=d)
    pool.write(pool.rows(sum(lens)), pool.rows(sum(lens)), lens, [0] * 7)
    pool.check()
    at = list(lens)
    for k, new in enumerate(([1, 1, 1, 1, 1, 1, 1], [1, 1, 1, 1, 1, 1, 1], [0, 40, 2, 64, 7, 1, 0], [3, 1, 33, 0, 60, 5, 31])):
        size = [20.0, 0.01, 1.0, 300.0][k]
        x, y = pool.rows(sum(new), size), pool.rows(sum(new), 1 / size)
        pool.write(x, y, new, at, one=k < 2)
        pool.check()
        before = pool.cache.clone()
        pool.write(x, y, new, at, one=k < 2)  # the same again changes nothing
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in
                   zip(before.tensors(), pool.cache.tensors()))
        at = [a + b for a, b in zip(at, new)]
    start = [0, 5, 31, 32, 0, 60, 199]
    count = [a - b for a, b in zip(at, start)]
    kw = dict(start=torch.tensor(start, dtype=torch.int32, device="cuda"))
    k, v = B.gdn_kv_read(pool.shape, pool.cache, pool.dev_table, cu_of(count).cuda(), sum(count), **kw)
    row = 0
    for n in range(7):
        for got, o in ((k, pool.k), (v, pool.v)):
            want, there = o.read(pool.table[n], start[n], count[n])
            assert there.all()
            assert np.array_equal(np64(got[row:row + count[n]]), torch.from_numpy(want).to(DT[t]).double().numpy())
        row += count[n]
    one, _ = B.gdn_kv_read(pool.shape, pool.cache, pool.dev_table[1:], None, 6, start=kw["start"][1:])
    first = np.cumsum([0] + count)[1:7]
    assert torch.equal(one, k[torch.from_numpy(first).cuda()])


def test_cache_of_special_values():
    pool = Pool(2, 1, 64, "f32", 32, [32] * 9, seed=1)
    x = pool.rows(9 * 20)
    x[0:20] = 0
    x[20:40] *= 1e-38
    x[40:60] *= 1e37
    x[61] = 3.4e38
    x[80, 0, 3] = INF
    x[81, 0, 4] = -INF
    x[82, 0, 5] = NAN
    x[100:120] = NAN
    x[120:140] = INF
    x[140, 0, 0] = 448.0 * 2 ** 7
    x[160, 0, 0] = float(np.nextafter(np.float32(448.0), np.float32(500)))
    pool.write(x, -x, [20] * 9, [0] * 9)
    pool.check()
    pool.write(pool.rows(9 * 5, 1e-3), pool.rows(9 * 5, 1e3), [5] * 9, [20] * 9)  # NaN codes go over too
    pool.check()


def test_cache_rows_and_pages_that_are_not_there():
    """Bad ids in the table, places past its width, rows behind the last sequence, slices of wider rows."""
    pool = Pool(4, 2, 128, "bf16", 64, [200, 100, 150], seed=2)
    pool.table[0, 1], pool.table[1, 0], pool.table[2, 2] = -5, 1 << 30, pool.cache.pages
    pool.dev_table.copy_(torch.from_numpy(pool.table))
    wide = torch.full((430, 5 * 128), NAN, dtype=BF16, device="cuda")
    k, v = wide[:, :256].unflatten(1, (2, 128)), wide[:, 256:512].unflatten(1, (2, 128))
    lens = [190, 90, 120]
    k[:400], v[:400] = pool.rows(400), pool.rows(400)
    pool.write(k, v, lens, [0, 3, 140])  # the last ones end past the table's width
    pool.check()
    out = [torch.full((430, 2, 128), 9.0, dtype=BF16, device="cuda") for _ in range(2)]
    B.gdn_kv_read(pool.shape, pool.cache, pool.dev_table, cu_of(lens).cuda(), 430,
                  start=torch.tensor([0, 3, 140], dtype=torch.int32, device="cuda"), k_out=out[0], v_out=out[1])
    row = 0
    for n, (m, s) in enumerate(zip(lens, [0, 3, 140])):
        for got, o in zip(out, (pool.k, pool.v)):
            want, there = o.read(pool.table[n], s, m)
            want[~there] = 9.0
            assert np.array_equal(np64(got[row:row + m]), torch.from_numpy(want).bfloat16().double().numpy())
        row += m
    assert all((x[400:] == 9).all() for x in out)


# ---- attention over the cache ------------------------------------------------------


def decode_check(pool, q, lens_q, kv_len, o, lse, what=""):
    at = 0
    for n, (m, L) in enumerate(zip(lens_q, kv_len)):
        k, tk = pool.k.read(pool.table[n], 0, L)
        v, _ = pool.v.read(pool.table[n], 0, L)
        wo, wl, bo, bl = A.decode_fwd(np64(q[at:at + m]), k, v, tk, float(pool.shape.scale), UNIT[pool.t], L)
        check(o[at:at + m], wo, bo, f"{what} o of {n}")
        check(lse[at:at + m], wl, bl, f"{what} lse of {n}")
        at += m


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


DECODE = [
    # Hq, Hkv, d, type, page, cached tokens
    (1, 1, 64, "bf16", 32, [1, 2, 31, 32, 33, 64, 65]),
    (8, 2, 128, "bf16", 64, [5, 0, 511, 512, 513, 1500, 130]),
    (16, 2, 256, "bf16", 96, [1, 700, 1025]),
    (5, 1, 64, "bf16", 64, [300, 9000]),
    (40, 2, 128, "bf16", 32, [600, 3]),
    (96, 1, 64, "bf16", 64, [600, 31]),       # 96 rows a token
    (4, 2, 64, "f32", 32, [70, 1100]),
    (6, 2, 128, "f32", 256, [513, 40]),
    (8, 1, 256, "f32", 64, [33, 520]),
    (70, 1, 128, "f32", 64, [100, 530]),
]


@pytest.mark.parametrize("Hq,Hkv,d,t,P,lens", DECODE)
def test_decode(Hq, Hkv, d, t, P, lens):
    pool = Pool(Hq, Hkv, d, t, P, lens, seed=d + Hq)
    pool.write(pool.rows(sum(lens)), pool.rows(sum(lens)), lens, [0] * len(lens))
    q = pool.queries(len(lens))
    o, lse = B.gdn_attn_decode(pool.shape, q, pool.cache, pool.dev_table, i32(lens), max(lens), want_lse=True)
    decode_check(pool, q, [1] * len(lens), lens, o, lse)
    # the bits depend on neither the batch nor max_len
    o2 = B.gdn_attn_decode(pool.shape, q, pool.cache, pool.dev_table, i32(lens), 20 * max(lens))
    assert torch.equal(o, o2)
    for n in range(len(lens)):
        one = B.gdn_attn_decode(pool.shape, q[n:n + 1], pool.cache, pool.dev_table[n:n + 1], i32(lens[n:n + 1]), lens[n] + 1)
        assert torch.equal(one[0], o[n]), n
    # nor on whether the tokens come by cu_seqlens
    o3 = B.gdn_attn_decode(pool.shape, q, pool.cache, pool.dev_table, i32(lens), max(lens),
                           cu_seqlens=cu_of([1] * len(lens)).cuda())
    assert torch.equal(o, o3)


@pytest.mark.parametrize("Hq,Hkv,d,t,P", [(4, 2, 64, "bf16", 64), (8, 2, 128, "bf16", 32), (16, 1, 256, "bf16", 64),
                                          (3, 1, 64, "f32", 96), (4, 1, 128, "f32", 64), (4, 2, 256, "f32", 32)])
def test_several_tokens_a_sequence(Hq, Hkv, d, t, P):
    """Few rows and many, in one batch; rows that see nothing (more new tokens than cached ones)."""
    new, kv = [1, 0, 5, 70, 150, 20, 64], [40, 7, 1200, 1300, 150, 8, 2100]
    pool = Pool(Hq, Hkv, d, t, P, kv, seed=d)
    pool.write(pool.rows(sum(kv)), pool.rows(sum(kv)), kv, [0] * 7)
    q = pool.queries(sum(new))
    cu = cu_of(new).cuda()
    o, lse = B.gdn_attn_decode(pool.shape, q, pool.cache, pool.dev_table, i32(kv), max(kv), cu_seqlens=cu, want_lse=True)
    decode_check(pool, q, new, kv, o, lse)
    row = 0
    for n, m in enumerate(new):  # the bits do not depend on the batch
        if m:
            one = B.gdn_attn_decode(pool.shape, q[row:row + m], pool.cache, pool.dev_table[n:n + 1], i32(kv[n:n + 1]),
                                    5000, cu_seqlens=cu_of([m]).cuda())
            assert torch.equal(one, o[row:row + m]), n
        row += m


@pytest.mark.parametrize("d,t,new", [(64, "bf16", 3), (128, "bf16", 3), (256, "f32", 2), (128, "bf16", 100),
                                     (64, "f32", 90), (256, "bf16", 64)])
def test_what_a_row_must_not_see(d, t, new):
    """NaN behind the last token (stale codes), in a later new token, in blocks without a page, and past max_len."""
    kv = [200, 333, 120]
    pool = Pool(4, 2, d, t, 32, kv, seed=4)
    pool.write(pool.rows(sum(kv)), pool.rows(sum(kv)), kv, [0] * 3)
    last = pool.rows(1)
    last[0, 1, 5] = NAN
    pool.write(pool.rows(1), last, [0, 1, 0], [0, 332, 0])  # the newest token's value
    pool.table[2, 1] = -1
    pool.dev_table.copy_(torch.from_numpy(pool.table))
    lens = [new] * 3
    q = pool.queries(3 * new)
    cu = cu_of(lens).cuda()
    o, lse = B.gdn_attn_decode(pool.shape, q, pool.cache, pool.dev_table, i32(kv), 400, cu_seqlens=cu, want_lse=True)
    hit = o[2 * new - 1, 2:, 5].clone()
    assert torch.isnan(hit).all()
    o[2 * new - 1, 2:, 5] = 0
    fixed = pool.v.codes.copy()
    pool.v.codes[(pool.v.codes & 127) == 127] = 0
    w = 0
    for n in range(3):
        k, there = pool.k.read(pool.table[n], 0, kv[n])
        v, _ = pool.v.read(pool.table[n], 0, kv[n])
        wo, wl, bo, bl = A.decode_fwd(np64(q[w:w + new]), k, v, there, float(pool.shape.scale), UNIT[t], kv[n])
        if n == 1:
            wo[new - 1, 2:, 5] = 0
        check(o[w:w + new], wo, bo, f"o of {n}")
        check(lse[w:w + new], wl, bl, f"lse of {n}")
        w += new
    pool.v.codes = fixed
    short = B.gdn_attn_decode(pool.shape, q, pool.cache, pool.dev_table, i32(kv), 100, cu_seqlens=cu)
    assert torch.isfinite(short).all()  # tokens past max_len are not seen


def test_no_tokens_and_no_pages():
    pool = Pool(4, 2, 64, "bf16", 64, [64, 64], seed=6)
    q = pool.queries(2)
    o, lse = B.gdn_attn_decode(pool.shape, q, pool.cache, pool.dev_table, i32([0, -3]), 64, want_lse=True)
    assert not o.any() and torch.isneginf(lse).all()
    none = torch.full((2, 1), -1, dtype=torch.int32, device="cuda")
    for cu, n in ((None, 2), (cu_of([40, 60]).cuda(), 100)):
        q = pool.queries(n)
        o, lse = B.gdn_attn_decode(pool.shape, q, pool.cache, none, i32([64, 60]), 700, cu_seqlens=cu, want_lse=True)
        assert not o.any() and torch.isneginf(lse).all()
    empty = torch.zeros(2, 0, dtype=torch.int32, device="cuda")
    o = B.gdn_attn_decode(pool.shape, pool.queries(2), pool.cache, empty, i32([5, 5]), 64)
    assert not o.any()


def test_a_pool_past_4_gb():
    shape = B.make_attn_shape(8, 8, 256, BF16)
    cache = B.KvCache(shape, 9000, 256, "cuda")  # 4.7 GB each of keys and values
    gen = torch.Generator().manual_seed(0)
    small = B.KvCache(shape, 4, 256, "cuda")
    far, near = i32([[8999, 8191, 8998]]), i32([[2, 0, 3]])
    k, v = (torch.randn(700, 8, 256, generator=gen).bfloat16().cuda() for _ in range(2))
    cu, q = cu_of([700]).cuda(), torch.randn(101, 8, 256, generator=gen).bfloat16().cuda()
    out = []
    for c, table in ((cache, far), (small, near)):
        B.gdn_kv_write(shape, k, v, c, table, cu_seqlens=cu)
        out.append([*B.gdn_kv_read(shape, c, table, cu, 700),
                    B.gdn_attn_decode(shape, q[:1], c, table, i32([700]), 768),
                    B.gdn_attn_decode(shape, q, c, table, i32([700]), 768, cu_seqlens=cu_of([101]).cuda())])
    assert all(torch.equal(a, b) for a, b in zip(*out))
    del cache


def test_a_long_cache():
    """Splits past sixteen: joined in groups."""
    L = 20000
    pool = Pool(8, 1, 128, "bf16", 256, [L, 300], seed=8)
    pool.write(pool.rows(L + 300), pool.rows(L + 300), [L, 300], [0, 0])
    q = pool.queries(2)
    o, lse = B.gdn_attn_decode(pool.shape, q, pool.cache, pool.dev_table, i32([L, 300]), L, want_lse=True)
    decode_check(pool, q, [1, 1], [L, 300], o, lse)
    short = B.gdn_attn_decode(pool.shape, q[1:], pool.cache, pool.dev_table[1:], i32([300]), 300)
    assert torch.equal(short[0], o[1])
    mid = [B.gdn_attn_decode(pool.shape, q[:1], pool.cache, pool.dev_table[:1], i32([8000]), m) for m in (8000, L)]
    assert torch.equal(*mid)  # joined one way and the other


@pytest.mark.parametrize("Hq,Hkv,d,t", [(2, 1, 64, "bf16"), (4, 1, 128, "f32"), (33, 1, 64, "bf16"), (32, 1, 64, "f32")])
def test_lengths_around_a_split(Hq, Hkv, d, t):
    """One token over lengths at and beside the ends of splits, and where splits grow."""
    lens = [511, 512, 513, 4095, 4096, 4097, 5121, 1]
    pool = Pool(Hq, Hkv, d, t, 128, lens, seed=5)
    pool.write(pool.rows(sum(lens)), pool.rows(sum(lens)), lens, [0] * len(lens))
    q = pool.queries(len(lens))
    o, lse = B.gdn_attn_decode(pool.shape, q, pool.cache, pool.dev_table, i32(lens), max(lens), want_lse=True)
    decode_check(pool, q, [1] * len(lens), lens, o, lse)
    for n in range(len(lens)):
        one = B.gdn_attn_decode(pool.shape, q[n:n + 1], pool.cache, pool.dev_table[n:n + 1], i32(lens[n:n + 1]), lens[n])
        assert torch.equal(one[0], o[n]), n
    o2 = B.gdn_attn_decode(pool.shape, q, pool.cache, pool.dev_table, i32(lens), 2 * max(lens),
                           cu_seqlens=cu_of([1] * len(lens)).cuda())
    assert torch.equal(o, o2)


@pytest.mark.parametrize("G,d,t", [(1, 64, "bf16"), (4, 128, "bf16"), (8, 256, "f32")])
def test_rows_around_a_kernels_limit(G, d, t):
    """31, 32, 33, 128, 256 and 264 rows a sequence over caches of several splits."""
    new = [max(1, r // G) for r in (31, 32, 33, 128, 256, 264)]
    lens = [1300 + 7 * n for n in new]
    pool = Pool(G, 1, d, t, 64, lens, seed=6)
    pool.write(pool.rows(sum(lens)), pool.rows(sum(lens)), lens, [0] * len(lens))
    q, cu = pool.queries(sum(new)), cu_of(new).cuda()
    o, lse = B.gdn_attn_decode(pool.shape, q, pool.cache, pool.dev_table, i32(lens), max(lens), cu_seqlens=cu, want_lse=True)
    decode_check(pool, q, new, lens, o, lse)
    at = 0
    for n, r in enumerate(new):
        one = B.gdn_attn_decode(pool.shape, q[at:at + r], pool.cache, pool.dev_table[n:n + 1], i32(lens[n:n + 1]), lens[n] + 600,
                                cu_seqlens=cu_of([r]).cuda())
        assert torch.equal(one, o[at:at + r]), n
        at += r


def test_decode_captured_in_a_graph():
    """Write and attend in one graph; the lengths grow between replays."""
    lens = [600, 33, 1, 1000]
    pool = Pool(8, 2, 128, "bf16", 64, [n + 50 for n in lens], seed=10)
    pool.write(pool.rows(sum(lens)), pool.rows(sum(lens)), lens, [0] * 4)
    k, v, q = pool.rows(4), pool.rows(4), pool.queries(4)
    start, kv = i32(lens), i32([n + 1 for n in lens])
    ws = torch.empty(B.attn_decode_workspace_bytes(pool.shape, 4, 4, 2000), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)

    def step():
        B.gdn_kv_write(pool.shape, k, v, pool.cache, pool.dev_table, start=start)
        B.gdn_attn_decode(pool.shape, q, pool.cache, pool.dev_table, kv, 2000, out=out, ws=ws)
    before = pool.cache.clone()
    step()
    for a, b in zip(pool.cache.tensors(), before.tensors()):
        a.view(torch.uint8).copy_(b.view(torch.uint8))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    at = list(lens)
    for r in range(5):
        k.copy_(pool.rows(4))
        v.copy_(pool.rows(4))
        q.copy_(pool.queries(4))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n in range(4):
            pool.k.write(np64(k[n:n + 1]), pool.table[n], at[n])
            pool.v.write(np64(v[n:n + 1]), pool.table[n], at[n])
        at = [a + 1 for a in at]
        pool.check()
        got = out.clone()
        want, lse = B.gdn_attn_decode(pool.shape, q, pool.cache, pool.dev_table, kv, 2000, want_lse=True)
        assert torch.equal(got, want), r
        decode_check(pool, q, [1] * 4, at, want, lse, f"replay {r}")
        start.add_(1)
        kv.add_(1)


# ---- together ------------------------------------------------------------------------


def test_a_layer_from_prompt_to_decode():
    """q and k normalised and rotated, attention over the prompt, the prompt into the cache, then tokens one at a time
    and a few at once, against the formulas."""
    Hq, Hkv, d, r = 8, 2, 128, 32
    lens, steps = [70, 1, 33], [1, 1, 4, 1]
    total = [n + sum(steps) for n in lens]
    pool = Pool(Hq, Hkv, d, "bf16", 32, total, seed=12)
    gen = torch.Generator().manual_seed(5)
    qk = B.make_qk_shape(Hq, Hkv, d, r, BF16, norm="rms", weight_offset=1.0)
    freq, _ = B.rope_freqs(r)
    w_q, w_k = 0.2 * torch.randn(d, generator=gen), 0.2 * torch.randn(d, generator=gen)
    kw = dict(w_q=w_q.cuda(), w_k=w_k.cuda())

    def project(n):
        row = torch.randn(n, (Hq + 2 * Hkv) * d, generator=gen).bfloat16().cuda()
        return [x.unflatten(1, (-1, d)) for x in row.split([Hq * d, Hkv * d, Hkv * d], 1)]

    def rotated(q, k, lens, start):
        qo, ko = B.gdn_qk_rotary(qk, q, k, freq.cuda(), cu_seqlens=cu_of(lens).cuda(), start=i32(start), **kw)
        pos = np.concatenate([np.arange(n) + s for n, s in zip(lens, start)])
        for x, y, w in ((q, qo, w_q), (k, ko, w_k)):
            want, bound = qk_fwd(np64(x), norm="rms", layout="half", r=r, eps=float(qk.eps), rope_scale=1.0, pos=pos,
                                 inv_freq=freq.double().numpy(), w=1.0 + w.double().numpy(), scale=1.0)
            check(y, want, bound, "rotated")
        return qo, ko
    q, k, v = project(sum(lens))
    q, k = rotated(q, k, lens, [0] * 3)
    p = dict(shape=pool.shape, q=q, k=k, v=v, cu=cu_of(lens).cuda(), cu_k=None, lens=lens, lens_k=lens, t="bf16",
             scale=float(pool.shape.scale))
    o, lse = forward(p)
    check_all(p, o, lse)
    pool.write(k, v, lens, [0] * 3)
    at = list(lens)
    for m in steps:
        new = [m] * 3
        q, k, v = project(3 * m)
        q, k = rotated(q, k, new, at)
        pool.write(k, v, new, at, one=m == 1)
        at = [a + m for a in at]
        cu = {} if m == 1 else dict(cu_seqlens=cu_of(new).cuda())
        o, lse = B.gdn_attn_decode(pool.shape, q, pool.cache, pool.dev_table, i32(at), max(total), want_lse=True, **cu)
        decode_check(pool, q, new, at, o, lse, f"at {at}")
    pool.check()
    k, v = B.gdn_kv_read(pool.shape, pool.cache, pool.dev_table, cu_of(at).cuda(), sum(at))
    p = dict(shape=pool.shape, q=q, k=k, v=v, cu=cu_of([steps[-1]] * 3).cuda(), cu_k=cu_of(at).cuda(),
             lens=[steps[-1]] * 3, lens_k=at, t="bf16", scale=p["scale"])
    o2, lse2 = forward(p)  # attention of the last tokens over what the cache gives back
    check_all(p, o2, lse2)


def test_a_layers_gradient():
    """q/k norms and rotation, attention, and both gradients, against the formulas in one go."""
    Hq, Hkv, d, lens = 4, 2, 64, [50, 9]
    gen = torch.Generator().manual_seed(6)
    T = sum(lens)
    q, k, v, do = (torch.randn(T, h, d, generator=gen).cuda() for h in (Hq, Hkv, Hkv, Hq))
    qk = B.make_qk_shape(Hq, Hkv, d, d, F32, norm="l2")
    freq, _ = B.rope_freqs(d)
    cu = cu_of(lens).cuda()
    s = B.make_attn_shape(Hq, Hkv, d, F32, scale=3.0)
    qo, ko = B.gdn_qk_rotary(qk, q, k, freq.cuda(), cu_seqlens=cu)
    o, lse = B.gdn_attn_prefill(s, qo, ko, v, cu)
    g = B.gdn_attn_bwd(s, qo, ko, v, cu, o, lse, do)
    h = B.gdn_qk_rotary_bwd(qk, q, k, g["dq"], g["dk"], freq.cuda(), cu_seqlens=cu)
    pos = np.concatenate([np.arange(n) for n in lens])
    c = dict(norm="l2", layout="half", r=d, eps=float(qk.eps), rope_scale=1.0, pos=pos, inv_freq=freq.double().numpy(),
             w=None, scale=1.0)
    (wq, bq), (wk, bk) = qk_fwd(np64(q), **c), qk_fwd(np64(k), **c)
    at = 0
    dq, dk, dv = (np.zeros_like(np64(x)) for x in (q, k, v))
    for n in lens:
        r = slice(at, at + n)
        w = A.attn_bwd(wq[r], wk[r], np64(v[r]), np64(do[r]), float(s.scale), UNIT["f32"], 0.0)
        dq[r], dk[r], dv[r] = w["dq"][0], w["dk"][0], w["dv"][0]
        at += n
    for got, x, dy in ((h["dq"], q, dq), (h["dk"], k, dk)):
        want = qk_bwd(np64(x), dy, **c)[0]
        # within 2^-16 of the gradient's size: some 2^-20 of each step through sums of up to 50 terms
        assert np.abs(np64(got) - want).max() < 2.0 ** -16 * np.abs(want).max()
    assert np.abs(np64(g["dv"]) - dv).max() < 2.0 ** -16 * np.abs(dv).max()
