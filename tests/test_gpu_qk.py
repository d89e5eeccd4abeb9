"""The q/k norms with rotary positions on the GPU against the fp64 oracle, and
together with the layers that take them."""

import numpy as np
import pytest
import torch

from gdn_helpers import bit_equal, make_inputs, to_dev
from linear_attention_rnn_gated_amd import binding as B
from oracle.qk_oracle import qk_bwd, qk_fwd

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
DT = {"f32": F32, "bf16": BF16}


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def check(got, want, bound, what):
    half = torch.finfo(got.dtype).eps / 2
    tol = bound + half * (np.abs(want) + bound) + 2.0 ** -126
    off = np.abs(np64(got) - want)
    bad = ~(off <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.nanmax(off / tol):.3g} of the bound"


def make(T, Hq, Hk, d, r, inp="bf16", out=None, norm="rms", layout="half", seed=0, far=100000, offset=1.0, scale=0.25,
         rope_scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    out = out or inp
    p = dict(q=rn(T, Hq, d).to(DT[inp]), k=rn(T, Hk, d).to(DT[inp]), w_q=None, w_k=None,
             pos=torch.randint(0, far + 1, (T,), generator=gen, dtype=torch.int32),
             inv_freq=(10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / max(r, 1))).float(),
             dq=rn(T, Hq, d).to(DT[out]), dk=rn(T, Hk, d).to(DT[out]))
    if norm == "rms":
        p["w_q"], p["w_k"] = 0.2 * rn(d), 0.2 * rn(d)
    p["shape"] = B.make_qk_shape(Hq, Hk, d, r, DT[inp], out_dtype=DT[out], norm=norm, layout=layout, scale=scale,
                                 rope_scale=rope_scale, weight_offset=offset)
    p["kw"] = dict(norm=norm, layout=layout, r=r, eps=float(p["shape"].eps), rope_scale=float(p["shape"].rope_scale))
    p["offset"] = offset
    return p


def on_gpu(p):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in p.items()}


def factor(p, name):
    return None if p["w_" + name] is None else p["offset"] + np64(p["w_" + name])


def oracle(p, name, pos=None):
    scale = float(p["shape"].scale) if name == "q" else 1.0
    return qk_fwd(np64(p[name]), pos=np64(p["pos"]) if pos is None else pos, inv_freq=np64(p["inv_freq"]),
                  w=factor(p, name), scale=scale, **p["kw"])


CASES = [
    # T, Hq, Hk, d, r, in, out, norm, layout
    (1, 1, 1, 8, 8, "f32", "f32", "l2", "half"),
    (3, 2, 1, 16, 8, "bf16", "f32", "rms", "interleaved"),
    (5, 3, 0, 64, 64, "bf16", "bf16", "l2", "half"),
    (33, 16, 16, 128, 128, "bf16", "bf16", "rms", "half"),
    (70, 16, 2, 128, 64, "f32", "bf16", "rms", "interleaved"),
    (9, 5, 3, 80, 40, "bf16", "bf16", "none", "half"),
    (17, 7, 1, 96, 24, "f32", "f32", "rms", "half"),
    (12, 3, 2, 192, 192, "bf16", "bf16", "l2", "interleaved"),
    (40, 32, 8, 256, 64, "bf16", "bf16", "rms", "half"),
    (6, 2, 2, 512, 512, "f32", "f32", "rms", "half"),
    (4, 1, 2, 504, 16, "bf16", "f32", "rms", "interleaved"),
    (11, 4, 4, 128, 0, "bf16", "bf16", "rms", "half"),
    (300, 40, 8, 64, 32, "bf16", "bf16", "none", "interleaved"),
    (2, 4000, 96, 8, 8, "bf16", "bf16", "rms", "half"),
    (3, 65, 1, 24, 8, "f32", "f32", "l2", "interleaved"),
    (2100, 1, 1, 512, 256, "bf16", "bf16", "rms", "interleaved"),
]


@pytest.mark.parametrize("T,Hq,Hk,d,r,inp,out,norm,layout", CASES)
def test_forward_and_gradient(T, Hq, Hk, d, r, inp, out, norm, layout):
    p = make(T, Hq, Hk, d, r, inp, out, norm, layout, seed=d + T, rope_scale=1.25 if r == 64 else 1.0)
    g = on_gpu(p)
    freq = g["inv_freq"] if r else None
    qo, ko = B.gdn_qk_rotary(p["shape"], g["q"], g["k"], freq, pos=g["pos"], w_q=g["w_q"], w_k=g["w_k"])
    assert qo.dtype == DT[out] and ko.shape == (T, Hk, d)
    got = B.gdn_qk_rotary_bwd(p["shape"], g["q"], g["k"], g["dq"], g["dk"], freq, pos=g["pos"], w_q=g["w_q"], w_k=g["w_k"])
    again = B.gdn_qk_rotary_bwd(p["shape"], g["q"], g["k"], g["dq"], g["dk"], freq, pos=g["pos"], w_q=g["w_q"],
                                w_k=g["w_k"])
    assert all(torch.equal(got[k], again[k]) for k in got)
    for name, y, H in (("q", qo, Hq), ("k", ko, Hk)):
        if H == 0:
            continue
        want, bound = oracle(p, name)
        check(y, want, bound, name)
        scale = float(p["shape"].scale) if name == "q" else 1.0
        dx, dw, bx, mag = qk_bwd(np64(p[name]), np64(p["d" + name]), pos=np64(p["pos"]), inv_freq=np64(p["inv_freq"]),
                                 w=factor(p, name), scale=scale, **p["kw"])
        assert got["d" + name].dtype == DT[inp]
        check(got["d" + name], dx, bx, "d" + name)
        if norm == "rms":
            # every term passes at most T H + 16 + 1024 additions and its own roundings (8 C)
            check(got["dw_" + name], dw, mag * (8 * 2.0 ** -20 + (T * H + 1040) * 2.0 ** -24), "dw_" + name)


def test_gradient_by_differences():
    p = make(7, 3, 2, 32, 16, "f32", norm="rms", seed=3)
    g = on_gpu(p)
    r = B.gdn_qk_rotary_bwd(p["shape"], g["q"], g["k"], g["dq"], g["dk"], g["inv_freq"], pos=g["pos"], w_q=g["w_q"],
                            w_k=g["w_k"])
    rng = np.random.default_rng(2)
    for name in ("q", "k"):
        scale = float(p["shape"].scale) if name == "q" else 1.0
        f = lambda x, w: (qk_fwd(x, pos=np64(p["pos"]), inv_freq=np64(p["inv_freq"]), w=w, scale=scale,  # noqa: E731
                                 **p["kw"])[0] * np64(p["d" + name])).sum()
        x, w = np64(p[name]), factor(p, name)
        v, u = rng.normal(size=x.shape), rng.normal(size=w.shape)
        want = (f(x + 1e-6 * v, w) - f(x - 1e-6 * v, w)) / 2e-6
        size = np.abs(np64(r["d" + name]) * v).sum()
        assert abs((np64(r["d" + name]) * v).sum() - want) <= 1e-5 * size + 1e-6
        want = (f(x, w + 1e-6 * u) - f(x, w - 1e-6 * u)) / 2e-6
        assert abs((np64(r["dw_" + name]) * u).sum() - want) <= 1e-5 * np.abs(np64(r["dw_" + name]) * u).sum() + 1e-6


def test_far_positions():
    """Positions to 2^31 - 1: the fp64 angle is off by at most 2^31 2^-53 turns, so fp32's bound holds as it is."""
    p = make(64, 2, 1, 64, 64, "f32", norm="none", seed=5, far=(1 << 31) - 2)
    p["pos"][0], p["pos"][1], p["pos"][2] = (1 << 31) - 1, 0, -7
    g = on_gpu(p)
    qo, ko = B.gdn_qk_rotary(p["shape"], g["q"], g["k"], g["inv_freq"], pos=g["pos"])
    check(qo, *oracle(p, "q"), "q")
    check(ko, *oracle(p, "k"), "k")


def test_positions_from_sequences_and_rows_behind():
    lens, start = [3, 0, 40, 1, 0], [7, 9, 100000, 0, 5]
    T, pad = sum(lens), 6
    p = make(T + pad, 4, 2, 128, 64, seed=6)
    pos = np.concatenate([np.arange(n) + s for n, s in zip(lens, start)])
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")
    g = on_gpu(p)
    st = torch.tensor(start, dtype=torch.int32, device="cuda")
    full = torch.tensor(list(pos) + [0] * pad, dtype=torch.int32, device="cuda")
    want = B.gdn_qk_rotary(p["shape"], g["q"], g["k"], g["inv_freq"], pos=full, w_q=g["w_q"], w_k=g["w_k"])
    qo, ko = torch.full_like(g["q"], 9.0), torch.full_like(g["k"], 9.0)
    B.gdn_qk_rotary(p["shape"], g["q"], g["k"], g["inv_freq"], cu_seqlens=cu, start=st, w_q=g["w_q"], w_k=g["w_k"],
                    q_out=qo, k_out=ko)
    assert torch.equal(qo[:T], want[0][:T]) and torch.equal(ko[:T], want[1][:T])
    assert bool((qo[T:] == 9).all()) and bool((ko[T:] == 9).all())
    plain, _ = B.gdn_qk_rotary(p["shape"], g["q"], g["k"], g["inv_freq"], cu_seqlens=cu, w_q=g["w_q"], w_k=g["w_k"])
    first = oracle(dict(p, q=p["q"][:T]), "q", np.concatenate([np.arange(n) for n in lens]))
    check(plain[:T], *first, "q")
    # the gradient leaves the rows behind out of the weights' sums too
    g["dq"][T:], g["q"][T:] = float("nan"), float("nan")
    r = B.gdn_qk_rotary_bwd(p["shape"], g["q"], g["k"], g["dq"], g["dk"], g["inv_freq"], cu_seqlens=cu, start=st,
                            w_q=g["w_q"], w_k=g["w_k"])
    assert bool(r["dw_q"].isfinite().all()) and bool(r["dq"][:T].isfinite().all())


def test_slices_in_place_and_other_channels():
    """q and k as slices of one projection, turned in place; nan in the part that is not rotated stays there."""
    p = make(50, 4, 2, 64, 32, norm="none", seed=7)
    g = on_gpu(p)
    g["q"][3, 1, 40], g["q"][4, 0, 63] = float("nan"), float("inf")
    want = B.gdn_qk_rotary(p["shape"], g["q"], g["k"], g["inv_freq"], pos=g["pos"])
    row = torch.full((50, 4 * 64 + 2 * 64 + 128), 3.0, dtype=BF16, device="cuda")
    row[:, :256], row[:, 256:384] = g["q"].flatten(1), g["k"].flatten(1)
    q, k = row[:, :256].unflatten(1, (4, 64)), row[:, 256:384].unflatten(1, (2, 64))
    B.gdn_qk_rotary(p["shape"], q, k, g["inv_freq"], pos=g["pos"], q_out=q, k_out=k)
    same = lambda a, b: torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))  # noqa: E731
    assert same(q, want[0]) and same(k, want[1]) and bool((row[:, 384:] == 3).all())
    assert bool(want[0][3, 1, :40].isfinite().all()) and int(want[0].isnan().sum()) == 1 and int(want[0].isinf().sum()) == 1


def test_offsets_past_32_bits():
    p = make(1300, 2, 2, 64, 64, seed=8)
    g = on_gpu(p)
    want = B.gdn_qk_rotary(p["shape"], g["q"], g["k"], g["inv_freq"], pos=g["pos"], w_q=g["w_q"], w_k=g["w_k"])
    big = torch.empty(1300, 1 << 21, dtype=BF16, device="cuda")
    q, k = big[:, :128].unflatten(1, (2, 64)), big[:, -128:].unflatten(1, (2, 64))
    q.copy_(g["q"])
    k.copy_(g["k"])
    B.gdn_qk_rotary(p["shape"], q, k, g["inv_freq"], pos=g["pos"], w_q=g["w_q"], w_k=g["w_k"], q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_zero_vectors_and_no_weights():
    p = make(4, 2, 1, 64, 32, "f32", norm="rms", seed=9)
    g = on_gpu(p)
    g["q"][1] = 0
    qo, _ = B.gdn_qk_rotary(p["shape"], g["q"], g["k"], g["inv_freq"], pos=g["pos"], w_q=g["w_q"], w_k=g["w_k"])
    assert bool((qo[1] == 0).all())
    r = B.gdn_qk_rotary_bwd(p["shape"], g["q"], g["k"], g["dq"], g["dk"], g["inv_freq"], pos=g["pos"], w_q=g["w_q"],
                            w_k=g["w_k"])
    assert bool(r["dq"].isfinite().all())
    a, _ = B.gdn_qk_rotary(p["shape"], g["q"], g["k"], g["inv_freq"], pos=g["pos"])
    b, _ = B.gdn_qk_rotary(p["shape"], g["q"], g["k"], g["inv_freq"], pos=g["pos"], w_q=torch.zeros_like(g["w_q"]),
                           w_k=torch.zeros_like(g["w_k"]))
    assert torch.equal(a, b)
    none = B.gdn_qk_rotary_bwd(p["shape"], g["q"][:0], g["k"][:0], g["dq"][:0], g["dk"][:0], g["inv_freq"],
                               pos=g["pos"][:0], w_q=g["w_q"], w_k=g["w_k"])
    assert bool((none["dw_q"] == 0).all()) and none["dq"].shape == (0, 2, 64)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("d", [8, 96, 128])
def test_weight_gradients_keep_q_and_k_apart(d, bad):
    """A NaN or an infinity in a head of q reaches dw_q and that head alone, and eps = 0 with more places in a wave than
    there are heads reaches nothing."""
    p = make(5, 2, 1, d, 8, "f32", seed=9)
    p["shape"] = B.make_qk_shape(2, 1, d, 8, F32, norm="rms", eps=0.0, weight_offset=p["offset"])
    g = on_gpu(p)
    args = (p["shape"], g["q"], g["k"], g["dq"], g["dk"], g["inv_freq"])
    kw = dict(pos=g["pos"], w_q=g["w_q"], w_k=g["w_k"])
    clean = B.gdn_qk_rotary_bwd(*args, **kw)
    assert all(torch.isfinite(t).all() for t in clean.values())
    for name, other in (("q", "k"), ("k", "q")):
        keep = g[name].clone()
        g[name][2, 0, 3] = bad
        got = B.gdn_qk_rotary_bwd(*args, **kw)
        g[name].copy_(keep)
        assert torch.equal(got["dw_" + other], clean["dw_" + other])
        assert torch.equal(got["d" + other], clean["d" + other])
        assert not torch.isfinite(got["d" + name][2, 0]).all() and not torch.isfinite(got["dw_" + name]).all()
        rest = torch.ones(5, g[name].shape[1], dtype=torch.bool, device="cuda")
        rest[2, 0] = False
        assert torch.equal(got["d" + name][rest], clean["d" + name][rest])


def test_captured_in_a_graph_and_on_a_stream():
    p = make(300, 8, 2, 128, 128, seed=10)
    g = on_gpu(p)
    ws = torch.empty(B.qk_workspace_bytes(p["shape"], 300), dtype=torch.uint8, device="cuda")

    def step():
        y = B.gdn_qk_rotary(p["shape"], g["q"], g["k"], g["inv_freq"], pos=g["pos"], w_q=g["w_q"], w_k=g["w_k"])
        r = B.gdn_qk_rotary_bwd(p["shape"], g["q"], g["k"], g["dq"], g["dk"], g["inv_freq"], pos=g["pos"],
                                w_q=g["w_q"], w_k=g["w_k"], ws=ws)
        return [*y, *[r[k] for k in sorted(r)]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(other, step()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for k in range(4):
        g["q"].copy_(torch.randn(300, 8, 128, generator=torch.Generator().manual_seed(k)).cuda())
        g["pos"].add_(1)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), k


def test_equals_the_layers_own_norm():
    """Norm "l2" without a rotation, in fp32: gdn_prefill's own normalisation, bit for bit."""
    inp = make_inputs([70, 40], 2, 4, 128, "f32", seed=11)
    d = to_dev(inp)
    own = B.make_shape(2, 4, 128, 64, F32, qk_l2norm=True, scale=0.5)
    given = B.make_shape(2, 4, 128, 64, F32, qk_l2norm=False, scale=1.0)
    a, ha = B.gdn_prefill(own, d["q"], d["k"], d["v"], d["beta"], d["g"], d["cu_seqlens"])
    s = B.make_qk_shape(2, 2, 128, 0, F32, norm="l2", scale=0.5)
    q, k = B.gdn_qk_rotary(s, d["q"], d["k"], None, cu_seqlens=d["cu_seqlens"])
    b, hb = B.gdn_prefill(given, q, k, d["v"], d["beta"], d["g"], d["cu_seqlens"])
    assert bit_equal(a, b) and bit_equal(ha, hb)


def test_block_prefill_then_decode():
    """A block as a model runs it: v through the gated linear recurrence, q and k normed and rotated, the gated delta
    rule on them.  Prefill of a prompt and token-by-token decode give one long prefill's bits."""
    lens, new, Hq, Hv, d = [40, 75], 60, 2, 4, 128
    total = [n + new for n in lens]
    inp = to_dev(make_inputs(total, Hq, Hv, d, "bf16", seed=12))
    T, N, D = sum(total), 2, Hv * d
    lg = (-torch.rand(T, D, generator=torch.Generator().manual_seed(1))).cuda()
    freq, rope_scale = B.rope_freqs(64, kind="yarn", factor=4.0, orig_len=4096.0)
    freq = freq.cuda()
    qk = B.make_qk_shape(Hq, Hq, d, 64, BF16, norm="l2", rope_scale=rope_scale)
    lru = B.make_lru_shape(D, BF16, F32, "norm")
    gdn = B.make_shape(Hq, Hv, d, 64, BF16, qk_l2norm=False)

    def prefill(rows, cu, lru_cache=None, gdn_cache=None):
        v, _ = B.gdn_lru_prefill(lru, inp["v"][rows].flatten(1), lg[rows], cu, cache=lru_cache)
        q, k = B.gdn_qk_rotary(qk, inp["q"][rows], inp["k"][rows], freq, cu_seqlens=cu)
        return B.gdn_prefill(gdn, q, k, v.view(-1, Hv, d), inp["beta"][rows].contiguous(), inp["g"][rows].contiguous(), cu,
                             cache=gdn_cache)[0]
    cut = lambda ns: torch.tensor([0] + list(np.cumsum(ns)), dtype=torch.int32, device="cuda")  # noqa: E731
    want = prefill(torch.arange(T, device="cuda"), cut(total))
    first = [0, total[0]]
    rows = torch.cat([torch.arange(first[n], first[n] + lens[n]) for n in range(N)]).cuda()
    lc, gc = B.LruCache(D, N, "cuda"), B.Cache(gdn, N, "cuda", BF16)
    assert bit_equal(prefill(rows, cut(lens), lc, gc), want[rows])
    for t in range(new):
        at = torch.tensor([first[n] + lens[n] + t for n in range(N)], device="cuda")
        pos = torch.tensor([lens[n] + t for n in range(N)], dtype=torch.int32, device="cuda")
        v = B.gdn_lru_decode_step(lru, inp["v"][at].flatten(1), lg[at], lc)
        q, k = B.gdn_qk_rotary(qk, inp["q"][at], inp["k"][at], freq, pos=pos)
        o = B.gdn_decode_step(gdn, q, k, v.view(N, Hv, d), inp["beta"][at], inp["g"][at], gc)
        assert bit_equal(o, want[at]), t


def test_refusals_on_the_gpu():
    p = make(4, 2, 1, 64, 32, norm="l2", seed=13)
    g = on_gpu(p)
    call = lambda **kw: B.gdn_qk_rotary(p["shape"], **{**dict(q=g["q"], k=g["k"], inv_freq=g["inv_freq"], pos=g["pos"]), **kw})  # noqa: E731
    for kw in (dict(pos=None), dict(cu_seqlens=g["pos"]), dict(pos=g["pos"].long()), dict(pos=g["pos"][:3]),
               dict(inv_freq=None), dict(inv_freq=g["inv_freq"].cpu()), dict(q=g["q"].float()), dict(k=g["k"][:3]),
               dict(q=g["q"].transpose(0, 1).contiguous().transpose(0, 1)), dict(start=g["pos"])):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(B.GdnError):       # weights with a norm that has none
        call(w_q=torch.ones(64, device="cuda"))
    with pytest.raises(B.GdnError):       # rows not a multiple of eight elements apart
        call(q=torch.zeros(4, 132, dtype=BF16, device="cuda")[:, :128].unflatten(1, (2, 64)))


@pytest.mark.parametrize("norm", ["rms", "l2"])
def test_smallest_heads_without_eps(norm):
    """eps = 0 and heads whose mean square lies around and below fp32's normal numbers.  Each square and each of their sums
    is off by 2^-150 there, so the sum of d = 64 squares of size s by 128 2^-150 / (64 s) of it, halved by the root, and the
    mean once more by 2^-150 / s."""
    sizes = [1e-10, 2e-19, 1.1e-19, 1e-19, 5e-20, 1e-20, 1e-21]
    T, d = len(sizes), 64
    gen = torch.Generator().manual_seed(20)
    x = (1 + torch.rand(T, 2, d, generator=gen)) * torch.tensor(sizes)[:, None, None]
    s = B.make_qk_shape(2, 0, d, 0, F32, norm=norm, eps=0.0, weight_offset=1.0)
    y, _ = B.gdn_qk_rotary(s, x.cuda(), None, None, pos=torch.zeros(T, dtype=torch.int32, device="cuda"))
    want, bound = qk_fwd(np64(x), norm=norm, layout="half", r=0, pos=np.zeros(T), inv_freq=np.zeros(0), eps=0.0,
                         w=np.ones(d) if norm == "rms" else None)
    low = 2 * 2.0 ** -150 / np.array(sizes)[:, None, None] ** 2
    check(y, want, bound + low * np.abs(want), "y")
