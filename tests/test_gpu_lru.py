"""The gated linear recurrence on the GPU against the fp64 oracle, and its bits
across prefill, continuation, decode, the trainer, batches, streams and graphs."""

import numpy as np
import pytest
import torch

from linear_attention_rnn_gated_amd import binding as B
from oracle.lru_oracle import lru_bwd, lru_fwd

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
DT = {"f32": F32, "bf16": BF16}


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()


def make(lens, D, x="bf16", g="f32", gate="none", h0=True, seed=0, resets=False):
    gen = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    lg = -torch.nn.functional.softplus(2 * rn(T, D))
    if resets and T:
        lg[torch.rand(T, generator=gen) < 0.05] = float("-inf")
        lg[torch.rand(T, D, generator=gen) < 0.02] = 0.0
    cu = torch.zeros(N + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(lens, dtype=torch.int64), 0)
    p = dict(x=rn(T, D).to(DT[x]), g=lg.to(DT[g]), cu=cu, gate=gate, lens=lens, D=D,
             h0=rn(N, D) if h0 else None, dO=rn(T, D).to(DT[x]), dhT=rn(N, D) if h0 else None)
    p["shape"] = B.make_lru_shape(D, DT[x], DT[g], gate)
    return p


def dev(p):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in p.items()}


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def bits(t):
    return t.detach().contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32).cpu()


def same(a, b):
    return a.shape == b.shape and a.dtype == b.dtype and torch.equal(bits(a), bits(b))


def check(got, want, bound, what):
    """|got - want| within the oracle's bound and half a step of the output's type (and fp32's smallest normal number)."""
    got = got.detach()
    half = torch.finfo(got.dtype).eps / 2
    g = np64(got)
    tol = bound + half * (np.abs(want) + bound) + 2.0 ** -126
    off = np.abs(g - want)
    bad = ~(off <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.nanmax(off / tol):.3g} of the bound"


def prefill(p, **kw):
    d = dev(p)
    return B.gdn_lru_prefill(p["shape"], d["x"], d["g"], d["cu"], h0=d["h0"], **kw)


SHAPES = [
    ([1], 1), ([5], 2), ([31], 3), ([32], 16), ([33], 17), ([0, 64, 0], 130), ([65, 1, 0, 97], 257), ([700], 64),
    ([40, 333], 520), ([2100], 24), ([1] * 70, 8), ([5000], 6),
    ([9000, 0, 40, 1], 33), ([3, 4200, 0, 2500], 40), ([300] * 12 + [7, 0, 1100], 100),
]


@pytest.mark.parametrize("lens,D", SHAPES)
@pytest.mark.parametrize("x,g,gate", [("bf16", "bf16", "norm"), ("f32", "f32", "complement"), ("bf16", "f32", "none"),
                                      ("f32", "bf16", "norm")])
def test_prefill_and_gradients(lens, D, x, g, gate):
    p = make(lens, D, x, g, gate, h0=D % 2 == 0, seed=D, resets=True)
    o, hT = prefill(p)
    xs, gs, cu, h0 = np64(p["x"]), np64(p["g"]), p["cu"].tolist(), np64(p["h0"])
    ro, rh, eo, eh = lru_fwd(xs, gs, cu, gate, h0)
    check(o, ro, eo, "o")
    check(hT, rh, eh, "hT")
    d = dev(p)
    r = B.gdn_lru_fwd_bwd(p["shape"], d["x"], d["g"], d["cu"], d["dO"], h0=d["h0"], dhT=d["dhT"])
    assert same(r["o"], o) and same(r["hT"], hT)
    want, bound = lru_bwd(xs, gs, cu, gate, np64(p["dO"]), h0, np64(p["dhT"]))
    for k in ("dx", "dg", "dh0"):
        assert r[k].dtype == {"dx": DT[x], "dg": DT[g], "dh0": F32}[k]
        check(r[k], want[k], bound[k], k)
    # the backward alone, and once more: the same bits
    only = B.gdn_lru_fwd_bwd(p["shape"], d["x"], d["g"], d["cu"], d["dO"], h0=d["h0"], dhT=d["dhT"], want_o=False)
    assert sorted(only) == ["dg", "dh0", "dx"]
    for k in only:
        assert same(only[k], r[k]), k


def test_gradient_by_differences():
    """The fp32 gradient along random directions against differences of the fp64 oracle's loss."""
    p = make([37, 70], 6, "f32", "f32", "norm", seed=9)
    d = dev(p)
    r = B.gdn_lru_fwd_bwd(p["shape"], d["x"], d["g"], d["cu"], d["dO"], h0=d["h0"], dhT=d["dhT"])
    xs, gs, h0, cu = np64(p["x"]), np64(p["g"]), np64(p["h0"]), p["cu"].tolist()

    def loss(x, g, h):
        o, hT, _, _ = lru_fwd(x, g, cu, "norm", h)
        return (o * np64(p["dO"])).sum() + (hT * np64(p["dhT"])).sum()
    rng = np.random.default_rng(1)
    _, bound = lru_bwd(xs, gs, cu, "norm", np64(p["dO"]), h0, np64(p["dhT"]))
    for at, (k, t) in enumerate((("dx", xs), ("dg", gs), ("dh0", h0))):
        v = rng.normal(size=t.shape)
        args, back = [xs, gs, h0], [xs, gs, h0]
        args[at], back[at] = t + 1e-6 * v, t - 1e-6 * v
        want = (loss(*args) - loss(*back)) / 2e-6
        got = (np64(r[k]) * v).sum()
        # the elements' bounds, plus the difference's own rounding: |loss| 2^-52 / 1e-6
        tol = ((bound[k] + 2.0 ** -24 * np.abs(np64(r[k]))) * np.abs(v)).sum() + 1e-9 * abs(loss(xs, gs, h0)) + 1e-6 * abs(want)
        assert abs(got - want) <= tol, (k, got, want, tol)


@pytest.mark.parametrize("x,g,gate,D", [("bf16", "f32", "norm", 300), ("f32", "f32", "none", 33), ("bf16", "bf16", "complement", 64)])
def test_decode_and_continuation_equal_one_prefill(x, g, gate, D):
    lens = [1, 40, 97, 32, 64, 130]
    p = make(lens, D, x, g, gate, seed=5, resets=True)
    d, cu, N = dev(p), p["cu"].tolist(), len(lens)
    o, hT = prefill(p)
    cache = B.gdn_lru_cache_init(p["shape"], N, "cuda", h0=d["h0"])
    # all tokens one at a time; the sequences end at different steps, so the finished ones keep a copy of their cache
    done = {}
    for t in range(max(lens)):
        rows = torch.tensor([min(cu[n] + t, cu[n + 1] - 1) for n in range(N)], device="cuda")
        step = B.gdn_lru_decode_step(p["shape"], d["x"][rows], d["g"][rows], cache)
        for n in range(N):
            if t < lens[n]:
                assert same(step[n], o[cu[n] + t]), (n, t)
            if t == lens[n] - 1:
                done[n] = cache.clone()
    for n in range(N):
        assert same(done[n].state()[n], done[n].A[n] * done[n].S[n] + done[n].B[n])
        assert int(done[n].pos[n, 0]) == lens[n] % 32 and bool((done[n].pos[n] == done[n].pos[n, 0]).all())
    # prefill of a part, continuation twice, decode of the last token
    cuts = [[0, 0, 1, 1], [0, 7, 39, 40], [33, 33, 96, 97], [0, 31, 31, 32], [32, 63, 63, 64], [64, 65, 129, 130]]
    parts = []
    cache = B.LruCache(D, N, "cuda")
    for a in range(3):
        seg = [(cu[n] + (0 if a == 0 else cuts[n][a - 1]), cu[n] + cuts[n][a]) for n in range(N)]
        rows = torch.cat([torch.arange(i, j) for i, j in seg]).cuda()
        c = torch.tensor([0] + list(np.cumsum([j - i for i, j in seg])), dtype=torch.int32)
        if a == 0:
            got, _ = B.gdn_lru_prefill(p["shape"], d["x"][rows], d["g"][rows], c.cuda(), h0=d["h0"], cache=cache)
        else:
            got, last = B.gdn_lru_prefill_continue(p["shape"], d["x"][rows], d["g"][rows], c.cuda(), cache)
        assert same(got, o[rows]), a
        parts.append(seg)
    live = [n for n in range(N) if cuts[n][3] > cuts[n][2]]
    sub = B.LruCache.of(*[t[live].contiguous() for t in cache.tensors()])
    rows = torch.tensor([cu[n + 1] - 1 for n in live], device="cuda")
    assert same(B.gdn_lru_decode_step(p["shape"], d["x"][rows], d["g"][rows], sub), o[rows])
    for i, n in enumerate(live):
        for a, b in zip(sub.tensors(), done[n].tensors()):
            assert torch.equal(a[i].view(torch.int32), b[n].view(torch.int32)), n


def test_prefill_cache_equals_decoded_cache_and_empty_sequences():
    p = make([0, 32, 45, 0], 40, seed=6)
    d = dev(p)
    cache = B.LruCache(40, 4, "cuda")
    _, hT = prefill(p, cache=cache)
    assert same(cache.S[0], d["h0"][0]) and bool((cache.A[0] == 1).all()) and bool((cache.B[0] == 0).all())
    assert cache.pos[:, 0].tolist() == [0, 0, 13, 0]
    assert same(hT[0], d["h0"][0]) and same(hT[1], cache.S[1])
    before = [t.clone() for t in cache.tensors()]
    zero = torch.zeros(5, dtype=torch.int32, device="cuda")
    o, h = B.gdn_lru_prefill_continue(p["shape"], d["x"][:0], d["g"][:0], zero, cache)
    assert o.shape == (0, 40) and all(torch.equal(a, b) for a, b in zip(before, cache.tensors()))
    assert same(h[2], hT[2])
    r = B.gdn_lru_fwd_bwd(p["shape"], d["x"], d["g"], d["cu"], d["dO"], h0=d["h0"], dhT=d["dhT"])
    assert same(r["dh0"][0], d["dhT"][0]) and same(r["hT"][3], d["h0"][3])


def kernels(call):
    """The names' launch counts of the library kernels that `call` runs, and what it returns."""
    B.profile_enable(True)
    try:
        r = call()
        torch.cuda.synchronize()
        names = ("k_lru_fwd", "k_lru_fold", "k_lru_chain", "k_lru_apply", "k_lru_grad", "k_lru_pos", "k_lru_train")
        return {k: B.profile_read(k)[1] for k in names}, r
    finally:
        B.profile_enable(False)


@pytest.mark.parametrize("D,gate", [(40, "norm"), (300, "none")])
def test_both_schedules_continue_to_the_same_bits(D, gate):
    """One long sequence of few channels takes the three steps, short ones the one pass; continued from caches that stand
    inside chunks, with sequences that bring no token, both equal one prefill."""
    lens, cut = [6000 * (1 if D == 300 else 2), 45, 100, 32], [17, 45, 64, 32]
    p = make(lens, D, "bf16", "bf16", gate, seed=60, resets=True)
    d, cu = dev(p), p["cu"].tolist()
    n, (o, hT) = kernels(lambda: prefill(p))
    assert n["k_lru_fold"] == n["k_lru_chain"] == n["k_lru_apply"] == 1 and n["k_lru_fwd"] == 0
    rows = lambda a, b: torch.cat([torch.arange(cu[i] + a[i], cu[i] + b[i]) for i in range(4)]).cuda()  # noqa: E731
    count = lambda a, b: torch.tensor([0] + list(np.cumsum([j - i for i, j in zip(a, b)])), dtype=torch.int32)  # noqa: E731
    cache, r = B.LruCache(D, 4, "cuda"), rows([0] * 4, cut)
    n, (first, _) = kernels(lambda: B.gdn_lru_prefill(p["shape"], d["x"][r], d["g"][r], count([0] * 4, cut).cuda(), h0=d["h0"],
                                                      cache=cache))
    assert n["k_lru_fwd"] == 1 and n["k_lru_fold"] == 0 and same(first, o[r])
    r = rows(cut, lens)
    n, (rest, last) = kernels(lambda: B.gdn_lru_prefill_continue(p["shape"], d["x"][r], d["g"][r], count(cut, lens).cuda(), cache))
    assert n["k_lru_fold"] == 1 and same(rest, o[r])
    full = B.LruCache(D, 4, "cuda")
    prefill(p, cache=full)
    for a, b in zip(cache.tensors(), full.tensors()):
        assert torch.equal(a.view(torch.int32), b.view(torch.int32))
    assert same(last[0], hT[0]) and same(last[1], cache.state()[1])
    # the same long sequence next to as many others as let the one pass have it
    many = make(lens[:1] * 40, 300, "bf16", "bf16", gate, seed=61)
    if D == 300:
        many["x"][:6000], many["g"][:6000], many["h0"][0] = p["x"][:6000], p["g"][:6000], p["h0"][0]
        n, (om, hm) = kernels(lambda: prefill(many))
        assert n["k_lru_fwd"] == 1 and n["k_lru_fold"] == 0 and same(om[:6000], o[:6000]) and same(hm[0], hT[0])


def test_batch_composition_does_not_change_bits():
    lens = [300, 7, 0, 2500, 64, 33]
    p = make(lens, 96, "bf16", "bf16", "norm", seed=7)
    d, cu = dev(p), p["cu"].tolist()
    o, hT = prefill(p)
    r = B.gdn_lru_fwd_bwd(p["shape"], d["x"], d["g"], d["cu"], d["dO"], h0=d["h0"], dhT=d["dhT"])
    for n in (0, 1, 3, 5):
        s = slice(cu[n], cu[n + 1])
        c = torch.tensor([0, lens[n]], dtype=torch.int32, device="cuda")
        o1, h1 = B.gdn_lru_prefill(p["shape"], d["x"][s].contiguous(), d["g"][s].contiguous(), c, h0=d["h0"][n:n + 1].contiguous())
        assert same(o1, o[s]) and same(h1[0], hT[n])
        a, b = d["x"][s].contiguous(), d["g"][s].contiguous()
        q = B.gdn_lru_fwd_bwd(p["shape"], a, b, c, d["dO"][s].contiguous(), h0=d["h0"][n:n + 1].contiguous(),
                              dhT=d["dhT"][n:n + 1].contiguous())
        for k in ("dx", "dg"):
            assert same(q[k], r[k][s]), (n, k)
        assert same(q["dh0"][0], r["dh0"][n])
    # channels are independent: a slice of them, an odd number, gives their bits
    part = B.make_lru_shape(31, BF16, BF16, "norm")
    o2, _ = B.gdn_lru_prefill(part, d["x"][:, 16:47], d["g"][:, 16:47], d["cu"], h0=d["h0"][:, 16:47].contiguous())
    assert same(o2, o[:, 16:47])


@pytest.mark.parametrize("lens,D,x,g,gate", [
    ([100, 256, 0, 1, 33, 64], 130, "bf16", "f32", "norm"),
    ([512, 31, 257, 32, 0, 300], 70, "f32", "bf16", "complement"),
    ([1000, 640, 1, 90, 1024], 33, "bf16", "bf16", "none"),
    ([0, 5, 40, 2, 64] * 20, 65, "f32", "f32", "norm"),
    ([0, 0], 7, "f32", "f32", "none"),
])
def test_both_trainer_schedules_give_the_same_bits(lens, D, x, g, gate):
    """Sequences that fit a round take one pass; with a longer one in the batch all take the three steps."""
    p = make(lens + [1025], D, x, g, gate, seed=23)
    d, T, N = dev(p), sum(lens), len(lens)

    def run(n, T):
        c, r = kernels(lambda: B.gdn_lru_fwd_bwd(p["shape"], d["x"][:T], d["g"][:T], d["cu"][:n + 1], d["dO"][:T],
                                                 h0=d["h0"][:n], dhT=d["dhT"][:n]))
        return r, (c["k_lru_train"], c["k_lru_grad"])
    three, k = run(N + 1, T + 1025)
    assert k == (0, 1)
    one, k = run(N, T)
    assert k == (1, 0)
    for key, t in one.items():
        assert same(t, three[key][:t.shape[0]]), key
    bw = B.gdn_lru_fwd_bwd(p["shape"], d["x"][:T], d["g"][:T], d["cu"][:N + 1], d["dO"][:T], h0=d["h0"][:N],
                           dhT=d["dhT"][:N], want_o=False)
    assert all(same(t, one[key]) for key, t in bw.items())


def test_trainer_of_many_sequences_next_to_a_long_one():
    """Enough sequences for the chains to go over many channels a block; the first four of them alone give the same bits."""
    lens = [1300] + [20, 0, 33] * 70
    p = make(lens, 330, "bf16", "f32", "norm", seed=29)
    d, T = dev(p), int(p["cu"][4])
    many = B.gdn_lru_fwd_bwd(p["shape"], d["x"], d["g"], d["cu"], d["dO"], h0=d["h0"], dhT=d["dhT"])
    few = B.gdn_lru_fwd_bwd(p["shape"], d["x"][:T], d["g"][:T], d["cu"][:5], d["dO"][:T], h0=d["h0"][:4], dhT=d["dhT"][:4])
    for key, t in few.items():
        assert same(t, many[key][:t.shape[0]]), key
    last = lambda name, n: d[name][-n:].clone()  # noqa: E731
    one = B.gdn_lru_fwd_bwd(p["shape"], last("x", 33), last("g", 33), torch.tensor([0, 33], dtype=torch.int32, device="cuda"),
                            last("dO", 33), h0=last("h0", 1), dhT=last("dhT", 1))
    for key, t in one.items():
        assert same(t, many[key][-t.shape[0]:]), key


def test_no_nan_crosses_into_another_sequences_gradient():
    lens = [70, 40, 33, 64, 100, 20]
    p = make(lens, 6, "f32", "f32", "norm", seed=18)
    cu, d = p["cu"].tolist(), dev(p)
    train = lambda: B.gdn_lru_fwd_bwd(p["shape"], d["x"], d["g"], d["cu"], d["dO"], h0=d["h0"], dhT=d["dhT"])  # noqa: E731
    want = train()
    payload = torch.tensor([0xffc0dead - (1 << 32), 0x7fc00000, 0xffc0dead - (1 << 32), 0x7f800001, -1, 0x7fffffff], dtype=torch.int32)
    d["x"][cu[0] + 5], d["dO"][cu[2] + 1] = float("nan"), float("inf")
    d["g"][cu[1] + 36] = d["g"][cu[4] + 66] = payload.view(F32).cuda()
    got = train()
    for n in (3, 5):
        for k in ("o", "dx", "dg"):
            assert same(got[k][cu[n]:cu[n + 1]], want[k][cu[n]:cu[n + 1]]), (n, k)
        assert same(got["hT"][n], want["hT"][n]) and same(got["dh0"][n], want["dh0"][n])
    for n, t in ((1, 36), (4, 66)):  # states behind the NaN, gradients in front of it
        assert bool(got["o"][cu[n] + t:cu[n + 1]].isnan().all()) and bool(got["dx"][cu[n]:cu[n] + t].isnan().all())
        assert same(got["o"][cu[n]:cu[n] + t], want["o"][cu[n]:cu[n] + t])
        assert same(got["dx"][cu[n] + t + 1:cu[n + 1]], want["dx"][cu[n] + t + 1:cu[n + 1]])


def test_wide_rows_in_place_and_rows_behind():
    """Slices of one projection's rows, o over x, rows past the last sequence untouched."""
    p = make([50, 0, 81], 48, "bf16", "bf16", "complement", seed=8)
    d, T = dev(p), 131
    want, hT = prefill(p)
    wide = torch.full((T + 9, 200), float("nan"), dtype=BF16, device="cuda")
    wide[:T, 8:56], wide[:T, 64:112] = d["x"], d["g"]
    x, g = wide[:, 8:56], wide[:, 64:112]
    cache = B.LruCache(48, 3, "cuda")
    o, h = B.gdn_lru_prefill(p["shape"], x, g, d["cu"], h0=d["h0"], out=x, cache=cache)
    assert same(wide[:T, 8:56], want) and same(h, hT)
    assert bool(wide[T:].isnan().all()) and bool(wide[:, :8].isnan().all()) and bool(wide[:, 56:64].isnan().all())
    assert same(wide[:T, 64:112], d["g"])
    r = B.gdn_lru_fwd_bwd(p["shape"], d["x"], d["g"], d["cu"], d["dO"], h0=d["h0"])
    out = {k: torch.full((T + 9, 64), 7.0, dtype=BF16, device="cuda")[:, 8:56] for k in ("dx", "dg", "o")}
    pad = lambda t: torch.cat([t, torch.full((9, 48), float("nan"), dtype=t.dtype, device="cuda")])  # noqa: E731
    q = B.gdn_lru_fwd_bwd(p["shape"], pad(d["x"]), pad(d["g"]), d["cu"], pad(d["dO"]), h0=d["h0"], out=out)
    for k in ("dx", "dg", "o"):
        assert same(q[k][:T], r[k]) and bool((q[k][T:] == 7).all()), k
    dec = torch.full((3, 100), 5.0, dtype=BF16, device="cuda")
    xs, gs = wide[:3, 64:112], wide[3:6, 64:112]
    a, b = cache.clone(), cache.clone()
    B.gdn_lru_decode_step(p["shape"], xs, gs, a, out=dec[:, 40:88])
    assert same(dec[:, 40:88], B.gdn_lru_decode_step(p["shape"], xs.contiguous(), gs.contiguous(), b))
    assert bool((dec[:, :40] == 5).all()) and bool((dec[:, 88:] == 5).all())


def test_long_rows_in_place_and_rows_behind():
    """The three steps over slices of wider rows: o over x, NaN behind the last sequence left alone and not read."""
    T, D = 7000, 40
    p = make([T], D, "bf16", "bf16", "norm", seed=16)
    d = dev(p)
    want, hT = prefill(p)
    grads = B.gdn_lru_fwd_bwd(p["shape"], d["x"], d["g"], d["cu"], d["dO"], h0=d["h0"])
    wide = torch.full((T + 33, 200), float("nan"), dtype=BF16, device="cuda")
    wide[:T, 8:48], wide[:T, 64:104], wide[:T, 120:160] = d["x"], d["g"], d["dO"]
    x, g, dO = wide[:, 8:48], wide[:, 64:104], wide[:, 120:160]
    out = {k: torch.full((T + 33, 64), 7.0, dtype=BF16, device="cuda")[:, 8:48] for k in ("o", "dx", "dg")}
    r = B.gdn_lru_fwd_bwd(p["shape"], x, g, d["cu"], dO, h0=d["h0"], out=out)
    for k in out:
        assert same(r[k][:T], grads[k]) and bool((r[k][T:] == 7).all()), k
    n, (o, h) = kernels(lambda: B.gdn_lru_prefill(p["shape"], x, g, d["cu"], h0=d["h0"], out=x))
    assert n["k_lru_fold"] == 1 and same(wide[:T, 8:48], want) and same(h, hT)
    assert bool(wide[T:].isnan().all()) and bool(wide[:, 48:64].isnan().all())


def test_offsets_past_32_bits():
    """Rows 2^21 elements apart: 1500 of them span 3e9 elements, 6 GB."""
    p = make([900, 600], 32, "bf16", "bf16", "norm", seed=10)
    d = dev(p)
    want = B.gdn_lru_fwd_bwd(p["shape"], d["x"], d["g"], d["cu"], d["dO"], h0=d["h0"])
    big = torch.empty(1500, 1 << 21, dtype=BF16, device="cuda")
    cols = {k: big[:, i * 64:i * 64 + 32] for i, k in enumerate(("x", "g", "dO", "o", "dx", "dg"))}
    for k in ("x", "g", "dO"):
        cols[k].copy_(d[k])
    r = B.gdn_lru_fwd_bwd(p["shape"], cols["x"], cols["g"], d["cu"], cols["dO"], h0=d["h0"],
                          out={k: cols[k] for k in ("o", "dx", "dg")})
    for k in ("o", "dx", "dg", "hT", "dh0"):
        assert same(r[k], want[k]), k


def test_growth_infinities_and_nan_stay_in_their_channel():
    p = make([90], 8, "f32", "f32", "none", seed=11)
    p["g"][:, 1] = 0.3                    # growing state
    p["x"][40, 2] = float("inf")
    p["x"][50, 3] = float("nan")
    p["g"][70, 2] = p["g"][70, 3] = float("-inf")
    o, hT = prefill(p)
    clean = dict(p, x=p["x"].clone(), g=p["g"].clone())
    clean["x"][40, 2] = clean["x"][50, 3] = 0.0
    oc, _ = prefill(clean)
    for c in (0, 1, 4, 5, 6, 7):
        assert same(o[:, c], oc[:, c])
    assert same(o[:40, 2], oc[:40, 2]) and bool(o[40:70, 2].isinf().all()) and same(o[:50, 3], oc[:50, 3])
    assert bool(o[50:, 3].isnan().all()) and bool(o[70:, 2].isnan().all())   # 0 times inf is NaN, as the formula has it
    ro, _, eo, _ = lru_fwd(np64(clean["x"]), np64(clean["g"]), [0, 90], "none", np64(clean["h0"]))
    check(oc, ro, eo, "o")


@pytest.mark.parametrize("most,D", [(6, 40), (90, 130), (400, 17)])
def test_many_sequences_continue(most, D):
    """More sequences than are packed by length, empty ones among them: a prefix, two continuations and a decode step equal
    one prefill of each."""
    N = 150
    gen = torch.Generator().manual_seed(most)
    lens = [int(v) for v in torch.randint(0, most, (N,), generator=gen)]
    p = make(lens, D, "bf16", "f32", "complement", seed=most)
    d, cu = dev(p), p["cu"].tolist()
    o, hT = prefill(p)
    ro, rh, eo, eh = lru_fwd(np64(p["x"]), np64(p["g"]), cu, "complement", np64(p["h0"]))
    check(o, ro, eo, "o")
    check(hT, rh, eh, "hT")
    cache, at = B.gdn_lru_cache_init(p["shape"], N, "cuda", h0=d["h0"]), [0] * N
    for step in range(3):
        to = [n if step == 2 else int(torch.randint(a, n + 1, (1,), generator=gen)) for a, n in zip(at, lens)]
        rows = torch.cat([torch.arange(cu[n] + at[n], cu[n] + to[n]) for n in range(N)]).cuda()
        c = torch.tensor([0] + list(np.cumsum([b - a for a, b in zip(at, to)])), dtype=torch.int32, device="cuda")
        got, last = B.gdn_lru_prefill_continue(p["shape"], d["x"][rows], d["g"][rows], c, cache)
        assert same(got, o[rows]), step
        at = to
    assert same(last, hT)
    full = B.LruCache(D, N, "cuda")
    prefill(p, cache=full)
    for a, b in zip(cache.tensors(), full.tensors()):
        assert torch.equal(a.view(torch.int32), b.view(torch.int32))


def test_positions_outside_a_chunk_are_clamped():
    p = make([40, 3, 2500], 300, seed=18)
    d = dev(p)
    for bad in (-3, 99, 32, -(1 << 31), (1 << 31) - 1):
        for lens in ([40, 3, 0], [40, 3, 2500]):
            cache = B.gdn_lru_cache_init(p["shape"], 3, "cuda", h0=d["h0"])
            cache.pos.fill_(bad)
            T = sum(lens)
            cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")
            out = torch.full((T + 40, 300), 3.0, dtype=BF16, device="cuda")
            pad = lambda t: torch.cat([t[:T], t[:40]])  # noqa: E731
            B.gdn_lru_prefill_continue(p["shape"], pad(d["x"]), pad(d["g"]), cu, cache, out=out)
            assert bool((out[T:] == 3).all()) and bool((cache.pos >= 0).all()) and bool((cache.pos < 32).all())
            cache.pos.fill_(bad)
            B.gdn_lru_decode_step(p["shape"], d["x"][:3], d["g"][:3], cache)
            assert bool((cache.pos >= 0).all()) and bool((cache.pos < 32).all())


@pytest.mark.parametrize("long", [False, True])
def test_no_nan_crosses_into_another_sequence(long):
    """Sequences that share a block's round, after ones whose states are NaN or infinite, and a NaN of every payload as g."""
    lens = [70, 40, 33, 64, 100] + ([9000] if long else [])
    p = make(lens, 6, "f32", "f32", "norm", seed=17)
    cu = p["cu"].tolist()
    want, wh = prefill(p)
    bad = dict(p, x=p["x"].clone(), g=p["g"].clone())
    bad["x"][cu[0] + 5], bad["x"][cu[2] + 1] = float("nan"), float("inf")
    payload = torch.tensor([0xffc0dead - (1 << 32), 0x7fc00000, 0xffc0dead - (1 << 32), 0x7f800001, -1, 0x7fffffff], dtype=torch.int32)
    bad["g"][cu[1] + 36] = payload.view(F32)
    bad["g"][cu[4] + 66] = payload.view(F32)
    o, h = prefill(bad)
    for n in (3, 5)[:1 + long]:
        assert same(o[cu[n]:cu[n + 1]], want[cu[n]:cu[n + 1]]) and same(h[n], wh[n]), n
    for n, t in ((0, 5), (1, 36), (2, 1), (4, 66)):   # until then as without it
        assert same(o[cu[n]:cu[n] + t], want[cu[n]:cu[n] + t]), n
    for n, t in ((0, 5), (1, 36), (4, 66)):
        assert bool(o[cu[n] + t:cu[n + 1]].isnan().all()) and bool(h[n].isnan().all())


def test_many_sequences_and_longest_channel_count():
    p = make([2] * 70000, 5, "bf16", "f32", "none", seed=12)
    o, hT = prefill(p)
    x, g = p["x"].double().view(-1, 2, 5), p["g"].double().view(-1, 2, 5)
    h = p["h0"].double()
    for t in range(2):
        h = g[:, t].exp() * h + x[:, t]
    # two tokens: within 2 C_STEP of terms below 16, and the rounding of an fp32 state
    assert float((hT.cpu().double() - h).abs().max()) < 16 * 2 * 2.0 ** -20
    q = make([3], 1 << 20, "bf16", "bf16", "norm", seed=13)
    o, _ = prefill(q)
    ro, _, eo, _ = lru_fwd(np64(q["x"]), np64(q["g"]), [0, 3], "norm", np64(q["h0"]))
    check(o, ro, eo, "o")


def test_host_copy_that_disagrees_stays_inside():
    """A device copy with other values than the host's gives wrong numbers but touches only the rows [0, T)."""
    p = make([40, 40], 16, seed=14)
    d = dev(p)
    x, g = d["x"], d["g"]
    out = torch.full((100, 16), 3.0, dtype=BF16, device="cuda")
    pad = lambda t: torch.cat([t, t[:20]])  # noqa: E731
    bad = torch.tensor([-5, 95, 30], dtype=torch.int32, device="cuda")
    B.gdn_lru_prefill(p["shape"], pad(x), pad(g), bad, h0=d["h0"], out=out, cu_seqlens_host=p["cu"])
    assert bool((out[80:] == 3).all())
    dx, dg = torch.full((100, 16), 3.0, dtype=BF16, device="cuda"), torch.full((100, 16), 3.0, device="cuda")
    B.gdn_lru_fwd_bwd(p["shape"], pad(x), pad(g), bad, pad(d["dO"]), h0=d["h0"], out=dict(o=out, dx=dx, dg=dg),
                      cu_seqlens_host=p["cu"])
    assert bool((out[80:] == 3).all()) and bool((dx[80:] == 3).all()) and bool((dg[80:] == 3).all())


def test_null_host_copy():
    """The C entry reads cu_seqlens back itself when the host copy is NULL."""
    import ctypes
    p = make([33, 20], 16, seed=15)
    d = dev(p)
    want, _ = prefill(p)
    o = torch.empty_like(d["x"])
    ws = torch.empty(B.lru_workspace_bytes(p["shape"], 2, 53, B.OP_PREFILL), dtype=torch.uint8, device="cuda")
    st = B.lib().gdn_lru_prefill(ctypes.byref(p["shape"]), 2, d["cu"].data_ptr(), None, d["x"].data_ptr(), 0,
                                 d["g"].data_ptr(), 0, d["h0"].data_ptr(), o.data_ptr(), 0, None, None,
                                 ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == B.GDN_OK and same(o, want)


def test_streams():
    """Two calls at once on their own streams and buffers; a call waits for its own stream's work alone."""
    ps = [make([1500, 700], 128, seed=20 + i, gate="norm") for i in range(2)]
    want = [prefill(p) for p in ps]
    ds = [dev(p) for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    got = []
    for p, d, s in zip(ps, ds, streams):
        with torch.cuda.stream(s):
            x = d["x"] * 1   # made on this stream just before
            got.append(B.gdn_lru_prefill(p["shape"], x, d["g"], d["cu"], h0=d["h0"], cu_seqlens_host=p["cu"]))
    torch.cuda.synchronize()
    for (o, h), (ro, rh) in zip(got, want):
        assert same(o, ro) and same(h, rh)


def test_two_graphs_share_a_workspace():
    """Two captured trainer steps (and a captured long prefill) on one workspace, replayed in turn."""
    ps = [make([3000, 40], 48, "bf16", "f32", "norm", seed=32), make([100, 2500], 48, "bf16", "f32", "none", seed=33)]
    ds = [dev(p) for p in ps]
    ws = torch.empty(max(B.lru_workspace_bytes(p["shape"], 2, sum(p["lens"])) for p in ps), dtype=torch.uint8, device="cuda")

    def step(p, d):
        r = B.gdn_lru_fwd_bwd(p["shape"], d["x"], d["g"], d["cu"], d["dO"], h0=d["h0"], ws=ws, cu_seqlens_host=p["cu"])
        o, h = B.gdn_lru_prefill(p["shape"], d["x"], d["g"], d["cu"], h0=d["h0"], ws=ws, cu_seqlens_host=p["cu"])
        return [*(r[k] for k in sorted(r)), o, h]
    want = [[t.clone() for t in step(p, d)] for p, d in zip(ps, ds)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for p, d in zip(ps, ds):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(p, d))
        graphs.append(g)
    for order in ((0, 1), (1, 0), (1, 1), (0, 0)):
        for i in order:
            for t in outs[i]:
                t.zero_()
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in set(order):
            for a, b in zip(outs[i], want[i]):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), (order, i)


def test_captured_in_a_graph():
    """Prefill with a cache, continuation, decode and the trainer in one graph: every replay equals the eager calls."""
    p = make([70, 20], 64, "bf16", "f32", "norm", seed=30)
    q = make([33, 5], 64, "bf16", "f32", "norm", seed=31)
    d, e = dev(p), dev(q)
    cache = B.LruCache(64, 2, "cuda")
    ws = torch.empty(B.lru_workspace_bytes(p["shape"], 2, 90), dtype=torch.uint8, device="cuda")

    def step():
        out = list(B.gdn_lru_prefill(p["shape"], d["x"], d["g"], d["cu"], h0=d["h0"], cache=cache, cu_seqlens_host=p["cu"]))
        out += B.gdn_lru_prefill_continue(p["shape"], e["x"], e["g"], e["cu"], cache, cu_seqlens_host=q["cu"])
        out.append(B.gdn_lru_decode_step(p["shape"], e["x"][:2], e["g"][:2], cache))
        r = B.gdn_lru_fwd_bwd(p["shape"], d["x"], d["g"], d["cu"], d["dO"], h0=d["h0"], ws=ws, cu_seqlens_host=p["cu"])
        return out + [r[k] for k in sorted(r)] + cache.tensors()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for k in range(4):
        d["x"].copy_(torch.randn(90, 64, generator=torch.Generator().manual_seed(k)).cuda())
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), k


def test_poisoned_buffers():
    """Outputs, workspace and a cache to be filled hold NaN patterns before; nothing of them shows."""
    p = make([100, 3], 72, "bf16", "bf16", "norm", seed=40)
    d = dev(p)
    res = []
    for fill in (0xFF, 0x00):
        ws = torch.full((B.lru_workspace_bytes(p["shape"], 2, 103),), fill, dtype=torch.uint8, device="cuda")
        cache = B.LruCache(72, 2, "cuda")
        for t in cache.tensors():
            t.view(torch.uint8).fill_(fill)
        o, h = prefill(p, cache=cache)
        r = B.gdn_lru_fwd_bwd(p["shape"], d["x"], d["g"], d["cu"], d["dO"], ws=ws)
        res.append([o, h, *cache.tensors(), *[r[k] for k in sorted(r)]])
    for a, b in zip(*res):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_refusals_on_the_gpu():
    p = make([40], 16, seed=50)
    d = dev(p)
    s = p["shape"]
    with pytest.raises(ValueError):
        B.gdn_lru_prefill(s, d["x"].float(), d["g"], d["cu"])
    with pytest.raises(ValueError):
        B.gdn_lru_prefill(s, d["x"][:39], d["g"], d["cu"])
    with pytest.raises(ValueError):
        B.gdn_lru_prefill(s, d["x"][:39], d["g"][:39], d["cu"])        # cu_seqlens past the rows
    with pytest.raises(ValueError):
        B.gdn_lru_prefill(s, d["x"], d["g"], d["cu"], h0=d["h0"].cpu())
    with pytest.raises(ValueError):
        B.gdn_lru_decode_step(s, d["x"], d["g"], B.LruCache(16, 39, "cuda"))
    with pytest.raises(ValueError):
        B.gdn_lru_fwd_bwd(s, d["x"], d["g"], d["cu"], d["dO"], want_o=False, out={"o": d["x"]})
    with pytest.raises(B.GdnError):
        B.gdn_lru_fwd_bwd(s, d["x"], d["g"], d["cu"], d["dO"], ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(B.GdnError):                                     # a start that is not 16-byte aligned
        B.gdn_lru_prefill(B.make_lru_shape(15, BF16), d["x"][:, 1:], d["g"][:, 1:], d["cu"])


def test_kernel_timing_names():
    p = make([40], 16, seed=51)
    B.profile_enable(True)
    try:
        prefill(p, cache=B.LruCache(16, 1, "cuda"))
        torch.cuda.synchronize()
        ms, n = B.profile_read("k_lru_")
        assert n == 2 and ms > 0
    finally:
        B.profile_enable(False)


STRAY = [[100, 6000, 6045], [-5, 7000, 30], [6045, 0, 6045], [3000, 3000, 3000], [6044, 6045, 1 << 30], [-(1 << 31), -1, 0]]


@pytest.mark.parametrize("stray", STRAY)
def test_host_copy_that_disagrees_stays_inside_three_steps(stray):
    """The schedules that keep chunks in the workspace, whose places follow from the device copy: a copy that starts behind
    row 0, steps back or ends elsewhere reads no cache that is not there and touches only the rows [0, T)."""
    lens, D, T = [6000, 45], 40, 6045
    p = make(lens, D, seed=62)
    d = dev(p)
    pad = lambda t: torch.cat([t, t[:60]])  # noqa: E731
    fresh = lambda dt=BF16: torch.full((T + 60, D), 3.0, dtype=dt, device="cuda")  # noqa: E731
    bad = torch.tensor(stray, dtype=torch.int32, device="cuda")
    x, g, dO = pad(d["x"]), pad(d["g"]), pad(d["dO"])
    cache = B.gdn_lru_cache_init(p["shape"], 2, "cuda", h0=d["h0"])
    cache.pos.fill_(17)
    for call in (lambda o: B.gdn_lru_prefill(p["shape"], x, g, bad, h0=d["h0"], out=o, cu_seqlens_host=p["cu"]),
                 lambda o: B.gdn_lru_prefill_continue(p["shape"], x, g, bad, cache, out=o, cu_seqlens_host=p["cu"])):
        out = fresh()
        n, (_, hT) = kernels(lambda: call(out))
        assert n["k_lru_fold"] == n["k_lru_apply"] == 1 and hT.shape == (2, D)
        assert bool((out[T:] == 3).all())
    out = dict(o=fresh(), dx=fresh(), dg=fresh(F32))
    n, _ = kernels(lambda: B.gdn_lru_fwd_bwd(p["shape"], x, g, bad, dO, h0=d["h0"], out=out, cu_seqlens_host=p["cu"]))
    assert n["k_lru_fold"] == n["k_lru_grad"] == 1
    assert all(bool((t[T:] == 3).all()) for t in out.values())
    # the right copy gives the right bits after it
    assert same(prefill(p)[0], B.gdn_lru_fwd_bwd(p["shape"], d["x"], d["g"], d["cu"], d["dO"], h0=d["h0"])["o"])


def test_a_reordered_cache_continues_its_sequences():
    """A batch whose cache tensors are assigned in another order, then cut: decode and continuation go on with what was
    assigned."""
    lens, D = [40, 7, 64, 33], 300
    p = make(lens, D, seed=63)
    d = dev(p)
    cache = B.LruCache(D, 4, "cuda")
    prefill(p, cache=cache)
    fixed, step = cache.clone(), make([1] * 4, D, seed=64)
    x, g = step["x"].cuda(), step["g"].cuda()
    want = B.gdn_lru_decode_step(p["shape"], x, g, fixed)
    order = torch.tensor([2, 0, 3, 1], device="cuda")
    cache.S, cache.A, cache.B, cache.pos = (t[order] for t in cache.tensors())
    assert same(B.gdn_lru_decode_step(p["shape"], x[order], g[order], cache), want[order])
    for a, b in zip(cache.tensors(), fixed.tensors()):
        assert torch.equal(a.view(torch.int32), b[order].view(torch.int32))
    cache.S, cache.A, cache.B, cache.pos = (t[1:3].clone() for t in cache.tensors())
    cu = torch.tensor([0, 5, 12], dtype=torch.int32, device="cuda")
    some = fixed.clone()
    some = B.LruCache.of(*[t[order[1:3]].contiguous() for t in some.tensors()])
    a, _ = B.gdn_lru_prefill_continue(p["shape"], d["x"][:12], d["g"][:12], cu, cache)
    b, _ = B.gdn_lru_prefill_continue(p["shape"], d["x"][:12], d["g"][:12], cu, some)
    assert same(a, b) and all(torch.equal(s.view(torch.int32), t.view(torch.int32)) for s, t in zip(cache.tensors(), some.tensors()))
    cache.A = cache.A[:1]
    with pytest.raises(ValueError):
        B.gdn_lru_decode_step(p["shape"], x[:2], g[:2], cache)


@pytest.mark.parametrize("gate", ["none", "complement", "norm"])
@pytest.mark.parametrize("lens", [[70, 40], [1100, 40]])
def test_a_nan_decay_reaches_its_own_tokens_gradient(lens, gate):
    """Both trainer schedules: a NaN in g makes dx at that token NaN where its weight depends on g, and dg always; the last
    token's dx without a gate is dO + dhT."""
    p = make(lens, 6, "f32", "f32", gate, seed=65)
    d, t = dev(p), lens[0] - 1
    at = [t, 33, sum(lens) - 1]
    d["g"][at[0], 1], d["g"][at[1], 2], d["g"][at[2], 3] = (float("nan"),) * 3
    n, r = kernels(lambda: B.gdn_lru_fwd_bwd(p["shape"], d["x"], d["g"], d["cu"], d["dO"], h0=d["h0"], dhT=d["dhT"]))
    assert n["k_lru_train"] == (lens[0] < 1024) and n["k_lru_grad"] == (lens[0] > 1024)
    for row, c in zip(at, (1, 2, 3)):
        assert bool(r["dg"][row, c].isnan()) and bool(r["o"][row, c].isnan())
        assert bool(r["dx"][row, c].isnan()) == (gate != "none"), (row, c)
    want, _ = lru_bwd(np64(d["x"]), np64(d["g"]), p["cu"].tolist(), gate, np64(d["dO"]), np64(d["h0"]), np64(d["dhT"]))
    for k in ("dx", "dg", "dh0"):
        assert np.array_equal(np.isnan(np64(r[k])), np.isnan(want[k])), k


@pytest.mark.parametrize("T", [64 * 3 + 5, 12000])
def test_growth_and_decay_to_the_ends_of_the_range(T):
    """Chunks whose sums of g go up to 88 and down by 88, in both schedules: within the oracle's bound, and 2^-145 of the
    largest state for what a chunk takes down below fp32's normal numbers (32 products, each off by 2^-150 at most)."""
    p = make([T], 40, "f32", "f32", "none", h0=False, seed=66)
    rise = (torch.arange(T) // 32 % 2 == 0)[:, None]
    p["g"] = torch.where(rise, 2.75, -2.75).expand(T, 40).contiguous()
    p["x"] = p["x"] * 1e-3
    p["x"][:31, 5] = 0.0                # a zero state and a zero sum up to the chunk's last token
    n, (o, hT) = kernels(lambda: prefill(p))
    assert n["k_lru_fold"] == (T > 2048)
    ro, rh, eo, eh = lru_fwd(np64(p["x"]), np64(p["g"]), [0, T], "none")
    lost = 2.0 ** -145 * np.abs(ro).max(0)
    check(o, ro, eo + lost, "o")
    check(hT, rh, eh + lost, "hT")
    assert float(o[:31, 5].abs().max()) == 0.0 and same(o[31, 5], p["x"][31, 5].cuda())
    assert float(o.abs().max()) > 1e33


@pytest.mark.parametrize("long", [False, True])
def test_gradient_of_a_growing_chunk(long):
    """One chunk whose g sums to 88, alone and next to a sequence past a round, in both trainer schedules."""
    lens = [32] + ([1100] if long else [])
    p = make(lens, 8, "f32", "f32", "none", seed=67)
    p["g"][:32] = 2.75
    for k in ("x", "dO", "h0", "dhT"):
        p[k] = p[k] * 1e-3
    d = dev(p)
    n, r = kernels(lambda: B.gdn_lru_fwd_bwd(p["shape"], d["x"], d["g"], d["cu"], d["dO"], h0=d["h0"], dhT=d["dhT"]))
    assert n["k_lru_grad"] == long
    want, bound = lru_bwd(np64(p["x"]), np64(p["g"]), p["cu"].tolist(), "none", np64(p["dO"]), np64(p["h0"]), np64(p["dhT"]))
    for k in ("dx", "dg", "dh0"):
        check(r[k], want[k], bound[k], k)
    assert float(r["dh0"][0].abs().max()) > 1e32


def test_a_state_that_a_chunk_takes_below_the_normal_numbers():
    p = make([32], 4, "f32", "f32", "none", seed=68)
    p["g"].fill_(float(np.log(0.03)))
    p["x"].zero_()
    p["h0"] = torch.tensor([[1e30, -1e25, 1.0, 3e38]])
    o, _ = prefill(p)
    ro, _, eo, _ = lru_fwd(np64(p["x"]), np64(p["g"]), [0, 32], "none", np64(p["h0"]))
    check(o, ro, eo + 2.0 ** -145 * np.abs(np64(p["h0"])), "o")


def test_weights_at_the_smallest_decays():
    """b = 1 - alpha and sqrt(1 - alpha^2) for |g| down to 2^-126; the root's is 0 for the few values below."""
    g = -torch.tensor([[2.0 ** -126, 1.5 * 2.0 ** -126, 1e-37, 1e-30, 1e-20, 1e-8, 3e-5, 0.01]])
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    x, gd = torch.ones(1, 8, device="cuda"), g.cuda()
    for gate in ("complement", "norm"):
        o, _ = B.gdn_lru_prefill(B.make_lru_shape(8, F32, F32, gate), x, gd, cu)
        ro, _, eo, _ = lru_fwd(np.ones((1, 8)), np64(g), [0, 1], gate)
        off = np.abs(np64(o) - ro)
        assert (off <= eo + 2.0 ** -24 * ro + 2.0 ** -148).all(), (gate, off / ro)
    tiny = -torch.tensor([[0.0, 1e-45, 1e-40, 2.0 ** -128]]).repeat(1, 2).cuda()
    s = B.make_lru_shape(8, F32, F32, "norm")
    o, _ = B.gdn_lru_prefill(s, x, tiny, cu)
    r = B.gdn_lru_fwd_bwd(s, x, tiny, cu, x)
    assert bool((o == 0).all()) and bool((r["dg"] == 0).all()) and bool((r["dx"] == 0).all())


def test_trainer_of_more_sequences_and_channels_than_narrow_chains_hold():
    """32768 sequences x 4096 channels, whose chains take 256 channels a block: the long one and its neighbours alone, and the
    last ones, give the same bits."""
    N, D = 32768, 4096
    lens = [1100] + [1] * (N - 1)
    T = sum(lens)
    gen = torch.Generator(device="cuda").manual_seed(69)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x, g, dO, h0, dhT = rn(T, D).bfloat16(), -rn(T, D).abs().bfloat16(), rn(T, D).bfloat16(), rn(N, D), rn(N, D)
    cu = torch.zeros(N + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(lens, dtype=torch.int64), 0)
    s = B.make_lru_shape(D, BF16, BF16, "norm")
    n, many = kernels(lambda: B.gdn_lru_fwd_bwd(s, x, g, cu.cuda(), dO, h0=h0, dhT=dhT, cu_seqlens_host=cu))
    assert n["k_lru_chain"] == n["k_lru_grad"] == 1
    few = B.gdn_lru_fwd_bwd(s, x[:1103], g[:1103], cu[:5].cuda(), dO[:1103], h0=h0[:4], dhT=dhT[:4])
    for key, t in few.items():
        assert same(t, many[key][:t.shape[0]]), key
    end = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
    last = B.gdn_lru_fwd_bwd(s, x[-3:].clone(), g[-3:].clone(), end, dO[-3:].clone(), h0=h0[-3:].clone(), dhT=dhT[-3:].clone())
    for key, t in last.items():
        assert same(t, many[key][-3:]), key


def test_short_sequences_next_to_long_ones_in_a_row():
    """Many short sequences with long neighbours, whose one pass would run them one after another: the same bits as in three
    batches, from the start and continued."""
    lens, D = [20] * 200 + [2000] * 8 + [0, 7], 96
    p = make(lens, D, "bf16", "f32", "complement", seed=70)
    d, cu, N = dev(p), p["cu"].tolist(), len(lens)
    n, (o, hT) = kernels(lambda: prefill(p))
    assert n["k_lru_fold"] == 1 and n["k_lru_fwd"] == 0
    for a, b in ((0, 40), (200, 203), (205, N)):
        r = slice(cu[a], cu[b])
        c = torch.tensor([v - cu[a] for v in cu[a:b + 1]], dtype=torch.int32, device="cuda")
        o1, h1 = B.gdn_lru_prefill(p["shape"], d["x"][r].clone(), d["g"][r].clone(), c, h0=d["h0"][a:b].clone())
        assert same(o1, o[r]) and same(h1, hT[a:b]), (a, b)
    cache, cut = B.gdn_lru_cache_init(p["shape"], N, "cuda", h0=d["h0"]), [min(v, 11 * (i % 5)) for i, v in enumerate(lens)]
    for at, to in (([0] * N, cut), (cut, lens)):
        rows = torch.cat([torch.arange(cu[i] + at[i], cu[i] + to[i]) for i in range(N)]).cuda()
        c = torch.tensor([0] + list(np.cumsum([j - i for i, j in zip(at, to)])), dtype=torch.int32, device="cuda")
        got, last = B.gdn_lru_prefill_continue(p["shape"], d["x"][rows], d["g"][rows], c, cache)
        assert same(got, o[rows])
    assert same(last, hT)


def test_no_host_copy():
    """cu_seqlens_host=False, as gdn_prefill takes it."""
    p = make([33, 0, 2500], 16, seed=71)
    d = dev(p)
    want, hT = prefill(p, cu_seqlens_host=p["cu"])
    o, h = prefill(p, cu_seqlens_host=False)
    r = B.gdn_lru_fwd_bwd(p["shape"], d["x"], d["g"], d["cu"], d["dO"], h0=d["h0"], cu_seqlens_host=False)
    assert same(o, want) and same(h, hT) and same(r["o"], want)
    cache = B.gdn_lru_cache_init(p["shape"], 3, "cuda", h0=d["h0"])
    assert same(B.gdn_lru_prefill_continue(p["shape"], d["x"], d["g"], d["cu"], cache, cu_seqlens_host=False)[0], want)


@pytest.mark.parametrize("x,g,gate,D", [("bf16", "f32", "norm", 300), ("f32", "f32", "none", 33), ("bf16", "bf16", "complement", 64)])
def test_decoded_states_are_the_prefills(x, g, gate, D):
    """A continuation without tokens gives the states: after token-by-token decode, after a prefill into a cache and by that
    prefill itself the same bits; A S + B in two roundings is next to them."""
    lens = [1, 40, 97, 32, 64, 130]
    p = make(lens, D, x, g, gate, seed=72)
    p["g"] = (p["g"].float() / 16).to(DT[g])     # slow decays: A S counts in the sum
    d, cu, N = dev(p), p["cu"].tolist(), len(lens)
    none, zeros = torch.zeros(N + 1, dtype=torch.int32, device="cuda"), (d["x"][:0], d["g"][:0])
    filled = B.LruCache(D, N, "cuda")
    _, hT = prefill(p, cache=filled)
    assert same(B.gdn_lru_prefill_continue(p["shape"], *zeros, none, filled)[1], hT)
    cache, seen = B.gdn_lru_cache_init(p["shape"], N, "cuda", h0=d["h0"]), 0
    for t in range(max(lens)):
        rows = torch.tensor([min(cu[n] + t, cu[n + 1] - 1) for n in range(N)], device="cuda")
        o = B.gdn_lru_decode_step(p["shape"], d["x"][rows], d["g"][rows], cache)
        _, now = B.gdn_lru_prefill_continue(p["shape"], *zeros, none, cache)
        if x == "f32":
            assert same(now, o), t
        for n in range(N):
            if t == lens[n] - 1:
                assert same(now[n], hT[n]), n
                seen += 1
        two = cache.A.double().abs() * cache.S.double().abs() + cache.B.double().abs()
        # a product, a sum and the fma, each off by 2^-24 of at most |A S| + |B| (and of the roundings before)
        assert bool(((cache.state().double() - now.double()).abs() <= 3.001 * 2.0 ** -24 * two + 2.0 ** -126).all()), t
    assert seen == N


# ---- both schedules: [6000, 45] tokens x 40 channels takes the three steps, [40, 45] the one pass ----
BOTH = [([40, 45], False), ([6000, 45], True)]


def launched(long, n, forward, train):
    """Whether n's launches are those of the three steps (long) or of the one pass, for the calls that ran."""
    want = dict.fromkeys(n, 0)
    if long:
        want.update(k_lru_fold=forward + train, k_lru_chain=forward + train, k_lru_apply=forward, k_lru_grad=train)
    else:
        want.update(k_lru_fwd=forward, k_lru_train=train)
    want["k_lru_pos"] = n["k_lru_pos"]
    return n == want


@pytest.mark.parametrize("lens,long", BOTH)
def test_poisoned_buffers_in_both_schedules(lens, long):
    p = make(lens, 40, "bf16", "f32", "norm", seed=73)
    d, T, N = dev(p), sum(lens), len(lens)
    begin = B.LruCache(40, N, "cuda")
    prefill(dict(p, x=p["x"][:50], g=p["g"][:50], cu=torch.tensor([0, 17, 50], dtype=torch.int32)), cache=begin)
    res = []
    for fill in (0xFF, 0x00, 0x7F):
        ws = lambda op: torch.full((B.lru_workspace_bytes(p["shape"], N, T, op),), fill, dtype=torch.uint8, device="cuda")  # noqa: E731
        cache, go = B.LruCache(40, N, "cuda"), begin.clone()
        for t in cache.tensors():
            t.view(torch.uint8).fill_(fill)
        out = torch.empty_like(d["x"])
        out.view(torch.uint8).fill_(fill)
        n, (o, h) = kernels(lambda: prefill(p, cache=cache, ws=ws(B.OP_PREFILL), out=out))
        assert launched(long, n, 1, 0)
        n, (c, hc) = kernels(lambda: B.gdn_lru_prefill_continue(p["shape"], d["x"], d["g"], d["cu"], go,
                                                                ws=ws(B.OP_PREFILL_CONTINUE)))
        assert launched(long, n, 1, 0)
        n, r = kernels(lambda: B.gdn_lru_fwd_bwd(p["shape"], d["x"], d["g"], d["cu"], d["dO"], h0=d["h0"], ws=ws(B.OP_FWD_BWD)))
        assert launched(long, n, 0, 1)
        res.append([o, h, c, hc, *cache.tensors(), *go.tensors(), *[r[k] for k in sorted(r)]])
    for other in res[1:]:
        for a, b in zip(res[0], other):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("lens,long", BOTH)
def test_offsets_past_32_bits_in_both_schedules(lens, long):
    """Rows that span more than 2^32 elements, for every row that the prefill, the continuation, the trainer and a decode step
    take."""
    p = make(lens, 40, "bf16", "bf16", "norm", seed=74)
    d, T = dev(p), sum(lens)
    ld = (1 << 20) if long else (1 << 26)
    big = torch.empty(T, ld, dtype=BF16, device="cuda")
    assert (T - 1) * ld > 1 << 32
    cols = {k: big[:, i * 64:i * 64 + 40] for i, k in enumerate(("x", "g", "dO", "o", "dx", "dg"))}
    for k in ("x", "g", "dO"):
        cols[k].copy_(d[k])
    caches = [B.LruCache(40, 2, "cuda") for _ in range(2)]
    n, (o, h) = kernels(lambda: B.gdn_lru_prefill(p["shape"], cols["x"], cols["g"], d["cu"], h0=d["h0"], cache=caches[0],
                                                  out=cols["o"]))
    assert launched(long, n, 1, 0)
    want, hT = prefill(p, cache=caches[1])
    assert same(o, want) and same(h, hT)
    n, (o, h) = kernels(lambda: B.gdn_lru_prefill_continue(p["shape"], cols["x"], cols["g"], d["cu"], caches[0], out=cols["o"]))
    assert launched(long, n, 1, 0)
    want, hT = B.gdn_lru_prefill_continue(p["shape"], d["x"], d["g"], d["cu"], caches[1])
    assert same(o, want) and same(h, hT)
    for a, b in zip(*(c.tensors() for c in caches)):
        assert torch.equal(a.view(torch.int32), b.view(torch.int32))
    want = B.gdn_lru_fwd_bwd(p["shape"], d["x"], d["g"], d["cu"], d["dO"], h0=d["h0"])
    n, r = kernels(lambda: B.gdn_lru_fwd_bwd(p["shape"], cols["x"], cols["g"], d["cu"], cols["dO"], h0=d["h0"],
                                             out={k: cols[k] for k in ("o", "dx", "dg")}))
    assert launched(long, n, 0, 1)
    for k in ("o", "dx", "dg", "hT", "dh0"):
        assert same(r[k], want[k]), k
    one, two = (B.gdn_lru_cache_init(p["shape"], T, "cuda") for _ in range(2))
    assert same(B.gdn_lru_decode_step(p["shape"], cols["x"], cols["g"], one, out=cols["o"]),
                B.gdn_lru_decode_step(p["shape"], d["x"], d["g"], two))


@pytest.mark.parametrize("long", [False, True])
def test_no_nan_crosses_into_another_sequences_gradient_in_both_schedules(long):
    lens = [70, 40, 33, 64, 100, 20] + ([1100] if long else [])
    p = make(lens, 6, "f32", "f32", "complement", seed=75)
    cu, d = p["cu"].tolist(), dev(p)

    def train():
        n, r = kernels(lambda: B.gdn_lru_fwd_bwd(p["shape"], d["x"], d["g"], d["cu"], d["dO"], h0=d["h0"], dhT=d["dhT"]))
        assert launched(long, n, 0, 1)
        return r
    want = train()
    payload = torch.tensor([0xffc0dead - (1 << 32), 0x7fc00000, 0xffc0dead - (1 << 32), 0x7f800001, -1, 0x7fffffff], dtype=torch.int32)
    d["x"][cu[0] + 5], d["dO"][cu[2] + 1] = float("nan"), float("inf")
    d["g"][cu[1] + 36] = d["g"][cu[4] + 66] = payload.view(F32).cuda()
    got = train()
    for n in (3, 5, 6)[:2 + long]:
        for k in ("o", "dx", "dg"):
            assert same(got[k][cu[n]:cu[n + 1]], want[k][cu[n]:cu[n + 1]]), (n, k)
        assert same(got["hT"][n], want["hT"][n]) and same(got["dh0"][n], want["dh0"][n])
    for n, t in ((1, 36), (4, 66)):  # states from the NaN on, gradients up to it
        assert bool(got["o"][cu[n] + t:cu[n + 1]].isnan().all()) and bool(got["dx"][cu[n]:cu[n] + t + 1].isnan().all())
        assert bool(got["dg"][cu[n] + t].isnan().all()) and bool(got["dh0"][n].isnan().all())
        assert same(got["o"][cu[n]:cu[n] + t], want["o"][cu[n]:cu[n] + t])
        assert same(got["dx"][cu[n] + t + 1:cu[n + 1]], want["dx"][cu[n] + t + 1:cu[n + 1]])


def test_both_schedules_on_their_own_streams():
    """A call in three steps, one in one pass and a trainer call at once, each on its own stream, workspace and cache."""
    ps = [make([6000, 45], 40, "bf16", "f32", "norm", seed=76), make([40, 45], 40, "bf16", "f32", "norm", seed=77)]
    want = [prefill(p) for p in ps]
    ds = [dev(p) for p in ps]
    train = lambda d: B.gdn_lru_fwd_bwd(ps[0]["shape"], d["x"], d["g"], d["cu"], d["dO"], h0=d["h0"], cu_seqlens_host=ps[0]["cu"])  # noqa: E731
    grads = train(ds[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(3):
        got = []
        for s, (p, d) in zip(streams, zip(ps, ds)):
            with torch.cuda.stream(s):
                got.append(B.gdn_lru_prefill(p["shape"], d["x"], d["g"], d["cu"], h0=d["h0"], cu_seqlens_host=p["cu"]))
        with torch.cuda.stream(streams[2]):
            r = train(ds[0])
        torch.cuda.synchronize()
        for (o, h), (ro, rh) in zip(got, want):
            assert same(o, ro) and same(h, rh)
        assert all(same(r[k], grads[k]) for k in r)


def test_accuracy_of_the_gates():
    """alpha, 1 - alpha and sqrt(1 - alpha^2) over four million g, in units of 2^-24.  alpha: its last rounding 1, p's polynomial
    0.3, p's and q's roundings 1.4 of at most 0.42 of it, f's rounding 0.25: 2.  1 - alpha: at n = 0 p's 1.7; at n = -1, where
    it is 0.29 at least, p's 1.2, f's 0.6 and its own 1: 3.  The root: half of 1 - alpha's 3, of 1 + alpha's 2 and of the
    product's 1, and the instruction's own 2: 5."""
    D, worst = 1 << 20, {}
    gen = torch.Generator().manual_seed(80)
    g = -torch.cat([torch.exp(torch.rand(2, D, generator=gen) * 40 - 36), torch.rand(1, D, generator=gen) * 2,
                    torch.rand(1, D, generator=gen) * 104])
    cu = torch.arange(5, dtype=torch.int32, device="cuda")
    gd = g.cuda()
    ones, e = torch.ones(4, D, device="cuda"), gd.double()
    for gate, want, units in (("none", e.exp(), 2), ("complement", -e.expm1(), 3), ("norm", (-(2 * e).expm1()).sqrt(), 5)):
        s = B.make_lru_shape(D, F32, F32, gate)
        o, _ = B.gdn_lru_prefill(s, ones * (gate != "none"), gd, cu, h0=ones * (gate == "none"), cu_seqlens_host=cu.cpu())
        off = (o.double() - want).abs() - 2.0 ** -149         # a step of the denormal numbers
        worst[gate] = float((off / want).max()) * 2 ** 24
        assert worst[gate] <= units, worst
    print("units of 2^-24:", worst)
