"""The gated linear recurrence and the q/k norms with rotary positions without a
GPU: refusals of the C ABI and of the binding (every call here fails before it
touches a GPU), rotary frequencies, and the oracles against closed forms and
differences."""

import ctypes
import math

import numpy as np
import pytest
import torch

from linear_attention_rnn_gated_amd import binding as B
from oracle.lru_oracle import lru_bwd, lru_fwd
from oracle.qk_oracle import qk_bwd, qk_fwd

P = ctypes.c_void_p(16)      # an aligned address that is never followed
ODD = ctypes.c_void_p(20)


def lru_shape(**kw):
    base = dict(D=8, in_dtype=B.GDN_BF16, g_dtype=B.GDN_F32, gate=0)
    base.update(kw)
    return B.LruShape(*[base[k] for k in ("D", "in_dtype", "g_dtype", "gate")])


def lru_prefill(s, cu, x=P, ldx=0, g=P, ldg=0, h0=None, o=P, ldo=0, hT=None, cache=None, cu_dev=P, ws=P,
                ws_bytes=1 << 40):
    host = (ctypes.c_int32 * len(cu))(*cu)
    return B.lib().gdn_lru_prefill(ctypes.byref(s), len(cu) - 1, cu_dev, host, x, ldx, g, ldg, h0, o, ldo, hT,
                                   cache, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(D=0), B.GDN_ERR_INVALID_ARG),
    (dict(D=(1 << 20) + 1), B.GDN_ERR_UNSUPPORTED),
    (dict(in_dtype=2), B.GDN_ERR_UNSUPPORTED),
    (dict(g_dtype=-1), B.GDN_ERR_UNSUPPORTED),
    (dict(gate=3), B.GDN_ERR_INVALID_ARG),
])
def test_lru_shape_claims(kw, want):
    s, L = lru_shape(**kw), B.lib()
    cache = B.LruCacheStruct(16, 16, 16, 16)
    cu = (ctypes.c_int32 * 2)(0, 5)
    assert lru_prefill(s, [0, 5]) == want
    assert L.gdn_lru_cache_init(ctypes.byref(s), 1, None, ctypes.byref(cache), None) == want
    assert L.gdn_lru_decode_step(ctypes.byref(s), 1, P, 0, P, 0, ctypes.byref(cache), P, 0, None) == want
    assert L.gdn_lru_fwd_bwd(ctypes.byref(s), 1, P, cu, P, 0, P, 0, None, P, 0, None, P, 0, P, P, 0, P, 0, P, P,
                             1 << 40, None) == want
    assert L.gdn_lru_workspace_bytes(ctypes.byref(s), 1, 5, B.OP_PREFILL) == 0


def test_lru_argument_checks():
    s, L = lru_shape(), B.lib()
    bad = B.GDN_ERR_INVALID_ARG
    assert lru_prefill(s, [1, 5]) == bad
    assert lru_prefill(s, [0, 5, 4]) == bad
    assert lru_prefill(s, [0, 5], x=None) == bad
    assert lru_prefill(s, [0, 5], o=None) == bad
    assert lru_prefill(s, [0, 5], g=ODD) == bad
    assert lru_prefill(s, [0, 5], h0=ODD) == bad
    assert lru_prefill(s, [0, 5], ldx=7) == bad           # shorter than a row
    assert lru_prefill(s, [0, 5], ldo=-8) == bad
    assert lru_prefill(s, [0, 5], cu_dev=None) == bad
    assert lru_prefill(s, [0, 5], cache=ctypes.byref(B.LruCacheStruct(16, 16, None, 16))) == bad
    assert lru_prefill(s, [0, 5], cache=ctypes.byref(B.LruCacheStruct(16, 16, 20, 16))) == bad
    need = L.gdn_lru_workspace_bytes(ctypes.byref(s), 1, 2049, B.OP_PREFILL)
    assert lru_prefill(s, [0, 2049], ws=None) == B.GDN_ERR_WORKSPACE
    assert lru_prefill(s, [0, 2049], ws_bytes=need - 1) == B.GDN_ERR_WORKSPACE
    assert lru_prefill(s, [0, 5], ws=ODD) == bad
    assert lru_prefill(s, [0]) == B.GDN_OK                # no sequence, nothing to do
    cache = B.LruCacheStruct(16, 16, 16, 16)
    cb = ctypes.byref(cache)
    cu = (ctypes.c_int32 * 2)(0, 5)
    assert L.gdn_lru_prefill_continue(ctypes.byref(s), 1, P, cu, P, 0, P, 0, None, P, 0, None, P, 1 << 40, None) == bad
    assert L.gdn_lru_prefill_continue(ctypes.byref(s), -1, P, cu, P, 0, P, 0, cb, P, 0, None, P, 1 << 40, None) == bad
    step = L.gdn_lru_decode_step
    assert step(ctypes.byref(s), 1, P, 0, P, 0, cb, None, 0, None) == bad
    assert step(ctypes.byref(s), 1, P, 4, P, 0, cb, P, 0, None) == bad
    assert step(ctypes.byref(s), -1, P, 0, P, 0, cb, P, 0, None) == bad
    assert step(ctypes.byref(s), 65536, P, 0, P, 0, cb, P, 0, None) == B.GDN_ERR_UNSUPPORTED
    assert step(ctypes.byref(s), 0, P, 0, P, 0, cb, P, 0, None) == B.GDN_OK
    assert L.gdn_lru_cache_init(ctypes.byref(s), 0, None, cb, None) == B.GDN_OK
    assert L.gdn_lru_cache_init(ctypes.byref(s), -1, None, cb, None) == bad


def test_lru_trainer_checks():
    s, L = lru_shape(), B.lib()
    cu = (ctypes.c_int32 * 2)(0, 100)

    def call(ws=P, ws_bytes=1 << 40, dO=P, dx=P, dg=P, dh0=P, lddx=0, lddo=0):
        return L.gdn_lru_fwd_bwd(ctypes.byref(s), 1, P, cu, P, 0, P, 0, None, dO, lddo, None, None, 0, None, dx, lddx,
                                 dg, 0, dh0, ws, ws_bytes, None)
    size = lambda n, t, op=B.OP_FWD_BWD: L.gdn_lru_workspace_bytes(ctypes.byref(s), n, t, op)  # noqa: E731
    need = size(1, 100)
    assert need >= (100 // 32 + 2) * 8 * 4 * 3
    assert call(ws=None) == B.GDN_ERR_WORKSPACE
    assert call(ws_bytes=need - 1) == B.GDN_ERR_WORKSPACE
    for kw in (dict(dO=None), dict(dx=None), dict(dg=None), dict(dh0=None), dict(dx=ODD), dict(lddx=3), dict(lddo=-1)):
        assert call(**kw) == B.GDN_ERR_INVALID_ARG, kw
    assert size(-1, 5) == 0 and size(1, -5) == 0 and size(1, 5, B.OP_DECODE) == 0
    assert size(1, 0) > 0 and size(3, 100) > size(1, 100)


def qk_shape(**kw):
    base = dict(H_q=2, H_k=1, d=64, r=32, in_dtype=1, out_dtype=1, norm=2, layout=0, eps=1e-6, scale=1.0,
                rope_scale=1.0, weight_offset=0.0)
    base.update(kw)
    return B.QkShape(*[base[f[0]] for f in B.QkShape._fields_])


def qk_call(s, T=3, pos=P, n=0, cu=None, start=None, freq=P, w_q=None, w_k=None, q=P, ldq=0, k=P, ldk=0, qo=P, ldqo=0,
            ko=P, ldko=0):
    return B.lib().gdn_qk_rotary(ctypes.byref(s), T, pos, n, cu, start, freq, w_q, w_k, q, ldq, k, ldk, qo, ldqo, ko,
                                 ldko, None)


def qk_grad(s, T=3, ws=P, ws_bytes=1 << 40, dw=P, dq=P, dko=P, lddq=0, w_q=None):
    return B.lib().gdn_qk_rotary_bwd(ctypes.byref(s), T, P, 0, None, None, P, w_q, None, P, 0, P, 0, P, 0, dko, 0, dq,
                                     lddq, P, 0, dw, dw, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(d=0), B.GDN_ERR_INVALID_ARG),
    (dict(d=60, r=0), B.GDN_ERR_UNSUPPORTED),
    (dict(d=520), B.GDN_ERR_UNSUPPORTED),
    (dict(r=20), B.GDN_ERR_UNSUPPORTED),
    (dict(r=72), B.GDN_ERR_INVALID_ARG),
    (dict(H_q=0), B.GDN_ERR_INVALID_ARG),
    (dict(H_k=-1), B.GDN_ERR_INVALID_ARG),
    (dict(H_q=5000), B.GDN_ERR_UNSUPPORTED),
    (dict(in_dtype=3), B.GDN_ERR_UNSUPPORTED),
    (dict(out_dtype=3), B.GDN_ERR_UNSUPPORTED),
    (dict(norm=3), B.GDN_ERR_INVALID_ARG),
    (dict(layout=2), B.GDN_ERR_INVALID_ARG),
    (dict(eps=-1.0), B.GDN_ERR_INVALID_ARG),
    (dict(scale=float("inf")), B.GDN_ERR_INVALID_ARG),
    (dict(rope_scale=float("nan")), B.GDN_ERR_INVALID_ARG),
])
def test_qk_shape_claims(kw, want):
    s = qk_shape(**kw)
    assert qk_call(s) == want
    assert qk_grad(s) == want
    assert B.lib().gdn_qk_workspace_bytes(ctypes.byref(s), 3) == 0


def test_qk_argument_checks():
    s, bad = qk_shape(), B.GDN_ERR_INVALID_ARG
    for kw in (dict(T=-1), dict(pos=None), dict(pos=None, cu=P, n=0), dict(pos=ODD), dict(freq=None), dict(q=None),
               dict(k=None), dict(qo=None), dict(ko=None), dict(qo=ODD), dict(ldq=127), dict(ldq=132), dict(ldko=-8),
               dict(ldqo=129), dict(n=-1)):
        assert qk_call(s, **kw) == bad, kw
    assert qk_call(qk_shape(norm=1), w_q=P) == bad        # weights without the weighted norm
    assert qk_call(s, T=1 << 31) == B.GDN_ERR_UNSUPPORTED
    assert qk_call(s, T=0) == B.GDN_OK
    need = B.lib().gdn_qk_workspace_bytes(ctypes.byref(s), 3)
    assert need >= 2 * 64 * 4
    assert qk_grad(s, ws=None) == B.GDN_ERR_WORKSPACE
    assert qk_grad(s, ws_bytes=need - 1) == B.GDN_ERR_WORKSPACE
    assert qk_grad(s, dq=None) == bad
    assert qk_grad(s, dko=None) == bad
    assert qk_grad(s, lddq=68) == bad
    assert qk_grad(qk_shape(norm=0)) == bad               # weight gradients without weights


def test_binding_refuses_tensors_off_the_gpu():
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    g = torch.zeros(4, 8)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    s = B.make_lru_shape(8, torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        B.gdn_lru_prefill(s, x, g, cu)
    with pytest.raises(ValueError, match="GPU"):
        B.gdn_lru_fwd_bwd(s, x, g, cu, x)
    with pytest.raises(ValueError, match="GPU"):
        B.gdn_lru_decode_step(s, x, g, None)
    with pytest.raises(ValueError, match="GPU"):
        B.LruCache.of(g, g, g, torch.zeros(4, 1, dtype=torch.int32))
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        B.gdn_qk_rotary(B.make_qk_shape(2, 2, 64, 0, torch.bfloat16), q, q, None, cu_seqlens=cu)


def test_binding_checks_strides_and_shapes():
    dev = torch.device("cpu")
    t = torch.zeros(6, 20)
    assert B._rows(t[:, 4:12], torch.float32, 6, 8, dev, "x") == 20
    assert B._rows(t[:1, 4:12], torch.float32, 1, 8, dev, "x") == 8
    for bad in (t[:, ::2], t.expand(6, 20)[:, :8].t(), t[:1, :8].expand(6, 8), t[:, :7], t[:, :8].double()):
        with pytest.raises(ValueError):
            B._rows(bad, torch.float32, 6, 8, dev, "x")
    q = torch.zeros(5, 48)
    assert B._heads(q[:, 16:32].unflatten(1, (2, 8)), torch.float32, 5, 2, 8, dev, "q") == 48
    for bad in (torch.zeros(5, 8, 2).transpose(1, 2), torch.zeros(2, 5, 8).transpose(0, 1),
                torch.zeros(1, 2, 8).expand(5, 2, 8)):
        with pytest.raises(ValueError):
            B._heads(bad, torch.float32, 5, 2, 8, dev, "q")
    with pytest.raises(ValueError):
        B._packed(torch.tensor([0, 9], dtype=torch.int32), None, dev, 8)
    with pytest.raises(ValueError):
        B._packed(torch.tensor([0, 9], dtype=torch.int32), False, dev, 9)


def test_calls_run_on_their_tensors_gpu(monkeypatch):
    """_launch makes the tensors' GPU current for the call where another one is, and takes that GPU's current stream."""
    log = []

    class Guard:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            log.append(("enter", self.dev.index))

        def __exit__(self, *a):
            log.append(("exit", self.dev.index))

    class Lib:
        @staticmethod
        def gdn_lru_decode_step(*args):
            log.append(("call", args))
            return B.GDN_OK
    monkeypatch.setattr(B, "_lib", Lib)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 100 + i, raising=False)
    monkeypatch.setattr(torch.cuda, "device", Guard)
    B._launch("gdn_lru_decode_step", torch.device("cuda", 0), 1)
    assert log == [("call", (1, 100))]
    log.clear()
    B._launch("gdn_lru_decode_step", torch.device("cuda", 1), 1)
    assert log == [("enter", 1), ("call", (1, 101)), ("exit", 1)]


# ---- rotary frequencies: the formulas written out ------------------------------


def test_rope_freqs_plain_linear_ntk():
    for r, base in ((2, 10000.0), (64, 10000.0), (128, 1e6)):
        i = np.arange(r // 2)
        f, c = B.rope_freqs(r, base)
        assert c == 1.0
        want = base ** (-2.0 * i / r)
        # formed in fp64 (pow and division, a few 2^-53) and rounded to fp32 once
        assert np.all(np.abs(f.numpy() - want) <= want * (2.0 ** -24 + 2.0 ** -50))
        f, c = B.rope_freqs(r, base, "linear", 4.0)
        assert c == 1.0 and np.all(np.abs(f.numpy() - want / 4) <= want / 4 * (2.0 ** -24 + 2.0 ** -50))
        if r > 2:
            f, _ = B.rope_freqs(r, base, "ntk", 8.0)
            want = (base * 8.0 ** (r / (r - 2))) ** (-2.0 * i / r)
            assert np.all(np.abs(f.numpy() - want) <= want * (2.0 ** -24 + 2.0 ** -48))


@pytest.mark.parametrize("kind", ["yarn", "bands"])
def test_rope_freqs_blended(kind):
    r, base, factor, orig, low, high = 128, 10000.0, 16.0, 4096.0, 1.0, 32.0
    f, c = B.rope_freqs(r, base, kind, factor, orig, low, high)
    f = f.double().numpy()
    plain = base ** (-2.0 * np.arange(r // 2) / r)
    turns = orig * plain / (2 * math.pi)
    near = lambda a, b: np.all(np.abs(a - b) <= b * 2.0 ** -23)  # noqa: E731
    pad = 2 if kind == "yarn" else 0     # the blend's ends are whole indices there
    keeps, scales = np.nonzero(turns >= high)[0], np.nonzero(turns <= low)[0]
    assert len(keeps) > 4 and len(scales) > 4
    assert near(f[keeps[:len(keeps) - pad]], plain[keeps[:len(keeps) - pad]])
    assert near(f[scales[pad:]], plain[scales[pad:]] / factor)
    share = (f / plain - 1 / factor) / (1 - 1 / factor)
    assert np.all(np.diff(share) <= 2e-6)
    if kind == "bands":
        mid = (turns > low) & (turns < high)
        assert np.allclose(share[mid], (turns[mid] - low) / (high - low), atol=2e-6)
        assert c == 1.0
    else:
        first = math.floor(r * math.log(orig / (high * 2 * math.pi)) / (2 * math.log(base)))
        last = math.ceil(r * math.log(orig / (low * 2 * math.pi)) / (2 * math.log(base)))
        want = 1 - np.clip((np.arange(r // 2) - first) / (last - first), 0, 1)
        assert np.allclose(share, want, atol=2e-6)
        assert abs(c - (0.1 * math.log(16.0) + 1)) < 1e-6
    assert B.rope_freqs(r, base, kind, factor, orig, low, high, attn=1.5)[1] == 1.5


@pytest.mark.parametrize("kw", [
    dict(r=3), dict(r=0), dict(r=-2), dict(base=1.0), dict(base=float("nan")), dict(kind="linear", factor=0.5),
    dict(kind="linear", factor=float("inf")), dict(kind="ntk", factor=2.0, r=2), dict(kind="yarn", factor=2.0),
    dict(kind="bands", factor=2.0, orig_len=100.0, low=4.0, high=4.0),
    dict(kind="yarn", factor=2.0, orig_len=100.0, attn=-1.0),
])
def test_rope_freqs_refusals(kw):
    kw = dict(dict(r=64), **kw)
    with pytest.raises(B.GdnError):
        B.rope_freqs(**kw)


def test_rope_freqs_refuses_unknown_kind_and_null():
    L = B.lib()
    s = B.RopeScaling(5, 1.0, 1.0, 1.0, 2.0, 0.0)
    buf, c = (ctypes.c_float * 4)(), ctypes.c_float()
    assert L.gdn_rope_freqs(8, 1e4, ctypes.byref(s), buf, ctypes.byref(c)) == B.GDN_ERR_INVALID_ARG
    assert L.gdn_rope_freqs(8, 1e4, None, None, ctypes.byref(c)) == B.GDN_ERR_INVALID_ARG
    assert L.gdn_rope_freqs(8, 1e4, None, buf, None) == B.GDN_ERR_INVALID_ARG
    assert L.gdn_rope_freqs(8, 1e4, None, buf, ctypes.byref(c)) == B.GDN_OK


# ---- the oracles ---------------------------------------------------------------


@pytest.mark.parametrize("gate", ["none", "complement", "norm"])
def test_lru_oracle_gradient_by_differences(gate):
    rng = np.random.default_rng(3)
    cu = [0, 5, 5, 12]
    x, g = rng.normal(size=(12, 3)), -np.abs(rng.normal(size=(12, 3))) - 0.05
    h0, dO, dhT = rng.normal(size=(3, 3)), rng.normal(size=(12, 3)), rng.normal(size=(3, 3))

    def loss(x, g, h0):
        o, hT, _, _ = lru_fwd(x, g, cu, gate, h0)
        return (o * dO).sum() + (hT * dhT).sum()
    r, _ = lru_bwd(x, g, cu, gate, dO, h0, dhT)
    for name, t, at in (("dx", x, 0), ("dg", g, 1), ("dh0", h0, 2)):
        for i in np.ndindex(t.shape):
            args = [x.copy(), g.copy(), h0.copy()]
            args[at][i] += 1e-6
            up = loss(*args)
            args[at][i] -= 2e-6
            # central difference: eps^2 truncation, 1e-16 / eps rounding of a loss of order 10
            assert abs((up - loss(*args)) / 2e-6 - r[name][i]) < 1e-7, (name, i)


def test_lru_oracle_closed_forms():
    # constant decay without input: h_t = a^t h0; a reset forgets the past; "complement" keeps a constant input's mean
    g, h0 = np.full((6, 1), math.log(0.5)), np.array([[3.0]])
    o, hT, _, _ = lru_fwd(np.zeros((6, 1)), g, [0, 6], "none", h0)
    assert np.allclose(o[:, 0], 3.0 * 0.5 ** np.arange(1, 7)) and np.allclose(hT, o[-1:])
    g[3] = -np.inf
    o, _, _, _ = lru_fwd(np.ones((6, 1)), g, [0, 6], "none", h0)
    assert o[3, 0] == 1.0
    o, _, _, _ = lru_fwd(np.ones((6, 1)), g, [0, 6], "complement", np.array([[1.0]]))
    assert np.allclose(o, 1.0)


@pytest.mark.parametrize("norm", ["none", "l2", "rms"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_qk_oracle_gradient_by_differences(norm, layout):
    rng = np.random.default_rng(4)
    x, dy, w = rng.normal(size=(2, 2, 16)), rng.normal(size=(2, 2, 16)), rng.normal(size=16)
    pos, freq = [3, 70000], 10000.0 ** (-np.arange(4) / 4)
    kw = dict(norm=norm, layout=layout, r=8, pos=pos, inv_freq=freq, eps=1e-6, scale=0.3, rope_scale=1.2)
    dx, dw, _, _ = qk_bwd(x, dy, w=w, **kw)
    f = lambda x, w: (qk_fwd(x, w=w, **kw)[0] * dy).sum()  # noqa: E731
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = 1e-6
        assert abs((f(x + e, w) - f(x - e, w)) / 2e-6 - dx[i]) < 1e-7
    if norm == "rms":
        for i in range(16):
            e = np.zeros(16)
            e[i] = 1e-6
            assert abs((f(x, w + e) - f(x, w - e)) / 2e-6 - dw[i]) < 1e-7


def test_qk_oracle_rotation_is_relative():
    # the product of two rotated vectors depends on the distance of their positions alone
    rng = np.random.default_rng(5)
    a, b = rng.normal(size=(1, 1, 8)), rng.normal(size=(1, 1, 8))
    freq = 100.0 ** (-np.arange(4) / 4)
    for layout in ("half", "interleaved"):
        y = lambda v, p: qk_fwd(v, "none", layout, 8, [p], freq)[0]  # noqa: E731
        assert abs((y(a, 5) * y(b, 2)).sum() - (y(a, 1005) * y(b, 1002)).sum()) < 1e-12


# ---- the cache's tensors -------------------------------------------------------


def test_cache_follows_assigned_tensors():
    """The struct of addresses is that of the tensors which the cache holds at the call."""
    c = B.LruCache(300, 4, "cpu")
    at = lambda: tuple(getattr(c.struct(), k) for k in ("S", "A", "B", "pos"))  # noqa: E731
    now = lambda: tuple(t.data_ptr() for t in c.tensors())  # noqa: E731
    assert at() == now() and c.struct() is c.struct()
    for name in ("S", "A", "B", "pos"):
        old = getattr(c, name)
        setattr(c, name, old[[2, 0, 3, 1]])
        assert getattr(c, name).data_ptr() != old.data_ptr() and at() == now(), name
    c.B.set_(torch.zeros(4, 300))            # other memory under the same tensor
    assert at() == now()
    order = torch.tensor([1, 3])
    c.S, c.A, c.B, c.pos = (t[order] for t in c.tensors())
    c.check(B.make_lru_shape(300, torch.float32), 2, torch.device("cpu"))
    assert (c.n, c.D) == (2, 300) and at() == now()
    c.S, c.A, c.B, c.pos = (t[:1] for t in c.tensors())     # the same addresses, fewer sequences
    assert at() == now() and c.n == 1
    with pytest.raises(ValueError):
        c.check(B.make_lru_shape(300, torch.float32), 2, torch.device("cpu"))


@pytest.mark.parametrize("name,bad", [
    ("A", torch.zeros(3, 8)), ("B", torch.zeros(4, 9)), ("S", torch.zeros(4, 16)[:, ::2]), ("A", torch.zeros(4, 8).double()),
    ("pos", torch.zeros(4, 2, dtype=torch.int32)), ("pos", torch.zeros(4, 1, dtype=torch.int64)),
    ("B", torch.zeros(8, 4).t()), ("S", torch.zeros(5, 8)),
])
def test_cache_refuses_tensors_that_do_not_fit(name, bad):
    c = B.LruCache(8, 4, "cpu")
    setattr(c, name, bad)
    with pytest.raises(ValueError):
        c.struct()


def test_no_host_copy_reads_the_device_copy_back(monkeypatch):
    """cu_seqlens_host=False, as gdn_prefill takes it: the calls go on with a copy that they read back and check."""
    seen = []
    x, g = torch.zeros(5, 8), torch.zeros(5, 8)
    cu, s = torch.tensor([0, 2, 5], dtype=torch.int32), B.make_lru_shape(8, torch.float32)
    monkeypatch.setattr(B, "_gpu", lambda t, name: t.device)
    monkeypatch.setattr(B, "_launch", lambda name, dev, *args: seen.append((name, args[1], args[3])))
    for host in (False, None, cu.clone()):
        B.gdn_lru_prefill(s, x, g, cu, cu_seqlens_host=host)
        B.gdn_lru_prefill_continue(s, x, g, cu, B.LruCache(8, 2, "cpu"), cu_seqlens_host=host)
        B.gdn_lru_fwd_bwd(s, x, g, cu, x, cu_seqlens_host=host)
        with pytest.raises(ValueError, match="past the 4 rows"):
            B.gdn_lru_prefill(s, x[:4], g[:4], cu, cu_seqlens_host=host)
    assert len(seen) == 9 and all(n == 2 and p for _, n, p in seen)


def test_exp_polynomial():
    """The recurrence's p(f) = f + f^2 q(f), with the coefficients that its source holds: within 2^-25.8 of e^f - 1."""
    import os
    import re
    src = open(os.path.join(os.path.dirname(B.__file__), "csrc", "gdn_lru.hip")).read()
    body = src[src.index("LruExp lru_exp(float g)"):]
    first = float(re.search(r"float q = ([0-9.e-]+)f;", body).group(1))
    rest = [float(v) for v in re.findall(r"q = fmaf\(q, f, ([0-9.e-]+)f\);", body)]
    assert len(rest) == 4
    f = np.linspace(-math.log(2) / 2, math.log(2) / 2, 400000)
    q = np.full_like(f, float(np.float32(first)))
    for c in rest:
        q = q * f + float(np.float32(c))
    off = np.abs((f + f * f * q) / np.expm1(f) - 1)
    assert off.max() < 2.0 ** -25.8


def test_cache_is_copied_and_restored():
    """As the other cache: deep copies and pickles hold tensors of their own, and their struct is of those."""
    import copy
    import pickle
    c = B.LruCache(40, 3, "cpu")
    for t in c.tensors()[:3]:
        t.normal_()
    for make in (copy.copy, copy.deepcopy, lambda c: pickle.loads(pickle.dumps(c))):
        c.struct()
        d = make(c)
        assert tuple(getattr(d.struct(), k) for k in ("S", "A", "B", "pos")) == tuple(t.data_ptr() for t in d.tensors())
        assert all(torch.equal(a, b) for a, b in zip(c.tensors(), d.tensors()))
        assert make is copy.copy or all(a.data_ptr() != b.data_ptr() for a, b in zip(c.tensors(), d.tensors()))
