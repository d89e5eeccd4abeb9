"""Attention and the 8-bit cache without a GPU: refusals of the C ABI and of the
binding (every call here fails before it touches a GPU), workspace sizes, and the
oracle against closed forms, differences and another e4m3."""

import ctypes

import numpy as np
import pytest
import torch

from linear_attention_rnn_gated_amd import binding as B
from oracle import attn_oracle as A

P = ctypes.c_void_p(16)      # an aligned address that is never followed
ODD = ctypes.c_void_p(20)
OFF = ctypes.c_void_p(18)    # not even an int32's address
BAD, UNS, WS = B.GDN_ERR_INVALID_ARG, B.GDN_ERR_UNSUPPORTED, B.GDN_ERR_WORKSPACE
BIG = 1 << 40


def shape(**kw):
    base = dict(H_q=4, H_kv=2, d=128, in_dtype=B.GDN_BF16, scale=0.1)
    base.update(kw)
    return B.AttnShape(*[base[k] for k in ("H_q", "H_kv", "d", "in_dtype", "scale")])


def cache(**kw):
    base = dict(k=16, v=16, k_scale=16, v_scale=16, pages=4, page_tokens=64)
    base.update(kw)
    return B.KvCacheStruct(*[base[k] for k in ("k", "v", "k_scale", "v_scale", "pages", "page_tokens")])


def prefill(s, N=1, cu_q=P, cu_k=None, T_q=5, T_k=5, q=P, ldq=0, k=P, ldk=0, v=P, ldv=0, o=P, ldo=0, lse=P):
    return B.lib().gdn_attn_prefill(ctypes.byref(s), N, cu_q, cu_k, T_q, T_k, q, ldq, k, ldk, v, ldv, o, ldo, lse, None)


def bwd(s, N=1, cu_q=P, cu_k=None, T_q=5, T_k=5, q=P, o=P, ldo=0, lse=P, dO=P, dq=P, dk=P, dv=P, lddk=0, ws=P,
        ws_bytes=BIG):
    return B.lib().gdn_attn_bwd(ctypes.byref(s), N, cu_q, cu_k, T_q, T_k, q, 0, P, 0, P, 0, o, ldo, lse, dO, 0, dq, 0,
                                dk, lddk, dv, 0, ws, ws_bytes, None)


def write(s, c, N=1, cu=P, start=None, T=5, k=P, ldk=0, v=P, table=P, width=3):
    return B.lib().gdn_kv_write(ctypes.byref(s), N, cu, start, T, k, ldk, v, 0, ctypes.byref(c) if c else None, table,
                                width, None)


def read(s, c, N=1, cu=P, T=5, k=P, v=P, ldv=0, table=P, width=3):
    return B.lib().gdn_kv_read(ctypes.byref(s), N, cu, None, T, ctypes.byref(c) if c else None, table, width, k, 0, v,
                               ldv, None)


def decode(s, c, N=1, cu=P, T=5, q=P, ldq=0, table=P, width=300, kv_len=P, max_len=9000, o=P, ldo=0, lse=None, ws=P,
           ws_bytes=BIG):
    return B.lib().gdn_attn_decode(ctypes.byref(s), N, cu, T, q, ldq, ctypes.byref(c) if c else None, table, width,
                                   kv_len, max_len, o, ldo, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(H_q=0), BAD), (dict(H_kv=0), BAD), (dict(d=0), BAD), (dict(scale=0.0), BAD), (dict(scale=-1.0), BAD),
    (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD), (dict(H_q=3), UNS), (dict(H_q=8192), UNS),
    (dict(d=96), UNS), (dict(d=512), UNS), (dict(in_dtype=2), UNS), (dict(scale=2.0 ** 127), UNS),
])
def test_shape_claims(kw, want):
    s, c, L = shape(**kw), cache(), B.lib()
    assert prefill(s) == want and bwd(s) == want and write(s, c) == want and read(s, c) == want
    assert decode(s, c) == want
    assert L.gdn_attn_workspace_bytes(ctypes.byref(s), 5, 5) == 0
    assert L.gdn_attn_decode_workspace_bytes(ctypes.byref(s), 1, 5, 9000) == 0


def test_prefill_argument_checks():
    s = shape()
    for kw in (dict(N=-1), dict(T_q=-1), dict(T_k=-1), dict(cu_q=None), dict(N=0), dict(T_k=6), dict(q=None),
               dict(k=None), dict(v=None), dict(o=None), dict(q=ODD), dict(k=ODD), dict(v=ODD), dict(o=ODD),
               dict(lse=OFF), dict(cu_q=OFF), dict(cu_k=OFF), dict(ldq=504), dict(ldq=516), dict(ldk=248),
               dict(ldv=260), dict(ldo=8)):
        assert prefill(s, **kw) == BAD, kw
    assert prefill(s, T_q=1 << 31, T_k=1 << 31) == UNS
    assert prefill(s, ldq=(1 << 22) + 8) == UNS and prefill(s, ldo=(1 << 22) + 8) == UNS
    assert prefill(s, N=0, T_q=0, T_k=0) == B.GDN_OK


def test_bwd_argument_checks():
    s = shape()
    for kw in (dict(N=-1), dict(cu_q=None), dict(o=None), dict(lse=None), dict(dO=None), dict(dq=None), dict(dk=None),
               dict(dv=None), dict(o=ODD), dict(lse=OFF), dict(dO=ODD), dict(dq=ODD), dict(dk=ODD), dict(dv=ODD),
               dict(ws=ODD), dict(ldo=8), dict(lddk=250)):
        assert bwd(s, **kw) == BAD, kw
    need = B.attn_workspace_bytes(s, 5, 5)
    assert need > 0 and bwd(s, ws=None) == WS and bwd(s, ws_bytes=need - 1) == WS
    assert bwd(s, N=0, T_q=0, T_k=0) == B.GDN_OK


def test_cache_argument_checks():
    s = shape()
    for call in (write, read, decode):
        assert call(s, None) == BAD
        for kw, want in ((dict(k=None), BAD), (dict(v_scale=None), BAD), (dict(k=20), BAD), (dict(k_scale=24), BAD),
                         (dict(pages=0), BAD), (dict(page_tokens=0), BAD), (dict(page_tokens=48), UNS),
                         (dict(page_tokens=1 << 21), UNS)):
            assert call(s, cache(**kw)) == want, (call, kw)
        c = cache()
        for kw in (dict(N=-1), dict(T=-1), dict(N=0), dict(cu=None), dict(cu=OFF), dict(table=None), dict(table=OFF),
                   dict(width=-1)):
            assert call(s, c, **kw) == BAD, (call, kw)
        assert call(s, c, T=1 << 31) == UNS
        assert call(s, c, N=0, T=0) == B.GDN_OK and call(s, c, N=0, T=0, cu=None) == B.GDN_OK
    c = cache()
    assert write(s, c, k=None) == BAD and write(s, c, start=OFF) == BAD and write(s, c, ldk=100) == BAD
    assert read(s, c, v=None) == BAD and read(s, c, ldv=100) == BAD
    for kw in (dict(q=None), dict(o=None), dict(kv_len=None), dict(q=ODD), dict(o=ODD), dict(kv_len=OFF), dict(lse=OFF),
               dict(ws=ODD), dict(max_len=-1), dict(ldq=8), dict(ldo=516)):
        assert decode(s, c, **kw) == BAD, kw
    assert decode(s, c, max_len=1 << 31) == UNS
    need = B.attn_decode_workspace_bytes(s, 1, 5, 9000)
    assert decode(s, c, ws=None) == WS and decode(s, c, ws_bytes=1 << 10) == WS and need > 1 << 10
    assert write(s, c, width=0, table=None) == B.GDN_OK  # no page: every write is dropped


def test_workspace_sizes():
    s = shape(H_q=32, H_kv=8)
    assert B.attn_decode_workspace_bytes(s, 64, 64, 512) > 0
    # one token a sequence: a row of results for each head and split
    assert B.attn_decode_workspace_bytes(s, 64, 64, 8192) == (64 * 32 * 16 * 130 * 4 // 256 + 1) * 256
    # many tokens: a share for each sequence, not a split for each row
    assert B.attn_decode_workspace_bytes(s, 1, 16384, 131072) < 16384 * 32 * 130 * 4 * 2
    assert B.attn_workspace_bytes(s, 32768) < 10 << 20
    # few keys: partial sums of a group's heads
    assert B.attn_workspace_bytes(s, 128) >= 4 * 2 * 128 * 8 * 128 * 4


def test_binding_needs_gpu_tensors():
    s = B.make_attn_shape(4, 2, 64, torch.bfloat16)
    q, k = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 3], dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU tensor"):
        B.gdn_attn_prefill(s, q, k, k, cu)
    with pytest.raises(ValueError, match="multiple of 32"):
        B.KvCache(s, 2, 48, "cpu")
    with pytest.raises(ValueError, match="GPU tensor"):
        B.KvCache.of(*B.KvCache(s, 2, 64, "cpu").tensors())
    assert s.scale == pytest.approx(1 / 8)


def test_oracle_attention_closed_forms():
    rng = np.random.default_rng(1)
    k = np.zeros((5, 1, 64))
    v = rng.standard_normal((5, 1, 64))
    o, lse, _, _ = A.attn_fwd(rng.standard_normal((5, 2, 64)), k, v, 1.0, 0.0)  # equal scores: running means
    want = np.cumsum(v[:, 0], axis=0) / np.arange(1, 6)[:, None]
    assert np.allclose(o[:, 0], want) and np.allclose(o[:, 1], want)
    assert np.allclose(lse, np.log(np.arange(1, 6))[:, None])
    o, lse, _, _ = A.attn_fwd(rng.standard_normal((5, 2, 64)), k[:2], v[:2], 1.0, 0.0)  # three queries see nothing
    assert not o[:3].any() and np.isneginf(lse[:3]).all() and np.allclose(o[3], v[0, 0]) and np.isfinite(lse[3:]).all()


def test_oracle_gradient_by_differences():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((4, 2, 8)), rng.standard_normal((6, 1, 8)), rng.standard_normal((6, 1, 8))
    do = rng.standard_normal((4, 2, 8))
    g = A.attn_bwd(q, k, v, do, 0.3, 0.0, 0.0)
    for name, x in (("dq", q), ("dk", k), ("dv", v)):
        for _ in range(6):
            at = tuple(rng.integers(0, n) for n in x.shape)
            was, h, f = x[at], 1e-5, []
            for e in (h, -h):
                x[at] = was + e
                f.append((A.attn_fwd(q, k, v, 0.3, 0.0)[0] * do).sum())
            x[at] = was
            assert abs((f[0] - f[1]) / (2 * h) - g[name][0][at]) < 1e-7


def test_oracle_e4m3_is_torchs():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(codes, A.VALUES, equal_nan=True)
    rng = np.random.default_rng(3)
    x = np.concatenate([rng.standard_normal(4000) * 2.0 ** rng.integers(-12, 9, 4000), A.VALUES[:126],
                        (A.VALUES[:126] + A.VALUES[1:127]) / 2, [448.0, 463.9, 2.0 ** -10, 1.5 * 2.0 ** -9]])
    x = x[np.abs(x) <= 448]
    x = np.concatenate([x, -x]).astype(np.float32).astype(np.float64)
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(A.quantise(x, 1.0), want)
    assert (A.quantise(np.array([np.inf, -np.inf, np.nan]), 1.0) & 127).tolist() == [127] * 3
    for m in (448.0, 448.1, 1.0, 0.0, 1e-40, 3e38, 1.75 * 2.0 ** 20):
        s = A.scale_of(np.array([m, np.inf]))
        assert m <= 448 * s and (s == 2.0 ** -117 or m > 224 * s)
