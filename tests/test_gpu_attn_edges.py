"""Attention over the cache and the cache's writes at the edges of what the entry
points allow: padded batches, sequences without new tokens, pages that are not there."""

import numpy as np
import pytest
import torch

from linear_attention_rnn_gated_amd import binding as B
from test_gpu_attn import BF16, DT, INF, NAN, Pool, _need_gpu, cu_of, decode_check, i32, np64  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,d,t,T,real,kv", [
    (4, 2, 64, "bf16", 64, 1, 300),
    (4, 2, 128, "bf16", 16, 15, 1500),
    (8, 1, 256, "bf16", 40, 3, 9000),   # joined in groups
    (6, 2, 64, "f32", 30, 10, 700),
    (4, 1, 128, "f32", 9, 7, 100),
    (4, 2, 64, "bf16", 64, 40, 1500),   # as many as the other kernel takes
    (4, 2, 64, "bf16", 64, 0, 1500),
    (40, 1, 64, "bf16", 8, 1, 600),     # one token fills it
])
def test_one_padded_sequence(Hq, Hkv, d, t, T, real, kv):
    """T rows, of which cu_seqlens has the first `real`: the others are left as they are."""
    pool = Pool(Hq, Hkv, d, t, 64, [kv], seed=d + real)
    pool.write(pool.rows(kv), pool.rows(kv), [kv], [0])
    q = pool.queries(T)
    q[real:] = NAN
    out = torch.full_like(q, 7.0)
    ws = torch.full((B.attn_decode_workspace_bytes(pool.shape, 1, T, kv),), 255, dtype=torch.uint8, device="cuda")
    args = (pool.cache, pool.dev_table, i32([kv]), kv)
    o, lse = B.gdn_attn_decode(pool.shape, q, *args, cu_seqlens=cu_of([real]).cuda(), out=out, want_lse=True, ws=ws)
    assert (o[real:] == 7).all()
    decode_check(pool, q, [real], [kv], o[:real], lse[:real])
    if real:
        exact = B.gdn_attn_decode(pool.shape, q[:real], *args, cu_seqlens=cu_of([real]).cuda())
        assert torch.equal(exact, o[:real])


def test_a_captured_chunk_that_gets_shorter():
    """One graph for chunks of one prompt: the last one has fewer tokens than the buffer."""
    T, L = 48, 700
    pool = Pool(4, 2, 128, "bf16", 64, [L + 200], seed=3)
    pool.write(pool.rows(L), pool.rows(L), [L], [0])
    q = pool.queries(T)
    cu, kv = cu_of([T]).cuda(), i32([L])
    ws = torch.empty(B.attn_decode_workspace_bytes(pool.shape, 1, T, 900), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), None
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        B.gdn_attn_decode(pool.shape, q, pool.cache, pool.dev_table, kv, 900, cu_seqlens=cu, out=out, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, lse = B.gdn_attn_decode(pool.shape, q, pool.cache, pool.dev_table, kv, 900, cu_seqlens=cu, out=out, ws=ws,
                                   want_lse=True)
    for real in (48, 20, 16, 15, 7, 1, 33, 0, 15):
        q.copy_(pool.queries(T))
        cu.copy_(cu_of([real]))
        out.fill_(3.0)
        ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert (out[real:] == 3).all(), real
        decode_check(pool, q, [real], [L], out[:real], lse[:real], f"{real} tokens")
