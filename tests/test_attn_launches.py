"""Which kernels attention's entry points launch, and over what grids, recorded on
the CPU (tests/native/launch_record.cpp)."""

import os
import shutil
import subprocess

import pytest

from linear_attention_rnn_gated_amd import binding as B

HERE = os.path.dirname(os.path.abspath(__file__))
F32, BF16 = B.GDN_F32, B.GDN_BF16


@pytest.fixture(scope="module")
def record(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("launch") / "launch_record")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-rdynamic", "-I", os.path.join(os.path.dirname(HERE), "include"),
                        os.path.join(HERE, "native", "launch_record.cpp"), "-o", exe, "-ldl"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-4000:]

    def run(*args):
        """([(kernel, grid x, grid y, threads a block)], status)"""
        r = subprocess.run([exe, B.LIB_PATH, *map(str, args)], capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, r.stderr
        *rows, last = r.stdout.splitlines()
        out = []
        for row in rows:
            name, x, y, z, threads = row.split()
            assert z == "1"
            known = [k for k in KERNELS if k + "I" in name or k + "E" in name]
            assert len(known) == 1, name
            out.append((known[0], int(x), int(y), int(threads)))
        return out, int(last.split()[1])
    return run


KERNELS = ("k_attn_decode", "k_attn_decode_wide", "k_attn_join", "k_attn_dq", "k_attn_dkv", "k_attn_sum", "k_attn_stat")


@pytest.mark.parametrize("Hq,Hkv,n,T", [(4, 2, 1, 64), (8, 1, 1, 4), (31, 1, 1, 2), (4, 2, 2, 64), (16, 2, 5, 5)])
@pytest.mark.parametrize("max_len", [100, 5000])
def test_packed_rows_may_be_fewer_than_the_buffer(record, Hq, Hkv, n, T, max_len):
    """cu_seqlens is read on the device: whatever T is, a sequence may have fewer rows than the wide kernel takes."""
    launches, rc = record("decode", Hq, Hkv, 64, BF16, 1, n, T, max_len)
    assert rc == B.GDN_OK
    assert ("k_attn_decode" in [k for k, *_ in launches]) == (Hq // Hkv < 32)
    assert ("k_attn_decode_wide" in [k for k, *_ in launches]) == (T * (Hq // Hkv) >= 32)
    assert ("k_attn_join" in [k for k, *_ in launches]) == (max_len > 512)


@pytest.mark.parametrize("Hq,Hkv,d,t,n,Tq,Tk,cut", [
    (8, 8, 128, BF16, 1, 1024, 20_000_000, "q"),   # a few queries over very many keys: the keys' gradients are not cut
    (8, 8, 128, BF16, 1, 1024, 30_000, "q"),
    (4, 1, 64, F32, 3, 1030, 1538, "both"),
    (64, 2, 256, BF16, 2, 100_000, 700, "k"),
    (32, 8, 128, BF16, 8, 32768, 32768, "none"),
])
def test_the_gradients_sums(record, Hq, Hkv, d, t, n, Tq, Tk, cut):
    """Only what was cut into parts is summed, over a grid of its own size."""
    launches, rc = record("bwd", Hq, Hkv, d, t, n, Tq, Tk)
    assert rc == B.GDN_OK
    grids = {k: (x, y) for k, x, y, _ in launches}
    assert (grids["k_attn_dq"][1] > 1) == (cut in ("q", "both"))
    assert (grids["k_attn_dkv"][1] > 1) == (cut in ("k", "both"))
    sizes = {"q": [Tq * Hq], "k": [Tk * Hkv] * 2, "both": [Tq * Hq] + [Tk * Hkv] * 2, "none": []}[cut]
    if sizes:
        assert grids["k_attn_sum"] == (-(-max(sizes) * d // 1024), len(sizes))
    assert ("k_attn_sum" in grids) == bool(sizes)
    assert ("k_attn_stat" in grids) == (t == BF16 and cut in ("q", "both"))
    assert all(x * y * threads < 1 << 32 for _, x, y, threads in launches)


@pytest.mark.parametrize("Hq,Hkv,d,n,T,max_len", [
    (32, 8, 128, 8, 200_000, 500),        # many rows, nothing to join
    (32, 8, 128, 1, 131_072, 131_072),
    (32, 8, 256, 3, 140_000, 20_000),     # more rows than one launch of the join holds
    (32, 8, 128, 1024, 1024, 1 << 20),    # many sequences that may become long
    (2, 1, 64, 1, 20, 40_000_000),        # more splits than a grid's second dimension holds
])
def test_large_calls_take_several_launches(record, Hq, Hkv, d, n, T, max_len):
    launches, rc = record("decode", Hq, Hkv, d, BF16, 1, n, T, max_len)
    assert rc == B.GDN_OK
    assert all(x * y * threads < 1 << 32 and y < 65536 for _, x, y, threads in launches)
    splits = -(-max_len // 512)
    halves = splits if splits <= 8 else max(8, -(-splits // 2))
    assert sum(y for k, _, y, _ in launches if k == "k_attn_decode") == halves
    assert sum(y for k, _, y, _ in launches if k == "k_attn_decode_wide") == (splits if T * Hq // Hkv >= 32 else 0)
    per = 1024 // d if splits <= 16 else 1
    assert sum(x * per for k, x, _, _ in launches if k == "k_attn_join") == (T * Hq if splits > 1 else 0)


def test_what_no_launch_holds_is_refused(record):
    for args in ((32, 8, 128, BF16, 1, 1 << 20, 1 << 20, 100), (32, 8, 128, BF16, 0, 1 << 21, 1 << 21, 100),
                 (32, 8, 128, BF16, 1, 1, 1 << 29, 100)):
        assert record("decode", *args) == ([], B.GDN_ERR_UNSUPPORTED), args
