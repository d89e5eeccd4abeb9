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
            known = [k for k in KERNELS if k + "I" in name]
            assert len(known) == 1, name
            out.append((known[0], int(x), int(y), int(threads)))
        return out, int(last.split()[1])
    return run


KERNELS = ("k_attn_decode", "k_attn_decode_wide", "k_attn_join", "k_attn_dq", "k_attn_dkv", "k_attn_sum")


@pytest.mark.parametrize("Hq,Hkv,n,T", [(4, 2, 1, 64), (8, 1, 1, 4), (31, 1, 1, 2), (4, 2, 2, 64), (16, 2, 5, 5)])
@pytest.mark.parametrize("max_len", [100, 5000])
def test_packed_rows_may_be_fewer_than_the_buffer(record, Hq, Hkv, n, T, max_len):
    """cu_seqlens is read on the device: whatever T is, a sequence may have fewer rows than the wide kernel takes."""
    launches, rc = record("decode", Hq, Hkv, 64, BF16, 1, n, T, max_len)
    assert rc == B.GDN_OK
    assert ("k_attn_decode" in [k for k, *_ in launches]) == (Hq // Hkv < 32)
    assert ("k_attn_decode_wide" in [k for k, *_ in launches]) == (T * (Hq // Hkv) >= 32)
    assert ("k_attn_join" in [k for k, *_ in launches]) == (max_len > 512)
