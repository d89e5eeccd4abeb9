"""Builds libgdn.so (HIP, gfx950) in-tree with hipcc.

Flags that are part of the arithmetic contract: -ffp-contract=off (the only
fused multiply-adds are the explicit fmaf calls), no fast-math, and packed
FP32 instructions disabled.  These are the same for every source; SOURCE_FLAGS
says beside them where a source's matrix sums stand, which changes no bits.  The
recurrences' kernels, whose bits have to agree, are one translation unit
(gdn_library.hip).
"""

import hashlib
import os
import subprocess
import sys
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libgdn.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

SOURCES = ["gdn_library.hip", "gdn_attn.hip", "gdn_kv.hip", "gdn_kv_wide.hip", "gdn_plan.cpp", "gdn_rope.cpp"]
INCLUDED = ["gdn_common.h", "gdn_mma.h", "gdn_attn_walk.h", "gdn_kv.h", "gdn_plan.h", "gdn_kernels.hip", "gdn_lru.hip", "gdn_qk.hip"]  # by the sources
FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++20",
    "-fPIC",
    "-ffp-contract=off",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
    "-Wno-unused-function",
]
SOURCE_FLAGS = {
    # MFMA accumulators in ordinary VGPRs: the 4-wave chunk scan otherwise
    # splits its accumulators into AGPRs and copies them back every chunk, and
    # attention over the cache for few rows does (decode 64: 117 us, without 134).
    # Elsewhere attention's accumulators stay in the AGPRs.
    "gdn_library.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"],
    "gdn_kv.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"],
}

def source_digest(extra_flags=()):
    """SHA-256 (first 16 hex digits) over the header, every source and the
    compile flags: part of gdn_contract_id(), so two builds that could differ in
    arithmetic never report the same id."""
    h = hashlib.sha256()
    for path in [os.path.join(ROOT, "include", "gdn.h"),
                 *[os.path.join(CSRC, s) for s in [*INCLUDED, *SOURCES]]]:
        with open(path, "rb") as f:
            h.update(f.read())
    h.update(" ".join([*FLAGS, str(SOURCE_FLAGS), *extra_flags]).encode())
    return h.hexdigest()[:16]


def build(verbose=False, extra_flags=()):
    """Compiles the sources side by side and links libgdn.so; returns its path."""
    digest = f'-DGDN_SOURCE_DIGEST="{source_digest(extra_flags)}"'
    with tempfile.TemporaryDirectory() as tmp:
        objects = [os.path.join(tmp, s + ".o") for s in SOURCES]
        cmds = [[HIPCC, *FLAGS, *SOURCE_FLAGS.get(s, []), *extra_flags, digest, "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                 "-c", os.path.join(CSRC, s), "-o", o] for s, o in zip(SOURCES, objects)]
        _run_all(cmds, verbose)
        _run_all([[HIPCC, *FLAGS, *extra_flags, "-shared", *objects, "-o", LIB + ".tmp"]], verbose)
    os.replace(LIB + ".tmp", LIB)
    return LIB


def _run_all(cmds, verbose):
    """Runs the commands at once and waits for all of them; raises if one fails."""
    running = []
    for cmd in cmds:
        if verbose:
            print(" ".join(cmd), flush=True)
        running.append(subprocess.Popen(cmd, stdout=subprocess.DEVNULL, stderr=subprocess.PIPE, text=True))
    # hipcc's host pass does not know the packed-fp32 feature and says so
    noise = "is not a recognized feature for this target"
    said = ["\n".join(l for l in p.communicate()[1].splitlines() if noise not in l) for p in running]
    if any(p.returncode for p in running):
        raise RuntimeError("hipcc failed:\n" + "\n".join(said))
    if verbose and any(s.strip() for s in said):
        print("\n".join(s for s in said if s.strip()), file=sys.stderr)


if __name__ == "__main__":
    print(build(verbose=True))
