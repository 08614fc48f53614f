"""Build libcarve.so (HIP kernels + C ABI) for gfx950 in-tree.

    python -m chunk_gated_delta_amd.build

Each translation unit is compiled in parallel with hipcc, then linked into
chunk_gated_delta_amd/libcarve.so next to this file.
"""
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libcarve.so")
BUILD = os.path.join(HERE, "_build")
SOURCES = ["carve_api.cpp", "fwd_kernels.hip", "bwd_kernels.hip", "decode_kernels.hip", "content_bwd_kernels.hip",
           "stream_kernels.hip", "width_kernels.hip", "attention/attn_api.cpp", "attention/swa_fwd.hip",
           "attention/swa_bwd.hip", "attention/weights.hip", "attention/cache_decode.hip", "attention/cache_fill.hip"]
ARCH = "gfx950"

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CFLAGS = [
    "-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
    # packed fp32 instructions stay off: hipcc would otherwise form v_pk_* fp32 ops by itself
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-result",
]


def source_digest(attention=False):
    """Digest of the delta rule's kernel sources (csrc/*, without csrc/attention), or of the attention
    operators' (csrc/attention/* and the device header that they share); measurements
    record it so that a later change to the kernels marks them stale."""
    import hashlib
    h = hashlib.sha256()
    if attention:
        files = ["carve_device.h"] + [os.path.join("attention", f) for f in sorted(os.listdir(os.path.join(CSRC, "attention")))]
    else:
        files = sorted(os.listdir(CSRC))
    for name in files:
        if name.endswith((".hip", ".h", ".cpp")):
            h.update(name.encode())
            with open(os.path.join(CSRC, name), "rb") as f:
                h.update(f.read())
    return h.hexdigest()[:16]


def _compile(src):
    obj = os.path.join(BUILD, os.path.splitext(os.path.basename(src))[0] + ".o")
    cmd = [HIPCC] + CFLAGS + (["-x", "hip"] if src.endswith(".cpp") else []) + \
        ["-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    err = "\n".join(line for line in r.stderr.splitlines() if "packed-fp32-ops" not in line)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{err}")
    return obj


def build(verbose=True):
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(max_workers=min(8, len(SOURCES))) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "-shared", "-fPIC", f"--offload-arch={ARCH}", "-Wl,--no-undefined", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stderr)
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build()
    sys.exit(0)
