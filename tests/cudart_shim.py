"""Child processes with cudart_shim.cpp in front of the CUDA runtime: what the
library asks of the runtime, and what it does where the runtime says no."""

import os
import subprocess
import sys

from split_backward_gemms_gb300 import build as B

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


def build(folder) -> str:
    B.build()
    out = os.path.join(str(folder), "cudart_shim.so")
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-shared", "-fPIC", "-I",
                    os.path.join(B.cuda_home(), "include"), os.path.join(HERE, "cudart_shim.cpp"), "-o", out, "-ldl"],
                   check=True)
    return out


def run(folder, code, fake=True, **env):
    """The launches that `code` made: (blocks, threads, cluster, programmatic, argument's bytes)."""
    so, log = os.path.join(str(folder), "cudart_shim.so"), os.path.join(str(folder), "launches")
    if not os.path.exists(so):
        build(folder)
    if os.path.exists(log):
        os.remove(log)
    env = dict({k: v for k, v in os.environ.items() if not k.startswith("ZB_")}, LD_PRELOAD=so, SHIM_LOG=log,
               SHIM_FAKE="1" if fake else "0", **env)
    r = subprocess.run([sys.executable, "-c", code], env=env, cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
    with open(log) as f:
        lines = [line.rstrip("\n").split(" ") for line in f]
    return [(int(a), int(b), int(c), int(d), bytes.fromhex(e)) for a, b, c, d, e in lines]
