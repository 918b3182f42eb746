"""Compile the gfx950 HIP sources into ``libsdtw.so`` (in-tree, beside this file),
and the same sources with SDTW_STRESS=1 into ``libsdtw_stress.so`` (pseudo-random
delays at every hand-off, for the stress tests only).

    python -m differentiable_series_alignment_amd.build [-v]

hipcc cross-compiles for gfx950 without a GPU.  Packed fp32 instructions are
disabled for the device code (``-packed-fp32-ops``); the host pass warns that
it does not know that feature, which is harmless.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libsdtw.so")
# Debug build of the same sources with pseudo-random sleeps at every hand-off
# (SDTW_STRESS=1): loaded only by the hand-off stress tests.
STRESS_LIB = os.path.join(HERE, "libsdtw_stress.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.hip")))


def _compile(src: str, obj: str, extra) -> list:
    return [HIPCC, f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-c",
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            "-Wall", "-Wno-unused-command-line-argument",
            "-I", INCLUDE, "-I", CSRC, *extra, src, "-o", obj]


def _run(cmd) -> tuple:
    """(exit status, messages) of a compiler's run."""
    pr = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    noise = "is not a recognized feature for this target"
    return pr.returncode, [ln for ln in pr.stdout.splitlines() if ln.strip() and noise not in ln]


def build(verbose: bool = False, extra=(), stress: bool = True) -> str:
    """Builds libsdtw.so and (stress=True) the stress variant, every source of
    both on its own, as many at a time as there are CPUs, at most 16 (on 8 the
    longest one's 45 s, where a library's sources one after the other take 90);
    returns the path of libsdtw.so."""
    libs = [(LIB, tuple(extra))]
    if stress:
        libs.append((STRESS_LIB, tuple(extra) + ("-DSDTW_STRESS=1",)))
    errors = []
    with tempfile.TemporaryDirectory() as tmp:
        jobs, links = [], []
        for i, (out, ex) in enumerate(libs):
            objs = []
            for src in sources():
                objs.append(os.path.join(tmp, f"{i}_{os.path.basename(src)}.o"))
                jobs.append((os.path.basename(src), _compile(src, objs[-1], ex)))
            links.append((os.path.basename(out), [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC",
                                                  *objs, "-o", out + ".tmp"]))
        with ThreadPoolExecutor(max_workers=min(16, os.cpu_count() or 1)) as pool:
            for step in (jobs, links):
                if verbose:
                    for _, cmd in step:
                        print(" ".join(cmd), flush=True)
                for (name, _), (rc, msgs) in zip(step, pool.map(_run, [cmd for _, cmd in step])):
                    if rc != 0:
                        errors.append(f"{name}:\n" + "\n".join(msgs))
                    elif verbose and msgs:
                        print("\n".join(msgs))
                if errors:
                    raise RuntimeError("hipcc failed:\n" + "\n".join(errors))
    for out, _ in libs:
        os.replace(out + ".tmp", out)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
