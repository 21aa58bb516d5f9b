"""Build the in-tree shared libraries with nvcc for sm_100a (B200).

  libkv4.so     the INT4 KV cache library (C ABI in include/kv4.h)
  libkv4gen.so  the GPU twin of the seeded input generator (tests and benchmark only)

Run ``python -m int4_kv_cache_append_b200.build`` (or ``__graft_entry__.build()``).  Sources
compile in parallel; a library is rebuilt only when a source or header is newer than it.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
COMMON = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "-ftz=false", "-prec-div=true", "-prec-sqrt=true",
          "-Xptxas", "-v"]

LIBS = {
    "libkv4.so": ["kv4_api.cu", "kv4_append.cu", "kv4_decode.cu", "kv4_bf16.cu", "kv4_mixed.cu", "kv4_rope.cu", "kv4_shared.cu"],
    "libkv4gen.so": ["kv4gen.cu"],
}


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> dict[str, str]:
    headers = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        [os.path.join(ROOT, "include", "kv4.h")]
    out = {}
    for lib, srcs in LIBS.items():
        target = os.path.join(HERE, lib)
        src_paths = [os.path.join(CSRC, s) for s in srcs]
        if force or _stale(target, src_paths + headers):
            tmp = target + f".tmp{os.getpid()}"
            objs = [tmp + "." + os.path.basename(s) + ".o" for s in src_paths]
            cmds = [[NVCC, *ARCH, *COMMON, "-I", os.path.join(ROOT, "include"), "-c", "-o", o, s] for o, s in zip(objs, src_paths)]
            try:
                with concurrent.futures.ThreadPoolExecutor(max_workers=os.cpu_count() or 1) as pool:
                    runs = list(pool.map(lambda c: subprocess.run(c, capture_output=True, text=True), cmds))
                if all(r.returncode == 0 for r in runs):
                    runs.append(subprocess.run([NVCC, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True))
            finally:
                for o in objs:
                    if os.path.exists(o):
                        os.remove(o)
            if any(r.returncode != 0 for r in runs):
                sys.stderr.write("".join(r.stdout + r.stderr for r in runs if r.returncode != 0))
                raise RuntimeError(f"nvcc failed for {lib}")
            if verbose:
                sys.stderr.write("".join(r.stderr for r in runs))
            os.replace(tmp, target)
        out[lib] = target
    return out


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
