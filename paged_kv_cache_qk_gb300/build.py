"""Build libpkvqk.so (the C-ABI library) in-tree with nvcc for sm_103a, and torch_calls.so.

    python -m paged_kv_cache_qk_gb300.build [--verbose-ptxas]

Each .cu under csrc/ is compiled in parallel to an object under _build/,
then linked into paged_kv_cache_qk_gb300/libpkvqk.so (CUDA runtime linked
statically, no libcuda link: the TMA encoder is fetched through the runtime's
driver entry-point query).  Beside it csrc/torch_calls.cpp, the binding's native part, becomes
paged_kv_cache_qk_gb300/torch_calls.so with the host compiler, against the installed torch.
The library needs nvcc alone: without torch torch_calls.so is left out (its calls take
tensors), and where it cannot be built the library is there before that is raised.
"""

from __future__ import annotations

import argparse
import concurrent.futures
import fcntl
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libpkvqk.so")
CALLS = os.path.join(PKG, "torch_calls.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
SOURCES = ["api.cu", "norm_rope_append.cu", "decode.cu", "combine.cu", "decode_static_ws.cu",
           "prefill.cu", "norm_rope_append_q8.cu", "decode_q8.cu", "verify_drafts.cu",
           "decode_scored.cu", "prefill_scored.cu"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def cxx() -> str:
    found = shutil.which("g++") or shutil.which("c++")
    if found is None:
        raise RuntimeError("no C++ compiler found")
    return found


def torch_dir() -> str | None:
    spec = importlib.util.find_spec("torch")   # its headers are wanted, not the module
    return None if spec is None else os.path.dirname(spec.origin)


def build(verbose_ptxas: bool = False, force: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with open(os.path.join(BUILD, "lock"), "w") as lock:
        fcntl.flock(lock, fcntl.LOCK_EX)       # processes that build at the same time
        return _build(verbose_ptxas, force)


def _build(verbose_ptxas: bool, force: bool) -> str:
    header = os.path.join(ROOT, "include", "pkvqk.h")
    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    deps = [header, __file__] + srcs + [os.path.join(CSRC, f) for f in os.listdir(CSRC)
                                        if f.endswith((".h", ".cuh"))]
    torch = torch_dir()
    with concurrent.futures.ThreadPoolExecutor(1) as pool:
        calls = None
        if torch is not None:
            calls_src = os.path.join(CSRC, "torch_calls.cpp")
            with open(os.path.join(torch, "version.py")) as f:
                against = f"{sysconfig.get_config_var('SOABI')}\n{torch}\n{f.read()}"
            # another torch may be older than what was built against this one
            if force or _stale(CALLS, [header, __file__, calls_src]) or _read(_stamp()) != against:
                calls = pool.submit(_compile_calls, calls_src, torch)
        if force or _stale(LIB, deps):
            _link([nvcc(), *ARCH, "-shared"], LIB, _compile_library(srcs, verbose_ptxas))
        if calls is not None:                  # links with the library
            _link([cxx(), "-shared"], CALLS,
                  [calls.result(), "-L" + os.path.join(torch, "lib"), "-ltorch_python",
                   "-ltorch_cpu", "-lc10", "-lc10_cuda", "-L" + PKG, "-l:libpkvqk.so",
                   "-Wl,-rpath,$ORIGIN"])
            with open(_stamp(), "w") as f:
                f.write(against)
    return LIB


def _stamp() -> str:
    return os.path.join(BUILD, "torch_calls.against")


def _read(path: str) -> str | None:
    if not os.path.exists(path):
        return None
    with open(path) as f:
        return f.read()


def _stale(out: str, deps: list) -> bool:
    return not os.path.exists(out) or any(os.path.getmtime(d) >= os.path.getmtime(out)
                                          for d in deps)


def _compile_library(srcs: list, verbose_ptxas: bool) -> list:
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2,-fvisibility=hidden",
                    "-I", os.path.join(ROOT, "include"), "--expt-relaxed-constexpr"]
    if verbose_ptxas:
        flags += ["-Xptxas", "-v"]
    procs = []
    objs = []
    for s in srcs:
        o = os.path.join(BUILD, os.path.basename(s).replace(".cu", ".o"))
        objs.append(o)
        procs.append((s, subprocess.Popen([nvcc(), *flags, "-c", s, "-o", o],
                                          stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for s, p in procs:
        out, _ = p.communicate()
        txt = out.decode(errors="replace")
        if verbose_ptxas or p.returncode != 0:
            sys.stderr.write(txt)
        if p.returncode != 0:
            failed.append(s)
    if failed:
        raise RuntimeError("compilation failed for: " + ", ".join(failed))
    return objs


def _compile_calls(src: str, torch: str) -> str:
    obj = os.path.join(BUILD, "torch_calls.o")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    include = [os.path.join(ROOT, "include"), os.path.join(torch, "include"),
               os.path.join(torch, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    _run([cxx(), "-std=c++17", "-O2", "-fPIC", "-fvisibility=hidden", *("-I" + i for i in include),
          "-c", src, "-o", obj], "compilation failed for: " + src)
    return obj


def _link(command: list, out: str, inputs: list) -> None:
    tmp = out + ".tmp"
    _run([*command, "-o", tmp, *inputs], "link failed: " + os.path.basename(out))
    os.replace(tmp, out)


def _run(command: list, failure: str) -> None:
    r = subprocess.run(command, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if r.returncode != 0:
        sys.stderr.write(r.stdout.decode(errors="replace"))
        raise RuntimeError(failure)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--verbose-ptxas", action="store_true")
    ap.add_argument("--force", action="store_true")
    args = ap.parse_args()
    print(build(verbose_ptxas=args.verbose_ptxas, force=args.force))


if __name__ == "__main__":
    main()
