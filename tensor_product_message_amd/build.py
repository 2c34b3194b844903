"""Build libconvtp.so (HIP, gfx950) in-tree with hipcc, and the Python bindings of
the training-step and the dense operators (_train.so, _dense.so, host code) with
g++.

    python -m tensor_product_message_amd.build [--incremental]

Every HIP source is compiled for gfx950 only, with packed-fp32 instruction
selection switched off (-Xclang -target-feature -Xclang -packed-fp32-ops) and
no implicit multiply-add contraction (-ffp-contract=off: every fused
multiply-add is an explicit __builtin_fmaf in the source).
The convolution kernels are compiled once per degree triple (l_in, l_sh,
l_out), 64 objects from csrc/convtp_triple.hip with -DCTP_L1/-DCTP_L2/-DCTP_L3,
in parallel, largest first; the linear layers once per element type (-DCTP_DENSE_TYPE).
--incremental skips objects newer than every
source (for development; the default rebuilds everything).
"""
from __future__ import annotations

import glob
import importlib.util
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libconvtp.so")
SOURCES = ["convtp_common.hip", "nodetp_kernels.hip", "graph_kernels.hip", "stream_probe.hip", "convtp_api.hip"]
# the operators of a training step (include/convtp_train.h), apart from the convolution's sources and headers
TRAIN_SOURCES = ["embed_kernels.hip", "norm_fwd.hip", "norm_bwd.hip", "norm_bwd_bwd.hip", "clip_kernels.hip", "train_api.hip"]
TRAIN_HEADERS = ["csrc/train_common.hpp", "csrc/train_kernels.hpp", "csrc/norm_common.hpp", "csrc/norm_sums.hpp",
                 "../include/convtp_train.h", "../include/convtp.h"]
# the dense operators (include/convtp_dense.h)
DENSE_SOURCES = ["ortho_kernels.hip", "dense_dispatch.hip", "dense_api.hip"]
DENSE_TYPED_SOURCE, DENSE_TYPES = "dense_linear.hip", ("f32", "bf16", "f16")
DENSE_HEADERS = ["csrc/dense_common.hpp", "csrc/dense_direct.hpp", "csrc/dense_kernels.hpp", "csrc/dense_linear.hpp",
                 "csrc/train_common.hpp", "../include/convtp_dense.h", "../include/convtp_train.h", "../include/convtp.h"]
# the Python bindings, extension modules next to the package's other files: source, module
BINDINGS = [("train_binding.cpp", os.path.join(HERE, "_train.so")), ("dense_binding.cpp", os.path.join(HERE, "_dense.so"))]
BINDING_HEADERS = ["csrc/binding_common.hpp", "../include/convtp_dense.h", "../include/convtp_train.h", "../include/convtp.h"]
TRIPLE_SOURCE = "convtp_triple.hip"
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
FLAGS = ["-O3", "-std=c++20", "-fPIC", f"--offload-arch={ARCH}",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         # fused multiply-adds only where the source writes __builtin_fmaf: the
         # compiler may not fuse a product into a later addition, so kernels
         # that share an arithmetic sequence (the backward's dY and the dY-only
         # kernel) round identically
         "-ffp-contract=off",
         "-Wall", "-Wno-unused-function", "-Wno-undefined-inline"]


def _paths(a: int, b: int, c: int) -> int:
    return sum(1 for p in range(a + 1) for q in range(b + 1) for r in range(c + 1) if abs(p - q) <= r <= p + q)


TRIPLES = sorted(((a, b, c) for a in range(4) for b in range(4) for c in range(4)),
                 key=lambda t: -_paths(*t))


def _compile(job) -> None:
    src, obj, defines = job
    cmd = [HIPCC, *FLAGS, *defines, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    msgs = [ln for ln in (r.stdout + r.stderr).splitlines() if "packed-fp32-ops" not in ln
            and "is not a recognized feature for this target" not in ln]
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src} {' '.join(defines)}:\n" + "\n".join(msgs))
    if msgs:
        print("\n".join(msgs), file=sys.stderr)


def _jobs(objdir: str):
    single = lambda names: [(s, os.path.join(objdir, s.replace(".hip", ".o")), []) for s in names]  # noqa: E731
    triples = [(TRIPLE_SOURCE, os.path.join(objdir, f"triple_{a}{b}{c}.o"),
                [f"-DCTP_L1={a}", f"-DCTP_L2={b}", f"-DCTP_L3={c}"]) for a, b, c in TRIPLES]
    typed = [(DENSE_TYPED_SOURCE, os.path.join(objdir, f"dense_linear_{t}.o"), [f"-DCTP_DENSE_TYPE={k}"])
             for k, t in enumerate(DENSE_TYPES)]
    return single(TRAIN_SOURCES) + typed + triples + single(DENSE_SOURCES + SOURCES)     # the longest first


def _build_binding(source: str, module: str) -> None:
    """Host code only (g++): torch's and Python's headers, the library's entry points are looked up at run time."""
    torch_dir = os.path.dirname(importlib.util.find_spec("torch").origin)
    include, lib = os.path.join(torch_dir, "include"), os.path.join(torch_dir, "lib")
    rocm = os.path.dirname(os.path.dirname(HIPCC))
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__",
           "-DUSE_ROCM", "-D_GLIBCXX_USE_CXX11_ABI=1"]
    for path in (include, os.path.join(include, "torch", "csrc", "api", "include"), os.path.join(rocm, "include"),
                 sysconfig.get_paths()["include"]):
        cmd += ["-isystem", path]
    tmp = module + ".tmp"
    cmd += [os.path.join(CSRC, source), "-o", tmp, f"-L{lib}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_hip"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {source}:\n{r.stdout}{r.stderr}")
    if r.stderr:
        print(r.stderr, file=sys.stderr)
    os.replace(tmp, module)


def build(verbose: bool = True, incremental: bool = False, workers: int = None) -> str:
    """Compile every HIP source and link libconvtp.so; returns its path."""
    objdir = os.path.join(HERE, "_build")
    os.makedirs(objdir, exist_ok=True)
    jobs = _jobs(objdir)
    todo = jobs
    bindings = BINDINGS
    if incremental:
        full = lambda paths: [os.path.normpath(os.path.join(HERE, p)) for p in paths]  # noqa: E731
        newest = lambda paths: max(os.path.getmtime(p) for p in paths)  # noqa: E731
        train, dense = full(TRAIN_HEADERS), full(DENSE_HEADERS)
        others = train + dense + full(BINDING_HEADERS)
        conv = [p for p in glob.glob(os.path.join(CSRC, "*.hpp")) if p not in others] + full(["../include/convtp.h"])

        def stale(src, target, headers):
            return not os.path.exists(target) or os.path.getmtime(target) < newest([os.path.join(CSRC, src), *headers])

        def headers_of(src):
            return train if src in TRAIN_SOURCES else dense if src in (*DENSE_SOURCES, DENSE_TYPED_SOURCE) else conv
        todo = [j for j in jobs if stale(j[0], j[1], headers_of(j[0]))]
        bindings = [b for b in BINDINGS if stale(*b, full(BINDING_HEADERS))]
    n = workers or min(16, os.cpu_count() or 8)
    with ThreadPoolExecutor(max_workers=n) as ex:
        jobs_done = [ex.submit(_build_binding, *b) for b in bindings]
        list(ex.map(_compile, todo))
        for f in jobs_done:
            f.result()
    tmp = LIB + ".tmp"
    subprocess.run([HIPCC, "-shared", "-fPIC", f"--offload-arch={ARCH}", "-o", tmp, *[j[1] for j in jobs]],
                   check=True)
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB} ({len(todo)} of {len(jobs)} objects compiled)")
    return LIB


if __name__ == "__main__":
    build(incremental="--incremental" in sys.argv)
