"""Compile the CUDA library (libgbgemm.so) in-tree for sm_103a with nvcc, and the torch binding of the
operators around the products (_gbgemm_torch.so) with the host compiler."""
from __future__ import annotations

import os
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libgbgemm.so")
BINDING = os.path.join(PKG, "_gbgemm_torch.so")
LOG_DIR = os.path.join(PKG, "_build")
SOURCES = ["gbgemm.cu", "rowwise.cu", "w4.cu"]
HEADERS = ["gemm_kernel.cuh", "host.h", "ptx.cuh", "probe.cuh", "rowwise.cuh", "w4_kernel.cuh"]
NVCC_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-lineinfo", "-std=c++17",
              "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden", "-Xptxas", "-v",
              "--diag-suppress", "177"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _stale(lib: str = LIB, files=tuple(SOURCES + HEADERS)) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    deps = [os.path.join(CSRC, f) for f in files] + [os.path.join(ROOT, "include", "gbgemm.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def _check_register_budgets(log: str) -> None:
    """Refuse a build whose kernels could block forever in setmaxnreg.inc: for every
    kernel with two epilogue warpgroups (384 threads), the launch register count
    times the threads must cover the budgets the warpgroups lower and raise to
    (constants of WarpLayout in gemm_kernel.cuh)."""
    import re
    src = open(os.path.join(CSRC, "gemm_kernel.cuh")).read()

    def const(name):
        return int(re.search(rf"static constexpr int {name} = (\d+);", src).group(1))

    control, epilogue = const("kRegsControl"), const("kRegsEpilogue")
    entries = re.findall(r"Compiling entry function '(\w+)'.*?Used (\d+) registers", log, flags=re.S)
    if not entries:
        raise RuntimeError("no kernels in the ptxas report")
    for name, regs in entries:
        if "gemm_persistent_kernel" not in name:
            continue
        m = re.search(r"Li(\d+)EEEv", name)  # the last template argument: epilogue warpgroups
        epi = int(m.group(1)) if m else 1
        if epi != 2:
            continue
        threads, need = 384, 128 * control + 256 * epilogue
        if int(regs) * threads < need:
            raise RuntimeError(f"{name} launches with {regs} registers/thread x {threads} threads, less than "
                               f"the {need} its warpgroup register budgets need")


TRACE_LIB = os.path.join(PKG, "libgbgemm_trace.so")


def build(force: bool = False, verbose: bool = False, trace: bool = False) -> str:
    """Build libgbgemm.so next to this file; the -Xptxas -v report goes to _build/ptxas.log.
    trace=True builds the instrumented libgbgemm_trace.so instead (-DGB_TRACE: the kernels
    record where each role waited; see gb_set_trace_buffer)."""
    out = TRACE_LIB if trace else LIB
    if not force and not _stale(out):
        return out
    os.makedirs(LOG_DIR, exist_ok=True)
    tag = f"{'trace.' if trace else ''}{os.getpid()}"
    flags = [*NVCC_FLAGS, *(["-DGB_TRACE"] if trace else [])]
    objs = [os.path.join(LOG_DIR, f"{s}.{tag}.o") for s in SOURCES]
    tmp = out + f".tmp{os.getpid()}"
    try:
        # one compiler process per source, all at once; their reports in the sources' order
        cmds = [[_nvcc(), *flags, "-c", os.path.join(CSRC, s), "-o", o] for s, o in zip(SOURCES, objs)]
        procs = [subprocess.Popen(c, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True) for c in cmds]
        logs = [p.communicate()[0] for p in procs]
        log = "".join(" ".join(c) + "\n" + text for c, text in zip(cmds, logs))
        failed = [p.returncode for p in procs if p.returncode]
        if not failed:
            link = subprocess.run([_nvcc(), *flags, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
            log += link.stdout + link.stderr
            failed = [link.returncode] if link.returncode else []
        with open(os.path.join(LOG_DIR, "ptxas_trace.log" if trace else "ptxas.log"), "w") as f:
            f.write(log)
        if failed:
            raise RuntimeError(f"nvcc failed ({failed[0]}):\n{log[-4000:]}")
        _check_register_budgets(log)
        if verbose:
            print(log)
        os.replace(tmp, out)
    finally:
        for path in (*objs, tmp):
            if os.path.exists(path):
                os.remove(path)
    return out


def _binding_command(out: str) -> list:
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    include = [*cpp_extension.include_paths(), sysconfig.get_paths()["include"]]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *[flag for path in include for flag in ("-isystem", path)], os.path.join(CSRC, "binding.cpp"), "-o", out,
            "-L" + lib, "-lc10", "-ltorch_cpu", "-ltorch", "-ltorch_python"]


def _binding_stamp() -> str:
    """What the binding is compiled for besides its source: a torch of another version, or elsewhere, needs another."""
    import torch
    return "\n".join([torch.__version__, *_binding_command(BINDING)])


def build_binding(force: bool = False) -> str:
    """Build _gbgemm_torch.so, the operators' binding to torch (argument marshalling only)."""
    stamp, kept = _binding_stamp(), os.path.join(LOG_DIR, "binding.stamp")
    if not force and not _stale(BINDING, ("binding.cpp",)) and os.path.exists(kept):
        with open(kept) as f:
            if f.read() == stamp:
                return BINDING
    os.makedirs(LOG_DIR, exist_ok=True)
    tmp = BINDING + f".tmp{os.getpid()}"
    try:
        res = subprocess.run(_binding_command(tmp), capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"the torch binding did not compile ({res.returncode}):\n{res.stderr[-4000:]}")
        os.replace(tmp, BINDING)
        with open(kept, "w") as f:
            f.write(stamp)
    finally:
        if os.path.exists(tmp):
            os.remove(tmp)
    return BINDING


if __name__ == "__main__":
    print(build(force=True, verbose=True))
    print(build_binding(force=True))
