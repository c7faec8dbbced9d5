"""Build libbl.so in-tree: nvcc for sm_103a, one translation unit per dtype compiled in
parallel, plus the host dispatcher; then, where torch is installed, _torch_binding.so, the training
operators' binding to torch tensors, with the host compiler against torch's headers. libbl.so needs
neither and is in place before the binding is looked at. The tuned selection tables (tuned/*.txt) are embedded as
string literals so the library needs no data files at run time (BL_TUNED_DIR still overrides).

Usage: python -m matrix_dense_linear_spd_gb300.build [--force] [--jobs N]
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import hashlib
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
TUNED = os.path.join(PKG, "tuned")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libbl.so")
BINDING = os.path.join(PKG, "_torch_binding.so")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-I", CSRC, "-I", INCLUDE]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _c_literal(text: str) -> str:
    out = []
    for line in text.splitlines(True):
        esc = line.replace("\\", "\\\\").replace('"', '\\"').replace("\n", "\\n")
        out.append(f'    "{esc}"')
    return "\n".join(out) if out else '    ""'


def gen_tables() -> str:
    """Write csrc/_tuned_tables.inc from tuned/*.txt; returns its content hash."""
    files = sorted(glob.glob(os.path.join(TUNED, "*.txt")))
    parts = ["// Generated by build.py from tuned/*.txt. Do not edit.",
             "static const char *const kTunedTables[][2] = {"]
    for f in files:
        name = os.path.basename(f)[:-4]
        parts.append(f'  {{"{name}",\n{_c_literal(open(f).read())}}},')
    if not files:
        parts.append('  {"", ""},')
    parts.append("};")
    text = "\n".join(parts) + "\n"
    path = os.path.join(CSRC, "_tuned_tables.inc")
    if not os.path.exists(path) or open(path).read() != text:
        with open(path, "w") as fh:
            fh.write(text)
    return hashlib.sha1(text.encode()).hexdigest()


def _deps_hash(src: str) -> str:
    h = hashlib.sha1()
    for f in [src] + sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
                            + glob.glob(os.path.join(CSRC, "*.inc")) + [os.path.join(INCLUDE, "bl.h")]):
        with open(f, "rb") as fh:
            h.update(fh.read())
    h.update(" ".join(ARCH + NVCC_FLAGS).encode())
    return h.hexdigest()


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    stamp = obj + ".sha"
    report = os.path.join(BUILD, os.path.basename(src) + ".ptxas.txt")
    digest = _deps_hash(src)
    if os.path.exists(obj) and os.path.exists(stamp) and open(stamp).read() == digest and \
            (src.endswith(".cpp") or os.path.exists(report)):
        return obj
    cmd = [nvcc()] + ARCH + NVCC_FLAGS + ["-Xptxas", "-v", "-c", src, "-o", obj]
    if src.endswith(".cpp"):
        cmd = [nvcc(), "-x", "cu"] + ARCH + NVCC_FLAGS + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if not src.endswith(".cpp"):
        # the ptxas resource report (registers, stack frame, spills) of every kernel of this
        # translation unit, for the register gate (tests/test_register_gate.py)
        with open(report, "w") as fh:
            fh.write(r.stderr)
    with open(stamp, "w") as fh:
        fh.write(digest)
    return obj


def _torch_dir() -> str:
    spec = importlib.util.find_spec("torch")          # without importing it
    if spec is None or not spec.submodule_search_locations:
        raise RuntimeError("torch not found: the training operators' binding needs its headers")
    return spec.submodule_search_locations[0]


def _compile_binding() -> str:
    src = os.path.join(CSRC, "binding", "torch_binding.cpp")
    obj = os.path.join(BUILD, "torch_binding.cpp.o")
    stamp = obj + ".sha"
    torch_dir = _torch_dir()
    with open(os.path.join(torch_dir, "version.py")) as fh:
        version = fh.read()
    flags = ["-O2", "-std=c++17", "-fPIC", "-I", os.path.join(torch_dir, "include"),
             "-I", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
             "-I", sysconfig.get_paths()["include"],
             "-I", os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    digest = hashlib.sha1((_deps_hash(src) + version + " ".join(flags)).encode()).hexdigest()
    if os.path.exists(obj) and os.path.exists(stamp) and open(stamp).read() == digest:
        return obj
    r = subprocess.run(["g++"] + flags + ["-c", src, "-o", obj], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {src}:\n{r.stdout}\n{r.stderr}")
    with open(stamp, "w") as fh:
        fh.write(digest)
    return obj


def _link_binding(obj: str) -> None:
    lib = os.path.join(_torch_dir(), "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, obj, LIB, "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10",
           f"-Wl,-rpath,{lib}", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)


def parse_ptxas(text: str):
    """[{name, registers, stack, spill_stores, spill_loads}] for every function in a ptxas -v
    report (the mangled name; functions that report no register line have registers None)."""
    import re
    out, cur = [], None
    for line in text.splitlines():
        m = re.search(r"Function properties for (\S+)", line)
        if m:
            cur = {"name": m.group(1), "registers": None, "stack": 0, "spill_stores": 0, "spill_loads": 0}
            out.append(cur)
            continue
        m = re.search(r"(\d+) bytes stack frame, (\d+) bytes spill stores, (\d+) bytes spill loads", line)
        if m and cur is not None:
            cur["stack"], cur["spill_stores"], cur["spill_loads"] = (int(x) for x in m.groups())
            continue
        m = re.search(r"Used (\d+) registers", line)
        if m and cur is not None:
            cur["registers"] = int(m.group(1))
    return out


def ptxas_reports():
    """{translation unit: parsed report} for the current build (build() first)."""
    res = {}
    for f in sorted(glob.glob(os.path.join(BUILD, "*.ptxas.txt"))):
        with open(f) as fh:
            res[os.path.basename(f)[: -len(".ptxas.txt")]] = parse_ptxas(fh.read())
    return res


def build(force: bool = False, jobs: int | None = None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    gen_tables()
    if force:
        for f in glob.glob(os.path.join(BUILD, "*")):
            os.remove(f)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))
    jobs = jobs or max(1, min(len(srcs), os.cpu_count() or 1))
    with cf.ThreadPoolExecutor(jobs) as ex:
        binding = ex.submit(_compile_binding) if importlib.util.find_spec("torch") else None
        objs = list(ex.map(_compile, srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + objs + ["-Xlinker", "--no-undefined", "-Xlinker", "-soname=libbl.so"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if binding is None:
        print("torch is not installed: the training operators' binding to its tensors is not built", file=sys.stderr)
    else:
        _link_binding(binding.result())
    return LIB


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--jobs", type=int, default=None)
    a = ap.parse_args(argv)
    print(build(a.force, a.jobs))


if __name__ == "__main__":
    main(sys.argv[1:])
