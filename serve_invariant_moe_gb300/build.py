"""Build libinvmoe.so in-tree with nvcc for sm_103a (no cmake, no torch extension machinery), and _marshal.so beside it.

Each .cu translation unit is compiled in parallel into ``_build/`` and linked
into ``serve_invariant_moe_gb300/libinvmoe.so``; csrc/marshal.cpp (the binding's
CPython helpers, against the installed torch's headers) becomes ``_marshal.so``.
A unit is recompiled only when it, or a header in csrc/ or include/, is newer
than its object file, the helpers also when torch or Python is another one.
"""
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libinvmoe.so")
MARSHAL = os.path.join(PKG, "_marshal.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
                     "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cpp")))


def _object(src):
    return os.path.join(BUILD, os.path.splitext(os.path.basename(src))[0] + ".o")


def _torch_dirs():
    """Headers and libraries of the installed torch."""
    import torch
    root = os.path.dirname(torch.__file__)
    return os.path.join(root, "include"), os.path.join(root, "lib"), int(torch._C._GLIBCXX_USE_CXX11_ABI)


def _host():
    """What the helpers' object was compiled against: torch's C++ interface and Python's change with their versions."""
    import torch
    return "\n".join([torch.__version__, torch.__file__, sys.version])


def _compile_command(src, obj, verbose_ptxas):
    if src.endswith(".cu"):
        return [nvcc()] + NVCC_FLAGS + (["-Xptxas", "-v"] if verbose_ptxas else []) + ["-c", src, "-o", obj]
    include, _, abi = _torch_dirs()
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={abi}",
            "-isystem", include, "-isystem", cuda, "-isystem", sysconfig.get_paths()["include"], "-c", src, "-o", obj]


def _link(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")


def _stale(out, inputs):
    return not os.path.exists(out) or os.path.getmtime(out) < max(os.path.getmtime(i) for i in inputs)


def _headers_mtime():
    m = 0.0
    for d in (CSRC, INCLUDE):
        for f in os.listdir(d):
            if f.endswith((".h", ".cuh", ".hpp")):
                m = max(m, os.path.getmtime(os.path.join(d, f)))
    return m


def _compile(src, verbose_ptxas=False):
    obj = _object(src)
    r = subprocess.run(_compile_command(src, obj, verbose_ptxas), capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compilation failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def build(force: bool = False, verbose_ptxas: bool = False, jobs: int = None) -> str:
    """Compile and link; returns the path of libinvmoe.so."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    hdr = _headers_mtime()
    todo = []
    marshal_src, stamp, host = os.path.join(CSRC, "marshal.cpp"), os.path.join(BUILD, "marshal.host"), _host()
    same_host = os.path.exists(stamp) and open(stamp).read() == host
    for s in srcs:
        obj = _object(s)
        if (force or verbose_ptxas or not os.path.exists(obj) or os.path.getmtime(obj) < max(os.path.getmtime(s), hdr)
                or (s == marshal_src and not same_host)):
            todo.append(s)
    logs = []
    if todo:
        with cf.ThreadPoolExecutor(max_workers=jobs or min(len(todo), os.cpu_count() or 4)) as ex:
            for obj, err in ex.map(lambda s: _compile(s, verbose_ptxas), todo):
                logs.append(err)
    objs = [_object(s) for s in srcs if s.endswith(".cu")]
    if todo or _stale(LIB, objs):
        _link([nvcc()] + ARCH + ["-shared", "-o", LIB + ".tmp"] + objs + ["-cudart", "static"])
        os.replace(LIB + ".tmp", LIB)
    marshal = _object(marshal_src)
    if todo or _stale(MARSHAL, [marshal, LIB]):
        torch_lib = _torch_dirs()[1]
        # libinvmoe.so is found beside it; torch's libraries are in the process already
        _link(["g++", "-shared", "-o", MARSHAL + ".tmp", marshal, "-L", PKG, "-l:libinvmoe.so", "-Wl,-rpath,$ORIGIN",
               "-L", torch_lib, f"-Wl,-rpath,{torch_lib}", "-lc10", "-ltorch_cpu", "-lc10_cuda", "-ltorch_cuda",
               "-ltorch_python"])
        os.replace(MARSHAL + ".tmp", MARSHAL)
    if not same_host:
        with open(stamp, "w") as f:
            f.write(host)
    if verbose_ptxas:
        sys.stderr.write("".join(logs))
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
