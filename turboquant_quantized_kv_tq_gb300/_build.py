"""Build the C-ABI library ``libtq.so`` in-tree for sm_103a (GB300).

Each translation unit is compiled in parallel with nvcc (CUDA sources) or g++ (host sources),
then linked into ``turboquant_quantized_kv_tq_gb300/_lib/libtq.so`` with the CUDA runtime linked
statically.  Beside it goes ``_lib/_tq_torch.so``, the Python extension of ``byte_cache`` (torch
tensors to the C ABI), where a torch with CUDA is installed; the library itself does not need torch.
Objects go to ``_build/`` at the repository root.
"""

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_DIR = os.path.join(PKG, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libtq.so")
EXT_SRC = os.path.join(CSRC, "python", "tq_torch.cpp")
EXT_PATH = os.path.join(LIB_DIR, "_tq_torch.so")
OBJ_DIR = os.path.join(ROOT, "_build", "obj")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _cuda_home():
    home = os.environ.get("CUDA_HOME") or os.environ.get("CUDA_PATH")
    if home and os.path.isdir(home):
        return home
    nvcc = shutil.which("nvcc")
    if nvcc:
        return os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    return "/usr/local/cuda"


def sources():
    return sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cpp")))


def _compile(src, extra_nvcc=()):
    cuda = _cuda_home()
    nvcc = os.path.join(cuda, "bin", "nvcc")
    out = os.path.join(OBJ_DIR, src + ".o")
    path = os.path.join(CSRC, src)
    if src.endswith(".cu"):
        cmd = [nvcc, *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-ffp-contract=off",
               "-I", INCLUDE, "-I", CSRC, *extra_nvcc, "-c", path, "-o", out]
    else:
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-ffp-contract=off", "-I", INCLUDE, "-I", CSRC,
               "-I", os.path.join(cuda, "include"), "-c", path, "-o", out]
    res = subprocess.run(cmd, capture_output=True, text=True)
    return src, res.returncode, res.stdout + res.stderr, out


def _torch_dir():
    """The folder of an installed torch with CUDA, or None."""
    try:
        import torch
    except ImportError:
        return None
    path = os.path.dirname(torch.__file__)
    return path if os.path.exists(os.path.join(path, "lib", "libc10_cuda.so")) else None


def _compile_ext(torch_dir):
    import sysconfig

    import torch
    inc = os.path.join(torch_dir, "include")
    out = os.path.join(OBJ_DIR, "tq_torch.cpp.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           "-I", INCLUDE, "-isystem", inc, "-isystem", os.path.join(_cuda_home(), "include"),
           "-I", sysconfig.get_paths()["include"], "-c", EXT_SRC, "-o", out]
    res = subprocess.run(cmd, capture_output=True, text=True)
    return EXT_SRC, res.returncode, res.stdout + res.stderr, out


def _link_ext(obj, torch_dir):
    lib = os.path.join(torch_dir, "lib")
    tmp = EXT_PATH + ".tmp"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", LIB_DIR, "-l:libtq.so", "-Wl,-rpath,$ORIGIN", "-L", lib,
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("linking _tq_torch.so failed:\n" + res.stdout + res.stderr)
    os.replace(tmp, EXT_PATH)


def _checked(result, verbose):
    src, rc, log, out = result
    if verbose and log.strip():
        print(f"[{src}]\n{log}", file=sys.stderr)
    if rc != 0:
        raise RuntimeError(f"compiling {src} failed:\n{log}")
    return out


def build(verbose=False, extra_nvcc=()):
    """Compile every source and link libtq.so, then the torch extension; raise RuntimeError on the first failure."""
    os.makedirs(OBJ_DIR, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    srcs = sources()
    torch_dir = _torch_dir()
    with ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        ext = ex.submit(_compile_ext, torch_dir) if torch_dir else None
        results = list(ex.map(lambda s: _compile(s, extra_nvcc), srcs))
    objs = [_checked(r, verbose) for r in results]
    cuda = _cuda_home()
    tmp = LIB_PATH + ".tmp"
    cmd = [os.path.join(cuda, "bin", "nvcc"), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("linking libtq.so failed:\n" + res.stdout + res.stderr)
    os.replace(tmp, LIB_PATH)
    if ext is not None:
        _link_ext(_checked(ext.result(), verbose), torch_dir)
    else:
        if os.path.exists(EXT_PATH):  # (of an earlier build, for another library)
            os.remove(EXT_PATH)
        if verbose:
            print("no torch with CUDA: _tq_torch.so (byte_cache) is not built", file=sys.stderr)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
