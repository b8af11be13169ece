"""Build libseqattn.so in-tree: one nvcc per translation unit, in parallel,
for sm_103a only, then one shared-library link; and beside it _marshal.so, the
binding's argument checks in C++ against the installed PyTorch.  Usage:

    python -m long_context_attention_seqattn_gb300.build [--force] [--verbose]
"""

import hashlib
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(PKG, "libseqattn.so")
MARSHAL_PATH = os.path.join(PKG, "_marshal.so")

SOURCES = ["seqattn_api.cu", "simt_f32.cu", "fwd_bf16.cu", "bwd_bf16.cu", "wgrad_bf16.cu",
           "linear_bf16.cu", "norm_rope.cu", "adamw.cu"]
LIBS = []
HEADERS = ["internal.h", "sm103_ptx.cuh"]
MARSHAL = "marshal.cpp"      # host only: g++, PyTorch's headers

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
          "-I", INCLUDE, "-I", CSRC]


def _nvcc():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def _fingerprint():
    h = hashlib.sha256()
    for f in SOURCES + HEADERS + [MARSHAL]:
        with open(os.path.join(CSRC, f), "rb") as fh:
            h.update(f.encode() + fh.read())
    with open(os.path.join(INCLUDE, "seqattn.h"), "rb") as fh:
        h.update(fh.read())
    h.update(" ".join(ARCH + CFLAGS + LIBS).encode())
    import torch
    h.update((torch.__version__ + sys.version).encode())     # what _marshal.so is compiled against
    return h.hexdigest()


def _marshal_commands():
    """Compile and link commands of _marshal.so."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    obj = os.path.join(BUILD_DIR, "marshal.o")
    cuda = os.path.dirname(os.path.dirname(_nvcc())) if os.path.isabs(_nvcc()) else "/usr/local/cuda"
    compile_ = ["g++", "-std=c++17", "-O2", "-fPIC", "-Wall", "-I", INCLUDE]
    for d in (os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
              os.path.join(cuda, "include"), sysconfig.get_paths()["include"]):
        compile_ += ["-isystem", d]
    compile_ += [f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                 "-c", os.path.join(CSRC, MARSHAL), "-o", obj]
    lib = os.path.join(root, "lib")
    link = ["g++", "-shared", "-o", MARSHAL_PATH + ".tmp", obj, "-L", PKG, "-l:libseqattn.so", "-L", lib, "-lc10",
            "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    return obj, compile_, link


def build(force=False, verbose=False):
    """Compile every CUDA translation unit for sm_103a and link libseqattn.so,
    then _marshal.so.  Skips the work when the sources (and the PyTorch that
    _marshal.so is compiled against) are unchanged since the last build."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    stamp = os.path.join(BUILD_DIR, "fingerprint")
    fp = _fingerprint()
    if not force and os.path.exists(LIB_PATH) and os.path.exists(MARSHAL_PATH) and os.path.exists(stamp):
        with open(stamp) as fh:
            if fh.read().strip() == fp:
                return LIB_PATH
    nvcc = _nvcc()

    marshal_obj, marshal_compile, marshal_link = _marshal_commands()

    def compile_one(src):
        if src == MARSHAL:
            return src, marshal_obj, subprocess.run(marshal_compile, capture_output=True, text=True)
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        cmd = [nvcc] + ARCH + CFLAGS + ["-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, r

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        results = list(ex.map(compile_one, SOURCES + [MARSHAL]))
    for src, _, r in results:
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"compiling {src} failed:\n{r.stdout}\n{r.stderr}")
    cmd = [nvcc] + ARCH + ["-shared", "-o", LIB_PATH + ".tmp"] + [o for s, o, _ in results if s != MARSHAL] + LIBS
    for path, cmd in ((LIB_PATH, cmd), (MARSHAL_PATH, marshal_link)):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(path + ".tmp", path)
    with open(stamp, "w") as fh:
        fh.write(fp)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
