"""Build step for the C-ABI library ``liblora_linear.so`` (sm_103a), in-tree.

Compiles the library's translation units in parallel with nvcc for
``-gencode arch=compute_103a,code=sm_103a`` and links them into
``mixed_lora_projection_gb300/liblora_linear.so`` (CUDA runtime linked statically, no
libcuda link: the tensor-map encoder is fetched through the runtime's driver entry
point, so the library also loads on a machine without a GPU). The operators' Python
binding, ``_layer_bind.so``, is the one unit compiled against PyTorch's headers; where there is
no PyTorch, run this file as a script, and the library alone is built.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "liblora_linear.so")
BIND = os.path.join(PKG, "_layer_bind.so")
BIND_FOR = os.path.join(BUILD, "layer_bind.for")       # the PyTorch and the Python that the binding was built for
BIND_SOURCE = "layer_bind.cpp"
SOURCES = ["kernels.cu", "kernels_w4.cu", "kernels_fp8.cu", "api.cpp", "planner.cpp", "noalloc.cu",
           "layer_ops.cu", "act_fp8.cu", "logprobs.cu", "attn_decode.cu", "attn_prompt.cu", "layer_api.cpp"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build liblora_linear.so")


def _sources():
    return [s for s in SOURCES if os.path.exists(os.path.join(CSRC, s))]


def bind_for() -> str:
    """What a binding is built for; file times do not tell, so it says so itself (``built_for``)."""
    import torch
    return f"PyTorch {torch.__version__}, {sys.implementation.cache_tag}"


def _stale() -> bool:
    outputs = [LIB]
    if _torch_flags():
        outputs += [BIND, BIND_FOR]
    if not all(os.path.exists(f) for f in outputs):
        return True
    if BIND in outputs:
        with open(BIND_FOR) as f:
            if f.read() != bind_for():
                return True
    t = min(os.path.getmtime(f) for f in outputs)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [
        os.path.join(ROOT, "include", h) for h in ("lora_linear.h", "lora_layer.h")]
    return any(os.path.getmtime(d) > t for d in deps if os.path.exists(d))


def _torch_flags() -> tuple[list, list] | None:
    """How the binding is compiled and linked against PyTorch; None where there is no PyTorch."""
    try:
        import torch
    except ImportError:
        return None
    root = os.path.dirname(torch.__file__)
    libs = os.path.join(root, "lib")
    return (["-I", os.path.join(root, "include"), "-I", sysconfig.get_paths()["include"],
             f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DLAYER_BIND_FOR="{bind_for()}"'],
            ["-L", libs, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-Xlinker", f"-rpath={libs}"])


def build(verbose: bool = False, ptxas_info: bool = False) -> str:
    """Builds the library, and the binding where PyTorch is there. The library is linked first: it needs neither
    PyTorch nor a binding that compiles."""
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    torch_flags = _torch_flags()
    common = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2", "-I", os.path.join(ROOT, "include")]

    def compile_one(src, flags=()):
        obj = os.path.join(BUILD, src + ".o")
        cmd = [nvcc, *ARCH, *common, "-c", os.path.join(CSRC, src), "-o", obj, *flags]
        if ptxas_info and src.endswith(".cu"):
            cmd += ["-Xptxas", "-v"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        log = r.stdout + r.stderr
        if (verbose or ptxas_info) and log.strip():
            print(log, file=sys.stderr)
        return obj

    def link(target, objs, flags=()):
        r = subprocess.run([nvcc, *ARCH, "-shared", "-o", target + ".tmp", *objs, *flags], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(target + ".tmp", target)

    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        objs = [ex.submit(compile_one, s) for s in srcs]
        bind = ex.submit(compile_one, BIND_SOURCE, torch_flags[0]) if torch_flags else None
        link(LIB, [o.result() for o in objs])
        if bind:
            link(BIND, [bind.result()], torch_flags[1])
            with open(BIND_FOR, "w") as f:
                f.write(bind_for())
    return LIB


def ensure_built() -> str:
    if _stale():
        return build()
    return LIB


if __name__ == "__main__":
    print(build(verbose=True, ptxas_info="--ptxas" in sys.argv))
