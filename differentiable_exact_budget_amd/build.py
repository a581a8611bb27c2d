"""Build the gfx950 HIP library liblapsum.so in-tree with hipcc, and with g++
the torch module of the expert operators (_experts_torch.so, host code only).

Every HIP source is compiled for gfx950 only; packed-fp32 instruction
selection is disabled (-Xclang -target-feature -Xclang -packed-fp32-ops).
"""
import concurrent.futures as cf
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
OUT = os.path.join(HERE, "liblapsum.so")
BUILD = os.path.join(ROOT, "_build")
TORCH_SOURCE = "experts_torch.cpp"
TORCH_OUT = os.path.join(HERE, "_experts_torch.so")

SOURCES = ["lapsum_sample.hip", "lapsum_stream.hip", "lapsum_sort.hip", "lapsum_ceiling.hip", "lapsum_topk.hip", "lapsum_batched.hip", "lapsum_heavy.hip", "lapsum_noalloc.hip", "lapsum_route.hip", "lapsum_tokens.hip",
           "lapsum_expert_linear.hip", "lapsum_expert_mfma.hip", "lapsum_expert_few.hip",
           "lapsum_host.cpp", "lapsum_experts_host.cpp"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = ["-O3", "-std=c++17", "-fPIC", "--offload-arch=gfx950", "-Xclang", "-target-feature", "-Xclang",
         "-packed-fp32-ops", "-Wall", "-Wno-unused-function", "-I", os.path.join(ROOT, "include")]
# The matrix kernels' loops are written in the order they are to be issued; the
# compiler's own scheduler lengthens live ranges past the register file there
# and spills (the weight gradient's step of 16384 x 2 rows, 2048 x 4096: 1.76 ms
# instead of 0.44 ms).
SOURCE_FLAGS = {"lapsum_expert_mfma.hip": ["-mllvm", "-enable-misched=false"]}


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [HIPCC, "-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj] + FLAGS + SOURCE_FLAGS.get(src, [])
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    err = "\n".join(ln for ln in (res.stderr or "").splitlines() if "packed-fp32-ops" not in ln
                    and "is not a recognized feature for this target" not in ln)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{err}")
    if verbose and err.strip():
        print(err, flush=True)
    return obj


def _run(cmd, what: str, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{res.stderr}")


def _compile_torch(verbose: bool) -> str:
    """The torch module's object, with the headers of the torch in use."""
    import torch
    import sysconfig
    root = os.path.dirname(torch.__file__)
    obj = os.path.join(BUILD, TORCH_SOURCE + ".o")
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], "/opt/rocm/include", os.path.join(ROOT, "include")]
    _run(["g++", "-c", os.path.join(CSRC, TORCH_SOURCE), "-o", obj, "-O2", "-std=c++17", "-fPIC", "-w",
          "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1", "-DTORCH_EXTENSION_NAME=_experts_torch",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
         + [f for d in inc for f in ("-isystem", d)], f"g++ on {TORCH_SOURCE}", verbose)
    return obj


def _link_torch(obj: str, verbose: bool) -> None:
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    _run(["g++", "-shared", "-o", TORCH_OUT + ".tmp", obj, "-L" + HERE, "-l:liblapsum.so", "-L" + libs, "-lc10",
          "-lc10_hip", "-ltorch_cpu", "-ltorch", "-ltorch_python", "-Wl,-rpath,$ORIGIN"], "link of the torch module",
         verbose)
    os.replace(TORCH_OUT + ".tmp", TORCH_OUT)


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(4, len(SOURCES))) as ex:
        torch_obj = ex.submit(_compile_torch, verbose)
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
        torch_obj = torch_obj.result()
    cmd = [HIPCC, "-shared", "-fPIC", "--offload-arch=gfx950", "-o", OUT + ".tmp"] + objs
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stderr}")
    os.replace(OUT + ".tmp", OUT)
    _link_torch(torch_obj, verbose)
    return OUT


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
