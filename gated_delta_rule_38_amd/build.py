"""Builds libkda.so (the gfx950 C-ABI library) in-tree with hipcc, and _layer_binding.so (the
extension module that passes torch tensors to its layer operators) with the host compiler.

    python -m gated_delta_rule_38_amd.build
"""
import concurrent.futures
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libkda.so")
SOURCES = ["kda_api.cpp", "kda_chunk.hip", "kda_chunk_pipe.hip", "kda_prep.hip", "kda_combine.hip", "kda_decode.hip",
           "kda_peak.hip", "kda_layer_api.cpp", "kda_conv.hip", "kda_qk_norm.hip", "kda_ssm.hip", "kda_ssm_decode.hip"]
# -packed-fp32-ops: no v_pk_*_f32 generation in device code.
FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def _compile(src: str, obj: str) -> None:
    cmd = [hipcc(), *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{r.stderr}")


def _build_binding() -> str:
    """_layer_binding.so, the torch side of the layer operators (host code only)."""
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths
    out = os.path.join(HERE, "_layer_binding.so")
    libdir = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-I{d}" for d in (*include_paths(), sysconfig.get_paths()["include"])),
           os.path.join(CSRC, "layer_binding.cpp"), "-o", out + ".tmp",
           f"-L{libdir}", f"-Wl,-rpath,{libdir}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on layer_binding.cpp:\n{r.stderr}")
    os.replace(out + ".tmp", out)
    return out


def build(verbose: bool = True) -> str:
    bdir = os.path.join(HERE, "_build")
    os.makedirs(bdir, exist_ok=True)
    objs = [os.path.join(bdir, os.path.splitext(s)[0] + ".o") for s in SOURCES]
    with concurrent.futures.ThreadPoolExecutor(max_workers=8) as ex:
        binding = ex.submit(_build_binding)
        list(ex.map(_compile, SOURCES, objs))
        binding.result()
    tmp = LIB + ".tmp"
    r = subprocess.run([hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build()
    sys.exit(0)
