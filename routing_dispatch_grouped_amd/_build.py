"""Build librdg.so (HIP, gfx950) in-tree with hipcc, and _binding.so, the part of the Python binding that is in C++."""
import concurrent.futures
import importlib.util
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT = os.path.join(PKG, "librdg.so")
BINDING = os.path.join(PKG, "_binding.so")
BUILD = os.path.join(PKG, "_build")

SOURCES = ["abi.hip", "route.hip", "dispatch.hip", "quant.hip", "pack.hip", "ffn.hip", "ffn_tiled.hip", "combine.hip",
           "kvplan.hip", "qkstore.hip", "attn.hip", "attn_tiles.hip",
           "abi_kv.hip", "addnorm.hip", "linear.hip", "linear_tiled.hip", "abi_layer.hip", "eplb.cpp", "tbo.cpp"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    # keep hand-written float code off the packed fp32 instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-result",
    "-I", INCLUDE, "-I", CSRC,
]


# host-only sources (no device code): the system C++ compiler, plain IEEE
# double arithmetic
CXX = os.environ.get("CXX", "g++")
CXXFLAGS = ["-O2", "-std=c++17", "-fPIC", "-ffp-contract=off", "-Wall", "-I", INCLUDE, "-I", CSRC]


def _compile(src):
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    if src.endswith(".cpp"):
        cmd = [CXX] + CXXFLAGS + ["-c", os.path.join(CSRC, src), "-o", obj]
    else:
        cmd = [HIPCC] + FLAGS + ["-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("compile failed for %s:\n%s\n%s" % (src, " ".join(cmd), r.stderr))
    return obj


def _compile_binding():
    """binding.cpp against torch's headers, found without importing torch."""
    obj = os.path.join(BUILD, "binding.o")
    include = os.path.join(_torch(), "include")
    cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-Wall", "-I", INCLUDE, "-isystem", include, "-isystem",
           os.path.join(include, "torch", "csrc", "api", "include"), "-isystem", sysconfig.get_paths()["include"],
           "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("compile failed for binding.cpp:\n%s\n%s" % (" ".join(cmd), r.stderr))
    return obj


def _torch():
    """torch's folder, None where there is no torch (the library needs none)."""
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec else None


def _link_binding(obj):
    """Next to librdg.so, which it finds by its own folder; torch's libraries are those that the process has loaded."""
    tmp = BINDING + ".tmp"
    cmd = [CXX, "-shared", "-o", tmp, obj, "-L", PKG, "-l:librdg.so", "-Wl,-rpath,$ORIGIN", "-L", os.path.join(_torch(), "lib"),
           "-lc10", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed for _binding.so:\n%s" % r.stderr)
    os.replace(tmp, BINDING)


def build(verbose=False):
    os.makedirs(BUILD, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(len(SOURCES) + 1, os.cpu_count() or 4)) as ex:
        binding = ex.submit(_compile_binding) if _torch() else None
        objs = list(ex.map(_compile, SOURCES))
    tmp = OUT + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s" % r.stderr)
    os.replace(tmp, OUT)
    if verbose:
        print("built", OUT)
    if binding is not None:
        _link_binding(binding.result())
    elif verbose:
        print("no torch here, so no", BINDING)
    return OUT


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
