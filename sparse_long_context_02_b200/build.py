"""Builds libdsa_b200.so (the CUDA kernels and the C ABI of include/dsa.h)
in place, for sm_100a."""
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB_PATH = os.path.join(HERE, "libdsa_b200.so")
SOURCES = [os.path.join(CSRC, "dsa_lib.cu")]
# the benchmark's L2 bandwidth and FP8 tensor-rate probes: a separate library,
# not part of the ABI
PROBE_SOURCE = os.path.join(CSRC, "probe_l2.cu")
PROBE_PATH = os.path.join(HERE, "libdsa_probe.so")
# the Python side's argument marshalling (host code, torch's C++ API)
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")
BINDING_PATH = os.path.join(HERE, "_native.so")
BINDING_STAMP = os.path.join(HERE, "_native.built_for")  # binding_key() of that file
DEPS = SOURCES + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cuh")] + [
    os.path.join(ROOT, "include", "dsa.h")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-shared", "-cudart", "static",
]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def build_probe(force: bool = False) -> str:
    deps = (PROBE_SOURCE, os.path.join(CSRC, "ptx.cuh"))
    if (not force and os.path.exists(PROBE_PATH)
            and os.path.getmtime(PROBE_PATH) >= max(os.path.getmtime(d) for d in deps)):
        return PROBE_PATH
    tmp = PROBE_PATH + f".tmp{os.getpid()}"
    subprocess.check_call([nvcc(), *NVCC_FLAGS, "-o", tmp, PROBE_SOURCE])
    os.replace(tmp, PROBE_PATH)
    return PROBE_PATH


def binding_key() -> str:
    """What the binding depends on beside its source: it reads tensors through
    torch's inline accessors and calls CPython's API, so it serves this torch and
    this Python only."""
    import torch
    return (f"torch {torch.__version__}, C++ ABI {int(torch._C._GLIBCXX_USE_CXX11_ABI)}, "
            f"Python {sysconfig.get_config_var('SOABI')}")


def _stamp() -> str:
    try:
        with open(BINDING_STAMP) as f:
            return f.read()
    except OSError:
        return ""


def build_binding(force: bool = False) -> str:
    deps = (BINDING_SOURCE, os.path.join(ROOT, "include", "dsa.h"))
    key = binding_key()
    if (not force and os.path.exists(BINDING_PATH) and _stamp() == key
            and os.path.getmtime(BINDING_PATH) >= max(os.path.getmtime(d) for d in deps)):
        return BINDING_PATH
    import torch
    at = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc())) or "/usr/local/cuda"
    tmp = BINDING_PATH + f".tmp{os.getpid()}"
    lib = os.path.join(at, "lib")
    subprocess.check_call([
        os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
        "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
        f'-DDSA_BUILT_FOR="{key}"',
        "-I", os.path.join(ROOT, "include"), "-isystem", os.path.join(at, "include"),
        "-isystem", os.path.join(at, "include", "torch", "csrc", "api", "include"),
        "-isystem", os.path.join(cuda, "include"),
        "-isystem", sysconfig.get_paths()["include"], "-o", tmp, BINDING_SOURCE,
        "-L", lib, f"-Wl,-rpath,{lib}", "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10",
        "-ldl"])
    if os.path.exists(BINDING_STAMP):  # never beside a file that it does not describe
        os.remove(BINDING_STAMP)
    os.replace(tmp, BINDING_PATH)
    with open(BINDING_STAMP, "w") as f:
        f.write(key)
    return BINDING_PATH


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    build_probe(force)
    build_binding(force)
    if (not force and os.path.exists(LIB_PATH)
            and os.path.getmtime(LIB_PATH) >= max(os.path.getmtime(d) for d in DEPS)):
        return LIB_PATH
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc(), *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           *(["-Xptxas", "-v"] if verbose_ptxas else []), "-o", tmp, *SOURCES]
    subprocess.check_call(cmd)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose_ptxas="-v" in sys.argv))
