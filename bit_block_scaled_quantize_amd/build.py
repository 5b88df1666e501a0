"""Build libnvfp4.so (the HIP kernels + C ABI) in-tree for gfx950 with hipcc,
and _native.so, the Python binding of the MoE-block operators, against it with
the host compiler.

Flags that matter for correctness:
  -ffp-contract=off            every a*b+c rounds twice, as the format's
                               definition is written (no FMA contraction);
  -fhip-fp32-correctly-rounded-divide-sqrt
                               the per-block division and reciprocal are
                               correctly rounded binary32 operations;
  -fno-gpu-flush-denormals-to-zero
                               binary32 subnormals are kept;
  -Xclang -target-feature -Xclang -packed-fp32-ops
                               no packed FP32 instructions are generated.
"""
import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libnvfp4.so")
BINDING = os.path.join(HERE, "_native.so")
BUILD = os.path.join(HERE, "_build")
SOURCES = ["quantize.hip", "gemm.hip", "mx.hip", "mx_gemm.hip", "norm.hip", "route.hip", "gemv.hip", "nvfp4_api.hip"]
ARCH = os.environ.get("NVFP4_OFFLOAD_ARCH", "gfx950")


def hipcc():
    exe = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(exe):
        raise RuntimeError("hipcc not found; the NVFP4 HIP library cannot be built")
    return exe


def flags():
    return ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
            "-ffp-contract=off", "-fhip-fp32-correctly-rounded-divide-sqrt",
            "-fno-gpu-flush-denormals-to-zero",
            # loops marked for full unrolling stay unrolled even when the body
            # is large (a rolled loop would index register arrays dynamically)
            "-mllvm", "-pragma-unroll-threshold=262144",
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            "-Wall", "-Wno-unused-function",
            "-I", CSRC, "-I", INCLUDE]


def _compile(src):
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [hipcc()] + flags() + ["-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def _compile_binding():
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        raise RuntimeError("no host C++ compiler found; the Python binding cannot be built")
    import torch  # (the C library is built without it)
    torch_dir = os.path.dirname(torch.__file__)
    inc = os.path.join(torch_dir, "include")
    obj = os.path.join(BUILD, "binding.o")
    # (the std::string of torch's own interface)
    abi = f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}"
    cmd = [cxx, "-O2", "-std=c++17", abi, "-fPIC", "-fvisibility=hidden", "-Wall", "-Wno-unused-function", "-I", INCLUDE,
           "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cxx} failed for binding.cpp:\n{r.stdout}\n{r.stderr}")
    return cxx, obj, os.path.join(torch_dir, "lib")


def _link_binding(cxx, obj, torch_lib):
    # torch is loaded before the module is imported; libnvfp4.so lies beside it
    tmp = BINDING + ".tmp"
    cmd = [cxx, "-shared", "-o", tmp, obj, "-L", HERE, "-l:libnvfp4.so", "-L", torch_lib, "-ltorch_python", "-ltorch_cpu",
           "-lc10", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + torch_lib]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the binding failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)


def build(verbose=False):
    """Compile every source and link libnvfp4.so and _native.so (always rebuilds)."""
    os.makedirs(BUILD, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_compile_binding)
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_binding(*binding.result())  # (the library is there whether or not the binding can be)
    if verbose:
        print(LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
