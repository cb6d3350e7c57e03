"""Build librcc.so in-tree: the CUDA kernels and the C-ABI host layer; and
_lm.so, the torch binding of the language-model operators.

nvcc, one -gencode for sm_103a, the translation units compiled in parallel,
static CUDA runtime, only the rcc_* symbols exported.  No fast-math: means use
IEEE division and bf16 outputs round to nearest even.
"""
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "librcc.so")
BINDING = os.path.join(HERE, "_lm.so")

NVCC = os.environ.get("NVCC", "nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
COMMON = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
          "-I", INCLUDE, "-I", CSRC]
SOURCES = ["gradsync.cu", "embedding.cu", "rmsnorm.cu", "linear_ce.cu", "rcc_host.cpp",
           "rcc_rank.cpp", "rcc_gradsync_host.cpp", "rcc_lm_host.cpp"]
# collectives_part.cu is compiled once per (element type, reduction, tree
# order) that the host dispatcher names: fp32 (0) and bf16 (1) x rank-order
# sum (0), tree sum (0, fast), max (1), min (2), copy (3).
PARTS = [(dt, red, fast) for dt in (0, 1)
         for red, fast in ((0, 0), (0, 1), (1, 0), (2, 0), (3, 0))]


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "rcc.h"))
    files.append(os.path.abspath(__file__))
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BINDING):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return all(os.path.getmtime(f) <= t for f in _inputs())


def binding_command(out: str):
    """g++ on lm_binding.cpp with Python's and torch's headers and libraries."""
    import importlib.util
    import sysconfig
    torch_dir = list(importlib.util.find_spec("torch").submodule_search_locations)[0]
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    lib = os.path.join(torch_dir, "lib")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-D_GLIBCXX_USE_CXX11_ABI=1",
            "-I", INCLUDE, "-I", sysconfig.get_paths()["include"],
            "-isystem", os.path.join(torch_dir, "include"),
            "-isystem", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
            "-isystem", cuda, os.path.join(CSRC, "lm_binding.cpp"), "-o", out,
            "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
            "-Wl,-rpath," + lib]


def build(force: bool = False, verbose: bool = False, defines=(), lib: str = LIB,
          objdir: str = OBJDIR) -> str:
    """Compile librcc.so.  `defines` (e.g. ["-DRCC_WAVES=8"]) rebuild the
    kernels with other tuning macros into `lib` / `objdir` (a comparison
    build that RCC_LIBRARY can point the binding at)."""
    defines = list(defines)
    if not force and not defines and lib == LIB and up_to_date():
        return LIB
    os.makedirs(objdir, exist_ok=True)
    jobs = []
    for dt, red, fast in PARTS:
        name = "collectives_part_%d_%d_%d" % (dt, red, fast)
        jobs.append((name, "collectives_part.cu",
                     ["-DRCC_PART_DT=%d" % dt, "-DRCC_PART_RED=%d" % red,
                      "-DRCC_PART_FAST=%d" % fast]))
    for src in SOURCES:
        jobs.append((os.path.splitext(src)[0], src, []))
    procs = []
    objs = []
    for name, src, defs in jobs:
        obj = os.path.join(objdir, name + ".o")
        objs.append(obj)
        cmd = [NVCC, *ARCH, *COMMON, *defines, *defs, "-c", os.path.join(CSRC, src), "-o", obj]
        if src.endswith(".cpp"):
            cmd = [NVCC, *COMMON, "-x", "c++", "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd))
        procs.append((name, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    binding = None
    if lib == LIB:
        binding = os.path.join(objdir, "_lm.%d.so" % os.getpid())
        procs.append(("lm_binding", subprocess.Popen(
            binding_command(binding), stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            failed.append((src, out.decode(errors="replace")))
        elif verbose and out:
            print(out.decode(errors="replace"))
    if failed:
        msg = "\n".join(f"--- {s}\n{o}" for s, o in failed)
        raise RuntimeError("librcc build failed:\n" + msg)
    tmp = lib + ".tmp%d" % os.getpid()
    link = [NVCC, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs,
            "-Xlinker", "--version-script=" + os.path.join(CSRC, "exports.map")]
    if verbose:
        print(" ".join(link))
    subprocess.run(link, check=True)
    os.replace(tmp, lib)
    if binding:
        os.replace(binding, BINDING)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
