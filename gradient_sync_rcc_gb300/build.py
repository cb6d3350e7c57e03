"""Build librcc.so in-tree: the CUDA kernels and the C-ABI host layer; and
_lm.so, the torch binding of the language-model operators.

nvcc, one -gencode for sm_103a, the translation units compiled in parallel,
static CUDA runtime, only the rcc_* symbols exported.  No fast-math: means use
IEEE division and bf16 outputs round to nearest even.

librcc.so needs nothing but nvcc.  Where torch is missing the binding is left
out; where it does not compile that is said, and librcc.so is built all the same.
"""
import importlib.metadata
import importlib.util
import os
import subprocess
import sys
import sysconfig

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
SOURCES = ["gradsync.cu", "embedding.cu", "rmsnorm.cu", "add_rmsnorm.cu",
           "rotary.cu", "adamw.cu", "linear_ce.cu", "rcc_host.cpp",
           "rcc_rank.cpp", "rcc_gradsync_host.cpp", "rcc_lm_host.cpp", "rcc_adamw_host.cpp"]
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


def _newer_than_inputs(path: str) -> bool:
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def _torch_dir():
    spec = importlib.util.find_spec("torch")
    return list(spec.submodule_search_locations)[0] if spec else None


def _binding_for() -> str:
    """What _lm.so is good for: this Python, and the torch that it finds."""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = "?"
    return "%s, torch %s in %s\n" % (sysconfig.get_config_var("SOABI"), version, _torch_dir())


def _binding_up_to_date() -> bool:
    """True also where there is no torch to build it for."""
    if not _torch_dir():
        return True
    stamp = os.path.join(OBJDIR, "_lm.for")
    if not _newer_than_inputs(BINDING) or not os.path.exists(stamp):
        return False
    with open(stamp) as f:
        return f.read() == _binding_for()


def up_to_date() -> bool:
    return _newer_than_inputs(LIB) and _binding_up_to_date()


def binding_command(out: str):
    """g++ on lm_binding.cpp with Python's and torch's headers and libraries."""
    torch_dir = _torch_dir()
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    lib = os.path.join(torch_dir, "lib")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-D_GLIBCXX_USE_CXX11_ABI=1",
            "-I", INCLUDE, "-I", sysconfig.get_paths()["include"],
            "-isystem", os.path.join(torch_dir, "include"),
            "-isystem", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
            "-isystem", cuda, os.path.join(CSRC, "lm_binding.cpp"), "-o", out,
            "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cuda", "-ltorch_cpu", "-ltorch_python",
            "-Wl,-rpath," + lib]


def _start_binding(out: str, verbose: bool):
    cmd = binding_command(out)
    if verbose:
        print(" ".join(cmd))
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)


def _finish_binding(proc, out: str) -> None:
    text, _ = proc.communicate()
    stamp = os.path.join(OBJDIR, "_lm.for")
    if os.path.exists(stamp):
        os.remove(stamp)
    if proc.returncode != 0:
        if os.path.exists(BINDING):
            os.remove(BINDING)
        print("note: _lm.so, the language-model operators' binding, did not build:\n"
              + text.decode(errors="replace"), file=sys.stderr)
        return
    os.replace(out, BINDING)
    with open(stamp, "w") as f:
        f.write(_binding_for())


def build(force: bool = False, verbose: bool = False, defines=(), lib: str = LIB,
          objdir: str = OBJDIR) -> str:
    """Compile librcc.so, and _lm.so where there is a torch.  `defines` (e.g.
    ["-DRCC_WAVES=8"]) rebuild the kernels with other tuning macros into `lib` /
    `objdir` (a comparison build that RCC_LIBRARY can point the binding at)."""
    defines = list(defines)
    if not force and not defines and lib == LIB and up_to_date():
        return LIB
    os.makedirs(objdir, exist_ok=True)
    binding = None
    if lib == LIB and _torch_dir() and (force or not _binding_up_to_date()):
        out = os.path.join(objdir, "_lm.%d.so" % os.getpid())
        binding = (_start_binding(out, verbose), out)
    try:
        if force or defines or lib != LIB or not _newer_than_inputs(LIB):
            _build_lib(verbose, defines, lib, objdir)
    finally:
        if binding:
            _finish_binding(*binding)
    return lib


def _build_lib(verbose: bool, defines, lib: str, objdir: str) -> None:
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


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
