"""In-tree build of libfsa.so (nvcc, sm_103a only) and of the serving calls' extension module.

The fused attention kernel is compiled once per (QK format, PV format) pair in
its own translation unit so that the pairs build in parallel."""
from __future__ import annotations

import glob
import os
import subprocess
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libfsa.so")
TORCH_SOURCE = os.path.join(CSRC, "fsa_torch.cpp")
TORCH_MODULE = os.path.join(PKG, "_fsa_torch.so")     # the serving calls' marshalling (a Python extension)

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I" + INCLUDE, "-I" + CSRC]

# (QK format, PV format): 0 E4M3, 1 E2M3, 2 E2M1, 3 E2M1 by the EFQ rule, 4 E3M2, 5 BF16, 6 NVFP4 (Q/K)
ATTN_PAIRS = [(qk, pv) for qk in (0, 1, 2, 4, 6) for pv in range(5)] + [(5, 5)]


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.sep not in c or os.path.exists(c)):
            return c
    return "nvcc"


def _units():
    units = [("fsa_api", os.path.join(CSRC, "fsa_api.cu"), []),
             ("fsa_quant", os.path.join(CSRC, "fsa_quant.cu"), []),
             ("fsa_peak", os.path.join(CSRC, "fsa_peak.cu"), [])]
    units += [(n, os.path.join(CSRC, n + ".cu"), []) for n in ("fsa_cache_api", "fsa_cache_attn", "fsa_cache", "fsa_rope", "fsa_append_rope", "fsa_cache_chunk")]
    units.append(("fsa_cache_attn_window", os.path.join(CSRC, "fsa_cache_attn.cu"), ["-DFSA_CACHE_WINDOW=1"]))
    for qk, pv in ATTN_PAIRS:
        units.append((f"fsa_attn_{qk}{pv}", os.path.join(CSRC, "fsa_attn.cu"),
                      [f"-DFSA_INST_QK={qk}", f"-DFSA_INST_PV={pv}"]))
    return units


def _torch_flags():
    """(compile, link) flags of csrc/fsa_torch.cpp against the installed torch."""
    import sysconfig
    import torch
    base = os.path.dirname(torch.__file__)
    nvcc = _nvcc()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc))) if os.path.sep in nvcc else "/usr/local/cuda"
    inc = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"], INCLUDE]
    lib = os.path.join(base, "lib")
    return (["-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
             *["-isystem" + i for i in inc]],
            ["-L" + lib, "-L" + PKG, "-l:libfsa.so", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
             "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib])


def _fresh(output: str, inputs) -> bool:
    return os.path.exists(output) and os.path.getmtime(output) >= max(os.path.getmtime(f) for f in [*inputs, __file__])


def _library_inputs():
    return [f for f in glob.glob(os.path.join(CSRC, "*")) if f != TORCH_SOURCE] + glob.glob(os.path.join(INCLUDE, "*.h"))


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stderr}")
    return r


def _replace(cmd, out, what):
    """Run a link command, its output put in place whole."""
    tmp = out + f".{os.getpid()}.tmp"
    _run([*cmd[:-1], "-o", tmp, *cmd[-1]], what)
    os.replace(tmp, out)


def build_library(force: bool = False, jobs: int | None = None, verbose: bool = False) -> str:
    """Compile every CUDA source for sm_103a and link libfsa.so in the package dir (nvcc only)."""
    if not force and _fresh(LIB, _library_inputs()):
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    nvcc = _nvcc()

    def compile_unit(u):
        name, src, defs = u
        obj = os.path.join(OBJ, name + ".o")
        r = _run([nvcc, *(["-Xptxas=-v"] if verbose else []), *ARCH, *FLAGS, *defs, "-c", src, "-o", obj],
                 f"nvcc failed for {name}")
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    with ThreadPoolExecutor(jobs or min(16, os.cpu_count() or 4)) as ex:
        objs = list(ex.map(compile_unit, _units()))
    _replace([nvcc, *ARCH, "-shared", "-cudart", "shared", "-Xlinker", "-soname=libfsa.so", objs], LIB, "link failed")
    return LIB


def _torch_stamp() -> str:
    """What the compiled module depends on besides its sources: the interpreter and torch."""
    import platform
    import torch
    return f"{platform.machine()} {platform.python_version()} {torch.__version__} {os.path.dirname(torch.__file__)}"


def _compile_torch(force: bool) -> str | None:
    """The object file of csrc/fsa_torch.cpp; None if the module is up to date."""
    stamp = os.path.join(OBJ, "fsa_torch.for")
    if not force and _fresh(TORCH_MODULE, [TORCH_SOURCE, os.path.join(INCLUDE, "fsa.h")]) and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read() == _torch_stamp():
                return None
    os.makedirs(OBJ, exist_ok=True)
    obj = os.path.join(OBJ, "fsa_torch.o")
    _run(["g++", *_torch_flags()[0], "-c", TORCH_SOURCE, "-o", obj], "g++ failed for fsa_torch")
    return obj


def _link_torch(obj: str | None) -> str:
    if obj is not None:
        _replace(["g++", "-shared", [obj, *_torch_flags()[1]]], TORCH_MODULE, "link of _fsa_torch failed")
        with open(os.path.join(OBJ, "fsa_torch.for"), "w") as f:
            f.write(_torch_stamp())
    return TORCH_MODULE


def build_torch_module(force: bool = False) -> str:
    """The extension module of the serving calls, against the installed torch (g++, the headers
    of torch and Python); libfsa.so first, if that is missing or stale."""
    build_library()
    return _link_torch(_compile_torch(force))


def build(force: bool = False, jobs: int | None = None, verbose: bool = False) -> str:
    """Both, at once.  libfsa.so does not need the module: where that cannot be built, a warning
    says why, and the serving calls raise."""
    with ThreadPoolExecutor(1) as ex:
        module = ex.submit(_compile_torch, force)
        build_library(force, jobs, verbose)
        try:
            _link_torch(module.result())
        except Exception as e:  # noqa: BLE001
            warnings.warn(f"libfsa.so is built, the serving calls' module is not: {e}", RuntimeWarning, stacklevel=2)
    return LIB
