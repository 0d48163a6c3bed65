"""Build libdetfold.so in-tree with nvcc for sm_103a.

Each ``csrc/*.cu`` translation unit compiles in parallel to an object under
``_build/``; the objects link into ``libdetfold.so`` beside this file. No
fast-math: binary32 adds keep round-to-nearest-even and subnormals
(``-ftz=false -prec-div=true -prec-sqrt=true``), and ``-fmad=false`` rules out
any multiply-add contraction.

The measurement probes (``csrc/probes/*.cu``, the latency floors that graphs
of small folds are compared against) link into a library of their own,
``libdetfold_probes.so``, which the fold library's binding never loads. The
decode-step attention operators (``csrc/attn/*.cu``) link into
``libdetfold_attn.so``, those of a step with drafted tokens (``csrc/tree/*.cu``)
into ``libdetfold_tree.so``, and the module that marshals torch tensors for both
(``csrc/binding/attn_binding.cpp``) into ``_attn_binding.so``, with the host
compiler against the installed torch's headers.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libdetfold.so")
PROBES_CSRC = os.path.join(CSRC, "probes")
PROBES_LIB = os.path.join(PKG, "libdetfold_probes.so")
ATTN_CSRC = os.path.join(CSRC, "attn")
ATTN_LIB = os.path.join(PKG, "libdetfold_attn.so")
TREE_CSRC = os.path.join(CSRC, "tree")
TREE_LIB = os.path.join(PKG, "libdetfold_tree.so")
BINDING_SRC = os.path.join(CSRC, "binding", "attn_binding.cpp")
BINDING_LIB = os.path.join(PKG, "_attn_binding.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "-ftz=false",
              "-prec-div=true", "-prec-sqrt=true", "-fmad=false", "-Xptxas", "-warn-spills"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libdetfold")
    return path


def _inputs() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + [os.path.join(INCLUDE, "detfold.h"), os.path.abspath(__file__)])


def _probe_inputs() -> list[str]:
    return sorted(glob.glob(os.path.join(PROBES_CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + [os.path.join(INCLUDE, "detfold.h"), os.path.join(INCLUDE, "detfold_probes.h"),
                     os.path.abspath(__file__)])


def _attn_inputs() -> list[str]:
    return sorted(glob.glob(os.path.join(ATTN_CSRC, "*.cu")) + glob.glob(os.path.join(ATTN_CSRC, "*.cuh"))
                  + [os.path.join(INCLUDE, "detfold.h"), os.path.join(INCLUDE, "detfold_attn.h"),
                     os.path.abspath(__file__)])


def _tree_inputs() -> list[str]:
    return sorted(glob.glob(os.path.join(TREE_CSRC, "*.cu")) + glob.glob(os.path.join(TREE_CSRC, "*.cuh"))
                  + glob.glob(os.path.join(ATTN_CSRC, "*.cuh"))
                  + [os.path.join(INCLUDE, h) for h in ("detfold.h", "detfold_attn.h", "detfold_tree.h")]
                  + [os.path.abspath(__file__)])


def _binding_inputs() -> list[str]:
    return [BINDING_SRC, *sorted(glob.glob(os.path.join(CSRC, "binding", "*.h"))),
            *[os.path.join(INCLUDE, h) for h in ("detfold.h", "detfold_attn.h", "detfold_tree.h")],
            os.path.abspath(__file__)]


def stale(lib: str = LIB, inputs=None) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(p) > t for p in (inputs if inputs is not None else _inputs()))


def build(force: bool = False, defines: dict | None = None, lib: str = LIB,
          build_dir: str = BUILD_DIR, verbose: bool = False) -> str:
    """Compile and link libdetfold.so (and, for the default library path, the
    probes, attention and drafted-token libraries and the latter two's Python
    binding); returns the fold library's path.

    ``defines`` adds -D macros (launch-shape knobs of csrc/detfold_launch.cuh).
    The C libraries do not depend on torch: a binding that cannot be built is a
    RuntimeWarning, and importing ``attention`` then fails.
    """
    default = lib == LIB
    attn_dir = os.path.join(build_dir, "attn")
    stamp = os.path.join(attn_dir, "binding.for")
    dflags = [f"-D{k}={v}" for k, v in (defines or {}).items()]
    with ThreadPoolExecutor(max_workers=1) as ex:
        binding = None
        if default and (force or _binding_stale(stamp)):
            binding = ex.submit(_compile_binding, attn_dir)  # beside the kernels
        if force or defines or stale(lib):
            _link(sorted(glob.glob(os.path.join(CSRC, "*.cu"))), lib, build_dir, dflags, verbose)
        if default and (force or stale(PROBES_LIB, _probe_inputs())):
            _link(sorted(glob.glob(os.path.join(PROBES_CSRC, "*.cu"))), PROBES_LIB,
                  os.path.join(build_dir, "probes"), [], verbose)
        if default and (force or stale(ATTN_LIB, _attn_inputs())):
            _link(sorted(glob.glob(os.path.join(ATTN_CSRC, "*.cu"))), ATTN_LIB,
                  attn_dir, [], verbose)
        if default and (force or stale(TREE_LIB, _tree_inputs())):
            _link(sorted(glob.glob(os.path.join(TREE_CSRC, "*.cu"))), TREE_LIB,
                  os.path.join(build_dir, "tree"), [], verbose)
        if binding is not None:
            try:
                _link_binding(binding.result())
                with open(stamp, "w") as f:
                    f.write(_binding_target())
            except (RuntimeError, OSError) as e:
                if os.path.exists(BINDING_LIB):
                    os.remove(BINDING_LIB)  # of older sources: not to be loaded
                warnings.warn(f"the attention operators' Python binding was not built: {e}", RuntimeWarning,
                              stacklevel=2)
    return lib


def _binding_target() -> str:
    """The torch and the Python that the binding is compiled against."""
    root = _torch_root()
    with open(os.path.join(root, "version.py")) as f:
        return "\n".join([sys.version, str(sysconfig.get_config_var("SOABI")), root, f.read()])


def _binding_stale(stamp: str) -> bool:
    if stale(BINDING_LIB, _binding_inputs()) or not os.path.exists(stamp):
        return True
    try:
        with open(stamp) as f:
            return f.read() != _binding_target()
    except (RuntimeError, OSError):
        return True


def _torch_root() -> str:
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("torch not found: the attention operators' marshalling module is built against it")
    return list(spec.submodule_search_locations)[0]


def _run(cmd: list[str], what: str) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _compile_binding(build_dir: str) -> str:
    os.makedirs(build_dir, exist_ok=True)
    root, obj = _torch_root(), os.path.join(build_dir, "attn_binding.o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    dirs = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(root, "include"),
            os.path.join(root, "include", "torch", "csrc", "api", "include"), cuda]
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", *[f"-I{d}" for d in dirs], "-c", BINDING_SRC,
          "-o", obj], "g++ on attn_binding.cpp")
    return obj


def _link_binding(obj: str) -> None:
    libs, tmp = os.path.join(_torch_root(), "lib"), BINDING_LIB + f".tmp{os.getpid()}"
    _run(["g++", "-shared", "-o", tmp, obj, f"-L{PKG}", "-l:libdetfold_attn.so", "-l:libdetfold_tree.so", "-Wl,-rpath,$ORIGIN", f"-L{libs}",
          "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"], "link of _attn_binding.so")
    os.replace(tmp, BINDING_LIB)


def _link(sources: list[str], lib: str, build_dir: str, dflags: list[str], verbose: bool) -> str:
    os.makedirs(build_dir, exist_ok=True)
    cc = nvcc()

    def compile_one(src: str) -> str:
        obj = os.path.join(build_dir, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, *dflags, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
        if verbose:
            cmd += ["-Xptxas", "-v"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            print(r.stdout + r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=max(1, min(len(sources), os.cpu_count() or 1))) as ex:
        objs = list(ex.map(compile_one, sources))
    tmp = lib + f".tmp{os.getpid()}"
    r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force=True))
