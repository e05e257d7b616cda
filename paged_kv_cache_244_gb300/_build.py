"""Compile the CUDA library in-tree: csrc/*.cu -> libpa_gb300.so, for sm_103a only, and the
native half of the Python binding, csrc_py/pa_torch.cpp -> _pa_torch.so, with the host compiler
against this interpreter's PyTorch.

Each translation unit compiles in parallel with nvcc (-gencode arch=compute_103a,
code=sm_103a, -O3, -lineinfo); the objects link into one shared library with the CUDA
runtime linked statically, so loading it needs only the driver.  Rebuilds only when a
source or header is newer than the library, or the native half was compiled against another
interpreter or PyTorch.  Where a host compiler, Python's headers or
PyTorch's are missing, the library is built all the same, with a warning, and the calls that
need the native half raise.
"""

from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
INCLUDE = ROOT / "include"
BUILD_DIR = PKG / "_build"
LIBRARY = PKG / "libpa_gb300.so"
NATIVE_SOURCE = PKG / "csrc_py" / "pa_torch.cpp"
NATIVE = PKG / "_pa_torch.so"
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and Path(cand).exists():
            return cand
    raise RuntimeError("nvcc not found: the CUDA library cannot be built")


def _sources():
    return sorted(CSRC.glob("*.cu"))


def _deps():
    return _sources() + sorted(CSRC.glob("*.cuh")) + sorted(CSRC.glob("*.h")) + sorted(INCLUDE.glob("*.h"))


def up_to_date() -> bool:
    if not LIBRARY.exists():
        return False
    t = LIBRARY.stat().st_mtime
    return all(p.stat().st_mtime <= t for p in _deps())


def cxx() -> str:
    return os.environ.get("CXX") or "g++"


def torch_dir() -> Path | None:
    """The installed PyTorch, found without importing it."""
    spec = importlib.util.find_spec("torch")
    return Path(spec.origin).resolve().parent if spec and spec.origin else None


def native_key() -> str:
    """The interpreter and the PyTorch that the native half is compiled against."""
    version = torch_dir() / "version.py" if torch_dir() else None
    text = version.read_text() if version and version.exists() else ""
    return f"{sysconfig.get_config_var('SOABI')}\n{version}\n{text}"


def native_up_to_date() -> bool:
    key = BUILD_DIR / "pa_torch.key"
    if not NATIVE.exists() or not key.exists() or key.read_text() != native_key():
        return False
    t = NATIVE.stat().st_mtime
    return all(p.stat().st_mtime <= t for p in [NATIVE_SOURCE, *INCLUDE.glob("*.h")])


def native_missing() -> str | None:
    """What the native half of the binding needs and is not there (None: nothing)."""
    if not shutil.which(cxx()):
        return f"no host compiler ({cxx()})"
    torch = torch_dir()
    if torch is None or not (torch / "include" / "torch" / "csrc" / "autograd" / "python_variable.h").exists():
        return "no PyTorch with its headers"
    if not (Path(sysconfig.get_paths()["include"]) / "Python.h").exists():
        return "no Python headers"
    return None


def _compile_native() -> Path:
    """The binding's object file (its link needs the library)."""
    inc = torch_dir() / "include"
    cuda = Path(nvcc()).resolve().parents[1] / "include"
    obj = BUILD_DIR / "pa_torch.o"
    cmd = [cxx(), "-c", str(NATIVE_SOURCE), "-o", str(obj), "-O2", "-std=c++17", "-fPIC",
           f"-I{INCLUDE}", f"-I{inc}", f"-I{inc}/torch/csrc/api/include", f"-I{cuda}",
           f"-I{sysconfig.get_paths()['include']}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"the compiler failed on {NATIVE_SOURCE.name}:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_native(obj: Path) -> None:
    libs = torch_dir() / "lib"
    tmp = NATIVE.with_name(NATIVE.name + f".tmp{os.getpid()}")
    cmd = [cxx(), "-shared", "-o", str(tmp), str(obj), f"-L{libs}", f"-L{PKG}",
           "-l:libpa_gb300.so", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda",
           f"-Wl,-rpath,{libs}", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"linking {NATIVE.name} failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, NATIVE)
    (BUILD_DIR / "pa_torch.key").write_text(native_key())


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> Path:
    ready = not force and up_to_date()
    if ready and native_up_to_date():
        return LIBRARY
    BUILD_DIR.mkdir(exist_ok=True)
    missing = native_missing()
    if missing:
        warnings.warn(f"{missing}: {NATIVE.name} is not built, the serving calls of the binding will raise",
                      RuntimeWarning, stacklevel=2)
    if ready:
        if not missing:
            _link_native(_compile_native())
        return LIBRARY
    cc = nvcc()
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                    f"-I{INCLUDE}", f"-I{CSRC}", "--expt-relaxed-constexpr"] + (extra_flags or [])

    def compile_one(src: Path) -> Path:
        obj = BUILD_DIR / (src.stem + ".o")
        cmd = [cc, "-c", str(src), "-o", str(obj)] + flags
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src.name}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=max(1, min(12, os.cpu_count() or 1))) as ex:
        native = None if missing else ex.submit(_compile_native)
        objs = list(ex.map(compile_one, _sources()))
    tmp = LIBRARY.with_name(LIBRARY.name + f".tmp{os.getpid()}")
    cmd = [cc, "-shared", "-o", str(tmp)] + ARCH + [str(o) for o in objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIBRARY)
    if native:
        _link_native(native.result())
    return LIBRARY


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
