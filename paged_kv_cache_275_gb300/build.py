"""Build libpagedkv.so in-tree with nvcc for sm_103a (GB300), and the compiled Python binding of some of its calls.

    python -m paged_kv_cache_275_gb300.build [--force] [--ptxas-verbose]

Each CUDA translation unit is compiled in parallel to ``_build/*.o`` and the
objects are linked into ``paged_kv_cache_275_gb300/libpagedkv.so`` against the
shared CUDA runtime.  Rebuilds only when a source or header is newer than the
library.  The binding (csrc/binding.cpp, host code against torch's headers) is compiled beside them into
``_binding.so``.  No cmake, no torch extension machinery.
"""
from __future__ import annotations

import argparse
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
INCLUDE = ROOT / "include"
BUILD = PKG / "_build"
LIB = PKG / "libpagedkv.so"
BINDING = PKG / "_binding.so"
SOURCES = ["capi.cu", "kv_append.cu", "rope_append.cu", "paged_decode.cu", "window_decode.cu", "prefix_decode.cu",
           "static_workspace.cu", "copy_blocks.cu", "block_manager.cpp", "paged_prefill.cu", "window_prefill.cu",
           "shared_prefix.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def cuda_home() -> Path:
    env = os.environ.get("CUDA_HOME") or os.environ.get("CUDA_PATH")
    if env:
        return Path(env)
    nvcc = shutil.which("nvcc")
    if nvcc:
        return Path(nvcc).resolve().parent.parent
    return Path("/usr/local/cuda")


def _nvcc() -> str:
    exe = cuda_home() / "bin" / "nvcc"
    return str(exe) if exe.exists() else "nvcc"


def _inputs() -> list[Path]:
    return ([CSRC / s for s in SOURCES] + [CSRC / "binding.cpp"] + list(CSRC.glob("*.h")) + list(CSRC.glob("*.cuh"))
            + list(INCLUDE.glob("*.h")) + [Path(__file__)])


STAMP = BUILD / "flags.txt"


def extra_flags() -> list[str]:
    """Extra nvcc flags from PKV_NVCC_FLAGS (launch-shape tuning, e.g. -DPKV_D128_WARPS=6)."""
    return os.environ.get("PKV_NVCC_FLAGS", "").split()


def _stamp() -> str:
    """What the binaries depend on besides the sources; the binding goes by the interpreter's ABI as well as by torch's."""
    return " ".join([*extra_flags(), "torch", importlib.metadata.version("torch"), "python",
                     str(sysconfig.get_config_var("SOABI"))])


def needs_build() -> bool:
    if not LIB.exists() or not BINDING.exists():
        return True
    if (STAMP.read_text() if STAMP.exists() else "") != _stamp():
        return True
    t = min(LIB.stat().st_mtime, BINDING.stat().st_mtime)
    return any(p.stat().st_mtime > t for p in _inputs())


def _compile_binding(obj: Path) -> subprocess.CompletedProcess:
    torch = Path(importlib.util.find_spec("torch").origin).parent
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-I", str(INCLUDE), "-I", str(torch / "include"),
           "-I", str(torch / "include" / "torch" / "csrc" / "api" / "include"), "-I", sysconfig.get_paths()["include"],
           "-I", str(cuda_home() / "include"), "-c", str(CSRC / "binding.cpp"), "-o", str(obj)]
    return subprocess.run(cmd, capture_output=True, text=True)


def _link_binding(obj: Path, out: Path) -> subprocess.CompletedProcess:
    torch_lib = Path(importlib.util.find_spec("torch").origin).parent / "lib"
    cmd = ["g++", "-shared", "-o", str(out), str(obj), "-L", str(PKG), "-l:libpagedkv.so", "-L", str(torch_lib),
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
           "-L", str(cuda_home() / "lib64"), "-lcudart", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{torch_lib}",
           f"-Wl,-rpath,{cuda_home() / 'lib64'}", f"-Wl,-rpath-link,{cuda_home() / 'lib64'}"]
    return subprocess.run(cmd, capture_output=True, text=True)


def compile_flags(ptxas_verbose: bool = False) -> list[str]:
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", str(INCLUDE), "-I", str(CSRC),
                    "--expt-relaxed-constexpr"] + extra_flags()
    if ptxas_verbose:
        flags += ["-Xptxas", "-v"]
    return flags


def build(force: bool = False, ptxas_verbose: bool = False, quiet: bool = False) -> Path:
    if not force and not ptxas_verbose and not needs_build():
        return LIB
    BUILD.mkdir(exist_ok=True)
    nvcc = _nvcc()
    flags = compile_flags(ptxas_verbose)

    def one(src: str):
        obj = BUILD / (Path(src).stem + ".o")
        cmd = [nvcc, *flags, "-c", str(CSRC / src), "-o", str(obj)]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, r

    binding_obj = BUILD / "binding.o"
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_compile_binding, binding_obj)
        results = list(ex.map(one, SOURCES))
    if binding.result().returncode != 0:
        sys.stderr.write(binding.result().stdout + binding.result().stderr)
        raise RuntimeError("g++ failed on binding.cpp")
    for src, _, r in results:
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError(f"nvcc failed on {src}")
        if (ptxas_verbose or r.stderr.strip()) and not quiet:
            sys.stderr.write(r.stderr)
    tmp = LIB.with_name(f"libpagedkv.so.tmp{os.getpid()}")
    link = [nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", str(tmp), *[str(o) for _, o, _ in results],
            "-Xlinker", f"-rpath,{cuda_home() / 'lib64'}"]
    r = subprocess.run(link, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("nvcc link failed")
    os.replace(tmp, LIB)
    tmp = BINDING.with_name(f"_binding.so.tmp{os.getpid()}")
    r = _link_binding(binding_obj, tmp)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("g++ link of the binding failed")
    os.replace(tmp, BINDING)
    STAMP.write_text(_stamp())
    return LIB


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--ptxas-verbose", action="store_true", help="print registers / spills / shared memory")
    args = ap.parse_args(argv)
    print(build(force=args.force, ptxas_verbose=args.ptxas_verbose))
    return 0


if __name__ == "__main__":
    raise SystemExit(main())
