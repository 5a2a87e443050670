"""Build the HIP library libfg.so for gfx950 and its torch extension fg_torch.so
(in-tree, next to this file)."""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB_DIR = os.path.join(HERE, "_lib")
LIB = os.path.join(LIB_DIR, "libfg.so")
SOURCES = [os.path.join(CSRC, n) for n in ("fg.hip", "fg_ops.hip", "fg_cache.hip", "fg_latent.hip")]
HEADERS = [os.path.join(CSRC, n) for n in ("fg_sync.hpp", "fg_gemm.hpp", "fg_plan.hpp", "fg_kernels.hpp", "fg_combine.hpp",
                                               "fg_entry.hpp", "fg_ops.hpp", "fg_norm.hpp", "fg_route.hpp", "fg_w4.hpp", "fg_moe.hpp",
                                               "fg_split.hpp", "fg_pages.hpp", "fg_paged.hpp", "fg_latent.hpp", "fg_prompt.hpp")] + [
    os.path.join(ROOT, "include", n) for n in ("fg.h", "fg_attention.h")]
EXTENSION = os.path.join(LIB_DIR, "fg_torch.so")
EXTENSION_SOURCE = os.path.join(CSRC, "fg_torch.cpp")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    # packed fp32 instructions are kept out of every code object on this part
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
    "-Wno-unused-command-line-argument",
]


def _extension_command(out: str) -> list[str]:
    """The torch extension holds no device code: the host compiler, torch's headers, libfg.so beside it."""
    from torch.utils import cpp_extension as T
    rocm = os.path.dirname(os.path.dirname(HIPCC))
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-DUSE_ROCM", "-D__HIP_PLATFORM_AMD__",
            *[f"-I{d}" for d in (os.path.join(ROOT, "include"), *T.include_paths(), os.path.join(rocm, "include"),
                                 sysconfig.get_paths()["include"])],
            EXTENSION_SOURCE, f"-L{LIB_DIR}", *[f"-L{d}" for d in T.library_paths()], "-l:libfg.so", "-ltorch_python", "-ltorch",
            "-ltorch_cpu", "-ltorch_hip", "-lc10", "-lc10_hip", f"-L{rocm}/lib", "-lamdhip64", "-Wl,-rpath,$ORIGIN", "-o", out]


def _run(what: str, cmd: list[str], verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"the compiler failed building {what}")


def build(verbose: bool = False) -> str:
    """Compile every HIP source into libfg.so, the sources side by side, then fg_torch.so; always recompiles."""
    os.makedirs(LIB_DIR, exist_ok=True)
    flags = [f for f in FLAGS if f != "-shared"]
    with tempfile.TemporaryDirectory(dir=LIB_DIR) as objects:
        made = [os.path.join(objects, os.path.basename(s) + ".o") for s in SOURCES]
        with ThreadPoolExecutor(len(SOURCES)) as pool:
            for done in [pool.submit(_run, os.path.basename(s), [HIPCC, *flags, "-c", s, "-o", o], verbose) for s, o in zip(SOURCES, made)]:
                done.result()
        _run("libfg.so", [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *made, "-o", LIB + ".tmp"], verbose)
    os.replace(LIB + ".tmp", LIB)
    _run("fg_torch.so", _extension_command(EXTENSION + ".tmp"), verbose)
    os.replace(EXTENSION + ".tmp", EXTENSION)
    return LIB


def device_asm(out_path: str) -> str:
    """Write the gfx950 assembly of the library (for inspection of the kernels)."""
    cmd = [HIPCC, *[f for f in FLAGS if f not in ("-shared", "-fPIC")], "--cuda-device-only", "-S",
           *SOURCES, "-o", out_path]
    subprocess.run(cmd, check=True)
    return out_path


if __name__ == "__main__":
    print(build(verbose=True))
