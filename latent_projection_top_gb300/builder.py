"""Build the route library (``_build/libroute.so``) for sm_103a with nvcc.

The translation units compile in parallel; ptxas resource usage (registers,
spills, shared memory) is written to ``_build/ptxas.log``.

``build(debug=True)`` builds the same sources with ``-DROUTE_DEBUG`` into
``_build/debug/libroute_debug.so``: every global index that the route step's
kernels compute is checked, and a failed check is reported through the device
status word (``route_device_status`` returns ROUTE_ERR_DEVICE_BOUNDS) instead
of faulting.  The layer operators' kernels are the same in both.  The binding loads it when the environment sets ROUTE_DEBUG_LIB=1.

With either goes the Python module of the layer operators' calls
(``csrc/layer_call.cpp``, host code only).  It reads tensors through torch's
and Python's binary interfaces, so its file's name says which of each it was
built for (``call_module()``).  The library is complete without it: where it
cannot be built (no torch, or no headers of torch's or Python's) ``build()``
warns, and the calls go through ctypes.
"""

from __future__ import annotations

import importlib.util
import os
import re
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libroute.so")
DEBUG_BUILD = os.path.join(BUILD, "debug")
DEBUG_LIB = os.path.join(DEBUG_BUILD, "libroute_debug.so")
INCLUDE = os.path.join(ROOT, "include")
CALL_SOURCE = os.path.join(CSRC, "layer_call.cpp")

SOURCES = ["decode_kernel.cu", "prefill_kernel.cu", "topk_kernel.cu", "stage_kernel.cu",
           "route_api.cu", "layer_gemm.cu", "layer_small.cu", "layer_elem.cu",
           "layer_norm.cu", "layer_api.cu", "dispatch_kernel.cu", "experts_kernel.cu",
           "experts_small.cu", "dropout_kernel.cu", "experts_api.cu"]
HEADERS = ["common.cuh", "sm103_ptx.cuh", "topk16.cuh", "twofloat.cuh", "api_util.h", "layer.cuh",
           "layer_math.cuh", "layer_ptx.cuh", "layer_plan.h", "experts.cuh"]

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                "-Xptxas", "-v", "-I", INCLUDE, "-I", CSRC]


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES + HEADERS]
    files += [os.path.join(INCLUDE, h) for h in ("route.h", "route_layer.h", "route_experts.h")]
    files.append(os.path.abspath(__file__))
    return files


def _stale(lib: str, inputs: list | None = None) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(f) > t for f in inputs or _inputs())


def _compile(src: str, build_dir: str, extra: list) -> tuple[str, str]:
    obj = os.path.join(build_dir, os.path.splitext(src)[0] + ".o")
    cmd = [NVCC] + FLAGS + extra + ["-c", os.path.join(CSRC, src), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{res.stdout}\n{res.stderr}")
    return obj, res.stderr


def _link(objs: list, lib: str) -> None:
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [NVCC] + ARCH + ["-shared", "-o", tmp] + objs + ["-cudart", "static"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, lib)


def _torch_dir() -> str | None:
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec else None


def call_module() -> str | None:
    """The calls' module for this Python and the torch that it would import
    (read from torch's version file: importing it takes seconds); None where
    there is no torch."""
    if _torch_dir() is None:
        return None
    text = open(os.path.join(_torch_dir(), "version.py")).read()
    version = re.search(r"""^__version__ = ['"]([^'"]+)""", text, re.M).group(1)
    return os.path.join(BUILD, f"_layer_call.torch-{version}.{sysconfig.get_config_var('SOABI')}.so")


def _build_call_module(force: bool) -> None:
    """Build the calls' module if it is stale; warn if that is not possible."""
    inputs = [CALL_SOURCE, *(os.path.join(INCLUDE, h) for h in ("route.h", "route_layer.h", "route_experts.h")),
              os.path.abspath(__file__)]
    module = None
    try:
        module = call_module()
        if module is None:
            raise RuntimeError("torch is not installed")
        if force or _stale(module, inputs):
            _compile_call_module()
    except Exception as e:  # the library and the binding work without it
        # one older than the entry points would call them by their old arguments
        if module is not None and os.path.exists(module) and _stale(module, inputs):
            os.remove(module)
        warnings.warn(f"the layer operators' calls will go through ctypes (2 to 5 us more each): {e}")


def _compile_call_module() -> None:
    import torch
    abi, torch = int(torch._C._GLIBCXX_USE_CXX11_ABI), _torch_dir()
    module = call_module()
    tmp = module + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", CALL_SOURCE,
           "-o", tmp, "-I", INCLUDE, "-I", sysconfig.get_paths()["include"],
           "-I", os.path.join(torch, "include"), "-L", os.path.join(torch, "lib"),
           f"-D_GLIBCXX_USE_CXX11_ABI={abi}", "-ltorch_python", "-ltorch_cpu", "-lc10"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for layer_call.cpp:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, module)


def build(force: bool = False, verbose: bool = False, debug: bool = False,
          both: bool = False) -> str:
    """Build the release library (or, with debug=True, the checked one; with
    both=True, both at once, their translation units in parallel).  Returns
    the path of the release library (of the debug one with debug=True)."""
    targets = [(LIB, BUILD, [])] if not debug or both else []
    if debug or both:
        targets.append((DEBUG_LIB, DEBUG_BUILD, ["-DROUTE_DEBUG"]))
    todo = [(lib, d, x) for lib, d, x in targets if force or _stale(lib)]
    os.makedirs(BUILD, exist_ok=True)
    if not todo:
        _build_call_module(force)
    if todo:
        for _, d, _ in todo:
            os.makedirs(d, exist_ok=True)
        jobs = [(src, d, x) for _, d, x in todo for src in SOURCES]
        with ThreadPoolExecutor(max_workers=len(jobs) + 1) as pool:
            module = pool.submit(_build_call_module, force)
            results = list(pool.map(lambda j: _compile(*j), jobs))
            module.result()
        for k, (lib, d, _) in enumerate(todo):
            part = results[k * len(SOURCES):(k + 1) * len(SOURCES)]
            with open(os.path.join(d, "ptxas.log"), "w") as f:
                for (o, log), src in zip(part, SOURCES):
                    f.write(f"==== {src}\n{log}\n")
            _link([o for o, _ in part], lib)
        if verbose:
            print(open(os.path.join(todo[0][1], "ptxas.log")).read())
    return DEBUG_LIB if debug and not both else LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, debug="--debug" in sys.argv,
                both="--both" in sys.argv))
