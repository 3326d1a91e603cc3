"""Build and load libdsa_indexer.so (the sm_103a CUDA library) in-tree.

The library is compiled with nvcc for ``sm_103a`` only and loaded with
ctypes; the tensor-level calls over it are a CPython module, compiled with
g++ when one of them is first made.  There is no fallback: if the library cannot be built or loaded the
calls raise.
"""
from __future__ import annotations

import contextlib
import ctypes
import fcntl
import os
import subprocess
import threading
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(BUILD, "libdsa_indexer.so")
CXX = os.environ.get("CXX", "g++")
NVCC = os.environ.get("NVCC", "nvcc")

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]

# Every symbol include/dsa_indexer.h declares.
EXPORTS = ("dsa_indexer_logits_decode", "dsa_indexer_logits_prefill",
           "dsa_indexer_logits_prefill_varlen", "dsa_indexer_topk_decode",
           "dsa_indexer_topk_decode_form",
           "dsa_indexer_topk_decode_static", "dsa_kcache_store",
           "dsa_qk_norm_rope", "dsa_latent_store", "dsa_latent_load",
           "dsa_latent_attention", "dsa_latent_attention_workspace",
           "dsa_request_slots", "dsa_kv_store", "dsa_block_bounds", "dsa_block_select",
           "dsa_paged_attention", "dsa_paged_attention_workspace",
           "dsa_status_string", "dsa_indexer_abi_version")

_lib = None
_lock = threading.Lock()


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    files = _sources()
    files += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return files


def _older(path, files) -> bool:
    return not os.path.exists(path) or any(os.path.getmtime(f) > os.path.getmtime(path) for f in files)


def calls_path() -> str:
    """The CPython module of the tensor-level calls (torch_calls.cpp).  It reads tensors by the
    layout of the torch that it was compiled with, so its name carries that torch's version and
    commit, and Python's version and machine: another torch has a file of its own."""
    import sysconfig
    import torch
    commit = (torch.version.git_version or "")[:10]
    return os.path.join(BUILD, f"_dsa_torch-{torch.__version__}-{commit}{sysconfig.get_config_var('EXT_SUFFIX')}")


def is_stale() -> bool:
    return _older(LIB_PATH, _deps())


def calls_stale() -> bool:
    return _older(calls_path(), [os.path.join(CSRC, "torch_calls.cpp"), os.path.join(INCLUDE, "dsa_indexer.h")])


@contextlib.contextmanager
def _one_builder():
    """Processes that find the build stale at the same time take turns: they share its files."""
    os.makedirs(BUILD, exist_ok=True)
    with open(os.path.join(BUILD, "lock"), "w") as f:
        fcntl.flock(f, fcntl.LOCK_EX)
        yield


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every .cu under csrc/ for sm_103a and link the shared library."""
    if force or is_stale():
        with _one_builder():
            if force or is_stale():
                _build(verbose)
    return LIB_PATH


def _build(verbose: bool = False) -> None:
    objs = []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [NVCC, *ARCH_FLAGS, *NVCC_FLAGS, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    srcs = _sources()
    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
        results = list(ex.map(compile_one, srcs))
    for obj, log in results:
        objs.append(obj)
        if verbose and log:
            print(log)
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [NVCC, *ARCH_FLAGS, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)


def build_calls(force: bool = False) -> str:
    """Compile the CPython module of the tensor-level calls (g++, torch's and Python's headers) and
    link it to the shared library, which is built first."""
    if force or calls_stale():
        build()
        with _one_builder():
            if force or calls_stale():
                _link_calls(_compile_calls())
    return calls_path()


def build_all(force: bool = False, verbose: bool = False) -> None:
    """Both, compiled side by side."""
    if not (force or is_stale() or calls_stale()):
        return
    with _one_builder(), ThreadPoolExecutor(max_workers=1) as ex:
        calls = ex.submit(_compile_calls) if force or calls_stale() else None
        if force or is_stale():
            _build(verbose)
        if calls:
            _link_calls(calls.result())


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stdout}\n{r.stderr}")


def _compile_calls() -> str:
    import sysconfig
    import torch
    base = os.path.join(os.path.dirname(torch.__file__), "include")
    include = [INCLUDE, base, os.path.join(base, "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"],
               os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")]
    obj = os.path.join(BUILD, "torch_calls.o")
    _run([CXX, "-O2", "-std=c++17", "-fPIC",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          *[f"-I{d}" for d in include], "-c", os.path.join(CSRC, "torch_calls.cpp"), "-o", obj],
         "compiling torch_calls.cpp")
    return obj


def _link_calls(obj):
    import torch
    tmp = calls_path() + f".tmp{os.getpid()}"
    _run([CXX, "-shared", obj, "-o", tmp, "-L" + BUILD, "-l:libdsa_indexer.so", "-Wl,-rpath,$ORIGIN",
          "-L" + os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python", "-ltorch_cpu",
          "-lc10", "-lc10_cuda"], "linking the tensor-level calls")
    os.replace(tmp, calls_path())


_calls = None


def load_calls():
    """The CPython module of the tensor-level calls (building it first if it is missing or stale)."""
    global _calls
    if _calls is None:
        load()
        build_calls()
        import importlib.machinery
        import importlib.util
        import torch  # noqa: F401  (its libraries are the module's)
        loader = importlib.machinery.ExtensionFileLoader("_dsa_torch", calls_path())
        spec = importlib.util.spec_from_loader("_dsa_torch", loader)
        _calls = importlib.util.module_from_spec(spec)
        loader.exec_module(_calls)
    return _calls


def load() -> ctypes.CDLL:
    """Load the library (building it first if it is missing or stale)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if is_stale():
            build()
        lib = ctypes.CDLL(LIB_PATH)
        vp, ll, ci = ctypes.c_void_p, ctypes.c_longlong, ctypes.c_int
        sig = [vp, vp, vp, vp, ll, ci, ci, vp, ll, vp, ci, ci, ci, ci, ci, vp, ll, vp, vp]
        for name in ("dsa_indexer_logits_decode", "dsa_indexer_logits_prefill"):
            fn = getattr(lib, name)
            fn.restype = ci
            fn.argtypes = sig
        lib.dsa_indexer_topk_decode.restype = ci
        lib.dsa_indexer_topk_decode.argtypes = [vp, vp, vp, vp, ll, ci, ci, vp, ll, vp, ci, ci,
                                                ci, ci, ci, ci, vp, vp, ll, vp, ll, vp, vp]
        lib.dsa_indexer_topk_decode_form.restype = ci
        lib.dsa_indexer_topk_decode_form.argtypes = [vp, vp, vp, vp, ll, ci, ci, vp, ll, vp, ci,
                                                     ci, ci, ci, ci, ci, vp, vp, ll, vp, ll, vp,
                                                     ci, vp]
        lib.dsa_indexer_logits_prefill_varlen.restype = ci
        lib.dsa_indexer_logits_prefill_varlen.argtypes = [vp, vp, vp, vp, ll, ci, ci, vp, ll, vp,
                                                          ci, vp, ci, ci, ci, ci, vp, ll, vp, vp]
        lib.dsa_indexer_topk_decode_static.restype = ci
        lib.dsa_indexer_topk_decode_static.argtypes = [vp, vp, vp, vp, ll, ci, ci, vp, ll, vp, ci,
                                                       ci, ci, ci, ci, ci, vp, vp, ll, vp, vp]
        lib.dsa_kcache_store.restype = ci
        lib.dsa_kcache_store.argtypes = [vp, vp, ci, vp, ll, ci, ci, ci, ci, vp, vp]
        cf = ctypes.c_float
        lib.dsa_qk_norm_rope.restype = ci
        lib.dsa_qk_norm_rope.argtypes = [vp, ll, ll, ci, vp, ll, ll, ci, ci, ci, ci, ci, vp, vp, vp,
                                         vp, cf, vp, vp, ci, ci, ci, ci, vp, ll, ll, vp, ll, ll, vp,
                                         vp]
        lib.dsa_latent_store.restype = ci
        lib.dsa_latent_store.argtypes = [vp, ll, vp, ll, ci, ci, ci, vp, cf, vp, vp, ci, ci, vp, vp,
                                         ll, ci, ci, ci, vp, vp]
        lib.dsa_latent_load.restype = ci
        lib.dsa_latent_load.argtypes = [vp, ll, ci, ci, ci, vp, ll, ci, vp, vp, ci, ci, ci, ci, vp,
                                        ll, vp, vp]
        lib.dsa_latent_attention.restype = ci
        lib.dsa_latent_attention.argtypes = [vp, ll, ll, vp, ll, ll, ci, ci, ci, ci, cf, vp, ll, ci,
                                             ci, ci, vp, ll, ci, vp, vp, ll, ci, vp, ll, ll, vp, vp,
                                             ll, vp, vp]
        lib.dsa_latent_attention_workspace.restype = ll
        lib.dsa_latent_attention_workspace.argtypes = []
        lib.dsa_request_slots.restype = ci
        lib.dsa_request_slots.argtypes = [vp, vp, ci, vp, ci, vp, ll, ci, ci, ci, vp, vp, vp, vp, vp,
                                          vp, vp]
        lib.dsa_kv_store.restype = ci
        lib.dsa_kv_store.argtypes = [vp, ll, ll, vp, ll, ll, ci, ci, ci, ci, vp, vp, ll, ll, ll, vp, ll,
                                     ll, ll, vp, vp, ci, ci, ci, vp, vp]
        lib.dsa_block_bounds.restype = ci
        lib.dsa_block_bounds.argtypes = [vp, ll, ll, ll, vp, ci, ci, ci, ci, ci, vp, ll, ci, vp, vp, ci,
                                         ci, vp, vp, vp, vp]
        lib.dsa_block_select.restype = ci
        lib.dsa_block_select.argtypes = [vp, ll, ll, ci, ci, ci, ci, ci, vp, vp, ci, vp, ll, ci, ci, vp,
                                         ci, ci, ci, vp, vp, vp]
        lib.dsa_paged_attention.restype = ci
        lib.dsa_paged_attention.argtypes = [vp, ll, ll, ci, ci, ci, ci, ci, cf, vp, ll, ll, ll, vp, ll,
                                            ll, ll, vp, vp, ci, ci, ci, vp, ll, ci, vp, vp, ll, ll, ci,
                                            vp, ll, ll, vp, vp, ll, vp, vp]
        lib.dsa_paged_attention_workspace.restype = ll
        lib.dsa_paged_attention_workspace.argtypes = [ci, ci, ci]
        lib.dsa_status_string.restype = ctypes.c_char_p
        lib.dsa_status_string.argtypes = [ci]
        lib.dsa_indexer_abi_version.restype = ci
        lib.dsa_indexer_abi_version.argtypes = []
        _lib = lib
        return lib
