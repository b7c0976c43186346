"""Build libgbfuse.so in-tree with nvcc for sm_103a, and the compiled part of the
Python binding with the host compiler.

Each CUDA translation unit under csrc/ is compiled to an object in parallel,
then linked into fusion_add_rmsnorm_gb300/libgbfuse.so with the CUDA runtime
linked statically (the library loads without a GPU driver; kernels need one).
Objects go to fusion_add_rmsnorm_gb300/_build/ (git-ignored).  A source whose
object is newer than the source and every header is not recompiled.  The library
needs neither torch nor Python's headers: it is linked before the binding is
looked at, and `--no-binding` leaves the binding out.
binding/decode_binding.cpp (the wrappers of the decode-step and block-scaled calls) becomes
fusion_add_rmsnorm_gb300/decode_binding<tag of this Python>.so against the
installed torch, whose version it carries; another Python or torch builds it anew.
"""
import concurrent.futures as cf
import glob
import importlib.util
import os
import runpy
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libgbfuse.so")
BINDING_SRC = os.path.join(HERE, "binding", "decode_binding.cpp")
TAG = sysconfig.get_config_var("EXT_SUFFIX")              # .cpython-<version>-<platform>.so
BINDING = os.path.join(HERE, "decode_binding" + TAG)
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC",
         "-Xcompiler", "-fvisibility=hidden", "-I", os.path.join(ROOT, "include")]


def nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or put it on PATH)")


def _headers():
    return glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h")) + glob.glob(os.path.join(HERE, "binding", "*.h"))


def _stale(src, obj, hdr_mtime):
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return t < os.path.getmtime(src) or t < hdr_mtime


def build(verbose=False, extra_flags=(), binding=True):
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdr_mtime = max([os.path.getmtime(h) for h in _headers()] + [0])
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]

    def compile_one(pair):
        src, obj = pair
        if not _stale(src, obj, hdr_mtime) and not extra_flags:
            return None
        cmd = [cc, *ARCH, *FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        return r.stderr if verbose else None

    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        binding_obj = ex.submit(compile_binding, hdr_mtime) if binding else None
        for out in ex.map(compile_one, zip(srcs, objs)):
            if out:
                sys.stderr.write(out)
    if not os.path.exists(LIB) or any(os.path.getmtime(o) > os.path.getmtime(LIB) for o in objs):
        tmp = LIB + ".tmp"
        cmd = [cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    if binding:
        link_binding(binding_obj.result())
    return LIB


def _torch_dir():
    # found, not imported: the paths are all that is needed
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("the binding needs torch (--no-binding builds the library alone)")
    return os.path.dirname(spec.origin)


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _torch_version():
    return runpy.run_path(os.path.join(_torch_dir(), "version.py"))["__version__"]


def compile_binding(hdr_mtime):
    version = _torch_version()
    obj = os.path.join(BUILD, "decode_binding" + os.path.splitext(TAG)[0] + ".o")
    built_for = obj[:-2] + ".torch"                        # torch version of the object
    if os.path.exists(built_for):
        with open(built_for) as f:
            same = f.read() == version
    else:
        same = False
    if not same or _stale(BINDING_SRC, obj, hdr_mtime):
        cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
        inc = [os.path.join(ROOT, "include"), sysconfig.get_paths()["include"], os.path.join(_torch_dir(), "include"), cuda]
        _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", f'-DGBF_BUILT_FOR_TORCH="{version}"',
              *[f"-I{p}" for p in inc], "-c", BINDING_SRC, "-o", obj], "g++ on decode_binding.cpp")
        with open(built_for, "w") as f:
            f.write(version)
    return obj


def link_binding(obj):
    if os.path.exists(BINDING) and os.path.getmtime(BINDING) >= max(os.path.getmtime(obj), os.path.getmtime(LIB)):
        return
    lib = os.path.join(_torch_dir(), "lib")
    tmp = BINDING + ".tmp"
    _run(["g++", "-shared", "-o", tmp, obj, f"-L{lib}", "-ltorch_python", "-lc10", "-lc10_cuda", "-ltorch_cpu", f"-L{HERE}",
          "-l:libgbfuse.so", f"-Wl,-rpath,{lib}", "-Wl,-rpath,$ORIGIN"], "link of decode_binding.so")
    os.replace(tmp, BINDING)
    untagged = os.path.join(os.path.dirname(BINDING), "decode_binding.so")   # as older builds left it, for any Python to import
    if os.path.exists(untagged):
        os.remove(untagged)


if __name__ == "__main__":
    v = "-v" in sys.argv
    extra = ("-Xptxas", "-v") if v else ()
    print(build(verbose=v, extra_flags=extra, binding="--no-binding" not in sys.argv))
