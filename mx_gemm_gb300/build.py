"""Build step for the CUDA library: compiles csrc/*.cu for sm_103a with nvcc
(one process per translation unit, in parallel) and links ``_build/libfg.so``
next to this file.  The CUDA runtime is linked statically; the driver's
tensor-map encoder is looked up at run time, so the library needs no
libcuda at link time.  csrc/fg_torch.cpp, the binding that allocates outputs
through torch, is compiled beside them with g++ into ``_build/fg_torch.so``,
which finds libfg.so next to itself and torch's libraries in the process.
The library does not need it: where it cannot be built (no g++, no headers of
torch or Python) a warning says why, and the operators that live in it raise
when they are first called.
"""
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "_build")
LIB = os.path.join(OUT, "libfg.so")
BINDING = os.path.join(OUT, "fg_torch.so")
MADE_FOR = os.path.join(OUT, "fg_torch.made_for")  # the torch and Python that the binding was compiled against
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xcompiler", "-fvisibility=hidden"]


def nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _header():
    return os.path.join(os.path.dirname(HERE), "include", "fg.h")


def _newer(target, deps):
    return os.path.exists(target) and all(os.path.getmtime(d) <= os.path.getmtime(target) for d in deps)


def library_up_to_date():
    return _newer(LIB, _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [_header()])


def running():
    """The torch and Python of this process, as the binding's build records them."""
    import torch
    return "torch %s, Python %d.%d\n" % (torch.__version__, sys.version_info[0], sys.version_info[1])


def made_for():
    """What the binding was compiled against (None: not recorded)."""
    try:
        with open(MADE_FOR, encoding="utf-8") as f:
            return f.read()
    except OSError:
        return None


def binding_up_to_date():
    return _newer(BINDING, [os.path.join(CSRC, "fg_torch.cpp"), _header()]) and made_for() == running()


def up_to_date():
    return library_up_to_date() and binding_up_to_date()


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("%s failed:\n%s%s" % (what, r.stdout, r.stderr))


def _compile_binding(obj):
    """csrc/fg_torch.cpp against the installed torch's headers."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    paths = cpp_extension.include_paths() + [sysconfig.get_paths()["include"], os.path.join(os.path.dirname(
        os.path.dirname(nvcc())), "include")]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wno-deprecated-declarations",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI]
    _run(cmd + ["-isystem" + p for p in paths] + ["-c", os.path.join(CSRC, "fg_torch.cpp"), "-o", obj],
         "g++ for fg_torch.cpp")


def _link_binding(obj):
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + ".tmp.%d" % os.getpid()
    _run(["g++", "-shared", "-o", tmp, obj, "-L" + OUT, "-l:libfg.so", "-Wl,-rpath,$ORIGIN", "-L" + libs, "-ltorch_python",
          "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-lc10", "-lc10_cuda"], "link of fg_torch.so")
    os.replace(tmp, BINDING)
    with open(MADE_FOR, "w", encoding="utf-8") as f:
        f.write(running())


def _attempt(step, *args):
    """What went wrong in a step of the binding's build, or None."""
    try:
        step(*args)
    except Exception as e:  # a missing compiler, header or module: the library is built all the same
        return e
    return None


def build(force=False, verbose=False):
    library, binding = force or not library_up_to_date(), force or not binding_up_to_date()
    if not (library or binding):
        return LIB
    os.makedirs(OUT, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(OUT, os.path.basename(src) + ".o")
        cmd = [cc] + ARCH + FLAGS + ["-c", src, "-o", obj]
        if verbose:
            cmd += ["-Xptxas", "-v"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s%s" % (src, r.stdout, r.stderr))
        return obj, r.stderr

    srcs = _sources()
    binding_obj = os.path.join(OUT, "fg_torch.cpp.o")
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 4))) as ex:
        other = ex.submit(_attempt, _compile_binding, binding_obj) if binding else None
        results = list(ex.map(compile_one, srcs)) if library else []
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    if library:
        tmp = LIB + ".tmp.%d" % os.getpid()
        _run([cc] + ARCH + ["-shared", "-o", tmp] + [o for o, _ in results] + ["-lcudart_static", "-ldl", "-lrt", "-lpthread"],
             "link")
        os.replace(tmp, LIB)
    if binding:
        wrong = other.result() or _attempt(_link_binding, binding_obj)
        if wrong is not None:
            if os.path.exists(BINDING):
                os.remove(BINDING)  # of other sources
            warnings.warn("fg_torch.so, the binding of the operators around the GEMM, was not built: %s" % wrong)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
