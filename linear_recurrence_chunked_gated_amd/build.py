"""Build libsf_gdn.so (HIP, gfx950) and the module _calls (the native Python
calls of the layer's operators) in the package directory.

    python -m linear_recurrence_chunked_gated_amd.build

Each translation unit is compiled to an object under _build/ in parallel,
then linked.  Packed-fp32 instruction forms are disabled for device code.  The
library and the module are stamped with a digest of the header they share, by
which the module is matched to the library when it is loaded.
"""
import hashlib
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libsf_gdn.so")
SOURCES = ["gdn_fwd.hip", "gdn_bwd.hip", "gdn_conv.hip", "sf_gdn_api.cpp"]
CALLS = os.path.join(HERE, "_calls" + sysconfig.get_config_var("EXT_SUFFIX"))
ARCH = "gfx950"

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CFLAGS = ["-x", "hip", "--offload-arch=" + ARCH, "-O3", "-std=c++17", "-fPIC",
          "-ffp-contract=fast", "-Wall", "-Wno-unused-result",
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          "-I", os.path.join(HERE, "..", "include")]


def _stamp():
    with open(os.path.join(HERE, "..", "include", "sf_gdn.h"), "rb") as f:
        return '-DSF_GDN_INTERFACE="%s"' % hashlib.sha256(f.read()).hexdigest()[:16]


def _compile(src):
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [HIPCC] + CFLAGS + [_stamp(), "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    msgs = "\n".join(l for l in (r.stdout + r.stderr).splitlines()
                     if "packed-fp32-ops" not in l)
    if r.returncode != 0:
        raise RuntimeError("compile failed: %s\n%s" % (" ".join(cmd), msgs))
    return obj, msgs


def _build_calls():
    """The CPython module _calls: host code on torch's headers, by g++."""
    import torch
    from torch.utils import cpp_extension
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = CALLS + ".tmp%d" % os.getpid()
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           "-fvisibility=hidden", "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI,
           _stamp(), "-I", sysconfig.get_paths()["include"]]
    for d in cpp_extension.include_paths():
        cmd += ["-isystem", d]
    cmd += [os.path.join(CSRC, "sf_gdn_calls.cpp"), "-o", tmp, "-L", lib, "-lc10", "-ltorch_cpu",
            "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("compile failed: %s\n%s%s" % (" ".join(cmd), r.stdout, r.stderr))
    os.replace(tmp, CALLS)
    return r.stdout + r.stderr


def _link(objects):
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [HIPCC, "--offload-arch=" + ARCH, "-shared", "-fPIC", "-o", tmp] + objects
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed: %s\n%s%s" % (" ".join(cmd), r.stdout, r.stderr))
    os.replace(tmp, LIB)


def build(verbose=False):
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        calls = ex.submit(_build_calls)
        results = list(ex.map(_compile, SOURCES))
        # the library needs hipcc alone: it is there whatever becomes of the module
        _link([o for o, _ in results])
        results.append((CALLS, calls.result()))
    if verbose:
        for _, m in results:
            if m.strip():
                print(m)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
