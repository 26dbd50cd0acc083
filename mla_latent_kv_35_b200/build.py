"""Build libmla_b200.so in-tree with nvcc for sm_100a, and the Python calls
(_pycall.so) with the host compiler.

    python -m mla_latent_kv_35_b200.build
"""

import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libmla_b200.so")
SOURCES = [os.path.join(HERE, "csrc", "api.cu")]
HEADER = os.path.join(ROOT, "include", "mla.h")
CALLS = os.path.join(HERE, "_pycall.so")
CALLS_SOURCE = os.path.join(HERE, "csrc", "pycall.cpp")
# What CALLS was built for: it fits one Python and one torch.
CALLS_STAMP = os.path.join(HERE, "_build", "pycall.txt")
DEPS = SOURCES + [os.path.join(HERE, "csrc", f) for f in os.listdir(os.path.join(HERE, "csrc"))
                  if f != "pycall.cpp"] + [HEADER]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "--expt-relaxed-constexpr",
    "-Xptxas", "-v",
]


def nvcc():
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.sep not in c or os.path.exists(c)):
            return c
    return "nvcc"


def up_to_date(target: str = LIB, deps=DEPS) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(d) <= t for d in deps if os.path.exists(d))


def _calls_stamp() -> str:
    import torch
    return f"{sys.version}\ntorch {torch.__version__}\n"


def calls_up_to_date() -> bool:
    if not up_to_date(CALLS, [CALLS_SOURCE, HEADER]) or not os.path.exists(CALLS_STAMP):
        return False
    with open(CALLS_STAMP) as f:
        return f.read() == _calls_stamp()


def _compile(cmd, target: str, verbose: bool):
    tmp = target + ".tmp"
    r = subprocess.run(cmd + ["-o", tmp], capture_output=True, text=True)
    if verbose or r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed building {os.path.basename(target)}")
    os.replace(tmp, target)


def build(force: bool = False, verbose: bool = False) -> str:
    include = ["-I", os.path.join(ROOT, "include")]
    if force or not calls_up_to_date():
        import torch
        t = os.path.dirname(torch.__file__)
        _compile([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC"] + include
                 + ["-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(t, "include"),
                    "-isystem", os.path.join(t, "include", "torch", "csrc", "api", "include"),
                    f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
                    CALLS_SOURCE, "-L", os.path.join(t, "lib"), "-ltorch_python", "-ltorch_cpu",
                    "-lc10"], CALLS, verbose)
        os.makedirs(os.path.dirname(CALLS_STAMP), exist_ok=True)
        with open(CALLS_STAMP, "w") as f:
            f.write(_calls_stamp())
    if force or not up_to_date():
        _compile([nvcc()] + NVCC_FLAGS + include + SOURCES, LIB, verbose)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
