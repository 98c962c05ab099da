"""Build libspecverify.so in-tree with hipcc for gfx950."""
import os
import shutil
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libspecverify.so")
SOURCES = ("specverify.hip", "beam.hip", "pages.hip", "tree.hip")

HIPCC_FLAGS = [
    "-O3", "-std=c++17", "--offload-arch=gfx950", "-fPIC",
    "-Wall", "-Wno-unused-result",
    # keep the compiler from emitting packed-fp32 VALU instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-fvisibility=hidden", "-DSPECVERIFY_BUILDING",
]


def hipcc_path() -> str:
    return shutil.which("hipcc") or "/opt/rocm/bin/hipcc"


# Host-side AddressSanitizer and UndefinedBehaviorSanitizer for the argument
# checks, plan and workspace layout (the device code is built as usual): each
# -fsanitize applies to the host compilation only.
HOST_SANITIZE_FLAGS = [
    "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
    "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer", "-g",
]


def build(verbose: bool = False, out: str = LIB, defines=(), host_sanitize: bool = False) -> str:
    """Compile the HIP sources into rejection_sampling_verify_07_amd/libspecverify.so
    (or `out`, with extra -D defines, for tuning builds; host_sanitize: a host
    ASan/UBSan build for the CPU tests of the argument checks)."""
    tmp = out + ".tmp"
    extra = HOST_SANITIZE_FLAGS if host_sanitize else []
    flags = [*HIPCC_FLAGS, *extra, *[f"-D{d}" for d in defines], "-I", os.path.join(ROOT, "include"), "-I", CSRC]

    def run(cmd):
        if verbose:
            print(" ".join(cmd))
        subprocess.run(cmd, check=True)

    # one object per source, compiled side by side
    with tempfile.TemporaryDirectory() as objdir:
        objs = [os.path.join(objdir, os.path.splitext(src)[0] + ".o") for src in SOURCES]
        with ThreadPoolExecutor(len(SOURCES)) as pool:
            list(pool.map(lambda so: run([hipcc_path(), *flags, "-c", os.path.join(CSRC, so[0]), "-o", so[1]]),
                          zip(SOURCES, objs)))
        run([hipcc_path(), *HIPCC_FLAGS, "-shared", *extra, *objs, "-o", tmp])
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    print(build(verbose=True))
