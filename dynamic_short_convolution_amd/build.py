"""Builds libdynconv.so (HIP kernels + C ABI) for gfx950 with hipcc, in the package dir.

Usage: python -m dynamic_short_convolution_amd.build   (or build() from Python).
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import re
import shutil
import subprocess
import sys

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG_DIR, "csrc")
BUILD_DIR = os.path.join(PKG_DIR, "_build")
LIB_PATH = os.path.join(PKG_DIR, "libdynconv.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

SOURCES = [
    "dynconv_abi.hip",
    "dynconv_stream.hip",
    "dynconv_stream_f32.hip",
    "dynconv_stream_bf16.hip",
    "dynconv_stream_f16.hip",
    "dynconv_lowrank.hip",
    "dynconv_lowrank_f32.hip",
    "dynconv_lowrank_bf16.hip",
    "dynconv_lowrank_f16.hip",
    "dynconv_lowrank_fast.hip",
    "dynconv_decode.hip",
    "dynconv_gemm.hip",
    "dynconv_delta_abi.hip",
    "dynconv_delta.hip",
    "dynconv_delta_f32.hip",
    "dynconv_delta_bf16.hip",
    "dynconv_delta_f16.hip",
    "dynconv_norm.hip",
    "dynconv_scan_abi.hip",
    "dynconv_scan.hip",
    "dynconv_scan_f32.hip",
    "dynconv_scan_bf16.hip",
    "dynconv_scan_f16.hip",
    "dynconv_pack.hip",
    "dynconv_groupnorm.hip",
    "dynconv_groupnorm_f32.hip",
    "dynconv_groupnorm_bf16.hip",
    "dynconv_groupnorm_f16.hip",
]

# -packed-fp32-ops: no v_pk_{add,mul,fma}_f32 are generated from ordinary float code.
COMPILE_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    "-Wno-unused-function",
    "-Xclang",
    "-target-feature",
    "-Xclang",
    "-packed-fp32-ops",
    # matrix-core results in ordinary VGPRs: no v_accvgpr_read copies before they are used
    "-mllvm",
    "-amdgpu-mfma-vgpr-form",
]

# Sources with kernels of more than 256 registers are built without the last two flags: past 256,
# the compiler's pass that moves VGPR-form matrix-core operands to accumulation registers has
# crashed here. Within 256 registers, as in bfloat16, the flags change these kernels' times
# by less than 2 %.
PLAIN_MFMA_SOURCES = ("dynconv_delta_f32.hip", "dynconv_delta_bf16.hip", "dynconv_delta_f16.hip")


def compile_flags(src: str) -> list[str]:
    return COMPILE_FLAGS[:-2] if src in PLAIN_MFMA_SOURCES else COMPILE_FLAGS


_VECTOR = re.compile(r"(?:v_(?!readlane|writelane|readfirstlane)|scratch_|ds_|global_|buffer_|flat_)")
_COPY = re.compile(r"(?:v_mov_b|v_accvgpr_|scratch_)")
_EXEC = re.compile(r"\bexec\b")


def misplaced_vector_code(listing: str) -> list[str]:
    """Vector instructions of an assembly listing that run under a divergent branch's execution mask
    though they belong behind it.

    The block where the lanes of a divergent branch meet begins by restoring the mask. When the
    compiler splits a register's live range at that block it can put the copy or spill before the
    restoring, if a scalar copy already stands there: lanes (or whole waves) that did not take the
    branch then keep what the register or its scratch place held before. Seen with this compiler: a
    spilled sum of the delta rule's chunk gradients (float32, 128-wide heads, two value heads per key
    head), lost in six of eight waves, with no diagnostic."""
    found = []
    joins = set(re.findall(r"s_cbranch_execz (\.LBB\d+_\d+)\b", listing))
    for m in re.finditer(r"^\s+(?:s_or_b64 exec, exec,|s_or_saveexec_b64).*$", listing, re.M):
        start = max(listing.rfind("\n.LBB", 0, m.start()), listing.rfind("\n; %bb.", 0, m.start()))
        if start < 0:
            continue
        head, *body = listing[start + 1:m.start()].split("\n")
        lines = [t for t in (x.split(";")[0].strip() for x in body) if t and not t.startswith(".")]
        if any(t.startswith(("s_cbranch", "s_branch")) or (_EXEC.search(t) and not re.match(r"s_and(n2)?_b64 vcc, exec", t))
               for t in lines):
            continue  # the mask was written since
        vector = [t for t in lines if _VECTOR.match(t)]
        # a block that no branch leads to may be the branch's own body: only copies and spills tell
        if vector and (head.split(":")[0] in joins or (head.startswith(";") and all(_COPY.match(t) for t in vector))):
            line = listing.count("\n", 0, m.start()) + 1
            found.append(f"line {line}, {head.split(':')[0]}: {'; '.join(vector[:3])}")
    return found


def _compile(src: str) -> str:
    stem = os.path.splitext(src)[0]
    obj, work = os.path.join(BUILD_DIR, stem + ".o"), os.path.join(BUILD_DIR, stem + ".tmp")
    shutil.rmtree(work, ignore_errors=True)
    os.makedirs(work)
    try:
        tmp = os.path.join(work, stem + ".o")
        cmd = [HIPCC, *compile_flags(src), "-save-temps=obj", "-c", os.path.join(CSRC, src), "-o", tmp]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"hipcc failed for {src}:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
        (name,) = glob.glob(os.path.join(work, "*amdgcn*.s"))
        with open(name) as f:
            found = misplaced_vector_code(f.read())
        if found:
            raise RuntimeError(f"{src}: vector code before the execution mask is restored:\n" + "\n".join(found[:10]))
        os.replace(tmp, obj)
    finally:
        shutil.rmtree(work, ignore_errors=True)
    return obj


def build(verbose: bool = False) -> str:
    """Compiles every source and links libdynconv.so; returns the library path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    jobs = min(len(SOURCES), os.cpu_count() or 1)
    with concurrent.futures.ThreadPoolExecutor(max_workers=jobs) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB_PATH + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB_PATH)
    if verbose:
        print(f"built {LIB_PATH}")
    return LIB_PATH


# Host-side code only, with AddressSanitizer and UndefinedBehaviorSanitizer on the host
# compile. Each object embeds the same device bundle of an empty source file instead of its
# kernels, so the library registers no kernels: only argument checking, planning and size
# queries can run (a launch would fail). Loaded with the clang ASan runtime
# preloaded (SANITIZER_RUNTIME) by a process that selects it through DYNCONV_LIBRARY.
ASAN_DIR = os.path.join(PKG_DIR, "_build_asan")
ASAN_LIB_PATH = os.path.join(ASAN_DIR, "libdynconv_hostsan.so")
SANITIZE_FLAGS = [
    "-Xarch_host", "-fsanitize=address",
    "-Xarch_host", "-fsanitize=undefined",
    "-Xarch_host", "-fno-sanitize-recover=undefined",
    "-Xarch_host", "-fno-omit-frame-pointer",
]


def sanitizer_runtime() -> str:
    """Path of the clang ASan runtime matching hipcc's compiler."""
    res = subprocess.run([os.path.join(os.path.dirname(HIPCC), "..", "lib", "llvm", "bin", "clang"),
                          "-print-file-name=libclang_rt.asan-x86_64.so"], capture_output=True, text=True)
    path = res.stdout.strip()
    if res.returncode != 0 or not os.path.isabs(path) or not os.path.exists(path):
        raise RuntimeError(f"no ASan runtime found ({res.stdout} {res.stderr})")
    return path


def build_host_sanitized() -> str:
    """Builds the host-only sanitized library; returns its path."""
    os.makedirs(ASAN_DIR, exist_ok=True)
    empty_src = os.path.join(ASAN_DIR, "empty.hip")
    empty_bin = os.path.join(ASAN_DIR, "empty.fatbin")
    with open(empty_src, "w") as f:
        f.write("// no kernels\n")
    cmd = [HIPCC, "-x", "hip", "--offload-arch=gfx950", "--cuda-device-only", "--no-offload-new-driver", "-c",
           empty_src, "-o", empty_bin]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"empty device bundle failed:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")

    def one(src: str) -> str:
        obj = os.path.join(ASAN_DIR, os.path.splitext(src)[0] + ".o")
        cmd = [HIPCC, "-x", "hip", "--cuda-host-only", "--no-offload-new-driver", "-Xclang", "-fcuda-include-gpubinary",
               "-Xclang", empty_bin, "-O1", "-g", "-std=c++17", "-fPIC", *SANITIZE_FLAGS, "-c",
               os.path.join(CSRC, src), "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"hipcc failed for {src}:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=min(len(SOURCES), os.cpu_count() or 1)) as ex:
        objs = list(ex.map(one, SOURCES))
    cmd = [HIPCC, "-shared", "-fPIC", *SANITIZE_FLAGS, "-shared-libasan", *objs, "-o", ASAN_LIB_PATH]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    return ASAN_LIB_PATH


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
