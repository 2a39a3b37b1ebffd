"""Compile the HIP library in-tree for gfx950.

``python -m selective_state_space_41_amd.build`` (or ``build()``) runs hipcc on the library's
sources (``SOURCES``, side by side) and links ``libvmscan.so`` next to this file; it always
recompiles.
``python -m selective_state_space_41_amd.build --probe`` builds only the issue-rate
microbenchmark (``csrc/probe.hip`` -> ``vmscan_probe``), which is not part of the library.
"""
import os
import re
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libvmscan.so")
SOURCES = ("vmscan.hip", "linattn.hip", "norm.hip", "rope.hip", "act8.hip", "groupnorm.hip", "gated_scan.hip")  # in csrc/
PROBE = os.path.join(PKG, "vmscan_probe")

# Packed fp32 VALU forms are kept out of every gfx950 code object.
HIP_FLAGS = ["-O3", "-std=c++17", "--offload-arch=gfx950", "-fPIC",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]


def _hipcc():
    h = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(h):
        raise RuntimeError("hipcc not found: the ROCm toolchain is required to build vmscan")
    return h


def _run(cmd):
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    # hipcc's host pass does not know the packed-fp32 feature name; that warning is harmless
    out = "\n".join(l for l in r.stdout.splitlines() if "packed-fp32-ops" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"build failed ({r.returncode}): {' '.join(cmd)}\n{out}")
    return out


# The hot kernels' occupancy is part of their design: each launch shape assumes that many waves per
# SIMD fit the registers (the Vim scan three, so that a Vim-Ti call is one round; the backward walk
# two; the SS2D walk four, two eight-wave workgroups per CU; the state-only passes many).  A change
# that costs a kernel a wave shows up only as a slower call, so the build reads the compiler's
# per-kernel resource report and fails when a kernel falls below its floor or spills where it should
# not (only the float32 backward walk is allowed a few bytes of scratch).
OCCUPANCY_FLOORS = [  # (kernel name fragment, minimum waves per SIMD)
    ("scan_pair_kernel", 3),
    ("bwd_scan_kernel", 2),
    ("walk_pair_kernel", 4),
    ("chunk_state_kernel", 6),
    ("bwd_ckpt_kernel", 6),
    ("adj_state_kernel", 6),
    ("lane_scan_kernel", 2),
    ("linattn_segment_kernelItLi64ELi64E", 4),
    ("linattn_passes_kernelItLi64ELi64E", 4),
    ("linattn_step_kernel", 6),
    ("gated_scan_fwd_kernel", 4),
    ("gated_scan_bwd_kernel", 4),
    ("groupnorm_sums_kernelItLb1", 4),
    ("groupnorm_dx_kernelItLb1", 6),
]
# Linear attention: workgroups per CU that the cuts of a call are planned with (kWalks of csrc/linattn.hip), by kernel, type
# and padded key channels, for 32, 64 and 128 value channels of a workgroup; 0: no such kernel.
WALKS_PER_CU = {
    "fwd": {"t": {32: (4, 3, 2), 64: (4, 3, 2), 128: (2, 2, 0)}, "f": {32: (4, 2, 1), 64: (3, 2, 0), 128: (2, 1, 0)}},
    "grad": {"t": {32: (0, 2, 1), 64: (0, 2, 1), 128: (0, 1, 1)}, "f": {32: (0, 1, 1), 64: (0, 1, 1), 128: (0, 1, 1)}},
}
LDS_PER_CU = 160 * 1024


def walk_floors():
    """[(kernel name fragment, workgroups per CU, waves per SIMD that makes)] of WALKS_PER_CU."""
    out = []
    for kernel, types in WALKS_PER_CU.items():
        for t, keys in types.items():
            for dk, per_cu in keys.items():
                for dv, n in zip((32, 64, 128), per_cu):
                    waves = 4 if kernel == "fwd" else 4 if (t, dk, dv) == ("f", 128, 128) else 8  # of a workgroup
                    if n:
                        out.append((f"linattn_{kernel}_kernelI{t}Li{dk}ELi{dv}E", n, n * waves // 4))
    return out


# Bytes per lane.  linattn_grad: twelve registers of its key waves, spilled once a block; with 2 waves per SIMD and no
# scratch the call takes 476 us instead of 424 (32 x 3136 tokens, 8 heads).
SCRATCH_ALLOWED = [("bwd_scan_kernelIf", 64), ("linattn_grad_kernelItLi64ELi64E", 48),
                   # the other walks of the gradient whose state does not fit beside the block's results
                   ("linattn_grad_kernelItLi128ELi128E", 260), ("linattn_grad_kernelIfLi128ELi128E", 36),
                   ("linattn_grad_kernelIfLi128ELi64E", 104),
                   # rows over 8192 channels: 16 waves of 128 registers
                   ("rmsnorm_bwd_kernelIffLi64ELi16ELi4E", 228), ("rmsnorm_bwd_kernelItfLi64ELi16ELi4E", 208),
                   ("rmsnorm_bwd_kernelIttLi64ELi16ELi4E", 204),
                   # runs of 8 float32 tokens (of 4, without: 20001 x 195 tokens 68 us instead of 65, 16 x 3136 x 256 116
                   # instead of 113), and float32 channels that are no multiple of 4 kept in 8 bits
                   ("gated_scan_bwd_kernelIf", 28), ("gated_scan_fwd_kernelIfLi8ELi16ELNS_6LayoutE1ELb1E", 12),
                   ("groupnorm_slab_bwd_kernelItLb1ELi8ELb0E", 28)]
# Kernels whose scratch is checked beside those with a floor.
SCRATCH_CHECKED = ("linattn_", "rmsnorm_", "rope_kernel", "act8_", "groupnorm_", "gated_scan_")


def kernel_resources(report):
    """Per-kernel {VGPRs, AGPRs, ScratchSize, Occupancy, LDS} from -Rpass-analysis=kernel-resource-usage."""
    res, cur = {}, None
    for line in report.splitlines():
        m = re.search(r"remark: Function Name: (\S+)", line)
        if m:
            cur = m.group(1)
            res[cur] = {}
            continue
        m = re.search(r"remark:\s+(VGPRs|AGPRs|ScratchSize \[bytes/lane\]|Occupancy \[waves/SIMD\]|"
                      r"LDS Size \[bytes/block\]): (\d+)", line)
        if m and cur:
            res[cur][m.group(1).split()[0]] = int(m.group(2))
    return res


def check_resources(res):
    """Problems with the hot kernels' occupancy or scratch (empty when all is well)."""
    bad = []
    for name, r in res.items():
        for frag, floor in OCCUPANCY_FLOORS:
            if frag in name and r.get("Occupancy", 0) < floor:
                bad.append(f"{name}: {r.get('Occupancy')} waves per SIMD (VGPRs {r.get('VGPRs')}, AGPRs "
                           f"{r.get('AGPRs')}), needs {floor}")
        for frag, per_cu, floor in walk_floors():
            if frag not in name:
                continue
            if r.get("Occupancy", 0) < floor:
                bad.append(f"{name}: {r.get('Occupancy')} waves per SIMD, {per_cu} workgroups per CU need {floor}")
            if r.get("LDS", 0) * per_cu > LDS_PER_CU:
                bad.append(f"{name}: {r.get('LDS')} bytes of LDS, planned with {per_cu} workgroups per CU")
        allowed = next((b for frag, b in SCRATCH_ALLOWED if frag in name), 0)
        if any(frag in name for frag in SCRATCH_CHECKED + tuple(f for f, _ in OCCUPANCY_FLOORS)) and r.get("ScratchSize", 0) > allowed:
            bad.append(f"{name}: {r.get('ScratchSize')} bytes of scratch per lane, at most {allowed}")
    return bad


def build(verbose=False):
    """Compile libvmscan.so and check the hot kernels' occupancy."""
    hipcc = _hipcc()
    tmp = LIB + ".tmp"
    objs = [os.path.join(PKG, "csrc", src[:-len(".hip")] + ".o") for src in SOURCES]

    def compile_one(src, obj):
        return _run([hipcc, *HIP_FLAGS, "-Rpass-analysis=kernel-resource-usage", "-I", os.path.join(ROOT, "include"),
                     "-c", "-o", obj, os.path.join(PKG, "csrc", src)])

    with ThreadPoolExecutor(len(SOURCES)) as pool:
        out = "\n".join(pool.map(compile_one, SOURCES, objs))
    _run([hipcc, *HIP_FLAGS, "-shared", "-o", tmp, *objs])
    res = kernel_resources(out)
    if not any(frag in name for name in res for frag, _ in OCCUPANCY_FLOORS):
        raise RuntimeError("build: the compiler printed no kernel resource report")
    bad = check_resources(res)
    bad += [f"{frag}: planned with, and not built" for frag, _, _ in walk_floors() if not any(frag in n for n in res)]
    if bad:
        raise RuntimeError("build: kernels below their occupancy floor:\n  " + "\n  ".join(bad))
    os.replace(tmp, LIB)
    if verbose:
        print("\n".join(l for l in out.splitlines() if "kernel-resource-usage" not in l and l.strip()))
    return LIB


def build_probe(verbose=False):
    """Compile the issue-rate microbenchmark executable (measures the gfx950 VALU, exp2 and
    scan-token rates the kernel design relies on)."""
    out = _run([_hipcc(), *HIP_FLAGS, "-o", PROBE + ".tmp", os.path.join(PKG, "csrc", "probe.hip")])
    os.replace(PROBE + ".tmp", PROBE)
    if verbose and out.strip():
        print(out)
    return PROBE


if __name__ == "__main__":
    print(build_probe(verbose="-v" in sys.argv) if "--probe" in sys.argv else build(verbose="-v" in sys.argv))
