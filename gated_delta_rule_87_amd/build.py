"""Build libkda.so (HIP kernels + C ABI) for gfx950, in-tree.

    python -m gated_delta_rule_87_amd.build

Compiles every source under csrc/ with hipcc for --offload-arch=gfx950 into
gated_delta_rule_87_amd/libkda.so. hipcc cross-compiles without a GPU.
"""
import concurrent.futures
import os
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libkda.so")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
HIPCC = os.path.join(ROCM, "bin", "hipcc")

SOURCES = ["kda_api.cpp", "kda_sched.hip", "kda_intra.hip", "kda_chain.hip", "kda_scan.hip", "kda_recurrent.hip",
           "kda_noalloc.hip", "kda_ops_api.cpp", "kda_glr.hip", "kda_layernorm.hip", "kda_cache.hip",
           "kda_layer_api.cpp", "kda_conv.hip", "kda_ssm.hip", "kda_rmsnorm.hip", "kda_beam.hip"]

FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
    # MFMA results stay in VGPRs: no v_accvgpr_read before the VALU uses them
    "-mllvm", "-amdgpu-mfma-vgpr-form",
]


# hipcc's host pass warns that it does not know the packed-fp32 feature: harmless
NOISE = "is not a recognized feature for this target"


def _run(cmd, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    err = "\n".join(ln for ln in r.stderr.splitlines() if NOISE not in ln)
    if r.returncode != 0:
        sys.stderr.write(err + "\n")
        raise RuntimeError("hipcc failed building libkda.so")
    if verbose and err.strip():
        sys.stderr.write(err + "\n")


def build(verbose: bool = False, extra_flags=(), out: str = LIB) -> str:
    """One hipcc per source, several at once, then the link."""
    compile_flags = [f for f in FLAGS if f != "-shared"]
    tmp = out + ".tmp"
    with tempfile.TemporaryDirectory() as objects:
        jobs = [(os.path.join(CSRC, s), os.path.join(objects, s + ".o")) for s in SOURCES]
        with concurrent.futures.ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
            done = [pool.submit(_run, [HIPCC, *compile_flags, *extra_flags, "-c", "-o", o, s], verbose)
                    for s, o in sorted(jobs, key=lambda j: -os.path.getsize(j[0]))]
            for d in done:
                d.result()
        _run([HIPCC, *FLAGS, *extra_flags, "-o", tmp, *[o for _, o in jobs]], verbose)
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    print(build(verbose=True))
