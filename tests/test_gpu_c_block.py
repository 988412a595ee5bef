"""The update of many tensors, the block boundary and the policy loss driven from plain C through include/zero_shard.h
(tests/capi/block_check.c): against the host update bit for bit, and against the host's double evaluation; refusals."""

import os
import shutil
import subprocess

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIBDIR = os.path.join(ROOT, "zero_partition_plan_amd")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_blocks_from_c(tmp_path):
    exe = tmp_path / "block_check"
    build = subprocess.run(
        ["gcc", "-std=gnu11", "-O1", "-Wall", "-Wextra", "-Werror", "-D__HIP_PLATFORM_AMD__",
         "-isystem", os.path.join(ROCM, "include"), "-I", os.path.join(ROOT, "include"),
         os.path.join(ROOT, "tests", "capi", "block_check.c"), "-o", str(exe),
         "-L", LIBDIR, "-l:libzero_shard.so", f"-Wl,-rpath,{LIBDIR}",
         "-L", os.path.join(ROCM, "lib"), "-lamdhip64", f"-Wl,-rpath,{os.path.join(ROCM, 'lib')}", "-lm"],
        capture_output=True, text=True)
    assert build.returncode == 0, build.stderr[-3000:]
    print("[gpu] C ABI block check", flush=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, (run.stdout + run.stderr)[-3000:]
    for what in ("update", "boundary", "policy loss"):
        assert f"{what}: 0 differ" in run.stdout, run.stdout
