"""The layer operators driven from plain C through include/zero_shard.h (tests/capi/layer_check.c): a linear layer
forward and backward on whole numbers, exact; the cross entropy of a label as a one-entry distillation loss, in two calls and
in one over the logits, against the host's double evaluation; refusals."""

import os
import shutil
import subprocess

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIBDIR = os.path.join(ROOT, "zero_partition_plan_amd")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_layer_from_c(tmp_path):
    exe = tmp_path / "layer_check"
    build = subprocess.run(
        ["gcc", "-std=gnu11", "-O1", "-Wall", "-Wextra", "-Werror", "-D__HIP_PLATFORM_AMD__",
         "-isystem", os.path.join(ROCM, "include"), "-I", os.path.join(ROOT, "include"),
         os.path.join(ROOT, "tests", "capi", "layer_check.c"), "-o", str(exe),
         "-L", LIBDIR, "-l:libzero_shard.so", f"-Wl,-rpath,{LIBDIR}",
         "-L", os.path.join(ROCM, "lib"), "-lamdhip64", f"-Wl,-rpath,{os.path.join(ROCM, 'lib')}", "-lm"],
        capture_output=True, text=True)
    assert build.returncode == 0, build.stderr[-3000:]
    print("[gpu] C ABI layer check", flush=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, (run.stdout + run.stderr)[-3000:]
    assert "linear layer: 0 differ" in run.stdout and "distillation loss: 0 differ" in run.stdout
