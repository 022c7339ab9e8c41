"""Latent decode plans whose CUDA calls fail (host code over a fake runtime, no GPU): see
tests/c/latent_plan_failures.cpp."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_plans_and_updates_that_fail(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    include = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    if cxx is None or not os.path.exists(os.path.join(include, "cuda_runtime.h")):
        pytest.skip("needs a C++ compiler and the CUDA headers")
    csrc = os.path.join(ROOT, "paged_kv_attention_32_gb300", "csrc")
    exe = str(tmp_path / "latent_plan_failures")
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-I", csrc, "-I", os.path.join(ROOT, "include"),
                        "-I", include, os.path.join(ROOT, "tests", "c", "latent_plan_failures.cpp"),
                        os.path.join(csrc, "latent_abi.cpp"), os.path.join(csrc, "latent_plan.cpp"),
                        "-ldl", "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
