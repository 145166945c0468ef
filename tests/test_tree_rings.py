"""The tcgen05 tree decode's rings between producers and consumers, modelled on the host under any schedule."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("rings") / "ring_model")
    src = os.path.join(ROOT, "tests", "ring_model.cu")
    r = subprocess.run([NVCC, "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "include"),
                        "-I", os.path.join(ROOT, "paged_kv_gqa_13_gb300", "csrc"), src, "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return out


def test_no_barrier_of_a_ring_gets_two_phases_ahead_of_a_role(model):
    r = subprocess.run([model], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "10 of 10 sound" in r.stdout, r.stdout


def test_the_model_finds_a_rule_that_waits_for_places_of_others(model):
    r = subprocess.run([model, "planted"], capture_output=True, text=True, timeout=300)
    # one producer alone (E4M3, narrow, head_dim 64 and 128) has no places of others
    assert r.returncode == 0 and "\n2 of 10 sound" in r.stdout, r.stdout
