"""The stages of the gated scan's copies (csrc/copy_stages.h) against a model of mbarriers (CPU): a wait that gives up is
followed by waits for exactly the copies that are under way."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "linear_recurrent_sequence_causal_gb300", "csrc")


def test_every_wait_sees_its_own_copy(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    exe = tmp_path / "copy_stages"
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", os.path.join(ROOT, "tests", "c", "copy_stages.cpp"),
                        "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_both_scans_take_a_copy_after_its_wait_is_known_to_have_passed():
    """The failed stage keeps its parity until the CTA has drained: taken() comes behind the drain."""
    src = open(os.path.join(CSRC, "gated_scan.cuh")).read()
    steps = re.findall(r"stages\.parity\(it\)|gated_drain\(p, sm, stages, it\)|stages\.taken\(it\)", src)
    assert steps == ["stages.parity(it)", "gated_drain(p, sm, stages, it)", "stages.taken(it)"] * 2
