"""Errors of the CUDA runtime around the 4-bit cache's launches, on a fake of the runtime (tests/kv4_launch_errors.cc).

A launch that succeeded returns ATTN_OK whatever another call left behind before; one that failed returns ATTN_ERR_CUDA,
launched nothing and leaves no error for a later call to take for its own.
"""

import os
import subprocess

import pytest

from attention_tiled_attn_b200 import build as attn_build

HERE = os.path.dirname(os.path.abspath(__file__))
ATTN_ERR_CUDA = -13


@pytest.fixture(scope="module")
def cases(tmp_path_factory):
    objects = [os.path.join(attn_build.BUILD_DIR, f"{name}.o") for name in ("kv4_sm100", "kv4_decode_sm100")]
    attn_build.build(force=not all(os.path.exists(o) for o in objects))
    exe = str(tmp_path_factory.mktemp("kv4") / "launch_errors")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(attn_build.nvcc()))), "include")
    subprocess.run(["g++", "-std=c++17", "-O1", os.path.join(HERE, "kv4_launch_errors.cc"), *objects, "-o", exe,
                    "-I", attn_build.CSRC, "-I", attn_build.INCLUDE, "-I", cuda], check=True)
    lines = subprocess.run([exe], check=True, capture_output=True, text=True, timeout=60).stdout.split("\n")
    return [line.split() for line in lines if line]


def test_a_launch_is_judged_by_its_own_status(cases):
    seen = 0
    for op, pending, failing, status, launches, left in cases:
        if failing == "-":
            assert (int(status), int(launches)) == (0, 1), f"{op} after error {pending}"
            assert left == pending  # another call's error is left to its own reader
            seen += 1
    assert seen == 12


def test_a_failed_launch_leaves_no_error_behind(cases):
    seen = 0
    for op, pending, failing, status, launches, left in cases:
        if failing != "-":
            assert (int(status), int(launches), int(left)) == (ATTN_ERR_CUDA, 0, 0), f"{op} with a failing {failing}"
            seen += 1
    assert seen == 16
