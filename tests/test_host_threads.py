"""Two host threads on one stream (no GPU: host_threads.cpp stands in for the HIP runtime): the launches of a call that
hands data on in the stream's scratch are not mixed with another call's."""

from __future__ import annotations

import os
import subprocess

import pytest

import persistent_gemm_amd as pg

HERE = os.path.dirname(os.path.abspath(__file__))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    pg.load()
    lib = pg.library_path()
    out = str(tmp_path_factory.mktemp("host_threads") / "host_threads")
    subprocess.run([os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-pthread", "-rdynamic", "-isystem",
                    os.path.join(ROCM, "include"), os.path.join(HERE, "host_threads.cpp"), lib, "-o", out,
                    "-Wl,-rpath," + os.path.dirname(lib), "-Wl,--allow-shlib-undefined"], check=True)
    return out


@pytest.mark.parametrize("calls", ["block_backward", "block_backward_capped", "norm_backward", "bf16_backward",
                                   "block_and_bf16", "block_and_norm", "relaid_scales", "release", "one_unit"])
def test_calls_on_one_stream_do_not_mix(program, calls):
    r = subprocess.run([program, calls], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stdout + r.stderr
