"""CPU check of the multi-query attention kernel's launch order: every CTA works on a
place inside the call, also in grids whose CTA numbers pass 32 bits (varlen batches of
many sequences with a large longest prompt and many splits)."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "tests", "native", "prefill_order_check.cpp")


def test_every_cta_has_a_place_inside_the_call(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    exe = tmp_path / "prefill_order_check"
    subprocess.run([cxx, "-O2", "-fwrapv", "-std=c++17", "-o", str(exe), SRC], check=True)
    r = subprocess.run([str(exe)], stdout=subprocess.PIPE, timeout=300)
    assert r.returncode == 0, r.stdout.decode()
