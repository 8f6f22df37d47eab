"""CPU check of the 8-bit decode kernel's ring: no warp reads a tile before it has landed.

Below 8 kv heads a CTA two warps share a head and take pairs of tiles in turn; a stage's
barrier is waited for by the parity of the stage's round.  The program compiled here uses
the kernel's stage counts and dealing rule and walks both warps over segments of all tile
counts, then runs the protocol with copies that land late and in any order.
"""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "tests", "native", "decode_ring_check.cpp")


def test_no_warp_skips_a_round_of_its_stages(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    exe = tmp_path / "decode_ring_check"
    subprocess.run([cxx, "-O2", "-std=c++17", "-o", str(exe), SRC], check=True)
    r = subprocess.run([str(exe)], stdout=subprocess.PIPE, timeout=300)
    assert r.returncode == 0, r.stdout.decode()
