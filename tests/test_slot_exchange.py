"""The warps of a row slot leave their loop at the same row when one of them
gives up, whichever of them is slow (csrc/slot_exchange.cuh, compiled for the
CPU; no GPU needed)."""
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "rmsnorm_backward_gb300", "csrc")


def test_a_slot_gives_up_at_one_row(tmp_path):
    exe = tmp_path / "slot_exchange"
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wno-unknown-pragmas", "-pthread", "-I", CSRC,
                        os.path.join(HERE, "slot_exchange.cpp"), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout[-2000:]
    assert r.stdout.splitlines()[-1].endswith(" 0 wrong")
