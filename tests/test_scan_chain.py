"""How the scan's tiles hand their state on (csrc/scan_chain.h), on the host:
tests/scan_chain_check.cpp compiles that header with g++ and runs tiles and
carriers in orders a device may give them, one where the carrier gives up among
them."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "gated_delta_rule_77_amd", "csrc")


@pytest.mark.timeout(300)
def test_tiles_get_their_state_in_every_order(tmp_path):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("g++ is needed to build the check")
    exe = str(tmp_path / "scan_chain_check")
    # no contraction: the recurrence's fused steps are written out
    subprocess.check_call([gxx, "-std=c++17", "-O2", "-ffp-contract=off", "-pthread", "-I", CSRC,
                           os.path.join(HERE, "scan_chain_check.cpp"), "-o", exe])
    r = subprocess.run([exe], capture_output=True, text=True, timeout=240)
    print(r.stdout)
    assert r.returncode == 0, r.stdout
    assert r.stdout.count(": right") == 30 and "WRONG" not in r.stdout
