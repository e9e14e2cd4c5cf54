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


@pytest.mark.parametrize("B,T,D,fits", [
    ((1 << 23) - 1, 1, 128, True), (1 << 23, 1, 128, False), (4194304, 1, 256, False), (4194303, 64, 256, True),
    (4194303, 96, 136, True), (4194303, 97, 8, True), (4194303, 97, 136, False), (1, 1 << 30, 8, False),
    (1, 805306272, 8, False), (1, 805306273, 8, False), (8, 100663200, 8, False), (9, 89478400, 8, True),
    (1, 805306176, 8, True), (8, 100663104, 8, True),   # (2^23 - 2) 96 and (2^20 - 2) 96: the carriers' places are taken off
])
def test_how_many_tiles_a_scan_may_have(B, T, D, fits):
    """2^23 - 1 workgroups of 512 threads: a tile each, and in up to eight columns
    of several tiles a carrier each."""
    import ctypes

    import gated_delta_rule_77_amd as pdn
    lib = pdn.load_library()
    fake = 0x10000   # never dereferenced: only the checks see it
    a = pdn.ScanArgs()
    a.B, a.T, a.D, a.dtype, a.log_dtype, a.gain = B, T, D, pdn.PDN_BF16, pdn.PDN_BF16, 0
    a.x = a.log_a = a.h = fake
    a.x_sb = a.log_a_sb = a.h_sb = T * D
    a.x_st = a.log_a_st = a.h_st = D
    a.workspace, a.workspace_bytes = fake, 1 << 62
    # (sizes past the limit of B T and B D are refused before that)
    over = B * T > 1 << 30 or B * D > 1 << 30
    assert lib.pdn_scan_check(ctypes.byref(a)) == (pdn.PDN_OK if fits and not over else pdn.PDN_EUNSUPPORTED)
