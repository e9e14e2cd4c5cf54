"""How the calls of include/pdn_block.h are dealt over the device, seen by their workspace
sizes (no GPU, nothing launched)."""
import ctypes

import pytest

import gated_delta_rule_77_amd as pdn
from test_block_host import _attn, _attnb, _paged, lib  # noqa: F401  the fixture


def _parts(lib, call, a, rows):
    """Workgroups that share a row's keys: each leaves d + 2 numbers of it."""
    n = ctypes.c_size_t(0)
    assert getattr(lib, pdn._BLOCK[call][2])(ctypes.byref(a), ctypes.byref(n)) == pdn.PDN_OK
    each = rows * (128 + 2) * 4
    assert n.value % each == 0 and n.value != each
    return max(1, n.value // each)


def _call(**kw):
    B, H, Hk, Tq, Tk = (kw[n] for n in ("B", "H", "Hk", "Tq", "Tk"))
    return _attn(q_sb=H * Tq * 128, q_sh=Tq * 128, k_sb=Hk * Tk * 128, k_sh=Tk * 128, v_sb=Hk * Tk * 128, v_sh=Tk * 128, v_st=128,
                 o_sb=H * Tq * 128, o_sh=Tq * 128, o_st=128, **kw)


# a part has 512 keys at the least (96 of fp32): of those that a workgroup's rows can see
@pytest.mark.parametrize("window", [1, 64, 200, 700, 2000, 4095, 4096, 0])
@pytest.mark.parametrize("Tq,Tk", [(4096, 4096), (500, 16384), (1, 16384), (4096, 300)])
@pytest.mark.parametrize("bf16", [True, False])
def test_windows_bound_the_parts(lib, window, Tq, Tk, bf16):  # noqa: F811
    H, Hk, types = 4, 4, dict(dtype=pdn.PDN_BF16, o_dtype=pdn.PDN_BF16) if bf16 else dict(dtype=pdn.PDN_F32, o_dtype=pdn.PDN_F32)
    parts = _parts(lib, "pdn_attn_fwd", _call(B=1, H=H, Hk=Hk, Tq=Tq, Tk=Tk, window=window, **types), H * Tq)
    sees = min(Tk, window + min(Tq, 128)) if window else Tk
    assert parts == 1 or parts * (512 if bf16 else 96) <= sees + 1
    if window == 0 and Tk > 4000:
        assert parts > 1


# fewer than nine parts are joined by lanes and may be short in fp32; long keys give more of the usual length
@pytest.mark.parametrize("Tk,least,most", [(300, 3, 3), (700, 7, 7), (1500, 8, 8), (2600, 10, 10), (11056, 22, 22)])
def test_short_parts_are_few_and_long_keys_have_many(lib, Tk, least, most):  # noqa: F811
    a = _call(B=2, H=12, Hk=12, Tq=113, Tk=Tk, window=0, dtype=pdn.PDN_F32, o_dtype=pdn.PDN_F32)
    assert least <= _parts(lib, "pdn_attn_fwd", a, 2 * 12 * 113) <= most


@pytest.mark.parametrize("window", [1, 64, 200, 700, 2000, 0])
@pytest.mark.parametrize("new", [1, 7, 400])
def test_windows_bound_the_parts_of_a_cache(lib, window, new):  # noqa: F811
    a = _paged(window=window, cache__B=2, cache__N=2 * new, cache__max_new=new, cache__table_width=256)  # of 64 tokens each
    parts = _parts(lib, "pdn_attn_paged", a, 2 * 8 * new)
    sees = window + min(new, 32) if window else 16384   # four heads share a key head: 128 rows are 32 tokens
    assert parts == 1 or parts * 512 <= sees + 1
    if window == 0:
        assert parts > 1


def test_first_keys_cost_the_backward_one_number_a_tile(lib):  # noqa: F811
    """The least first key of each 32 queries; every part of the workspace ends at 256 bytes."""
    sizes = []
    for first in (0x10000, None):
        a, n = _attnb(fwd__Tq=6400, fwd__Tk=6400, fwd__first=first), ctypes.c_size_t(0)
        for name in ("fwd__q", "fwd__k", "fwd__v", "fwd__o", "d_o", "dq", "dk", "dv"):
            path = name.split("__")
            at = a.fwd if len(path) == 2 else a
            stem = {"d_o": "do"}.get(path[-1], path[-1])
            for s, step in (("sb", 1 << 24), ("sh", 1 << 20), ("st", 128)):
                setattr(at, stem + "_" + s, step)
        assert lib.pdn_attn_bwd_workspace_size(ctypes.byref(a), ctypes.byref(n)) == pdn.PDN_OK
        sizes.append(n.value)
    assert sizes[0] - sizes[1] == -(-4 * 2 * 200 // 256) * 256
