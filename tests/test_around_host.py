"""Host-side checks of the operators around the recurrence (no GPU, nothing
launched): struct mirrors, refusals, workspace sizes, the inverse frequencies,
and the references' own consistency."""
import ctypes
import math
import os
import re
import subprocess

import numpy as np
import pytest

import around_ref as ref
import gated_delta_rule_77_amd as pdn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # never dereferenced: only the checks see it


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(pdn.LIB_PATH):
        from gated_delta_rule_77_amd import build
        build.build()
    return pdn.load_library()


STRUCTS = {"pdn_qk_norm_args": pdn.QkNormArgs, "pdn_qk_norm_bwd_args": pdn.QkNormBwdArgs,
           "pdn_out_norm_args": pdn.OutNormArgs, "pdn_out_norm_bwd_args": pdn.OutNormBwdArgs,
           "pdn_scan_args": pdn.ScanArgs, "pdn_scan_bwd_args": pdn.ScanBwdArgs,
           "pdn_scan_step_args": pdn.ScanStepArgs}


def test_exports_every_declared_symbol(lib):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "pdn_layer.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(pdn_[a-z_0-9]+)\s*\(", src))
    assert names == set(pdn.EXPORTED_LAYER)
    out = subprocess.run(["nm", "-D", "--defined-only", pdn.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert names <= set(re.findall(r"\bT (pdn_[a-z_0-9]+)", out))


def test_struct_layouts_match_the_header(tmp_path):
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "pdn_layer.h"', "int main(void){"]
    for c, m in STRUCTS.items():
        lines.append('printf("%s %%zu\\n", sizeof(%s));' % (c, c))
        lines += ['printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (c, f, c, f) for f, _ in m._fields_]
    lines += ['printf("mark %d\\nversion %d\\n", PDN_SCAN_MARK, PDN_LAYER_VERSION);', "return 0;}"]
    (tmp_path / "l.c").write_text("\n".join(lines))
    subprocess.check_call(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(tmp_path / "l.c"), "-o", str(tmp_path / "l")])
    got = dict(l.split() for l in subprocess.check_output([str(tmp_path / "l")], text=True).splitlines())
    for c, m in STRUCTS.items():
        assert int(got[c]) == ctypes.sizeof(m), c
        for f, _ in m._fields_:
            assert int(got[c + "." + f]) == getattr(m, f).offset, (c, f)
    assert int(got["mark"]) == pdn.PDN_SCAN_MARK
    assert int(got["version"]) == pdn.PDN_LAYER_VERSION == pdn.load_library().pdn_layer_version()


def test_binding_refuses_a_library_of_another_layer_version(tmp_path):
    for layer in ("", "int pdn_layer_version(void) { return %d; }" % (pdn.PDN_LAYER_VERSION + 1)):
        stub = tmp_path / "stub.c"
        stub.write_text("\n".join(
            ["int pdn_abi_version(void) { return %d; }" % pdn.PDN_ABI_VERSION,
             "const char *pdn_strerror(int c) { (void)c; return \"stub\"; }", layer] +
            ["int %s(void *a, void *b) { (void)a; (void)b; return -1; }" % n
             for n in pdn.EXPORTED if n not in ("pdn_abi_version", "pdn_strerror")]))
        so = tmp_path / ("libstub%d.so" % len(layer))
        subprocess.check_call(["gcc", "-shared", "-fPIC", str(stub), "-o", str(so)])
        with pytest.raises(RuntimeError, match="pdn_layer.h"):
            pdn.load_library(str(so))


def _qk():
    a = pdn.QkNormArgs()
    a.B, a.T, a.H, a.Hq, a.Hk, a.d = 2, 100, 8, 8, 2, 128
    a.dtype, a.norm, a.eps, a.q_scale, a.k_scale = pdn.PDN_BF16, pdn.PDN_NORM_RMS, 1e-6, 1.0, 1.0
    a.rot_dim, a.rope_layout, a.rope_scale, a.inv_freq, a.positions = 64, pdn.PDN_ROPE_HALF, 1.0, FAKE, FAKE
    a.wq = a.wk = a.xq = a.xk = a.q = a.k = FAKE
    a.xq_sb, a.xq_st, a.xq_sh = 100 * 2304, 2304, 128
    a.xk_sb, a.xk_st, a.xk_sh = 100 * 2304, 2304, 128
    return a


def _qkb():
    a = pdn.QkNormBwdArgs()
    a.fwd = _qk()
    a.dq = a.dk = a.dxq = a.dxk = a.dwq = a.dwk = FAKE
    a.dxq_sb, a.dxq_st, a.dxq_sh = 100 * 1280, 1280, 128
    a.dxk_sb, a.dxk_st, a.dxk_sh = 100 * 1280, 1280, 128
    a.workspace, a.workspace_bytes = FAKE, 1 << 40
    return a


def _out():
    a = pdn.OutNormArgs()
    a.B, a.H, a.T, a.dv, a.o_dtype, a.dtype, a.act, a.eps = 2, 8, 100, 96, pdn.PDN_F32, pdn.PDN_BF16, pdn.PDN_ACT_SILU, 1e-6
    a.o = a.w = a.z = a.y = FAKE
    a.z_sb, a.z_st, a.z_sh = 100 * 768, 768, 96
    a.y_sb, a.y_st, a.y_sh = 100 * 768, 768, 96
    return a


def _outb():
    a = pdn.OutNormBwdArgs()
    a.fwd = _out()
    a.dy = a.d_o = a.dz = a.dw = FAKE
    a.dy_sb, a.dy_st, a.dy_sh = 100 * 768, 768, 96
    a.dz_sb, a.dz_st, a.dz_sh = 100 * 768, 768, 96
    a.workspace, a.workspace_bytes = FAKE, 1 << 40
    return a


def _scan():
    a = pdn.ScanArgs()
    a.B, a.T, a.D, a.dtype, a.log_dtype, a.gain = 2, 1000, 72, pdn.PDN_BF16, pdn.PDN_F32, pdn.PDN_GAIN_NORM
    a.x = a.log_a = a.h0 = a.hT = a.h = a.marks = FAKE
    a.x_sb, a.x_st, a.log_a_sb, a.log_a_st, a.h_sb, a.h_st = 72000, 72, 72000, 72, 72000, 72
    a.workspace, a.workspace_bytes = FAKE, 1 << 40
    return a


def _scanb():
    a = pdn.ScanBwdArgs()
    a.fwd = _scan()
    a.dh = a.dhT = a.dx = a.dlog_a = a.dh0 = FAKE
    a.dh_sb, a.dh_st, a.dx_sb, a.dx_st, a.dlog_a_sb, a.dlog_a_st = 72000, 72, 72000, 72, 72000, 72
    a.workspace, a.workspace_bytes = FAKE, 1 << 40
    return a


def _step():
    a = pdn.ScanStepArgs()
    a.B, a.D, a.dtype, a.log_dtype, a.gain = 4, 72, pdn.PDN_BF16, pdn.PDN_BF16, pdn.PDN_GAIN_COMPLEMENT
    a.x = a.log_a = a.h_prev = a.h_next = a.h = FAKE
    a.x_sb = a.log_a_sb = a.h_sb = 72
    return a


KINDS = {"pdn_qk_norm_fwd": _qk, "pdn_qk_norm_bwd": _qkb, "pdn_out_norm_fwd": _out, "pdn_out_norm_bwd": _outb,
         "pdn_scan_fwd": _scan, "pdn_scan_bwd": _scanb, "pdn_scan_step": _step}


def _check(lib, call, a):
    return getattr(lib, pdn._AROUND[call][1])(ctypes.byref(a))


@pytest.mark.parametrize("call", KINDS)
def test_valid_arguments_and_nothing(lib, call):
    assert _check(lib, call, KINDS[call]()) == pdn.PDN_OK
    assert getattr(lib, pdn._AROUND[call][1])(None) == pdn.PDN_EINVAL
    assert getattr(lib, call)(None, None) == pdn.PDN_EINVAL
    size = pdn._AROUND[call][2]
    if size:
        n = ctypes.c_size_t(0)
        a = KINDS[call]()
        assert getattr(lib, size)(ctypes.byref(a), ctypes.byref(n)) == pdn.PDN_OK
        assert getattr(lib, size)(None, ctypes.byref(n)) == pdn.PDN_EINVAL
        assert getattr(lib, size)(ctypes.byref(a), None) == pdn.PDN_EINVAL
        assert n.value > 0
        a.workspace_bytes = n.value
        assert _check(lib, call, a) == pdn.PDN_OK
        a.workspace_bytes = n.value - 1
        assert _check(lib, call, a) == pdn.PDN_EWORKSPACE
        assert getattr(lib, call)(ctypes.byref(a), None) == pdn.PDN_EWORKSPACE
        a.workspace, a.workspace_bytes = None, n.value
        assert _check(lib, call, a) == pdn.PDN_EWORKSPACE
        a.workspace = FAKE + 4
        assert _check(lib, call, a) == pdn.PDN_EINVAL


E, N = pdn.PDN_EINVAL, pdn.PDN_EUNSUPPORTED
REFUSED = [
    ("pdn_qk_norm_fwd", {"B": 0}, E), ("pdn_qk_norm_fwd", {"T": -1}, E), ("pdn_qk_norm_fwd", {"H": 0}, E),
    ("pdn_qk_norm_fwd", {"Hq": 3}, E), ("pdn_qk_norm_fwd", {"Hk": 0}, E), ("pdn_qk_norm_fwd", {"Hq": 16}, E),
    ("pdn_qk_norm_fwd", {"d": 96}, N), ("pdn_qk_norm_fwd", {"dtype": 2}, E), ("pdn_qk_norm_fwd", {"norm": 3}, E),
    ("pdn_qk_norm_fwd", {"eps": 0.0}, E), ("pdn_qk_norm_fwd", {"eps": -1e-6}, E), ("pdn_qk_norm_fwd", {"eps": math.nan}, E),
    ("pdn_qk_norm_fwd", {"eps": 1e-41}, E), ("pdn_qk_norm_fwd", {"eps": math.inf}, E),
    ("pdn_qk_norm_fwd", {"norm": 0}, E),                      # weights without a norm
    ("pdn_qk_norm_fwd", {"q_scale": math.inf}, E), ("pdn_qk_norm_fwd", {"k_scale": math.nan}, E),
    ("pdn_qk_norm_fwd", {"rot_dim": 8}, N), ("pdn_qk_norm_fwd", {"rot_dim": 144}, E), ("pdn_qk_norm_fwd", {"rot_dim": -16}, E),
    ("pdn_qk_norm_fwd", {"rope_layout": 2}, E), ("pdn_qk_norm_fwd", {"inv_freq": None}, E),
    ("pdn_qk_norm_fwd", {"rope_scale": math.nan}, E), ("pdn_qk_norm_fwd", {"positions": FAKE + 8}, E),
    ("pdn_qk_norm_fwd", {"xq": None}, E), ("pdn_qk_norm_fwd", {"k": None}, E), ("pdn_qk_norm_fwd", {"xk": FAKE + 2}, E),
    ("pdn_qk_norm_fwd", {"xq_st": 2300}, E), ("pdn_qk_norm_fwd", {"xk_sh": -128}, E), ("pdn_qk_norm_fwd", {"xq_sb": 1 << 60}, E),
    ("pdn_qk_norm_fwd", {"wq": FAKE + 4}, E), ("pdn_qk_norm_fwd", {"B": 1 << 22, "H": 8}, N),
    ("pdn_qk_norm_fwd", {"B": 1 << 16, "T": 1 << 15}, N),
    # more workgroups than a launch has room for
    ("pdn_qk_norm_fwd", {"B": 1 << 14, "T": 1 << 15, "H": 1, "Hq": 1, "Hk": 1}, N),
    ("pdn_out_norm_fwd", {"B": 1 << 14, "T": 1 << 14, "H": 1, "dv": 256}, N),
    ("pdn_scan_fwd", {"B": 1 << 20, "T": 1000, "D": 8}, N),
    ("pdn_scan_bwd", {"fwd.B": 1 << 20, "fwd.T": 1000, "fwd.D": 8}, N),
    ("pdn_qk_norm_bwd", {"fwd.Hk": 5}, E), ("pdn_qk_norm_bwd", {"dq": None}, E), ("pdn_qk_norm_bwd", {"dxk": None}, E),
    ("pdn_qk_norm_bwd", {"dwq": None}, E), ("pdn_qk_norm_bwd", {"fwd.wk": None}, E), ("pdn_qk_norm_bwd", {"dxq_sh": 64}, E),
    ("pdn_qk_norm_bwd", {"dxk_st": 0}, E), ("pdn_qk_norm_bwd", {"dxq_sb": 1280}, E), ("pdn_qk_norm_bwd", {"dk": FAKE + 8}, E),
    ("pdn_out_norm_fwd", {"dv": 40}, N), ("pdn_out_norm_fwd", {"dv": 272}, N), ("pdn_out_norm_fwd", {"dv": 0}, E),
    ("pdn_out_norm_fwd", {"o_dtype": 5}, E), ("pdn_out_norm_fwd", {"act": 3}, E), ("pdn_out_norm_fwd", {"act": 0}, E),
    ("pdn_out_norm_fwd", {"z": None}, E), ("pdn_out_norm_fwd", {"y": None}, E), ("pdn_out_norm_fwd", {"y_st": 760}, E),
    ("pdn_out_norm_fwd", {"z_sh": 97}, E), ("pdn_out_norm_fwd", {"eps": 0.0}, E), ("pdn_out_norm_fwd", {"o": FAKE + 4}, E),
    ("pdn_out_norm_bwd", {"dw": None}, E), ("pdn_out_norm_bwd", {"dz": None}, E), ("pdn_out_norm_bwd", {"d_o": None}, E),
    ("pdn_out_norm_bwd", {"dz_st": 8}, E), ("pdn_out_norm_bwd", {"dy": None}, E), ("pdn_out_norm_bwd", {"fwd.dv": 8}, N),
    ("pdn_scan_fwd", {"D": 12}, N), ("pdn_scan_fwd", {"D": 0}, E), ("pdn_scan_fwd", {"T": -1}, E), ("pdn_scan_fwd", {"gain": 3}, E),
    ("pdn_scan_fwd", {"dtype": 0, "log_dtype": 1}, N), ("pdn_scan_fwd", {"log_dtype": 2}, E), ("pdn_scan_fwd", {"x": None}, E),
    ("pdn_scan_fwd", {"h": None}, E), ("pdn_scan_fwd", {"h_st": 64}, E), ("pdn_scan_fwd", {"h_st": 0}, E),
    ("pdn_scan_fwd", {"x_st": 73}, E), ("pdn_scan_fwd", {"log_a_st": 74}, E), ("pdn_scan_fwd", {"h0": FAKE + 4}, E),
    ("pdn_scan_fwd", {"marks": FAKE + 8}, E), ("pdn_scan_fwd", {"B": 1 << 21, "T": 1 << 10}, N),
    ("pdn_scan_fwd", {"B": 1 << 16, "D": 1 << 16}, N),
    ("pdn_scan_bwd", {"dh": None}, E), ("pdn_scan_bwd", {"dx": None}, E), ("pdn_scan_bwd", {"dlog_a": FAKE + 4}, E),
    ("pdn_scan_bwd", {"dx_st": 8}, E), ("pdn_scan_bwd", {"dhT": FAKE + 2}, E), ("pdn_scan_bwd", {"fwd.gain": -1}, E),
    ("pdn_scan_step", {"B": 0}, E), ("pdn_scan_step", {"D": 20}, N), ("pdn_scan_step", {"h_next": None}, E),
    ("pdn_scan_step", {"h_sb": 8}, E), ("pdn_scan_step", {"x_sb": -72}, E), ("pdn_scan_step", {"h_prev": FAKE + 4}, E),
]


@pytest.mark.parametrize("call,change,code", REFUSED, ids=lambda v: str(v))
def test_refusals(lib, call, change, code):
    a = KINDS[call]()
    for f, v in change.items():
        t = a
        for part in f.split(".")[:-1]:
            t = getattr(t, part)
        setattr(t, f.split(".")[-1], v)
    assert _check(lib, call, a) == code
    assert getattr(lib, call)(ctypes.byref(a), None) == code   # before any launch


def test_what_is_not_read_is_not_checked(lib):
    a = _qk()
    a.T, a.xq, a.q = 0, None, None
    assert _check(lib, "pdn_qk_norm_fwd", a) == pdn.PDN_OK
    a = _qk()
    a.B, a.xq_sb, a.xk_sb = 1, 3, -5             # the stride of a dimension of size 1
    assert _check(lib, "pdn_qk_norm_fwd", a) == pdn.PDN_OK
    a = _qk()
    a.rot_dim, a.inv_freq, a.rope_layout = 0, None, 9
    assert _check(lib, "pdn_qk_norm_fwd", a) == pdn.PDN_OK
    a = _qkb()
    a.fwd.q = a.fwd.k = None
    assert _check(lib, "pdn_qk_norm_bwd", a) == pdn.PDN_OK
    a = _qkb()                                   # heads before tokens is an order like another
    a.dxq_sb, a.dxq_sh, a.dxq_st = 100 * 1024, 100 * 128, 128
    assert _check(lib, "pdn_qk_norm_bwd", a) == pdn.PDN_OK
    a = _scan()
    a.x_st, a.x_sb, a.log_a_sb = 0, 0, 0         # inputs may repeat
    assert _check(lib, "pdn_scan_fwd", a) == pdn.PDN_OK
    a = _scan()
    a.T, a.workspace, a.workspace_bytes = 1, None, 0     # one workgroup's span
    assert _check(lib, "pdn_scan_fwd", a) == pdn.PDN_OK
    a.T = 1000
    assert _check(lib, "pdn_scan_fwd", a) == pdn.PDN_EWORKSPACE


def test_calls_without_a_gpu_tensor_are_refused():
    torch = pytest.importorskip("torch")
    x = torch.zeros(1, 4, 8)
    with pytest.raises(ValueError, match="device memory"):
        pdn.pdn_scan_fwd(x, x, x)
    with pytest.raises(ValueError, match="device memory"):
        pdn.pdn_qk_norm_fwd(x, x, x, x)
    with pytest.raises(ValueError, match="device memory"):
        pdn.pdn_out_norm_fwd(x, x)


def test_marks():
    with pytest.raises(pdn.PdnError):
        pdn.pdn_scan_marks(-1)
    m = pdn.PDN_SCAN_MARK
    assert [pdn.pdn_scan_marks(t) for t in (0, 1, m, m + 1, 10 * m - 1)] == [0, 1, 1, 2, 10]


def test_inverse_frequencies():
    f, s = pdn.pdn_rope_freqs(64, 10000.0)
    np.testing.assert_allclose(f, 10000.0 ** (-np.arange(0, 64, 2) / 64), rtol=1e-14)
    assert s == 1.0
    g, s = pdn.pdn_rope_freqs(64, 10000.0, pdn.PDN_ROPE_LINEAR, 4.0)
    np.testing.assert_allclose(g, np.array(f) / 4, rtol=1e-14)
    g, s = pdn.pdn_rope_freqs(64, 10000.0, pdn.PDN_ROPE_BASE, 8.0)
    assert g[0] == 1.0 and abs(g[-1] * 8 / f[-1] - 1) < 1e-12 and s == 1.0
    g, s = pdn.pdn_rope_freqs(128, 10000.0, pdn.PDN_ROPE_BY_PARTS, 16.0, 4096)
    f = 10000.0 ** (-np.arange(0, 128, 2) / 128)
    turns = 4096 * f / (2 * np.pi)
    np.testing.assert_allclose(np.array(g)[turns > 32], f[turns > 32], rtol=1e-14)
    np.testing.assert_allclose(np.array(g)[turns < 1], f[turns < 1] / 16, rtol=1e-14)
    assert np.all(np.diff(g) < 0) and abs(s - (0.1 * math.log(16.0) + 1)) < 1e-7
    g, s = pdn.pdn_rope_freqs(128, 10000.0, pdn.PDN_ROPE_BY_PARTS, 1.0, 4096)
    np.testing.assert_allclose(g, f, rtol=1e-14)
    assert s == 1.0
    for bad in ((0, 1e4), (3, 1e4), (64, 1.0), (64, math.inf), (64, 1e4, 4), (64, 1e4, 1, 0.5), (64, 1e4, 3, 2.0, 0), (2, 1e4, 2, 2.0)):
        with pytest.raises(pdn.PdnError):
            pdn.pdn_rope_freqs(*bad)


def test_reference_gradients_against_differences():
    """The references' hand-written gradients against central differences of
    their forwards, in 64 bits (step 1e-5: errors about 1e-9)."""
    rng = np.random.default_rng(5)

    def slope(f, x, g, h=1e-5):
        v = rng.standard_normal(x.shape)
        return (f(x + h * v) - f(x - h * v)) / (2 * h), (g * v).sum()

    x, w = rng.standard_normal((2, 3, 2, 16)), rng.standard_normal(16)
    g = rng.standard_normal((2, 4, 3, 16))
    for norm in (0, 1, 2):
        for layout in (0, 1):
            rot = ref.rotation(rng.integers(0, 9, (2, 3)), np.array([0.7, 0.1, 0.02]), 16, layout, 1.2)
            wv = w if norm else None
            f = lambda t: (ref.qk_one(t, wv, 0.3, 4, norm, 1e-3, rot)[0] * g).sum()
            dx, _, dw, _ = ref.qk_one_bwd(x, wv, 0.3, g, norm, 1e-3, rot)
            a, b = slope(f, x, dx)
            assert abs(a - b) < 1e-7 * max(1, abs(a))
            if norm:
                a, b = slope(lambda u: (ref.qk_one(x, u, 0.3, 4, norm, 1e-3, rot)[0] * g).sum(), w, dw)
                assert abs(a - b) < 1e-7 * max(1, abs(a))
    o, z, dy = rng.standard_normal((2, 3, 4, 16)), rng.standard_normal((2, 4, 3, 16)), rng.standard_normal((2, 4, 3, 16))
    for kind in (0, 1, 2):
        (do, _), dz, (dw, _) = ref.out_bwd(o, w, z, dy, kind, 1e-3)
        for f, at, grad in ((lambda t: ref.out_fwd(t, w, z, kind, 1e-3), o, do), (lambda t: ref.out_fwd(o, t, z, kind, 1e-3), w, dw),
                            (lambda t: ref.out_fwd(o, w, t, kind, 1e-3), z, dz[0] if kind else 0 * z)):
            a, b = slope(lambda t: (f(t)[0] * dy).sum(), at, grad)
            assert abs(a - b) < 1e-7 * max(1, abs(a))
    x, la, h0 = rng.standard_normal((2, 9, 4)), -rng.uniform(0.05, 1, (2, 9, 4)), rng.standard_normal((2, 4))
    dh, dhT = rng.standard_normal((2, 9, 4)), rng.standard_normal((2, 4))
    for kind in (0, 1, 2):
        f = lambda a, b, c: (lambda h: (h * dh).sum() + (h[:, -1] * dhT).sum())(ref.scan_fwd(a, b, c, kind)[0])
        dx, dla, dh0 = (p[0] for p in ref.scan_bwd(x, la, h0, dh, dhT, kind))
        for a, b in (slope(lambda t: f(t, la, h0), x, dx), slope(lambda t: f(x, t, h0), la, dla), slope(lambda t: f(x, la, t), h0, dh0)):
            assert abs(a - b) < 1e-7 * max(1, abs(a))
