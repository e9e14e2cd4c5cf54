"""Host-side checks of the operators of include/pdn_block.h (no GPU, nothing
launched): struct mirrors, refusals, workspace sizes, the cache's map and the
generator compiled for the CPU, and the references' own consistency."""
import ctypes
import math
import os
import re
import subprocess

import pytest
import torch

import block_ref as ref
import gated_delta_rule_77_amd as pdn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # never dereferenced: only the checks see it


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(pdn.LIB_PATH):
        from gated_delta_rule_77_amd import build
        build.build()
    return pdn.load_library()


STRUCTS = {"pdn_add_norm_args": pdn.AddNormArgs, "pdn_add_norm_bwd_args": pdn.AddNormBwdArgs, "pdn_attn_args": pdn.AttnArgs,
           "pdn_attn_bwd_args": pdn.AttnBwdArgs, "pdn_cache": pdn.Cache, "pdn_cache_append_args": pdn.CacheAppendArgs,
           "pdn_attn_paged_args": pdn.AttnPagedArgs}


def test_exports_every_declared_symbol(lib):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "pdn_block.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(pdn_[a-z_0-9]+)\s*\(", src))
    assert names == set(pdn.EXPORTED_BLOCK)
    out = subprocess.run(["nm", "-D", "--defined-only", pdn.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert names <= set(re.findall(r"\bT (pdn_[a-z_0-9]+)", out))


def test_struct_layouts_match_the_header(tmp_path):
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "pdn_block.h"', "int main(void){"]
    for c, m in STRUCTS.items():
        lines.append('printf("%s %%zu\\n", sizeof(%s));' % (c, c))
        lines += ['printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (c, f, c, f) for f, _ in m._fields_]
    lines += ['printf("version %d\\ne4m3 %d\\n", PDN_BLOCK_VERSION, PDN_E4M3);', "return 0;}"]
    (tmp_path / "l.c").write_text("\n".join(lines))
    subprocess.check_call(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(tmp_path / "l.c"), "-o", str(tmp_path / "l")])
    got = dict(l.split() for l in subprocess.check_output([str(tmp_path / "l")], text=True).splitlines())
    for c, m in STRUCTS.items():
        assert int(got[c]) == ctypes.sizeof(m), c
        for f, _ in m._fields_:
            assert int(got[c + "." + f]) == getattr(m, f).offset, (c, f)
    assert int(got["version"]) == pdn.PDN_BLOCK_VERSION == pdn.load_library().pdn_block_version()
    assert int(got["e4m3"]) == pdn.PDN_E4M3


def _fill(a, **kw):
    for n, v in kw.items():
        at = a
        *path, last = n.split("__")
        for p in path:
            at = getattr(at, p)
        setattr(at, last, v)
    return a


def _norm(**kw):
    a = _fill(pdn.AddNormArgs(), B=2, T=100, D=768, dtype=pdn.PDN_BF16, s_dtype=pdn.PDN_F32, y_dtype=pdn.PDN_E4M3, group=128, eps=1e-6,
              drop_p=0.1, seed=FAKE, w=FAKE, x=FAKE * 3, x_sb=76800, x_st=768, res=FAKE, res_sb=76800, res_st=768, s=FAKE * 2, s_sb=76800,
              s_st=768, y=FAKE, y_sb=76800, y_st=768, y_scale=FAKE)
    return _fill(a, **kw)


def _normb(**kw):
    a = _fill(pdn.AddNormBwdArgs(), B=2, T=100, D=768, dtype=pdn.PDN_BF16, s_dtype=pdn.PDN_F32, y_dtype=pdn.PDN_BF16, eps=1e-6, drop_p=0.1,
              seed=FAKE, w=FAKE, dw=FAKE, s=FAKE, s_sb=76800, s_st=768, dy=FAKE, dy_sb=76800, dy_st=768, ds=FAKE, ds_sb=76800, ds_st=768,
              dres=FAKE * 2, dres_sb=76800, dres_st=768, dx=FAKE, dx_sb=76800, dx_st=768, workspace=FAKE, workspace_bytes=1 << 40)
    return _fill(a, **kw)


def _attn(a=None, **kw):
    a = _fill(a or pdn.AttnArgs(), B=2, H=8, Hk=2, Tq=100, Tk=2000, d=128, dtype=pdn.PDN_BF16, o_dtype=pdn.PDN_BF16, window=0, scale=0.1,
              first=FAKE, q=FAKE, q_sb=102400, q_sh=12800, q_st=128, k=FAKE, k_sb=512000, k_sh=256000, k_st=128, v=FAKE, v_sb=512000,
              v_sh=128, v_st=256, o=FAKE, o_sb=102400, o_sh=128, o_st=1024, lse=FAKE, workspace=FAKE, workspace_bytes=1 << 40)
    return _fill(a, **kw)


def _attnb(**kw):
    a = pdn.AttnBwdArgs()
    _attn(a.fwd)
    _fill(a, g_dtype=pdn.PDN_BF16, d_o=FAKE, do_sb=102400, do_sh=128, do_st=1024, dq=FAKE, dq_sb=102400, dq_sh=12800, dq_st=128, dk=FAKE,
          dk_sb=512000, dk_sh=256000, dk_st=128, dv=FAKE, dv_sb=512000, dv_sh=128, dv_st=256, workspace=FAKE, workspace_bytes=1 << 40)
    return _fill(a, **kw)


def _cache(c):
    _fill(c, B=4, N=20, max_new=9, Hk=2, d=128, dtype=pdn.PDN_BF16, pages=50, page_size=64, table_width=20, k_pages=FAKE, k_sp=16384,
          k_st=256, k_sh=128, v_pages=FAKE, v_sp=16384, v_st=256, v_sh=128, table=FAKE, lens=FAKE, starts=FAKE)


def _append(**kw):
    a = pdn.CacheAppendArgs()
    _cache(a.cache)
    _fill(a, k=FAKE, k_sn=512, k_sh=128, v=FAKE, v_sn=512, v_sh=128)
    return _fill(a, **kw)


def _paged(**kw):
    a = pdn.AttnPagedArgs()
    _cache(a.cache)
    _fill(a, H=8, o_dtype=pdn.PDN_F32, window=0, scale=0.1, q=FAKE, q_sn=1024, q_sh=128, o=FAKE, o_sn=1024, o_sh=128, lse=FAKE,
          workspace=FAKE, workspace_bytes=1 << 40)
    return _fill(a, **kw)


KINDS = {"pdn_add_norm_fwd": _norm, "pdn_add_norm_bwd": _normb, "pdn_attn_fwd": _attn, "pdn_attn_bwd": _attnb,
         "pdn_cache_append": _append, "pdn_attn_paged": _paged}


def _check(lib, call, a):
    return getattr(lib, pdn._BLOCK[call][1])(ctypes.byref(a))


@pytest.mark.parametrize("call", KINDS)
def test_valid_arguments_and_nothing(lib, call):
    assert _check(lib, call, KINDS[call]()) == pdn.PDN_OK
    assert getattr(lib, pdn._BLOCK[call][1])(None) == pdn.PDN_EINVAL
    assert getattr(lib, call)(None, None) == pdn.PDN_EINVAL
    size = pdn._BLOCK[call][2]
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
        a.workspace = None
        assert _check(lib, call, a) == pdn.PDN_EWORKSPACE
        a.workspace, a.workspace_bytes = FAKE + 8, n.value
        assert _check(lib, call, a) == pdn.PDN_EINVAL


INF, NAN = math.inf, math.nan
REFUSED = [
    ("pdn_add_norm_fwd", "EINVAL", [dict(B=0), dict(T=-1), dict(D=0), dict(dtype=2), dict(dtype=7), dict(s_dtype=2), dict(y_dtype=3), dict(eps=0.0),
                                    dict(eps=NAN), dict(eps=-1.0), dict(drop_p=1.0), dict(drop_p=-0.1), dict(drop_p=NAN), dict(seed=None),
                                    dict(drop_p=0.0), dict(seed=FAKE + 4), dict(w=FAKE + 4), dict(y_scale=None), dict(y_scale=FAKE + 2),
                                    dict(group=48), dict(group=-1), dict(group=768), dict(y_dtype=pdn.PDN_BF16), dict(s=None), dict(x=None),
                                    dict(y=None), dict(x=FAKE + 8), dict(res=FAKE + 8), dict(y=FAKE + 4), dict(x_st=772), dict(x_st=-768),
                                    dict(s_st=760), dict(y_st=767), dict(y_st=764), dict(y_st=760), dict(s=FAKE, s_sb=153600),
                                    dict(drop_p=0.0, seed=None, res=None), dict(drop_p=0.0, seed=None, res=None, s=None),
                                    dict(D=96, group=64)]),
    ("pdn_add_norm_fwd", "EUNSUPPORTED", [dict(D=772), dict(D=16392), dict(dtype=pdn.PDN_F32, s_dtype=pdn.PDN_BF16), dict(B=1 << 16, T=128)]),
    ("pdn_add_norm_bwd", "EINVAL", [dict(B=0), dict(T=-1), dict(y_dtype=pdn.PDN_E4M3), dict(dw=None), dict(w=None), dict(dw=FAKE + 4), dict(s=None),
                                    dict(dy=None), dict(dres=None), dict(dres_st=760), dict(dx=FAKE + 8), dict(seed=None), dict(dy_st=772),
                                    dict(dres=FAKE, dres_sb=153600), dict(eps=INF)]),
    ("pdn_add_norm_bwd", "EUNSUPPORTED", [dict(D=772), dict(D=16392), dict(dtype=pdn.PDN_F32, s_dtype=pdn.PDN_BF16)]),
    ("pdn_attn_fwd", "EINVAL", [dict(B=0), dict(H=0), dict(Hk=0), dict(Hk=3), dict(Tq=-1), dict(Tk=-1), dict(d=0), dict(dtype=2), dict(o_dtype=2),
                                dict(window=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=INF), dict(scale=NAN), dict(first=FAKE + 2),
                                dict(lse=FAKE + 2), dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(q=FAKE + 8), dict(k_st=132),
                                dict(v_st=-256), dict(o_st=512), dict(o_sh=64)]),
    ("pdn_attn_fwd", "EUNSUPPORTED", [dict(d=96), dict(d=256), dict(dtype=pdn.PDN_F32, o_dtype=pdn.PDN_BF16), dict(B=1 << 22), dict(H=4096),
                                      dict(Tk=(1 << 30) + 1), dict(Tq=1 << 29)]),
    ("pdn_attn_bwd", "EINVAL", [dict(fwd__lse=None), dict(d_o=None), dict(dq=None), dict(dk=None), dict(dv=None), dict(g_dtype=2), dict(dk_st=64),
                                dict(dq=FAKE + 8), dict(dv_sh=64), dict(fwd__scale=0.0), dict(fwd__o=None), dict(do_st=1028)]),
    ("pdn_attn_bwd", "EUNSUPPORTED", [dict(fwd__d=32), dict(fwd__dtype=pdn.PDN_F32, fwd__o_dtype=pdn.PDN_F32)]),
    ("pdn_cache_append", "EINVAL", [dict(cache__B=0), dict(cache__N=-1), dict(cache__max_new=-1), dict(cache__Hk=0), dict(cache__pages=0),
                                    dict(cache__table_width=0), dict(cache__dtype=2), dict(cache__page_size=0), dict(cache__k_pages=None),
                                    dict(cache__v_pages=None), dict(cache__table=None), dict(cache__lens=None), dict(cache__table=FAKE + 2),
                                    dict(cache__lens=FAKE + 1), dict(cache__starts=FAKE + 2), dict(cache__k_st=64), dict(cache__k_sp=16376),
                                    dict(cache__starts=None, cache__N=21), dict(cache__starts=None, cache__max_new=4), dict(k=None), dict(v=None),
                                    dict(k=FAKE + 8), dict(v_sn=516)]),
    ("pdn_cache_append", "EUNSUPPORTED", [dict(cache__page_size=48), dict(cache__page_size=8), dict(cache__page_size=2048), dict(cache__d=132),
                                          dict(cache__B=1 << 21), dict(cache__table_width=1 << 25)]),
    ("pdn_attn_paged", "EINVAL", [dict(H=0), dict(H=3), dict(o_dtype=2), dict(window=-2), dict(scale=0.0), dict(q=None), dict(o=None),
                                  dict(lse=FAKE + 1), dict(q_sn=1028), dict(o_sh=64), dict(cache__lens=None), dict(cache__starts=None, cache__N=21)]),
    ("pdn_attn_paged", "EUNSUPPORTED", [dict(cache__d=96), dict(cache__dtype=pdn.PDN_F32, o_dtype=pdn.PDN_BF16), dict(H=1 << 13),
                                        dict(cache__page_size=24), dict(cache__max_new=1 << 29)]),
]


REFUSED += [  # steps from token to token past the lanes' offsets; a scale that log2(e) takes past fp32
    ("pdn_attn_fwd", "EUNSUPPORTED", [dict(B=1, k_st=(1 << 28) + 8), dict(B=1, v_st=(1 << 28) + 8)]),
    ("pdn_attn_fwd", "EINVAL", [dict(scale=3e38)]),
    ("pdn_attn_bwd", "EUNSUPPORTED", [dict(fwd__q_st=(1 << 28) + 8), dict(do_st=(1 << 28) + 8), dict(fwd__k_st=1 << 29)]),
    ("pdn_attn_paged", "EUNSUPPORTED", [dict(cache__k_st=(1 << 28) + 8), dict(cache__v_st=1 << 30)]),
]


@pytest.mark.parametrize("call,code,change", [(c, e, k) for c, e, ks in REFUSED for k in ks],
                         ids=lambda v: v if isinstance(v, str) else "-".join("%s=%s" % i for i in v.items()))
def test_refusals(lib, call, code, change):
    assert _check(lib, call, KINDS[call](**change)) == getattr(pdn, "PDN_" + code)


ACCEPTED = [
    ("pdn_add_norm_fwd", [dict(T=0, x=None, y=None, s=FAKE), dict(s=FAKE), dict(res=None), dict(drop_p=1e-9), dict(group=0), dict(D=16384, x_st=16384,
     res_st=16384, s_st=16384, y_st=16384, T=1, B=1), dict(drop_p=0.0, seed=None, res=None, s=None, s_dtype=pdn.PDN_BF16),
     dict(B=1, x_sb=-5, y_sb=3), dict(x_st=0), dict(seed=FAKE + 8)]),
    ("pdn_add_norm_bwd", [dict(T=0), dict(ds=None), dict(dx=None), dict(dres=FAKE), dict(w=None, dw=None)]),
    ("pdn_attn_fwd", [dict(Tq=0), dict(Tk=0), dict(Tq=300, Tk=100, q_sb=400000, q_sh=40000, o_sb=400000), dict(window=1), dict(window=2 ** 31 - 1), dict(lse=None, first=None), dict(k_sh=0),
                      dict(o_dtype=pdn.PDN_F32), dict(first=FAKE + 4)]),
    ("pdn_attn_bwd", [dict(fwd__Tq=0), dict(fwd__Tk=0), dict(g_dtype=pdn.PDN_F32), dict(fwd__workspace=None), dict(fwd__o_dtype=pdn.PDN_F32)]),
    ("pdn_cache_append", [dict(cache__N=0, k=None), dict(cache__starts=None), dict(cache__d=8), dict(cache__max_new=0)]),
    ("pdn_attn_paged", [dict(cache__N=0, q=None, o=None), dict(cache__starts=None), dict(lse=None), dict(window=2 ** 31 - 1)]),
]


ACCEPTED += [
    ("pdn_attn_fwd", [dict(k_st=1 << 28, v_st=1 << 28), dict(q_st=1 << 40), dict(Tk=1, k_st=1 << 40)]),
    ("pdn_attn_bwd", [dict(fwd__q_st=1 << 28, do_st=1 << 28), dict(fwd__Tq=1, fwd__q_st=1 << 40)]),
    ("pdn_attn_paged", [dict(cache__k_st=1 << 28, cache__v_st=1 << 28)]),
    ("pdn_cache_append", [dict(k_sn=1 << 40)]),
]


@pytest.mark.parametrize("call,change", [(c, k) for c, ks in ACCEPTED for k in ks],
                         ids=lambda v: v if isinstance(v, str) else "-".join("%s=%s" % i for i in v.items()))
def test_accepted(lib, call, change):
    assert _check(lib, call, KINDS[call](**change)) == pdn.PDN_OK


def test_binding_refuses_host_tensors():
    x = torch.zeros(1, 1, 8)
    with pytest.raises(ValueError, match="device memory"):
        pdn.pdn_add_norm_fwd(x, x)
    t = torch.zeros(1, 1, 1, 64)
    with pytest.raises(ValueError, match="device memory"):
        pdn.pdn_attn_fwd(t, t, t, t)
    with pytest.raises(ValueError, match="device memory"):
        pdn.pdn_attn_paged(t[0], t[0], t, t, None, None)


# -- the cache's map and the generator, compiled for the CPU ------------------

@pytest.fixture(scope="module")
def host_map(tmp_path_factory):
    """The kernels' own header as plain C++."""
    at = tmp_path_factory.mktemp("map")
    (at / "hip").mkdir()
    (at / "hip" / "hip_runtime.h").write_text("#pragma once\n#define __host__\n#define __device__\n#define __forceinline__ inline\n")
    (at / "m.cpp").write_text('''
#include "pages.h"
#include "philox.h"
extern "C" void sequence(const int *table, const int *lens, const int *starts, int B, int N, int width, int pages, int shift, int b, int *out) {
    pdn::PageMap m{table, lens, starts, B, N, width, pages, shift};
    const pdn::Sequence s = pdn::sequence_of(m, b);
    out[0] = s.start; out[1] = s.n; out[2] = s.len;
}
extern "C" int page(const int *table, int B, int width, int pages, int shift, int b, int token) {
    pdn::PageMap m{table, nullptr, nullptr, B, 0, width, pages, shift};
    return pdn::page_of(m, b, token);
}
extern "C" int keeps(unsigned long long key, unsigned long long call, unsigned long long n, unsigned threshold) {
    return pdn::philox_keeps(pdn::philox(key, call, n / 8), n % 8, threshold);
}
extern "C" void words(unsigned long long key, unsigned long long call, unsigned long long block, unsigned *out) {
    const pdn::Philox p = pdn::philox(key, call, block);
    for (int i = 0; i < 4; ++i) out[i] = p.w[i];
}
''')
    so = at / "m.so"
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", str(at),
                           "-I", os.path.join(ROOT, "gated_delta_rule_77_amd", "csrc"), str(at / "m.cpp"), "-o", str(so)])
    return ctypes.CDLL(str(so))


def _ints(*v):
    return (ctypes.c_int * len(v))(*v)


def test_pages_and_sequences_that_lead_nowhere_stay_inside(host_map):
    big, small = 2 ** 31 - 1, -2 ** 31
    for entry in (small, -1, 0, 5, 6, 7, big):
        table = _ints(*[entry] * 12)
        for token in (0, 15, 16, 63):
            assert 0 <= host_map.page(table, 3, 4, 7, 4, 2, token) < 7
            if 0 <= entry < 7:
                assert host_map.page(table, 3, 4, 7, 4, 2, token) == entry
    out = _ints(0, 0, 0)
    for length in (small, -1, 0, 40, 64, 65, big):
        for starts in ((0, 3, 9, 10), (small, big, small, big), (9, 3, 0, -5), (big,) * 4, (0, 0, 0, 0), (10, 10, 10, 11)):
            for b in range(3):
                host_map.sequence(None, _ints(length, length, length), _ints(*starts), 3, 10, 4, 7, 4, b, out)
                start, n, held = out
                assert 0 <= start <= 10 and 0 <= n <= 10 - start and 0 <= held <= 64
                if 0 <= length <= 64:
                    assert held == length
                if 0 <= starts[b] <= starts[b + 1] <= 10:
                    assert (start, n) == (starts[b], starts[b + 1] - starts[b])
                else:
                    assert n == 0
    host_map.sequence(None, _ints(5, 6, 7), None, 3, 12, 4, 7, 4, 2, out)
    assert tuple(out) == (8, 4, 7)


def test_generator_is_the_published_one(host_map):
    out = (ctypes.c_uint * 4)()
    # the paper's own known answers for philox4x32-10
    for ctr, key, want in (((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
                           ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
                           ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
                            (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1))):
        host_map.words(ctypes.c_ulonglong(key[0] | key[1] << 32), ctypes.c_ulonglong(ctr[2] | ctr[3] << 32),
                       ctypes.c_ulonglong(ctr[0] | ctr[1] << 32), out)
        assert tuple(out) == want


def test_generator_against_python(host_map):
    for seed in ((0, 0), (12345, 7), (-1, -2), (2 ** 63 - 1, -2 ** 63)):
        keep, factor = ref.philox_keeps(seed, 4096, 0.3)
        t = round(0.3 * 65536)
        got = [host_map.keeps(ctypes.c_ulonglong(seed[0] % 2 ** 64), ctypes.c_ulonglong(seed[1] % 2 ** 64), ctypes.c_ulonglong(n), t) for n in range(4096)]
        assert torch.tensor(got).bool().equal(keep)
        assert abs(keep.double().mean().item() - 0.7) < 5 * math.sqrt(0.21 / 4096)
        assert factor == 65536 / (65536 - t)


# -- the references against themselves ----------------------------------------

def test_attention_reference_is_the_gradient():
    torch.manual_seed(0)
    mk = lambda *s: torch.randn(*s, dtype=torch.float64)  # noqa: E731
    first = torch.tensor([[0, 0, 2, 2, 9]])
    q, k, v, do = mk(1, 4, 5, 8), mk(1, 2, 7, 8), mk(1, 2, 7, 8), mk(1, 4, 5, 8)
    mask = ref.seen(5, 7, 3, first)
    leaves = [t.requires_grad_() for t in (q, k, v)]
    s = (q @ k.repeat_interleave(2, 1).mT * 0.3).masked_fill(~mask[:, None], -1e30)
    o = (torch.softmax(s, -1) * mask[:, None]) @ v.repeat_interleave(2, 1)
    want = torch.autograd.grad(o, leaves, do)
    q, k, v = (t.detach() for t in leaves)
    f = ref.attn(q, k, v, 0.3, mask, "fp32")
    assert torch.allclose(f["o"], o.detach(), atol=1e-12)
    got = ref.attn_bwd(q, k, v, f["o"], do, 0.3, mask, "fp32", False)
    for g, n in zip(want, ("dq", "dk", "dv")):
        assert torch.allclose(got[n][0], g, atol=1e-12)
    # and against differences
    for t, n in ((q, "dq"), (k, "dk"), (v, "dv")):
        step = torch.zeros_like(t)
        step[0, 0, 3, 1] = 1e-6
        args = [x + step if x is t else x for x in (q, k, v)], [x - step if x is t else x for x in (q, k, v)]
        hi, lo = ((ref.attn(*a, 0.3, mask, "fp32")["o"] * do).sum() for a in args)
        assert abs((hi - lo) / 2e-6 - got[n][0][0, 0, 3, 1]) < 1e-7


def test_seam_reference_is_the_gradient():
    torch.manual_seed(1)
    mk = lambda *s: torch.randn(*s, dtype=torch.float64)  # noqa: E731
    s, dy, ds, w = mk(2, 3, 16).requires_grad_(), mk(2, 3, 16), mk(2, 3, 16), mk(16).requires_grad_()
    y = ref.seam_norm(s, w, 1e-3)[0]
    gs, gw = torch.autograd.grad((y * dy).sum() + (s * ds).sum(), (s, w))
    got = ref.seam_bwd(s.detach(), dy, ds, w.detach(), 1e-3, None, 1.0)
    assert torch.allclose(got["dres"][0], gs, atol=1e-12) and torch.allclose(got["dw"][0], gw, atol=1e-12)
