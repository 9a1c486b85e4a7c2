"""Host-side argument checks of append, read, block selection and the attend
over selected blocks, and of E2M1 caches in the decode calls: errors are found
before any launch (no GPU needed)."""
import ctypes
import os

import pytest

F32, BF16, E4M3, E2M1 = 0, 1, 2, 3
OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    from gqa_kv_cache_gb300 import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from gqa_kv_cache_gb300 import build as b
        b.build()
    return _lib.load()


def _opt(scales=True, groups=True, **kw):
    from gqa_kv_cache_gb300 import _lib
    o = _lib.GqaOptions()
    if scales:
        o.k_scale = o.v_scale = 256
    if groups:
        o.k_group_scale = o.v_group_scale = 512
    for n, v in kw.items():
        setattr(o, n, v)
    return ctypes.byref(o)


def _append(lib, **kw):
    a = dict(k=256, v=256, dt=BF16, kc=256, vc=256, ln=256, cu=256, sl=None, box=None, bb=0, B=2, T=3, Hkv=2, D=64,
             R=2, Smax=64, kv=E2M1, opt=_opt())
    a.update(kw)
    return lib.gqa_append(a["k"], a["v"], a["dt"], a["kc"], a["vc"], a["ln"], a["cu"], a["sl"], a["box"], a["bb"],
                          a["B"], a["T"], a["Hkv"], a["D"], a["R"], a["Smax"], a["kv"], None, None, a["opt"])


def test_append_checks(lib):
    assert _append(lib, B=0) == OK and _append(lib, T=0) == OK
    for bad in (dict(k=None), dict(vc=None), dict(ln=None), dict(cu=None), dict(dt=E4M3), dict(kv=9), dict(kv=-1),
                dict(Hkv=0), dict(D=0), dict(Smax=0), dict(R=1), dict(T=-1), dict(opt=None), dict(k=264),
                dict(opt=_opt(scales=False)), dict(opt=_opt(groups=False)), dict(opt=_opt(k_group_scale=520)),
                dict(box=256, bb=0), dict(box=256, bb=7), dict(box=260, bb=16)):
        assert _append(lib, **bad) == INVALID, bad
    assert _append(lib, D=24) == UNSUPPORTED
    assert _append(lib, Smax=4096, box=256, bb=2048) == UNSUPPORTED


def test_read_checks(lib):
    def call(**kw):
        a = dict(kc=256, ln=256, cu=256, sl=None, ko=256, vo=256, dt=F32, B=1, T=4, Hkv=1, D=32, R=1, Smax=8, kv=E4M3,
                 opt=_opt(groups=False))
        a.update(kw)
        return lib.gqa_read(a["kc"], 256, a["ln"], a["cu"], a["sl"], a["ko"], a["vo"], a["dt"], a["B"], a["T"],
                            a["Hkv"], a["D"], a["R"], a["Smax"], a["kv"], None, None, a["opt"])
    assert call(B=0) == OK
    for bad in (dict(kc=None), dict(ko=None), dict(vo=8), dict(dt=E2M1), dict(kv=E2M1), dict(opt=None), dict(R=0)):
        assert call(**bad) == INVALID, bad


def test_paged_checks(lib):
    def rows(fn, table=256, nb=4, bs=16, mb=2, B=1):
        if fn == "append":
            return lib.gqa_append_paged(256, 256, BF16, 256, 256, table, 256, 256, None, B, 2, 1, 64, nb, bs, mb, BF16,
                                        None, None, None)
        return lib.gqa_read_paged(256, 256, table, 256, 256, 256, 256, BF16, B, 2, 1, 64, nb, bs, mb, BF16, None, None,
                                  None)
    for fn in ("append", "read"):
        assert rows(fn, B=0) == OK
        for bad in (dict(table=None), dict(nb=0), dict(bs=0), dict(mb=0), dict(bs=1 << 16, mb=1 << 16)):
            assert rows(fn, **bad) == INVALID, (fn, bad)


def _select(lib, **kw):
    a = dict(q=256, dt=BF16, box=256, ln=256, ids=256, B=1, Hq=4, Hkv=2, D=128, R=1, NB=8, bs=16, n=4, first=1, last=1)
    a.update(kw)
    return lib.gqa_select_blocks(a["q"], a["dt"], a["box"], a["ln"], None, a["ids"], 256, 256, a["B"], a["Hq"],
                                 a["Hkv"], a["D"], a["R"], a["NB"], a["bs"], a["n"], a["first"], a["last"], None, None)


def test_select_checks(lib):
    assert _select(lib, B=0) == OK
    for bad in (dict(q=None), dict(box=None), dict(ids=None), dict(ln=None), dict(dt=E4M3), dict(Hq=5), dict(NB=0),
                dict(bs=0), dict(n=0), dict(first=-1), dict(last=0), dict(first=3, last=2), dict(R=0), dict(q=264),
                dict(NB=1 << 16, bs=1 << 16)):
        assert _select(lib, **bad) == INVALID, bad
    for bad in (dict(D=96), dict(NB=16385), dict(R=1 << 20, NB=4096), dict(n=1 << 28)):
        assert _select(lib, **bad) == UNSUPPORTED, bad
    assert lib.gqa_select_blocks_paged(256, BF16, 256, None, 256, 256, 256, 256, 1, 4, 2, 128, 64, 16, 8, 4, 1, 1,
                                       None, None) == INVALID
    assert lib.gqa_select_blocks_paged(256, BF16, 256, 256, 256, 256, 256, 256, 1, 4, 2, 128, 0, 16, 8, 4, 1, 1,
                                       None, None) == INVALID


def _selected(lib, **kw):
    a = dict(q=256, dt=BF16, kc=256, tb=256, sl=256, out=256, B=1, Hq=4, Hkv=2, D=128, pool=64, bs=16, n=4, kv=BF16,
             opt=_opt(grid_ctas=8))
    a.update(kw)
    return lib.gqa_attend_selected(a["q"], a["dt"], a["kc"], 256, a["tb"], a["sl"], a["out"], a["B"], a["Hq"],
                                   a["Hkv"], a["D"], a["pool"], a["bs"], a["n"], a["kv"], None, 0, None, None, a["opt"])


def test_attend_selected_checks(lib):
    assert _selected(lib, B=0) == OK
    for bad in (dict(q=None), dict(tb=None), dict(sl=None), dict(out=None), dict(Hq=5), dict(Hkv=0), dict(pool=0),
                dict(bs=0), dict(n=0), dict(opt=_opt(window=4)), dict(opt=_opt(kept_prefix=1)),
                dict(opt=_opt(head_sink=256)), dict(opt=_opt(kept_prefix_rows=256)), dict(kv=E2M1, opt=None),
                dict(kv=7)):
        assert _selected(lib, **bad) == INVALID, bad
    for bad in (dict(kv=E4M3), dict(kv=E2M1, D=32), dict(kv=E2M1, Hq=18)):
        assert _selected(lib, **bad) == UNSUPPORTED, bad
    assert _selected(lib, kv=E2M1) == 4                   # no workspace


def test_e2m1_in_the_decode_calls(lib):
    P = 256

    def attend(opt, D=128, Hq=8, q=BF16, R=1, Smax=64, kernel_D=None):
        return lib.gqa_attend(P, q, P, P, P, None, P, 1, Hq, 2, D, R, Smax, E2M1, None, 0, None, None, opt)
    assert attend(None) == INVALID
    assert attend(_opt(groups=False, grid_ctas=8)) == INVALID
    assert attend(_opt(scales=False, grid_ctas=8)) == INVALID
    assert attend(_opt(v_group_scale=264, grid_ctas=8)) == INVALID
    assert attend(_opt(grid_ctas=8)) == 4 and attend(_opt(grid_ctas=8), q=F32, D=64) == 4      # no workspace
    for kernel in (1, 3, 4):
        assert attend(_opt(kernel=kernel, grid_ctas=8)) == UNSUPPORTED
    assert attend(_opt(grid_ctas=8), D=256) == UNSUPPORTED
    assert attend(_opt(grid_ctas=8), Hq=18) == UNSUPPORTED
    assert attend(_opt(grid_ctas=8), R=1 << 12, Smax=1 << 20) == UNSUPPORTED                   # 2^33 vectors
    assert lib.gqa_decode_multi(P, P, P, P, P, P, P, None, P, 1, 1, 1, 8, 2, 128, 1, 64, E2M1, None, 0, None, None,
                                _opt(grid_ctas=8)) == UNSUPPORTED
    o = _opt(grid_ctas=8)
    assert lib.gqa_workspace_bytes(4, 8, 2, 128, E2M1, o) > 0
    assert lib.gqa_workspace_bytes(4, 8, 2, 32, E2M1, o) == 0
    assert lib.gqa_workspace_bytes_multi(4, 8, 2, 128, E2M1, 2, o) == 0
    assert lib.gqa_decode_step_noalloc(P, P, P, P, P, P, None, P, 1, 8, 2, 128, 1, 64, E2M1, None, None) != OK


def test_binding_refuses_host_tensors():
    import torch

    import gqa_kv_cache_gb300 as gqa
    x = torch.zeros(1, 1, 64)
    c = torch.zeros(1, 1, 4, 64)
    n = torch.zeros(1, dtype=torch.int32)
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        gqa.append(x, x, c, c, n, cu)
    with pytest.raises(ValueError):
        gqa.read(c, c, n, cu, 1)
    with pytest.raises(ValueError):
        gqa.select_blocks(x, torch.zeros(1, 1, 1, 2, 64, dtype=torch.bfloat16), n, 2, block_size=4)


def test_capture_id_checks(lib):
    assert lib.gqa_stream_capture_id(None, None) == INVALID
