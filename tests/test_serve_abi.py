"""Host-side argument checks of rotary positions, eviction, 8-bit caches and
capped, biased or counted scores: errors are found before any launch (no GPU
needed)."""
import ctypes
import os

import pytest
import torch

F32, BF16, E4M3, E2M1, I8 = 0, 1, 2, 3, 4
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4
P = 256


@pytest.fixture(scope="module")
def lib():
    from gqa_kv_cache_gb300 import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from gqa_kv_cache_gb300 import build as b
        b.build()
    return _lib.load()


def _opt(**kw):
    from gqa_kv_cache_gb300 import _lib
    o = _lib.GqaOptions()
    for n, v in kw.items():
        setattr(o, n, v)
    return ctypes.byref(o)


def _rotate(lib, **kw):
    a = dict(q=P, k=P, qo=P, ko=P, dt=BF16, st=(ctypes.c_int64 * 8)(), pos=P, ln=None, cu=None, f=P, il=0, B=0, T=4,
             Hq=4, Hkv=2, D=64, dim=64)
    a.update(kw)
    return lib.gqa_rotate(a["q"], a["k"], a["qo"], a["ko"], a["dt"], a["st"], a["pos"], a["ln"], a["cu"], a["f"], 1.0,
                          a["il"], a["B"], a["T"], a["Hq"], a["Hkv"], a["D"], a["dim"], None, None)


def test_rotate_checks(lib):
    assert _rotate(lib, T=0) == OK
    for bad in (dict(dt=E4M3), dict(T=-1), dict(Hq=0, Hkv=0), dict(Hq=-1), dict(dim=0), dict(dim=3), dict(dim=66),
                dict(D=0), dict(q=None), dict(ko=None), dict(f=None), dict(st=None), dict(q=257), dict(f=260),
                dict(pos=None), dict(pos=None, cu=P, B=1), dict(pos=None, ln=P, B=1), dict(pos=None, cu=P, ln=P, B=-1)):
        assert _rotate(lib, **bad) == INVALID, bad
    assert _rotate(lib, D=1026, dim=64) == UNSUPPORTED
    assert _rotate(lib, Hq=1 << 20) == UNSUPPORTED


def _evict(lib, **kw):
    a = dict(k=P, v=P, w=P, ln=P, sl=None, ids=P, nl=512, ko=None, vo=None, wo=None, os=0, B=2, Hkv=2, D=64, R=2, S=64,
             kv=BF16, n=8, first=1, last=1)
    a.update(kw)
    return lib.gqa_evict(a["k"], a["v"], a["w"], a["ln"], a["sl"], a["ids"], a["nl"], a["ko"], a["vo"], a["wo"], a["os"],
                         a["B"], a["Hkv"], a["D"], a["R"], a["S"], a["kv"], a["n"], a["first"], a["last"], None, None)


def test_evict_checks(lib):
    assert _evict(lib, B=0) == OK
    for bad in (dict(k=None), dict(w=None), dict(ln=None), dict(ids=None), dict(nl=None), dict(nl=P), dict(B=-1),
                dict(Hkv=0), dict(D=0), dict(R=1), dict(S=0), dict(kv=9), dict(kv=-1), dict(n=0), dict(first=-1),
                dict(last=-1), dict(first=5, last=4), dict(k=264), dict(w=258), dict(ko=P), dict(wo=P),
                dict(ko=P, vo=P, os=7), dict(ko=264, vo=P, os=8), dict(ko=P, vo=1 << 20, os=8),
                dict(ko=1 << 20, vo=P + 2 * 2 * 64 * 128 - 16, os=8), dict(ko=1 << 20, vo=1 << 20, os=8),
                dict(ko=1 << 20, vo=1 << 22, wo=P, os=8)):
        assert _evict(lib, **bad) == INVALID, bad
    for bad in (dict(kv=I8), dict(kv=E2M1), dict(D=12), dict(B=1 << 20, Hkv=64, sl=P), dict(kv=E4M3, D=24)):
        assert _evict(lib, **bad) == UNSUPPORTED, bad
    for bad in (dict(table=None), dict(nb=0), dict(bs=0), dict(mb=0), dict(bs=1 << 16, mb=1 << 16)):
        a = dict(table=P, nb=4, bs=16, mb=2)
        a.update(bad)
        assert lib.gqa_evict_paged(P, P, P, a["table"], P, P, 512, None, None, None, 0, 1, 1, 64, a["nb"], a["bs"], a["mb"],
                                   BF16, 4, 0, 1, None, None) == INVALID, bad


def test_append_and_read_of_8_bits(lib):
    def append(kv=I8, box=None, S=64, opt=None, k=P):
        return lib.gqa_append(k, P, BF16, P, P, P, P, None, box, 16, 2, 3, 2, 64, 2, S, kv, None, None, opt)

    good = dict(k_block_scale=P, v_block_scale=P, scale_block=16)
    for bad in (None, _opt(), _opt(**{**good, "k_block_scale": 0}), _opt(**{**good, "v_block_scale": 258}),
                _opt(**{**good, "scale_block": 0}), _opt(**{**good, "scale_block": 24})):
        assert append(opt=bad) == INVALID
    assert append(opt=_opt(**good), box=P) == UNSUPPORTED
    assert append(opt=_opt(**good), k=264) == INVALID
    assert lib.gqa_read(P, P, P, P, None, P, P, BF16, 2, 3, 2, 64, 2, 64, I8, None, None, None) == INVALID
    assert lib.gqa_read_paged(P, P, P, P, P, P, P, BF16, 1, 3, 2, 64, 4, 16, 2, I8, None, None, _opt(k_block_scale=P)) \
        == INVALID


def test_blocks_past_32_bits_are_refused(lib):
    """The appends number a block's groups of 16 elements in 32 bits: larger blocks were written in part."""
    for S, D, want in ((1 << 30, 64, UNSUPPORTED), (1 << 29, 64, UNSUPPORTED), (1 << 28, 128, UNSUPPORTED)):
        big = _opt(k_block_scale=P, v_block_scale=P, scale_block=S, grid_ctas=8)
        assert lib.gqa_append(P, P, BF16, P, P, P, P, None, None, 0, 1, 3, 1, D, 1, S, I8, None, None, big) == want
        assert lib.gqa_append_paged(P, P, BF16, P, P, P, P, P, None, 1, 3, 1, D, 1, S, 1, I8, None, None, big) == want
        assert lib.gqa_decode_step_ex(P, P, P, P, P, P, None, P, 1, 1, 1, D, 1, S, I8, None, 0, None, None, big) == want
        assert lib.gqa_attend(P, BF16, P, P, P, None, P, 1, 1, 1, D, 1, S, I8, None, 0, None, None, big) == WORKSPACE
    heads = 1 << 18                                       # and a token's elements
    wide = _opt(k_block_scale=P, v_block_scale=P, scale_block=1, grid_ctas=8, score_cap=2.0)
    for kv in (I8, BF16):
        assert lib.gqa_decode_step_ex(P, P, P, P, P, P, None, P, 1, heads, heads, 128, 1, 1, kv, None, 0, None, None,
                                      wide) == UNSUPPORTED


def test_sizes_near_the_end_of_32_bits_are_refused(lib):
    """Loops step a few thousand places, and tiles a few hundred slots, behind the last one."""
    for bad in (dict(n=(1 << 30) + 1, last=0), dict(n=2 ** 31 - 1), dict(ko=1 << 20, vo=1 << 60, os=2 ** 31 - 1),
                dict(ko=1 << 20, vo=1 << 60, os=(1 << 30) + 1)):
        assert _evict(lib, **bad) == UNSUPPORTED, bad
        assert lib.gqa_evict_paged(P, P, P, P, P, P, 512, bad.get("ko"), bad.get("vo"), None, bad.get("os", 0), 1, 1, 64, 4, 16,
                                   2, BF16, bad.get("n", 8), 0, 0, None, None) == UNSUPPORTED
    block = dict(k_block_scale=P, v_block_scale=P)
    for blocks in (2 ** 31 // 16 - 1, 2 ** 31 // 16 - 64):
        for kv, opt in ((I8, _opt(grid_ctas=8, **block)), (BF16, _opt(grid_ctas=8, score_cap=2.0))):
            assert lib.gqa_attend_paged(P, BF16, P, P, P, P, P, 1, 8, 2, 128, 64, 16, blocks, kv, None, 0, None, None,
                                        opt) == UNSUPPORTED
            assert lib.gqa_attend_paged(P, BF16, P, P, P, P, P, 1, 8, 2, 128, 64, 16, blocks // 2, kv, None, 0, None, None,
                                        opt) == WORKSPACE


def _attend(lib, kv=BF16, D=128, Hq=8, Hkv=2, S=64, dt=BF16, **opt):
    opt.setdefault("grid_ctas", 8)
    return lib.gqa_attend(P, dt, P, P, P, None, P, 1, Hq, Hkv, D, 1, S, kv, None, 0, None, None, _opt(**opt))


def test_attend_checks(lib):
    good = dict(k_block_scale=P, v_block_scale=P, scale_block=16)
    assert _attend(lib, I8, **good) == WORKSPACE and _attend(lib, score_cap=30.0) == WORKSPACE
    assert _attend(lib, head_slopes=P) == WORKSPACE and _attend(lib, I8, **good, kernel=2) == WORKSPACE
    for bad in (dict(), dict(k_block_scale=P), {**good, "scale_block": 0}, {**good, "scale_block": 48},
                {**good, "score_cap": -1.0}):
        assert _attend(lib, I8, **bad) == INVALID, bad
    for bad in (dict(score_cap=-1.0), dict(score_cap=float("nan")), dict(score_cap=float("inf")), dict(score_cap=2.0 ** 61),
                dict(score_cap=2.0 ** -61), dict(head_slopes=258),
                dict(weights=258)):
        assert _attend(lib, **bad) == INVALID, bad
    for bad in (dict(kv=F32), dict(D=32), dict(Hq=18), dict(kernel=1), dict(kernel=3), dict(kernel=4)):
        assert _attend(lib, score_cap=30.0, **bad) == UNSUPPORTED, bad
    for bad in (dict(D=96), dict(Hq=18), dict(kernel=1)):
        assert _attend(lib, I8, **good, **bad) == UNSUPPORTED, bad
    # counted weights without their scratch
    n = lib.gqa_weights_scratch_bytes(1, 8, 2, 64)
    assert n > 0
    for bad in (dict(), dict(weights_scratch=P, weights_scratch_bytes=n - 1), dict(weights_scratch=264, weights_scratch_bytes=n)):
        assert _attend(lib, weights=P, **bad) == WORKSPACE, bad
    assert lib.gqa_weights_scratch_bytes(1, 8, 3, 64) == 0 and lib.gqa_weights_scratch_bytes(1, 8, 2, 0) == 0


def test_steps_that_take_neither(lib):
    good = dict(k_block_scale=P, v_block_scale=P, scale_block=16, grid_ctas=8)
    assert lib.gqa_decode_multi(P, P, P, P, P, P, P, None, P, 1, 2, 2, 8, 2, 128, 1, 64, I8, None, 0, None, None,
                                _opt(**good)) == UNSUPPORTED
    assert lib.gqa_decode_multi(P, P, P, P, P, P, P, None, P, 1, 2, 2, 8, 2, 128, 1, 64, BF16, None, 0, None, None,
                                _opt(score_cap=2.0, grid_ctas=8)) == UNSUPPORTED
    assert lib.gqa_workspace_bytes_multi(1, 8, 2, 128, I8, 2, _opt(**good)) == 0
    for bad in (dict(score_cap=2.0), dict(head_slopes=P), dict(weights=P)):
        assert lib.gqa_attend_selected(P, BF16, P, P, P, P, P, 1, 4, 2, 128, 64, 16, 4, BF16, None, 0, None, None,
                                       _opt(**bad)) == INVALID
    assert lib.gqa_attend_selected(P, BF16, P, P, P, P, P, 1, 4, 2, 128, 64, 16, 4, I8, None, 0, None, None,
                                   _opt(**good)) == UNSUPPORTED


def test_rotary_tables_on_the_host():
    import math

    import gqa_kv_cache_gb300 as gqa
    import serve_reference as R
    for scaling in (None, dict(kind="linear", factor=3.0), dict(kind="ntk", factor=8.0),
                    dict(kind="bands", factor=8.0, original=4096, low=1.0, high=32.0)):
        rot = gqa.Rotary(64, base=10000.0, scaling=scaling, device="cpu")
        f, _ = R.frequencies(64, 10000.0, scaling)
        got = torch.tensor([(int(x) % 2 ** 64) / 2 ** 64 for x in rot.freqs], dtype=torch.float64) * 2 * math.pi
        # both are 64-bit floats of a power: a few steps of 2^-52, and 2^-64 turns of fixed point
        assert ((got - f).abs() <= 1e-14 * f + 2.0 ** -60).all()
    for bad in (dict(dim=0), dict(dim=3), dict(dim=64, layout="x"), dict(dim=64, base=0.0),
                dict(dim=64, scaling=dict(kind="x")), dict(dim=64, scaling=dict(kind="linear")),
                dict(dim=64, scaling=dict(kind="linear", factor=-1.0)), dict(dim=2, scaling=dict(kind="ntk", factor=2.0)),
                dict(dim=64, scaling=dict(kind="linear", factor=2.0, low=1.0)),
                dict(dim=64, scaling=dict(kind="bands", factor=2.0, original=64, low=4.0, high=4.0))):
        with pytest.raises(ValueError):
            gqa.Rotary(bad.pop("dim"), device="cpu", **bad)


def test_threads_have_scratch_of_their_own(monkeypatch):
    """A counted call's kernels hand scores on through the scratch: two threads on one stream must not share it."""
    import threading

    import gqa_kv_cache_gb300 as gqa
    monkeypatch.setattr(gqa, "_stream", lambda stream, device=None: 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    device, got, meet = torch.device("cpu"), [], threading.Barrier(2)

    def call():
        got.append((gqa._scratch(device, 1000), gqa._scratch(device, 2000)))
        meet.wait(30)                    # this call is still under way when the other thread's begins

    first, second = (threading.Thread(target=call) for _ in range(2))
    first.start()
    while not got and first.is_alive():
        pass
    second.start()
    first.join()
    second.join()
    (a, b), (c, d) = got
    assert a is b and c is d and a.data_ptr() != c.data_ptr()


def _exact_turns(dim, base, scaling):
    """Frequencies over 2 pi, times 2^64, in decimal: powers by exp and ln, pi by Machin's formula."""
    from decimal import Decimal as Dec

    def atan_of(n):                      # atan(1 / n)
        x, k, total = Dec(1) / n, 0, Dec(0)
        while abs(x) > Dec(10) ** -118:
            total += (-1) ** k * x / (2 * k + 1)
            x, k = x / (n * n), k + 1
        return total

    two_pi = 2 * (16 * atan_of(5) - 4 * atan_of(239))
    k = {n: Dec(v) for n, v in (scaling or {}).items() if n != "kind"}
    kind = (scaling or {}).get("kind")
    ln = Dec(base).ln() + (k["factor"].ln() * dim / (dim - 2) if kind == "ntk" else 0)
    out = []
    for i in range(dim // 2):
        f = (-2 * i * ln / dim).exp()
        if kind == "linear":
            f /= k["factor"]
        if kind == "bands":
            u = (k["original"] * f / two_pi - k["low"]) / (k["high"] - k["low"])
            u = min(max(u, Dec(0)), Dec(1))
            f = f * u + f * (1 - u) / k["factor"]
        out.append(f / two_pi % 1 * 2 ** 64)
    return out


@pytest.mark.parametrize("base", [10000.0, 500000.0, 1e6, 0.5])
@pytest.mark.parametrize("scaling", [None, dict(kind="linear", factor=0.05), dict(kind="linear", factor=3.0),
                                     dict(kind="ntk", factor=8.0),
                                     dict(kind="bands", factor=8.0, original=4096, low=1.0, high=32.0)])
def test_rotary_tables_are_rounded_once(base, scaling):
    """An angle is a position times the table's entry: an entry from a 64-bit float would be 2^-56 of a turn off,
    2^-25 at far positions."""
    import decimal

    import gqa_kv_cache_gb300 as gqa
    for dim in (4, 64, 104, 128):
        rot = gqa.Rotary(dim, base=base, scaling=scaling, device="cpu")
        with decimal.localcontext() as c:
            c.prec = 120
            for got, want in zip(rot.freqs.tolist(), _exact_turns(dim, base, scaling)):
                off = (got - want) % 2 ** 64
                assert min(off, 2 ** 64 - off) <= decimal.Decimal("0.5000001")


def test_rotary_takes_any_size_of_scaling():
    import gqa_kv_cache_gb300 as gqa
    rot = gqa.Rotary(4, scaling=dict(kind="ntk", factor=1e300), device="cpu")   # a base of 10^604
    assert rot.freqs.tolist()[1] == 0
    with pytest.raises(ValueError):
        gqa.Rotary(4, scaling=dict(kind="linear", factor=1e-300), device="cpu")
