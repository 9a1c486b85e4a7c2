"""Attention over a 4-bit (E2M1) cache against the 64-bit definition: head
layouts, widths, lengths from one slot, odd capacities, every addressing and
page size, modifiers, cut units, bad content, graphs and streams."""
import math

import pytest
import torch

from cache_reference import Problem, attend_tolerance, quantise_e2m1, values_e2m1

pytestmark = pytest.mark.gpu


def _gpu(p):
    d = dict(q=p.q, lengths=p.lengths, k=p.kv[0], v=p.kv[1], kg=p.groups[0], vg=p.groups[1], ks=p.g[0], vs=p.g[1])
    if p.table is not None:
        d["table"] = p.table
    if p.slots is not None:
        d["slots"] = p.slots
    return {n: t.contiguous().cuda() for n, t in d.items()}


def _scales(t):
    return dict(k_scale=t["ks"], v_scale=t["vs"], k_group_scale=t["kg"], v_group_scale=t["vg"])


def _attend(p, t, **kw):
    import gqa_kv_cache_gb300 as gqa
    if p.table is not None:
        return gqa.attend_paged(t["q"], t["k"], t["v"], t["table"], t["lengths"], **_scales(t), **kw)
    return gqa.attend(t["q"], t["k"], t["v"], t["lengths"], t.get("slots"), **_scales(t), **kw)


def _decode(p, t, kn, vn, **kw):
    import gqa_kv_cache_gb300 as gqa
    if p.table is not None:
        return gqa.decode_step_paged(t["q"], kn, vn, t["k"], t["v"], t["table"], t["lengths"], **_scales(t), **kw)
    return gqa.decode_step(t["q"], kn, vn, t["k"], t["v"], t["lengths"], t.get("slots"), **_scales(t), **kw)


def _check(p, got, slots=None, sink=None, rows=None):
    got = got.double().cpu()
    for b in range(p.B) if rows is None else rows:
        want, vmax, amax = p.expect(b, None if slots is None else slots[b], sink)
        err = float((got[b] - want).abs().max())
        assert err <= attend_tolerance(p.D, vmax, amax), (b, p.lens[b], err)


LENS = [1, 2, 15, 16, 17, 31, 127, 128, 129, 300, 511]


@pytest.mark.parametrize("q_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 2), (128, 5, 5), (64, 16, 2), (64, 3, 1), (128, 14, 2)])
@pytest.mark.parametrize("layout", ["dense", "slots", "paged"])
def test_attend(layout, D, Hq, Hkv, q_dtype):
    p = Problem("e2m1", layout, LENS, Hq, Hkv, D, 513 if layout != "paged" else 512, q_dtype=q_dtype, seed=D + Hq)
    t = _gpu(p)
    keep = {n: x.clone() for n, x in t.items()}
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    _check(p, _attend(p, t, status=st))               # one CTA a unit
    _check(p, _attend(p, t, status=st, grid_ctas=11))  # units cut by CTAs
    assert int(st) == 0
    for n in keep:
        assert torch.equal(keep[n], t[n]), f"{n} written by a read-only attend"


@pytest.mark.parametrize("grid", [1, 3, 40, 500])
def test_cut_units(grid):
    """Units shared by few and by many CTAs, and merged past one pass."""
    p = Problem("e2m1", "dense", [4100, 1, 700], 4, 1, 128, 4101, seed=3)
    t = _gpu(p)
    _check(p, _attend(p, t, grid_ctas=grid))
    p = Problem("e2m1", "paged", [4100, 60, 700], 8, 1, 64, 4112, seed=4, q_dtype=torch.float32)
    t = _gpu(p)
    _check(p, _attend(p, t, grid_ctas=grid))


@pytest.mark.parametrize("bs", [1, 5, 8, 16, 24, 32, 128, 256])
def test_page_sizes(bs):
    p = Problem("e2m1", "paged", [1, 7, 8, 200, 255, 256], 6, 2, 128, 512, bs=bs, seed=bs)
    t = _gpu(p)
    _check(p, _attend(p, t))
    _check(p, _attend(p, t, grid_ctas=5))


@pytest.mark.parametrize("grid", [0, 6])
@pytest.mark.parametrize("layout", ["dense", "slots", "paged"])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_step_appends(layout, D, grid):
    """The appended token's bytes are the format's, and it is attended as stored."""
    lens = [0, 1, 15, 16, 127, 128, 300]
    p = Problem("e2m1", layout, lens, 8, 2, D, 320, seed=9, extra=1)
    gen = torch.Generator().manual_seed(1)
    kn, vn = (torch.randn(p.B, 2, D, generator=gen).bfloat16() for _ in range(2))
    t = _gpu(p)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = _decode(p, t, kn.cuda(), vn.cuda(), status=st, grid_ctas=grid).double().cpu()
    assert int(st) == 0
    for i, x in enumerate((kn, vn)):
        c, s, _, _ = quantise_e2m1(x, p.g[i].view(-1, 1))
        for b, n in enumerate(lens):
            at = (int(p.table[b, n // p.bs]), slice(None), n % p.bs) if layout == "paged" else \
                (int(p.slots[b]) if p.slots is not None else b, slice(None), n)
            p.kv[i][at], p.groups[i][at] = c[b], s[b]
    assert torch.equal(t["k"].cpu(), p.kv[0]) and torch.equal(t["v"].cpu(), p.kv[1])
    assert torch.equal(t["kg"].cpu(), p.groups[0]) and torch.equal(t["vg"].cpu(), p.groups[1])
    p.lens = [n + 1 for n in lens]
    _check(p, got)


def test_window_prefix_and_sink():
    p = Problem("e2m1", "dense", [5, 100, 400, 900], 8, 2, 128, 901, seed=11)
    t = _gpu(p)
    sink = torch.randn(8, generator=torch.Generator().manual_seed(2))
    for window, prefix in ((1, 0), (60, 0), (130, 37), (40, 300), (2000, 4)):
        slots = [[[j for j in range(n) if j > n - 1 - window or j < prefix]] * 2 for n in p.lens]
        for grid in (0, 13):
            _check(p, _attend(p, t, window=window, kept_prefix=prefix, sink=sink.cuda(), grid_ctas=grid), slots, sink)
    pp = Problem("e2m1", "paged", [5, 100, 400, 900], 8, 2, 64, 912, seed=12)
    tt = _gpu(pp)
    slots = [[[j for j in range(n) if j > n - 1 - 100 or j < 20]] * 2 for n in pp.lens]
    _check(pp, _attend(pp, tt, window=100, kept_prefix=20), slots)


def test_slots_outside_the_softmax_never_matter():
    """Stale slots and slots between prefix and window hold NaN scales."""
    p = Problem("e2m1", "dense", [33, 200, 641], 4, 1, 128, 650, seed=5)
    t = _gpu(p)
    for window, prefix in ((0, 0), (100, 10)):
        a = _attend(p, t, window=window, kept_prefix=prefix)
        u = {n: x.clone() for n, x in t.items()}
        for b, n in enumerate(p.lens):
            dead = [j for j in range(p.Smax) if j >= n or (window and prefix <= j <= n - 1 - window)]
            for name in ("kg", "vg"):
                u[name][b, :, dead] = 0x7F
        assert torch.equal(a, _attend(p, u, window=window, kept_prefix=prefix))


def test_nan_in_a_valid_slot_reaches_its_row_alone():
    p = Problem("e2m1", "dense", [50, 300], 4, 2, 128, 301, seed=6)
    for where in ("kg", "vg"):
        t = _gpu(p)
        t[where][1, 1, 7, 2] = 0x7F
        out = _attend(p, t).cpu()
        _check(p, out, rows=[0])
        want, vmax, amax = p.expect(1)
        assert (out[1, :2].double() - want[:2]).abs().max() <= attend_tolerance(128, vmax, amax)
        if where == "kg":
            assert torch.isnan(out[1, 2:]).all()
        else:
            assert torch.isnan(out[1, 2:, 32:48]).all() and torch.isfinite(out[1, 2:, :32]).all()


def test_wide_range_of_queries_and_scores():
    """Queries far outside f16's range and scores that rise along the row."""
    p = Problem("e2m1", "dense", [700, 513], 4, 1, 128, 700, seed=7)
    p.q = (p.q.float() * torch.tensor([1e-6, 1.0, 300.0, 2e5])[None, :, None]).bfloat16()
    _check(p, _attend(p, _gpu(p)))
    p = Problem("e2m1", "dense", [1024], 2, 1, 64, 1024, seed=8, q_dtype=torch.float32)
    p.q.fill_(3.0)
    ramp = torch.arange(1024).float()[None, None, :, None] / 40 + torch.zeros(1, 1, 1024, 64)
    p.kv[0], p.groups[0], _, _ = quantise_e2m1(ramp, p.g[0].view(-1, 1, 1))
    _check(p, _attend(p, _gpu(p)))


def test_bad_content():
    """Bad rows give NaN and their status bit, the others are right; nothing else is written."""
    p = Problem("e2m1", "paged", [40, 300, 20, 100], 4, 2, 128, 320, seed=13, extra=1)
    t = _gpu(p)
    t["lengths"][2] = 0
    t["table"][1, 3] = -1
    t["table"][3, 2] = 10 ** 6
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = _attend(p, t, status=st).cpu()
    assert int(st) == 1 | 4
    assert torch.isnan(out[1:]).all()
    _check(p, out, rows=[0])
    p = Problem("e2m1", "slots", [40, 300, 20], 4, 2, 128, 320, seed=14)
    t = _gpu(p)
    t["lengths"][0] = 321
    t["slots"][1] = p.B + 4
    st.zero_()
    out = _attend(p, t, status=st).cpu()
    assert int(st) == 1 | 2 and torch.isnan(out[:2]).all()
    _check(p, out, rows=[2])
    # a decode step whose append slot cannot be addressed writes nothing
    keep = t["k"].clone(), t["kg"].clone()
    new = torch.ones(3, 2, 128, dtype=torch.bfloat16, device="cuda")
    t["lengths"][:] = torch.tensor([320, 10, -1], dtype=torch.int32)
    out = _decode(p, t, new, new, status=st)
    assert torch.isnan(out).all() and torch.equal(keep[0], t["k"]) and torch.equal(keep[1], t["kg"])


def test_offsets_past_32_bits():
    """The last row of a cache of more than 2^32 bytes of codes."""
    R, Hkv, Smax, D = 9, 8, 1 << 20, 128
    p = Problem("e2m1", "dense", [777], 8, 8, D, 1024, seed=15)
    big = [torch.empty(R, Hkv, Smax, n, dtype=torch.uint8, device="cuda") for n in (64, 64, 8, 8)]
    assert big[0].numel() > 2 ** 32
    for x, y in zip(big, (*p.kv, *p.groups)):
        x[R - 1, :, Smax - 1024:].fill_(0)
        x[R - 1, :, :1024] = y[0].cuda()
    t = _gpu(p)
    t["k"], t["v"], t["kg"], t["vg"] = big
    t["slots"] = torch.tensor([R - 1], dtype=torch.int32, device="cuda")
    _check(p, _attend(p, t))
    new = torch.randn(1, Hkv, D, dtype=torch.bfloat16, device="cuda")
    t["lengths"] = torch.tensor([Smax - 1], dtype=torch.int32, device="cuda")
    _decode(p, t, new, new, window=8)
    c, s, _, _ = quantise_e2m1(new.cpu()[0], p.g[0].view(-1, 1))
    assert torch.equal(big[0][R - 1, :, Smax - 1].cpu(), c) and torch.equal(big[2][R - 1, :, Smax - 1].cpu(), s)


def test_graphs_and_streams():
    """Two captured steps replayed side by side, and a call on a stream of its own, give the eager bits."""
    ps = [Problem("e2m1", "dense", [3000 + 13 * i, 50, 2000], 8, 2, 128, 3100, seed=20 + i) for i in range(2)]
    ts = [_gpu(p) for p in ps]
    want = [_attend(p, t) for p, t in zip(ps, ts)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = _attend(ps[0], ts[0], stream=side)
    side.synchronize()
    assert torch.equal(other, want[0])
    graphs, outs = [], []
    for p, t in zip(ps, ts):
        out = torch.empty_like(want[0])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _attend(p, t, out=out)
        graphs.append(g)
        outs.append(out)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for o in outs:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)


def test_output_of_a_stream_is_its_own_memory():
    """What the current stream just freed may still be read there: the output of a
    call on another stream comes from that stream's memory."""
    p = Problem("e2m1", "dense", [100, 20], 8, 2, 128, 112, seed=22)
    t, side = _gpu(p), torch.cuda.Stream()
    freed = [torch.empty(2, 8, 128, device="cuda") for _ in range(4)]
    at = {x.data_ptr() for x in freed}
    torch.cuda.synchronize()
    del freed
    out = _attend(p, t, stream=side)
    side.synchronize()
    assert out.data_ptr() not in at
    _check(p, out)


def test_same_bits_twice_and_empty_batch():
    import gqa_kv_cache_gb300 as gqa
    p = Problem("e2m1", "paged", [900, 64, 333], 8, 1, 128, 912, seed=30)
    t = _gpu(p)
    assert torch.equal(_attend(p, t), _attend(p, t))
    e = gqa.attend(t["q"][:0], torch.empty(0, 1, 16, 64, dtype=torch.uint8, device="cuda"),
                   torch.empty(0, 1, 16, 64, dtype=torch.uint8, device="cuda"), t["lengths"][:0],
                   k_scale=t["ks"], v_scale=t["vs"],
                   k_group_scale=torch.empty(0, 1, 16, 8, dtype=torch.uint8, device="cuda"),
                   v_group_scale=torch.empty(0, 1, 16, 8, dtype=torch.uint8, device="cuda"))
    assert e.shape == (0, 8, 128)


def test_typed_caches():
    """The cache under torch's own 4-bit and 8-bit types gives the same bits."""
    p = Problem("e2m1", "dense", [100, 33], 4, 2, 64, 128, seed=40)
    t = _gpu(p)
    want = _attend(p, t)
    u = {**t, "kg": t["kg"].view(torch.float8_e4m3fn), "vg": t["vg"].view(torch.float8_e4m3fn)}
    if hasattr(torch, "float4_e2m1fn_x2"):
        u.update(k=t["k"].view(torch.float4_e2m1fn_x2), v=t["v"].view(torch.float4_e2m1fn_x2))
    assert torch.equal(_attend(p, u), want)


def test_many_short_rows():
    """More units than CTAs, most of one tile; a few units a CTA in the copies at once."""
    lens = [1 + (37 * i) % 150 for i in range(700)]
    for D, q in ((128, torch.bfloat16), (64, torch.float32)):
        p = Problem("e2m1", "slots", lens, 4, 2, D, 151, seed=41, q_dtype=q)
        t = _gpu(p)
        _check(p, _attend(p, t), rows=range(0, 700, 7))
        _check(p, _attend(p, t, grid_ctas=300), rows=range(0, 700, 7))


FORMS = [(1, 128, torch.bfloat16), (2, 64, torch.float32), (4, 128, torch.float32), (5, 128, torch.bfloat16),
         (8, 64, torch.bfloat16), (8, 128, torch.float32)]


@pytest.mark.parametrize("G,D,q", FORMS)
def test_modifiers_in_both_forms(G, D, q):
    """Windows, prefixes, sinks and stale NaN for up to four query rows a head and for more."""
    p = Problem("e2m1", "paged", [5, 100, 641, 900], 2 * G, 2, D, 960, bs=24, seed=50 + G, q_dtype=q)
    t = _gpu(p)
    sink = torch.randn(2 * G, generator=torch.Generator().manual_seed(G))
    for window, prefix, grid in ((1, 0, 0), (130, 37, 13), (40, 300, 7)):
        slots = [[[j for j in range(n) if j > n - 1 - window or j < prefix]] * 2 for n in p.lens]
        kw = dict(window=window, kept_prefix=prefix, sink=sink.cuda(), grid_ctas=grid)
        a = _attend(p, t, **kw)
        _check(p, a, slots, sink)
        u = {n: x.clone() for n, x in t.items()}
        for b, n in enumerate(p.lens):
            for j in range(-(-n // p.bs) * p.bs):
                if j >= n or (prefix <= j <= n - 1 - window):
                    for name in ("kg", "vg"):
                        u[name][int(p.table[b, j // p.bs]), :, j % p.bs] = 0x7F
        assert torch.equal(a, _attend(p, u, **kw))


@pytest.mark.parametrize("G,D,q", FORMS)
def test_nan_and_range_in_both_forms(G, D, q):
    p = Problem("e2m1", "dense", [50, 300, 513], 2 * G, 2, D, 513, seed=60 + G, q_dtype=q)
    # rows of very different size in one product
    p.q = (p.q.float() * torch.logspace(-6, 4, 2 * G)[None, :, None]).to(q)
    t = _gpu(p)
    _check(p, _attend(p, t))
    for where in ("kg", "vg"):
        u = {n: x.clone() for n, x in t.items()}
        u[where][1, 1, 7, 2] = 0x7F
        for grid in (0, 3):
            out = _attend(p, u, grid_ctas=grid).cpu()
            _check(p, out, rows=[0, 2])
            want, vmax, amax = p.expect(1)
            assert (out[1, :G].double() - want[:G]).abs().max() <= attend_tolerance(D, vmax, amax)
            bad = torch.isnan(out[1, G:])
            assert bad.all() if where == "kg" else bad[:, 32:48].all() and not bad[:, :32].any() and not bad[:, 48:].any()


@pytest.mark.parametrize("grid", [0, 5])
@pytest.mark.parametrize("G,D", [(1, 128), (3, 64), (4, 128), (6, 128), (8, 64)])
def test_decode_step_in_both_forms(G, D, grid):
    """The appended token is attended as stored, alone and with others, in whole and cut units."""
    lens = [0, 15, 127, 700]
    p = Problem("e2m1", "slots", lens, 2 * G, 2, D, 701, seed=70 + G)
    gen = torch.Generator().manual_seed(G)
    kn, vn = (torch.randn(p.B, 2, D, generator=gen).bfloat16() for _ in range(2))
    t = _gpu(p)
    got = _decode(p, t, kn.cuda(), vn.cuda(), grid_ctas=grid)
    for i, x in enumerate((kn, vn)):
        c, s, _, _ = quantise_e2m1(x, p.g[i].view(-1, 1))
        for b, n in enumerate(lens):
            p.kv[i][int(p.slots[b]), :, n], p.groups[i][int(p.slots[b]), :, n] = c[b], s[b]
    assert torch.equal(t["k"].cpu(), p.kv[0]) and torch.equal(t["vg"].cpu(), p.groups[1])
    p.lens = [n + 1 for n in lens]
    _check(p, got)


def test_refusals():
    import gqa_kv_cache_gb300 as gqa
    p = Problem("e2m1", "dense", [5], 8, 2, 128, 16, seed=31)
    t = _gpu(p)
    bf = torch.zeros(1, 2, 128, dtype=torch.bfloat16, device="cuda")
    for kernel in ("simt", "unit", "tc5"):
        with pytest.raises(gqa.GqaError):
            _attend(p, t, kernel=kernel)
    with pytest.raises(gqa.GqaError):                    # no head scales
        gqa.attend(t["q"], t["k"], t["v"], t["lengths"], k_group_scale=t["kg"], v_group_scale=t["vg"])
    with pytest.raises(TypeError):                       # one group scale
        gqa.attend(t["q"], t["k"], t["v"], t["lengths"], k_scale=t["ks"], v_scale=t["vs"], k_group_scale=t["kg"])
    with pytest.raises(ValueError):                      # scales of another shape
        _attend(p, {**t, "kg": t["kg"][..., :4].contiguous()})
    with pytest.raises(ValueError):                      # a cache that is not contiguous
        _attend(p, {**t, "k": t["k"].transpose(1, 2).contiguous().transpose(1, 2)})
    with pytest.raises(TypeError):                       # a float32 query of a decode step
        _decode(p, {**t, "q": t["q"].float()}, bf, bf)
    with pytest.raises(ValueError):                      # more rows than lengths
        _attend(p, {**t, "q": t["q"].repeat(2, 1, 1)})
    with pytest.raises(TypeError):                       # a status word of the host, or of another type
        _attend(p, t, status=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError):
        _attend(p, t, status=torch.zeros(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):                      # a workspace of the host
        _attend(p, t, workspace=torch.zeros(1 << 20, dtype=torch.uint8))
    w = Problem("e2m1", "dense", [5], 9, 1, 128, 16, seed=32)
    with pytest.raises(gqa.GqaError):                    # G = 9
        _attend(w, _gpu(w))
    w = Problem("e2m1", "dense", [5], 2, 1, 32, 16, seed=33)
    with pytest.raises(gqa.GqaError):                    # D = 32
        _attend(w, _gpu(w))
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    with pytest.raises((gqa.GqaError, ValueError, TypeError)):   # no multi-token step
        gqa.decode_multi(t["q"], bf, bf, t["k"], t["v"], t["lengths"], cu, max_q_len=1, k_scale=t["ks"],
                         v_scale=t["vs"])


def test_values_helper_matches_torch():
    """The 64-bit reading of the format agrees with torch's own E4M3 and a table of the sixteen codes."""
    b = torch.arange(256, dtype=torch.uint8)
    from cache_reference import e4m3_values
    mine, theirs = e4m3_values(), b.view(torch.float8_e4m3fn).double()
    assert torch.equal(torch.isnan(mine), torch.isnan(theirs)) and torch.equal(mine.nan_to_num(), theirs.nan_to_num())
    c = torch.tensor([[0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE]], dtype=torch.uint8)
    s = torch.tensor([[0x38]], dtype=torch.uint8)        # 1.0
    v = values_e2m1(c, s, torch.tensor([1.0]))[0]
    assert v.tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]
    assert math.copysign(1, float(v[8])) == -1


SINKS = [(1, 128, torch.bfloat16), (1, 64, torch.float32), (4, 128, torch.bfloat16), (4, 64, torch.float32),
         (3, 128, torch.float32), (8, 128, torch.bfloat16), (8, 64, torch.float32), (6, 128, torch.float32)]


@pytest.mark.parametrize("grid", [1, 0])
@pytest.mark.parametrize("G,D,q_dtype", SINKS)
def test_many_small_weights_behind_a_large_one(G, D, q_dtype, grid):
    """Slots whose weights are 2^-30 to 2^-33 of the largest, which carries no value:
    the output is theirs alone. grid 1: one CTA meets all of them behind the large
    one, slots 0, 32, 64 and 96, one for each warp."""
    import gqa_kv_cache_gb300 as gqa
    n = 131072
    sinks = [0, 32, 64, 96]
    k = torch.zeros(1, 1, n, D // 2, dtype=torch.uint8)
    v = torch.full((1, 1, n, D // 2), 0x22, dtype=torch.uint8)   # 1, 1
    v[..., 1::2] = 0xA3                                  # 1.5, -1
    one = torch.full((1, 1, n, D // 16), 0x38, dtype=torch.uint8)
    k[0, 0, sinks, 0], v[0, 0, sinks] = 2, 0             # dim 0 is 1
    octaves = [32.5, 31.5, 30.0, 33.0, 32.0, 31.0, 30.5, 32.8][:G]
    q = torch.zeros(1, G, D)
    q[0, :, 0] = torch.tensor(octaves) * math.log(2) * math.sqrt(D)
    q = q.to(q_dtype)
    t = dict(q=q, lengths=torch.tensor([n], dtype=torch.int32), k=k, v=v, kg=one, vg=one.clone(), ks=torch.ones(1),
             vs=torch.ones(1))
    t = {x: y.cuda() for x, y in t.items()}
    got = gqa.attend(t["q"], t["k"], t["v"], t["lengths"], grid_ctas=grid, **_scales(t)).double().cpu()[0]
    w = torch.exp(-q[0, :, 0].double() / math.sqrt(D))   # of the others, against the sinks' 1
    val = torch.tensor([1.0, 1.0, 1.5, -1.0], dtype=torch.float64).repeat(D // 4)
    want = ((n - 4) * w / (4 + (n - 4) * w))[:, None] * val
    rel = ((got - want) / want).abs().amax(1)
    # scores of 33 ln 2: a float32 query's 22 bits and up to four roundings, 2^-24
    # each, are 2^-16.5 of a weight; its own error 2^-49 of the largest one is 2^-16
    # of it; the sums' roundings 2^-16
    assert float(rel.max()) <= 2.0 ** -14


@pytest.mark.parametrize("kind", ["bf16", "e2m1"])
def test_a_capture_fills_its_workspace_once(kind, monkeypatch):
    """One zero-filled workspace a capture, not one a call."""
    import gqa_kv_cache_gb300 as gqa
    lens = [3000, 50, 2000]
    p = Problem(kind, "dense", lens, 8, 2, 128, 3100, seed=20)
    q, ln, kv = p.q.cuda(), p.lengths.cuda(), [x.cuda() for x in p.kv]
    kw = {}
    if kind == "e2m1":
        kw = dict(k_scale=p.g[0].cuda(), v_scale=p.g[1].cuda(), k_group_scale=p.groups[0].cuda(),
                  v_group_scale=p.groups[1].cuda())
    want = gqa.attend(q, *kv, ln, **kw)
    torch.cuda.synchronize()
    made, zeros = [], torch.zeros
    monkeypatch.setattr(torch, "zeros", lambda *a, **k: made.append(a) or zeros(*a, **k))
    for turn in (1, 2):
        g, outs = torch.cuda.CUDAGraph(), [torch.empty_like(want) for _ in range(4)]
        with torch.cuda.graph(g):
            for o in outs:
                gqa.attend(q, *kv, ln, out=o, **kw)
        assert len(made) == turn
        for _ in range(3):
            for o in outs:
                o.fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(o, want) for o in outs)


def test_two_streams_of_a_capture():
    """Steps on two streams of one capture may run at once: a workspace each. Larger
    sizes later in the capture change nothing."""
    ps = [Problem("e2m1", "dense", [3000 - 7 * i, 50, 2000] * (1 + i), 8, 2, 128, 3100, seed=60 + i) for i in range(3)]
    ts = [_gpu(p) for p in ps]
    want = [_attend(p, t) for p, t in zip(ps, ts)]
    torch.cuda.synchronize()
    g, side, outs = torch.cuda.CUDAGraph(), torch.cuda.Stream(), [[torch.empty_like(w) for w in want] for _ in range(3)]
    with torch.cuda.graph(g):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        for p, t, *o in zip(ps, ts, *outs):
            _attend(p, t, out=o[0])
            with torch.cuda.stream(side):
                _attend(p, t, out=o[1])
            _attend(p, t, out=o[2], stream=side)
        here.wait_stream(side)
    for _ in range(20):
        for o in outs:
            for x in o:
                x.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        for o in outs:
            assert all(torch.equal(x, w) for x, w in zip(o, want))
    assert all(torch.equal(_attend(p, t), w) for p, t, w in zip(ps, ts, want))
