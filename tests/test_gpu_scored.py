"""Capped, distance-biased and counted scores over bfloat16 and 8-bit caches."""
import math

import pytest
import torch

import gqa_kv_cache_gb300 as gqa
import serve_reference as R

pytestmark = pytest.mark.gpu


class Case:
    """A random cache; ``row`` gives its values in 64 bits."""

    def __init__(self, kind, layout, lens, Hkv, G, D, Smax, bs=16, qt=torch.bfloat16, seed=0, room=0):
        self.gen = g = torch.Generator().manual_seed(seed)
        self.kind, self.lens, self.Hkv, self.G, self.D, self.bs, self.Smax = kind, lens, Hkv, G, D, bs, Smax
        B = len(lens)
        self.shape, self.table, self.slots = R.layout_of(layout, B, Hkv, Smax, bs, g, [n + room for n in lens])
        self.q = torch.randn(B, Hkv * G, D, generator=g).to(qt)
        self.kv, self.scales, self.kw = [], [None, None], {}
        for i in range(2):
            x = torch.randn(*self.shape, D, generator=g)
            if kind == "int8":
                self.kv.append((x * 34).round().clamp(-127, 127).to(torch.int8))
                s = self.shape[:2] if self.table is not None else (*self.shape[:2], Smax // bs)
                self.scales[i] = 0.02 + 0.02 * torch.rand(s, generator=g)
            else:
                self.kv.append(x.bfloat16())
        if kind == "int8":
            self.kw = dict(k_block_scale=self.scales[0].cuda(), v_block_scale=self.scales[1].cuda())
        self.g = [x.cuda() for x in self.kv]

    def row(self, i, b, n):
        x = R.row_slots(self.kv[i], b, n, self.table, self.slots, self.bs).double()
        if self.kind != "int8":
            return x
        s = self.scales[i]
        if self.table is not None:
            t = s[self.table[b, :-(-n // self.bs)].long()].T
        else:
            t = s[int(self.slots[b]) if self.slots is not None else b]
        return x * torch.repeat_interleave(t.double(), self.bs, 1)[:, :n, None]

    def attend(self, lens=None, **kw):
        n = torch.tensor(self.lens if lens is None else lens, dtype=torch.int32).cuda()
        if self.table is not None:
            return gqa.attend_paged(self.q.cuda(), *self.g, self.table.cuda(), n, **self.kw, **kw)
        return gqa.attend(self.q.cuda(), *self.g, n, None if self.slots is None else self.slots.cuda(), **self.kw, **kw)

    def expect(self, cap=0.0, slopes=None, window=0, prefix=0, sink=None, lens=None):
        """Per row: out, its tolerance, counts (Hkv, n), their tolerance."""
        got = []
        for b, n in enumerate(self.lens if lens is None else lens):
            k, v, ok = self.row(0, b, n), self.row(1, b, n), R.attended(n, window, prefix)
            shape = (self.Hkv, self.G)
            o, w, e = R.attention(self.q[b].double().view(*shape, self.D), k, v, cap,
                                  None if slopes is None else slopes.view(shape), ok,
                                  None if sink is None else sink.view(shape))
            got.append((o.reshape(-1, self.D), R.out_tolerance(w, e, float(v[:, ok].abs().max())), w.sum(1),
                        R.count_tolerance(w, e)))
        return got

    def check(self, out, want, weights=None, base=None):
        for b, (o, tol, w, wtol) in enumerate(want):
            err = (out[b].cpu().double() - o).abs().max()
            assert err <= tol, (b, float(err / tol))
            if weights is not None:
                n = w.shape[1]
                got = R.row_slots(weights.cpu(), b, n, self.table, self.slots, self.bs).double()
                was = R.row_slots(base, b, n, self.table, self.slots, self.bs).double()
                bound = wtol + 2.0 ** -24 * (was + w)
                assert ((got - was - w).abs() <= bound).all(), (b, float(((got - was - w).abs() / bound).max()))


KINDS = ["bf16", "int8"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("layout,bs", [("dense", 32), ("slots", 16), ("paged", 16), ("paged", 24), ("paged", 64)])
@pytest.mark.parametrize("D,G,qt", [(128, 4, torch.bfloat16), (64, 8, torch.float32), (128, 6, torch.float32),
                                    (64, 1, torch.bfloat16), (128, 3, torch.float32)])
def test_all_at_once(kind, layout, bs, D, G, qt):
    lens = [1, 15, 16, 33, 130, 517]
    c = Case(kind, layout, lens, 2, G, D, -(-576 // bs) * bs, bs, qt, seed=D + G)
    slopes = torch.exp2(-torch.arange(1, 2 * G + 1).float() / 2)
    sink = torch.randn(2 * G, generator=c.gen)
    for kw in (dict(), dict(cap=5.0), dict(slopes=slopes), dict(cap=2.0, slopes=slopes, window=100, prefix=20, sink=sink)):
        want = c.expect(**kw)
        args = dict(window=kw.get("window", 0), kept_prefix=kw.get("prefix", 0), score_cap=kw.get("cap", 0.0),
                    head_slopes=slopes.cuda() if "slopes" in kw else None, sink=sink.cuda() if "sink" in kw else None)
        for grid in (0, 1, 5, 33):
            base = torch.rand(c.shape, generator=c.gen)
            weights = base.cuda()
            out = c.attend(grid_ctas=grid, weights=weights, **args)
            c.check(out, want, weights, base)
            touched = torch.zeros(c.shape, dtype=torch.bool)
            for b, n in enumerate(lens):
                ok = R.attended(n, args["window"], args["kept_prefix"]).expand(2, -1)
                R.put_row(touched, b, n, ok, c.table, c.slots, bs)
            assert torch.equal(weights.cpu()[~touched], base[~touched])      # other counts are left
            if kw or kind == "int8":
                c.check(c.attend(grid_ctas=grid, **args), want)


@pytest.mark.parametrize("kind", KINDS)
def test_a_cap_far_above_the_scores_changes_little(kind):
    """cap = 2^20: c tanh(s / c) is s to s^3 / (3 c^2); tanhf to its steps."""
    c = Case(kind, "dense", [100, 400], 2, 4, 128, 512, seed=3)
    c.check(c.attend(score_cap=2.0 ** 20), c.expect(cap=2.0 ** 20))
    small = c.attend(score_cap=1e-6)                              # every score the same: the mean of the values
    for b, n in enumerate(c.lens):
        v = c.row(1, b, n)
        mean = v.mean(1)[:, None].expand(-1, 4, -1).reshape(-1, 128)
        assert (small[b].cpu().double() - mean).abs().max() <= (2e-6 + 2.0 ** -17) * v.abs().max()


@pytest.mark.parametrize("kind", KINDS)
def test_masked_places_may_hold_anything(kind):
    lens = [35, 70]                                               # windows from slots 16 and 51 on
    c = Case(kind, "dense", lens, 1, 5, 64, 96, seed=4)
    want = c.expect(cap=10.0, window=19)
    for i in range(2):
        if kind == "bf16":
            c.g[i][:, :, 75:] = math.nan
            c.g[i][:, :, :10] = math.inf
        else:
            c.kw["kv"[i] + "_block_scale"][:, :, 5:] = math.nan
            c.kw["kv"[i] + "_block_scale"][:, :, 0] = math.nan
    base = torch.zeros(c.shape)
    weights = base.cuda()
    c.check(c.attend(score_cap=10.0, window=19, weights=weights), want, weights, base)


@pytest.mark.parametrize("layout,bs", [("dense", 16), ("paged", 24)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("where", [slice(0, 300), slice(170, 600), slice(500, 699)])
@pytest.mark.parametrize("slopes", [False, True])
def test_slots_masked_by_keys_of_minus_infinity(layout, bs, D, where, slopes):
    # scores of minus infinity: those slots weigh nothing, tiles full of them too
    n, G = 700, 4
    c = Case("bf16", layout, [n], 2, G, D, 720, bs=bs, seed=31)
    c.q[..., 0] = c.q[..., 0].abs() + 0.25
    ok = torch.ones(n, dtype=torch.bool)
    ok[where] = False
    k = R.row_slots(c.kv[0], 0, n, c.table, None, bs).clone()
    k[:, ~ok, 0] = -math.inf
    R.put_row(c.kv[0], 0, n, k, c.table, None, bs)
    c.g[0].copy_(c.kv[0])
    sl = 0.05 * torch.randn(2 * G, generator=c.gen) if slopes else None
    o, w, e = R.attention(c.q[0].double().view(2, G, D), k.double(), c.row(1, 0, n), 0.0,
                          None if sl is None else sl.view(2, G), ok)
    weights = torch.zeros(*c.shape, device="cuda")
    out = c.attend(weights=weights, **({} if sl is None else dict(head_slopes=sl.cuda())))
    vmax = float(c.row(1, 0, n).abs().max())
    c.check(out, [(o.reshape(-1, D), R.out_tolerance(w, e, vmax), w.sum(1), R.count_tolerance(w, e))], weights,
            torch.zeros(*c.shape))


@pytest.mark.parametrize("layout,bs", [("dense", 16), ("paged", 24)])
@pytest.mark.parametrize("D,G", [(64, 4), (128, 5)])
@pytest.mark.parametrize("where", [slice(0, 300), slice(500, 699)])
def test_float32_queries_over_keys_of_minus_infinity(layout, bs, D, G, where):
    # a query's elements with remainders of either sign, and without any, meet infinite keys
    n = 700
    c = Case("bf16", layout, [n], 2, G, D, 720, bs, torch.float32, seed=33)
    c.q[..., 0] = c.q[..., 0].abs() + 0.25
    c.q[0, ::3, 0] = c.q[0, ::3, 0].bfloat16().float()
    ok = torch.ones(n, dtype=torch.bool)
    ok[where] = False
    k = R.row_slots(c.kv[0], 0, n, c.table, None, bs).clone()
    k[:, ~ok, 0] = -math.inf
    R.put_row(c.kv[0], 0, n, k, c.table, None, bs)
    c.g[0].copy_(c.kv[0])
    for cap in (0.0, 8.0):
        if cap:                               # capped, they are the smallest score there is
            s = torch.einsum("hgd,hnd->hgn", c.q[0].double().view(2, G, D), k.double()) / math.sqrt(D)
            w = torch.softmax(cap * torch.tanh(s / cap), -1)
            v, e = c.row(1, 0, n), torch.full_like(w, 2.0 ** -16)   # (D / 16 + 6) 2^-23 of sums up to 100 / sqrt(D)
            o = torch.einsum("hgn,hnd->hgd", w, v)
        else:
            o, w, e = R.attention(c.q[0].double().view(2, G, D), k.double(), c.row(1, 0, n), 0.0, None, ok)
        want = [(o.reshape(-1, D), R.out_tolerance(w, e, float(c.row(1, 0, n).abs().max())), w.sum(1), R.count_tolerance(w, e))]
        for grid in (0, 3):
            weights = torch.zeros(c.shape, device="cuda")
            c.check(c.attend(weights=weights, score_cap=cap, grid_ctas=grid), want, weights, torch.zeros(c.shape))


@pytest.mark.parametrize("layout,bs", [("dense", 16), ("paged", 24)])
@pytest.mark.parametrize("D,G,qt", [(64, 4, torch.bfloat16), (128, 5, torch.float32)])
def test_values_of_infinity(layout, bs, D, G, qt):
    """An infinite value gives its element infinity of its sign, infinities of both signs NaN, other elements nothing."""
    n = 700
    c = Case("bf16", layout, [n], 2, G, D, 720, bs, qt, seed=34)
    v = R.row_slots(c.kv[1], 0, n, c.table, None, bs).clone()
    good = v.clone()
    for j, d, x in ((3, 1, math.inf), (699, 7, -math.inf), (350, 8, math.inf), (351, 8, math.inf), (10, 20, math.inf),
                    (600, 20, -math.inf)):
        v[:, j, d], good[:, j, d] = x, 0
    R.put_row(c.kv[1], 0, n, v, c.table, None, bs)
    c.g[1].copy_(c.kv[1])
    o, w, e = R.attention(c.q[0].double().view(2, G, D), c.row(0, 0, n), good.double())
    tol = R.out_tolerance(w, e, float(good.abs().max()))
    for grid in (0, 3, 33):
        out = c.attend(score_cap=2.0 ** 40, grid_ctas=grid)[0].cpu().double()
        assert (out[:, 1] == math.inf).all() and (out[:, 7] == -math.inf).all() and (out[:, 8] == math.inf).all()
        assert out[:, 20].isnan().all()
        rest = torch.ones(D, dtype=torch.bool)
        rest[[1, 7, 8, 20]] = False
        assert ((out - o.reshape(-1, D))[:, rest].abs() <= tol).all()


def test_scores_that_are_not_finite():
    """A NaN key gives its row NaN and no other; -inf scores count as nothing."""
    c = Case("bf16", "dense", [40, 40], 1, 2, 64, 48, seed=5)
    c.g[0][0, 0, 7, 3] = math.nan
    weights = torch.zeros(c.shape, device="cuda")
    out = c.attend(weights=weights)
    assert out[0].isnan().all() and weights[0, 0, :40].isnan().all() and not weights[0, 0, 40:].any()
    want = c.expect()
    assert (out[1].cpu().double() - want[1][0]).abs().max() <= want[1][1]
    d = Case("bf16", "dense", [40], 1, 2, 64, 48, seed=6)
    d.q = d.q.abs()
    d.kv[0][0, 0, 7] = -math.inf
    d.g[0] = d.kv[0].cuda()
    weights = torch.zeros(d.shape, device="cuda")
    out = d.attend(weights=weights)
    assert out.isfinite().all() and float(weights[0, 0, 7]) == 0.0
    assert abs(float(weights.sum()) - 2.0) <= 2 * 2.0 ** -15


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("layout", ["dense", "paged"])
def test_decode_step(kind, layout):
    lens = [0, 5, 31, 64, 300]
    c = Case(kind, layout, lens, 2, 4, 128, 320, seed=8, room=1)
    k, v = (torch.randn(5, 2, 128, generator=c.gen).bfloat16() for _ in range(2))
    slopes = torch.rand(8, generator=c.gen)
    weights = torch.zeros(c.shape, device="cuda")
    at = torch.tensor(lens, dtype=torch.int32).cuda()
    kw = dict(score_cap=3.0, head_slopes=slopes.cuda(), weights=weights, **c.kw)
    if c.table is not None:
        out = gqa.decode_step_paged(c.q.cuda(), k.cuda(), v.cuda(), *c.g, c.table.cuda(), at, **kw)
    else:
        out = gqa.decode_step(c.q.cuda(), k.cuda(), v.cuda(), *c.g, at, **kw)
    after = [n + 1 for n in lens]
    if kind == "bf16":
        for i, x in enumerate((k, v)):
            for b, n in enumerate(lens):
                row = R.row_slots(c.kv[i], b, n + 1, c.table, None, 16).clone()
                row[:, n] = x[b]
                R.put_row(c.kv[i], b, n + 1, row, c.table, None, 16)
            assert torch.equal(c.g[i].cpu(), c.kv[i])
    else:                                                          # the codes' own test is test_gpu_block8
        c.kv = [x.cpu() for x in c.g]
        c.scales = [c.kw["k_block_scale"].cpu(), c.kw["v_block_scale"].cpu()]
    c.check(out, c.expect(cap=3.0, slopes=slopes, lens=after), weights, torch.zeros(c.shape))


def test_long_rows_and_many_pieces():
    """One row of 60000 slots cut among every CTA, its counts summing to the heads."""
    c = Case("int8", "paged", [60000], 1, 8, 64, 60032, bs=64, seed=9)
    base = torch.zeros(c.shape)
    weights = base.cuda()
    c.check(c.attend(weights=weights), c.expect(), weights, base)
    weights.zero_()
    c.check(c.attend(weights=weights, grid_ctas=700), c.expect(), weights, base)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("layout,bs", [("paged", 16), ("paged", 24), ("paged", 64), ("slots", 16)])
@pytest.mark.parametrize("sign", [1, -1])
def test_slopes_over_long_rows(kind, layout, bs, sign):
    """Rows of many tiles and pages with steep and flat slopes of either sign, whole and in pieces."""
    lens = [9000, 4097, 300, 6001]
    c = Case(kind, layout, lens, 1, 6, 128, -(-9024 // bs) * bs, bs, torch.float32, seed=11)
    slopes = sign * torch.exp2(-torch.tensor([0.5, 2.0, 4.0, 7.0, 10.0, 14.0]))
    base = torch.zeros(c.shape)
    for kw in (dict(), dict(window=3000, prefix=70)):
        want = c.expect(slopes=slopes, **kw)
        for grid in (0, 3, 61):
            weights = base.cuda()
            out = c.attend(head_slopes=slopes.cuda(), weights=weights, grid_ctas=grid, window=kw.get("window", 0),
                           kept_prefix=kw.get("prefix", 0))
            c.check(out, want, weights, base)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("layout,bs", [("dense", 64), ("paged", 16), ("paged", 24)])
@pytest.mark.parametrize("D,G,qt", [(64, 4, torch.float32), (128, 6, torch.bfloat16)])
def test_large_biases_of_the_slots_that_win(kind, layout, bs, D, G, qt):
    """Negative slopes in long rows: the slots that weigh have the largest biases, of which their scores must not
    take the rounding. What is rounded is the bias less the winning slot's (and what a reference lies below the
    largest score: 12 and 10 in base 2): the common part of all biases leaves the softmax as it is."""
    lens = [100001, 48013]
    c = Case(kind, layout, lens, 1, G, D, -(-100032 // bs) * bs, bs, qt, seed=21)
    slopes = -torch.tensor([0.70710678, 0.25, 3.0, 0.01, 11.0, 0.1])[:G]
    for window, prefix in ((0, 0), (30011, 7)):
        want = []
        for b, n in enumerate(lens):
            ok = R.attended(n, window, prefix)
            k, v = c.row(0, b, n)[0, ok], c.row(1, b, n)[0, ok]
            q = c.q[b].double()
            s = q @ k.T / math.sqrt(D)
            bias = slopes.double()[:, None] * (torch.arange(n)[ok] - (n - 1)).double()
            w = torch.softmax(s + bias, -1)
            near = (bias - bias.gather(1, (s + bias).argmax(-1, keepdim=True))).abs()
            big = (q.abs() @ k.abs().T).amax(-1, keepdim=True) / math.sqrt(D)
            err = R.score_error(D, big, s.abs() + near + 24)
            full, d = torch.zeros(1, G, n, dtype=torch.float64), torch.zeros(1, G, n, dtype=torch.float64)
            full[0][:, ok], d[0][:, ok] = w, err
            want.append((w @ v, R.out_tolerance(full, d, float(v.abs().max())), full.sum(1), R.count_tolerance(full, d)))
        base = torch.zeros(c.shape)
        for grid in (0, 3):
            weights = base.cuda()
            out = c.attend(head_slopes=slopes.cuda(), weights=weights, window=window, kept_prefix=prefix, grid_ctas=grid)
            c.check(out, want, weights, base)


def test_rows_that_share_blocks_all_count():
    # three rows with the first 8 blocks in common, as after a common prompt
    lens = [150, 163, 200]
    c = Case("bf16", "paged", lens, 2, 4, 64, 208, seed=41)
    c.table[:, :8] = c.table[0, :8]
    want = c.expect()
    weights = torch.zeros(c.shape, device="cuda")
    out = c.attend(weights=weights)
    c.check(out, want)
    got = weights.cpu().double()
    total, bound = torch.zeros(c.shape, dtype=torch.float64), torch.zeros(c.shape, dtype=torch.float64)
    for b, n in enumerate(lens):
        for j in range(-(-n // 16)):
            m = min(16, n - 16 * j)
            total[int(c.table[b, j]), :, :m] += want[b][2][:, 16 * j:16 * j + m]
            bound[int(c.table[b, j]), :, :m] += want[b][3][:, 16 * j:16 * j + m]
    assert ((got - total).abs() <= bound + 3 * 2.0 ** -24 * total).all()


def test_bad_rows():
    c = Case("bf16", "paged", [40, 40, 40], 2, 2, 64, 64, seed=10)
    c.table[1, 1] = -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    weights = torch.zeros(c.shape, device="cuda")
    out = c.attend(lens=[40, 40, 65], weights=weights, status=status)
    assert int(status) == 5 and out[1:].isnan().all() and out[0].isfinite().all()
    assert weights[c.table[1, 0].long()].isnan().all()
    assert not weights[c.table[2, :3].long()].any()
    assert abs(float(weights[c.table[0, :3].long()].sum()) - 4.0) < 1e-3


def test_refusals():
    c = Case("bf16", "dense", [20, 20], 2, 2, 64, 32)
    w = torch.zeros(c.shape, device="cuda")
    for bad in (dict(head_slopes=torch.zeros(3, device="cuda")), dict(head_slopes=torch.zeros(4, device="cuda").double()),
                dict(weights=w[:, :1].contiguous()), dict(weights=w.double()), dict(k_scale=w[0, :, 0], score_cap=1.0),
                dict(wait_limit_cycles=5, score_cap=1.0)):
        with pytest.raises(TypeError):
            c.attend(**bad)
    for bad in (dict(weights=w.cpu()), dict(head_slopes=torch.zeros(4)),
                dict(weights=torch.zeros(2, 32, 2, device="cuda").transpose(1, 2))):
        with pytest.raises(ValueError):
            c.attend(**bad)
    for bad in (dict(score_cap=-1.0), dict(score_cap=math.inf), dict(score_cap=math.nan), dict(score_cap=1.0, kernel="simt")):
        with pytest.raises(gqa.GqaError):
            c.attend(**bad)
    q, n = c.q.cuda(), torch.tensor([20, 20], dtype=torch.int32).cuda()
    with pytest.raises(TypeError):
        gqa.attend(q, c.g[0].float(), c.g[1].float(), n, score_cap=2.0)
    d = Case("bf16", "dense", [20], 1, 9, 64, 32)
    with pytest.raises(gqa.GqaError):
        d.attend(score_cap=2.0)
