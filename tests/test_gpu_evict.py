"""Eviction: the kept slots, and the vectors and counts moved, exactly."""
import math

import pytest
import torch

import gqa_kv_cache_gb300 as gqa
import serve_reference as R

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.uint8}


class Case:
    def __init__(self, kind, layout, lens, Hkv, D, Smax, bs=16, seed=0, counts="spread"):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.Hkv, self.D, self.bs, self.Smax = lens, Hkv, D, bs, Smax
        self.shape, self.table, self.slots = R.layout_of(layout, len(lens), Hkv, Smax, bs, g, lens)
        if kind == "e4m3":
            self.kv = [torch.randint(0, 256, (*self.shape, D), generator=g).to(torch.uint8) for _ in range(2)]
        else:
            self.kv = [torch.randn(*self.shape, D, generator=g).to(TYPES[kind]) for _ in range(2)]
        w = torch.rand(self.shape, generator=g)
        self.w = {"spread": torch.where(w < 0.1, 0.0, torch.exp2(-20 * w)), "same": torch.ones_like(w),
                  "zero": torch.where(w < 0.5, 0.0, -0.0), "few": (w * 4).floor(), "signs": w - 0.5}[counts]

    def index(self):
        return None if self.slots is None else self.slots.cuda()

    def run(self, n_keep, w=None, lens=None, **kw):
        """Evicts on the GPU: (ids, lengths, k, v, weights) afterwards."""
        k, v, w = self.kv[0].cuda(), self.kv[1].cuda(), (self.w if w is None else w).cuda()
        n = torch.tensor(self.lens if lens is None else lens, dtype=torch.int32).cuda()
        if self.table is not None:
            ids, new = gqa.evict_paged(k, v, self.table.cuda(), w, n, n_keep, **kw)
        else:
            ids, new = gqa.evict(k, v, w, n, n_keep, self.index(), **kw)
        return ids.cpu(), new.cpu(), k.cpu(), v.cpu(), w.cpu()

    def expect(self, n_keep, n_first, n_last):
        ids = torch.full((len(self.lens), self.Hkv, n_keep), -1, dtype=torch.int32)
        k, v, w = self.kv[0].clone(), self.kv[1].clone(), self.w.clone()
        for b, n in enumerate(self.lens):
            if n == 0:
                continue
            rows = [R.row_slots(x, b, n, self.table, self.slots, self.bs).clone() for x in (k, v, w)]
            for h in range(self.Hkv):
                at = R.kept(rows[2][h], n, n_keep, n_first, n_last)
                ids[b, h, :len(at)] = torch.tensor(at, dtype=torch.int32)
                for x in rows:
                    x[h, :len(at)] = x[h, at].clone()
                if n > n_keep:
                    rows[2][h, len(at):] = 0.0
            for x, y in zip((k, v, w), rows):
                R.put_row(x, b, n, y, self.table, self.slots, self.bs)
        return ids, torch.tensor([min(n, n_keep) for n in self.lens], dtype=torch.int32), k, v, w


def _same(got, want):
    for a, b in zip(got, want):
        if a.dtype.is_floating_point:
            assert torch.equal(a.isnan(), b.isnan())
            a, b = a.nan_to_num(nan=0.0, posinf=9.0, neginf=-9.0), b.nan_to_num(nan=0.0, posinf=9.0, neginf=-9.0)
        assert torch.equal(a, b)


@pytest.mark.parametrize("layout,bs", [("dense", 16), ("slots", 16), ("paged", 16), ("paged", 24)])
@pytest.mark.parametrize("kind,D", [("bf16", 128), ("f32", 64), ("e4m3", 64), ("e4m3", 16), ("bf16", 24)])
@pytest.mark.parametrize("n_keep,n_first,n_last", [(1, 0, 0), (40, 4, 8), (257, 0, 1), (16, 8, 8), (600, 3, 300)])
def test_in_place_and_elsewhere(layout, bs, kind, D, n_keep, n_first, n_last):
    lens = [0, 1, 40, 41, 300, 1000]
    c = Case(kind, layout, lens, 2, D, -(-1008 // bs) * bs, bs, seed=n_keep)
    want = c.expect(n_keep, n_first, n_last)
    _same(c.run(n_keep, n_first=n_first, n_last=n_last), want)
    B, slots = len(lens), n_keep + 3
    fill = torch.randint(0, 100, (B, 2, slots, D)).to(c.kv[0].dtype)
    k2, v2, w2 = fill.cuda(), fill.cuda(), torch.full((B, 2, slots), -5.0, device="cuda")
    ids, new, k, v, w = c.run(n_keep, n_first=n_first, n_last=n_last, k_out=k2, v_out=v2, weights_out=w2)
    _same((ids, new, k, v, w), (*want[:2], *c.kv, c.w))                # the cache is only read
    for b, n in enumerate(want[1].tolist()):
        for out, x in ((k2, want[2]), (v2, want[3])):
            if n:
                assert torch.equal(out[b, :, :n].cpu(), R.row_slots(x, b, n, c.table, c.slots, bs))
            assert torch.equal(out[b, :, n:].cpu(), fill[b, :, n:])
        if n:
            assert torch.equal(w2[b, :, :n].cpu(), R.row_slots(want[4], b, n, c.table, c.slots, bs))
        assert not w2[b, :, n:].any()


@pytest.mark.parametrize("counts", ["same", "zero", "few", "signs"])
def test_equal_counts_go_to_the_lowest_slot(counts):
    c = Case("bf16", "dense", [700, 5000], 1, 64, 9008, counts=counts)
    for n_keep, n_first, n_last in ((64, 0, 0), (1000, 10, 20), (4999, 0, 1)):
        _same(c.run(n_keep, n_first=n_first, n_last=n_last), c.expect(n_keep, n_first, n_last))


def test_counts_that_are_not_finite():
    c = Case("f32", "dense", [200], 1, 16, 208, seed=3)
    c.w[0, 0, 50], c.w[0, 0, 60], c.w[0, 0, 70], c.w[0, 0, 80] = math.nan, math.inf, -math.inf, math.nan
    for n_keep in (1, 2, 3, 50, 199):
        _same(c.run(n_keep, n_first=0, n_last=0), c.expect(n_keep, 0, 0))


def test_a_row_longer_than_the_cached_counts():
    """40000 slots: part of the counts is read again; kept slots many chunks apart."""
    c = Case("e4m3", "paged", [40000, 16384, 16385], 1, 16, 40000, bs=32, seed=4)
    for n_keep in (100, 20000):
        _same(c.run(n_keep, n_first=1, n_last=5), c.expect(n_keep, 1, 5))


@pytest.mark.parametrize("counts", ["spread", "same", "few"])
def test_long_rows_elsewhere(counts):
    """Long rows of few heads (several CTAs each), into other buffers; many equal counts among them."""
    c = Case("e4m3", "paged", [40000, 7, 33333], 1, 16, 40000, bs=32, seed=6, counts=counts)
    for n_keep, n_first, n_last in ((9000, 2, 3), (500, 0, 0)):
        want = c.expect(n_keep, n_first, n_last)
        k2, v2 = (torch.zeros(3, 1, n_keep, 16, dtype=torch.uint8, device="cuda") for _ in range(2))
        w2 = torch.zeros(3, 1, n_keep, device="cuda")
        ids, new, *_ = c.run(n_keep, n_first=n_first, n_last=n_last, k_out=k2, v_out=v2, weights_out=w2)
        _same((ids, new), want[:2])
        for b, n in enumerate(want[1].tolist()):
            for out, x in ((k2, want[2]), (v2, want[3]), (w2, want[4])):
                assert torch.equal(out[b, :, :n].cpu(), R.row_slots(x, b, n, c.table, c.slots, 32))


def test_many_rows():
    """More (row, head) pairs than SMs, rows longer than the counts that one CTA holds: in place and elsewhere."""
    lens = [(i * 7919) % 17000 for i in range(80)]
    c = Case("e4m3", "dense", lens, 2, 16, 17000, seed=7)
    want = c.expect(64, 1, 2)
    _same(c.run(64, n_first=1, n_last=2), want)
    k2, v2 = (torch.zeros(80, 2, 64, 16, dtype=torch.uint8, device="cuda") for _ in range(2))
    ids, new, *_ = c.run(64, n_first=1, n_last=2, k_out=k2, v_out=v2)
    _same((ids, new), want[:2])
    for b, n in enumerate(want[1].tolist()):
        assert torch.equal(k2[b, :, :n].cpu(), want[2][b, :, :n]) and torch.equal(v2[b, :, :n].cpu(), want[3][b, :, :n])


def test_bad_rows_stay():
    c = Case("bf16", "paged", [100, 100, 100, 100], 2, 64, 112, seed=5)
    c.table[1, 3], c.table[2, 0] = -1, 99999
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids, new, k, v, w = c.run(20, lens=[100, 100, 100, 113], status=status)
    assert int(status) == 1 | 4 and new.tolist() == [20, 0, 0, 0] and (ids[1:] == -1).all()
    c.lens = [100, 0, 0, 0]
    want = c.expect(20, 0, 1)
    _same((k, v, w), want[2:])
    d = Case("bf16", "slots", [30], 1, 64, 32)
    d.slots[0] = 77
    status.zero_()
    ids, new, k, v, w = d.run(20, status=status)
    assert int(status) == 2 and new.tolist() == [0]
    _same((k, v, w), (*d.kv, d.w))


def test_refusals():
    c = Case("bf16", "dense", [30, 30], 2, 64, 32)
    k, v, w = c.kv[0].cuda(), c.kv[1].cuda(), c.w.cuda()
    n = torch.tensor([30, 30], dtype=torch.int32).cuda()
    out = torch.zeros(2, 2, 8, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(n_keep=0), dict(n_first=-1), dict(n_first=5, n_last=5), dict(k_out=out), dict(k_out=out, v_out=out[:, :, :7]),
                dict(k_out=out.float(), v_out=out.float()), dict(weights_out=w[..., :8].contiguous())):
        with pytest.raises(ValueError):
            gqa.evict(k, v, w, n, **{"n_keep": 8, **bad})
    for bad in (lambda: gqa.evict(k.to(torch.int8), v.to(torch.int8), w, n, 8), lambda: gqa.evict(k, v, w.double(), n, 8),
                lambda: gqa.evict(k, v, w[:, :1].contiguous(), n, 8), lambda: gqa.evict(k, v, w, n.long(), 8),
                lambda: gqa.evict(k.half(), v.half(), w, n, 8)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(ValueError):
        gqa.evict(k, v.float(), w, n, 8)
