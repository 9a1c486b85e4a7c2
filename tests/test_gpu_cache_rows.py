"""append and read: packed tokens into float32, bfloat16, E4M3 and E2M1 caches
and back, against the formats' 64-bit definitions; key bounds; bad content."""
import math

import pytest
import torch

from cache_reference import E2M1_MIDS, cache_values, e4m3_values, quantise_e2m1

pytestmark = pytest.mark.gpu

KINDS = ["f32", "bf16", "e4m3", "e2m1"]
CACHE = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.uint8, "e2m1": torch.uint8}


class Case:
    """Tokens for B rows at starts `at`, `n` tokens each, and an empty cache."""

    def __init__(self, kind, layout, at, n, Hkv, D, cap, bs=16, dtype=torch.bfloat16, seed=0, pad=0, bounds=False):
        gen = torch.Generator().manual_seed(seed)
        self.kind, self.layout, self.at, self.n, self.D, self.bs, self.cap = kind, layout, at, n, D, bs, cap
        self.B, self.Hkv, self.T = len(at), Hkv, sum(n)
        self.x = [(torch.randn(self.T + pad, Hkv, D, generator=gen) * (1 + i)).to(dtype) for i in range(2)]
        self.g = [(0.75 + 0.5 * torch.rand(Hkv, generator=gen)) * (1 + i) * 4 / 448 / (6 if kind == "e2m1" else 1)
                  for i in range(2)]
        cu = [0]
        for v in n:
            cu.append(cu[-1] + v)
        self.cu = torch.tensor(cu, dtype=torch.int32)
        self.lengths = torch.tensor(at, dtype=torch.int32)
        self.table = self.slots = None
        if layout == "paged":
            nb = cap // bs
            perm = torch.randperm(self.B * nb, generator=gen).view(self.B, nb).int()
            held = torch.tensor([-(-(a + v) // bs) for a, v in zip(at, n)])
            self.table = torch.where(torch.arange(nb) < held[:, None], perm, -1)
            lead = (self.B * nb, Hkv, bs)
        else:
            self.slots = torch.randperm(self.B + 3, generator=gen)[:self.B].int() if layout == "slots" else None
            lead = (self.B + (3 if layout == "slots" else 0), Hkv, cap)
        row = D // 2 if kind == "e2m1" else D
        self.kv = [torch.zeros(*lead, row).to(CACHE[kind]).cuda() for _ in range(2)]
        self.groups = [torch.zeros(*lead, D // 16, dtype=torch.uint8, device="cuda") for _ in range(2)] \
            if kind == "e2m1" else [None, None]
        self.bounds = None
        if bounds:
            shape = lead[:2] if layout == "paged" else (*lead[:2], cap // bs)
            self.bounds = torch.full((*shape, 2, D), 0.25, dtype=torch.bfloat16, device="cuda")

    def scales(self):
        kw = {}
        if self.kind in ("e4m3", "e2m1"):
            kw = dict(k_scale=self.g[0].cuda(), v_scale=self.g[1].cuda())
        if self.kind == "e2m1":
            kw.update(k_group_scale=self.groups[0], v_group_scale=self.groups[1])
        return kw

    def append(self, **kw):
        import gqa_kv_cache_gb300 as gqa
        a = [x.cuda() for x in self.x] + self.kv
        kw = {**self.scales(), **({"k_bounds": self.bounds} if self.bounds is not None else {}), **kw}
        if self.table is not None:
            gqa.append_paged(*a, self.table.cuda(), self.lengths.cuda(), self.cu.cuda(), **kw)
        else:
            gqa.append(*a, self.lengths.cuda(), self.cu.cuda(), None if self.slots is None else self.slots.cuda(), **kw)

    def read(self, **kw):
        import gqa_kv_cache_gb300 as gqa
        T = len(self.x[0])
        if self.table is not None:
            return gqa.read_paged(*self.kv, self.table.cuda(), self.lengths.cuda(), self.cu.cuda(), T,
                                  **self.scales(), **kw)
        return gqa.read(*self.kv, self.lengths.cuda(), self.cu.cuda(), T,
                        None if self.slots is None else self.slots.cuda(), **self.scales(), **kw)

    def where(self, b, s):
        """Index of slot s of row b in the cache (the heads' axis free)."""
        if self.table is not None:
            return int(self.table[b, s // self.bs]), slice(None), s % self.bs
        return (int(self.slots[b]) if self.slots is not None else b), slice(None), s

    def tokens(self):
        for b in range(self.B):
            for i in range(self.n[b]):
                yield int(self.cu[b]) + i, b, self.at[b] + i


def _check_bytes(c):
    """Every token's bytes are the format's, every other byte is as it was."""
    for i in range(2):
        got, g = c.kv[i].cpu(), c.g[i].view(-1, 1)
        want = torch.zeros_like(got)
        if c.kind == "e2m1":
            codes, scales, _, y = quantise_e2m1(c.x[i], g)
            ws = torch.zeros_like(c.groups[i].cpu())
        for t, b, s in c.tokens():
            at = c.where(b, s)
            if c.kind == "e2m1":
                mine, ref = got[at], codes[t]
                if not torch.equal(mine, ref):
                    # a float32 quotient may reach a border that the exact one misses by 2^-24
                    for sh in (0, 4):
                        off = ((mine >> sh) & 15) != ((ref >> sh) & 15)
                        q = y[t].view(c.Hkv, -1, 2)[..., sh // 4].abs()
                        near = ((q[..., None] - E2M1_MIDS).abs() <= 2.0 ** -24 * E2M1_MIDS).any(-1)
                        assert bool((~off | near).all()), (t, b, s)
                    ref = mine
                want[at], ws[at] = ref, scales[t]
            elif c.kind == "e4m3":
                q = (c.x[i][t].float() / g).clamp(-448, 448)     # float32 quotient, as the format says
                want[at] = q.to(torch.float8_e4m3fn).view(torch.uint8)
            else:
                want[at] = c.x[i][t].to(got.dtype)
        assert torch.equal(got, want)
        if c.kind == "e2m1":
            assert torch.equal(c.groups[i].cpu(), ws)


def _check_read(c, dtype, got):
    for i in range(2):
        vals = cache_values(c.kind, c.kv[i].cpu(), None if c.groups[i] is None else c.groups[i].cpu(), c.g[i])
        for t, b, s in c.tokens():
            want = vals[c.where(b, s)]
            # one rounding to float32 (the product), one to the output type
            tol = want.abs() * (torch.finfo(dtype).eps / 2 + 2.0 ** -24) * (1 + 2.0 ** -8)
            assert bool(((got[i][t].double().cpu() - want).abs() <= tol).all()), (t, b, s)


LAYOUTS = ["dense", "slots", "paged"]
SHAPES = [([0, 5, 16], [1, 1, 1], 2, 128), ([0, 3, 17, 40], [70, 0, 33, 1], 3, 64), ([9], [200], 1, 256),
          ([0, 31], [16, 18], 5, 16)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_append_and_read(shape, kind, layout, dtype):
    at, n, Hkv, D = SHAPES[shape]
    c = Case(kind, layout, at, n, Hkv, D, 224, dtype=dtype, seed=shape)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.append(status=st)
    _check_bytes(c)
    keep = [x.clone() for x in c.kv]
    _check_read(c, dtype, c.read(dtype=dtype, status=st))
    assert int(st) == 0 and all(torch.equal(a, b) for a, b in zip(keep, c.kv))


@pytest.mark.parametrize("kind", ["e4m3", "e2m1", "bf16"])
def test_many_tokens(kind):
    """More tokens than one CTA a token; odd starts."""
    c = Case(kind, "paged", [3, 0, 1000], [2500, 1, 1777], 2, 64, 2800, bs=16, seed=4, bounds=True)
    c.append()
    _check_bytes(c)
    _check_bounds(c, {})
    _check_read(c, torch.bfloat16, c.read())


def _bounds_now(c):
    """{(b, block): (lo, hi)} (Hkv, D) that the bounds must hold after one call."""
    want = {}
    for t, b, s in c.tokens():
        key = (b, s // c.bs)
        x = c.x[0][t].float()
        lo, hi = x.clone(), x.clone()
        if c.x[0].dtype == torch.float32:                # rounded outwards
            lo, hi = _down(x), -_down(-x)
        if s % c.bs == 0:
            want[key] = (lo, hi)
        else:
            old = want.get(key) or c.before[key]
            want[key] = (torch.minimum(old[0], lo), torch.maximum(old[1], hi))
    return want


def _down(x):
    y = x.to(torch.bfloat16)
    up = y.float() > x
    z = torch.where(up, torch.nextafter(y, torch.full_like(y, -math.inf)), y)
    return z.float()


def _bound_at(c, b, j):
    if c.table is not None:
        v = c.bounds[int(c.table[b, j])]
    else:
        v = c.bounds[int(c.slots[b]) if c.slots is not None else b, :, j]
    return v[:, 0].float().cpu(), v[:, 1].float().cpu()


def _check_bounds(c, before):
    """The touched blocks' bounds, and that no other block's changed from 0.25."""
    q = 0.25 * torch.ones(c.Hkv, c.D)
    c.before = {k: before.get(k, (q, q)) for k in {(b, s // c.bs) for _, b, s in c.tokens()}}
    want = _bounds_now(c)
    for (b, j), (lo, hi) in want.items():
        l, h = _bound_at(c, b, j)
        assert torch.equal(l, lo) and torch.equal(h, hi), (b, j)
    assert int((c.bounds != 0.25).any(-1).any(-1).sum()) <= len(want) * c.Hkv
    return want


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("bs", [1, 8, 16, 64])
def test_bounds(layout, bs, dtype):
    at, n = [0, 5, 64, 100], [40, 90, 3, 64]
    c = Case("e2m1", layout, at, n, 2, 64, 256, bs=bs, dtype=dtype, seed=bs, bounds=True)
    c.append()
    _check_bytes(c)
    want = _check_bounds(c, {})
    # more tokens behind them widen the last blocks
    more = Case("e2m1", layout, [a + v for a, v in zip(at, n)], [1, 1, 70, 2], 2, 64, 256, bs=bs, dtype=dtype,
                seed=bs + 1)
    more.table, more.slots, more.kv, more.groups, more.bounds = c.table, c.slots, c.kv, c.groups, c.bounds
    if layout == "paged":                                # the pages of the new tokens
        used = set(c.table[c.table >= 0].tolist())
        free = iter(x for x in range(len(c.kv[0])) if x not in used)
        for b in range(4):
            for j in range(-(-(more.at[b] + more.n[b]) // bs)):
                if c.table[b, j] < 0:
                    c.table[b, j] = next(free)
    more.append()
    q = 0.25 * torch.ones(2, 64)
    more.before = {(b, s // bs): want.get((b, s // bs), (q, q)) for _, b, s in more.tokens()}
    for (b, j), (lo, hi) in _bounds_now(more).items():
        l, h = _bound_at(more, b, j)
        assert torch.equal(l, lo) and torch.equal(h, hi), (b, j)


@pytest.mark.parametrize("kind", ["e2m1", "bf16"])
def test_wide_tokens_and_16_byte_alignment(kind):
    """More scale groups a token than a CTA has threads; vectors and caches that
    begin 16 bytes past a 32-byte boundary."""
    c = Case(kind, "dense", [3, 0], [20, 5], 40, 128, 32, bs=16, seed=5, bounds=True)
    c.append()
    _check_bytes(c)
    _check_bounds(c, {})
    _check_read(c, torch.bfloat16, c.read())
    c = Case(kind, "paged", [3, 0], [20, 40], 2, 64, 64, bs=16, seed=6, bounds=True)

    def shifted(x):
        n = 16 // x.element_size()
        y = torch.empty(x.numel() + n, dtype=x.dtype, device="cuda")[n:].view(x.shape)
        assert y.data_ptr() % 32 == 16
        return y.copy_(x)
    c.kv = [shifted(x) for x in c.kv]
    x = [shifted(y) for y in c.x]
    c.x = x
    c.append()
    c.x = [y.cpu() for y in x]
    _check_bytes(c)
    _check_bounds(c, {})
    out = [shifted(torch.zeros(60, 2, 64, dtype=torch.bfloat16)) for _ in range(2)]
    _check_read(c, torch.bfloat16, c.read(k_out=out[0], v_out=out[1]))


def test_single_tokens_of_many_rows():
    """One token a row, more rows than CTAs: every run its own block."""
    B = 3000
    c = Case("e2m1", "paged", [i % 48 for i in range(B)], [1] * B, 2, 64, 48, bs=16, seed=7, bounds=True)
    c.append()
    _check_bytes(c)
    _check_bounds(c, {})
    _check_read(c, torch.bfloat16, c.read())


def test_special_values():
    """Zero groups, values that overflow the scale, infinities and NaN."""
    c = Case("e2m1", "dense", [0], [6], 1, 32, 8, dtype=torch.float32)
    x = torch.zeros(6, 1, 32)
    x[1, 0, :16] = 1e-30                                 # scale 0: reads back 0
    x[2, 0, 3] = 1e9                                     # saturates at 6 * 448 g
    x[3, 0, 5] = math.inf
    x[4, 0, 7] = math.nan
    x[5, 0, 0], x[5, 0, 1] = -0.0, -3.0
    c.x = [x, x.clone()]
    c.append()
    k, v = c.read(dtype=torch.float32)
    for i, y in enumerate((k.cpu()[:, 0], v.cpu()[:, 0])):
        top = 6 * 448 * float(c.g[i][0])
        assert y[0].abs().max() == 0 and y[1].abs().max() == 0
        assert abs(float(y[2, 3]) - top) <= 2.0 ** -23 * top and float(y[2, :16].abs().sum()) == float(y[2, 3])
        assert abs(float(y[3, 5]) - top) <= 2.0 ** -23 * top
        assert torch.isnan(y[4, :16]).all() and torch.equal(y[4, 16:], torch.zeros(16))
        assert float(y[5, 0]) == 0.0 and abs(float(y[5, 1]) + 3.0) <= 3.0 / 16
    c = Case("e4m3", "dense", [0], [2], 1, 32, 8, dtype=torch.float32)
    c.x = [torch.full((2, 1, 32), 1e9), torch.full((2, 1, 32), math.nan)]
    c.append()
    k, v = c.read(dtype=torch.float32)
    assert torch.equal(k.cpu(), torch.full((2, 1, 32), 448.0) * c.g[0]) and torch.isnan(v).all()
    assert math.isnan(float(e4m3_values()[127]))


@pytest.mark.parametrize("kind", ["e2m1", "bf16"])
def test_padding_is_left_alone(kind):
    """Packed rows behind the last sequence: not written to the cache, not overwritten by a read."""
    c = Case(kind, "dense", [0, 4], [3, 5], 2, 64, 16, seed=1, pad=9)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.append(status=st)
    _check_bytes(c)
    ko, vo = (torch.full((17, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    got = c.read(k_out=ko, v_out=vo, status=st)
    assert got[0] is ko and got[1] is vo and int(st) == 0
    _check_read(c, torch.bfloat16, got)
    assert bool((ko[8:] == 7).all()) and bool((vo[8:] == 7).all())


def test_bad_content():
    c = Case("e2m1", "paged", [0, 10, 20], [20, 5, 4], 2, 64, 64, bs=16, seed=2, bounds=True)
    good = c.table.clone()
    c.table[0, 1] = -1                                   # tokens 16 .. 19 of row 0
    c.lengths[1] = 62                                    # 5 tokens do not fit
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.append(status=st)
    assert int(st) == 1 | 4
    st.zero_()
    k, v = c.read(status=st)
    assert int(st) == 1 | 4
    assert torch.isnan(k[16:25]).all() and torch.isfinite(k[:16]).all() and torch.isfinite(k[25:]).all()
    c.n, c.at = [16, 0, 4], [0, 10, 20]
    c.table = good
    c.x = [torch.cat([y[:16], y[25:]]) for y in c.x]
    c.cu = torch.tensor([0, 16, 16, 20], dtype=torch.int32)
    _check_bytes(c)
    # slot id out of range, offsets outside the packed rows
    c = Case("bf16", "slots", [0, 0], [2, 2], 1, 64, 8, seed=3)
    c.slots[0] = 5
    st.zero_()
    c.append(status=st)
    assert int(st) == 2 and float(c.kv[0][int(c.slots[1])].abs().sum()) > 0
    assert float(c.kv[0].abs().sum()) == float(c.kv[0][int(c.slots[1])].abs().sum())
    c = Case("bf16", "dense", [0, 0], [2, 2], 1, 64, 8, seed=3)
    c.cu = torch.tensor([0, 2, 99], dtype=torch.int32)
    st.zero_()
    c.append(status=st)
    assert int(st) == 32 and float(c.kv[0][1].abs().sum()) == 0 and float(c.kv[0][0].abs().sum()) > 0


@pytest.mark.parametrize("cu", [[0, 5, 3, 8], [0, 8, 8, 7], [0, 4, -1, 8]])
def test_decreasing_offsets_are_reported(cu):
    """A row whose offsets decrease has no token that could tell."""
    import gqa_kv_cache_gb300 as gqa
    x = torch.zeros(8, 2, 64, dtype=torch.bfloat16, device="cuda")
    kv = [torch.zeros(3, 2, 32, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    at = [torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 0, 0], cu)]
    for call in (lambda st: gqa.append(x, x, *kv, *at, status=st), lambda st: gqa.read(*kv, *at, 8, status=st)):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        call(st)
        assert int(st) == 32


def test_graph_and_stream():
    c = Case("e2m1", "dense", [0, 7], [30, 9], 2, 128, 64, seed=6, bounds=False)
    c.append()
    want = [x.clone() for x in (*c.kv, *c.groups)]
    k0, v0 = c.read()
    for x in (*c.kv, *c.groups):
        x.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.append(stream=side)
    k1, v1 = c.read(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (*c.kv, *c.groups)))
    assert torch.equal(k0, k1) and torch.equal(v0, v1)


def test_offsets_past_32_bits():
    """Elements of a cache beyond 2^32."""
    D, Hkv, Smax, R = 128, 8, 1 << 20, 5
    c = Case("e4m3", "dense", [Smax - 3], [3], Hkv, D, 16, seed=8)
    c.kv = [torch.empty(R, Hkv, Smax, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
    assert c.kv[0].numel() > 2 ** 32
    c.slots = torch.tensor([R - 1], dtype=torch.int32)
    c.append()
    k, v = c.read(dtype=torch.float32)
    for i, y in enumerate((k, v)):
        want = (c.x[i].float() / c.g[i].view(-1, 1)).clamp(-448, 448).to(torch.float8_e4m3fn).float() * c.g[i].view(-1, 1)
        assert torch.equal(y.cpu(), want)


def test_empty_calls():
    c = Case("bf16", "dense", [0], [0], 1, 64, 8)
    c.append()
    k, v = c.read()
    assert k.shape == (0, 1, 64) and float(c.kv[0].abs().sum()) == 0


def test_refusals():
    import gqa_kv_cache_gb300 as gqa
    c = Case("e2m1", "dense", [0], [2], 2, 64, 8)
    a = [x.cuda() for x in c.x] + c.kv
    ln, cu = c.lengths.cuda(), c.cu.cuda()
    with pytest.raises(gqa.GqaError):                    # no head scales
        gqa.append(*a, ln, cu, k_group_scale=c.groups[0], v_group_scale=c.groups[1])
    with pytest.raises(TypeError):                       # cu_q of another length
        gqa.append(*a, ln, cu[:1], **c.scales())
    with pytest.raises(TypeError):                       # cu_q of another type
        gqa.append(*a, ln, cu.long(), **c.scales())
    with pytest.raises(TypeError):                       # vectors of a type that is not taken
        gqa.append(a[0].half(), a[1].half(), *c.kv, ln, cu, **c.scales())
    with pytest.raises(ValueError):                      # vectors of other heads
        gqa.append(a[0][:, :1].contiguous(), a[1][:, :1].contiguous(), *c.kv, ln, cu, **c.scales())
    with pytest.raises(ValueError):                      # on the host
        gqa.append(c.x[0], c.x[1], *c.kv, ln, cu, **c.scales())
    with pytest.raises(ValueError):                      # a strided cache
        gqa.append(a[0], a[1], c.kv[0][:, :, ::2], c.kv[1][:, :, ::2], ln, cu, **c.scales())
    with pytest.raises(TypeError):                       # bounds of another type
        gqa.append(*a, ln, cu, k_bounds=torch.zeros(1, 2, 1, 2, 64, device="cuda"), **c.scales())
    with pytest.raises(ValueError):                      # blocks that do not divide the capacity
        gqa.append(*a, ln, cu, k_bounds=torch.zeros(1, 2, 3, 2, 64, dtype=torch.bfloat16, device="cuda"), **c.scales())
    with pytest.raises(TypeError):                       # an output type that is not offered
        gqa.read(*c.kv, ln, cu, 2, dtype=torch.float16, **c.scales())
    with pytest.raises(ValueError):                      # an output of another shape
        gqa.read(*c.kv, ln, cu, 2, k_out=torch.empty(3, 2, 64, dtype=torch.bfloat16, device="cuda"), **c.scales())
    b = Case("bf16", "dense", [0], [2], 1, 24, 8)        # D not a multiple of 16
    with pytest.raises(gqa.GqaError):
        b.append()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("cu,bad,free", [([0, 2, 99], [2, 3, 4, 5], []), ([1, 3, 7], [3, 4, 5], [0]),
                                         ([-2, 3, 5], [0, 1, 2], [5]), ([0, 2, 6], [], [])])
def test_read_of_a_row_with_bad_offsets_is_nan(cu, bad, free, kind, dtype):
    """A row whose offsets leave the packed tokens: its tokens among them read as
    NaN, those of no row are left as they were, the others are right."""
    c = Case(kind, "dense", [0, 0], [3, 3], 2, 64, 8, dtype=dtype, seed=9)
    c.append()
    c.cu = torch.tensor(cu, dtype=torch.int32)
    out = [torch.full((6, 2, 64), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.read(dtype=dtype, k_out=out[0], v_out=out[1], status=st)
    assert int(st) == (32 if bad else 0)
    for i, y in enumerate(out):
        vals = cache_values(kind, c.kv[i].cpu(), None if c.groups[i] is None else c.groups[i].cpu(), c.g[i])
        for t in range(6):
            if t in free:
                assert bool((y[t] == 7).all()), t
            elif t in bad:
                assert bool(torch.isnan(y[t]).all()), t
            else:
                b = max(x for x in range(2) if cu[x] <= t)
                want = vals[b, :, t - cu[b]]
                tol = want.abs() * (torch.finfo(dtype).eps / 2 + 2.0 ** -24) * (1 + 2.0 ** -8)
                assert bool(((y[t].double().cpu() - want).abs() <= tol).all()), t


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", ["e4m3", "e2m1"])
@pytest.mark.parametrize("D", [64, 128])
def test_negative_zeros_keep_their_sign(D, kind, dtype):
    """-0.0 is stored as -0, whatever the group's other values, and by the decode step as by append."""
    import gqa_kv_cache_gb300 as gqa
    B, Hkv = 6, 2
    c = Case(kind, "dense", [0] * B, [1] * B, Hkv, D, 16, dtype=dtype, seed=D)
    for x in c.x:
        x[:, :, ::3] = -0.0
        x[1, :, 16:32] = -0.0                            # a group of nothing else: scale 0
        x[2, :, 17] = -1e9                               # past the largest scale
        x[3] *= 1e-3                                     # scales near E4M3's smallest
        x[4, :, :16] = 0.0
        x[4, :, 5] = -0.0
    c.append()
    _check_bytes(c)
    if kind == "e2m1" and dtype == torch.bfloat16:
        kv, gs = [torch.zeros_like(x) for x in c.kv], [torch.zeros_like(x) for x in c.groups]
        q = torch.zeros(B, 2 * Hkv, D, dtype=dtype, device="cuda")
        gqa.decode_step(q, c.x[0].cuda(), c.x[1].cuda(), *kv, c.lengths.cuda(), k_scale=c.g[0].cuda(),
                        v_scale=c.g[1].cuda(), k_group_scale=gs[0], v_group_scale=gs[1])
        assert all(torch.equal(a, b) for a, b in zip(kv + gs, c.kv + c.groups))


@pytest.mark.parametrize("g", [1e-34, 1e30])
def test_negative_zeros_under_extreme_scales(g):
    c = Case("e2m1", "dense", [0], [4], 1, 32, 8, dtype=torch.float32, seed=3)
    c.g = [torch.tensor([g], dtype=torch.float32)] * 2
    c.x = [x * (100 * g) for x in c.x]
    for x in c.x:
        x[:, :, ::3] = -0.0
    c.append()
    _check_bytes(c)
