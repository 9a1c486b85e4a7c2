"""The 8-bit cache with block scales: writing, reading, attending, decoding.

Codes and scales are compared exactly (the format is float32 arithmetic rounded
to nearest even); values read back are one float32 product, rounded once."""
import math

import pytest
import torch

import gqa_kv_cache_gb300 as gqa
import serve_reference as R

pytestmark = pytest.mark.gpu


class Case:
    """An 8-bit cache written by the definition (CPU) and by the library."""

    def __init__(self, layout, B, Hkv, D, Smax, bs, held, seed=0):
        self.gen = torch.Generator().manual_seed(seed)
        shape, self.table, self.slots = R.layout_of(layout, B, Hkv, Smax, bs, self.gen, held)
        self.B, self.Hkv, self.D, self.bs, self.Smax = B, Hkv, D, bs, Smax
        self.k, self.v = (R.Cache8(shape, D, bs, self.table, self.slots) for _ in range(2))
        self.gk, self.gv = self.k.codes.cuda(), self.v.codes.cuda()
        self.kw = dict(k_block_scale=self.k.scale.cuda(), v_block_scale=self.v.scale.cuda())
        self.lens = [0] * B

    def index(self):
        return dict(block_table=self.table.cuda()) if self.table is not None else \
            dict(slot_ids=None if self.slots is None else self.slots.cuda())

    def _call(self, name, *args, **kw):
        i = self.index()
        if self.table is not None:
            return getattr(gqa, name + "_paged")(*args[:4], i["block_table"], *args[4:], **self.kw, **kw)
        return getattr(gqa, name)(*args, slot_ids=i["slot_ids"], **self.kw, **kw)

    def append(self, counts, dtype=torch.bfloat16, scale=1.0, pad=0, new=None, both=True):
        T = sum(counts)
        k, v = new if new is not None else ((torch.randn(T + pad, self.Hkv, self.D, generator=self.gen) * scale).to(dtype)
                                            for _ in range(2))
        cu = torch.tensor([sum(counts[:b]) for b in range(self.B + 1)], dtype=torch.int32)
        lens = torch.tensor(self.lens, dtype=torch.int32)
        for b, n in enumerate(counts):
            self.k.append(b, self.lens[b], k[int(cu[b]):int(cu[b]) + n].float())
            self.v.append(b, self.lens[b], v[int(cu[b]):int(cu[b]) + n].float())
        if both:
            self._call("append", k.cuda(), v.cuda(), self.gk, self.gv, lens.cuda(), cu.cuda())
        self.lens = [a + n for a, n in zip(self.lens, counts)]
        return k, v

    def same(self):
        for ref, codes, scale in ((self.k, self.gk, "k_block_scale"), (self.v, self.gv, "v_block_scale")):
            assert torch.equal(self.kw[scale].cpu().nan_to_num(nan=-1.0), ref.scale.nan_to_num(nan=-1.0))
            assert torch.equal(codes.cpu(), ref.codes)

    def read(self, dtype, T, start, counts, **kw):
        cu = torch.tensor([sum(counts[:b]) for b in range(self.B + 1)], dtype=torch.int32).cuda()
        lens = torch.tensor(start, dtype=torch.int32).cuda()
        if self.table is not None:
            return gqa.read_paged(self.gk, self.gv, self.table.cuda(), lens, cu, T, dtype=dtype, **self.kw, **kw)
        return gqa.read(self.gk, self.gv, lens, cu, T, None if self.slots is None else self.slots.cuda(), dtype=dtype,
                        **self.kw, **kw)

    def attend(self, q, n, **kw):
        n = torch.tensor(n, dtype=torch.int32).cuda()
        return self._call("attend", q, self.gk, self.gv, n, **kw) if self.table is None else \
            gqa.attend_paged(q, self.gk, self.gv, self.table.cuda(), n, **self.kw, **kw)


@pytest.mark.parametrize("layout", ["dense", "slots", "paged"])
@pytest.mark.parametrize("D,bs,dtype", [(128, 16, torch.bfloat16), (64, 8, torch.float32), (16, 24, torch.bfloat16),
                                        (48, 32, torch.float32), (256, 64, torch.bfloat16), (128, 1, torch.bfloat16)])
def test_prompts_then_tokens(layout, D, bs, dtype):
    Smax = -(-300 // bs) * bs
    c = Case(layout, 4, 3, D, Smax, bs, [Smax] * 4, seed=D + bs)
    c.append([0, 1, bs + 3, 70], dtype, pad=2)
    c.same()
    for scale in (0.5, 1.0, 3.0, 40.0, 1.0, 700.0):
        c.append([1, 0, 2, 1], dtype, scale)
        c.same()
    c.append([bs, 3 * bs + 1, 1, 0], dtype)
    c.same()
    n = c.lens
    k, v = c.read(torch.float32, sum(n) + 1, [0] * 4, n)
    at = 0
    for b in range(4):
        assert torch.equal(k[at:at + n[b]].cpu().double(), c.k.row(b, n[b]).float().double().transpose(0, 1)) if n[b] else True
        assert torch.equal(v[at:at + n[b]].cpu().double(), c.v.row(b, n[b]).float().double().transpose(0, 1)) if n[b] else True
        at += n[b]
    k16, _ = c.read(torch.bfloat16, sum(n) + 1, [0] * 4, n)
    assert torch.equal(k16[:sum(n)], k[:sum(n)].bfloat16())


def test_zeros_tiny_huge_and_values_that_are_not_finite():
    c = Case("paged", 1, 1, 64, 128, 16, [128])
    z = torch.zeros(4, 1, 64)
    c.append([4], torch.float32, new=(z, z))                  # a block of zeros: scale 0 ...
    c.same()
    c.append([2], torch.float32, scale=1.0)                   # ... takes the next tokens' scale
    c.same()
    c.append([10], torch.float32, scale=1e-42)
    c.append([3], torch.float32, scale=1e-42)                 # a subnormal scale
    c.same()
    c.append([3], torch.float32, scale=1e36)                  # 2^260 times as much: the earlier codes are 0
    c.same()
    c.append([10], torch.float32)
    x = torch.randn(4, 1, 64, generator=c.gen)
    y = x.clone()
    y[2, 0, 5] = math.inf
    c.append([4], torch.float32, new=(y, x))
    c.same()
    k, v = c.read(torch.float32, 4, [32], [4])
    assert k.isnan().all() and v.isfinite().all()
    c.append([4], torch.float32)                              # the block's scale stays NaN
    c.same()
    assert c.read(torch.float32, 8, [32], [8])[0].isnan().all()
    c.append([8], torch.float32)
    c.append([1], torch.float32, scale=3e38 / 6)
    c.same()


def test_a_block_written_again():
    """A row cut back and written again: the scale starts afresh where a block does."""
    c = Case("dense", 1, 2, 128, 64, 16, [64])
    c.append([40], scale=9.0)
    c.lens = [16]
    c.append([20], scale=0.1)
    c.same()
    c.lens = [18]
    c.append([1], scale=0.1)
    c.same()


def test_growth_error_stays_under_a_step():
    """Tokens that double in size one by one: every value is within a step of the block's final scale."""
    c = Case("dense", 1, 1, 64, 16, 16, [16])
    xs = []
    for i in range(16):
        x = torch.randn(1, 1, 64, generator=c.gen) * 1.3 ** i
        c.append([1], torch.float32, new=(x, x))
        xs.append(x)
    c.same()
    k, _ = c.read(torch.float32, 16, [0], [16])
    step = float(c.kw["k_block_scale"][0, 0, 0])
    assert (k.cpu() - torch.cat(xs)).abs().max() <= step * (1 + 2.0 ** -10)


def test_bad_rows_write_nothing():
    c = Case("paged", 3, 2, 64, 64, 16, [64] * 3)
    c.table[1, 1] = -1
    k, v = (torch.randn(60, 2, 64).bfloat16().cuda() for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 20, 40, 60], dtype=torch.int32).cuda()
    gqa.append_paged(k, v, c.gk, c.gv, c.table.cuda(), torch.tensor([50, 0, 10], dtype=torch.int32).cuda(), cu, status=status,
                     **c.kw)
    assert int(status) == 1 | 4
    c.k.append(2, 10, k[40:].float().cpu())
    c.v.append(2, 10, v[40:].float().cpu())
    c.k.append(1, 0, k[20:36].float().cpu())                  # the tokens of the usable block
    c.v.append(1, 0, v[20:36].float().cpu())
    c.same()


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cu,T", [([0, 5, 3, 8], 8), ([0, 8, 8, 7], 8), ([0, 4, -1, 8], 8), ([0, 10] * 24 + [0], 10),
                                  ([0, 5000] * 160, 5000), ([0, 700, 0, 700, 20, 5000] * 40, 5000),
                                  ([0] + [5000, 4990] * 300, 5000)])
def test_decreasing_offsets_are_reported(cu, T, paged, dtype):
    """Rows whose offsets fall and rise again name more runs than there are tokens: reported, and nothing but
    the rows' own slots is written."""
    B, bs, S = len(cu) - 1, 16, 5008
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, 2, 16, generator=g).to(dtype).cuda()
    spare = 2 * (S // bs) if paged else 2
    # all rows in the same cache row (what they write there is undefined), the others must stay as they are
    codes = [torch.full((spare, 2, bs, 16) if paged else (spare, 2, S, 16), 77, dtype=torch.int8, device="cuda")
             for _ in range(2)]
    scales = [torch.full((spare, 2) if paged else (spare, 2, S // bs), 3.0, device="cuda") for _ in range(2)]
    kw = dict(k_block_scale=scales[0], v_block_scale=scales[1])
    at = [torch.zeros(B, dtype=torch.int32, device="cuda"), torch.tensor(cu, dtype=torch.int32, device="cuda")]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if paged:
        table = torch.arange(S // bs, dtype=torch.int32, device="cuda").expand(B, -1).contiguous()
        gqa.append_paged(x, x, *codes, table, *at, status=status, **kw)
    else:
        gqa.append(x, x, *codes, *at, torch.zeros(B, dtype=torch.int32, device="cuda"), status=status, **kw)
    assert int(status) == 32
    half = spare // 2
    blocks = -(-T // bs)
    for c, s in zip(codes, scales):
        assert (c[half:] == 77).all() and (s[half:] == 3).all()
        assert ((c[blocks:half] == 77).all() and (s[blocks:half] == 3).all()) if paged else \
            ((c[0, :, blocks * bs:] == 77).all() and (s[0, :, blocks:] == 3).all())


# ---- attention ----

def _expect(c, q, n, window=0, prefix=0, sink=None):
    """Outputs, their tolerance."""
    B, Hq, D = q.shape
    outs, tols = [], []
    for b in range(B):
        k, v = c.k.row(b, n[b]), c.v.row(b, n[b])
        ok = R.attended(n[b], window, prefix)
        s = None if sink is None else sink.cpu().view(c.Hkv, -1)
        o, w, e = R.attention(q[b].double().cpu().view(c.Hkv, -1, D), k, v, ok=ok, sink=s)
        outs.append(o.reshape(Hq, D))
        tols.append(R.out_tolerance(w, e, float(v[:, ok].abs().max())))
    return torch.stack(outs), torch.stack(tols)


def _close(got, want, tol):
    err = (got.cpu().double() - want).abs().amax((1, 2))
    assert (err <= tol).all(), (err / tol).tolist()


@pytest.mark.parametrize("layout", ["dense", "slots", "paged"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 3, 4, 5, 8])
@pytest.mark.parametrize("qt", [torch.bfloat16, torch.float32])
def test_attend(layout, D, G, qt):
    bs = {"dense": 32, "slots": 24, "paged": 16}[layout]
    lens = [1, 15, 17, 64, 129, 300, 1151]
    c = Case(layout, 7, 2, D, 1152, bs, lens, seed=G)
    c.append(lens)
    q = torch.randn(7, 2 * G, D, generator=c.gen).to(qt).cuda()
    want, tol = _expect(c, q, lens)
    for grid in (0, 1, 3, 40):
        _close(c.attend(q, lens, grid_ctas=grid), want, tol)
    sink = torch.randn(2 * G, generator=c.gen).cuda()
    for kw in (dict(window=40), dict(window=40, kept_prefix=5), dict(sink=sink), dict(window=1, kept_prefix=33, sink=sink)):
        want, tol = _expect(c, q, lens, kw.get("window", 0), kw.get("kept_prefix", 0), kw.get("sink"))
        for grid in (0, 5):
            _close(c.attend(q, lens, grid_ctas=grid, **kw), want, tol)


@pytest.mark.parametrize("bs", [8, 16, 24, 64, 128])
def test_attend_page_sizes(bs):
    lens = [1, bs, bs + 1, 5 * bs - 1, 777]
    c = Case("paged", 5, 2, 128, -(-777 // bs) * bs, bs, lens, seed=bs)
    c.append(lens)
    q = torch.randn(5, 12, 128, generator=c.gen).bfloat16().cuda()
    want, tol = _expect(c, q, lens)
    _close(c.attend(q, lens), want, tol)


@pytest.mark.parametrize("G", [2, 8])
def test_scales_far_apart(G):
    """Blocks whose scales differ by many octaves, in both directions, and blocks of zeros."""
    n = 16 * 24
    c = Case("paged", 2, 1, 64, n, 16, [n, n], seed=5)
    for j in range(24):
        size = [1.0, 1e-9, 300.0, 0.0, 1e5, 1e-20, 7.0, 1e12][j % 8]
        k = torch.randn(32, 1, 64, generator=c.gen).bfloat16()
        v = (torch.randn(32, 1, 64, generator=c.gen) * (size if j else 0.0)).bfloat16()
        c.append([16, 16], new=(k, v))
    c.same()
    q = torch.randn(2, G, 64, generator=c.gen).cuda()
    want, tol = _expect(c, q, [n, n])
    _close(c.attend(q, [n, n]), want, tol)
    for first in (16, 32, 64):                                # short rows: small scales alone
        want, tol = _expect(c, q, [first, first])
        _close(c.attend(q, [first, first]), want, tol + 1e-30)


def test_what_is_not_attended_does_not_matter():
    """NaN scales and any codes behind the row's end, before its window, and in unused blocks."""
    lens = [37, 70]
    c = Case("paged", 2, 2, 128, 96, 16, lens, seed=6)
    c.append(lens)
    q = torch.randn(2, 8, 128, generator=c.gen).bfloat16().cuda()
    want, tol = _expect(c, q, lens, window=20)
    used = torch.zeros(c.gk.shape[0], dtype=torch.bool)
    for b, n in enumerate(lens):
        used[c.table[b, (n - 20) // 16:-(-n // 16)].long()] = True
    for t in c.kw.values():
        t[~used.cuda()] = math.nan
    c.gk[~used.cuda()] = 127
    c.table[:, 0] = -1
    _close(c.attend(q, lens, window=20), want, tol)
    d = Case("dense", 1, 1, 64, 64, 16, [33])
    d.append([33])
    q = torch.randn(1, 2, 64, generator=d.gen).cuda()
    want, tol = _expect(d, q, [33])
    for t in d.kw.values():
        t[0, 0, 3] = math.nan
    _close(d.attend(q, [33]), want, tol)
    for t in d.kw.values():
        t[0, 0, 0] = math.nan
    assert d.attend(q, [33]).isnan().all()


@pytest.mark.parametrize("layout", ["dense", "slots", "paged"])
@pytest.mark.parametrize("D,Hkv,G", [(128, 2, 4), (64, 1, 7)])
def test_decode_step(layout, D, Hkv, G):
    lens = [0, 1, 15, 16, 200]
    c = Case(layout, 5, Hkv, D, 224, 16, [n + 1 for n in lens], seed=7)
    c.append(lens, scale=0.5)
    for _ in range(3):
        q = torch.randn(5, Hkv * G, D, generator=c.gen).bfloat16()
        at = torch.tensor(c.lens, dtype=torch.int32).cuda()
        if c.table is not None and any(n % 16 == 0 and c.table[b, n // 16] < 0 for b, n in enumerate(c.lens)):
            break
        k, v = c.append([1] * 5, scale=2.0, both=False)
        if c.table is None:
            out = gqa.decode_step(q.cuda(), k.cuda(), v.cuda(), c.gk, c.gv, at, None if c.slots is None else c.slots.cuda(),
                                  **c.kw)
        else:
            out = gqa.decode_step_paged(q.cuda(), k.cuda(), v.cuda(), c.gk, c.gv, c.table.cuda(), at, **c.kw)
        c.same()
        want, tol = _expect(c, q, c.lens)
        _close(out, want, tol)


def test_bad_rows_give_nan():
    c = Case("paged", 4, 1, 64, 64, 16, [64] * 4)
    c.append([40, 40, 40, 40])
    c.table[1, 1] = -1
    c.table[2, 0] = 10 ** 6
    q = torch.randn(4, 2, 64).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for n, bits in (([40, 40, 40, 65], 5), ([40, 40, 40, 0], 5)):
        out = c.attend(q, n, status=status)
        assert out[0].isfinite().all() and out[1:].isnan().all() and int(status) == bits
    ws = gqa.workspace_bytes(4, 2, 1, 64, torch.int8)
    buf = torch.zeros(ws, dtype=torch.uint8, device="cuda")
    for grid in (0, 7):
        c.attend(q, [40, 40, 40, 65], workspace=buf, grid_ctas=grid and 2)
        assert not buf.any()


def test_refusals():
    c = Case("dense", 2, 2, 128, 64, 16, [64, 64])
    c.append([20, 20])
    q, n = torch.zeros(2, 4, 128, device="cuda"), torch.tensor([20, 20], dtype=torch.int32).cuda()
    new = q[:, :2].contiguous()
    ks, vs = c.kw["k_block_scale"], c.kw["v_block_scale"]

    def attend(**kw):
        return gqa.attend(q, c.gk, c.gv, n, **{**c.kw, **kw})

    for bad in (dict(k_block_scale=None), dict(v_block_scale=vs.double()), dict(k_scale=ks[:, 0, 0]),
                dict(k_group_scale=c.gk, v_group_scale=c.gk)):
        with pytest.raises(TypeError):
            attend(**bad)
    for bad in (dict(k_block_scale=ks[:, :1]), dict(k_block_scale=ks[..., :3].contiguous()), dict(v_block_scale=vs.cpu()),
                dict(k_block_scale=ks.expand(2, 2, 4).transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises(ValueError):
            attend(**bad)
    with pytest.raises(TypeError):                            # block scales of another kind of cache
        gqa.attend(q, c.gk.bfloat16(), c.gv.bfloat16(), n, **c.kw)
    with pytest.raises(TypeError):
        gqa.append(new, new, c.gk.bfloat16(), c.gv.bfloat16(), n, n.new_tensor([0, 1, 2]), **c.kw)
    with pytest.raises(gqa.GqaError):
        attend(kernel="simt")
    with pytest.raises(gqa.GqaError):                         # key bounds are not kept for it
        gqa.append(new, new, c.gk, c.gv, n, n.new_tensor([0, 1, 2]), **c.kw,
                   k_bounds=torch.zeros(2, 2, 4, 2, 128, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError):
        gqa.decode_step(q, new, new, c.gk, c.gv, n, **c.kw)
    with pytest.raises(TypeError):
        gqa.decode_multi(q.bfloat16(), new.bfloat16(), new.bfloat16(), c.gk, c.gv, n, n.new_tensor([0, 1, 2]), max_q_len=1)
    with pytest.raises(gqa.GqaError):
        gqa.attend(torch.zeros(2, 18, 128, device="cuda"), c.gk, c.gv, n, **c.kw)
