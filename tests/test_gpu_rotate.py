"""Rotary positions against the 64-bit definition.

Tolerance. cos and sin are off by less than 2^-23 (the angle's rest is a 30-bit
integer rounded to float32: 2^-26 of a quarter turn; sincospif: 2 steps; the
factor: one), the two products and their sum by three roundings of 2^-24: in
all under 6 2^-24 (|x| + |y|) m; the result is rounded once to its type."""
import math

import pytest
import torch

import gqa_kv_cache_gb300 as gqa
import serve_reference as R

pytestmark = pytest.mark.gpu
BANDS = dict(kind="bands", factor=8.0, original=8192, low=1.0, high=4.0, attention=1.25)


def _check(got, x, positions, dim, base, layout, scaling):
    want = R.rotate(x.cpu(), positions.cpu(), dim, base, layout, scaling)
    m = (scaling or {}).get("attention", 1.0)
    big = x.cpu().double().abs().amax(-1, keepdim=True) * 2 * m
    tol = 6 * 2.0 ** -24 * big + torch.finfo(x.dtype).eps / 2 * want.abs() * (1 + 2.0 ** -8)
    err = (got.cpu().double() - want).abs()
    assert (err <= tol).all(), float((err / tol).max())
    assert torch.equal(got[..., dim:].cpu(), x[..., dim:].cpu())


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,Hq,Hkv,D,dim", [(1, 8, 2, 128, 128), (7, 6, 1, 64, 40), (33, 3, 3, 128, 64), (5, 1, 1, 16, 2),
                                            (2000, 5, 1, 128, 104), (3, 2, 2, 96, 96), (4, 1, 2, 10, 6)])
def test_against_the_definition(T, Hq, Hkv, D, dim, dtype, layout):
    g = torch.Generator().manual_seed(T * 131 + D)
    q, k = torch.randn(T, Hq, D, generator=g).to(dtype).cuda(), torch.randn(T, Hkv, D, generator=g).to(dtype).cuda()
    pos = torch.randint(-5, 200000, (T,), generator=g).int().cuda()
    pos[0] = 2 ** 31 - 1
    for scaling in (None, BANDS):
        rot = gqa.Rotary(dim, layout=layout, scaling=scaling)
        a, b = gqa.rotate(q, k, rot, pos)
        _check(a, q, pos, dim, 10000.0, layout, scaling)
        _check(b, k, pos, dim, 10000.0, layout, scaling)


@pytest.mark.parametrize("scaling", [dict(kind="linear", factor=4.0), dict(kind="linear", factor=0.05),
                                     dict(kind="ntk", factor=8.0), BANDS])
def test_scaling(scaling):
    g = torch.Generator().manual_seed(1)
    q = torch.randn(64, 2, 128, generator=g).cuda()
    pos = torch.arange(64).mul(1999).int().cuda()
    a, none = gqa.rotate(q, None, gqa.Rotary(128, base=500000.0, scaling=scaling), pos)
    assert none is None
    _check(a, q, pos, 128, 500000.0, "half", scaling)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("shift", [0, 1, 8])
def test_parts_of_a_projection_and_in_place(layout, shift):
    """q and k as views of one tensor (16-byte aligned or not), turned in place; the rest stays."""
    T, Hq, Hkv, D = 19, 4, 2, 64
    g = torch.Generator().manual_seed(2)
    flat = torch.randn(T, (Hq + 2 * Hkv) * D + 8 + shift, generator=g).bfloat16().cuda()
    before = flat.clone()
    q = flat[:, shift:shift + Hq * D].view(T, Hq, D)
    k = flat[:, shift + Hq * D:shift + (Hq + Hkv) * D].view(T, Hkv, D)
    pos = torch.arange(T).int().cuda() * 77
    rot = gqa.Rotary(48, layout=layout)
    wq, wk = gqa.rotate(q, k, rot, pos)
    a, b = gqa.rotate(q, k, rot, pos, q_out=q, k_out=k)
    assert a is q and b is k
    assert torch.equal(wq, q) and torch.equal(wk, k)
    _check(wq, before[:, shift:shift + Hq * D].view(T, Hq, D), pos, 48, 10000.0, layout, None)
    keep = torch.ones_like(flat, dtype=torch.bool)
    keep[:, shift:shift + (Hq + Hkv) * D] = False
    assert torch.equal(flat[keep], before[keep])


def test_positions_of_rows():
    """lengths and cu_q in the place of positions; tokens of no row are copied, and bad offsets reported."""
    T, D = 12, 64
    g = torch.Generator().manual_seed(3)
    q = torch.randn(T, 2, D, generator=g).cuda()
    lengths = torch.tensor([5, 100, 0], dtype=torch.int32).cuda()
    cu = torch.tensor([0, 4, 4, 9], dtype=torch.int32).cuda()
    rot = gqa.Rotary(D)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    a, _ = gqa.rotate(q, None, rot, lengths=lengths, cu_q=cu, status=status)
    pos = torch.tensor([5, 6, 7, 8, 0, 1, 2, 3, 4, 0, 0, 0]).int().cuda()
    b, _ = gqa.rotate(q, None, rot, pos)
    assert torch.equal(a, b) and int(status) == 0
    assert torch.equal(a[9:], q[9:])
    bad = torch.tensor([0, 4, 4, 99], dtype=torch.int32).cuda()
    a, _ = gqa.rotate(q, None, rot, lengths=lengths, cu_q=bad, status=status)
    assert int(status) == 32 and torch.equal(a[:4], b[:4]) and torch.equal(a[4:], q[4:])


def test_scores_depend_on_the_distance():
    """q at i and k at j: the product depends on i - j alone (to rounding), far positions among them."""
    g = torch.Generator().manual_seed(4)
    D = 128
    x, y = torch.randn(1, 1, D, generator=g).cuda(), torch.randn(1, 1, D, generator=g).cuda()
    rot = gqa.Rotary(D)
    at = torch.tensor([0, 1000, 10 ** 6, 2 ** 30], dtype=torch.int32).cuda()
    q, _ = gqa.rotate(x.expand(4, 1, D).contiguous(), None, rot, at + 17)
    k, _ = gqa.rotate(y.expand(4, 1, D).contiguous(), None, rot, at)
    s = (q.double() * k.double()).sum(-1).flatten()
    # the table's angles are 2^-65 of a turn off: at 2^30 2^-35 turns; products: D roundings of 8 2^-24 |x| |y|
    assert (s - s[0]).abs().max() <= 16 * 2.0 ** -24 * float(x.norm() * y.norm()) * math.sqrt(D)


@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_angles_of_far_positions(base):
    """cos and sin themselves (the pairs are (1, 0)) at positions of 31 bits, angles reduced in decimal.

    Tolerance: 2^-34 of a turn from the table and 2^-32 from its cut (2e-9 radians), 2.4e-8 from the rest of the
    angle in float32 (at most pi / 4), one step of sincospif (6e-8): 8.6e-8, under 2^-23."""
    import decimal
    dim = 128
    at = [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 12345, 2 ** 30 + 1, -(2 ** 30) - 77, 10 ** 9, 123456789, 0, 1]
    x = torch.zeros(len(at), 1, dim, device="cuda")
    x[..., :dim // 2] = 1
    got, _ = gqa.rotate(x, None, gqa.Rotary(dim, base=base), torch.tensor(at, dtype=torch.int32, device="cuda"))
    want = torch.empty(len(at), dim, dtype=torch.float64)
    with decimal.localcontext() as c:
        c.prec = 60
        two_pi = 2 * decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
        for i in range(dim // 2):
            turns = (-2 * i * decimal.Decimal(base).ln() / dim).exp() / two_pi
            for t, pos in enumerate(at):
                a = float((pos * turns) % 1 * two_pi)
                want[t, i], want[t, i + dim // 2] = math.cos(a), math.sin(a)
    assert (got[:, 0].cpu().double() - want).abs().max() <= 2.0 ** -23


def test_empty():
    rot = gqa.Rotary(64)
    q = torch.zeros(0, 2, 64, device="cuda")
    a, _ = gqa.rotate(q, None, rot, torch.zeros(0, dtype=torch.int32, device="cuda"))
    assert a.shape == (0, 2, 64)


def test_an_output_whose_tokens_or_heads_share_memory_is_refused():
    q = torch.zeros(4, 2, 64, device="cuda")
    pos, rot = torch.zeros(4, dtype=torch.int32, device="cuda"), gqa.Rotary(64)
    for out in (q[:1].expand(4, 2, 64), q[:, :1].expand(4, 2, 64)):
        with pytest.raises(ValueError):
            gqa.rotate(q, None, rot, pos, q_out=out)
    got = gqa.rotate(q[:1, :1].expand(4, 2, 64), None, rot, pos)[0]     # inputs may
    assert got.shape == q.shape and not got.any()


def test_refusals():
    q, k = torch.zeros(4, 2, 64, device="cuda"), torch.zeros(4, 1, 64, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    rot = gqa.Rotary(64)
    for bad in (lambda: gqa.rotate(None, None, rot, pos), lambda: gqa.rotate(q, k, gqa.Rotary(66), pos),
                lambda: gqa.rotate(q, k.bfloat16(), rot, pos), lambda: gqa.rotate(q, k[:3], rot, pos),
                lambda: gqa.rotate(q, k, rot), lambda: gqa.rotate(q, k, rot, pos, lengths=pos, cu_q=pos),
                lambda: gqa.rotate(q, None, rot, pos, k_out=k), lambda: gqa.rotate(q, k, rot, pos, q_out=q[:, :1]),
                lambda: gqa.rotate(q.cpu(), None, rot, pos),
                lambda: gqa.rotate(q.transpose(1, 2).contiguous().transpose(1, 2), None, rot, pos)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: gqa.rotate(q.half(), None, rot, pos), lambda: gqa.rotate(q, k, rot, pos.long()),
                lambda: gqa.rotate(q, k, rot, pos[:3])):
        with pytest.raises(TypeError):
            bad()
