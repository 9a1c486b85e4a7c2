"""Block selection against the 64-bit definition (ties, borders, NaN, forced
blocks, bad content) and the attention over the kept blocks; and a whole run:
prompts written with bounds, then steps of append, select and attend."""
import math

import pytest
import torch

from cache_reference import Problem, attend_tolerance, block_scores, select

pytestmark = pytest.mark.gpu


def _bounds(p):
    """Key bounds of a problem's cache over its valid slots, as append keeps them
    from keys that are exactly what the cache holds, rounded to bfloat16 outwards."""
    if p.table is not None:
        out = torch.zeros(p.kv[0].shape[0], p.Hkv, 2, p.D)
    else:
        out = torch.zeros(p.kv[0].shape[0], p.Hkv, -(-p.Smax // p.bs), 2, p.D)
    for b in range(p.B):
        k = p.row(b, 0).float()
        for j in range(-(-p.lens[b] // p.bs)):
            x = k[:, j * p.bs:(j + 1) * p.bs]
            v = torch.stack([x.amin(1), x.amax(1)], 1)
            if p.table is not None:
                out[int(p.table[b, j])] = v
            else:
                out[int(p.slots[b]) if p.slots is not None else b, :, j] = v
    return out.bfloat16()


def _bound(p, box, b, h):
    n = -(-p.lens[b] // p.bs)
    if p.table is not None:
        v = box[p.table[b, :n].long(), h]
    else:
        v = box[int(p.slots[b]) if p.slots is not None else b, h, :n]
    return v[:, 0], v[:, 1]


def _select(p, box, n, first=1, last=1, q=None, **kw):
    import gqa_kv_cache_gb300 as gqa
    q = (p.q if q is None else q).cuda()
    if p.table is not None:
        return gqa.select_blocks_paged(q, box.cuda(), p.table.cuda(), p.lengths.cuda(), n, block_size=p.bs,
                                       n_first=first, n_last=last, **kw)
    return gqa.select_blocks(q, box.cuda(), p.lengths.cuda(), n, None if p.slots is None else p.slots.cuda(),
                             block_size=p.bs, n_first=first, n_last=last, **kw)


def _want(p, box, n, first=1, last=1):
    G = p.Hq // p.Hkv
    ids = torch.full((p.B, p.Hkv, n), -1, dtype=torch.int32)
    for b in range(p.B):
        for h in range(p.Hkv):
            s = block_scores(p.q[b, h * G:(h + 1) * G], *_bound(p, box, b, h)).tolist()
            kept = select(s, n, first, last)
            ids[b, h, :len(kept)] = torch.tensor(kept, dtype=torch.int32)
    return ids


def _check_tables(p, sel, ids):
    """The table and the slot counts follow from the ids."""
    table, lens = sel.table.cpu().view(p.B, p.Hkv, -1), sel.lengths.cpu().view(p.B, p.Hkv)
    nb = -(-p.Smax // p.bs)
    for b in range(p.B):
        for h in range(p.Hkv):
            kept = [j for j in ids[b, h].tolist() if j >= 0]
            if p.table is not None:
                want = [int(p.table[b, j]) * p.Hkv + h for j in kept]
            else:
                r = int(p.slots[b]) if p.slots is not None else b
                want = [(r * p.Hkv + h) * nb + j for j in kept]
            assert table[b, h].tolist() == want + [-1] * (ids.shape[2] - len(kept))
            assert int(lens[b, h]) == sum(min(p.bs, p.lens[b] - j * p.bs) for j in kept)


def _attend(p, sel, t):
    import gqa_kv_cache_gb300 as gqa
    kw = {}
    if p.kind == "e2m1":
        kw = dict(k_scale=p.g[0].cuda(), v_scale=p.g[1].cuda(), k_group_scale=t[2], v_group_scale=t[3])
    return gqa.attend_selected(p.q.cuda(), t[0], t[1], sel, **kw)


def _check_attend(p, sel, ids, got=None):
    t = [x.cuda() if x is not None else None for x in (*p.kv, *p.groups)]
    got = (_attend(p, sel, t) if got is None else got).double().cpu()
    for b in range(p.B):
        slots = [[s for j in ids[b, h].tolist() if j >= 0 for s in range(j * p.bs, min((j + 1) * p.bs, p.lens[b]))]
                 for h in range(p.Hkv)]
        want, vmax, amax = p.expect(b, slots)
        # a bfloat16 cache's weights enter the products as 16 bits: another 2^-15
        tol = attend_tolerance(p.D, vmax, amax) + (2.0 ** -15 * vmax if p.kind == "bf16" else 0)
        assert float((got[b] - want).abs().max()) <= tol, b


@pytest.mark.parametrize("layout", ["dense", "slots", "paged"])
@pytest.mark.parametrize("kind,D,Hq,Hkv,q", [("e2m1", 128, 8, 2, torch.bfloat16), ("e2m1", 64, 3, 3, torch.float32),
                                             ("bf16", 128, 12, 2, torch.bfloat16), ("bf16", 64, 4, 2, torch.bfloat16),
                                             ("f32", 64, 4, 2, torch.float32)])
def test_select_and_attend(layout, kind, D, Hq, Hkv, q):
    p = Problem(kind, layout, [1, 16, 17, 500, 1000, 1024], Hq, Hkv, D, 1024, seed=D + Hq, q_dtype=q)
    box = _bounds(p)
    for n, first, last in ((6, 1, 1), (9, 0, 2), (64, 1, 1), (100, 2, 3)):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        sel = _select(p, box, n, first, last, status=st)
        ids = sel.ids.cpu()
        assert torch.equal(ids, _want(p, box, n, first, last)) and int(st) == 0
        _check_tables(p, sel, ids)
        _check_attend(p, sel, ids)


@pytest.mark.parametrize("bs,n_blocks", [(8, 3000), (64, 700), (16, 16384)])
def test_long_rows(bs, n_blocks):
    """Many blocks a row: every cluster size, the bounds drawn directly."""
    gen = torch.Generator().manual_seed(bs)
    for B, Hkv in ((1, 1), (3, 2)) if n_blocks < 16384 else ((1, 1),):
        p = Problem("bf16", "dense", [1] * B, 2 * Hkv, Hkv, 128, bs, bs=bs, seed=1)
        p.lens = [n_blocks * bs - 3 * b for b in range(B)]
        p.Smax = n_blocks * bs
        p.lengths = torch.tensor(p.lens, dtype=torch.int32)
        x = torch.randn(B, Hkv, n_blocks, 2, 128, generator=gen).sort(3).values.bfloat16()
        for n in (2, 65, 300):
            assert torch.equal(_select(p, x, n).ids.cpu(), _want(p, x, n))


@pytest.mark.parametrize("D,G,q", [(256, 3, torch.float32), (64, 16, torch.bfloat16), (256, 12, torch.bfloat16)])
def test_widths_and_wide_groups(D, G, q):
    """Selection alone, for head widths and group sizes that only some attends take."""
    p = Problem("f32", "slots", [700, 33, 1000], 2 * G, 2, D, 1008, seed=G, q_dtype=q)
    box = _bounds(p)
    for n, first, last in ((5, 0, 1), (20, 2, 2)):
        assert torch.equal(_select(p, box, n, first, last).ids.cpu(), _want(p, box, n, first, last))


@pytest.mark.parametrize("kind", ["e2m1", "bf16"])
def test_steps_without_waiting(kind):
    """Steps of append, select, attend and decode queued back to back give the
    bits of the same steps with a wait after every call."""
    import gqa_kv_cache_gb300 as gqa
    B, Hq, Hkv, D, bs, Smax, steps = 5, 8, 2, 128, 16, 2048, 60
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(steps, 3, B, Hkv, D, generator=gen, device="cuda").bfloat16()
    q = torch.randn(steps, B, Hq, D, generator=gen, device="cuda").bfloat16()
    pre = torch.randn(2, B * 700, Hkv, D, generator=gen, device="cuda").bfloat16()
    g = torch.full((Hkv,), 0.002, device="cuda")
    at = torch.tensor([[700 + 2 * i] * B for i in range(steps + 1)], dtype=torch.int32, device="cuda")
    zero, cu0 = torch.zeros(B, dtype=torch.int32, device="cuda"), (torch.arange(B + 1, device="cuda") * 700).int()
    cu = torch.arange(B + 1, device="cuda").int()
    one = torch.ones(B, dtype=torch.int32, device="cuda")
    now = [at[i] + one for i in range(steps)]
    torch.cuda.synchronize()

    def run(wait):
        row = D // 2 if kind == "e2m1" else D
        kv = [torch.zeros(B, Hkv, Smax, row, dtype=torch.uint8 if kind == "e2m1" else torch.bfloat16, device="cuda")
              for _ in range(2)]
        kw = {}
        if kind == "e2m1":
            gs = [torch.zeros(B, Hkv, Smax, D // 16, dtype=torch.uint8, device="cuda") for _ in range(2)]
            kw = dict(k_scale=g, v_scale=g, k_group_scale=gs[0], v_group_scale=gs[1])
        box = torch.zeros(B, Hkv, Smax // bs, 2, D, dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        outs = []

        def done(y):
            if wait:
                torch.cuda.synchronize()
            return y
        done(gqa.append(pre[0], pre[1], *kv, zero, cu0, k_bounds=box, **kw))
        for i in range(steps):
            done(gqa.append(x[i, 0], x[i, 1], *kv, at[i], cu, k_bounds=box, **kw))
            sel = done(gqa.select_blocks(q[i], box, now[i], 9, block_size=bs))
            outs.append(done(gqa.attend_selected(q[i], *kv, sel, **kw)))
            # the next slot's token by the decode step, its bounds by an append of the same
            outs.append(done(gqa.decode_step(q[i], x[i, 2], x[i, 1], *kv, now[i], **kw)))
            done(gqa.append(x[i, 2], x[i, 1], *kv, now[i], cu, k_bounds=box, **kw))
            outs.extend(done(gqa.read(*kv, at[i], cu, B, **kw)))
        torch.cuda.synchronize()
        return outs, kv
    a, ka = run(True)
    for _ in range(3):
        b, kb = run(False)
        assert all(torch.equal(u, v) for u, v in zip(a, b)) and all(torch.equal(u, v) for u, v in zip(ka, kb))


def test_ties_and_borders():
    """Equal scores go to the lowest index; scores that float32 cannot tell apart are told apart."""
    B, n_blocks, bs, D = 1, 200, 16, 128
    p = Problem("bf16", "dense", [1], 2, 1, D, bs, bs=bs, seed=2)
    p.lens, p.Smax = [n_blocks * bs], n_blocks * bs
    p.lengths = torch.tensor(p.lens, dtype=torch.int32)
    gen = torch.Generator().manual_seed(3)
    one = torch.randn(1, 1, 1, 2, D, generator=gen).sort(3).values.bfloat16()
    same = one.expand(B, 1, n_blocks, 2, D).contiguous()
    assert _select(p, same, 20).ids.cpu()[0, 0].tolist() == list(range(19)) + [n_blocks - 1]
    assert _select(p, torch.zeros_like(same), 7).ids.cpu()[0, 0].tolist() == list(range(6)) + [n_blocks - 1]
    few = same.clone()
    few[0, 0, [31, 77, 150]] = (one * 2).bfloat16()[0, 0]            # three higher or lower, the rest equal
    assert torch.equal(_select(p, few, 20).ids.cpu(), _want(p, few, 20))
    # a large term that cancels leaves differences far below float32's rounding of the sum
    close = torch.zeros(B, 1, n_blocks, 2, D)
    q = torch.zeros(1, 2, D)
    q[:, :, 0], q[:, :, 1], q[:, :, 2] = 1024.0, -1024.0, 2.0 ** -12
    close[..., 0] = 256.0
    close[..., 1] = 256.0
    close[..., 2] = torch.randperm(n_blocks, generator=gen).float()[None, None, :, None] / 256
    close = close.bfloat16()
    p.q = q.bfloat16()
    assert torch.equal(_select(p, close, 30).ids.cpu(), _want(p, close, 30))
    assert torch.equal(_select(p, close, 30, 0, 1).ids.cpu(), _want(p, close, 30, 0, 1))


def test_nan_and_infinite_bounds():
    n_blocks, bs, D = 90, 16, 64
    p = Problem("bf16", "dense", [1], 4, 1, D, bs, bs=bs, seed=4)
    p.lens, p.Smax = [n_blocks * bs - 1], n_blocks * bs
    p.lengths = torch.tensor(p.lens, dtype=torch.int32)
    x = torch.randn(1, 1, n_blocks, 2, D, generator=torch.Generator().manual_seed(5)).sort(3).values
    x[0, 0, 40, :, 3] = math.nan
    x[0, 0, 13, 1, 2] = math.inf
    x[0, 0, 60, 0, 2] = -math.inf
    x = x.bfloat16()
    for n in (4, 5, 30):
        assert torch.equal(_select(p, x, n).ids.cpu(), _want(p, x, n))
    p.q[0, 1, 5] = math.nan                              # every score NaN: the lowest indexes
    assert _select(p, x, 6).ids.cpu()[0, 0].tolist() == [0, 1, 2, 3, 4, n_blocks - 1]


@pytest.mark.parametrize("n", [3, 4, 6])
def test_scores_past_float32(n):
    """Finite bounds whose score, or only a part of its sum, leaves float32's range."""
    p = Problem("bf16", "dense", [40 * 16], 1, 1, 64, 40 * 16, seed=8)
    p.q = torch.ones(1, 1, 64, dtype=torch.bfloat16)
    x = torch.randn(1, 1, 40, 2, 64, generator=torch.Generator().manual_seed(4)).sort(3).values.bfloat16()
    x[0, 0, 9, 1, :2] = 3e38
    x[0, 0, 30, 1, 5:9] = 3e38
    x[0, 0, 17, 1, :2] = 2e38                            # 4e38 and then back to the lowest of all
    x[0, 0, 17, :, 4:33:28] = -3e38
    assert torch.equal(_select(p, x, n).ids.cpu(), _want(p, x, n))


def test_blocks_behind_the_row_never_matter():
    p = Problem("bf16", "paged", [100, 333], 4, 2, 128, 512, seed=6)
    box = _bounds(p)
    want = _select(p, box, 5).ids
    used = set(p.table[p.table >= 0].tolist())
    for j in range(len(box)):
        if j not in used:
            box[j] = math.nan
    assert torch.equal(_select(p, box, 5).ids, want)


def test_bad_content():
    import gqa_kv_cache_gb300 as gqa
    p = Problem("e2m1", "paged", [300, 200, 100, 50], 4, 2, 128, 320, seed=7)
    box = _bounds(p)
    good = _want(p, box, 4)
    p.table[1, 5] = -1
    p.table[3, 0] = 999                                  # n <= n_select: every block kept
    p.lengths[2] = 0
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sel = _select(p, box, 4, status=st)
    assert int(st) == 1 | 4
    ids = sel.ids.cpu()
    assert torch.equal(ids[0], good[0]) and bool((ids[1:] == -1).all())
    assert bool((sel.table.cpu().view(4, -1)[1:] == -1).all()) and sel.lengths.cpu().view(4, -1)[1:].sum() == 0
    st.zero_()
    t = [x.cuda() for x in (*p.kv, *p.groups)]
    out = gqa.attend_selected(p.q.cuda(), t[0], t[1], sel, k_scale=p.g[0].cuda(), v_scale=p.g[1].cuda(),
                              k_group_scale=t[2], v_group_scale=t[3], status=st)
    assert int(st) == 1 and torch.isnan(out[1:]).all() and torch.isfinite(out[0]).all()
    p = Problem("bf16", "slots", [300, 200], 4, 2, 128, 320, seed=8)
    p.slots[0] = -1
    st.zero_()
    sel = _select(p, _bounds(p), 4, status=st)
    assert int(st) == 2 and int(sel.ids[0].max()) == -1 and int(sel.ids[1].min()) >= 0


def test_reuse_stream_and_graph():
    p = Problem("e2m1", "dense", [4000, 90, 2500], 8, 2, 128, 4096, seed=9)
    box = _bounds(p).cuda()
    t = [x.cuda() for x in (*p.kv, *p.groups)]
    sel = _select(p, box, 24)
    want_ids, want = sel.ids.clone(), _attend(p, sel, t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = _select(p, box, 24, stream=side)
    side.synchronize()
    assert torch.equal(other.ids, want_ids)
    sel._buf.fill_(-7)
    assert _select(p, box, 24, selection=sel) is sel and torch.equal(sel.ids, want_ids)
    import gqa_kv_cache_gb300 as gqa
    q, ln = p.q.cuda(), p.lengths.cuda()
    kw = dict(k_scale=p.g[0].cuda(), v_scale=p.g[1].cuda(), k_group_scale=t[2], v_group_scale=t[3])
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        kept = gqa.select_blocks(q, box, ln, 24, block_size=p.bs)
        out = gqa.attend_selected(q, t[0], t[1], kept, **kw)
    for _ in range(3):
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(kept.ids, want_ids)


@pytest.mark.parametrize("kind", ["e2m1", "bf16"])
def test_a_run_of_steps(kind):
    """Prompts written with bounds, then steps: append, select, attend. Every
    step's ids and outputs follow from the cache's own content."""
    import gqa_kv_cache_gb300 as gqa
    B, Hq, Hkv, D, bs, nb = 3, 8, 2, 128, 16, 40
    lens = [300, 17, 511]
    p = Problem(kind, "paged", lens, Hq, Hkv, D, bs * nb, bs=bs, seed=10, extra=8)
    gen = torch.Generator().manual_seed(11)
    t = [torch.zeros_like(x).cuda() if x is not None else None for x in (*p.kv, *p.groups)]
    box = torch.zeros(p.kv[0].shape[0], Hkv, 2, D, dtype=torch.bfloat16, device="cuda")
    g = [x.cuda() for x in p.g]
    table = p.table.cuda()
    kw = {}
    if kind == "e2m1":
        kw = dict(k_scale=g[0], v_scale=g[1], k_group_scale=t[2], v_group_scale=t[3])

    def put(at, n):
        x = [torch.randn(sum(n), Hkv, D, generator=gen).bfloat16() for _ in range(2)]
        cu = torch.tensor([0, *torch.tensor(n).cumsum(0).tolist()], dtype=torch.int32)
        gqa.append_paged(x[0].cuda(), x[1].cuda(), t[0], t[1], table, torch.tensor(at, dtype=torch.int32).cuda(),
                         cu.cuda(), k_bounds=box, **kw)
        return x[0], cu

    keys = [[] for _ in range(B)]                        # the keys as given: the bounds are theirs
    x, cu = put([0] * B, lens)
    for b in range(B):
        keys[b] += list(x[int(cu[b]):int(cu[b + 1])])
    for step in range(4):
        n = [1, 1, 2] if step == 2 else [1] * B
        x, cu = put(p.lens, n)
        for b in range(B):
            keys[b] += list(x[int(cu[b]):int(cu[b + 1])])
        p.lens = [len(k) for k in keys]
        p.lengths = torch.tensor(p.lens, dtype=torch.int32)
        p.q = torch.randn(B, Hq, D, generator=gen).bfloat16()
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        sel = gqa.select_blocks_paged(p.q.cuda(), box, table, p.lengths.cuda(), 8, block_size=bs, n_last=2, status=st)
        out = gqa.attend_selected(p.q.cuda(), t[0], t[1], sel, status=st, **kw)
        assert int(st) == 0
        p.kv = [t[0].cpu(), t[1].cpu()]
        p.groups = [None if y is None else y.cpu() for y in t[2:]]
        ref = torch.zeros_like(box.cpu())
        for b in range(B):
            for j in range(-(-p.lens[b] // bs)):
                part = torch.stack(keys[b][j * bs:(j + 1) * bs])
                ref[int(p.table[b, j])] = torch.stack([part.amin(0), part.amax(0)], 1)
        used = p.table[p.table >= 0].long()
        live = torch.tensor([int(p.table[b, j]) for b in range(B) for j in range(-(-p.lens[b] // bs))])
        assert torch.equal(box.cpu()[live], ref[live]) and len(used) >= len(live)
        ids = sel.ids.cpu()
        assert torch.equal(ids, _want(p, ref, 8, 1, 2))
        _check_attend(p, sel, ids, out)


@pytest.mark.parametrize("layout", ["dense", "paged"])
def test_a_selection_of_another_cache_is_refused(layout):
    """A selection names blocks of one pool: another block size or number of rows
    would be other slots."""
    import gqa_kv_cache_gb300 as gqa
    p = Problem("bf16", layout, [200, 100], 4, 2, 128, 256, bs=32)
    box, kv = _bounds(p), [x.cuda() for x in p.kv]
    sel = _select(p, box, 4)
    gqa.attend_selected(p.q.cuda(), *kv, sel)
    p.bs, p.lengths = 16, torch.tensor([100, 50], dtype=torch.int32)
    half = _select(p, box, 4)                            # pages (or bounds) of 32 taken for 16
    with pytest.raises(ValueError):
        gqa.attend_selected(p.q.cuda(), *kv, half)
    with pytest.raises(ValueError):
        gqa.attend_selected(p.q.cuda(), *[torch.cat([x, x]) for x in kv], sel)
    empty = gqa.Selection(2, 2, 4, 32, torch.device("cuda", 0))
    with pytest.raises(ValueError):
        gqa.attend_selected(p.q.cuda(), *kv, empty)


def test_all_blocks_kept_is_the_plain_attend():
    import gqa_kv_cache_gb300 as gqa
    p = Problem("e2m1", "dense", [256, 100, 33], 8, 2, 128, 256, seed=12)
    t = [x.cuda() for x in (*p.kv, *p.groups)]
    kw = dict(k_scale=p.g[0].cuda(), v_scale=p.g[1].cuda(), k_group_scale=t[2], v_group_scale=t[3])
    sel = _select(p, _bounds(p), 16)
    a = gqa.attend_selected(p.q.cuda(), t[0], t[1], sel, **kw)
    b = gqa.attend(p.q.cuda(), t[0], t[1], p.lengths.cuda(), **kw)
    assert float((a - b).abs().max()) <= 1e-5 * float(b.abs().max())


def test_refusals():
    import gqa_kv_cache_gb300 as gqa
    p = Problem("bf16", "dense", [100], 4, 2, 128, 128, seed=13)
    box = _bounds(p)
    for n, first, last in ((2, 2, 1), (4, -1, 1), (4, 0, 0)):
        with pytest.raises(gqa.GqaError):
            _select(p, box, n, first, last)
    with pytest.raises(ValueError):
        _select(p, box, 0)
    with pytest.raises(TypeError):
        _select(p, box.float(), 4)
    with pytest.raises(ValueError):                      # Hq not a multiple of Hkv
        _select(p, box, 4, q=p.q[:, :3].contiguous())
    with pytest.raises(TypeError):                       # bounds of another width
        _select(p, box[..., :64].contiguous(), 4)
    sel = _select(p, box, 4)
    with pytest.raises(ValueError):                      # a selection of other sizes
        _select(p, box, 5, selection=sel)
    k, v = (x.cuda() for x in p.kv)
    with pytest.raises(ValueError):                      # a cache of other heads
        gqa.attend_selected(p.q.cuda(), k[:, :1].contiguous(), v[:, :1].contiguous(), sel)
    f8 = torch.zeros(1, 2, 128, 128, dtype=torch.uint8, device="cuda")
    g = torch.ones(2, device="cuda")
    with pytest.raises(gqa.GqaError):                    # an E4M3 cache
        gqa.attend_selected(p.q.cuda(), f8, f8.clone(), sel, k_scale=g, v_scale=g)
    with pytest.raises(ValueError):                      # a workspace of the host
        gqa.attend_selected(p.q.cuda(), k, v, sel, workspace=torch.zeros(1 << 20, dtype=torch.uint8))
    wide = torch.zeros(1, 2, 17000, 2, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(gqa.GqaError):                    # too many blocks a row
        gqa.select_blocks(p.q.cuda(), wide, p.lengths.cuda(), 4, block_size=16)


def test_terms_that_a_matrix_step_drops():
    """Blocks whose scores hold a few large terms and hundreds that a sum in
    float32's width drops one by one; all of a block's dropped terms have one sign,
    so that its float32 score is far from the exact one."""
    D, nb = 256, 40
    p = Problem("bf16", "dense", [1], 2, 1, D, 16, seed=1)
    p.lens, p.Smax = [nb * 16], nb * 16
    p.lengths = torch.tensor(p.lens, dtype=torch.int32)
    q, x = torch.zeros(1, 2, D), torch.zeros(1, 1, nb, 2, D)
    small = 1.9921875 * 2.0 ** -12
    q[0, 0], q[0, 1] = 2.0 ** -14, -2.0 ** -14           # the weights of the upper and of the lower bounds
    x[..., 0, :], x[..., 1, :] = -small, small           # every term 2^-26 * 1.99
    x[:, :, 1::2] *= -1                                  # of the odd blocks: below zero
    big = [0, 4, 32, 36]                                 # a term of 1 in each of the sums side by side
    q[0, 1, big], x[..., 0, big] = -1.0, -1.0
    x[:, :, 1::2, 1, 128] = 15 / 32                      # and 480 * 2^-24 more, exact in any order
    p.q, x = q.bfloat16(), x.bfloat16()
    assert torch.equal(_select(p, x, 10, 0, 1).ids.cpu(), _want(p, x, 10, 0, 1))


def test_a_selection_of_another_shape_is_refused():
    """As many (block, head) pairs, but other blocks: rows and blocks a row exchanged, or dense and paged."""
    import gqa_kv_cache_gb300 as gqa
    B, Hkv, D, bs = 2, 2, 128, 16
    q = torch.randn(B, 4, D).bfloat16().cuda()
    ln = torch.tensor([128, 100], dtype=torch.int32, device="cuda")
    pool = [torch.randn(64, Hkv, bs, D).bfloat16().cuda() for _ in range(2)]
    table = torch.arange(2 * 8, dtype=torch.int32, device="cuda").view(2, 8)
    kept = {}
    for R in (4, 8):
        box = torch.zeros(R, Hkv, 64 // R, 2, D, dtype=torch.bfloat16, device="cuda")
        kept[R] = gqa.select_blocks(q, box, ln, 4, block_size=bs)
    kept["paged"] = gqa.select_blocks_paged(q, box.view(64, Hkv, 2, D), table, ln, 4, block_size=bs)
    cache = {R: [x.view(R, Hkv, -1, D) for x in pool] for R in (4, 8)}
    cache["paged"] = pool
    for a in kept:
        for b in cache:
            if a == b:
                gqa.attend_selected(q, *cache[b], kept[a])
            else:
                with pytest.raises(ValueError):
                    gqa.attend_selected(q, *cache[b], kept[a])


def test_a_selection_that_failed_is_not_attended():
    import gqa_kv_cache_gb300 as gqa
    p = Problem("bf16", "dense", [200, 100], 4, 2, 128, 256)
    box, kv = _bounds(p), [x.cuda() for x in p.kv]
    sel = gqa.Selection(2, 2, 4, 16, torch.device("cuda", 0))
    with pytest.raises(gqa.GqaError):
        _select(p, box, 4, 4, 4, selection=sel)
    with pytest.raises(ValueError):
        gqa.attend_selected(p.q.cuda(), *kv, sel)


def _drawn(B, Hkv, G, D, lens, nb, bs, layout, seed, q_dtype=torch.bfloat16):
    gen = torch.Generator().manual_seed(seed)
    p = Problem("bf16", "dense", [1] * B, G * Hkv, Hkv, D, bs, bs=bs, seed=seed, q_dtype=q_dtype)
    p.lens, p.Smax = lens, nb * bs
    p.lengths = torch.tensor(lens, dtype=torch.int32)
    if layout == "paged":
        perm = torch.randperm(B * nb, generator=gen).view(B, nb).int()
        held = torch.tensor([-(-n // bs) for n in lens])
        p.table = torch.where(torch.arange(nb) < held[:, None], perm, -1)
        shape = (B * nb, Hkv, 2, D)
    else:
        shape = (B, Hkv, nb, 2, D)
    box = torch.randn(shape, generator=gen).sort(-2).values.bfloat16()
    return p, box


@pytest.mark.parametrize("layout", ["dense", "paged"])
@pytest.mark.parametrize("D,G,q_dtype", [(64, 2, torch.float32), (128, 6, torch.bfloat16), (256, 1, torch.bfloat16)])
def test_many_units(D, G, q_dtype, layout):
    """More (row, cache head) pairs than two a multiprocessor: uneven rows, and
    among them equal scores, scores too close for float32 (more of them than are
    ranked directly), NaN and infinite bounds."""
    B, Hkv, nb, bs = 64, 8, 220, 16
    assert B * Hkv > 2 * torch.cuda.get_device_properties(0).multi_processor_count
    lens = [1 + (b * 997) % (nb * bs) if b % 8 else nb * bs - b for b in range(B)]
    p, box = _drawn(B, Hkv, G, D, lens, nb, bs, layout, D, q_dtype)
    gen = torch.Generator().manual_seed(1)
    for b in range(0, B, 8):
        at = (lambda h, j: (p.table[b, j].long(), h)) if layout == "paged" else (lambda h, j: (b, h, j))
        j = torch.arange(-(-lens[b] // bs))
        for h in range(Hkv):
            if h % 4 == 0:
                box[at(h, j)] = box[at(h, j[:1])]        # equal scores
            elif h % 4 == 1:                             # a large term that cancels
                q = p.q.view(B, Hkv, G, D)
                q[b, h] = 0
                q[b, h, 0, 0], q[b, h, 0, 1], q[b, h, 0, 2] = 1024.0, -1024.0, 2.0 ** -12
                x = torch.zeros(len(j), 2, D)
                x[..., :2] = 256.0
                x[..., 2] = (torch.randperm(len(j), generator=gen).float() / 256)[:, None]
                box[at(h, j)] = x.bfloat16()
            elif h % 4 == 2:
                box[at(h, j[40])], box[at(h, j[7])] = math.nan, math.inf
    for n, first, last in ((5, 0, 1), (100, 2, 3)):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        assert torch.equal(_select(p, box, n, first, last, status=st).ids.cpu(), _want(p, box, n, first, last))
        assert int(st) == 0


@pytest.mark.parametrize("nb", [256, 300, 511])
def test_two_ctas_a_unit(nb):
    """Few units of 256 to 511 blocks: a cluster of two."""
    p, box = _drawn(2, 2, 4, 128, [nb * 16, nb * 16 - 37], nb, 16, "dense", nb)
    for n in (3, 64, 200):
        assert torch.equal(_select(p, box, n).ids.cpu(), _want(p, box, n))


@pytest.mark.parametrize("q_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("G", [1, 6, 8])
def test_weights_of_a_bfloat16_cache_are_whole(G, q_dtype):
    """Every eighth slot of the largest weight and no value, the others of one smaller
    weight and the value 1: the output follows that weight, and an error of its
    rounding is not averaged out (16 bits of it: up to 2^-17)."""
    import gqa_kv_cache_gb300 as gqa
    D, n, bs = 128, 1024, 64
    q = torch.zeros(1, G, D)
    q[0, :, 0] = torch.tensor([3.0, 5.1, 7.7, 9.3, 11.9, 13.2, 15.7, 17.3][-G:])
    q = q.to(q_dtype)
    k, v = torch.zeros(1, 1, n, D).bfloat16(), torch.ones(1, 1, n, D).bfloat16()
    k[0, 0, ::8, 0], v[0, 0, ::8] = 1.0, 0.0
    box = torch.zeros(1, 1, n // bs, 2, D, dtype=torch.bfloat16, device="cuda")
    ln = torch.tensor([n], dtype=torch.int32, device="cuda")
    sel = gqa.select_blocks(q.cuda(), box, ln, n // bs, block_size=bs)
    got = gqa.attend_selected(q.cuda(), k.cuda(), v.cuda(), sel).double().cpu()[0]
    w = 7 * torch.exp(-q[0, :, 0].double() / math.sqrt(D))
    rel = (got / (w / (1 + w))[:, None] - 1).abs().amax(1)
    # scores of up to 1.53: three roundings of 2^-24 are 2^-21 of a weight; its 24 bits,
    # the exponential and the sums' roundings 2^-21 together. A float32 query enters as
    # two bfloat16, |q - hi| <= 2^-9 |q| and |q - hi - lo| <= 2^-9 |q - hi|: 2^-18 of a score
    assert float(rel.max()) <= 2.0 ** -20 + (1.53 * 2.0 ** -18 if q_dtype == torch.float32 else 0)
