"""Rotary positions, the cache, counted attention and eviction together, as a
serving loop runs them; on other streams, and captured and replayed."""
import pytest
import torch

import gqa_kv_cache_gb300 as gqa
import serve_reference as R

pytestmark = pytest.mark.gpu
B, Hq, Hkv, D, S = 3, 8, 2, 64, 256


def _inputs(n, gen):
    """Packed projections (n tokens a row)."""
    return [torch.randn(B * n, h, D, generator=gen).bfloat16().cuda() for h in (Hq, Hkv, Hkv)]


def test_a_loop_with_eviction():
    """A prompt, decode steps that count their weights, a cut of the rows, further steps: against 64 bits on what
    the cache then holds."""
    gen = torch.Generator().manual_seed(0)
    rot = gqa.Rotary(D, scaling=dict(kind="linear", factor=2.0))
    k_cache, v_cache = (torch.zeros(B, Hkv, S, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    weights = torch.zeros(B, Hkv, S, device="cuda")
    lengths = torch.zeros(B, dtype=torch.int32, device="cuda")
    q, k, v = _inputs(100, gen)
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda") * 100
    gqa.rotate(q, k, rot, lengths=lengths, cu_q=cu, q_out=q, k_out=k)
    gqa.append(k, v, k_cache, v_cache, lengths, cu)
    lengths = lengths + 100
    position = lengths.clone()
    one = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    for step in range(30):
        if step == 15:
            before = [x.cpu() for x in (k_cache, v_cache, weights)]
            ids, new = gqa.evict(k_cache, v_cache, weights, lengths, 64, n_first=4, n_last=16)
            for b in range(B):
                for h in range(Hkv):
                    at = R.kept(before[2][b, h], int(lengths[b]), 64, 4, 16)
                    assert ids[b, h].tolist() == at
                    for x, y in zip(before, (k_cache, v_cache, weights)):
                        assert torch.equal(y[b, h, :64].cpu(), x[b, h, at])
            lengths = new
        q, k, v = _inputs(1, gen)
        gqa.rotate(q, k, rot, position, q_out=q, k_out=k)
        out = gqa.decode_step(q, k, v, k_cache, v_cache, lengths, score_cap=30.0, weights=weights)
        n = int(lengths[0]) + 1
        o, w, e = R.attention(q[0].cpu().double().view(Hkv, -1, D), k_cache[0, :, :n].cpu().double(),
                              v_cache[0, :, :n].cpu().double(), 30.0)
        assert (out[0].cpu().double() - o.reshape(Hq, D)).abs().max() <= R.out_tolerance(w, e, float(v_cache[0].abs().max()))
        lengths = lengths + 1
        position = position + 1
    # every step gave each head's queries weights that sum to one; eviction dropped some
    total = weights.sum((1, 2))
    assert (total <= 30 * Hq * (1 + 2.0 ** -15)).all() and (total >= 15 * Hq * (1 - 2.0 ** -15)).all()
    assert not weights[:, :, int(lengths[0]):].any()
    read, _ = gqa.read(k_cache, v_cache, lengths - 1, one, B)
    assert torch.equal(read, k)


def test_biases_and_windows_of_a_row_that_was_cut_count_slots():
    """What evict says of head_slopes and window: distances are those of the kept slots."""
    gen = torch.Generator().manual_seed(5)
    k, v = (torch.randn(1, Hkv, S, D, generator=gen).bfloat16().cuda() for _ in range(2))
    w, n = torch.rand(1, Hkv, S, generator=gen).cuda(), torch.tensor([200], dtype=torch.int32).cuda()
    _, n = gqa.evict(k, v, w, n, 40, n_first=2, n_last=8)
    q, slopes = torch.randn(1, Hq, D, generator=gen), torch.rand(Hq, generator=gen)
    for window in (0, 12):
        out = gqa.attend(q.cuda(), k, v, n, head_slopes=slopes.cuda(), window=window)
        o, weight, e = R.attention(q[0].double().view(Hkv, -1, D), k[0, :, :40].cpu().double(), v[0, :, :40].cpu().double(),
                                   slopes=slopes.view(Hkv, -1), ok=R.attended(40, window))
        assert (out[0].cpu().double() - o.reshape(Hq, D)).abs().max() <= R.out_tolerance(weight, e, float(v.abs().max()))


def _steps(stream=None, workspace=None):
    """A fixed run of all the calls; returns every output."""
    gen = torch.Generator().manual_seed(1)
    state = dict(
        k8=torch.zeros(B, Hkv, S, D, dtype=torch.int8, device="cuda"), v8=torch.zeros(B, Hkv, S, D, dtype=torch.int8, device="cuda"),
        ks=torch.zeros(B, Hkv, S // 16, device="cuda"), vs=torch.zeros(B, Hkv, S // 16, device="cuda"),
        w=torch.zeros(B, Hkv, S, device="cuda"), kb=torch.randn(B, Hkv, S, D, generator=gen).bfloat16().cuda(),
        vb=torch.randn(B, Hkv, S, D, generator=gen).bfloat16().cuda(), inputs=_inputs(90, gen), token=_inputs(1, gen),
        cu=torch.arange(B + 1, dtype=torch.int32, device="cuda") * 90, zero=torch.zeros(B, dtype=torch.int32, device="cuda"),
        n=torch.full((B,), 90, dtype=torch.int32, device="cuda"), rot=gqa.Rotary(D))

    def run(s):
        kw = dict(k_block_scale=s["ks"], v_block_scale=s["vs"])
        q, k = gqa.rotate(*s["inputs"][:2], s["rot"], lengths=s["zero"], cu_q=s["cu"], stream=stream)
        gqa.append(k, s["inputs"][2], s["k8"], s["v8"], s["zero"], s["cu"], **kw, stream=stream)
        q1, k1 = gqa.rotate(*s["token"][:2], s["rot"], s["n"], stream=stream)
        a = gqa.decode_step(q1, k1, s["token"][2], s["k8"], s["v8"], s["n"], **kw, weights=s["w"], stream=stream)
        b = gqa.attend(q1, s["kb"], s["vb"], s["n"], score_cap=20.0, weights=s["w"], stream=stream)
        ids, new = gqa.evict(s["kb"], s["vb"], s["w"], s["n"], 32, stream=stream)
        c = gqa.attend(q1, s["kb"], s["vb"], new, stream=stream)
        return q, a, b, ids, new, c

    return state, run


def test_other_streams_and_graphs():
    state, run = _steps()
    want = [x.clone() for x in run(state)]
    cache = [state[n].clone() for n in ("k8", "v8", "ks", "vs", "w", "kb", "vb")]
    torch.cuda.synchronize()
    # the same on a stream given by argument, and as the current stream
    side = torch.cuda.Stream()
    state, run = _steps(side)
    torch.cuda.synchronize()
    got = run(state)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(a, state[n]) for a, n in zip(cache, ("k8", "v8", "ks", "vs", "w", "kb", "vb")))
    # captured once, replayed on fresh contents
    state, run = _steps()
    start = {n: state[n].clone() for n in ("k8", "v8", "ks", "vs", "w", "kb", "vb")}
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        run(state)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(state)
    for _ in range(3):
        for n, x in start.items():
            state[n].copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_graphs_side_by_side():
    """Two captured attends with counted weights, replayed at once on two streams."""
    graphs = []
    for seed in range(2):
        g = torch.Generator().manual_seed(seed)
        q = torch.randn(B, Hq, D, generator=g).cuda()
        k, v = (torch.randn(B, Hkv, 4096, D, generator=g).bfloat16().cuda() for _ in range(2))
        n = torch.tensor([4096, 17, 3000], dtype=torch.int32).cuda()
        w = torch.zeros(B, Hkv, 4096, device="cuda")
        want = gqa.attend(q, k, v, n, score_cap=9.0, weights=w).clone()
        once = w.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = gqa.attend(q, k, v, n, score_cap=9.0, weights=w)
        graphs.append((graph, out, w, want, once, (q, k, v, n)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for _, out, w, _, _, _ in graphs:
            w.zero_()
            out.zero_()
        torch.cuda.synchronize()
        for s, (graph, *_) in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for _, out, w, want, once, _ in graphs:
            assert torch.equal(out, want) and torch.equal(w, once)


def test_two_threads_count_on_one_stream():
    """Counted attends of two threads, on the default stream of both: each has the counts it has alone."""
    import threading
    jobs = []
    for seed in range(2):
        g = torch.Generator().manual_seed(seed)
        q = torch.randn(B, Hq, D, generator=g).cuda()
        k, v = (torch.randn(B, Hkv, 1024, D, generator=g).bfloat16().cuda() for _ in range(2))
        n = torch.tensor([1024, 17, 300], dtype=torch.int32).cuda()
        once = torch.zeros(B, Hkv, 1024, device="cuda")
        out = gqa.attend(q, k, v, n, weights=once)
        jobs.append((q, k, v, n, once, out))
    torch.cuda.synchronize()
    got = [[], []]

    def run(i):
        q, k, v, n, once, _ = jobs[i]
        for _ in range(300):
            w = torch.zeros_like(once)
            got[i].append((gqa.attend(q, k, v, n, weights=w), w))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for (*_, once, out), runs in zip(jobs, got):
        assert len(runs) == 300
        assert all(torch.equal(w, once) and torch.equal(o, out) for o, w in runs)


def test_runs_give_the_same_bits():
    state, run = _steps()
    start = {n: state[n].clone() for n in ("k8", "v8", "ks", "vs", "w", "kb", "vb")}
    first = [x.clone() for x in run(state)]
    for n, x in start.items():
        state[n].copy_(x)
    assert all(torch.equal(a, b) for a, b in zip(run(state), first))


def test_empty_batches():
    """No rows, or rows without tokens: nothing is launched or written."""
    k8 = torch.zeros(2, Hkv, S, D, dtype=torch.int8, device="cuda")
    kw = dict(k_block_scale=torch.zeros(2, Hkv, 4, device="cuda"), v_block_scale=torch.zeros(2, Hkv, 4, device="cuda"))
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    q = torch.zeros(0, Hq, D, dtype=torch.bfloat16, device="cuda")
    new = torch.zeros(0, Hkv, D, dtype=torch.bfloat16, device="cuda")
    assert gqa.attend(q, k8, k8, none, **kw).shape == (0, Hq, D)
    assert gqa.decode_step(q, new, new, k8, k8, none, **kw).shape == (0, Hq, D)
    kb = torch.zeros(2, Hkv, S, D, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(2, Hkv, S, device="cuda")
    assert gqa.attend(q, kb, kb, none, score_cap=3.0, weights=w).shape == (0, Hq, D)
    ids, lengths = gqa.evict(kb, kb, w, none, 8)
    assert ids.shape == (0, Hkv, 8) and lengths.shape == (0,)
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    gqa.append(new, new, k8, k8, none, one, **kw)
    gqa.append(torch.ones(3, Hkv, D, device="cuda"), torch.ones(3, Hkv, D, device="cuda"), k8, k8.clone(),
               torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda"), **kw)
    assert not k8.any() and not kw["k_block_scale"].any()
    a, _ = gqa.rotate(torch.ones(3, 1, D, device="cuda"), None, gqa.Rotary(D), lengths=none, cu_q=one)
    assert (a == 1).all()                                         # tokens of no row


def test_decode_steps_with_bad_rows():
    """A row that cannot take its token is left as it is and gives NaN; the others are served."""
    g = torch.Generator().manual_seed(3)
    for kind in (torch.int8, torch.bfloat16):
        cache = [torch.ones(3, Hkv, S, D, dtype=kind, device="cuda") for _ in range(2)]
        kw = dict(k_block_scale=torch.ones(3, Hkv, 16, device="cuda"), v_block_scale=torch.ones(3, Hkv, 16, device="cuda")) \
            if kind == torch.int8 else dict(score_cap=4.0)
        weights = torch.zeros(3, Hkv, S, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        q, k, v = _inputs(1, g)
        at = torch.tensor([S, 7, -1], dtype=torch.int32).cuda()
        out = gqa.decode_step(q, k, v, *cache, at, status=status, weights=weights, **kw)
        assert int(status) == 1 and out[0].isnan().all() and out[2].isnan().all() and out[1].isfinite().all()
        assert (cache[0][0] == 1).all() and (cache[0][2] == 1).all() and not weights[0].any() and not weights[2].any()
        assert abs(float(weights[1].sum()) - Hq) < 1e-4
        ids = torch.tensor([0, 9, 1], dtype=torch.int32).cuda()
        status.zero_()
        out = gqa.decode_step(q, k, v, *cache, at.clamp(0, 9), ids, status=status, **kw)
        assert int(status) == 2 and out[1].isnan().all() and out[0].isfinite().all()
