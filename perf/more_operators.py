"""Measured cases of what a serving step does around its cache: rotary
positions, writes into and attention over an 8-bit cache with a scale for each
(block of slots, cache head), attention with capped or distance-biased scores,
and eviction by accumulated attention weight.

Rotary positions. Over the first `dim` elements of a head, pair i turns by the
angle pos f_i and is multiplied by m: (x, y) -> m (x cos - y sin, x sin + y cos).
Pair i is (i, i + dim / 2) in the "half" layout and (2i, 2i + 1) in the
"interleaved" one. f_i = base^(-2i / dim), for long contexts scaled by s:
"linear" f / s; "ntk" another base, base s^(dim / (dim - 2)); "bands" with
r = original f / (2 pi) turns within the original length and
u = clamp((r - low) / (high - low), 0, 1): f (u + (1 - u) / s).

The 8-bit cache. A block's values are c t with int8 c and the block's float32
scale t (one a cache head). A block that begins with a new token has
t = max|x| / 127; one that gets tokens behind earlier ones keeps its scale t0
where it holds them, else it doubles (t = t0 2^k, the smallest k with
max|x| / 127 <= t; the earlier codes become rint(c / 2^k)); codes are rint(x / t)
(0 where t is 0), in float32.

Scores. s = q.k / sqrt(D); with a cap s' = cap tanh(s / cap); with slopes
s' + slope_h (j - L), L the query's position. A window W attends the last W slots.

Eviction. Every attended slot's weights are summed over the queries of a cache
head and added to its count; a row longer than n_keep slots keeps its first
n_first, its last n_last, and of the others those with the highest counts
(ties to the lowest slot), in ascending order.

Sizes are the repository's decode workloads (llama3_8b, long_context,
ragged_slots, paged, pr1_fp32) and smaller or ragged ones around them.
"""
import math
import random

import torch

own = False

CHUNK = 1 << 26


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one decode step of llama3_8b: q and k of 32 tokens, launch-bound
        dict(name="rotate_token", op="rotate", T=32, Hq=32, Hkv=8, D=128, dim=128, style="half", scaling="none",
             base=500000.0, pos_hi=4095, q="bf16"),
        # long prompts, half of each head turned, frequencies stretched for a longer context
        dict(name="rotate_prompts", op="rotate", T=65521, Hq=48, Hkv=8, D=128, dim=64, style="interleaved",
             scaling="bands", base=10000.0, pos_hi=131071, q="bf16"),
        # one decode step's tokens into an 8-bit cache, llama3_8b heads: most blocks hold earlier tokens
        dict(name="write8_token", op="write", layout="dense", B=32, R=32, Hkv=8, D=128, Smax=4096, block=16, q_lo=1,
             q_hi=1, len_lo=1024, len_hi=4094, out="bf16"),
        # ragged prompts behind earlier ones into a paged 8-bit cache
        dict(name="write8_prompts", op="write", layout="paged", B=64, R=0, Hkv=8, D=128, Smax=2112, block=16, q_lo=1,
             q_hi=2047, len_lo=0, len_hi=61, out="f32"),
        # llama3_8b's decode step (append and attend) over an 8-bit cache
        dict(name="decode8_llama3_8b", op="attend", kind="int8", step="decode", layout="dense", B=32, R=32, Hq=32,
             Hkv=8, D=128, Smax=4096, block=64, len_lo=1024, len_hi=4095, dist="uniform", q="bf16", key_scale=1.0,
             cap=0.0, slopes=False, window=0, weights=False),
        # four long contexts over an 8-bit cache, G = 8
        dict(name="attend8_long_context", op="attend", kind="int8", step="attend", layout="dense", B=4, R=4, Hq=64,
             Hkv=8, D=128, Smax=131072, block=64, len_lo=32768, len_hi=131071, dist="uniform", q="bf16", key_scale=3.0,
             cap=0.0, slopes=False, window=0, weights=False),
        # the paged workload (bfloat16, 16-slot blocks, G = 6) with scores capped at 50
        dict(name="capped_paged", op="attend", kind="bf16", step="attend", layout="paged", B=64, R=0, Hq=48, Hkv=8,
             D=128, Smax=16384, block=16, len_lo=512, len_hi=16383, dist="uniform", q="bf16", key_scale=3.0, cap=50.0,
             slopes=False, window=0, weights=False),
        # continuous batching with very uneven lengths over an 8-bit cache, distance bias, float32 queries
        dict(name="biased_ragged_slots", op="attend", kind="int8", step="attend", layout="slots", B=256, R=512, Hq=32,
             Hkv=4, D=128, Smax=8192, block=16, len_lo=16, len_hi=8191, dist="log", q="f32", key_scale=1.0, cap=0.0,
             slopes=True, window=0, weights=False),
        # two short sequences, D = 64, with the slots' weights counted: latency
        dict(name="counted_small", op="attend", kind="bf16", step="attend", layout="dense", B=2, R=2, Hq=8, Hkv=2,
             D=64, Smax=256, block=16, len_lo=1, len_hi=255, dist="uniform", q="f32", key_scale=1.0, cap=0.0,
             slopes=False, window=0, weights=True),
        # four long contexts over a bfloat16 cache with the slots' weights counted
        dict(name="counted_long_context", op="attend", kind="bf16", step="attend", layout="dense", B=4, R=4, Hq=64,
             Hkv=8, D=128, Smax=131072, block=64, len_lo=32768, len_hi=131071, dist="uniform", q="bf16", key_scale=3.0,
             cap=0.0, slopes=False, window=0, weights=True),
        # one sequence cut to 512 slots: latency
        dict(name="evict_one_row", op="evict", kind="e4m3", layout="dense", B=1, R=1, Hkv=8, D=128, Smax=8192, block=16,
             len_lo=8001, len_hi=8001, n_keep=512, n_first=4, n_last=64),
        # the paged workload's rows cut to 2048 slots each
        dict(name="evict_paged", op="evict", kind="bf16", layout="paged", B=64, R=0, Hkv=8, D=128, Smax=16384, block=16,
             len_lo=512, len_hi=16383, n_keep=2048, n_first=4, n_last=256),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["rotate", "write", "attend", "attend", "attend", "evict"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    if op == "rotate":
        q = rng.choice(["bf16", "bf16", "f32"])
        return dict(op=op, T=_log(rng, 1, 65536 if q == "bf16" else 32768), Hq=Hkv * rng.randint(1, 6), Hkv=Hkv, D=D,
                    dim=rng.choice([D, D, D // 2, D - 24]), style=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "ntk", "bands"]), base=rng.choice([10000.0, 500000.0]),
                    pos_hi=_log(rng, 1000, 1000000), q=q)
    layout = rng.choice(["dense", "slots", "paged"])
    if op == "write":
        B = _log(rng, 1, 128)
        q_hi = _log(rng, 1, max(1, 65536 // B))
        block = rng.choice([8, 16, 24, 32, 64, 128])
        len_hi = rng.choice([0, rng.randint(1, 500)])
        Smax = -(-(len_hi + q_hi) // block) * block
        return dict(op=op, layout=layout, B=B, R=0 if layout == "paged" else B + (rng.randint(0, B) if layout == "slots" else 0),
                    Hkv=Hkv, D=D, Smax=Smax, block=block, q_lo=rng.randint(1, q_hi), q_hi=q_hi, len_lo=0, len_hi=len_hi,
                    out=rng.choice(["bf16", "f32"]))
    block = rng.choice([8, 16, 24, 32, 64])
    Smax = -(-_log(rng, 64, 130000) // block) * block
    room = 4 * 131072 * 8 * 128 // 2   # elements of a case's keys
    B = _log(rng, 1, max(1, min(256, room // (Smax * Hkv * D))))
    rows = 0 if layout == "paged" else B + (rng.randint(0, B) if layout == "slots" else 0)
    lo = rng.randint(1, max(1, Smax // 2))
    if op == "evict":
        n_keep = _log(rng, 16, max(16, min(8192, Smax // 2)))
        return dict(op=op, kind=rng.choice(["bf16", "bf16", "e4m3", "f32"]), layout=layout, B=B, R=rows, Hkv=Hkv, D=D,
                    Smax=Smax, block=block, len_lo=lo, len_hi=Smax - 1, n_keep=n_keep, n_first=rng.randint(0, 8),
                    n_last=rng.randint(0, 8))
    step = rng.choice(["attend", "attend", "decode"])
    more = rng.choice(["", "", "cap", "slopes", "weights", "weights", "all"])
    kind = rng.choice(["int8", "bf16"]) if more else "int8"
    return dict(op=op, kind=kind, step=step, layout=layout, B=B, R=rows, Hq=Hkv * rng.randint(1, 8), Hkv=Hkv, D=D,
                Smax=Smax, block=block, len_lo=lo, len_hi=Smax - 1, dist=rng.choice(["uniform", "log"]),
                q=rng.choice(["bf16", "f32"]) if step == "attend" else "bf16", key_scale=rng.choice([1.0, 3.0]),
                cap=rng.choice([20.0, 50.0]) if more in ("cap", "all") else 0.0, slopes=more in ("slopes", "all"),
                window=rng.choice([0, 0, 1 + Smax // 3]), weights=more in ("weights", "all"))


def _spread(n, lo, hi, log=False):
    """n lengths spread evenly over lo..hi (or over their logarithm)."""
    if not log:
        return [lo + int((hi - lo + 1) * (i + 0.5) / n) for i in range(n)]
    a, b = math.log(max(lo, 1)), math.log(hi + 1)
    return [min(hi, max(lo, int(math.exp(a + (b - a) * (i + 0.5) / n)))) for i in range(n)]


def _size(kind):
    return {"f32": 4, "bf16": 2, "int8": 1, "e4m3": 1}[kind]


def work(case):
    Hkv, D = case["Hkv"], case["D"]
    if case["op"] == "rotate":
        n = case["T"] * (case["Hq"] + Hkv) * D
        return {"bytes": 2 * n * _size(case["q"]) + 4 * case["T"], "flops": 3 * n * case["dim"] // D}
    B, bs = case["B"], case["block"]
    if case["op"] == "write":
        lens, q_lens = _spread(B, case["len_lo"], case["len_hi"]), _spread(B, case["q_lo"], case["q_hi"])
        T, es = sum(q_lens), _size(case["out"])
        seen = T + sum(n % bs for n in lens)               # read back: the blocks' earlier tokens too
        blocks = seen // bs + B
        return {"bytes": 2 * Hkv * (T * (2 * D + D) + seen * (D + es * D) + blocks * 8), "flops": 6 * T * Hkv * D}
    lens = _spread(B, case["len_lo"], case["len_hi"], case.get("dist") == "log")
    if case["op"] == "evict":
        kept = sum(min(n, case["n_keep"]) for n in lens)
        return {"bytes": Hkv * (4 * sum(lens) + kept * (4 * D * _size(case["kind"]) + 8)), "flops": Hkv * sum(lens)}
    Hq, es = case["Hq"], _size(case["kind"])
    if case["window"]:
        lens = [min(n, case["window"]) for n in lens]
    n = B * Hq * D * (_size(case["q"]) + 4) + sum(lens) * Hkv * 2 * es * D
    if es == 1:
        n += sum(lens) // bs * Hkv * 8
    if case["weights"]:
        n += sum(lens) * Hkv * 8
    if case["step"] == "decode":
        n += 2 * B * Hkv * D * (2 + es) + 2 * B * Hkv * D * (es + 2)      # written, and read back
    return {"bytes": n, "flops": 4 * sum(lens) * Hq * D}


# ----------------------------------------------------------------- inputs --

def _normal(shape, gen, scale=1.0, dtype=torch.bfloat16):
    out = torch.empty(math.prod(shape), dtype=dtype, device="cuda")
    for i in range(0, out.numel(), CHUNK):
        m = min(CHUNK, out.numel() - i)
        out[i:i + m] = torch.randn(m, generator=gen, device="cuda").mul_(scale).to(dtype)
    return out.view(shape)


def _codes(shape, gen):
    """Codes of an 8-bit cache's normal values, the block's largest near 127."""
    out = torch.empty(math.prod(shape), dtype=torch.int8, device="cuda")
    for i in range(0, out.numel(), CHUNK):
        m = min(CHUNK, out.numel() - i)
        out[i:i + m] = torch.randn(m, generator=gen, device="cuda").mul_(34.0).round_().clamp_(-127, 127).to(torch.int8)
    return out.view(shape)


SCALING = {"none": None, "linear": dict(kind="linear", factor=4.0), "ntk": dict(kind="ntk", factor=8.0),
           "bands": dict(kind="bands", factor=8.0, original=8192, low=1.0, high=4.0, attention=1.2)}


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    rng = random.Random(seed)
    c = dict(case)
    s = {"case": c}
    Hkv, D = c["Hkv"], c["D"]
    if c["op"] == "rotate":
        dtype = torch.bfloat16 if c["q"] == "bf16" else torch.float32
        s["q"], s["k"] = _normal((c["T"], c["Hq"], D), gen, 1.0, dtype), _normal((c["T"], Hkv, D), gen, 1.0, dtype)
        s["positions"] = torch.randint(0, c["pos_hi"] + 1, (c["T"],), generator=gen, device=dev, dtype=torch.int32)
        if own:
            import gqa_kv_cache_gb300 as gqa
            s["rotary"] = gqa.Rotary(c["dim"], base=c["base"], layout=c["style"], scaling=SCALING[c["scaling"]],
                                     device=dev)
        return s
    B, Smax, bs = c["B"], c["Smax"], c["block"]
    lens = _spread(B, c["len_lo"], c["len_hi"], c.get("dist") == "log")
    q_lens = _spread(B, c["q_lo"], c["q_hi"]) if c["op"] == "write" else [1] * B
    rng.shuffle(lens)
    rng.shuffle(q_lens)
    grows = c["op"] == "write" or c.get("step") == "decode"
    s["lengths"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["cu_q"] = torch.tensor([sum(q_lens[:b]) for b in range(B + 1)], dtype=torch.int32, device=dev)
    s["T"] = sum(q_lens)
    s["slot_ids"] = s["table"] = None
    if c["layout"] == "paged":
        nb = Smax // bs
        shape, blocks, counts = (B * nb, Hkv, bs, D), (B * nb, Hkv), (B * nb, Hkv, bs)
        held = torch.tensor([-(-(a + (n if grows else 0)) // bs) for a, n in zip(lens, q_lens)], device=dev)
        s["table"] = torch.randperm(B * nb, generator=gen, device=dev).view(B, nb).to(torch.int32)
        s["table"] = torch.where(torch.arange(nb, device=dev) < held[:, None], s["table"], -1)
    else:
        R = c["R"]
        shape, blocks, counts = (R, Hkv, Smax, D), (R, Hkv, Smax // bs), (R, Hkv, Smax)
        if c["layout"] == "slots":
            s["slot_ids"] = torch.randperm(R, generator=gen, device=dev)[:B].to(torch.int32)
    kind = c.get("kind", "int8")
    key_scale = c.get("key_scale", 1.0)
    if kind == "int8":
        s["k"], s["v"] = _codes(shape, gen), _codes(shape, gen)
        # the largest of a block's normal values lies between three and five deviations
        s["ks"] = (0.024 + 0.016 * torch.rand(blocks, generator=gen, device=dev)) * key_scale
        s["vs"] = 0.024 + 0.016 * torch.rand(blocks, generator=gen, device=dev)
    elif kind == "e4m3":
        s["k"], s["v"] = (_normal(shape, gen, 40.0, torch.float8_e4m3fn) for _ in range(2))
    else:
        dtype = torch.bfloat16 if kind == "bf16" else torch.float32
        s["k"], s["v"] = _normal(shape, gen, key_scale, dtype), _normal(shape, gen, 1.0, dtype)
    if grows:
        s["k_new"], s["v_new"] = _normal((s["T"], Hkv, D), gen, key_scale), _normal((s["T"], Hkv, D), gen)
    if c["op"] == "write":
        # what is read back: the new tokens and those before them in their first block
        first = [n // bs * bs for n in lens]
        total = [0]
        for a, n, m in zip(first, lens, q_lens):
            total.append(total[-1] + n + m - a)
        s["read_at"] = torch.tensor(first, dtype=torch.int32, device=dev)
        s["read_cu"] = torch.tensor(total, dtype=torch.int32, device=dev)
        s["read_T"] = total[-1]
        return s
    if c["op"] == "evict":
        # counts fall over many octaves; some slots were never attended
        w = torch.rand(counts, generator=gen, device=dev)
        s["weights"] = torch.where(w < 0.05, 0.0, torch.exp2(-12.0 * w) * (0.5 + w * w)).float()
        s["k2"], s["v2"] = (torch.zeros((B, Hkv, c["n_keep"], D), dtype=s["k"].dtype, device=dev) for _ in range(2))
        s["w2"] = torch.zeros((B, Hkv, c["n_keep"]), device=dev)
        return s
    s["q"] = _normal((B, c["Hq"], D), gen, 1.0, torch.float32 if c["q"] == "f32" else torch.bfloat16)
    if c["slopes"]:
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, c["Hq"] + 1, device=dev) / c["Hq"]).float()
    if c["weights"]:
        s["weights"] = torch.zeros(counts, device=dev)
    return s


# ------------------------------------------------------------ plain forms --

def _frequencies(c):
    """Angles a position, 64 bits, and the factor m."""
    i = torch.arange(0, c["dim"], 2, device="cuda").double() / c["dim"]
    k = SCALING[c["scaling"]]
    if k is None:
        return c["base"] ** -i, 1.0
    if k["kind"] == "linear":
        return c["base"] ** -i / k["factor"], 1.0
    if k["kind"] == "ntk":
        return (c["base"] * k["factor"] ** (c["dim"] / (c["dim"] - 2))) ** -i, 1.0
    f = c["base"] ** -i
    u = ((k["original"] * f / (2 * math.pi) - k["low"]) / (k["high"] - k["low"])).clamp(0, 1)
    return f * (u + (1 - u) / k["factor"]), k["attention"]


def _plain_rotate(s):
    c = s["case"]
    f, m = _frequencies(c)
    angle = s["positions"].double()[:, None] * f                  # far positions: 64 bits
    cos, sin = (torch.cos(angle) * m).float()[:, None], (torch.sin(angle) * m).float()[:, None]
    out = []
    for x in (s["q"], s["k"]):
        y = x.float()
        turned, rest = y[..., :c["dim"]], y[..., c["dim"]:]
        if c["style"] == "half":
            a, b = turned[..., :c["dim"] // 2], turned[..., c["dim"] // 2:]
            turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        else:
            a, b = turned[..., 0::2], turned[..., 1::2]
            turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        out.append(torch.cat([turned, rest], -1).to(x.dtype))
    return {"q": out[0], "k": out[1]}


def _places(s, lengths, cu, T):
    """Flat (token, head) indices of packed tokens' slots and blocks."""
    c = s["case"]
    bs = c["block"]
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu[1:], t.int(), right=True)
    slot = lengths[b].long() + t - cu[b]
    h = torch.arange(c["Hkv"], device="cuda")
    if c["layout"] == "paged":
        block = s["table"][b, slot // bs].long()[:, None] * c["Hkv"] + h
        return block * bs + (slot % bs)[:, None], block, slot
    row = s["slot_ids"][b].long() if s["slot_ids"] is not None else b
    line = row[:, None] * c["Hkv"] + h
    return line * c["Smax"] + slot[:, None], line * (c["Smax"] // bs) + (slot // bs)[:, None], slot


def _plain_write(s):
    c = s["case"]
    bs, D = c["block"], c["D"]
    at, block, slot = _places(s, s["lengths"], s["cu_q"], s["T"])
    # of every row the slots before its first token in that token's block
    one = torch.arange(c["B"] + 1, dtype=torch.int32, device="cuda")
    _, first, begin = _places(s, s["lengths"], one, c["B"])
    inner = torch.arange(bs, device="cuda")
    held = inner < (begin % bs)[:, None]                                   # (B, bs)
    if c["layout"] == "paged":
        old = first[..., None] * bs + inner                                # (B, Hkv, bs)
    else:
        nb = c["Smax"] // bs
        old = (first // nb * c["Smax"] + first % nb * bs)[..., None] + inner
    for name in ("k", "v"):
        x = s[name + "_new"].float()
        flat, scale = s[name].view(-1, D), s[name + "s"].view(-1)
        top = torch.zeros_like(scale).scatter_reduce_(0, block.flatten(), x.abs().amax(-1).flatten(), "amax")
        top = top / torch.full_like(top, 127.0)                            # a division, not a product with 1 / 127
        fresh = torch.zeros_like(scale, dtype=torch.bool)
        fresh[block[slot % bs == 0].flatten()] = True
        was = scale.clone()
        mr, er = torch.frexp(top)
        ms, es = torch.frexp(was)
        k = (er - es + (mr > ms).int()).clamp(min=0)
        k = torch.where((top > was) & (was > 0), k, 0)
        now = torch.where(fresh | (was == 0), top, torch.ldexp(was, k))
        hit = torch.zeros_like(fresh)
        hit[block.flatten()] = True
        scale.copy_(torch.where(hit, now, was))
        less = torch.exp2(-k.float())[first][..., None, None]              # (B, Hkv, 1, 1)
        was8 = flat[old].float()
        flat[old] = torch.where((held[:, None] & ~fresh[first][..., None])[..., None], torch.round(was8 * less), was8).to(torch.int8)
        t = scale[block][..., None]
        flat[at] = torch.round(torch.where(t > 0, x / t, 0.0)).clamp(-127, 127).to(torch.int8)


def _plain_read(s, lengths, cu, T, dtype):
    at, block, _ = _places(s, lengths, cu, T)
    got = [s[n].view(-1, s["case"]["D"])[at] for n in ("k", "v")]
    if "ks" in s:
        got = [x.float() * s[n].view(-1)[block][..., None] for x, n in zip(got, ("ks", "vs"))]
    return [x.to(dtype) for x in got]


def _rows(s, name):
    """The batch's cache rows as float32 (B, Hkv, Smax, D)."""
    c = s["case"]
    x = s[name]
    if c["layout"] == "paged":
        page = s["table"].clamp(min=0).long()
        x = x[page].float()
        if c["kind"] == "int8":
            x = x * s[name + "s"][page][..., None, None]
        return x.transpose(1, 2).flatten(2, 3)
    rows = slice(0, c["B"]) if s["slot_ids"] is None else s["slot_ids"].long()
    y = x[rows].float()
    if c["kind"] == "int8":
        y = (y.unflatten(2, (-1, c["block"])) * s[name + "s"][rows][..., None, None]).flatten(2, 3)
    return y


def _plain_attend(s):
    c = s["case"]
    B, Hkv, Hq, D, Smax = c["B"], c["Hkv"], c["Hq"], c["D"], c["Smax"]
    n = s["lengths"] + (1 if c["step"] == "decode" else 0)
    j = torch.arange(Smax, device="cuda")
    ok = j < n[:, None]
    if c["window"]:
        ok = ok & (j >= n[:, None] - c["window"])
    ok = ok[:, None, None]                                                 # (B, 1, 1, Smax)
    x = (s["q"].float().view(B, Hkv, -1, D) @ _rows(s, "k").transpose(-1, -2)) * (1.0 / math.sqrt(D))
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    if c["slopes"]:
        x = x + s["slopes"].view(1, Hkv, -1, 1) * (j - (n[:, None] - 1)).float()[:, None, None]
    x = torch.where(ok, x, -math.inf)
    w = torch.exp(x - x.amax(-1, keepdim=True))
    w = w / w.sum(-1, keepdim=True)
    out = (w @ torch.where(ok[:, :, 0, :, None], _rows(s, "v"), 0.0)).view(B, Hq, D)
    if not c["weights"]:
        return out
    mass = torch.where(ok[:, :, 0], w.sum(2), 0.0)                         # (B, Hkv, Smax)
    if c["layout"] == "paged":
        real = s["table"] >= 0
        s["weights"][s["table"][real].long()] += mass.unflatten(2, (-1, c["block"])).transpose(1, 2)[real]
    else:
        rows = s["slot_ids"].long() if s["slot_ids"] is not None else torch.arange(B, device="cuda")
        s["weights"][rows] += mass
    return out


def _plain_evict(s):
    c = s["case"]
    B, Hkv, D, n_keep = c["B"], c["Hkv"], c["D"], c["n_keep"]
    n = s["lengths"].long()[:, None, None]
    j = torch.arange(c["Smax"], device="cuda")
    if c["layout"] == "paged":
        page = s["table"].clamp(min=0).long()
        w, k, v = (x[page].transpose(1, 2).flatten(2, 3) for x in (s["weights"], s["k"].view(torch.uint8), s["v"].view(torch.uint8)))
    else:
        rows = s["slot_ids"].long() if s["slot_ids"] is not None else torch.arange(B, device="cuda")
        w, k, v = s["weights"][rows], s["k"].view(torch.uint8)[rows], s["v"].view(torch.uint8)[rows]
    key = torch.where((j < c["n_first"]) | (j >= n - c["n_last"]), math.inf, w)
    key = torch.where(j < n, key, -math.inf)
    ids = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :n_keep]
    ids = torch.where(ids < n, ids, c["Smax"]).sort(-1).values
    if n_keep > c["Smax"]:
        ids = torch.cat([ids, ids.new_full((B, Hkv, n_keep - c["Smax"]), c["Smax"])], -1)
    some = ids < c["Smax"]
    at = ids.clamp(max=c["Smax"] - 1)
    for out, x in ((s["k2"], k), (s["v2"], v)):
        y = torch.gather(x, 2, at[..., None].expand(-1, -1, -1, x.shape[-1]))
        out.view(torch.uint8).copy_(torch.where(some[..., None], y, out.view(torch.uint8)))
    s["w2"].copy_(torch.where(some, torch.gather(w, 2, at), 0.0))
    return torch.where(some, ids, -1).int(), s["lengths"].clamp(max=n_keep)


# ---------------------------------------------------------------- one pass --

def _values(x):
    """What 8-bit vectors stand for (others as they are)."""
    return x.float() if x.dtype == torch.float8_e4m3fn else x


def run(s):
    if own:
        return _own(s)
    c = s["case"]
    if c["op"] == "rotate":
        return _plain_rotate(s)
    if c["op"] == "write":
        _plain_write(s)
        k, v = _plain_read(s, s["read_at"], s["read_cu"], s["read_T"], torch.bfloat16 if c["out"] == "bf16" else torch.float32)
        return {"k": k, "v": v, "k_scale": s["ks"], "v_scale": s["vs"]}
    if c["op"] == "evict":
        ids, lengths = _plain_evict(s)
        return {"ids": ids, "lengths": lengths, "k": _values(s["k2"]), "v": _values(s["v2"]), "weights": s["w2"]}
    if c["step"] == "decode":
        if c["kind"] == "int8":
            _plain_write(s)
        else:
            at, _, _ = _places(s, s["lengths"], s["cu_q"], s["T"])
            s["k"].view(-1, c["D"])[at] = s["k_new"]
            s["v"].view(-1, c["D"])[at] = s["v_new"]
    got = {}
    if c["weights"]:
        s["weights"].zero_()
        got["weights"] = s["weights"]
    got["out"] = _plain_attend(s)
    if c["step"] == "decode":
        got["k"], got["v"] = _plain_read(s, s["lengths"], s["cu_q"], s["T"], torch.bfloat16)
        if "ks" in s:
            got["k_scale"], got["v_scale"] = s["ks"], s["vs"]
    return got


def _own(s):
    import gqa_kv_cache_gb300 as gqa

    c = s["case"]
    if c["op"] == "rotate":
        q, k = gqa.rotate(s["q"], s["k"], s["rotary"], s["positions"])
        return {"q": q, "k": k}
    paged = c["layout"] == "paged"
    if c["op"] == "evict":
        kw = dict(n_first=c["n_first"], n_last=c["n_last"], k_out=s["k2"], v_out=s["v2"], weights_out=s["w2"])
        if paged:
            ids, lengths = gqa.evict_paged(s["k"], s["v"], s["table"], s["weights"], s["lengths"], c["n_keep"], **kw)
        else:
            ids, lengths = gqa.evict(s["k"], s["v"], s["weights"], s["lengths"], c["n_keep"], s["slot_ids"], **kw)
        return {"ids": ids, "lengths": lengths, "k": _values(s["k2"]), "v": _values(s["v2"]), "weights": s["w2"]}
    kw = dict(k_block_scale=s["ks"], v_block_scale=s["vs"]) if "ks" in s else {}
    if c["op"] == "write":
        dtype = torch.bfloat16 if c["out"] == "bf16" else torch.float32
        if paged:
            gqa.append_paged(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["lengths"], s["cu_q"], **kw)
            k, v = gqa.read_paged(s["k"], s["v"], s["table"], s["read_at"], s["read_cu"], s["read_T"], dtype=dtype, **kw)
        else:
            gqa.append(s["k_new"], s["v_new"], s["k"], s["v"], s["lengths"], s["cu_q"], s["slot_ids"], **kw)
            k, v = gqa.read(s["k"], s["v"], s["read_at"], s["read_cu"], s["read_T"], s["slot_ids"], dtype=dtype, **kw)
        return {"k": k, "v": v, "k_scale": s["ks"], "v_scale": s["vs"]}
    if c["cap"]:
        kw["score_cap"] = c["cap"]
    if c["slopes"]:
        kw["head_slopes"] = s["slopes"]
    if c["window"]:
        kw["window"] = c["window"]
    if c["weights"]:
        s["weights"].zero_()
        kw["weights"] = s["weights"]
    if c["step"] == "decode":
        if paged:
            out = gqa.decode_step_paged(s["q"], s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["lengths"], **kw)
        else:
            out = gqa.decode_step(s["q"], s["k_new"], s["v_new"], s["k"], s["v"], s["lengths"], s["slot_ids"], **kw)
    elif paged:
        out = gqa.attend_paged(s["q"], s["k"], s["v"], s["table"], s["lengths"], **kw)
    else:
        out = gqa.attend(s["q"], s["k"], s["v"], s["lengths"], s["slot_ids"], **kw)
    got = {"out": out, "weights": s["weights"]} if c["weights"] else {"out": out}
    if c["step"] == "decode":
        scales = dict(k_block_scale=s["ks"], v_block_scale=s["vs"]) if "ks" in s else {}
        if paged:
            got["k"], got["v"] = gqa.read_paged(s["k"], s["v"], s["table"], s["lengths"], s["cu_q"], s["T"], **scales)
        else:
            got["k"], got["v"] = gqa.read(s["k"], s["v"], s["lengths"], s["cu_q"], s["T"], s["slot_ids"], **scales)
        if scales:
            got["k_scale"], got["v_scale"] = s["ks"], s["vs"]
    return got


# ------------------------------------------------------ 64-bit definitions --

def _turns(c):
    """Angle a position of every pair, by a loop over the pairs, and m."""
    k, out = SCALING[c["scaling"]], []
    for i in range(c["dim"] // 2):
        e = 2 * i / c["dim"]
        f = math.exp(-e * math.log(c["base"]))
        if k and k["kind"] == "linear":
            f /= k["factor"]
        elif k and k["kind"] == "ntk":
            f = math.exp(-e * (math.log(c["base"]) + math.log(k["factor"]) * c["dim"] / (c["dim"] - 2)))
        elif k:
            r = k["original"] * f / (2 * math.pi)
            u = min(1.0, max(0.0, (r - k["low"]) / (k["high"] - k["low"])))
            f = u * f + (1 - u) * f / k["factor"]
        out.append(f)
    return torch.tensor(out, dtype=torch.float64, device="cuda"), (k or {}).get("attention", 1.0)


def _exact_rotate(s):
    c = s["case"]
    f, m = _turns(c)
    got = {}
    for name in ("q", "k"):
        x, parts = s[name], []
        step = max(1, CHUNK // (x.shape[1] * x.shape[2] * 4))
        for t in range(0, c["T"], step):
            y = x[t:t + step].double()
            turn = torch.polar(torch.full_like(f, m).expand(y.shape[0], -1), s["positions"][t:t + step].double()[:, None] * f)[:, None]
            head = y[..., :c["dim"]]
            z = torch.complex(*head.chunk(2, -1)) if c["style"] == "half" else torch.view_as_complex(head.unflatten(-1, (-1, 2)).contiguous())
            z = z * turn
            z = torch.cat([z.real, z.imag], -1) if c["style"] == "half" else torch.view_as_real(z).flatten(-2)
            parts.append(torch.cat([z, y[..., c["dim"]:]], -1))
        got[name] = torch.cat(parts)
    return got


def _row_of(s, b):
    return int(s["slot_ids"][b]) if s["slot_ids"] is not None else b


def _written(s, name):
    """Per row the blocks that hold the row's new tokens after the write: codes
    (Hkv, n, block, D) and scales (Hkv, n), both in 64 bits, their places and the first slot."""
    c = s["case"]
    bs, Hkv, D = c["block"], c["Hkv"], c["D"]
    lens, cu = s["lengths"].tolist(), s["cu_q"].tolist()
    for b in range(c["B"]):
        n, m = lens[b], cu[b + 1] - cu[b]
        j0, j1 = n // bs, -(-(n + m) // bs)
        if c["layout"] == "paged":
            where = (s["table"][b, j0:j1].long(),)
            codes, t0 = s[name][where[0]].transpose(0, 1), s[name + "s"][where[0]].T
        else:
            r = _row_of(s, b)
            where = (r, j0, j1)
            codes = s[name][r].view(Hkv, -1, bs, D)[:, j0:j1]
            t0 = s[name + "s"][r, :, j0:j1]
        codes, t = codes.double().contiguous().clone(), t0.double().clone()
        x = s[name + "_new"][cu[b]:cu[b + 1]].double().transpose(0, 1)               # (Hkv, m, D)
        line = torch.zeros(Hkv, (j1 - j0) * bs, D, dtype=torch.float64, device="cuda")
        at = n - j0 * bs
        line[:, at:at + m] = x
        line = line.view(Hkv, -1, bs, D)
        r = (line.abs().amax((2, 3)) / 127).float().double()
        fine = r.clone()
        if at:                                                                       # the first block goes on
            a, w = t[:, 0], r[:, 0]
            k = torch.ceil(torch.log2(torch.where((a > 0) & (w > a), w / a, 1.0))).clamp(min=0)
            k = torch.where((a > 0) & (a * torch.exp2(k) < w), k + 1, k)
            fine[:, 0] = torch.where(a > 0, a * torch.exp2(k), w)
            codes[:, 0, :at] = torch.round(codes[:, 0, :at] * torch.exp2(-k)[:, None, None])
        quot = torch.where(fine[..., None, None] > 0, line / fine.clamp(min=1e-300)[..., None, None], 0.0).float().double()
        new = torch.round(quot).clamp(-127, 127).flatten(1, 2)
        codes.view(Hkv, -1, D)[:, at:at + m] = new[:, at:at + m]
        yield b, codes, fine, where, at + m


def _exact_write(s):
    got = {}
    for name in ("k", "v"):
        parts, scales = [], s[name + "s"].double().clone()
        for b, codes, t, where, n in _written(s, name):
            parts.append((codes * t[..., None, None]).flatten(1, 2)[:, :n].transpose(0, 1))
            if len(where) == 1:
                scales[where[0]] = t.T
            else:
                scales[where[0], :, where[1]:where[2]] = t
        got[name], got[name + "_scale"] = torch.cat(parts), scales
    return {n: got[n] for n in ("k", "v", "k_scale", "v_scale")}


def _exact_attend(s):
    c = s["case"]
    Hkv, bs, D = c["Hkv"], c["block"], c["D"]
    lens = s["lengths"].tolist()
    new, got = {}, {}
    if c["step"] == "decode":
        got = {"k": s["k_new"].double(), "v": s["v_new"].double()}
        if c["kind"] == "int8":
            for name in ("k", "v"):
                new[name] = {b: (codes * t[..., None, None]).flatten(1, 2)[:, :n] for b, codes, t, _, n in _written(s, name)}
                got[name] = torch.stack([new[name][b][:, -1] for b in range(c["B"])])
            got = {**got, "k_scale": None, "v_scale": None}               # held in the write's cases
    mass = torch.zeros_like(s["weights"], dtype=torch.float64) if c["weights"] else None
    outs = []
    for b in range(c["B"]):
        n = lens[b] + (c["step"] == "decode")
        lo = max(0, n - c["window"]) if c["window"] else 0
        pair = []
        for name in ("k", "v"):
            if c["layout"] == "paged":
                pages = s["table"][b, :-(-n // bs)].long()
                x = s[name][pages].double()
                if c["kind"] == "int8":
                    x = x * s[name + "s"][pages].double()[..., None, None]
                x = x.permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :n]
            else:
                r = _row_of(s, b)
                x = s[name][r, :, :n].double()
                if c["kind"] == "int8":
                    x = x * torch.repeat_interleave(s[name + "s"][r].double(), bs, -1)[:, :n, None]
            x = x.clone()
            if c["step"] == "decode":
                if c["kind"] == "int8":
                    x[:, n - new[name][b].shape[1]:] = new[name][b]
                else:
                    x[:, n - 1] = s[name + "_new"][b].double()
            pair.append(x[:, lo:])
        z = torch.einsum("hgd,hnd->hgn", s["q"][b].double().view(Hkv, -1, D), pair[0]) / math.sqrt(D)
        if c["cap"]:
            z = torch.tanh(z / c["cap"]) * c["cap"]
        if c["slopes"]:
            z = z - s["slopes"].double().view(Hkv, -1, 1) * torch.arange(n - 1 - lo, -1, -1, device="cuda").double()
        p = torch.softmax(z, -1)
        outs.append(torch.einsum("hgn,hnd->hgd", p, pair[1]).reshape(c["Hq"], D))
        if mass is not None:
            w = p.sum(1)
            if c["layout"] == "paged":
                full = torch.zeros(Hkv, -(-n // bs) * bs, dtype=torch.float64, device="cuda")
                full[:, lo:n] = w
                mass[s["table"][b, :-(-n // bs)].long()] = full.view(Hkv, -1, bs).transpose(0, 1)
            else:
                mass[_row_of(s, b), :, lo:n] = w
    got["out"] = torch.stack(outs)
    return {**got, "weights": mass} if c["weights"] else got


def _exact_evict(s):
    c = s["case"]
    got = {"k": s["k2"].double(), "v": s["v2"].double(), "weights": torch.zeros_like(s["w2"], dtype=torch.float64)}
    for b, n in enumerate(s["lengths"].tolist()):
        for name, x in (("weights", s["weights"]), ("k", s["k"]), ("v", s["v"])):
            if c["layout"] == "paged":
                x = x[s["table"][b, :-(-n // c["block"])].long()].transpose(0, 1).flatten(1, 2)[:, :n]
            else:
                x = x[_row_of(s, b), :, :n]
            if name == "weights":
                chosen = torch.arange(n, device="cuda").expand(c["Hkv"], -1)
                if n > c["n_keep"]:
                    rank = x[:, c["n_first"]:n - c["n_last"]].double()
                    order = torch.argsort(-rank, dim=-1, stable=True)[:, :c["n_keep"] - c["n_first"] - c["n_last"]]
                    ends = torch.cat([chosen[:, :c["n_first"]], chosen[:, n - c["n_last"]:]], 1)
                    chosen = torch.cat([ends, order + c["n_first"]], 1).sort(-1).values
            for h in range(c["Hkv"]):
                got[name][b, h, :chosen.shape[1]] = x[h].double()[chosen[h]]
    return {"ids": None, "lengths": None, **got}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotate":
        return _exact_rotate(s)
    if case["op"] == "write":
        return _exact_write(s)
    if case["op"] == "attend":
        return _exact_attend(s)
    return _exact_evict(s)
