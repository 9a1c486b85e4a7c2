"""Measured cases of the cache operators: writing tokens into a quantised cache
and reading them back, attention over a 4-bit (E2M1) cache, and sparse
attention over the blocks that a bound on the scores selects.

An E2M1 cache holds D / 2 bytes a vector (dim 2i in the low nibble of byte i),
one E4M3 scale per 16 dims and one float32 scale g per cache head:

    s = E4M3(min(max|x| / (6 g), 448)),  t = s g,  value = E2M1(x / t) t

with round to nearest, ties to even (and 0 where t is 0).

Sizes are the repository's decode workloads (llama3_8b, long_context,
ragged_slots, paged, pr1_fp32) and smaller or ragged ones around them.
"""
import math
import random

import torch

own = False

GROUP = 16
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
CHUNK = 1 << 26


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one decode step's new tokens, llama3_8b heads: a launch-bound write
        dict(name="write_token", op="write", kind="e2m1", layout="dense", B=32, R=32, Hkv=8, D=128, Smax=4096,
             block=16, bounds=True, q_lo=1, q_hi=1, len_lo=1024, len_hi=4094, out="bf16", key_scale=1.0),
        # speculative tokens of 256 sequences into an E4M3 cache by slot id
        dict(name="write_spec_e4m3", op="write", kind="e4m3", layout="slots", B=256, R=512, Hkv=4, D=128, Smax=8192,
             block=64, bounds=False, q_lo=1, q_hi=8, len_lo=16, len_hi=8183, out="bf16", key_scale=1.0),
        # ragged prompts into a paged 4-bit cache, key bounds kept for selection
        dict(name="write_prompts_paged", op="write", kind="e2m1", layout="paged", B=64, R=0, Hkv=8, D=128, Smax=2112,
             block=16, bounds=True, q_lo=1, q_hi=2047, len_lo=0, len_hi=61, out="bf16", key_scale=1.0),
        # one very long prompt
        dict(name="write_long", op="write", kind="e2m1", layout="dense", B=1, R=1, Hkv=8, D=128, Smax=131072,
             block=64, bounds=True, q_lo=131071, q_hi=131071, len_lo=0, len_hi=0, out="bf16", key_scale=3.0),
        # pr1_fp32's sizes: two short sequences, float32 queries, D = 64
        dict(name="attend_small", op="attend", step="attend", layout="dense", B=2, R=2, Hq=8, Hkv=2, D=64, Smax=256,
             block=16, len_lo=1, len_hi=255, dist="uniform", q="f32", key_scale=1.0),
        # llama3_8b's decode step (append and attend)
        dict(name="decode_llama3_8b", op="attend", step="decode", layout="dense", B=32, R=32, Hq=32, Hkv=8, D=128,
             Smax=4096, block=16, len_lo=1024, len_hi=4095, dist="uniform", q="bf16", key_scale=1.0),
        # four long contexts, G = 8
        dict(name="attend_long_context", op="attend", step="attend", layout="dense", B=4, R=4, Hq=64, Hkv=8, D=128,
             Smax=131072, block=64, len_lo=32768, len_hi=131071, dist="uniform", q="bf16", key_scale=3.0),
        # continuous batching with very uneven lengths, float32 queries
        dict(name="attend_ragged_slots", op="attend", step="attend", layout="slots", B=256, R=512, Hq=32, Hkv=4, D=128,
             Smax=8192, block=16, len_lo=16, len_hi=8191, dist="log", q="f32", key_scale=1.0),
        # the paged workload, 16-slot blocks, G = 6
        dict(name="attend_paged", op="attend", step="attend", layout="paged", B=64, R=0, Hq=48, Hkv=8, D=128,
             Smax=16384, block=16, len_lo=512, len_hi=16383, dist="uniform", q="bf16", key_scale=1.0),
        # one sequence, few blocks kept: latency
        dict(name="sparse_one_row", op="sparse", kind="e2m1", layout="dense", B=1, R=1, Hq=32, Hkv=8, D=128, Smax=8192,
             block=32, n_select=16, n_first=1, n_last=2, len_lo=8001, len_hi=8001, dist="uniform", q="bf16",
             key_scale=1.0),
        # four long contexts over a bfloat16 cache, 64 of up to 2048 blocks kept
        dict(name="sparse_long_bf16", op="sparse", kind="bf16", layout="dense", B=4, R=4, Hq=64, Hkv=8, D=128,
             Smax=131072, block=64, n_select=64, n_first=1, n_last=1, len_lo=32768, len_hi=131071, dist="uniform",
             q="bf16", key_scale=3.0),
        # the paged workload over a 4-bit cache, 64 of up to 1024 blocks kept
        dict(name="sparse_paged", op="sparse", kind="e2m1", layout="paged", B=64, R=0, Hq=48, Hkv=8, D=128, Smax=16384,
             block=16, n_select=64, n_first=1, n_last=4, len_lo=512, len_hi=16383, dist="uniform", q="bf16",
             key_scale=1.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["write", "attend", "attend", "sparse", "sparse"])
    layout = rng.choice(["dense", "slots", "paged"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.randint(1, 8)
    if op == "write":
        B = _log(rng, 1, 128)
        q_hi = _log(rng, 1, max(1, 65536 // B))
        q_lo = rng.randint(1, q_hi)
        block = rng.choice([8, 16, 32, 64])
        len_hi = rng.choice([0, rng.randint(1, 500)])
        Smax = -(-(len_hi + q_hi) // block) * block
        return dict(op=op, kind=rng.choice(["e2m1", "e2m1", "e4m3"]), layout=layout, B=B,
                    R=0 if layout == "paged" else B + (rng.randint(0, B) if layout == "slots" else 0), Hkv=Hkv, D=D,
                    Smax=Smax, block=block, bounds=rng.random() < 0.5, q_lo=q_lo, q_hi=q_hi, len_lo=0, len_hi=len_hi,
                    out=rng.choice(["bf16", "f32"]), key_scale=1.0)
    room = 4 * 131072 * 8 * 128 // (2 if op == "sparse" else 1)   # elements of a case's keys
    Smax = _log(rng, 64, 131072)
    B = _log(rng, 1, max(1, min(256, room // (Smax * Hkv * D * 2))))
    block = rng.choice([8, 16, 32, 64]) if op == "attend" else rng.choice([16, 32, 64])
    if op == "sparse":
        block = max(block, -(-Smax // 8192))
        block = 16 if block <= 16 else 32 if block <= 32 else 64
    if layout == "paged" or op == "sparse":
        Smax = -(-Smax // block) * block
    lo = rng.randint(1, max(1, Smax // 2))
    case = dict(op=op, layout=layout, B=B, R=0 if layout == "paged" else B + (rng.randint(0, B) if layout == "slots" else 0),
                Hq=Hq, Hkv=Hkv, D=D, Smax=Smax, block=block, len_lo=lo, len_hi=Smax - 1,
                dist=rng.choice(["uniform", "log"]), q=rng.choice(["bf16", "f32"]), key_scale=rng.choice([1.0, 3.0]))
    if op == "attend":
        case["step"] = rng.choice(["attend", "decode"])
        if case["step"] == "decode":
            case["q"] = "bf16"
        return case
    case["kind"] = rng.choice(["e2m1", "bf16"])
    case["n_select"] = _log(rng, 4, max(4, min(256, Smax // block)))
    case["n_first"] = rng.randint(0, 2)
    case["n_last"] = rng.randint(1, 2)
    return case


def _spread(n, lo, hi, log=False):
    """n lengths spread evenly over lo..hi (or over their logarithm)."""
    if not log:
        return [lo + int((hi - lo + 1) * (i + 0.5) / n) for i in range(n)]
    a, b = math.log(max(lo, 1)), math.log(hi + 1)
    return [min(hi, max(lo, int(math.exp(a + (b - a) * (i + 0.5) / n)))) for i in range(n)]


def _row_bytes(case):
    kind, D = case.get("kind", "e2m1"), case["D"]
    return D // 2 + D // GROUP if kind == "e2m1" else D if kind == "e4m3" else 2 * D


def work(case):
    B, Hkv, D, row = case["B"], case["Hkv"], case["D"], _row_bytes(case)
    if case["op"] == "write":
        T = sum(_spread(B, case["q_lo"], case["q_hi"]))
        es = 2 if case["out"] == "bf16" else 4
        n = 2 * T * Hkv * (2 * D + 2 * row + es * D)
        if case["bounds"]:
            n += T * Hkv * 4 * D // case["block"]
        return {"bytes": n, "flops": 2 * T * Hkv * D * 4}
    lens = _spread(B, case["len_lo"], case["len_hi"], case["dist"] == "log")
    Hq = case["Hq"]
    n = B * Hq * D * ((2 if case["q"] == "bf16" else 4) + 4)
    if case["op"] == "attend":
        if case["step"] == "decode":
            n += 2 * B * Hkv * (4 * D + 2 * row)
        return {"bytes": n + sum(lens) * Hkv * 2 * row, "flops": 4 * sum(lens) * Hq * D}
    bs, k = case["block"], case["n_select"]
    blocks = sum(-(-v // bs) for v in lens)
    slots = sum(min(v, k * bs - (-v) % bs) for v in lens)
    return {"bytes": n + blocks * Hkv * 4 * D + slots * Hkv * 2 * row + 4 * B * Hkv * k,
            "flops": blocks * Hkv * 4 * D + 4 * slots * Hq * D}


# ----------------------------------------------------------------- inputs --

def _normal(shape, gen, scale=1.0, dtype=torch.bfloat16):
    out = torch.empty(math.prod(shape), dtype=dtype, device="cuda")
    for i in range(0, out.numel(), CHUNK):
        m = min(CHUNK, out.numel() - i)
        out[i:i + m] = torch.randn(m, generator=gen, device="cuda").mul_(scale).to(dtype)
    return out.view(shape)


def _quantised(shape, gen, scale, g):
    """A cache of N(0, scale^2) values (..., Hkv, slots, D) as E2M1 codes and
    group scales, a chunk of its first axis at a time."""
    codes = torch.empty(*shape[:-1], shape[-1] // 2, dtype=torch.uint8, device="cuda")
    groups = torch.empty(*shape[:-1], shape[-1] // GROUP, dtype=torch.uint8, device="cuda")
    step = max(1, CHUNK // math.prod(shape[1:]))
    for i in range(0, shape[0], step):
        n = min(step, shape[0] - i)
        x = torch.randn((n, *shape[1:]), generator=gen, device="cuda").mul_(scale)
        codes[i:i + n], groups[i:i + n] = _to_e2m1(x, g.view(-1, 1, 1))
    return codes, groups


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    rng = random.Random(seed)
    c = dict(case)
    B, Hkv, D, Smax, bs = c["B"], c["Hkv"], c["D"], c["Smax"], c["block"]
    kind = c.get("kind", "e2m1")
    s = {"case": c}
    # heads' largest values differ by up to a third
    top = 5.0 * (0.75 + 0.5 * torch.rand(2, Hkv, generator=gen, device=dev)) / (448.0 * (6.0 if kind == "e2m1" else 1.0))
    s["k_scale"], s["v_scale"] = (top[0] * c["key_scale"]).contiguous(), top[1].contiguous()
    if c["op"] == "write":
        q_lens = _spread(B, c["q_lo"], c["q_hi"])
        lens = _spread(B, c["len_lo"], c["len_hi"])
    else:
        lens = _spread(B, c["len_lo"], c["len_hi"], c["dist"] == "log")
        q_lens = [1] * B
    rng.shuffle(lens)
    rng.shuffle(q_lens)
    s["lengths"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    cu = [0]
    for n in q_lens:
        cu.append(cu[-1] + n)
    s["cu_q"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    s["T"] = cu[-1]
    if c["layout"] == "paged":
        nb = Smax // bs
        shape = (B * nb, Hkv, bs, D)
        s["table"] = torch.randperm(B * nb, generator=gen, device=dev).view(B, nb).to(torch.int32)
        held = torch.tensor([-(-(a + (n if c["op"] == "write" or c.get("step") == "decode" else 0)) // bs)
                             for a, n in zip(lens, q_lens)], device=dev)
        s["table"] = torch.where(torch.arange(nb, device=dev) < held[:, None], s["table"], -1)
    else:
        shape = (c["R"], Hkv, Smax, D)
        s["slot_ids"] = (torch.randperm(c["R"], generator=gen, device=dev)[:B].to(torch.int32)
                         if c["layout"] == "slots" else None)
    if c["op"] == "write" or c.get("step") == "decode":
        s["k_new"] = _normal((s["T"], Hkv, D), gen, c["key_scale"])
        s["v_new"] = _normal((s["T"], Hkv, D), gen)
    if c["op"] == "write":
        width = D // 2 if kind == "e2m1" else D
        s["k"] = torch.zeros((*shape[:-1], width), dtype=torch.uint8, device=dev)
        s["v"] = torch.zeros_like(s["k"])
        if kind == "e2m1":
            s["kg"] = torch.zeros((*shape[:-1], D // GROUP), dtype=torch.uint8, device=dev)
            s["vg"] = torch.zeros_like(s["kg"])
        if c["bounds"]:
            flat = shape[:2] if c["layout"] == "paged" else (*shape[:2], Smax // bs)
            s["bounds"] = torch.zeros((*flat, 2, D), dtype=torch.bfloat16, device=dev)
            s["bounds"][..., 0, :] = -0.5      # the block's earlier tokens
            s["bounds"][..., 1, :] = 0.5
        return s
    s["q"] = _normal((B, c["Hq"], D), gen, dtype=torch.float32 if c["q"] == "f32" else torch.bfloat16)
    if kind == "bf16":
        s["k"] = _normal(shape, gen, c["key_scale"])
        s["v"] = _normal(shape, gen)
    else:
        s["k"], s["kg"] = _quantised(shape, gen, c["key_scale"], s["k_scale"])
        s["v"], s["vg"] = _quantised(shape, gen, 1.0, s["v_scale"])
    if c["op"] == "sparse":
        s["bounds"] = _bounds_of(s)
    return s


def _bounds_of(s):
    """Element-wise smallest and largest key of every block of a prepared
    cache, over its valid slots."""
    c = s["case"]
    bs, D = c["block"], c["D"]
    kind = c["kind"]
    k = s["k"] if c["layout"] == "paged" else s["k"].view(c["R"], c["Hkv"], -1, bs, s["k"].shape[-1])
    valid = torch.full(k.shape[:-2], bs, dtype=torch.int32, device="cuda")
    j = torch.arange(c["Smax"] // bs, device="cuda")
    left = (s["lengths"][:, None] - j * bs).clamp(0, bs).int()       # slots each block of a row holds
    if c["layout"] == "paged":
        at = s["table"] >= 0
        valid[s["table"][at].long()] = left[at][:, None]
    else:
        rows = s["slot_ids"].long() if s["slot_ids"] is not None else torch.arange(c["B"], device="cuda")
        valid[rows] = left[:, None]
    kg = None if kind == "bf16" else s["kg"].view(*k.shape[:-1], c["D"] // GROUP)
    out = torch.empty((*k.shape[:-2], 2, D), dtype=torch.bfloat16, device="cuda")
    step = max(1, CHUNK // max(1, k[0].numel()))
    shape = (-1, 1, 1) if c["layout"] == "paged" else (-1, 1, 1, 1)
    for i in range(0, k.shape[0], step):
        x = k[i:i + step].float() if kind == "bf16" else _of_e2m1(k[i:i + step], kg[i:i + step],
                                                                  s["k_scale"].view(shape))
        ok = (torch.arange(bs, device="cuda") < valid[i:i + step, ..., None])[..., None]
        out[i:i + step, ..., 0, :] = torch.where(ok, x, math.inf).amin(-2)
        out[i:i + step, ..., 1, :] = torch.where(ok, x, -math.inf).amax(-2)
    return out


# ------------------------------------------------------------ plain forms --

def _to_e2m1(x, g):
    """float32 x (..., D) with head scale g (broadcast to x[..., :1]) as packed
    codes (..., D / 2) and E4M3 group scales (..., D / 16)."""
    v = x.unflatten(-1, (-1, GROUP))
    amax = v.abs().amax(-1)
    groups = (amax / (g * 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    t = (groups.float() * g)[..., None]
    y = torch.where(t > 0, v / t, 0.0)
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code + 8 * torch.signbit(y).to(torch.uint8)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), groups.view(torch.uint8)


def _of_e2m1(codes, groups, g):
    """Values of packed codes (..., D / 2), float32."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    pair = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    t = groups.view(torch.float8_e4m3fn).float() * g
    return (lut[pair.int()].unflatten(-1, (-1, GROUP)) * t[..., None]).flatten(-2)


def _slots(s):
    """Flat index of the (token, head) slot of every packed token of a
    prepared state, and of the block it lies in."""
    c = s["case"]
    t = torch.arange(s["T"], device="cuda")
    b = torch.searchsorted(s["cu_q"][1:], t.int(), right=True)
    slot = s["lengths"][b].long() + t - s["cu_q"][b]
    h = torch.arange(c["Hkv"], device="cuda")
    bs = c["block"]
    if c["layout"] == "paged":
        page = s["table"][b, slot // bs].long()
        block = page[:, None] * c["Hkv"] + h
        return block * bs + (slot % bs)[:, None], block, slot
    row = s["slot_ids"][b].long() if s["slot_ids"] is not None else b
    line = row[:, None] * c["Hkv"] + h
    return line * c["Smax"] + slot[:, None], line * (c["Smax"] // bs) + (slot // bs)[:, None], slot


def _plain_write(s):
    """Quantises the new tokens into the cache."""
    c = s["case"]
    at, block, slot = _slots(s)
    for name in ("k", "v"):
        x, g = s[name + "_new"].float(), s[name + "_scale"].view(-1, 1)
        if c.get("kind", "e2m1") == "e2m1":
            codes, groups = _to_e2m1(x, g)
            s[name].view(-1, c["D"] // 2)[at] = codes
            s[name + "g"].view(-1, c["D"] // GROUP)[at] = groups
        else:
            y = (x / g).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
            s[name].view(-1, c["D"])[at] = y.view(torch.uint8)
    if c.get("bounds"):
        flat = s["bounds"].view(-1, 2, c["D"])
        fresh = block[slot % c["block"] == 0]              # blocks that begin with a new token
        flat[fresh, 0], flat[fresh, 1] = math.inf, -math.inf
        wide = flat.float()
        index = block.reshape(-1, 1).expand(-1, c["D"])
        keys = s["k_new"].float().view(-1, c["D"])
        wide[:, 0].scatter_reduce_(0, index, keys, "amin")
        wide[:, 1].scatter_reduce_(0, index, keys, "amax")
        flat.copy_(wide)


def _plain_read(s, dtype):
    c = s["case"]
    at, _, _ = _slots(s)
    out = []
    for name in ("k", "v"):
        g = s[name + "_scale"].view(-1, 1)
        if c.get("kind", "e2m1") == "e2m1":
            x = _of_e2m1(s[name].view(-1, c["D"] // 2)[at], s[name + "g"].view(-1, c["D"] // GROUP)[at], g)
        else:
            x = s[name].view(-1, c["D"])[at].view(torch.float8_e4m3fn).float() * g
        out.append(x.to(dtype))
    return out


def _rows(s, name):
    """The batch's cache rows as float32 (B, Hkv, Smax, D)."""
    c = s["case"]
    parts = [s[name]] if c.get("kind", "e2m1") == "bf16" else [s[name], s[name + "g"]]
    if c["layout"] == "paged":
        page = s["table"].clamp(min=0).long()
        parts = [p[page].transpose(1, 2).flatten(2, 3) for p in parts]
    elif s["slot_ids"] is not None:
        parts = [p[s["slot_ids"].long()] for p in parts]
    if len(parts) == 1:
        return parts[0].float()
    return _of_e2m1(parts[0], parts[1], s[name + "_scale"].view(-1, 1, 1))


def _softmax_sum(q, k, v, ok):
    """Attention of q (B, Hkv, G, D) over k, v (B, Hkv, S, D) where ok (B, Hkv or 1, S)."""
    x = (q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(q.shape[-1]))
    x = torch.where(ok[:, :, None], x, -math.inf)
    w = torch.exp(x - x.amax(-1, keepdim=True))
    return (w @ torch.where(ok[..., None], v, 0.0)) / w.sum(-1, keepdim=True)


def _plain_attend(s):
    c = s["case"]
    n = s["lengths"] + (1 if c["step"] == "decode" else 0)
    ok = (torch.arange(c["Smax"], device="cuda") < n[:, None])[:, None]
    q = s["q"].float().view(c["B"], c["Hkv"], -1, c["D"])
    return _softmax_sum(q, _rows(s, "k"), _rows(s, "v"), ok).view(c["B"], c["Hq"], c["D"])


def _plain_select(s):
    """Ids (B, Hkv, n_select) of the kept blocks, ascending, -1 after the last."""
    c = s["case"]
    bs, n = c["block"], c["n_select"]
    nb = c["Smax"] // bs
    if c["layout"] == "paged":
        box = s["bounds"][s["table"].clamp(min=0).long()].transpose(1, 2)
    elif s["slot_ids"] is not None:
        box = s["bounds"][s["slot_ids"].long()]
    else:
        box = s["bounds"]
    q = s["q"].double().view(c["B"], c["Hkv"], -1, c["D"])     # near scores are told apart in 64 bits
    up, down = q.clamp(min=0).sum(2), q.clamp(max=0).sum(2)
    score = (box[..., 1, :].double() @ up[..., None] + box[..., 0, :].double() @ down[..., None])[..., 0]
    blocks = ((s["lengths"] + bs - 1) // bs)[:, None, None]
    j = torch.arange(nb, device="cuda")
    score = torch.where((j < c["n_first"]) | (j >= blocks - c["n_last"]), math.inf, score)
    score = torch.where(j < blocks, score, -math.inf)
    kept = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :n]
    kept = torch.where(kept < blocks, kept, nb).sort(-1).values
    if n > nb:
        kept = torch.cat([kept, kept.new_full((*kept.shape[:-1], n - nb), nb)], -1)
    return torch.where(kept < nb, kept, -1).int()


def _plain_sparse(s):
    c = s["case"]
    bs, B, Hkv, D = c["block"], c["B"], c["Hkv"], c["D"]
    ids = _plain_select(s)
    j = ids.clamp(min=0).long()
    h = torch.arange(Hkv, device="cuda")[:, None]
    if c["layout"] == "paged":
        page = s["table"][torch.arange(B, device="cuda")[:, None, None], j].long()
        at = page * Hkv + h
    else:
        row = s["slot_ids"].long() if s["slot_ids"] is not None else torch.arange(B, device="cuda")
        at = (row[:, None, None] * Hkv + h) * (c["Smax"] // bs) + j
    got = []
    for name in ("k", "v"):
        x = s[name].view(-1, bs, s[name].shape[-1])[at]
        if c["kind"] != "bf16":
            x = _of_e2m1(x, s[name + "g"].view(-1, bs, D // GROUP)[at], s[name + "_scale"].view(-1, 1, 1, 1))
        got.append(x.float().flatten(2, 3))
    slot = j[..., None] * bs + torch.arange(bs, device="cuda")
    ok = ((ids >= 0)[..., None] & (slot < s["lengths"][:, None, None, None])).flatten(2)
    q = s["q"].float().view(B, Hkv, -1, D)
    return {"ids": ids, "out": _softmax_sum(q, got[0], got[1], ok).view(B, c["Hq"], D)}


# ---------------------------------------------------------------- one pass --

def run(s):
    if own:
        return _own(s)
    c = s["case"]
    if c["op"] == "write":
        _plain_write(s)
        k, v = _plain_read(s, torch.bfloat16 if c["out"] == "bf16" else torch.float32)
        return {"k": k, "v": v, "bounds": s["bounds"]} if c["bounds"] else {"k": k, "v": v}
    if c["op"] == "sparse":
        return _plain_sparse(s)
    if c["step"] == "attend":
        return {"out": _plain_attend(s)}
    _plain_write(s)
    k, v = _plain_read(s, torch.bfloat16)
    return {"out": _plain_attend(s), "k": k, "v": v}


def _own(s):
    import gqa_kv_cache_gb300 as gqa

    c = s["case"]
    kw = {}
    if c.get("kind", "e2m1") != "bf16":
        kw = dict(k_scale=s["k_scale"], v_scale=s["v_scale"])
        if "kg" in s:
            kw.update(k_group_scale=s["kg"], v_group_scale=s["vg"])
    paged = c["layout"] == "paged"
    if c["op"] == "write":
        dtype = torch.bfloat16 if c["out"] == "bf16" else torch.float32
        box = dict(k_bounds=s["bounds"]) if c["bounds"] else {}
        if paged:
            gqa.append_paged(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["lengths"], s["cu_q"], **kw, **box)
            k, v = gqa.read_paged(s["k"], s["v"], s["table"], s["lengths"], s["cu_q"], s["T"], dtype=dtype, **kw)
        else:
            gqa.append(s["k_new"], s["v_new"], s["k"], s["v"], s["lengths"], s["cu_q"], s["slot_ids"], **kw, **box)
            k, v = gqa.read(s["k"], s["v"], s["lengths"], s["cu_q"], s["T"], s["slot_ids"], dtype=dtype, **kw)
        return {"k": k, "v": v, **({"bounds": s["bounds"]} if c["bounds"] else {})}
    if c["op"] == "sparse":
        if paged:
            kept = gqa.select_blocks_paged(s["q"], s["bounds"], s["table"], s["lengths"], c["n_select"],
                                           block_size=c["block"], n_first=c["n_first"], n_last=c["n_last"])
        else:
            kept = gqa.select_blocks(s["q"], s["bounds"], s["lengths"], c["n_select"], s["slot_ids"],
                                     block_size=c["block"], n_first=c["n_first"], n_last=c["n_last"])
        return {"ids": kept.ids, "out": gqa.attend_selected(s["q"], s["k"], s["v"], kept, **kw)}
    if c["step"] == "attend":
        if paged:
            return {"out": gqa.attend_paged(s["q"], s["k"], s["v"], s["table"], s["lengths"], **kw)}
        return {"out": gqa.attend(s["q"], s["k"], s["v"], s["lengths"], s["slot_ids"], **kw)}
    if paged:
        out = gqa.decode_step_paged(s["q"], s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["lengths"], **kw)
        k, v = gqa.read_paged(s["k"], s["v"], s["table"], s["lengths"], s["cu_q"], s["T"], **kw)
    else:
        out = gqa.decode_step(s["q"], s["k_new"], s["v_new"], s["k"], s["v"], s["lengths"], s["slot_ids"], **kw)
        k, v = gqa.read(s["k"], s["v"], s["lengths"], s["cu_q"], s["T"], s["slot_ids"], **kw)
    return {"out": out, "k": k, "v": v}


# ------------------------------------------------------ 64-bit definitions --

def _round_to(x, low, drop):
    """x >= 0 in 64 bits to a format whose smallest normal is 2^low, with `drop` fraction bits; ties to even."""
    e = torch.floor(torch.log2(x.clamp(min=2.0 ** low)))
    e = torch.where(torch.exp2(e) > x.clamp(min=2.0 ** low), e - 1, e)
    step = torch.exp2(e - drop)
    return torch.round(x / step) * step


def _stored(x, g, kind):
    """What the cache holds for x (..., Hkv, D), head scales g (Hkv,), in 64 bits."""
    x, g = x.double(), g.double()[:, None]
    if kind == "e4m3":
        y = x / g
        return torch.sign(y) * _round_to(y.abs().clamp(max=448.0), -6, 3).clamp(max=448.0) * g
    v = x.reshape(*x.shape[:-1], -1, GROUP)
    s = _round_to((v.abs().max(-1).values / (6 * g)).clamp(max=448.0), -6, 3)
    t = (s * g)[..., None]
    y = torch.where(t > 0, v / t.clamp(min=1e-300), torch.zeros_like(v))
    return (torch.sign(y) * _round_to(y.abs().clamp(max=6.0), 0, 1).clamp(max=6.0) * t).reshape(x.shape)


def _e2m1_row(codes, groups, g):
    """Codes (Hkv, n, D / 2) of one row in 64 bits: sign, two exponent bits, one fraction bit."""
    n = torch.stack([codes.long() % 16, codes.long() // 16], -1).reshape(*codes.shape[:-1], -1)
    e, m = (n // 2) % 4, (n % 2).double()
    mag = torch.where(e > 0, torch.exp2((e - 1).double()) * (1 + m / 2), m / 2)
    b = groups.long()
    ge, gm = (b // 8) % 16, (b % 8).double()
    s = torch.where(ge > 0, torch.exp2((ge - 7).double()) * (1 + gm / 8), torch.exp2(torch.tensor(-9.0)).item() * gm)
    s = torch.repeat_interleave(s, GROUP, -1)
    return torch.where(n >= 8, -mag, mag) * s * g.double()[:, None, None]


def _line(s, name, b, n):
    """Slots 0 .. n - 1 of row b as (Hkv, n, D) in 64 bits."""
    c = s["case"]
    parts = [s[name]] + ([s[name + "g"]] if name + "g" in s else [])
    if c["layout"] == "paged":
        pages = s["table"][b, :-(-n // c["block"])].long()
        parts = [p[pages].permute(1, 0, 2, 3).reshape(c["Hkv"], -1, p.shape[-1])[:, :n] for p in parts]
    else:
        r = int(s["slot_ids"][b]) if s["slot_ids"] is not None else b
        parts = [p[r, :, :n] for p in parts]
    return parts[0].double() if len(parts) == 1 else _e2m1_row(parts[0], parts[1], s[name + "_scale"])


def _attention(q, k, v):
    """q (Hkv, G, D) over k, v (Hkv, n, D)."""
    x = torch.einsum("hgd,hnd->hgn", q, k) / math.sqrt(q.shape[-1])
    w = torch.softmax(x, -1)
    return torch.einsum("hgn,hnd->hgd", w, v)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    B, Hkv, D = c["B"], c["Hkv"], c["D"]
    if c["op"] == "write":
        step = max(1, CHUNK // (Hkv * D))
        kv = [torch.cat([_stored(s[n + "_new"][i:i + step], s[n + "_scale"], c["kind"]) for i in range(0, s["T"], step)])
              for n in ("k", "v")]
        got = {"k": kv[0], "v": kv[1]}
        return {**got, "bounds": None} if c["bounds"] else got
    lens = [int(n) for n in s["lengths"]]
    q = s["q"].double().view(B, Hkv, -1, D)
    if c["op"] == "sparse":
        ids, bs, out = _plain_select(s).long(), c["block"], []
        for b in range(B):
            k, v = (_line(s, n, b, lens[b]) for n in ("k", "v"))
            rows = []
            for h in range(Hkv):
                j = ids[b, h][ids[b, h] >= 0]
                at = (j[:, None] * bs + torch.arange(bs, device="cuda")).reshape(-1)
                at = at[at < lens[b]]
                rows.append(_attention(q[b, h][None], k[h, at][None], v[h, at][None]))
            out.append(torch.cat(rows).reshape(c["Hq"], D))
        return {"ids": None, "out": torch.stack(out)}
    new = [None, None]
    if c["step"] == "decode":
        new = [_stored(s[n + "_new"], s[n + "_scale"], "e2m1") for n in ("k", "v")]
    out = []
    for b in range(B):
        k, v = (_line(s, n, b, lens[b]) for n in ("k", "v"))
        if c["step"] == "decode":
            k, v = (torch.cat([x, y[b][:, None]], 1) for x, y in zip((k, v), new))
        out.append(_attention(q[b], k, v).reshape(c["Hq"], D))
    got = {"out": torch.stack(out)}
    return {**got, "k": new[0], "v": new[1]} if c["step"] == "decode" else got
