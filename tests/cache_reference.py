"""Plain 64-bit definitions of the cache formats, the key bounds, the block
selection and the attention over chosen slots, and random problems for them.
Everything here runs on the CPU."""
import math

import torch

E2M1_VALUES = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
E2M1_MIDS = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)
GROUP = 16


def e4m3_values():
    """The values of the 256 E4M3 bytes (NaN at 0x7f and 0xff)."""
    b = torch.arange(256)
    e, m = (b >> 3) & 15, (b & 7).double()
    v = torch.where(e > 0, torch.exp2((e - 7).double()) * (1 + m / 8), torch.full_like(m, 2.0 ** -9) * m)
    v[(b & 127) == 127] = math.nan
    return torch.where(b >= 128, -v, v)


def _nearest(a, values):
    """Index of the value nearest to a >= 0 (ascending values; ties to the even index)."""
    mids = (values[1:] + values[:-1]) / 2
    at = torch.searchsorted(mids, a)                    # a == mid: the lower one
    tie = (at < len(mids)) & (mids[at.clamp(max=len(mids) - 1)] == a)
    return torch.where(tie & (at % 2 == 1), at + 1, at)


def quantise_e2m1(x, g):
    """Codes (..., D / 2), scale bytes (..., D / 16) and t (..., D / 16) of x
    (..., D), g broadcastable to (..., 1): 64-bit quotients of the float32 inputs."""
    v = x.double().unflatten(-1, (-1, GROUP))
    amax = v.abs().amax(-1)
    g6 = (6.0 * g.float()).double()                     # float32(6 g), as the format says float32 arithmetic
    pos = e4m3_values()[:127]
    s = _nearest((amax / g6).clamp(max=448.0), pos)
    t = (pos[s].float() * g.float()).double()           # float32(s g)
    y = torch.where((t > 0)[..., None], v / torch.where(t > 0, t, 1.0)[..., None], 0.0)
    code = _nearest(y.abs().clamp(max=6.0), E2M1_VALUES)
    code = (code + 8 * torch.signbit(y).long()).flatten(-2)
    s = torch.where(torch.isnan(amax), 127, s)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8), s.to(torch.uint8), t, y.flatten(-2)


def values_e2m1(codes, scales, g):
    """float64 values of an E2M1 cache's vectors; g broadcastable to (..., 1)."""
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    v = E2M1_VALUES[n & 7] * torch.where(n >= 8, -1.0, 1.0)
    t = (e4m3_values()[scales.long()].float() * g.float()).double()
    return (v.unflatten(-1, (-1, GROUP)) * t[..., None]).flatten(-2)


def cache_values(kind, cache, groups, g):
    """float64 values of a cache (..., Hkv, S, row); g (Hkv,)."""
    gg = None if g is None else g.view(-1, 1, 1)
    if kind == "e2m1":
        return values_e2m1(cache, groups, gg)
    if kind == "e4m3":
        return e4m3_values()[cache.long()] * gg.double()
    return cache.double()


def attention(q, k, v, sink=None):
    """q (G, D) over k, v (n, D), 64 bits; sink (G,) logits or None."""
    x = q.double() @ k.T / math.sqrt(q.shape[-1])
    if sink is not None:
        x = torch.cat([x, sink.double()[:, None]], 1)
    w = torch.softmax(x, -1)
    return (w if sink is None else w[:, :-1]) @ v


def block_scores(q, lo, hi):
    """q (G, D); lo, hi (n, D): 64-bit bound scores of the blocks."""
    q = q.double()
    return hi.double() @ q.clamp(min=0).sum(0) + lo.double() @ q.clamp(max=0).sum(0)


def select(scores, n_select, n_first, n_last):
    """Ascending ids of the kept blocks of one (row, cache head)."""
    n = len(scores)
    if n <= n_select:
        return list(range(n))
    forced = [j for j in range(n) if j < n_first or j >= n - n_last]
    rest = [j for j in range(n) if j not in set(forced)]
    key = {j: (math.inf if math.isnan(scores[j]) else float(scores[j]), math.isnan(scores[j])) for j in rest}
    rest.sort(key=lambda j: (not key[j][1], -key[j][0], j))
    return sorted(forced + rest[:n_select - len(forced)])


class Problem:
    """A random cache problem on the CPU: tensors under the binding's names.
    ``lens`` are the valid slots of each row; paged rows get only the blocks
    that hold their first ``room`` slots (the others are -1)."""

    def __init__(self, kind, layout, lens, Hq, Hkv, D, Smax, bs=16, q_dtype=torch.bfloat16, seed=0, scale=1.0,
                 extra=0):
        gen = torch.Generator().manual_seed(seed)
        self.kind, self.layout, self.lens = kind, layout, list(lens)
        self.B, self.Hq, self.Hkv, self.D, self.Smax, self.bs = len(lens), Hq, Hkv, D, Smax, bs
        B = self.B
        self.g = [scale * (0.75 + 0.5 * torch.rand(Hkv, generator=gen)) * 4 / 448 / (6 if kind == "e2m1" else 1)
                  for _ in range(2)]
        self.q = torch.randn(B, Hq, D, generator=gen).to(q_dtype)
        self.lengths = torch.tensor(lens, dtype=torch.int32)
        self.table = self.slots = None
        if layout == "paged":
            nb = -(-Smax // bs)
            pool = B * nb + 3
            perm = torch.randperm(pool, generator=gen)[:B * nb].view(B, nb).int()
            held = torch.tensor([-(-(n + extra) // bs) for n in lens])
            self.table = torch.where(torch.arange(nb) < held[:, None], perm, -1)
            shape = (pool, Hkv, bs, D)
        else:
            R = B + (4 if layout == "slots" else 0)
            self.slots = torch.randperm(R, generator=gen)[:B].int() if layout == "slots" else None
            shape = (R, Hkv, Smax, D)
        self.kv, self.groups = [], []
        for i in range(2):
            x = torch.randn(shape, generator=gen) * scale
            if kind == "e2m1":
                c, s, _, _ = quantise_e2m1(x, self.g[i].view(-1, 1, 1))
                self.kv.append(c)
                self.groups.append(s)
            elif kind == "e4m3":
                y = (x / self.g[i].view(-1, 1, 1)).clamp(-448, 448).to(torch.float8_e4m3fn)
                self.kv.append(y.view(torch.uint8))
                self.groups.append(None)
            else:
                self.kv.append(x.to(torch.bfloat16 if kind == "bf16" else torch.float32))
                self.groups.append(None)

    def row(self, b, i, n=None):
        """Slots 0 .. n - 1 of row b of K (i = 0) or V (i = 1): (Hkv, n, D), 64 bits."""
        n = self.lens[b] if n is None else n
        parts = [self.kv[i]] + ([self.groups[i]] if self.groups[i] is not None else [])
        if self.table is not None:
            pages = self.table[b, :-(-n // self.bs)].long()
            parts = [p[pages].transpose(0, 1).flatten(1, 2)[:, :n] for p in parts]
        else:
            r = int(self.slots[b]) if self.slots is not None else b
            parts = [p[r, :, :n] for p in parts]
        return cache_values(self.kind, parts[0], parts[1] if len(parts) > 1 else None, self.g[i])

    def expect(self, b, slots=None, sink=None, new=None):
        """(Hq, D) attention of row b over `slots` (per head lists, or all), and
        the largest |V| and sum |q k| / sqrt(D) met."""
        G = self.Hq // self.Hkv
        k, v = self.row(b, 0), self.row(b, 1)
        if new is not None:
            k, v = (torch.cat([x, y[:, None]], 1) for x, y in zip((k, v), new))
        out, vmax, amax = [], 0.0, 0.0
        for h in range(self.Hkv):
            at = slice(None) if slots is None else torch.tensor(slots[h])
            q = self.q[b, h * G:(h + 1) * G]
            kk, vv = k[h][at], v[h][at]
            out.append(attention(q, kk, vv, None if sink is None else sink[h * G:(h + 1) * G]))
            vmax = max(vmax, float(vv.abs().max()))
            amax = max(amax, float((q.double().abs() @ kk.abs().T).max()) / math.sqrt(self.D))
        return torch.cat(out), vmax, amax


def attend_tolerance(D, vmax, amax):
    """Largest error of an output element (float32 sums over exact products).
    A score is a sum of D / 16 matrix steps, each truncated to 2^-23 of the sum
    of magnitudes amax, and of few roundings more (a float32 query enters as 22
    bits: another 2^-22); a relative error e of the weights moves the output by
    at most 2 e vmax (numerator and denominator); the exponential, the weights'
    own 22 bits, the running sums of a few thousand slots and the merge stay
    under 2^-17 together."""
    return vmax * (2 * (D / 16 + 4) * 2.0 ** -23 * amax + 2.0 ** -17)
