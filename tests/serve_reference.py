"""Plain definitions, on the CPU, of rotary positions, the 8-bit cache with
block scales, capped / biased / counted attention and eviction."""
import math

import torch


def layout_of(name, B, Hkv, Smax, bs, gen, held):
    """(shape without D, table, slot ids) of a cache; held: slots a row needs."""
    if name == "paged":
        nb = -(-Smax // bs)
        pool = B * nb + 3
        perm = torch.randperm(pool, generator=gen)[:B * nb].view(B, nb).int()
        need = torch.tensor([-(-n // bs) for n in held])
        return (pool, Hkv, bs), torch.where(torch.arange(nb) < need[:, None], perm, -1), None
    if name == "slots":
        return (B + 3, Hkv, Smax), None, torch.randperm(B + 3, generator=gen)[:B].int()
    return (B, Hkv, Smax), None, None


def row_slots(x, b, n, table, slots, bs):
    """Slots 0 .. n - 1 of batch row b of a cache-shaped tensor x: (Hkv, n, ...)."""
    if table is None:
        return x[int(slots[b]) if slots is not None else b][:, :n]
    pages = x[table[b, :-(-n // bs)].long()]
    return pages.transpose(0, 1).flatten(1, 2)[:, :n]


def put_row(x, b, n, new, table, slots, bs):
    """Writes new (Hkv, n, ...) into slots 0 .. n - 1 of row b."""
    if table is None:
        x[int(slots[b]) if slots is not None else b, :, :n] = new
        return
    for j in range(-(-n // bs)):
        m = min(bs, n - j * bs)
        x[int(table[b, j]), :, :m] = new[:, j * bs:j * bs + m]


class Cache8:
    """An 8-bit cache on the CPU: codes and block scales by the definition."""

    def __init__(self, shape, D, bs, table, slots):
        self.codes = torch.zeros(*shape, D, dtype=torch.int8)
        self.scale = torch.zeros(shape[:2] if table is not None else (*shape[:2], shape[2] // bs))
        self.bs, self.table, self.slots = bs, table, slots

    def block(self, b, j):
        """(codes (Hkv, bs, D), scales (Hkv,)) of block j of row b, views."""
        if self.table is not None:
            p = int(self.table[b, j])
            return self.codes[p], self.scale[p]
        r = int(self.slots[b]) if self.slots is not None else b
        return self.codes[r, :, j * self.bs:(j + 1) * self.bs], self.scale[r, :, j]

    def append(self, b, start, x):
        """x (n, Hkv, D) float32 into slots start .. of row b."""
        n, at = x.shape[0], 0
        while at < n:
            slot = start + at
            j, first = slot // self.bs, slot % self.bs
            m = min(self.bs - first, n - at)
            codes, scale = self.block(b, j)
            for h in range(x.shape[1]):
                y = x[at:at + m, h].float()
                top = y.abs().max()
                need = top / torch.tensor(127.0)
                old = scale[h].clone()
                if not torch.isfinite(top):
                    t = torch.tensor(math.nan)
                elif first == 0 or old <= 0:
                    t = need
                else:
                    t, k = old, 0
                    while t < need:
                        t, k = t * 2, k + 1
                    if k:
                        codes[h, :first] = torch.round(codes[h, :first].double() * 2.0 ** -k).to(torch.int8)
                scale[h] = t
                q = torch.where(t > 0, y / t, 0.0) if t > 0 else torch.zeros_like(y)
                codes[h, first:first + m] = torch.round(q).clamp(-127, 127).to(torch.int8)
            at += m

    def row(self, b, n):
        """Values of slots 0 .. n - 1, (Hkv, n, D), 64 bits."""
        c = row_slots(self.codes, b, n, self.table, self.slots, self.bs).double()
        nb = -(-n // self.bs)
        t = torch.stack([self.block(b, j)[1] for j in range(nb)], 1).double()
        return c * torch.repeat_interleave(t, self.bs, 1)[:, :n, None]


def attended(n, window=0, prefix=0):
    j = torch.arange(n)
    return (j > n - 1 - window) | (j < prefix) if window else torch.ones(n, dtype=torch.bool)


def attention(q, k, v, cap=0.0, slopes=None, ok=None, sink=None):
    """q (Hkv, G, D), k and v (Hkv, n, D), 64 bits. Returns out (Hkv, G, D),
    weights (Hkv, G, n), and the scores' magnitudes that rounding acts on."""
    n = k.shape[1]
    at = torch.ones(n, dtype=torch.bool) if ok is None else ok
    s = torch.einsum("hgd,hnd->hgn", q, k[:, at]) / math.sqrt(q.shape[-1])
    if cap:
        s = cap * torch.tanh(s / cap)
    y = s
    bias = torch.zeros_like(s)
    if slopes is not None:
        bias = slopes.double()[..., None] * (torch.arange(n)[at] - (n - 1)).double()
        y = s + bias
    z = y if sink is None else torch.cat([y, sink.double()[..., None]], -1)
    w = torch.softmax(z, -1)[..., :y.shape[-1]]
    out = torch.einsum("hgn,hnd->hgd", w, v[:, at])
    full = torch.zeros(*w.shape[:2], n, dtype=torch.float64)
    full[..., at] = w
    # largest magnitude a product's sum meets, and what the cap and bias round
    big = torch.einsum("hgd,hnd->hgn", q.abs(), k[:, at].abs()).amax(-1, keepdim=True) / math.sqrt(q.shape[-1])
    d = score_error(q.shape[-1], big, s.abs() + bias.abs())
    err = torch.zeros_like(full)
    err[..., at] = d
    return out, full, err


def score_error(D, amax, formed):
    """Bound of a score's error. The product: D / 16 matrix steps truncated to
    2^-23 of the sum of magnitudes, and four roundings more (the key scale, the
    factor, a float32 query's 2^-22). What is formed from it: tanhf (one step),
    the cap's product, the bias' product and sum: five roundings of 2^-24 of the
    magnitudes at hand, doubled for the change to base 2."""
    return (D / 16 + 6) * 2.0 ** -23 * amax + 10 * 2.0 ** -24 * formed


def out_tolerance(w, err, vmax):
    """First order: sum w_j e_j |v_j - out| <= 2 vmax sum w_j e_j; the
    exponential (2^-22), the weights' parts (2^-22), running sums of a few
    thousand slots and the merge stay under 2^-17 together."""
    return 2 * vmax * (w * err).sum(-1).max() + 2.0 ** -17 * vmax


def count_tolerance(w, err):
    """A weight's relative error is its score's, the denominator's mean, and
    2^-19 of the exponentials and sums."""
    mean = (w * err).sum(-1, keepdim=True)
    return (w * (err + mean + 2.0 ** -19)).sum(1) + 1e-30


def frequencies(dim, base, scaling):
    out = []
    k = scaling or {}
    for i in range(dim // 2):
        b = base * k["factor"] ** (dim / (dim - 2)) if k.get("kind") == "ntk" else base
        f = b ** (-2.0 * i / dim)
        if k.get("kind") == "linear":
            f /= k["factor"]
        if k.get("kind") == "bands":
            r = k["original"] * f / (2 * math.pi)
            u = min(1.0, max(0.0, (r - k["low"]) / (k["high"] - k["low"])))
            f = f * u + f * (1 - u) / k["factor"]
        out.append(f)
    return torch.tensor(out, dtype=torch.float64), k.get("attention", 1.0)


def rotate(x, positions, dim, base, layout, scaling):
    """x (T, H, D) turned, 64 bits."""
    f, m = frequencies(dim, base, scaling)
    a = positions.double()[:, None] * f
    c, s = (torch.cos(a) * m)[:, None], (torch.sin(a) * m)[:, None]
    y = x.double().clone()
    i, j = (slice(0, dim // 2), slice(dim // 2, dim)) if layout == "half" else (slice(0, dim, 2), slice(1, dim, 2))
    u, v = y[..., i].clone(), y[..., j].clone()
    y[..., i], y[..., j] = u * c - v * s, u * s + v * c
    return y


def kept(w, n, n_keep, n_first, n_last):
    """Ascending kept slots of counts w (>= n,)."""
    if n <= n_keep:
        return list(range(n))
    mid = list(range(n_first, n - n_last))
    mid.sort(key=lambda j: (0, 0.0, j) if math.isnan(w[j]) else (1, -float(w[j]), j))
    return sorted(list(range(n_first)) + list(range(n - n_last, n)) + mid[:n_keep - n_first - n_last])
