"""References in 64 bits for the 8-bit cache and eviction calls, written from
their definitions (torch in float64, Python loops), and seeded inputs."""
from __future__ import annotations

import math

import torch

BS = 16
DTYPES = {"f16": torch.float16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def scale_of(amax: float, fmt: str) -> float:
    """The block scale of a largest magnitude."""
    if amax == 0:
        return 0.0
    if fmt == "e4m3":  # smallest power of two with 448 s >= amax
        k = -60
        while 448.0 * 2.0 ** k < amax:
            k += 1
        return 2.0 ** k
    # smallest number of 8 significant bits with 127 s >= amax
    e = math.frexp(amax / 127.0)[1] - 8
    n = math.floor(math.ldexp(amax / 127.0, -e)) - 1
    while 127.0 * math.ldexp(n, e) < amax:
        n += 1
    return math.ldexp(n, e)


# every finite e4m3 value from its definition: sign, 4 exponent bits (bias 7), 3 mantissa bits
E4M3_VALUES = [(m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
               for e in range(16) for m in range(8) if not (e == 15 and m == 7)]


def round_code(t: torch.Tensor, fmt: str) -> torch.Tensor:
    """float64 values to the format's nearest (ties to even), saturated; NaN to NaN (e4m3) or 0 (int8)."""
    if fmt == "int8":
        return torch.nan_to_num(torch.round(t), nan=0.0, posinf=127.0, neginf=-127.0).clamp(-127, 127)
    table = torch.tensor(E4M3_VALUES, dtype=torch.float64, device=t.device)
    a = t.abs().clamp(max=448.0)
    hi = torch.searchsorted(table, a.nan_to_num(0.0).contiguous()).clamp(max=len(E4M3_VALUES) - 1)
    lo = (hi - 1).clamp(min=0)
    dh, dl = table[hi] - a, a - table[lo]
    pick_lo = (dl < dh) | ((dl == dh) & (lo % 2 == 0))  # even code = even mantissa
    r = torch.where(pick_lo, table[lo], table[hi])
    return torch.where(t.isnan(), t, torch.copysign(r, t))


def quantise_blocks(x: torch.Tensor, fmt: str):
    """A cache in `fmt` of the values x (fp16 [blocks, heads, 16, dim]), with scales (None for f16)."""
    if fmt == "f16":
        return x.clone(), None
    amax = x.double().abs().amax(dim=(2, 3)).cpu()
    s = torch.tensor([[scale_of(float(v), fmt) for v in row] for row in amax], dtype=torch.float64).to(x.device)
    codes = round_code(x.double() / torch.where(s > 0, s, 1.0)[:, :, None, None], fmt)
    return to_codes(codes, fmt), s.float()


def to_codes(values64: torch.Tensor, fmt: str) -> torch.Tensor:
    return values64.float().to(DTYPES[fmt])


def values(cache: torch.Tensor, scales) -> torch.Tensor:
    """What a cache stands for, in 64 bits."""
    v = cache.float().double() if cache.dtype == torch.float8_e4m3fn else cache.double()
    return v if scales is None else v * scales.double()[:, :, None, None]


class Case:
    """A paged cache with sequences of the given lengths, blocks handed out from a seeded permutation;
    slots past a sequence's end hold NaN (f16, e4m3) or -128 (int8)."""

    def __init__(self, lens, heads, hkv, dim, fmt, seed=0, device="cpu", spare=2, extra_cols=0, spread=2.0, room=None):
        g = torch.Generator(device=device).manual_seed(seed)
        gc = torch.Generator().manual_seed(seed)
        self.lens, self.heads, self.hkv, self.dim, self.fmt, self.device = list(lens), heads, hkv, dim, fmt, device
        cover = room or self.lens
        need = [-(-n // BS) for n in cover]
        blocks = sum(need) + spare
        perm = torch.randperm(blocks, generator=gc).to(torch.int32)
        self.free = perm[sum(need):].tolist()
        cols = max(1, max(need, default=1)) + extra_cols
        tables = torch.full((len(self.lens), cols), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            tables[b, :n] = perm[at:at + n]
            at += n
        self.tables = tables.to(device)
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32, device=device)
        mag = torch.exp(spread * (torch.rand(2, blocks, hkv, 1, 1, generator=g, device=device) - 0.5))
        half = lambda *s: torch.randn(*s, generator=g, device=device)
        k = (half(blocks, hkv, BS, dim) * mag[0]).half()
        v = (half(blocks, hkv, BS, dim) * mag[1]).half()
        self.k, self.ks = quantise_blocks(k, fmt)
        self.v, self.vs = quantise_blocks(v, fmt)
        junk = torch.tensor(-128, dtype=torch.int8) if fmt == "int8" else torch.tensor(math.nan)
        for b, n in enumerate(self.lens):
            if n % BS:
                blk = int(tables[b, n // BS])
                for c in (self.k, self.v):
                    c[blk, :, n % BS:] = junk.to(c.dtype).to(device)
        for blk in self.free:  # blocks of nobody
            for c in (self.k, self.v):
                c[blk] = junk.to(c.dtype).to(device)
            if self.ks is not None:
                self.ks[blk] = math.nan
                self.vs[blk] = math.nan
        self.q = half(len(self.lens), heads, dim).half()
        self.scale = 1.0 / math.sqrt(dim)
        self.max_len = max(self.lens, default=0)

    def cache(self):
        return self.k, self.v, self.ks, self.vs

    def tokens(self, b, n=None):
        """K and V of sequence b's first n tokens, [hkv, n, dim] in 64 bits."""
        n = self.lens[b] if n is None else n
        ids = self.tables[b, :-(-n // BS)].long()
        out = []
        for c, s in ((self.k, self.ks), (self.v, self.vs)):
            raw = c.view(torch.uint8)[ids].view(c.dtype) if c.element_size() == 1 else c[ids]
            x = values(raw, None if s is None else s[ids])
            out.append(x.permute(1, 0, 2, 3).reshape(x.shape[1], -1, x.shape[3])[:, :n])
        return out


def attend(q, k, v, scale, mask=None):
    """One kv head group: q [g, n, d], k and v [t, d] in 64 bits.  Returns the output, the probabilities,
    sum p |v|, and the largest scale * sum |q k|."""
    s = q @ k.T * scale
    if mask is not None:
        s = s.masked_fill(~mask, -math.inf)
    p = torch.softmax(s, dim=-1)
    size = (q.abs() @ k.abs().T * abs(scale)).amax() if k.shape[0] else torch.zeros(())
    return p @ v, p, p @ v.abs(), float(size)


def score_error(dim, size):
    """Bound of a score's error, in natural units: a dot product of `dim` exact products added in 32 bits in any
    order, dim roundings of at most 2^-23 of the largest partial sum each (tensor cores truncate), and 8 further
    roundings of the score itself (block scale, softmax scale, base change, differences)."""
    return (dim + 8) * 2.0 ** -23 * size


def decode_reference(c: Case):
    """out, its bound, weights, their bound (all [B, ...], 64 bits).

    out: p enters the product rounded to fp16 (2^-11), a score error e changes p by a factor within exp(+-2 e) (its own and
    the sum's), exp2 and 32-bit sums add at most 2^-18; the output is rounded to fp16 (2^-11, subnormals 2^-25)."""
    B, g = len(c.lens), c.heads // c.hkv
    out = torch.zeros(B, c.heads, c.dim, dtype=torch.float64, device=c.device)
    bound = torch.zeros_like(out)
    w = torch.zeros(B, c.hkv, max(1, c.max_len), dtype=torch.float64, device=c.device)
    wb = torch.zeros_like(w)
    for b, n in enumerate(c.lens):
        if n == 0:
            continue
        k, v = c.tokens(b)
        for h in range(c.hkv):
            q = c.q[b, h * g:(h + 1) * g].double()
            o, p, a, size = attend(q, k[h], v[h], c.scale)
            e = math.expm1(2 * score_error(c.dim, size)) + 2.0 ** -18
            out[b, h * g:(h + 1) * g] = o
            bound[b, h * g:(h + 1) * g] = 2.0 ** -11 * o.abs() + (2.0 ** -11 * 1.01 + e) * a + 2.0 ** -25
            w[b, h, :n] = p.sum(dim=0)
            wb[b, h, :n] = p.sum(dim=0) * (e + g * 2.0 ** -24)
    return out, bound, w, wb


def prefix_reference(c: Case, new_lens, q, k_new, v_new, rounded=False):
    """out and its bound for chunks behind c's contexts.  Beyond decode_reference: probabilities under 2^-24 of the
    row's largest may be lost or rounded by 2^-25, and the sum may run over the rounded ones (2^-11 more).  `rounded`:
    context values are rounded to fp16 (2^-11 of K in the scores and of V in the sum)."""
    g = c.heads // c.hkv
    out = torch.zeros(q.shape, dtype=torch.float64, device=c.device)
    bound = torch.zeros_like(out)
    at = 0
    for b, n in enumerate(c.lens):
        m = new_lens[b]
        if m == 0:
            continue
        kc, vc = c.tokens(b)
        mask = torch.cat([torch.ones(m, n, dtype=torch.bool), torch.ones(m, m, dtype=torch.bool).tril()], 1).to(c.device)
        for h in range(c.hkv):
            k = torch.cat([kc[h], k_new[at:at + m, h].double()])
            v = torch.cat([vc[h], v_new[at:at + m, h].double()])
            for j in range(h * g, (h + 1) * g):
                o, p, a, size = attend(q[at:at + m, j].double(), k, v, c.scale, mask)
                r = 2.0 ** -11 if rounded else 0.0
                e = math.expm1(2 * (score_error(c.dim, size) + r * size)) + 2.0 ** -18
                out[at:at + m, j] = o
                bound[at:at + m, j] = (2.0 ** -11 * o.abs() + (2 * 2.0 ** -11 * 1.01 + r + e) * a
                                       + (n + m) * 2.0 ** -24 * v.abs().max() + 2.0 ** -25)
        at += m
    return out, bound


def append_reference(c: Case, new_lens, k_new, v_new):
    """The caches and scales after the append, as (k, v, ks, vs) with codes as float64 values."""
    res = []
    for cache, scales, new in ((c.k, c.ks, k_new), (c.v, c.vs, v_new)):
        codes = (cache.float() if cache.dtype != torch.float16 else cache).double()
        sc = None if scales is None else scales.double()
        at = 0
        for b, ctx in enumerate(c.lens):
            pos = ctx
            while pos < ctx + new_lens[b]:
                lo = pos % BS
                n = min(BS - lo, ctx + new_lens[b] - pos)
                blk = int(c.tables[b, pos // BS])
                x = new[at:at + n].double().transpose(0, 1)  # [hkv, n, dim]
                if c.fmt == "f16":
                    codes[blk, :, lo:lo + n] = x
                else:
                    for h in range(c.hkv):
                        # (a tensor divisor: by a number, torch multiplies by its rounded reciprocal on the GPU)
                        fin = x[h][x[h].isfinite()].abs()
                        s0 = float(sc[blk, h]) if lo else 0.0
                        s1 = max(s0, scale_of(float(fin.max()) if fin.numel() else 0.0, c.fmt))
                        if lo and s1 > s0:
                            codes[blk, h, :lo] = round_code(codes[blk, h, :lo] * s0 / x.new_tensor(s1), c.fmt)
                        codes[blk, h, lo:lo + n] = round_code(x[h] / x.new_tensor(s1) if s1 else x[h], c.fmt)
                        sc[blk, h] = s1
                at += n
                pos += n
        res += [codes, sc]
    return res[0], res[2], res[1], res[3]


def evict_reference(c: Case, weights, keep, sinks, recent):
    """Per sequence and kv head the kept positions, by Python's sort."""
    kept = []
    for b, n in enumerate(c.lens):
        k = min(keep[b], n)
        r = min(recent, k)
        s = min(sinks, k - r)
        rows = []
        for h in range(c.hkv):
            w = weights[b, h, :n].cpu().tolist()
            rank = lambda t: (-(w[t] if w[t] == w[t] else -math.inf), t)
            mid = sorted(range(s, n - r), key=rank)[:k - r - s]
            rows.append(sorted(list(range(s)) + mid + list(range(n - r, n))))
        kept.append(rows)
    return kept
