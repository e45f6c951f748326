"""References for block allocation, rotary put and linear attention, written from their definitions (Python
loops; torch in float64), with bounds on what 32-bit sums and 16-bit operands may be off."""
from __future__ import annotations

import math

import torch

BS = 16
H16 = 2.0 ** -11  # half a step of fp16, relative
TINY16 = 2.0 ** -25  # half a step of its subnormals
U32 = 2.0 ** -24


def blocks(n):
    return -(-n // BS)


def alloc(tables, free, count, held, ctx, new, num_tokens, num_blocks=None):
    """What pa_kv_alloc leaves for valid lengths: dict of lists, and whether blocks ran out."""
    tables, free = [list(r) for r in tables], list(free)
    num_blocks = len(free) if num_blocks is None else num_blocks
    n0 = [blocks(h) for h in held]
    n1 = [blocks(c + q) for c, q in zip(ctx, new)]
    short = False
    for b in range(len(held)):
        for i in range(n1[b], n0[b]):
            free[count] = tables[b][i]
            count += 1
    lens, served, out_of = [], [], False
    wanted = 0
    top = count
    for b in range(len(held)):
        need = max(0, n1[b] - n0[b])
        wanted += need
        ok = need == 0 or wanted <= top
        short |= not ok
        if ok:
            for i in range(n0[b], n1[b]):
                count -= 1
                tables[b][i] = free[count]
        served.append(ok)
        lens.append(ctx[b] + new[b] if ok else ctx[b])
    loc, slots, positions = [0], [], []
    for b in range(len(held)):
        for i in range(new[b]):
            p = ctx[b] + i
            positions.append(p)
            slots.append(tables[b][p // BS] * BS + p % BS if served[b] else -1)
        loc.append(loc[-1] + new[b])
    pad = num_tokens - len(slots)
    return dict(tables=tables, free=free, count=count, loc=loc, lens=lens, slots=slots + [-1] * pad,
                positions=positions + [-1] * pad), short


def rotate(x, pos, table, pairs):
    """float64 rotation of x [tokens, heads, dim], and a bound on a 32-bit one that is rounded to fp16."""
    rot = table.shape[1]
    y = x.double().clone()
    mag = x.double().abs()
    c, s = table[pos, :rot // 2].double()[:, None], table[pos, rot // 2:].double()[:, None]
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if pairs else (i, i + rot // 2)
        xa, xb = x[..., a].double(), x[..., b].double()
        y[..., a] = xa * c[..., i] - xb * s[..., i]
        y[..., b] = xb * c[..., i] + xa * s[..., i]
        mag[..., a] = (xa * c[..., i]).abs() + (xb * s[..., i]).abs()
        mag[..., b] = (xb * c[..., i]).abs() + (xa * s[..., i]).abs()
    # a product and a fused sum in 32 bits, then fp16 (a sum just below a power of two may round by its own step)
    return y, H16 * y.abs() * (1 + 2.0 ** -10) + 3 * U32 * mag + TINY16


def linear(q, k, v, s0, g, scale, chunked=True):
    """One sequence of linear attention in float64: q [T, H, D], k / v [T, Hkv, D], s0 [Hkv, D, D], g [Hkv].

    Returns out, states and bounds on both.  What they count (terms: the products that a value sums):
      out     its rounding to fp16; with `chunked`, one rounding to fp16 of each score and of each entry of a
              state, half a step each (whose subnormals are 2^-14 of the largest normal's step: 2^-29 of the row's
              or the state's largest); 32-bit sums of at most 2 * D + T terms; decays as below;
      states  exp(g n) in 32 bits, off by (|g n| + 4) units (its argument's rounding and its own), two 16-bit halves
              of v (2^-22), a unit a step of 16 tokens in the tensor cores' sums of a block of 256 tokens (which may
              truncate: two units), and one a token or block for the chain.
    """
    T, H, D = q.shape
    hkv = k.shape[1]
    G = H // hkv
    dev = q.device
    q, k, v, s0 = q.double(), k.double(), v.double(), s0.double()
    t = torch.arange(T, device=dev, dtype=torch.float64)
    out, out_b = torch.zeros(T, H, D, dtype=torch.float64, device=dev), torch.zeros(T, H, D, dtype=torch.float64, device=dev)
    st, st_b = s0.clone(), torch.zeros_like(s0)
    for h in range(hkv):
        gh = float(g[h])
        pw = lambda n: torch.where(n == 0, 1.0, torch.exp(torch.where(n == 0, 0.0, n * gh)))
        x = lambda n: torch.where(torch.isfinite(n * gh), (n * gh).abs(), 0.0)  # |g n|; a decay of 0 is exact
        apart = t[:, None] - t
        seen = apart >= 0
        apart = apart.clamp(min=0)
        for j in range(h * G, (h + 1) * G):
            p = torch.where(seen, (q[:, j] @ k[:, h].T) * pw(apart), 0.0)
            pa = torch.where(seen, (q[:, j].abs() @ k[:, h].abs().T) * pw(apart) * (x(apart) + 8 + D), 0.0)
            inter, far = (q[:, j] @ s0[h]) * pw(t + 1)[:, None], (q[:, j].abs() @ s0[h].abs()) * pw(t + 1)[:, None]
            o = (p @ v[:, h] + inter) * scale
            units = 2 * U32 * (pa @ v[:, h].abs() + (far * (x(t + 1)[:, None] + 2 * D + T + 16)) + T * (p.abs() @ v[:, h].abs()))
            lost = 0.0
            if chunked:
                # scores of a token's own block are rounded, those of earlier blocks are in the state
                state_abs = far + (torch.where(seen, (q[:, j].abs() @ k[:, h].abs().T) * pw(apart), 0.0) @ v[:, h].abs())
                lost = H16 * (1 + 2.0 ** -10) * (p.abs() @ v[:, h].abs() + state_abs)
                lost = lost + 2.0 ** -28 * state_abs.amax(dim=1, keepdim=True) * math.sqrt(D)
            out[:, j] = o
            out_b[:, j] = H16 * (1 + 2.0 ** -10) * o.abs() + abs(scale) * (units + lost) + TINY16
        n, last = T - 1 - t, torch.tensor(float(T), dtype=torch.float64, device=dev)
        whole = pw(last)
        st[h] = s0[h] * whole + (k[:, h] * pw(n)[:, None]).T @ v[:, h]
        per = 40 + 2 * T  # (a token-by-token chain; a block's is shorter)
        st_b[h] = U32 * 2 * (s0[h].abs() * whole * (float(x(last)) + per)
                             + (k[:, h].abs() * (pw(n) * (x(n) + per))[:, None]).T @ v[:, h].abs()) + 2.0 ** -140
    return out, st, out_b, st_b


def check(got, want, bound, what=""):
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    if got.dtype == torch.float16:
        # from 65520 on (the largest, 65504, and half of the step of 32 above it) a value rounds to infinity
        bad &= ~(torch.isinf(got) & (got.double().sign() == want.sign()) & (want.abs() + bound >= 65520.0))
    if bool(bad.any()):
        i = int(torch.argmax(torch.where(bad, off / bound.clamp(min=1e-300), torch.zeros_like(off)).flatten()))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; at {i}: {float(got.flatten()[i])} for "
                             f"{float(want.flatten()[i])}, bound {float(bound.flatten()[i]):.3g}")


class LinearCase:
    """Packed sequences of linear attention with states in a shuffled pool; what no call may touch holds NaN."""

    def __init__(self, new, heads, hkv, dim, ctx=None, g=None, seed=0, device="cuda", pad=3, spare=2, size=1.0, scale=None):
        gen = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=gen, device=device)
        B, T = len(new), sum(new)
        self.new, self.heads, self.hkv, self.dim, self.device = list(new), heads, hkv, dim, device
        self.ctx = [100] * B if ctx is None else list(ctx)
        self.scale = 1.0 / math.sqrt(dim) if scale is None else scale
        self.q, self.k, self.v = (torch.full((T + pad, n, dim), math.nan, dtype=torch.float16, device=device)
                                  for n in (heads, hkv, hkv))
        for x in (self.q, self.k, self.v):
            x[:T] = (rand(T, *x.shape[1:]) * size).half()
        self.out = torch.full_like(self.q, 7.0)
        self.g = torch.tensor([-(2.0 ** (-8.0 * (h + 1) / hkv)) for h in range(hkv)] if g is None else g,
                              dtype=torch.float32, device=device)
        self.states = torch.full((B + spare, hkv, dim, dim), math.nan, device=device)
        order = torch.randperm(B + spare, generator=torch.Generator().manual_seed(seed))[:B].to(torch.int32)
        self.slots = order.to(device)
        for b in range(B):
            if self.ctx[b] > 0:
                self.states[int(order[b])] = rand(hkv, dim, dim) * size * size
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device=device)
        self.loc = ints([sum(new[:b]) for b in range(B + 1)])
        self.ctx_lens = ints(self.ctx)
        self.before = self.states.clone()

    def check(self, out, states, chunked=True):
        """Every sequence against its reference; everything else as it was."""
        at, loc = 0, self.loc.tolist()
        untouched = torch.ones(states.shape[0], dtype=torch.bool)
        for b, n in enumerate(self.new):
            slot = int(self.slots[b])
            if n == 0 or slot < 0:
                continue
            untouched[slot] = False
            rows = slice(loc[b], loc[b + 1])
            s0 = self.before[slot] if self.ctx[b] > 0 else torch.zeros_like(self.before[slot])
            o, s, ob, sb = linear(self.q[rows], self.k[rows], self.v[rows], s0, self.g, self.scale, chunked)
            check(out[rows], o, ob, f"sequence {b} out")
            check(states[slot], s, sb, f"sequence {b} state")
        same = lambda x, y: torch.equal(x.nan_to_num(nan=-77.0), y.nan_to_num(nan=-77.0))
        assert same(states[untouched.to(states.device)], self.before[untouched.to(states.device)]), "a state that no sequence has was written"
        assert bool((out[loc[-1]:] == 7.0).all()), "rows behind the last sequence were written"
