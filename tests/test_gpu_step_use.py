"""Block allocation, rotary put, the paged attention calls and linear attention run together, as a serving loop runs
them, and the step's calls on streams and in graphs."""
import math

import pytest
import torch

import step_helpers as S
from paged_kv_cache_308_gb300 import binding as pb

pytestmark = pytest.mark.gpu
BS = 16


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def status():
    torch.cuda.synchronize()
    return pb.pa_get_device_status()


def attention(q, k, v, first, scale):
    """Causal attention in float64 of new tokens q (from position `first` on) over all tokens' k and v."""
    G = q.shape[1] // k.shape[1]
    out = torch.empty(q.shape, dtype=torch.float64, device=q.device)
    seen = torch.arange(k.shape[0], device=q.device)[None] <= first + torch.arange(q.shape[0], device=q.device)[:, None]
    for h in range(q.shape[1]):
        s = (q[:, h].double() @ k[:, h // G].double().T * scale).masked_fill(~seen, -math.inf)
        out[:, h] = torch.softmax(s, dim=1) @ v[:, h // G].double()
    return out


class Model:
    """A paged attention layer with rotary positions and a linear attention layer, for `rows` sequences at a time."""

    def __init__(self, rows, blocks=40, heads=8, hkv=2, dim=64, cols=12):
        self.rows, self.heads, self.hkv, self.dim, self.cols = rows, heads, hkv, dim, cols
        self.gen = torch.Generator(device="cuda").manual_seed(5)
        self.cache = [torch.full((blocks, hkv, BS, dim), math.nan, dtype=torch.float16, device="cuda") for _ in range(2)]
        self.tables = torch.full((rows, cols), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(blocks, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
        self.count = ints([blocks])
        self.lens = ints([0] * rows)
        self.states = torch.full((rows + 2, hkv, dim, dim), math.nan, device="cuda")
        self.slots = ints([(3 * b + 1) % (rows + 2) for b in range(rows)])
        self.g = torch.tensor([-0.01, -0.3][:hkv], device="cuda")
        ang = torch.arange(256, device="cuda")[:, None] * 0.5 ** torch.arange(dim // 4, device="cuda")
        self.table = torch.cat([ang.cos(), ang.sin()], dim=1).float().contiguous()  # half of the dims turn
        self.history = [dict(k=[], v=[], lk=[], lv=[]) for _ in range(rows)]

    def step(self, ctx, new, pad=4):
        rows, heads, hkv, dim = self.rows, self.heads, self.hkv, self.dim
        T = sum(new)
        half = lambda *s: torch.randn(*s, generator=self.gen, device="cuda").half()
        q, k, v = half(T + pad, heads, dim), half(T + pad, hkv, dim), half(T + pad, hkv, dim)
        lq, lk, lv = half(T + pad, heads, dim), half(T + pad, hkv, dim), half(T + pad, hkv, dim)
        held, self.lens = self.lens, torch.empty_like(self.lens)
        context, query, loc = ints(ctx), ints(new), ints([-1] * (rows + 1))
        slots, positions = ints([-7] * (T + pad)), ints([-7] * (T + pad))
        pb.pa_kv_alloc(self.tables, self.free, self.count, context, query, loc, self.lens, slots, positions, held_lens=held)
        q2, k2 = torch.zeros_like(q), torch.zeros_like(k)
        pb.pa_kv_put(q2, k2, q, k, v, *self.cache, slots, positions, self.table)
        out, lout = torch.zeros_like(q), torch.zeros_like(q)
        scale = 1 / math.sqrt(dim)
        if max(new) == 1 and min(new) == 1:
            pb.pa_kv_decode(out[:T], q2[:T], *self.cache, None, None, self.tables, self.lens, scale, max_seq_len=self.cols * BS)
            pb.pa_linear_decode(lout[:T], lq[:T], lk[:T], lv[:T], self.states, self.slots, self.g, scale)
        else:
            pb.pa_kv_prefix(out, q2, k2, v, *self.cache, None, None, self.tables, context, loc, scale,
                            max_context_len=self.cols * BS, max_query_len=max(new))
            pb.pa_linear_prefix(lout, lq, lk, lv, self.states, self.slots, self.g, context, loc, scale, max_query_len=max(new))
        assert status() == 0
        # everything against the sequences' whole histories
        at = 0
        for b, n in enumerate(new):
            h = self.history[b]
            for key in h:
                del h[key][ctx[b]:]
            if not n:
                continue
            rows_ = slice(at, at + n)
            pos = torch.arange(ctx[b], ctx[b] + n, device="cuda")
            kr, kb = S.rotate(k[rows_], pos, self.table, False)
            S.check(k2[rows_], kr, kb, "rotated keys")
            for key, x in (("k", k2), ("v", v), ("lk", lk), ("lv", lv)):
                h[key] += list(x[rows_])
            keys, values = torch.stack(h["k"]), torch.stack(h["v"])
            want = attention(q2[rows_], keys, values, ctx[b], scale)
            # the attention kernels round p and v's products as the framework's other tests allow them
            assert bool(((out[rows_].double() - want).abs() <= 2e-3 + 1e-2 * want.abs()).all()), f"row {b}"
            full_q = torch.cat([torch.zeros(ctx[b], heads, dim, device="cuda").half(), lq[rows_]])
            o, s, ob, sb = S.linear(full_q, torch.stack(h["lk"]), torch.stack(h["lv"]),
                                    torch.zeros(hkv, dim, dim, device="cuda"), self.g, scale)
            S.check(lout[rows_], o[ctx[b]:], ob[ctx[b]:], f"row {b} linear")
            S.check(self.states[int(self.slots[b])], s, sb, f"row {b} state")
            at += n
        assert bool((out[T:] == 0).all()) and bool((lout[T:] == 0).all())
        # every block is free, or in one row
        lens = self.lens.tolist()
        used = [x for b in range(rows) for x in self.tables[b, :S.blocks(lens[b])].tolist()]
        free = self.free[:self.count.item()].tolist()
        assert sorted(used + free) == list(range(self.free.shape[0]))


def test_serving_loop():
    m = Model(3)
    m.step([0, 0, 0], [37, 0, 5])
    m.step([37, 0, 5], [20, 64, 1])
    for _ in range(17):
        m.step(m.lens.tolist(), [1, 1, 1])
    a, b, c = m.lens.tolist()
    m.step([a, 0, c], [30, 0, 1])       # the second one ended
    m.step([a + 30, 0, c + 1], [1, 50, 1])  # another takes its row and its state's slot
    m.step([0, 50, c + 2], [9, 2, 3])   # the first row starts again at once
    m.step(m.lens.tolist(), [1, 1, 1])


def test_tokens_taken_back():
    """Tokens written ahead are taken back: the next step goes on from fewer than the row holds."""
    held, ctx, new = [40, 17], [33, 15], [2, 20]
    tables = ints([[5, 6, 7, -1], [1, 2, -1, -1]])
    free, count = ints([9, 8, 4, 3, -1, -1, -1, -1, -1, -1]), ints([4])
    loc, lens, slots, pos = ints([0] * 3), ints([0] * 2), ints([0] * 22), ints([0] * 22)
    pb.pa_kv_alloc(tables, free, count, ints(ctx), ints(new), loc, lens, slots, pos, held_lens=ints(held))
    want, short = S.alloc([[5, 6, 7, -1], [1, 2, -1, -1]], [9, 8, 4, 3] + [-1] * 6, 4, held, ctx, new, 22)
    assert status() == 0 and not short
    assert tables.tolist() == want["tables"] and slots.tolist() == want["slots"] and count.item() == want["count"]


def test_eight_bit_cache_behind_put():
    """Rotation without a cache, then the append that knows block scales."""
    T, heads, hkv, dim = 40, 8, 2, 128
    g = torch.Generator(device="cuda").manual_seed(7)
    half = lambda *s: torch.randn(*s, generator=g, device="cuda").half()
    q, k, v = half(T, heads, dim), half(T, hkv, dim), half(T, hkv, dim)
    tables, free, count = ints([[-1] * 4]), ints([3, 1, 2, 0]), ints([4])
    loc, lens, slots, pos = ints([0, 0]), ints([0]), ints([0] * T), ints([0] * T)
    pb.pa_kv_alloc(tables, free, count, ints([0]), ints([T]), loc, lens, slots, pos)
    ang = torch.rand(T, dim // 2, generator=g, device="cuda") * 6
    pb.pa_kv_put(q, k, q, k, v, None, None, None, pos, torch.cat([ang.cos(), ang.sin()], dim=1))
    kc, vc = (torch.zeros(4, hkv, BS, dim, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(4, hkv, device="cuda") for _ in range(2))
    pb.pa_kv_append(kc, vc, ks, vs, k, v, tables, ints([0]), loc, max_query_len=T)
    out = torch.empty(1, heads, dim, dtype=torch.float16, device="cuda")
    pb.pa_kv_decode(out, q[-1:].contiguous(), kc, vc, ks, vs, tables, lens, 0.1, max_seq_len=64)
    assert status() == 0
    ids = tables[0, :3].long()
    value = lambda c, s: (c.float().double() * s.double()[:, :, None, None])[ids].transpose(0, 1).flatten(1, 2)[:, :T].transpose(0, 1)
    want = attention(q[-1:], value(kc, ks), value(vc, vs), T - 1, 0.1)
    assert bool(((out.double() - want).abs() <= 2e-3 + 1e-2 * want.abs()).all())
    # (e4m3 holds the rotated keys to half a step of 3 bits, 2^-4, and below its normals of half of 2^-9 scales)
    back = value(kc, ks)
    most = ks[ids].repeat_interleave(BS, dim=0)[:T, :, None].double()
    assert bool(((back - k.double()).abs() <= 2.0 ** -4 * k.double().abs() + 2.0 ** -10 * most).all())


def test_decode_loop_in_a_graph():
    """A step that hands out its own blocks, replayed: lengths live on the device."""
    rows, steps = 5, 40
    start = [3, 16, 0, 31, 15]
    need = [S.blocks(n) for n in start]
    tables_l, ids, at = [], list(range(60)), 0
    for n in need:
        tables_l.append(ids[at:at + n] + [-1] * (8 - n))
        at += n
    stack = ids[at:] + [-1] * at
    tables, free, count = ints(tables_l), ints(stack), ints([60 - at])
    ctx, lens, one = ints(start), ints([0] * rows), ints([1] * rows)
    loc, slots, pos = ints([0] * (rows + 1)), ints([0] * (rows + 2)), ints([0] * (rows + 2))

    def run():
        pb.pa_kv_alloc(tables, free, count, ctx, one, loc, lens, slots, pos)
        ctx.copy_(lens)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        run()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    want = dict(tables=tables_l, free=stack, count=60 - at, lens=start)
    for step in range(steps + 1):
        if step:
            g.replay()
        want, short = S.alloc(want["tables"], want["free"], want["count"], want["lens"], want["lens"], [1] * rows, rows + 2)
        assert status() == 0 and not short
        assert tables.tolist() == want["tables"] and slots.tolist() == want["slots"] and pos.tolist() == want["positions"]
        assert count.item() == want["count"] and ctx.tolist() == want["lens"]


def test_put_in_a_graph_and_on_another_stream():
    q, k, v = (torch.randn(9, n, 64, device="cuda").half() for n in (4, 2, 2))
    cache = [torch.zeros(3, 2, BS, 64, dtype=torch.float16, device="cuda") for _ in range(2)]
    slots, pos = ints(list(range(20, 29))), ints(list(range(9)))
    table = torch.rand(9, 32, device="cuda")
    eager, s = [torch.zeros_like(q), torch.zeros_like(k)], torch.cuda.Stream()
    torch.cuda.synchronize()
    pb.pa_kv_put(*eager, q, k, v, *cache, slots, pos, table, s)
    s.synchronize()
    want = [x.clone() for x in eager + cache]
    outs = [torch.zeros_like(q), torch.zeros_like(k)]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        pb.pa_kv_put(*outs, q, k, v, *cache, slots, pos, table)
    for c in cache:
        c.zero_()
    g.replay()
    assert status() == 0
    assert all(torch.equal(x, y) for x, y in zip(want, outs + cache))
    yr, yb = S.rotate(q, pos.long(), table, False)
    S.check(outs[0], yr, yb)


def test_alloc_on_two_streams_at_once():
    made, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for i in range(2):
        held = [(37 * j + 11 * i) % 90 for j in range(300)]
        made.append((held, S, i))
    cases = []
    for held, _, i in made:
        rows = [[-1] * 12 for _ in held]
        ids, at = list(range(4000)), 0
        for b, n in enumerate(held):
            for x in range(S.blocks(n)):
                rows[b][x] = ids[at]
                at += 1
        stack = ids[at:] + [-1] * at
        new = [(b * 7 + i) % 60 for b in range(300)]
        cases.append((held, rows, stack, 4000 - at, new))
    tensors = []
    torch.cuda.synchronize()
    for (held, rows, stack, count, new), s in zip(cases, streams):
        T = sum(new) + 3
        t = dict(tables=ints(rows), free=ints(stack), count=ints([count]), loc=ints([0] * 301), lens=ints([0] * 300),
                 slots=ints([0] * T), pos=ints([0] * T), ctx=ints(held), new=ints(new))
        tensors.append(t)
    torch.cuda.synchronize()
    for t, s in zip(tensors, streams):
        pb.pa_kv_alloc(t["tables"], t["free"], t["count"], t["ctx"], t["new"], t["loc"], t["lens"], t["slots"], t["pos"], s)
    assert status() == 0
    for (held, rows, stack, count, new), t in zip(cases, tensors):
        want, short = S.alloc(rows, stack, count, held, held, new, sum(new) + 3)
        assert not short and t["tables"].tolist() == want["tables"] and t["slots"].tolist() == want["slots"]
        assert t["count"].item() == want["count"] and t["pos"].tolist() == want["positions"]
