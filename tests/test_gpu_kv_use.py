"""The 8-bit cache and eviction calls as a server uses them: one after the other
over one pool, on streams, in graphs, with bad tables and lengths, and with
caches past 32-bit offsets."""
import math

import pytest
import torch

import kv_helpers as K
from kv_helpers import BS
from test_gpu_kv import DEV, _chunks, append, check, check_evict, decode, evict, pb, same, same_cache, status

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("fmt", ["f16", "e4m3", "int8"])
def test_prompt_decode_evict_decode(fmt):
    """Two prompt chunks, decoding with the weights added up, eviction into fresh blocks of the same
    pool, decoding on from there: every call against the references on the cache as it stands."""
    heads, hkv, dim, B = 8, 2, 128, 3
    c = K.Case([0, 0, 0], heads, hkv, dim, fmt, seed=41, device=DEV, room=[160, 100, 200], spare=24)
    width = 256
    w = torch.zeros(B, hkv, width, device=DEV)

    def prompt(new, seed):
        q, k_new, v_new, loc = _chunks(c, new, seed)
        ref, bound = K.prefix_reference(c, new, q, k_new, v_new)
        out = torch.full_like(q, math.nan)
        pb().pa_kv_prefix(out, q, k_new, v_new, *c.cache(), c.tables, c.seq_lens, loc, c.scale,
                          max_context_len=max(c.lens), max_query_len=max(new))
        check(out, ref, bound, "prefix")
        cache = K.append_reference(c, new, k_new, v_new)
        append(c, new, k_new, v_new, loc)
        same_cache(c, cache)
        c.lens = [a + b for a, b in zip(c.lens, new)]
        c.seq_lens += ints(new)
        c.max_len = max(c.lens)

    def steps(n, seed):
        for i in range(n):
            q, k_new, v_new, loc = _chunks(c, [1] * B, seed + i)
            append(c, [1] * B, k_new, v_new, loc)
            c.lens = [a + 1 for a in c.lens]
            c.seq_lens += 1
            c.max_len = max(c.lens)
            c.q = q
            ref, bound, ww, wb = K.decode_reference(c)
            before = w.clone()
            out = torch.full_like(q, math.nan)
            pb().pa_kv_decode(out, q, *c.cache(), c.tables, c.seq_lens, c.scale, max_seq_len=c.max_len, weights_in=w,
                              weights_out=w)
            check(out, ref, bound, "decode")
            for b, n_b in enumerate(c.lens):
                want = before[b, :, :n_b].double() + ww[b, :, :n_b]
                check(w[b, :, :n_b], want, wb[b, :, :n_b] + 2.0 ** -24 * want + 1e-30, "weights")

    prompt([100, 33, 128], 42)
    prompt([40, 50, 1], 44)
    steps(6, 50)
    # down to 64 tokens a sequence (the second keeps fewer), into blocks that nobody uses
    keep = [64, 20, 64]
    free = list(c.free)
    dst = torch.full((B, 6), -1, dtype=torch.int32)
    for b in range(B):
        for j in range(4):
            dst[b, j] = free.pop()
        # (two more blocks to decode on)
        dst[b, 4], dst[b, 5] = free.pop(), free.pop()
    kept = torch.full((B, hkv, 64), -5, dtype=torch.int32, device=DEV)
    lens = ints([0] * B)
    w2 = torch.zeros(B, hkv, width, device=DEV)
    want = K.evict_reference(c, w, keep, 4, 8)
    rows = [[c.tokens(b)[kv][h][torch.tensor(want[b][h], device=DEV)] for kv in range(2)]
            for b in range(B) for h in range(hkv)]
    pb().pa_kv_evict(*c.cache(), c.tables, c.seq_lens, *c.cache(), dst.to(DEV), ints(keep), w, kept, lens, w2,
                     max_seq_len=c.max_len, max_keep_len=64, sinks=4, recent=8)
    assert status() == 0
    assert lens.tolist() == keep
    for b in range(B):
        for h in range(hkv):
            assert kept[b, h, :keep[b]].tolist() == want[b][h]
            assert torch.equal(w2[b, h, :keep[b]], w[b, h][kept[b, h, :keep[b]].long()])
    old_w, w = w, w2
    c.tables, c.lens, c.seq_lens, c.max_len = dst.to(DEV), list(keep), lens, 64
    # the moved rows: the same values, or (8 bits) rounded to the scale of their new block
    for b in range(B):
        for h in range(hkv):
            for kv in range(2):
                now, was = c.tokens(b)[kv][h], rows[b * hkv + h][kv]
                scales = (c.ks, c.vs)[kv]
                step = 0.0
                if fmt == "int8":
                    step = scales[c.tables[b].long()[torch.arange(keep[b], device=DEV) // BS], h].double()[:, None] / 2
                if fmt == "e4m3":  # only values in the new scale's subnormal range round, by half of 2^-9
                    step = scales[c.tables[b].long()[torch.arange(keep[b], device=DEV) // BS], h].double()[:, None] * 2.0 ** -10
                assert bool(((now - was).abs() <= step).all())
    steps(20, 80)
    assert status() == 0 and bool((old_w >= 0).all())


def test_decode_of_sequences_that_share_blocks():
    c = K.Case([64, 64, 50], 8, 2, 64, "e4m3", seed=60, device=DEV)
    c.tables[1, :3] = c.tables[0, :3]
    c.tables[2, :2] = c.tables[0, :2]
    ref, bound, _, _ = K.decode_reference(c)
    check(decode(c), ref, bound)


@pytest.mark.parametrize("fmt", ["f16", "e4m3"])
def test_a_length_bound_above_the_lengths_changes_nothing(fmt):
    c = K.Case([700, 0, 33, 1000], 8, 2, 128, fmt, seed=61, device=DEV, extra_cols=200)
    ref, bound, _, _ = K.decode_reference(c)
    for bound_len in (1000, 1001, 4000):
        out = torch.full_like(c.q, math.nan)
        pb().pa_kv_decode(out, c.q, *c.cache(), c.tables, c.seq_lens, c.scale, max_seq_len=bound_len)
        assert status() == 0
        check(out, ref, bound)


def test_empty_calls():
    c = K.Case([0, 0], 4, 2, 64, "int8", seed=62, device=DEV)
    out = torch.full_like(c.q, math.nan)
    w = torch.full((2, 2, 4), -7.0, device=DEV)
    pb().pa_kv_decode(out, c.q, *c.cache(), c.tables, c.seq_lens, c.scale, max_seq_len=0, weights_out=w)
    assert status() == 0 and bool((out == 0).all()) and bool((w == -7).all())
    kept = torch.full((2, 2, 0), -5, dtype=torch.int32, device=DEV)
    lens = ints([9, 9])
    pb().pa_kv_evict(*c.cache(), c.tables, c.seq_lens, c.k.clone(), c.v.clone(), c.ks.clone(), c.vs.clone(), c.tables,
                     ints([0, 0]), w, kept, lens, max_seq_len=4, max_keep_len=0)
    assert status() == 0 and lens.tolist() == [0, 0]


# ---- streams and graphs

def test_on_another_stream():
    c = K.Case([900, 77], 8, 2, 64, "int8", seed=63, device=DEV)
    ref, bound, _, _ = K.decode_reference(c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [torch.full_like(c.q, math.nan) for _ in range(3)]
    args = (c.q, *c.cache(), c.tables, c.seq_lens, c.scale)
    pb().pa_kv_decode(outs[0], *args, s, max_seq_len=900)                # a Stream
    pb().pa_kv_decode(outs[1], *args, s.cuda_stream, max_seq_len=900)    # its handle
    with torch.cuda.stream(s):
        pb().pa_kv_decode(outs[2], *args, max_seq_len=900)               # the current one
    torch.cuda.synchronize()
    for o in outs:
        check(o, ref, bound)


def test_two_calls_at_once():
    cs = [K.Case([3000 + 100 * i, 50], 8, 2, 128, "e4m3", seed=64 + i, device=DEV) for i in range(2)]
    refs = [K.decode_reference(c) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    outs = [[torch.full_like(c.q, math.nan) for _ in range(20)] for c in cs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for i in range(20):
        for c, s, o in zip(cs, streams, outs):
            with torch.cuda.stream(s):
                pb().pa_kv_decode(o[i], c.q, *c.cache(), c.tables, c.seq_lens, c.scale, max_seq_len=c.max_len)
    torch.cuda.synchronize()
    for o, (ref, bound, _, _) in zip(outs, refs):
        for x in o:
            check(x, ref, bound)
    assert status() == 0


def test_captured_calls_follow_the_lengths_of_their_replay():
    """A decoding step (append, decode with weights) and an eviction, captured once and replayed as the
    sequences grow: nothing is fixed at capture but the bounds."""
    c = K.Case([30, 5], 4, 2, 64, "e4m3", seed=66, device=DEV, room=[128, 128], spare=20)
    q, k_new, v_new, loc = _chunks(c, [1, 1], 67)
    w = torch.zeros(2, 2, 128, device=DEV)
    out = torch.empty_like(q)
    ws = torch.empty(pb().pa_kv_decode_workspace_size(2, 128, 4, 2, 64, c.k.dtype, weights=True), dtype=torch.uint8,
                     device=DEV)
    append(c, [1, 1], k_new, v_new, loc)  # (warm-up; the same again below)

    def step():
        pb().pa_kv_append(*c.cache(), k_new, v_new, c.tables, c.seq_lens, loc, max_query_len=1)
        c.seq_lens.add_(1)
        pb().pa_kv_decode(out, q, *c.cache(), c.tables, c.seq_lens, c.scale, max_seq_len=128, weights_in=w, weights_out=w,
                          workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step()
    c.seq_lens.copy_(ints([30, 5]))
    w.zero_()
    for i in range(25):
        qn, kn, vn, _ = _chunks(c, [1, 1], 100 + i)
        q.copy_(qn), k_new.copy_(kn), v_new.copy_(vn)
        want = K.append_reference(c, [1, 1], k_new, v_new)
        before = w.clone()
        g.replay()
        torch.cuda.synchronize()
        same_cache(c, want)
        c.lens = [a + 1 for a in c.lens]
        c.max_len = max(c.lens)
        c.q = q
        ref, bound, ww, wb = K.decode_reference(c)
        check(out, ref, bound)
        for b, n in enumerate(c.lens):
            x = before[b, :, :n].double() + ww[b, :, :n]
            check(w[b, :, :n], x, wb[b, :, :n] + 2.0 ** -24 * x + 1e-30)
    assert status() == 0
    keep = [16, 50]
    d = evict(c, w, keep, 2, 3)  # eager
    dst = {k: (torch.zeros_like(v) if v is not None else None) for k, v in d.items()}
    dst["tables"] = d["tables"]
    for x in ("k", "v", "ks", "vs", "w"):
        dst[x].copy_(torch.full(dst[x].shape, -5.0 if x == "w" else 9.0, device=DEV).to(dst[x].dtype))
    dst["kept"].fill_(-5)
    keeps = ints([1, 1])
    with torch.cuda.stream(s):
        s.wait_stream(torch.cuda.current_stream())
        g2 = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g2, stream=s):
            pb().pa_kv_evict(*c.cache(), c.tables, c.seq_lens, dst["k"], dst["v"], dst["ks"], dst["vs"], dst["tables"], keeps, w,
                             dst["kept"], dst["lens"], dst["w"], max_seq_len=128, max_keep_len=50, sinks=2, recent=3)
    keeps.copy_(ints(keep))
    torch.cuda.synchronize()
    g2.replay()
    torch.cuda.synchronize()
    check_evict(c, w, keep, 2, 3, dst)
    assert status() == 0


def test_prefix_captured_with_its_workspace():
    c = K.Case([100, 17], 4, 2, 64, "int8", seed=68, device=DEV, spread=1.0)
    new = [20, 33]
    q, k_new, v_new, loc = _chunks(c, new, 69)
    ref, bound = K.prefix_reference(c, new, q, k_new, v_new)
    ws = torch.empty(pb().pa_kv_prefix_workspace_size(2, 100, 2, 64, c.k.dtype), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(q)
    call = lambda: pb().pa_kv_prefix(out, q, k_new, v_new, *c.cache(), c.tables, c.seq_lens, loc, c.scale, max_context_len=100,
                                     max_query_len=33, workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call()
    for _ in range(3):
        out.fill_(math.nan)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        check(out, ref, bound)
    assert status() == 0


# ---- bad tables and lengths: reported, and nothing else is disturbed

def _flags(st):
    return bool(st & 1), bool(st & 2)  # block id, length


@pytest.mark.parametrize("fmt", ["f16", "int8"])
@pytest.mark.parametrize("bad", [-1, -2 ** 31, 10 ** 6, 2 ** 31 - 1])
def test_decode_reports_bad_block_ids(fmt, bad):
    c = K.Case([700, 40, 90], 4, 2, 64, fmt, seed=70, device=DEV)
    ref, bound, _, _ = K.decode_reference(c)
    c.tables[0, 7] = bad
    out = torch.full_like(c.q, math.nan)
    for kw in ({}, dict(mode="single"), dict(mode="split"), dict(partition_size=64)):
        pb().pa_kv_decode(out, c.q, *c.cache(), c.tables, c.seq_lens, c.scale, max_seq_len=700, **kw)
        assert _flags(status()) == (True, False)
        check(out[1:], ref[1:], bound[1:])


@pytest.mark.parametrize("fmt", ["f16", "e4m3"])
def test_tokens_of_a_bad_block_get_no_weight(fmt):
    c = K.Case([700, 40, 90], 4, 2, 64, fmt, seed=74, device=DEV)
    c.tables[0, 7] = -1
    before = torch.rand(3, 2, 700, device=DEV)
    out = torch.empty_like(c.q)
    for kw in ({}, dict(mode="single"), dict(mode="split"), dict(partition_size=64)):
        ws = torch.full((1 << 22,), 0.5, device=DEV)  # what an earlier call may have left as scores
        got = before.clone()
        pb().pa_kv_decode(out, c.q, *c.cache(), c.tables, c.seq_lens, c.scale, max_seq_len=700, weights_in=got,
                          weights_out=got, workspace=ws, **kw)
        assert _flags(status()) == (True, False)
        assert torch.equal(got[0, :, 112:128], before[0, :, 112:128])
        # the others' still add up to one a query head (2^-12 for p's sum of 684 terms, half an ulp of the sums)
        rest = (got - before)[0].double().sum(dim=1)
        assert bool(((rest - 2).abs() < 1e-3).all())


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_prefix_with_a_bad_block_does_not_read_an_old_workspace(fmt):
    c = K.Case([128, 64], 4, 2, 64, fmt, seed=75, device=DEV)
    q, k_new, v_new, loc = _chunks(c, [20, 9], 76)
    c.tables[0, 3] = 10 ** 6
    outs = []
    for fill in (0x00, 0x7f):
        ws = torch.full((1 << 22,), fill, dtype=torch.uint8, device=DEV)
        out = torch.empty_like(q)
        pb().pa_kv_prefix(out, q, k_new, v_new, *c.cache(), c.tables, c.seq_lens, loc, c.scale, max_context_len=128,
                          max_query_len=20, workspace=ws)
        assert _flags(status()) == (True, False)
        outs.append(out.clone())
    assert torch.equal(outs[0], outs[1]) and bool(torch.isfinite(outs[0]).all())


@pytest.mark.parametrize("bad", [-1, 701, 2 ** 31 - 1, -2 ** 31])
def test_decode_reports_bad_lengths(bad):
    c = K.Case([700, 40, 90], 4, 2, 64, "e4m3", seed=71, device=DEV)
    ref, bound, w, wb = K.decode_reference(c)
    c.seq_lens[1] = bad
    for kw in ({}, dict(mode="single"), dict(mode="split"), dict(partition_size=64)):
        out = torch.full_like(c.q, math.nan)
        got = torch.full((3, 2, 700), -7.0, device=DEV)
        pb().pa_kv_decode(out, c.q, *c.cache(), c.tables, c.seq_lens, c.scale, max_seq_len=700, weights_out=got, **kw)
        assert _flags(status()) == (False, True)
        for b in (0, 2):
            check(out[b], ref[b], bound[b])
            check(got[b, :, :c.lens[b]], w[b, :, :c.lens[b]], wb[b, :, :c.lens[b]] + 1e-30)
        assert bool((got[1] == -7).all())


@pytest.mark.parametrize("fmt", ["f16", "e4m3"])
def test_append_reports_bad_tables_and_lengths(fmt):
    def fresh():
        c = K.Case([10, 20, 5], 2, 2, 64, fmt, seed=72, device=DEV, room=[60, 60, 60])
        new = [30, 5, 20]
        _, k_new, v_new, loc = _chunks(c, new, 73)
        return c, new, k_new, v_new, loc

    c, new, k_new, v_new, loc = fresh()
    good = c.tables.clone()
    keep = [x.clone() if x is not None else None for x in c.cache()]
    c.tables[0, 1] = 10 ** 6
    append(c, new, k_new, v_new, loc)
    assert _flags(status()) == (True, False)
    # the other blocks got their tokens: those of a sequence without the bad block
    c2, *_ = fresh()
    append(c2, new, k_new, v_new, loc)
    status()
    skip = int(good[0, 1])
    for got, want, was in zip(c.cache(), c2.cache(), keep):
        if got is not None:
            others = [i for i in range(got.shape[0]) if i != skip]
            raw = lambda t: t.view(torch.uint8 if t.element_size() == 1 else torch.int16 if t.element_size() == 2 else torch.int32)
            assert torch.equal(raw(got)[others], raw(want)[others]) and torch.equal(raw(got)[skip], raw(was)[skip])

    for change in ("ctx_negative", "ctx_long", "loc_negative", "loc_order", "loc_end", "over_bound"):
        c, new, k_new, v_new, loc = fresh()
        keep = [x.clone() if x is not None else None for x in c.cache()]
        most = max(new)
        if change == "ctx_negative":
            c.seq_lens[1] = -3
        if change == "ctx_long":
            c.seq_lens[1] = c.tables.shape[1] * BS - 2  # 5 more do not fit
        if change == "loc_negative":
            loc[0] = -4
        if change == "loc_order":
            loc[2] = 10
        if change == "loc_end":
            loc[3] = 1000
        if change == "over_bound":
            most = 29
        pb().pa_kv_append(*c.cache(), k_new, v_new, c.tables, c.seq_lens, loc, max_query_len=most)
        assert _flags(status())[1], change
        victims = {"ctx_negative": [1], "ctx_long": [1], "loc_negative": [0], "loc_order": [1], "loc_end": [2],
                   "over_bound": [0]}[change]
        for b in victims:  # the sequence's blocks are as they were
            ids = c.tables[b][c.tables[b] >= 0].long()
            for got, was in zip(c.cache(), keep):
                if got is not None:
                    raw = lambda t: t.view(torch.uint8 if t.element_size() == 1 else torch.int16 if t.element_size() == 2 else torch.int32)
                    assert torch.equal(raw(got)[ids], raw(was)[ids]), change


@pytest.mark.parametrize("change", ["order", "negative", "end", "ctx"])
def test_append_reports_bad_lengths_in_a_large_batch(change):
    # a batch whose tile slots are packed: the report does not hang on which sequences the search meets
    lens = [3] * 100
    c = K.Case(lens, 2, 2, 64, "int8", seed=91, device=DEV, room=[40] * 100)
    new = [1] * 99 + [30]
    _, k_new, v_new, loc = _chunks(c, new, 92)
    if change == "order":
        loc[50] = 5
    if change == "negative":
        loc[50] = -2 ** 31
    if change == "end":
        loc[100] = 2 ** 31 - 1
    if change == "ctx":
        c.seq_lens[7] = 2 ** 31 - 1
    append(c, new, k_new, v_new, loc)
    assert _flags(status()) == (False, True)


def test_evict_reports_bad_tables_and_lengths():
    c = K.Case([100, 200, 50], 2, 2, 64, "int8", seed=74, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(75)
    w = torch.rand(3, 2, 200, generator=g, device=DEV)
    kept = torch.full((3, 2, 64), -5, dtype=torch.int32, device=DEV)
    lens = ints([-5] * 3)
    pool = [torch.full((12,) + tuple(x.shape[1:]), 9.0, device=DEV).to(x.dtype) for x in c.cache()]
    dst = torch.arange(12, dtype=torch.int32, device=DEV).view(3, 4)

    def call(seq_lens, keep, tables=None, dst_tables=None):
        kept.fill_(-5)
        lens.fill_(-5)
        for x in pool:
            x.copy_(torch.full(x.shape, 9.0, device=DEV).to(x.dtype))
        pb().pa_kv_evict(*c.cache(), tables if tables is not None else c.tables, ints(seq_lens), *pool,
                         dst_tables if dst_tables is not None else dst, ints(keep), w, kept, lens, max_seq_len=200,
                         max_keep_len=64, sinks=2, recent=4)
        return _flags(status())

    ok = [100, 200, 50]
    for seq_lens, keep in (([100, -1, 50], [20] * 3), ([100, 201, 50], [20] * 3), (ok, [20, 65, 20]), (ok, [20, -1, 20]),
                           ([100, 2 ** 31 - 1, 50], [20] * 3)):
        assert call(seq_lens, keep) == (False, True)
        assert lens.tolist() == [20, -5, 20] and bool((kept[1] == -5).all())
        assert bool((pool[0][4:8].float() == 9).all()) and bool((pool[2][4:8] == 9).all())
        want = K.evict_reference(c, w, [20, 20, 20], 2, 4)
        for b in (0, 2):
            assert [kept[b, h, :20].tolist() for h in range(2)] == want[b]
    bad = c.tables.clone()
    bad[1, 0] = -1  # holds the sinks, so it is read
    assert call(ok, [20] * 3, tables=bad) == (True, False) and lens.tolist() == [20] * 3
    bad = dst.clone()
    bad[1, 1] = 12
    assert call(ok, [20] * 3, dst_tables=bad) == (True, False)
    assert bool((pool[0][5].float() == 9).all())


def test_prefix_reports_bad_tables_and_lengths():
    c = K.Case([100, 60, 30], 4, 2, 64, "e4m3", seed=76, device=DEV, spread=1.0)
    new = [8, 9, 10]
    q, k_new, v_new, loc = _chunks(c, new, 77)
    ref, bound = K.prefix_reference(c, new, q, k_new, v_new)
    good = c.tables.clone()
    out = torch.full_like(q, math.nan)
    call = lambda: pb().pa_kv_prefix(out, q, k_new, v_new, *c.cache(), c.tables, c.seq_lens, loc, c.scale, max_context_len=100,
                                     max_query_len=10)
    c.tables[1, 1] = 10 ** 6
    call()
    assert _flags(status())[0]
    check(out[:8], ref[:8], bound[:8])
    check(out[17:], ref[17:], bound[17:])
    c.tables = good
    c.seq_lens[1] = 101
    out.fill_(math.nan)
    call()
    assert _flags(status())[1]
    check(out[:8], ref[:8], bound[:8])
    check(out[17:], ref[17:], bound[17:])


# ---- large sizes

@pytest.mark.parametrize("fmt", ["f16", "e4m3"])
def test_offsets_past_32_bits(fmt):
    """Blocks whose bytes lie beyond 2^32 from the pool's start: append, decode, prefix, eviction."""
    hkv, dim = 16, 256
    blocks = 2 ** 33 // (hkv * BS * dim) if fmt == "e4m3" else 2 ** 32 // (hkv * BS * dim)
    blocks += 40
    dt = K.DTYPES[fmt]
    k, v = (torch.zeros(blocks, hkv, BS, dim, dtype=torch.uint8 if fmt == "e4m3" else dt, device=DEV).view(dt) for _ in range(2))
    ks, vs = ((torch.zeros(blocks, hkv, device=DEV) for _ in range(2)) if fmt == "e4m3" else (None, None))
    c = K.Case([40, 70], 2 * hkv, hkv, dim, "f16", seed=78, device=DEV)  # (for its lengths and queries)
    c.fmt, c.k, c.v, c.ks, c.vs = fmt, k, v, ks, vs
    c.tables = ints([[blocks - 1 - i for i in range(0, 14, 2)], [blocks - 20 - i for i in range(7)]])
    lens = c.lens
    c.lens, c.seq_lens = [0, 0], ints([0, 0])
    q, k_new, v_new, loc = _chunks(c, lens, 79)
    append(c, lens, k_new, v_new, loc)
    assert status() == 0
    at = 0
    for b, n in enumerate(lens):  # the rows are where they belong
        for i in (0, n - 1):
            blk = int(c.tables[b, i // BS])
            row = k[blk, :, i % BS].float()
            if ks is not None:
                row = row * ks[blk][:, None]
            x = k_new[at + i].float()
            assert bool(((row - x).abs() <= x.abs() * 2.0 ** -4 + 1e-3).all())
        at += n
    c.lens, c.seq_lens, c.max_len = lens, ints(lens), max(lens)
    ref, bound, w, wb = K.decode_reference(c)
    out, got = decode(c, weights=True)
    check(out, ref, bound)
    q, k_new, v_new, loc = _chunks(c, [3, 5], 80)
    ref, bound = K.prefix_reference(c, [3, 5], q, k_new, v_new)
    out = torch.full_like(q, math.nan)
    pb().pa_kv_prefix(out, q, k_new, v_new, *c.cache(), c.tables, c.seq_lens, loc, c.scale, max_context_len=70, max_query_len=5)
    assert status() == 0
    check(out, ref, bound)
    # evict from the pool's end into it again
    dst = ints([[blocks - 30], [blocks - 31]])
    kept = torch.full((2, hkv, 16), -5, dtype=torch.int32, device=DEV)
    n = ints([0, 0])
    want = K.evict_reference(c, got, [16, 16], 1, 2)
    was = [c.tokens(b)[0] for b in range(2)]
    pb().pa_kv_evict(*c.cache(), c.tables, c.seq_lens, *c.cache(), dst, ints([16, 16]), got, kept, n, max_seq_len=70,
                     max_keep_len=16, sinks=1, recent=2)
    assert status() == 0 and n.tolist() == [16, 16]
    for b in range(2):
        for h in range(hkv):
            assert kept[b, h].tolist() == want[b][h]
            now = K.values(k.view(torch.uint8)[[blocks - 30 - b]].view(dt) if ks is not None else k[[blocks - 30 - b]],
                           None if ks is None else ks[[blocks - 30 - b]])[0, h]
            step = 0.0 if ks is None else float(ks[blocks - 30 - b, h]) * 2.0 ** -10
            assert bool(((now - was[b][h][kept[b, h].long()]).abs() <= step).all())


def test_wide_weights_rows_and_many_sequences():
    # rows of weights much longer than the sequences, 3000 sequences of a few tokens
    g = torch.Generator().manual_seed(81)
    lens = torch.randint(0, 6, (3000,), generator=g).tolist()
    c = K.Case(lens, 2, 1, 64, "int8", seed=82, device=DEV)
    ref, bound, w, wb = K.decode_reference(c)
    for kw in ({}, dict(mode="split")):
        out = torch.full_like(c.q, math.nan)
        got = torch.full((3000, 1, 1000), -7.0, device=DEV)
        pb().pa_kv_decode(out, c.q, *c.cache(), c.tables, c.seq_lens, c.scale, max_seq_len=c.max_len, weights_out=got, **kw)
        assert status() == 0
        check(out, ref, bound)
        n = c.max_len
        live = torch.arange(n, device=DEV) < c.seq_lens[:, None, None]
        check(torch.where(live, got[..., :n].double(), 0.0), torch.where(live, w[..., :n], 0.0), wb[..., :n] + 1e-30)
        assert bool((got[..., n:] == -7).all()) and bool((torch.where(live, -7.0, got[..., :n].double()) == -7).all())


def test_wrong_tensors_are_refused():
    c = K.Case([20], 4, 2, 64, "int8", seed=83, device=DEV)
    out = torch.empty_like(c.q)
    call = lambda **kw: pb().pa_kv_decode(**{**dict(out=out, q=c.q, k_cache=c.k, v_cache=c.v, k_scales=c.ks, v_scales=c.vs,
                                                    block_tables=c.tables, seq_lens=c.seq_lens, scale=c.scale,
                                                    max_seq_len=20), **kw})
    for kw, err in ((dict(q=c.q.float()), TypeError), (dict(q=c.q.cpu()), ValueError), (dict(k_scales=None), ValueError),
                    (dict(v_scales=c.vs[:, :1]), ValueError), (dict(v_cache=c.v[:-1]), ValueError),
                    (dict(v_cache=c.v.view(torch.uint8)), TypeError), (dict(seq_lens=c.seq_lens.long()), TypeError),
                    (dict(block_tables=c.tables[0]), ValueError), (dict(out=out[:, :2]), ValueError),
                    (dict(k_cache=c.k.transpose(1, 2)), ValueError), (dict(weights_in=torch.zeros(1, 2, 20, device=DEV)), ValueError),
                    (dict(weights_out=torch.zeros(1, 3, 20, device=DEV)), ValueError),
                    (dict(workspace=torch.empty(9, device="cpu")), ValueError)):
        with pytest.raises(err):
            call(**kw)
    with pytest.raises(pb().PaDecodeError):
        call(weights_out=torch.zeros(1, 2, 19, device=DEV))  # rows shorter than the bound
    with pytest.raises(pb().PaDecodeError):
        call(max_seq_len=33)  # more than the table's row
    with pytest.raises(pb().PaDecodeError):
        call(weights_out=torch.zeros(1, 2, 20, device=DEV), workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
