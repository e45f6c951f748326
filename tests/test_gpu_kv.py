"""The 8-bit cache and eviction calls on the GPU against 64-bit references."""
import math

import pytest
import torch

import kv_helpers as K
from kv_helpers import BS, DTYPES

pytestmark = pytest.mark.gpu
DEV = "cuda"


def pb():
    from paged_kv_cache_308_gb300 import binding
    return binding


def status():
    torch.cuda.synchronize()
    return pb().pa_get_device_status()


def check(got, ref, bound, what=""):
    err = (got.double() - ref).abs()
    bad = ~(err <= bound)  # NaN is bad too
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds, worst excess {float((err - bound).max()):.3g}"


def decode(c, weights=False, w_in=None, **kw):
    out = torch.full_like(c.q, math.nan)
    more = {}
    if weights:
        w = torch.full((len(c.lens), c.hkv, max(1, c.max_len)), -7.0, device=DEV)
        more = {"weights_out": w, "weights_in": w_in}
    pb().pa_kv_decode(out, c.q, *c.cache(), c.tables, c.seq_lens, c.scale, max_seq_len=c.max_len, **more, **kw)
    assert status() == 0
    return (out, w) if weights else out


SHAPES = [(24, 4, 256), (32, 8, 128), (8, 1, 64), (3, 3, 256), (7, 1, 128), (10, 2, 64)]


@pytest.mark.parametrize("fmt", ["f16", "e4m3", "int8"])
@pytest.mark.parametrize("heads,hkv,dim", SHAPES)
def test_decode_lengths(fmt, heads, hkv, dim):
    # lengths at block, warp and partition borders, an empty sequence among them; NaN past every end
    c = K.Case([1, 15, 16, 17, 0, 64, 65, 127, 255, 513, 700], heads, hkv, dim, fmt, seed=3, device=DEV, extra_cols=3)
    ref, bound, w, wb = K.decode_reference(c)
    out, got = decode(c, weights=True)
    check(out, ref, bound, "out")
    for b, n in enumerate(c.lens):
        check(got[b, :, :n], w[b, :, :n], wb[b, :, :n] + 1e-30, "weights")
        assert bool((got[b, :, n:] == -7).all())  # nothing is written past the end
    # in the same form the output has the same bits without the weights
    for mode in ("single", "split"):
        assert torch.equal(decode(c, mode=mode), decode(c, weights=True, mode=mode)[0])


@pytest.mark.parametrize("fmt", ["f16", "e4m3", "int8"])
@pytest.mark.parametrize("part", [0, 16, 64, 496, 1024])
def test_decode_partitions(fmt, part):
    c = K.Case([1000, 3, 497], 12, 2, 128, fmt, seed=4, device=DEV)
    ref, bound, w, wb = K.decode_reference(c)
    out, got = decode(c, weights=True, partition_size=part)
    check(out, ref, bound)
    for b, n in enumerate(c.lens):
        check(got[b, :, :n], w[b, :, :n], wb[b, :, :n] + 1e-30)
    single = decode(c, mode="single")
    check(single, ref, bound)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dim,hkv", [(64, 2), (128, 2), (256, 1)])
def test_decode_one_long_sequence(fmt, dim, hkv):
    c = K.Case([20011], 4 * hkv, hkv, dim, fmt, seed=5, device=DEV)
    ref, bound, w, wb = K.decode_reference(c)
    out, got = decode(c, weights=True)
    check(out, ref, bound)
    check(got, w, wb + 1e-30)
    assert torch.equal(decode(c), decode(c))  # fixed partitions: the same bits again


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_decode_peaked_and_unlike_blocks(fmt):
    # block scales spread over e^16, one key far above the rest: its value alone is the output
    c = K.Case([400, 90], 8, 2, 128, fmt, seed=6, device=DEV, spread=16.0)
    ref, bound, w, wb = K.decode_reference(c)
    out, got = decode(c, weights=True)
    check(out, ref, bound)
    for b, n in enumerate(c.lens):
        check(got[b, :, :n], w[b, :, :n], wb[b, :, :n] + 1e-30)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_decode_zero_scales_and_extreme_codes(fmt):
    c = K.Case([48, 40], 4, 1, 64, fmt, seed=7, device=DEV)
    top = 448.0 if fmt == "e4m3" else 127.0
    for b in range(2):
        blk = int(c.tables[b, 0])
        c.ks[blk] = 0.0                       # all scores of the block are 0
        blk = int(c.tables[b, 1])
        c.k[blk] = torch.tensor(top).to(c.k.dtype)
        c.v[blk] = torch.tensor(-top).to(c.k.dtype)
        c.vs[blk] = 0.0 if b else 2.0 ** -10
    ref, bound, w, wb = K.decode_reference(c)
    out, got = decode(c, weights=True)
    check(out, ref, bound)


def test_decode_accumulates_in_place_and_from_another_array():
    c = K.Case([200, 31], 8, 2, 128, "int8", seed=8, device=DEV)
    _, _, w, wb = K.decode_reference(c)
    base = torch.rand(2, 2, 250, device=DEV)
    acc = base.clone()
    out = torch.empty_like(c.q)
    call = lambda i, o: pb().pa_kv_decode(out, c.q, *c.cache(), c.tables, c.seq_lens, c.scale, max_seq_len=200,
                                          weights_in=i, weights_out=o)
    call(acc, acc)
    call(acc, acc)
    other = torch.full_like(base, 5.0)
    call(base, other)
    assert status() == 0
    for b, n in enumerate(c.lens):
        x = base[b, :, :n].double()
        # two additions: each rounds the sum by 2^-24
        check(acc[b, :, :n], x + 2 * w[b, :, :n], 2 * wb[b, :, :n] + 2.0 ** -23 * (x + 2 * w[b, :, :n]))
        check(other[b, :, :n], x + w[b, :, :n], wb[b, :, :n] + 2.0 ** -24 * (x + w[b, :, :n]))
        assert torch.equal(acc[b, :, n:], base[b, :, n:]) and bool((other[b, :, n:] == 5).all())


def _chunks(c, new, seed, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    half = lambda h: (torch.randn(sum(new), h, c.dim, generator=g, device=DEV) * scale).half()
    loc = [0]
    for n in new:
        loc.append(loc[-1] + n)
    return half(c.heads), half(c.hkv), half(c.hkv), torch.tensor(loc, dtype=torch.int32, device=DEV)


def append(c, new, k_new, v_new, loc):
    pb().pa_kv_append(*c.cache(), k_new, v_new, c.tables, c.seq_lens, loc, max_query_len=max(new))


def same(got, want, what):
    g = got.float().double() if got.element_size() == 1 else got.double()
    bad = ~((g == want) | (g.isnan() & want.isnan()))
    n = int(bad.sum())
    if n:
        at = bad.nonzero()[:3].tolist()
        raise AssertionError(f"{what}: {n} of {bad.numel()} differ, first {[(i, float(g[tuple(i)]), float(want[tuple(i)])) for i in at]}")


def same_cache(c, ref):
    k, v, ks, vs = ref
    for what, got, want in (("ks", c.ks, ks), ("vs", c.vs, vs), ("k", c.k, k), ("v", c.v, v)):
        if want is not None:
            same(got, want, what)


@pytest.mark.parametrize("fmt", ["f16", "e4m3", "int8"])
@pytest.mark.parametrize("hkv,dim", [(4, 256), (3, 128), (1, 64), (5, 64)])
def test_append(fmt, hkv, dim):
    ctx = [0, 1, 15, 16, 17, 100, 31, 40]
    new = [1, 1, 1, 1, 20, 50, 0, 8]
    c = K.Case(ctx, hkv, hkv, dim, fmt, seed=9, device=DEV, room=[a + b for a, b in zip(ctx, new)])
    for s, f in ((c.ks, 8.0), (c.vs, 0.125)):  # some scales grow, some do not
        if s is not None:
            s[::2] /= f
    _, k_new, v_new, loc = _chunks(c, new, 10)
    k_new[::3] *= 30
    ref = K.append_reference(c, new, k_new, v_new)
    append(c, new, k_new, v_new, loc)
    assert status() == 0
    same_cache(c, ref)
    append(c, new, k_new, v_new, loc)  # again: the same cache
    assert status() == 0
    same_cache(c, ref)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_token_by_token_is_the_repeated_definition(fmt):
    c = K.Case([3], 2, 2, 64, fmt, seed=11, device=DEV, room=[64])
    _, k_new, v_new, _ = _chunks(c, [40], 12)
    k_new *= torch.exp(torch.linspace(-6, 3, 40, device=DEV))[:, None, None].half()  # scales grow often
    loc = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    for i in range(40):
        ref = K.append_reference(c, [1], k_new[i:i + 1], v_new[i:i + 1])
        append(c, [1], k_new[i:i + 1].contiguous(), v_new[i:i + 1].contiguous(), loc)
        same_cache(c, ref)
        c.lens[0] += 1
        c.seq_lens += 1
    assert status() == 0


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_special_values(fmt):
    # zeros, subnormal halves, the largest half, infinities and NaN, ties between codes
    c = K.Case([0, 5, 2, 0, 0], 1, 1, 64, fmt, seed=13, device=DEV, room=[16] * 5)
    new = [4, 3, 2, 1, 6]
    _, k_new, v_new, loc = _chunks(c, new, 14)
    k_new[0:4] = 0
    k_new[4:7, 0, ::2] = math.inf
    k_new[4:7, 0, 1::4] = math.nan
    k_new[7:9] = 65504.0
    k_new[9] = 0.0
    k_new[9, 0, 3] = -math.inf
    k_new[10:16] = 2.0 ** -24
    k_new[11, 0, :32] = 0.0
    v_new[10:16, 0] = (torch.arange(6 * 64, device=DEV).view(6, 64) / 2.0 - 127.0).clamp(-127, 127).half()
    v_new[10, 0, 0] = 127.0
    ref = K.append_reference(c, new, k_new, v_new)
    append(c, new, k_new, v_new, loc)
    assert status() == 0
    same_cache(c, ref)


@pytest.mark.parametrize("fmt", ["f16", "e4m3", "int8"])
def test_append_padded_batch_and_large_chunk(fmt):
    # rows behind the last sequence are not read, entries of max_query_len above the real lengths only cost blocks
    c = K.Case([7, 0], 2, 2, 128, fmt, seed=15, device=DEV, room=[1007, 300])
    new = [1000, 300]
    _, k_new, v_new, loc = _chunks(c, new, 16)
    pad = torch.full((50, 2, 128), math.nan, dtype=torch.float16, device=DEV)
    ref = K.append_reference(c, new, k_new, v_new)
    pb().pa_kv_append(*c.cache(), torch.cat([k_new, pad]), torch.cat([v_new, pad]), c.tables, c.seq_lens, loc,
                      max_query_len=1300)
    assert status() == 0
    same_cache(c, ref)


@pytest.mark.parametrize("fmt", ["f16", "e4m3", "int8"])
@pytest.mark.parametrize("heads,hkv,dim", [(24, 4, 256), (8, 2, 128), (5, 1, 64)])
def test_prefix(fmt, heads, hkv, dim):
    ctx, new = [0, 1, 33, 500, 16], [5, 40, 1, 70, 0]
    c = K.Case(ctx, heads, hkv, dim, fmt, seed=17, device=DEV, extra_cols=2, spread=1.0)
    q, k_new, v_new, loc = _chunks(c, new, 18)
    ref, bound = K.prefix_reference(c, new, q, k_new, v_new)
    out = torch.full_like(q, math.nan)
    pb().pa_kv_prefix(out, q, k_new, v_new, *c.cache(), c.tables, c.seq_lens, loc, c.scale, max_context_len=500,
                      max_query_len=70)
    assert status() == 0
    check(out, ref, bound)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("form", ["persistent", "grid", "warp"])
@pytest.mark.parametrize("dim", [64, 256])
def test_prefix_kernels_and_scales(fmt, form, dim):
    # every kernel form; block scales e^8 apart, some of them 0, for INT8 of 24 significant bits
    ctx, new = [200, 7, 1000], [70, 150, 3]
    c = K.Case(ctx, 6, 2, dim, fmt, seed=84, device=DEV, spread=4.0)
    if fmt == "int8":
        c.ks *= 1.2345678
        c.vs *= 0.8765432
    for s in (c.ks, c.vs):
        s[int(c.tables[2, 5])] = 0.0
    q, k_new, v_new, loc = _chunks(c, new, 85)
    flags = {"persistent": 0, "grid": pb().PA_FLAG_PREFIX_GRID, "warp": pb().PA_FLAG_PREFIX_WARP_MMA}[form]
    ref, bound = K.prefix_reference(c, new, q, k_new, v_new, rounded=form == "warp" and fmt == "int8")
    out = torch.full_like(q, math.nan)
    pb().pa_kv_prefix(out, q, k_new, v_new, *c.cache(), c.tables, c.seq_lens, loc, c.scale, max_context_len=1000,
                      max_query_len=150, flags=flags)
    assert status() == 0
    check(out, ref, bound)


def test_prefix_negative_scale_and_special_blocks():
    # a negative softmax scale; NaN codes past the context's end in a block with a factor
    c = K.Case([37, 90], 4, 2, 128, "int8", seed=86, device=DEV, spread=2.0)
    c.scale = -c.scale
    q, k_new, v_new, loc = _chunks(c, [40, 20], 87)
    ref, bound = K.prefix_reference(c, [40, 20], q, k_new, v_new)
    out = torch.full_like(q, math.nan)
    pb().pa_kv_prefix(out, q, k_new, v_new, *c.cache(), c.tables, c.seq_lens, loc, c.scale, max_context_len=90,
                      max_query_len=40)
    assert status() == 0
    check(out, ref, bound)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_prefix_without_context(fmt):
    c = K.Case([0, 0], 4, 2, 64, fmt, seed=19, device=DEV)
    q, k_new, v_new, loc = _chunks(c, [20, 3], 20)
    ref, bound = K.prefix_reference(c, [20, 3], q, k_new, v_new)
    out = torch.full_like(q, math.nan)
    pb().pa_kv_prefix(out, q, k_new, v_new, *c.cache(), c.tables, c.seq_lens, loc, c.scale, max_context_len=0,
                      max_query_len=20)
    assert status() == 0
    check(out, ref, bound)


def evict(c, w, keep, sinks, recent, seed=0, dst_w=True, blocks=None, max_len=None):
    """Evict into fresh blocks of a second pool; returns everything written."""
    mk = max(keep)
    need = [-(-min(a, b) // BS) for a, b in zip(keep, c.lens)]
    total = sum(need) + 2
    perm = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    tables = torch.full((len(c.lens), max(1, -(-mk // BS))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        tables[b, :n] = perm[at:at + n]
        at += n
    fill = lambda t: torch.full((total,) + tuple(t.shape[1:]), 9.0, device=DEV).to(t.dtype)
    d = dict(k=fill(c.k), v=fill(c.v), ks=None if c.ks is None else fill(c.ks), vs=None if c.vs is None else fill(c.vs),
             tables=tables.to(DEV), kept=torch.full((len(c.lens), c.hkv, mk), -5, dtype=torch.int32, device=DEV),
             lens=torch.full((len(c.lens),), -5, dtype=torch.int32, device=DEV),
             w=torch.full((len(c.lens), c.hkv, mk + 3), -5.0, device=DEV) if dst_w else None)
    pb().pa_kv_evict(*c.cache(), c.tables, c.seq_lens, d["k"], d["v"], d["ks"], d["vs"], d["tables"],
                     torch.tensor(keep, dtype=torch.int32, device=DEV), w, d["kept"], d["lens"], d["w"],
                     max_seq_len=max_len or c.max_len, max_keep_len=mk, sinks=sinks, recent=recent)
    assert status() == 0
    return d


def check_evict(c, w, keep, sinks, recent, d):
    kept = K.evict_reference(c, w, keep, sinks, recent)
    want_k = torch.full(d["k"].shape, 9.0, dtype=torch.float64, device=DEV)
    want_v = want_k.clone()
    want_ks = None if c.ks is None else torch.full(d["ks"].shape, 9.0, dtype=torch.float64, device=DEV)
    want_vs = None if c.ks is None else want_ks.clone()
    raw = lambda t: t.float().double() if t.element_size() == 1 else t.double()
    for b, n in enumerate(c.lens):
        k = min(keep[b], n)
        assert int(d["lens"][b]) == k
        for h in range(c.hkv):
            pos = torch.tensor(kept[b][h], dtype=torch.long, device=DEV)
            assert d["kept"][b, h, :k].tolist() == kept[b][h]
            assert bool((d["kept"][b, h, k:] == -5).all())
            if d["w"] is not None:
                x, y = d["w"][b, h, :k], w[b, h][pos]
                assert bool(((x == y) | (x.isnan() & y.isnan())).all())
                assert bool((d["w"][b, h, k:] == -5).all())
            if k == 0:
                continue
            blk = c.tables[b].long()[pos // BS]
            to = d["tables"][b].long()
            for cache, scales, want, want_s in ((c.k, c.ks, want_k, want_ks), (c.v, c.vs, want_v, want_vs)):
                rows = raw(cache.view(torch.uint8)[blk, h, pos % BS].view(cache.dtype)
                           if cache.element_size() == 1 else cache[blk, h, pos % BS])
                for i in range(0, k, BS):
                    r = rows[i:i + BS]
                    t = int(to[i // BS])
                    if scales is not None:
                        s0 = scales[blk[i:i + BS], h].double()
                        s1 = s0.max()
                        r = K.round_code(r * s0[:, None] / s1, c.fmt) if float(s1) > 0 else r
                        want_s[t, h] = s1
                    want[t, h, :len(r)] = r
    if c.ks is not None:
        same(d["ks"], want_ks, "ks")
        same(d["vs"], want_vs, "vs")
    same(d["k"], want_k, "k")  # 9 as a code is 9 in every format
    same(d["v"], want_v, "v")


@pytest.mark.parametrize("fmt", ["f16", "e4m3", "int8"])
@pytest.mark.parametrize("hkv,dim", [(4, 256), (2, 128), (3, 64)])
@pytest.mark.parametrize("sinks,recent", [(0, 0), (4, 16), (3, 1)])
def test_evict(fmt, hkv, dim, sinks, recent):
    lens = [0, 1, 15, 16, 17, 100, 333, 40]
    keep = [5, 1, 7, 16, 3, 40, 100, 64]
    c = K.Case(lens, hkv, hkv, dim, fmt, seed=21, device=DEV, extra_cols=1)
    g = torch.Generator(device=DEV).manual_seed(22)
    w = torch.rand(len(lens), hkv, 340, generator=g, device=DEV) ** 6
    w = torch.where(torch.rand(w.shape, generator=g, device=DEV) < 0.3, torch.zeros_like(w), w)  # many equal
    check_evict(c, w, keep, sinks, recent, evict(c, w, keep, sinks, recent))


@pytest.mark.parametrize("keep,sinks,recent", [([0, 0], 4, 4), ([2, 3], 4, 8), ([10, 12], 4, 8), ([12, 200], 0, 500),
                                               ([300, 1], 1, 0)])
def test_evict_budgets_below_the_protected_tokens(keep, sinks, recent):
    c = K.Case([120, 260], 2, 2, 64, "int8", seed=23, device=DEV)
    w = torch.rand(2, 2, 260, generator=torch.Generator(device=DEV).manual_seed(24), device=DEV)
    check_evict(c, w, keep, sinks, recent, evict(c, w, keep, sinks, recent, dst_w=False))


@pytest.mark.parametrize("kind", ["equal", "negative", "special", "tiny"])
def test_evict_orders_weights(kind):
    c = K.Case([200, 77], 2, 2, 64, "f16", seed=25, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(26)
    w = torch.rand(2, 2, 200, generator=g, device=DEV)
    if kind == "equal":
        w = torch.full_like(w, 0.25)
    if kind == "negative":
        w = w - 0.5
        w[:, :, ::5] = -0.0
        w[:, :, 1::5] = 0.0
    if kind == "special":
        w[:, :, ::3] = math.nan
        w[:, :, 1::7] = math.inf
        w[:, :, 2::7] = -math.inf
    if kind == "tiny":
        w = w * 1e-42  # subnormal numbers
    for keep in ([50, 20], [190, 77], [199, 1]):
        check_evict(c, w, keep, 2, 3, evict(c, w, keep, 2, 3))


@pytest.mark.parametrize("B,n,keep", [(2, 9000, 1000), (2, 20000, 19999), (2, 40000, 5), (2, 40001, 20000), (8, 14001, 3000),
                                      (20, 26003, 2000), (90, 13000, 50)])
def test_evict_long(B, n, keep):
    # lengths that one block has to itself, and that 2, 4 and 8 blocks of a cluster share
    c = K.Case([n] + [50] * (B - 1), 2, 2, 64, "e4m3", seed=27, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(28)
    w = torch.rand(B, 2, n, generator=g, device=DEV) ** 8
    w = torch.where(w < 0.01, torch.zeros_like(w), w)
    want, recent = [keep] + [20] * (B - 1), 64 if keep > 64 else 1
    check_evict(c, w, want, 4, recent, evict(c, w, want, 4, recent))


def test_evict_more_tokens_than_the_blocks_can_hold():
    # beyond the shared memory of a whole cluster the weights are read again in every round
    n = 400003
    c = K.Case([n], 1, 1, 64, "f16", seed=29, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(30)
    w = torch.rand(1, 1, n, generator=g, device=DEV) ** 3
    w = torch.where(w < 0.2, torch.zeros_like(w), w)
    check_evict(c, w, [150001], 4, 100, evict(c, w, [150001], 4, 100))


@pytest.mark.parametrize("fmt", ["f16", "int8"])
@pytest.mark.parametrize("B", [31, 32, 33, 70, 1100])
def test_append_finds_its_sequence_in_large_batches(fmt, B):
    g = torch.Generator().manual_seed(B)
    ctx = torch.randint(0, 40, (B,), generator=g).tolist()
    new = torch.randint(0, 20, (B,), generator=g).tolist()
    new[0], new[-1], new[B // 2] = 0, 50, 90
    c = K.Case(ctx, 5, 5, 64, fmt, seed=31, device=DEV, room=[a + b for a, b in zip(ctx, new)])
    _, k_new, v_new, loc = _chunks(c, new, 32)
    ref = K.append_reference(c, new, k_new, v_new)
    append(c, new, k_new, v_new, loc)
    assert status() == 0
    same_cache(c, ref)


@pytest.mark.parametrize("fmt", ["f16", "e4m3", "int8"])
@pytest.mark.parametrize("B,top,long,hkv,dim", [(200, 60, 0, 2, 64), (33, 300, 2500, 3, 128), (64, 40, 5000, 1, 256), (700, 20, 0, 1, 64),
                                                (5, 900, 0, 16, 64)])
def test_decode_ragged_batches(fmt, B, top, long, hkv, dim):
    # runs of blocks that cross many sequences, empty ones among them, one long sequence in the middle
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, top + 1, (B,), generator=g).tolist()
    lens[0] = lens[-1] = 0
    if long:
        lens[B // 2] = long
    c = K.Case(lens, 3 * hkv, hkv, dim, fmt, seed=33, device=DEV)
    ref, bound, w, wb = K.decode_reference(c)
    out, got = decode(c, weights=True)
    check(out, ref, bound)
    for b, n in enumerate(c.lens):
        check(got[b, :, :n], w[b, :, :n], wb[b, :, :n] + 1e-30)
        assert bool((got[b, :, n:] == -7).all())
    assert torch.equal(decode(c), out) and torch.equal(decode(c), out)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("heads,hkv,dim,ctx,new", [(24, 4, 256, [1500], [3]), (32, 8, 128, [2100, 0, 64, 700], [37, 5, 1, 0]),
                                                   (8, 1, 64, [4003, 100, 1, 1000, 513], [1, 150, 17, 40, 64]),
                                                   (3, 3, 256, [1023, 1024], [1, 130])])
def test_prefix_in_key_ranges(fmt, heads, hkv, dim, ctx, new):
    # few query tiles after long contexts; sequences shorter than a range, without context, without a chunk
    c = K.Case(ctx, heads, hkv, dim, fmt, seed=35, device=DEV)
    q, k_new, v_new, loc = _chunks(c, new, 36)
    ref, bound = K.prefix_reference(c, new, q, k_new, v_new)
    first = None
    for fill in (0x00, 0xff):  # whatever the workspace holds
        ws = torch.full((pb().pa_kv_prefix_workspace_size(len(ctx), max(ctx), hkv, dim, DTYPES[fmt]),), fill,
                        dtype=torch.uint8, device=DEV)
        out = torch.full_like(q, math.nan)
        pb().pa_kv_prefix(out, q, k_new, v_new, *c.cache(), c.tables, c.seq_lens, loc, c.scale, max_context_len=max(ctx),
                          max_query_len=max(new), workspace=ws)
        assert status() == 0
        check(out, ref, bound)
        assert first is None or torch.equal(first, out)
        first = out


@pytest.mark.parametrize("mode", ["auto", "split"])
@pytest.mark.parametrize("fmt", ["f16", "e4m3", "int8"])
@pytest.mark.parametrize("heads,hkv,dim,B", [(6, 1, 256, 1), (24, 4, 256, 3), (32, 8, 128, 8), (8, 8, 64, 20), (7, 1, 128, 70),
                                             (3, 3, 64, 2)])
def test_decode_forms(mode, fmt, heads, hkv, dim, B):
    # few and short sequences in clusters of 2, 4 and 8 CTAs (auto) and in equal shares: lengths that leave CTAs and warps
    # without blocks, one block past a round, none
    lens = ([1000, 0, 1, 64, 65, 513, 130, 16] + [(37 * i) % 600 for i in range(B)])[:B]
    c = K.Case(lens, heads, hkv, dim, fmt, seed=34, device=DEV, extra_cols=2)
    ref, bound, w, wb = K.decode_reference(c)
    start = torch.rand(B, hkv, c.max_len, device=DEV)
    for again in range(2):
        out, got = decode(c, weights=True, w_in=start, mode=mode)
        check(out, ref, bound)
        for b, n in enumerate(c.lens):
            # (adding the old weight rounds the sum once more, by 2^-24 of at most 1 + the heads)
            check(got[b, :, :n], w[b, :, :n] + start[b, :, :n].double(), wb[b, :, :n] + (1 + heads / hkv) * 2.0 ** -24)
            assert bool((got[b, :, n:] == -7).all())
        plain = decode(c, mode=mode)  # (with and without the weights the form may differ)
        check(plain, ref, bound)
        if again:
            assert torch.equal(plain, first[0]) and torch.equal(out, first[1]) and torch.equal(got, first[2])
        first = plain, out, got


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_decode_value_scales_far_apart(fmt):
    # the block with the weight has values 2^-30 of its neighbours', whose keys are far below
    c = K.Case([64, 100, 33], 4, 1, 128, fmt, seed=34, device=DEV, spread=0.0)
    for b in range(3):
        for j in range(-(-c.lens[b] // BS)):
            c.vs[int(c.tables[b, j])] *= 2.0 ** (-30 if j == b else 0)
            if j != b:
                c.ks[int(c.tables[b, j])] = 0.0  # scores 0
    # scores of the small blocks: about 60 above the rest
    for b in range(3):
        blk = int(c.tables[b, b])
        c.k[blk] = torch.tensor(1.0).to(c.k.dtype).to(DEV)
        c.ks[blk] = 30.0
    c.q.fill_(0.18)
    ref, bound, w, wb = K.decode_reference(c)
    out, got = decode(c, weights=True)
    check(out.double() * 2 ** 12, ref * 2 ** 12, bound * 2 ** 12)
    for b, n in enumerate(c.lens):
        check(got[b, :, :n], w[b, :, :n], wb[b, :, :n] + 1e-30)
    tiny = K.Case([40], 4, 1, 64, fmt, seed=35, device=DEV)
    tiny.vs[tiny.tables[0].long()] = 1e-42  # a subnormal scale: zero in fp16
    assert bool((decode(tiny) == 0).all())


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_to_blocks_with_a_callers_scales(fmt):
    # scales of 24 significant bits, and a code of -128: quotients are rounded to 32 bits first
    c = K.Case([5, 9], 2, 2, 64, fmt, seed=88, device=DEV, room=[16, 16])
    c.ks *= 1.2345678
    c.vs *= 0.000123456
    if fmt == "int8":
        c.k[int(c.tables[0, 0]), 0, 1, ::3] = -128
    _, k_new, v_new, loc = _chunks(c, [4, 7], 89)
    k_new *= 0.1
    old = [(c.k.clone(), c.ks.clone()), (c.v.clone(), c.vs.clone())]
    append(c, [4, 7], k_new, v_new, loc)
    assert status() == 0
    for (codes, scales), got, got_s, new in zip(old, (c.k, c.v), (c.ks, c.vs), (k_new, v_new)):
        for b, (n, m) in enumerate(zip(c.lens, (4, 7))):
            blk = int(c.tables[b, 0])
            x = new[int(loc[b]):int(loc[b]) + m].float().transpose(0, 1)
            for h in range(2):
                s0 = scales[blk, h]
                s1 = torch.maximum(s0, s0.new_tensor(K.scale_of(float(x[h].abs().max()), fmt)))
                assert float(got_s[blk, h]) == float(s1)
                want = K.round_code((x[h] / s1).double(), fmt)
                same(got[blk, h, n:n + m], want, "new")
                was = codes[blk, h, :n].float()
                want = K.round_code(((was * s0) / s1).double(), fmt) if float(s1) > float(s0) else was.double()
                same(got[blk, h, :n], want, "old")


@pytest.mark.parametrize("mode", ["auto", "single", "split"])
def test_decode_blocks_of_minus_infinity(mode):
    # scores of -infinity fill whole blocks, partitions and one head's whole sequence: they weigh nothing; a sequence
    # without any other score has none to normalise (NaN), as a softmax of -infinity alone
    c = K.Case([1100, 40, 700, 20], 4, 2, 64, "f16", seed=90, device=DEV)
    c.q[:, :, 0] = 1.0
    for b, upto in ((0, 600), (1, 16), (2, 0), (3, 20)):
        for t in range(upto):
            c.k[int(c.tables[b, t // BS]), :, t % BS, 0] = -math.inf
    ref, bound, w, wb = K.decode_reference(c)
    out = torch.full_like(c.q, 7.0)
    got = torch.full((4, 2, 1100), -7.0, device=DEV)
    pb().pa_kv_decode(out, c.q, *c.cache(), c.tables, c.seq_lens, c.scale, max_seq_len=1100, weights_out=got, mode=mode)
    assert status() == 0
    for b in range(3):  # (the bound of a dot product with infinities is none: a plain tolerance for fp16 outputs)
        err = (out[b].double() - ref[b]).abs()
        assert bool((err <= 2.0 ** -10 * (1 + ref[b].abs())).all())
        assert bool(((got[b, :, :c.lens[b]].double() - w[b, :, :c.lens[b]]).abs() <= 1e-5 * (1 + w[b, :, :c.lens[b]])).all())
    assert bool(out[3].isnan().all()) and bool(ref[3].isnan().all())
