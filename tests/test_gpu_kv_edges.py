"""Calls of the 8-bit cache's operators at the edges of what their arguments
allow, on the GPU against the 64-bit references."""
import math

import pytest
import torch

import kv_helpers as K
from test_gpu_kv import DEV, _chunks, check, check_evict, evict, pb, status

pytestmark = pytest.mark.gpu


def prefix_tiles(c, new):
    """Query tiles of a pa_kv_prefix call: 128 rows each, a token having one row per head of its kv head."""
    return -(-max(new) // (128 // (c.heads // c.hkv))) * c.hkv * len(new)


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def prefix(c, q, k_new, v_new, loc, new, flags=0, workspace=None):
    out = torch.full_like(q, math.nan)
    pb().pa_kv_prefix(out, q, k_new, v_new, *c.cache(), c.tables, c.seq_lens, loc, c.scale, max_context_len=c.max_len,
                      max_query_len=max(new), flags=flags, workspace=workspace)
    assert status() == 0
    return out


@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-45, -1e-45])
@pytest.mark.parametrize("fmt", ["f16", "e4m3", "int8"])
@pytest.mark.parametrize("form", ["grid", "ranges", "persistent", "warp"])
def test_prefix_with_a_softmax_scale_of_zero(form, fmt, scale):
    # equal scores: the mean of the visible V
    ctx, new = ([1500, 0, 700], [3, 37, 1]) if form == "ranges" else ([100, 0, 33], [40, 17, 1])
    if form == "persistent":
        ctx, new = ctx * 4, [70] + new * 3 + [0, 9]
    c = K.Case(ctx, 16, 8 if form == "persistent" else 2, 64, fmt, seed=93, device=DEV, spread=1.0)
    c.scale = scale
    q, k_new, v_new, loc = _chunks(c, new, 94)
    flags = pb().PA_FLAG_PREFIX_GRID if form == "grid" else pb().PA_FLAG_PREFIX_WARP_MMA if form == "warp" else 0
    assert (prefix_tiles(c, new) > sms()) == (form == "persistent")
    ref, bound = K.prefix_reference(c, new, q, k_new, v_new, rounded=form == "warp" and fmt == "int8")
    if form == "ranges" and fmt == "f16":  # (the fp16 cache's key ranges are a call of their own)
        out = torch.full_like(q, math.nan)
        pb().pa_prefix_split(out, q, k_new, v_new, c.k, c.v, c.tables, c.seq_lens, loc, 16, 2, 64, 16, scale,
                             max_context_len=c.max_len, max_query_len=max(new), parts=3, units=prefix_tiles(c, new))
        assert status() == 0
    else:
        out = prefix(c, q, k_new, v_new, loc, new, flags)
    check(out, ref, bound)


@pytest.mark.parametrize("fmt", ["f16", "e4m3", "int8"])
@pytest.mark.parametrize("heads,hkv,dim", [(12, 4, 64), (16, 4, 128), (24, 4, 256), (7, 7, 64)])
def test_prefix_with_more_query_tiles_than_the_device_has_sms(fmt, heads, hkv, dim):
    # the form whose CTAs claim tile after tile: ragged contexts and chunks, some empty, unlike block scales (for INT8 of
    # 24 significant bits), so that a factor of the tile, sequence or head before would show; the same bits as a CTA a tile
    g = torch.Generator().manual_seed(dim + hkv)
    B = 24
    ctx = [0, 511, 16, 17, 1] + torch.randint(0, 500, (B - 5,), generator=g).tolist()
    new = [33, 1, 0, 200, 16] + torch.randint(0, 130, (B - 5,), generator=g).tolist()
    ctx[9] = new[11] = 0
    c = K.Case(ctx, heads, hkv, dim, fmt, seed=95, device=DEV, spread=4.0, extra_cols=1)
    if fmt == "int8":
        c.ks *= 1.2345678
        c.vs *= 0.8765432
    if fmt != "f16":
        for s in (c.ks, c.vs):
            s[int(c.tables[3, 1])] = 0.0
    q, k_new, v_new, loc = _chunks(c, new, 96)
    assert prefix_tiles(c, new) > 2 * sms()
    ref, bound = K.prefix_reference(c, new, q, k_new, v_new)
    size = pb().pa_kv_prefix_workspace_size(B, c.max_len, hkv, dim, K.DTYPES[fmt])
    for fill in (0x00, 0xff):  # (and again: the claims begin at the first tile)
        ws = torch.full((size,), fill, dtype=torch.uint8, device=DEV) if size else None
        out = prefix(c, q, k_new, v_new, loc, new, workspace=ws)
        check(out, ref, bound)
        assert torch.equal(out, prefix(c, q, k_new, v_new, loc, new, pb().PA_FLAG_PREFIX_GRID))


@pytest.mark.parametrize("fmt,exponent,exact", [("e4m3", -15, True), ("e4m3", 7, True), ("e4m3", -22, False), ("e4m3", 8, False),
                                                ("int8", -24, True), ("int8", 8, True), ("int8", -28, False)])
def test_prefix_over_the_smallest_and_largest_scales(fmt, exponent, exact):
    # the fp16 copy of the context: exact for the scales that the header names, its rounding outside of them
    s = 2.0 ** exponent
    ctx, new = [200, 33, 700], [40, 5, 3]
    c = K.Case(ctx, 6, 2, 64, fmt, seed=104, device=DEV, spread=0.0)
    factor = 1.0 if fmt == "e4m3" else 1.2109375  # (8 significant bits)
    c.ks.fill_(s * factor), c.vs.fill_(s * factor)
    for x in (c.k, c.v):  # every code, the smallest ones too
        codes = (torch.tensor([a * b for a in K.E4M3_VALUES for b in (1, -1)]) if fmt == "e4m3" else
                 torch.arange(-127, 128).float()).to(DEV)
        pick = torch.randint(0, codes.numel(), x.shape, generator=torch.Generator(device=DEV).manual_seed(105), device=DEV)
        live = x.float().isfinite() if fmt == "e4m3" else x != -128
        x.copy_(torch.where(live, codes[pick].to(x.dtype).float(), x.float()).to(x.dtype))
    size = 100 * s
    c.scale = 1 / (8 * size)
    q, k_new, v_new, loc = _chunks(c, new, 106)
    k_new, v_new = ((x.double() * size).clamp(-65504, 65504).half() for x in (k_new, v_new))
    copy = K.Case(ctx, 6, 2, 64, "f16", seed=104, device=DEV)
    copy.scale, copy.tables = c.scale, c.tables
    copy.k, copy.v = ((x.float() * s).clamp(-65504, 65504).half() for x in (c.k, c.v))
    copy.ks, copy.vs = (torch.full_like(x, factor) for x in (c.ks, c.vs))
    for b in range(3):
        for a, h in zip(c.tokens(b), copy.tokens(b)):
            assert torch.equal(a, h) == exact
    ref, bound = K.prefix_reference(copy, new, q, k_new, v_new)
    for flags in (0, pb().PA_FLAG_PREFIX_GRID):
        check(prefix(c, q, k_new, v_new, loc, new, flags), ref, bound)


@pytest.mark.parametrize("fmt", ["f16", "int8"])
@pytest.mark.parametrize("form", ["grid", "ranges", "persistent", "warp"])
def test_prefix_reports_offsets_whose_difference_wraps_around(form, fmt):
    # 2^31 - 3 and -2^31 + 2 are five apart in 32 bits: no sequence of five tokens, and no row there to read or write
    few = form != "persistent"
    ctx, new = ([1500, 700] if form == "ranges" else [20, 90], [5, 5]) if few else ([20] * 12, [70] + [5] * 11)
    c = K.Case(ctx, 16, 2 if few else 8, 64, fmt, seed=102, device=DEV)
    q, k_new, v_new, loc = _chunks(c, new, 103)
    assert (prefix_tiles(c, new) > sms()) == (form == "persistent")
    ref, bound = K.prefix_reference(c, new, q, k_new, v_new, rounded=form == "warp" and fmt == "int8")
    loc[1], loc[2] = 2 ** 31 - 3, -2 ** 31 + 2
    flags = pb().PA_FLAG_PREFIX_GRID if form == "grid" else pb().PA_FLAG_PREFIX_WARP_MMA if form == "warp" else 0
    out = torch.full_like(q, 7.0)
    pb().pa_kv_prefix(out, q, k_new, v_new, *c.cache(), c.tables, c.seq_lens, loc, c.scale, max_context_len=c.max_len,
                      max_query_len=max(new), flags=flags)
    assert status() == pb().PA_DEV_BAD_SEQ_LEN
    at = sum(new[:3])  # the sequences behind them have their rows
    assert bool((out[:at] == 7).all())
    check(out[at:], ref[at:], bound[at:])


@pytest.mark.parametrize("place", ["seq_lens", "keep_lens"])
@pytest.mark.parametrize("hkv,lens", [(2, [20000, 50]), (8, [(37 * i) % 700 for i in range(60)]), (1, [30, 0, 5]),
                                      (2, [26003] + [100] * 19)])
def test_evict_writes_the_new_lengths_in_place_of_the_old(hkv, lens, place):
    # in clusters, in more blocks than the SMs hold at once, with sequences below their budget: the same as into an
    # array of their own, for the later blocks too, which find the lengths where they were
    c = K.Case(lens, hkv, hkv, 64, "int8", seed=97, device=DEV)
    w = torch.rand(len(lens), hkv, c.max_len, generator=torch.Generator(device=DEV).manual_seed(98), device=DEV)
    keep = [(29 * i + 11) % 60 for i in range(len(lens))]
    d = evict(c, w, keep, 2, 3)
    check_evict(c, w, keep, 2, 3, d)
    for replayed in (False, True):
        seq, want = c.seq_lens.clone(), torch.tensor(keep, dtype=torch.int32, device=DEV)
        new = seq if place == "seq_lens" else want
        got = {n: torch.full_like(t, -5) if n in ("kept", "w") else torch.full(t.shape, 9.0, device=DEV).to(t.dtype)
               for n, t in d.items() if n not in ("tables", "lens")}
        call = lambda: pb().pa_kv_evict(*c.cache(), c.tables, seq, got["k"], got["v"], got["ks"], got["vs"], d["tables"], want,
                                        w, got["kept"], new, got["w"], max_seq_len=c.max_len, max_keep_len=max(keep), sinks=2,
                                        recent=3)
        if replayed:
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            g = torch.cuda.CUDAGraph()
            with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
                call()
            g.replay()
        else:
            call()
        assert status() == 0
        check_evict(c, w, keep, 2, 3, {**got, "lens": new, "tables": d["tables"]})
        other, was = (want, keep) if new is seq else (seq, c.lens)
        assert other.tolist() == list(was)


def test_evict_in_place_leaves_a_bad_length():
    c = K.Case([100, 200], 2, 2, 64, "f16", seed=99, device=DEV)
    w = torch.rand(2, 2, 200, device=DEV)
    seq = torch.tensor([100, 201], dtype=torch.int32, device=DEV)
    dst = torch.arange(2, dtype=torch.int32, device=DEV).view(2, 1)
    pool = [torch.zeros(2, 2, 16, 64, dtype=torch.float16, device=DEV) for _ in range(2)]
    pb().pa_kv_evict(c.k, c.v, None, None, c.tables, seq, *pool, None, None, dst,
                     torch.tensor([9, 9], dtype=torch.int32, device=DEV), w,
                     torch.zeros(2, 2, 16, dtype=torch.int32, device=DEV), seq, max_seq_len=200, max_keep_len=16)
    assert status() == pb().PA_DEV_BAD_SEQ_LEN and seq.tolist() == [9, 201]


def test_evict_refuses_outputs_over_the_lengths():
    c = K.Case([100, 90], 1, 1, 64, "f16", seed=100, device=DEV)
    w = torch.rand(2, 1, 100, device=DEV)
    room = torch.zeros(64, dtype=torch.int32, device=DEV)
    seq, keep, new = room[:2], torch.tensor([9, 9], dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    seq.copy_(c.seq_lens)
    dst = torch.arange(2, dtype=torch.int32, device=DEV).view(2, 1)
    pool = [torch.zeros(2, 1, 16, 64, dtype=torch.float16, device=DEV) for _ in range(2)]
    call = lambda kept, dst_w: pb().pa_kv_evict(c.k, c.v, None, None, c.tables, seq, *pool, None, None, dst, keep, w, kept, new,
                                                dst_w, max_seq_len=100, max_keep_len=16)
    kept = torch.zeros(2, 1, 16, dtype=torch.int32, device=DEV)
    for bad in ((room[:32].view(2, 1, 16), None), (room[1:33].view(2, 1, 16), None),
                (kept, room[:32].view(torch.float32).view(2, 1, 16))):
        with pytest.raises(pb().PaDecodeError):
            call(*bad)
    torch.cuda.synchronize()
    assert seq.tolist() == [100, 90] and new.tolist() == [0, 0]
    call(room[2:34].view(2, 1, 16), None)  # right behind them
    assert status() == 0 and new.tolist() == [9, 9] and seq.tolist() == [100, 90]


@pytest.mark.parametrize("opt", [dict(), dict(mode="single"), dict(mode="split"), dict(partition_size=64)])
@pytest.mark.parametrize("fmt", ["f16", "e4m3"])
@pytest.mark.parametrize("B", [1, 2, 70])
def test_decode_of_empty_sequences_in_every_form(B, fmt, opt):
    c = K.Case([0] * B, 4, 2, 64, fmt, seed=101, device=DEV)
    w = torch.full((B, 2, 4), -7.0, device=DEV)
    for weights in (None, w):
        out = torch.full_like(c.q, math.nan)
        pb().pa_kv_decode(out, c.q, *c.cache(), c.tables, c.seq_lens, c.scale, max_seq_len=0, weights_out=weights, **opt)
        assert status() == 0 and bool((out == 0).all()) and bool((w == -7).all())
    # a length that the bound of 0 does not allow is reported
    c.seq_lens[B - 1] = 3
    out = torch.full_like(c.q, math.nan)
    pb().pa_kv_decode(out, c.q, *c.cache(), c.tables, c.seq_lens, c.scale, max_seq_len=0, **opt)
    assert status() == pb().PA_DEV_BAD_SEQ_LEN and bool((out[:B - 1] == 0).all()) and bool(out[B - 1].isnan().all())


def _raw_append(k, v, ks, vs, new_k, new_v, ctx):
    """Append new_k and new_v ([blocks, heads, tokens, dim]) to blocks that hold ctx tokens each, a sequence a block."""
    B, hkv, n, dim = new_k.shape
    rows = lambda x: x.transpose(1, 2).reshape(B * n, hkv, dim).contiguous()
    ints = lambda x: torch.as_tensor(x, dtype=torch.int32, device=DEV)
    pb().pa_kv_append(k, v, ks, vs, rows(new_k), rows(new_v), torch.arange(B, dtype=torch.int32, device=DEV).view(B, 1),
                      ints([ctx] * B), torch.arange(0, B * n + 1, n, dtype=torch.int32, device=DEV), max_query_len=n)
    assert status() == 0


def test_int8_codes_of_every_half_in_every_scale():
    # A code is the integer nearest to x / s, ties to even; s has 8 significant bits.  Its exponent only shifts the
    # quotients, so 128 scales and all halves are every case.  In 64 bits x / s (11 bits over 8) is a tie exactly or further
    # from one than its rounding, so the reference's round is the quotient's.
    halves = torch.arange(0, 0x7c00, dtype=torch.int16, device=DEV).view(torch.float16)
    x = torch.cat([halves, -halves])                       # 63488
    per = 15 * 256                                         # new tokens of a block of 16, the first being there already
    n = -(-x.numel() // per)
    x = torch.nn.functional.pad(x, (0, n * per - x.numel())).view(1, n, 15, 256)
    s = torch.arange(128, 256, device=DEV).float() * 2
    hkv = 8
    x = torch.where(x.float().abs() > 127 * s[:, None, None, None], torch.zeros_like(x), x)  # so that no scale grows
    new = x.reshape(128 * n // hkv, hkv, 15, 256)
    scales = s[:, None].expand(128, n).reshape(-1, hkv).contiguous()
    k = torch.zeros(new.shape[0], hkv, 16, 256, dtype=torch.int8, device=DEV)
    v, ks, vs = k.clone(), scales.clone(), scales.clone()
    _raw_append(k, v, ks, vs, new, -new, 1)
    want = torch.round(new.double() / scales.double()[:, :, None, None]).clamp(-127, 127).to(torch.int8)
    assert torch.equal(ks, scales) and torch.equal(vs, scales)
    assert torch.equal(k[:, :, 1:], want) and torch.equal(v[:, :, 1:], -want)
    assert bool((k[:, :, 0] == 0).all())


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_every_code_from_every_scale_to_every_larger_one(fmt):
    # A block whose scale grows from s0 to s1 has its codes c rounded again to c s0 / s1.  INT8: all pairs of 8-bit
    # significands, s1 up to 2^9 of s0 (there every code is 0); E4M3: all powers of two that an append can make.  c s0 and
    # s1 are exact in 64 bits, and their quotient (15 bits over 8) is a tie exactly or further from one than its rounding.
    # (torch's pow on the GPU is not exact at powers of two)
    powers = lambda lo, hi: torch.tensor([2.0 ** i for i in range(lo, hi + 1)], dtype=torch.float64, device=DEV)
    if fmt == "int8":
        codes = torch.arange(-127, 128, device=DEV).float()
        s1, s0, e = torch.meshgrid(torch.arange(128, 256, device=DEV).double(), torch.arange(128, 256, device=DEV).double(),
                                   powers(-9, 0), indexing="ij")
        s0 = s0 * e
        s0, s1 = s0[s0 < s1], s1[s0 < s1]
        top = 127 * s1
    else:
        codes = torch.tensor(K.E4M3_VALUES + [-c for c in K.E4M3_VALUES], device=DEV)
        s1, s0 = torch.meshgrid(powers(-32, 8), powers(-32, 8), indexing="ij")
        s0, s1 = s0[s0 < s1], s1[s0 < s1]
        top = (448 * s1).clamp(max=65504)
    # the largest half whose scale is s1: one that does not exceed `top`
    a = top.half()
    a = torch.where(a.double() > top, (a.view(torch.int16) - 1).view(torch.float16), a)
    assert bool((a.double() <= top).all()) and bool(a.isfinite().all())
    hkv, dim = 4, 64
    pad = -s0.numel() % (2 * hkv)
    s0, s1, a = (torch.cat([t, t[:1].expand(pad)]) for t in (s0, s1, a))
    old = torch.nn.functional.pad(codes, (0, 256 - codes.numel())).view(4, dim)  # four tokens
    dt = K.DTYPES[fmt]

    def side(s0, s1, a):
        cache = torch.zeros(s0.shape[0], hkv, 16, dim, device=DEV)
        cache[:, :, :4] = old
        new = torch.zeros(s0.shape[0], hkv, 1, dim, dtype=torch.float16, device=DEV)
        new[:, :, 0, 5] = a
        return cache.to(dt), s0.float(), new

    half = s0.numel() // 2
    parts = [[t[i * half:(i + 1) * half].view(-1, hkv).contiguous() for t in (s0, s1, a)] for i in range(2)]
    (k, ks, new_k), (v, vs, new_v) = side(*parts[0]), side(*parts[1])
    _raw_append(k, v, ks, vs, new_k, new_v, 4)
    for got, scales, (p0, p1, top) in ((k, ks, parts[0]), (v, vs, parts[1])):
        assert torch.equal(scales.double(), p1)
        for at in range(0, got.shape[0], 4096):
            r = slice(at, at + 4096)
            want = K.round_code(old.double() * (p0[r] / p1[r])[:, :, None, None] if fmt == "e4m3" else
                                old.double() * p0[r][:, :, None, None] / p1[r][:, :, None, None], fmt)
            assert torch.equal(got[r, :, :4].float().double(), want)
            assert torch.equal(got[r, :, 4, 5].float().double(), K.round_code(top[r].double() / p1[r], fmt))
