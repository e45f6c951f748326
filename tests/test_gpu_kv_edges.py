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
