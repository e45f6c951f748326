"""The 8-bit cache and eviction calls without a GPU: their references against
closed forms, argument checks, workspace sizes."""
import ctypes
import math

import pytest
import torch

import kv_helpers as K
from paged_kv_cache_308_gb300 import binding as pb

FAKE = 0x10000  # a 16-byte aligned non-null address that no call dereferences


def cache(fmt=pb.PA_KV_E4M3, nb=100, hkv=4, D=256, bs=16, **p):
    d = dict(k_cache=FAKE, v_cache=FAKE, k_scales=FAKE, v_scales=FAKE)
    d.update(p)
    return pb.pa_kv_cache(d["k_cache"], d["v_cache"], d["k_scales"], d["v_scales"], nb, hkv, D, bs, fmt)


def decode_args(c=None, heads=24, B=2, mbps=50, max_len=800, scale=0.0625, stride=800, w_in=0, w_out=0, **p):
    d = dict(out=FAKE, q=FAKE, bt=FAKE, lens=FAKE)
    d.update(p)
    return pb.pa_kv_decode_args(d["out"], d["q"], c or cache(), d["bt"], d["lens"], w_in, w_out, stride, B, mbps,
                                max_len, heads, scale)


def append_args(c=None, B=2, T=10, mbps=50, max_q=5, **p):
    d = dict(k=FAKE, v=FAKE, bt=FAKE, ctx=FAKE, loc=FAKE)
    d.update(p)
    return pb.pa_kv_append_args(c or cache(), d["k"], d["v"], d["bt"], d["ctx"], d["loc"], B, T, mbps, max_q)


def prefix_args(c=None, heads=24, B=2, T=10, mbps=50, max_ctx=800, max_q=5, scale=0.0625, **p):
    d = dict(out=FAKE, q=FAKE, k=FAKE, v=FAKE, bt=FAKE, ctx=FAKE, loc=FAKE)
    d.update(p)
    return pb.pa_kv_prefix_args(d["out"], d["q"], d["k"], d["v"], c or cache(), d["bt"], d["ctx"], d["loc"], B, T, mbps,
                                max_ctx, max_q, heads, scale)


def evict_args(src=None, dst=None, B=2, mbps=50, dmbps=10, max_len=800, max_keep=160, ws=800, dws=160, sinks=0, recent=0,
               **p):
    d = dict(bt=FAKE, dbt=FAKE + 64, lens=FAKE, keep=FAKE, w=FAKE, dw=FAKE + 64, kept=FAKE, new=FAKE)
    d.update(p)
    return pb.pa_kv_evict_args(src or cache(), dst or cache(), d["bt"], d["dbt"], d["lens"], d["keep"], d["w"], d["dw"],
                               d["kept"], d["new"], ws, dws, B, mbps, dmbps, max_len, max_keep, sinks, recent)


def call(fn, a, opts=None, ws=None, n=0):
    if fn in ("pa_kv_append", "pa_kv_evict"):
        return getattr(pb.lib, fn)(ctypes.byref(a), None)
    return getattr(pb.lib, fn)(ctypes.byref(a), ctypes.byref(opts) if opts else None, ws, n, None)


BAD_CACHES = [(dict(fmt=3), pb.PA_ERR_INVALID_ARG), (dict(fmt=-1), pb.PA_ERR_INVALID_ARG),
              (dict(hkv=0), pb.PA_ERR_INVALID_ARG), (dict(nb=-1), pb.PA_ERR_INVALID_ARG),
              (dict(D=96), pb.PA_ERR_UNSUPPORTED), (dict(bs=32), pb.PA_ERR_UNSUPPORTED),
              (dict(nb=1 << 31), pb.PA_ERR_UNSUPPORTED), (dict(nb=1 << 26), pb.PA_ERR_UNSUPPORTED),
              (dict(k_cache=0), pb.PA_ERR_INVALID_ARG), (dict(v_cache=FAKE + 8), pb.PA_ERR_INVALID_ARG),
              (dict(k_scales=0), pb.PA_ERR_INVALID_ARG), (dict(v_scales=FAKE + 2), pb.PA_ERR_INVALID_ARG)]


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_bad_caches_are_refused(kw, code):
    for fn, make in (("pa_kv_append", append_args), ("pa_kv_decode", decode_args), ("pa_kv_prefix", prefix_args)):
        assert call(fn, make(cache(**kw))) == code, fn
    assert call("pa_kv_evict", evict_args(src=cache(**kw), dst=cache(**kw))) == code


@pytest.mark.parametrize("kw,code", [
    (dict(heads=23), pb.PA_ERR_INVALID_ARG), (dict(heads=36), pb.PA_ERR_UNSUPPORTED), (dict(heads=0), pb.PA_ERR_INVALID_ARG),
    (dict(B=-1), pb.PA_ERR_INVALID_ARG), (dict(B=65536), pb.PA_ERR_INVALID_ARG), (dict(max_len=801), pb.PA_ERR_INVALID_ARG),
    (dict(max_len=-1), pb.PA_ERR_INVALID_ARG), (dict(scale=math.nan), pb.PA_ERR_INVALID_ARG),
    (dict(scale=math.inf), pb.PA_ERR_INVALID_ARG), (dict(out=0), pb.PA_ERR_INVALID_ARG), (dict(q=FAKE + 8), pb.PA_ERR_INVALID_ARG),
    (dict(bt=0), pb.PA_ERR_INVALID_ARG), (dict(lens=FAKE + 2), pb.PA_ERR_INVALID_ARG),
    (dict(w_out=FAKE, stride=799), pb.PA_ERR_INVALID_ARG), (dict(w_in=FAKE), pb.PA_ERR_INVALID_ARG),
    (dict(w_out=FAKE + 1), pb.PA_ERR_INVALID_ARG)])
def test_decode_refusals(kw, code):
    assert call("pa_kv_decode", decode_args(**kw)) == code


def test_decode_options_and_workspace_are_checked():
    big = dict(ws=FAKE, n=1 << 40)
    for o, code in ((dict(mode="fused"), pb.PA_ERR_INVALID_ARG), (dict(mode="flat"), pb.PA_ERR_INVALID_ARG),
                    (dict(partition_size=-16), pb.PA_ERR_INVALID_ARG), (dict(partition_size=24), pb.PA_ERR_INVALID_ARG),
                    (dict(warps=4, stages=2), pb.PA_ERR_UNSUPPORTED)):
        assert call("pa_kv_decode", decode_args(), pb.make_opts(**o), **big) == code, o
    o = pb.make_opts(partition_size=64)
    n = pb.pa_kv_decode_workspace_size(2, 800, 24, 4, 256, torch.float8_e4m3fn, partition_size=64)
    up = lambda x: -(-x // 256) * 256
    rows = 2 * 24 * 13
    assert n == up(rows * 8) + rows * 256 * 4
    assert call("pa_kv_decode", decode_args(), o, FAKE, n - 1) == pb.PA_ERR_WORKSPACE
    assert call("pa_kv_decode", decode_args(), o, None, n) == pb.PA_ERR_WORKSPACE
    assert call("pa_kv_decode", decode_args(), o, FAKE + 16, n) == pb.PA_ERR_WORKSPACE
    # the weights add the scores of 50 whole blocks
    assert pb.pa_kv_decode_workspace_size(2, 800, 24, 4, 256, torch.float8_e4m3fn, partition_size=64, weights=True) == n + 2 * 24 * 800 * 4
    for bad in ((0, 800, 24, 4, 256), (2, 0, 24, 4, 256), (2, 800, 0, 4, 256), (2, 800, 24, 0, 256), (2, 800, 24, 4, 96)):
        assert pb.pa_kv_decode_workspace_size(*bad, torch.int8) == 0
    assert pb.pa_kv_decode_workspace_size(2, 800, 24, 4, 256, torch.int8, partition_size=24) == 0


def test_decode_workspace_follows_the_plan():
    size = lambda B, L, **kw: pb.pa_kv_decode_workspace_size(B, L, 24, 4, 256, torch.int8, **kw)
    # one CTA or one cluster per (sequence, kv head): nothing to merge; the weights still need the scores, and the sums
    # where another launch adds them
    up = lambda x: -(-x // 256) * 256
    assert size(1, 128) == 0 and size(8, 128) == 0 and size(8, 4000, mode="single") == 0
    assert size(8, 128, weights=True) == 8 * 24 * 128 * 4
    assert size(8, 4000, mode="single", weights=True) == up(8 * 24 * 8) + 8 * 24 * 4000 * 4
    assert size(1, 2048) == 0 and size(8, 512) == 0 and size(2, 4096) == 0
    assert size(8, 512, weights=True) == 8 * 24 * 512 * 4 and size(2, 2048, weights=True) == 2 * 24 * 2048 * 4
    # longer ones, and one sequence with the weights: partials
    assert size(1, 2049) > 0 and size(2, 4097) > 0 and size(8, 512, mode="split") > 0
    assert size(1, 512, weights=True) > 24 * 512 * 4 and size(2, 2049, weights=True) > 2 * 24 * 2064 * 4
    # equal shares: per kv head a slot for every CTA, every warp and every sequence
    one, two = size(8, 100000), size(9, 100000)
    assert 0 < two - one < 24 * 256 * 4 + 24 * 8 + 1024
    assert size(8, 100000) == size(8, 5000)  # whatever the lengths
    # the weights add fp32 scores of whole blocks
    assert size(8, 5000, weights=True) == one + 8 * 24 * 5008 * 4
    assert size(2, 0) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), pb.PA_ERR_INVALID_ARG), (dict(T=-1), pb.PA_ERR_INVALID_ARG), (dict(max_q=0), pb.PA_ERR_INVALID_ARG),
    (dict(max_q=-1), pb.PA_ERR_INVALID_ARG), (dict(mbps=-1), pb.PA_ERR_INVALID_ARG), (dict(mbps=1 << 28), pb.PA_ERR_UNSUPPORTED),
    (dict(k=0), pb.PA_ERR_INVALID_ARG), (dict(v=FAKE + 8), pb.PA_ERR_INVALID_ARG), (dict(ctx=0), pb.PA_ERR_INVALID_ARG),
    (dict(loc=FAKE + 1), pb.PA_ERR_INVALID_ARG), (dict(bt=0), pb.PA_ERR_INVALID_ARG)])
def test_append_refusals(kw, code):
    assert call("pa_kv_append", append_args(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(heads=23), pb.PA_ERR_INVALID_ARG), (dict(heads=36), pb.PA_ERR_UNSUPPORTED), (dict(B=65536), pb.PA_ERR_INVALID_ARG),
    (dict(max_ctx=801), pb.PA_ERR_INVALID_ARG), (dict(max_q=0), pb.PA_ERR_INVALID_ARG), (dict(scale=math.nan), pb.PA_ERR_INVALID_ARG),
    (dict(k=0), pb.PA_ERR_INVALID_ARG), (dict(out=FAKE + 2), pb.PA_ERR_INVALID_ARG), (dict(), pb.PA_ERR_WORKSPACE)])
def test_prefix_refusals(kw, code):
    assert call("pa_kv_prefix", prefix_args(**kw)) == code


def test_prefix_workspace():
    n = pb.pa_kv_prefix_workspace_size(2, 800, 4, 256, torch.int8)
    # K and V in fp16, the copy's table, the factors of INT8's scales
    copy = lambda L: 2 * (2 * -(-L // 16) * 4 * 16 * 256 * 2)
    assert pb.pa_kv_prefix_workspace_size(2, 496, 4, 256, torch.float8_e4m3fn) == copy(496) + 256
    assert pb.pa_kv_prefix_workspace_size(2, 496, 4, 256, torch.int8) == copy(496) + 256 + 2 * 31 * 4 * 8 + 64
    # from 512 tokens on the states of split query tiles: 128 rows of 256 numbers and two for each SM
    states = n - copy(800) - 512 - 2 * 50 * 4 * 8 - 128
    assert states > 0 and states % (128 * 258 * 4) == 0
    assert pb.pa_kv_prefix_workspace_size(2, 800, 4, 256, torch.float8_e4m3fn) == copy(800) + 512 + states
    # (none where the batch has more heads than half the SMs)
    assert pb.pa_kv_prefix_workspace_size(200, 800, 4, 256, torch.float8_e4m3fn) == 100 * copy(800) + 40192
    assert pb.pa_kv_prefix_workspace_size(2, 800, 4, 256, torch.float16) == 0
    assert pb.pa_kv_prefix_workspace_size(2, 0, 4, 256, torch.int8) == 0
    for ws, size in ((FAKE, n - 1), (None, n), (FAKE + 16, n)):
        assert call("pa_kv_prefix", prefix_args(cache(fmt=pb.PA_KV_INT8)), None, ws, size) == pb.PA_ERR_WORKSPACE
    # an fp16 copy whose rows would not fit 32 bits
    big = prefix_args(cache(nb=20000), B=30000, T=30000, mbps=20000, max_ctx=320000)
    assert call("pa_kv_prefix", big, None, FAKE, 1 << 62) == pb.PA_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), pb.PA_ERR_INVALID_ARG), (dict(max_len=801), pb.PA_ERR_INVALID_ARG), (dict(max_keep=161), pb.PA_ERR_INVALID_ARG),
    (dict(sinks=-1), pb.PA_ERR_INVALID_ARG), (dict(recent=-1), pb.PA_ERR_INVALID_ARG), (dict(ws=799), pb.PA_ERR_INVALID_ARG),
    (dict(dws=159), pb.PA_ERR_INVALID_ARG), (dict(w=0), pb.PA_ERR_INVALID_ARG), (dict(kept=0), pb.PA_ERR_INVALID_ARG),
    (dict(new=0), pb.PA_ERR_INVALID_ARG), (dict(keep=FAKE + 2), pb.PA_ERR_INVALID_ARG), (dict(dw=FAKE), pb.PA_ERR_INVALID_ARG),
    (dict(dbt=FAKE), pb.PA_ERR_INVALID_ARG),
    (dict(dst=cache(fmt=pb.PA_KV_INT8)), pb.PA_ERR_INVALID_ARG), (dict(dst=cache(hkv=2)), pb.PA_ERR_INVALID_ARG),
    (dict(dst=cache(D=128)), pb.PA_ERR_INVALID_ARG), (dict(src=cache(nb=0)), pb.PA_ERR_INVALID_ARG)])
def test_evict_refusals(kw, code):
    assert call("pa_kv_evict", evict_args(**kw)) == code


def test_lengths_past_2_to_the_30_are_refused():
    top = 1 << 30
    wide = dict(mbps=1 << 27, stride=1 << 31)
    for n in (top + 1, 2 ** 31 - 1):
        assert call("pa_kv_decode", decode_args(B=1, max_len=n, **wide), None, FAKE, 1 << 62) == pb.PA_ERR_UNSUPPORTED
        assert call("pa_kv_evict", evict_args(mbps=1 << 27, max_len=n, ws=1 << 31)) == pb.PA_ERR_UNSUPPORTED
        assert call("pa_kv_evict", evict_args(dmbps=1 << 27, max_keep=n, dws=1 << 31)) == pb.PA_ERR_UNSUPPORTED
        assert call("pa_kv_append", append_args(T=n, max_q=n)) == pb.PA_ERR_UNSUPPORTED
        assert pb.pa_kv_decode_workspace_size(1, n, 24, 4, 256, torch.int8) == 0
    big = (2 ** 31 - 16)
    assert call("pa_kv_decode", decode_args(), pb.make_opts(partition_size=big), FAKE, 1 << 62) == pb.PA_ERR_UNSUPPORTED
    assert pb.pa_kv_decode_workspace_size(1, 100, 24, 4, 256, torch.int8, partition_size=big) == 0
    # and the largest one is accepted up to its workspace: 24 heads, partitions of 2^30 and of 2^20 tokens
    for part, slots in ((top, 1), (1 << 20, 1 << 10)):
        o = pb.make_opts(partition_size=part)
        n = pb.pa_kv_decode_workspace_size(1, top, 24, 4, 256, torch.int8, partition_size=part)
        assert n == (slots * 24 * (8 + 256 * 4) if slots > 1 else 0)
        if n:
            assert call("pa_kv_decode", decode_args(B=1, max_len=top, **wide), o, FAKE, n - 1) == pb.PA_ERR_WORKSPACE


def test_null_arguments_and_empty_calls():
    for fn in ("pa_kv_append", "pa_kv_evict"):
        assert getattr(pb.lib, fn)(None, None) == pb.PA_ERR_INVALID_ARG
    for fn in ("pa_kv_decode", "pa_kv_prefix"):
        assert getattr(pb.lib, fn)(None, None, None, 0, None) == pb.PA_ERR_INVALID_ARG
    # no sequences or no tokens: nothing to do, nothing looked at
    assert call("pa_kv_append", append_args(B=0, k=0, bt=0)) == pb.PA_OK
    assert call("pa_kv_append", append_args(T=0, k=0)) == pb.PA_OK
    assert call("pa_kv_decode", decode_args(B=0, q=0)) == pb.PA_OK
    assert call("pa_kv_prefix", prefix_args(T=0, q=0)) == pb.PA_OK
    assert call("pa_kv_evict", evict_args(B=0, w=0, kept=0)) == pb.PA_OK


@pytest.mark.skipif(torch.cuda.is_available(), reason="needs a machine without a GPU")
def test_calls_fail_cleanly_without_a_device():
    assert call("pa_kv_append", append_args()) == pb.PA_ERR_CUDA
    assert call("pa_kv_decode", decode_args(), None, FAKE, 1 << 40) == pb.PA_ERR_CUDA
    assert call("pa_kv_prefix", prefix_args(), None, FAKE, 1 << 40) == pb.PA_ERR_CUDA
    assert call("pa_kv_evict", evict_args()) == pb.PA_ERR_CUDA


def test_binding_refuses_cpu_tensors_and_unknown_types():
    k = torch.zeros(2, 1, 16, 64, dtype=torch.int8)
    s = torch.zeros(2, 1)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        pb.pa_kv_append(k, k, s, s, None, None, None, i, i, max_query_len=1)
    with pytest.raises(TypeError):
        pb.pa_kv_append(k.to(torch.uint8), k, s, s, None, None, None, i, i, max_query_len=1)


def test_structs_match_the_header():
    # field names in the header's order, for every struct of the calls
    import re
    text = re.sub(r"/\*.*?\*/", "", open(pb.HEADER_PATH).read(), flags=re.S)
    for name in ("pa_kv_cache", "pa_kv_append_args", "pa_kv_decode_args", "pa_kv_prefix_args", "pa_kv_evict_args"):
        body = re.search(r"typedef struct \{([^{}]*)\} %s;" % name, text).group(1)
        fields = re.findall(r"(\w+)\s*;", body)
        assert fields == [n for n, _ in getattr(pb, name)._fields_], name
    for k in ("F16", "E4M3", "INT8"):
        assert int(re.search(r"PA_KV_%s = (\d)" % k, text).group(1)) == getattr(pb, "PA_KV_" + k)


# ---- the references

def test_scale_reference():
    assert K.scale_of(448.0, "e4m3") == 1.0 and K.scale_of(448.1, "e4m3") == 2.0 and K.scale_of(1.75, "e4m3") == 2.0 ** -8
    assert K.scale_of(127.0, "int8") == 1.0 and K.scale_of(254.0, "int8") == 2.0
    s = K.scale_of(128.0, "int8")
    assert s == math.ceil(128 / 127 * 128) / 128 and K.scale_of(0.0, "int8") == 0.0


def test_rounding_reference_is_torch_rounding():
    # torch's own conversion rounds to nearest even too, below its largest value
    x = torch.cat([torch.linspace(-460, 460, 20001), torch.linspace(-0.05, 0.05, 20001)]).double()
    ref = x.clamp(-448, 448).float().to(torch.float8_e4m3fn).double()
    assert torch.equal(K.round_code(x.float().double(), "e4m3"), ref)


def test_decode_reference_closed_forms():
    c = K.Case([33], 2, 1, 64, "int8", seed=1)
    c.q.zero_()  # equal scores: the mean of V, weight 1 / 33 for each of two heads
    out, _, w, _ = K.decode_reference(c)
    _, v = c.tokens(0)
    assert torch.allclose(out[0, 0], v[0].mean(dim=0), atol=1e-14)
    assert torch.allclose(w[0, 0], torch.full((33,), 2 / 33, dtype=torch.float64), atol=1e-15)


def test_evict_reference_small():
    c = K.Case([6], 1, 1, 64, "f16", seed=1)
    w = torch.tensor([[[5.0, 1.0, 3.0, 3.0, math.nan, 0.0]]])
    assert K.evict_reference(c, w, [3], 0, 0) == [[[0, 2, 3]]]
    assert K.evict_reference(c, w, [3], 0, 1) == [[[0, 2, 5]]]
    assert K.evict_reference(c, w, [3], 2, 1) == [[[0, 1, 5]]]
    assert K.evict_reference(c, w, [1], 2, 3) == [[[5]]]
    assert K.evict_reference(c, w, [9], 2, 3) == [[[0, 1, 2, 3, 4, 5]]]
