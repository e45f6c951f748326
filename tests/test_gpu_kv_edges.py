"""Calls of the 8-bit cache's operators at the edges of what their arguments
allow, on the GPU against the 64-bit references."""
import math

import pytest
import torch

import kv_helpers as K
from test_gpu_kv import DEV, _chunks, check, pb, status

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
