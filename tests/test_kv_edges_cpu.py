"""Arguments of the 8-bit cache's calls at the edges of what is allowed, without a GPU."""
import pytest
import torch

from paged_kv_cache_308_gb300 import binding as pb
from test_kv_cpu import FAKE, cache, call, decode_args, evict_args

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="accepted arguments with addresses that no GPU may read")
AWAY = FAKE + (1 << 20)


@pytest.mark.parametrize("kw", [dict(new=FAKE + 4), dict(new=FAKE - 4), dict(new=AWAY + 4, keep=AWAY),
                                dict(new=AWAY - 4, keep=AWAY), dict(new=FAKE, keep=FAKE + 4)])
def test_evict_refuses_new_lengths_that_overlap_the_old(kw):
    # two sequences: eight bytes each; the same array is written in place, one beside it is an array of its own
    assert call("pa_kv_evict", evict_args(**kw)) == pb.PA_ERR_INVALID_ARG


@no_gpu
@pytest.mark.parametrize("kw", [dict(new=FAKE), dict(new=FAKE + 8), dict(new=FAKE - 8), dict(new=AWAY, keep=AWAY),
                                dict(new=AWAY, keep=AWAY + 8)])
def test_evict_takes_new_lengths_in_place_or_apart(kw):
    assert call("pa_kv_evict", evict_args(**kw)) == pb.PA_ERR_CUDA  # (as far as the device)


@no_gpu
@pytest.mark.parametrize("fmt", ["F16", "E4M3", "INT8"])
@pytest.mark.parametrize("opt", [dict(), dict(mode="single"), dict(mode="split"), dict(partition_size=64),
                                 dict(mode="split", partition_size=16)])
@pytest.mark.parametrize("B,hkv", [(1, 4), (2, 4), (5, 1), (300, 8)])
def test_decode_of_empty_sequences_needs_no_workspace(B, hkv, opt, fmt):
    dtype = {"F16": torch.float16, "E4M3": torch.float8_e4m3fn, "INT8": torch.int8}[fmt]
    for weights in (False, True):
        assert pb.pa_kv_decode_workspace_size(B, 0, 2 * hkv, hkv, 64, dtype, weights=weights, **opt) == 0
        a = decode_args(cache(fmt=getattr(pb, "PA_KV_" + fmt), hkv=hkv, D=64), heads=2 * hkv, B=B, max_len=0,
                        w_out=AWAY if weights else 0)
        assert call("pa_kv_decode", a, pb.make_opts(**opt), None, 0) == pb.PA_ERR_CUDA  # (as far as the device)


@no_gpu
@pytest.mark.parametrize("opt", [dict(), dict(mode="single"), dict(mode="split"), dict(partition_size=64)])
@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("B,L", [(1, 1), (1, 128), (1, 5000), (2, 1), (2, 512), (9, 700), (300, 600), (3, 33)])
def test_decode_takes_the_workspace_that_its_size_names(B, L, weights, opt):
    n = pb.pa_kv_decode_workspace_size(B, L, 8, 4, 128, torch.int8, weights=weights, **opt)
    a = decode_args(cache(fmt=pb.PA_KV_INT8, D=128), heads=8, B=B, mbps=400, max_len=L, stride=L, w_out=AWAY if weights else 0)
    assert call("pa_kv_decode", a, pb.make_opts(**opt), FAKE if n else None, n) == pb.PA_ERR_CUDA
    if n:
        assert call("pa_kv_decode", a, pb.make_opts(**opt), FAKE, n - 1) == pb.PA_ERR_WORKSPACE
