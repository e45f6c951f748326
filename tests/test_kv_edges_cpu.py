"""Arguments of the 8-bit cache's calls at the edges of what is allowed, without a GPU."""
import pytest
import torch

from paged_kv_cache_308_gb300 import binding as pb
from test_kv_cpu import FAKE, call, evict_args

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
