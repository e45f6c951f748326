"""What the binding and the C interface of a serving step's calls refuse before anything reaches a GPU."""
import pytest
import torch

from paged_kv_cache_308_gb300 import binding as pb


@pytest.fixture
def reached(monkeypatch):
    """The names of the library calls that were reached; none is made."""
    names = []
    monkeypatch.setattr(pb, "_call", lambda name, *a: names.append(name))
    return names


def ints(n):
    return torch.zeros(n, dtype=torch.int32)


def rows(*shape):
    return torch.zeros(shape, dtype=torch.float16)


def test_cpu_tensors_are_refused(reached):
    q, k, states, g = rows(3, 4, 64), rows(3, 2, 64), torch.zeros(3, 2, 64, 64), torch.zeros(2)
    with pytest.raises(ValueError, match="block_tables"):
        pb.pa_kv_alloc(ints((2, 4)), ints(8), ints(1), ints(2), ints(2), ints(3), ints(2), ints(3), ints(3))
    with pytest.raises(ValueError, match="q must be"):
        pb.pa_kv_put(q, k, q, k, None, None, None, None, ints(3), torch.zeros(8, 64))
    with pytest.raises(ValueError, match="q must be"):
        pb.pa_kv_put(q, k, q, k, k, rows(2, 2, 16, 64), rows(2, 2, 16, 64), ints(3), ints(3), torch.zeros(8, 64))
    with pytest.raises(ValueError, match="q must be"):
        pb.pa_linear_decode(q, q, k, k, states, ints(3), g, 1.0)
    with pytest.raises(ValueError, match="q must be"):
        pb.pa_linear_prefix(q, q, k, k, states, ints(1), g, ints(1), ints(2), 1.0, max_query_len=3)
    assert reached == []
