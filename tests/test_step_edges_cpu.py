"""What the binding and the C interface of a serving step's calls refuse before anything reaches a GPU."""
import ctypes

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


@pytest.fixture
def as_on_gpu(monkeypatch):
    """Every tensor says that it is on device 0."""
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)


# one token's row for all of them; rows that overlap the next
def spread(x, step, T=5):
    return x.as_strided((T,) + x.shape[1:], (step,) + x.stride()[1:])


@pytest.mark.parametrize("which", ["q", "k", "v"])
@pytest.mark.parametrize("step", [0, 8, 64])
def test_put_refuses_tokens_that_share_memory(reached, as_on_gpu, which, step):
    t = dict(q=rows(5, 4, 64), k=rows(5, 2, 64), v=rows(5, 2, 64))
    t[which] = spread(t[which], step)
    caches = rows(2, 2, 16, 64), rows(2, 2, 16, 64)
    with pytest.raises(ValueError, match=which):
        pb.pa_kv_put(rows(5, 4, 64), rows(5, 2, 64), t["q"], t["k"], t["v"], *caches, ints(5), ints(5), torch.zeros(8, 64))
    assert reached == []


def test_put_takes_rows_of_a_joint_projection_and_single_tokens(reached, as_on_gpu):
    joint = rows(5, 8, 64)
    caches = rows(2, 2, 16, 64), rows(2, 2, 16, 64)
    for T, step in ((5, 512), (1, 0), (1, 8), (0, 512)):
        q, k, v = (spread(joint[:, a:b], step, T) for a, b in ((0, 4), (4, 6), (6, 8)))
        pb.pa_kv_put(rows(T, 4, 64), None, q, k, v, *caches, ints(T), ints(T), torch.zeros(8, 64))
    assert reached == ["pa_kv_put"] * 4


# ---- the C interface: outputs over arrays that a call reads

FAKE = 0x100000  # aligned addresses that no call dereferences
FAR = 1 << 28


def put_code(strides=(0, 0, 0), **over):
    at = {n: FAKE + (i + 1) * FAR for i, n in enumerate(["kc", "vc", "q_out", "k_out", "q", "k", "v", "slots", "pos", "cs"])}
    at.update({n: at[x] + off for n, (x, off) in over.items()})
    cache = pb.pa_kv_cache(at["kc"], at["vc"], 0, 0, 10, 2, 16 * 8, 16, pb.PA_KV_F16)
    a = pb.pa_kv_put_args(cache, at["q_out"], at["k_out"], at["q"], at["k"], at["v"], at["slots"], at["pos"], at["cs"],
                          *strides, 4, 8, 128, 100, 0)
    return pb.lib.pa_kv_put(ctypes.byref(a), None)


@pytest.mark.parametrize("out,size", [("q_out", 4 * 8 * 256), ("k_out", 4 * 2 * 256), ("kc", 10 * 2 * 16 * 256), ("vc", 10 * 2 * 16 * 256)])
@pytest.mark.parametrize("array", ["slots", "pos", "cs"])
def test_put_outputs_over_slots_positions_and_factors(out, size, array):
    assert put_code(**{array: (out, 0)}) == pb.PA_ERR_INVALID_ARG
    assert put_code(**{array: (out, size - 16)}) == pb.PA_ERR_INVALID_ARG
    if array == "cs":
        assert put_code(**{out: (array, 100 * 128 * 4 - 16)}) == pb.PA_ERR_INVALID_ARG


def test_put_strides_past_32_bits():
    for i in range(3):
        for far in (1 << 31, (1 << 62) + 8, (1 << 63) - 8):
            assert put_code(strides=[far if j == i else 0 for j in range(3)]) == pb.PA_ERR_UNSUPPORTED


def linear_code(fn, hkv=4, max_q=5, **over):
    at = {n: FAKE + (i + 1) * FAR for i, n in enumerate(["states", "out", "q", "k", "v", "g", "slots", "ctx", "loc", "ws"])}
    at.update({n: at[x] + off for n, (x, off) in over.items()})
    state = pb.pa_linear_state(at["states"], 5, hkv, 128)
    if fn == "pa_linear_decode":
        a = pb.pa_linear_decode_args(at["out"], at["q"], at["k"], at["v"], state, at["g"], at["slots"], 10, 8, 0.1)
        return pb.lib.pa_linear_decode(ctypes.byref(a), None)
    a = pb.pa_linear_prefix_args(at["out"], at["q"], at["k"], at["v"], state, at["g"], at["slots"], at["ctx"], at["loc"], 3, 10,
                                 max_q, 8, 0.1)
    return pb.lib.pa_linear_prefix(ctypes.byref(a), at["ws"], pb.lib.pa_linear_prefix_workspace_size(3, 10, max_q, 8, hkv, 128), None)


LINEAR_SIZES = dict(out=10 * 8 * 256, states=5 * 4 * 128 * 128 * 4, q=10 * 8 * 256, k=10 * 4 * 256, v=10 * 4 * 256, g=16, slots=12,
                    ctx=12, loc=16)


@pytest.mark.parametrize("out", ["out", "states"])
@pytest.mark.parametrize("array", ["ctx", "loc"])
@pytest.mark.parametrize("max_q", [5, 20])
def test_linear_outputs_over_lengths(out, array, max_q):
    for off in (0, LINEAR_SIZES[out] - 4):
        assert linear_code("pa_linear_prefix", max_q=max_q, **{array: (out, off)}) == pb.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("array", sorted(LINEAR_SIZES))
def test_linear_workspace_over_other_arrays(array):
    need = pb.lib.pa_linear_prefix_workspace_size(3, 10, 20, 8, 4, 128)
    assert need % 256 == 0
    assert linear_code("pa_linear_prefix", max_q=20, **{array: ("ws", 0)}) == pb.PA_ERR_INVALID_ARG
    assert linear_code("pa_linear_prefix", max_q=20, **{array: ("ws", need - 256)}) == pb.PA_ERR_INVALID_ARG
    assert linear_code("pa_linear_prefix", max_q=20, ws=(array, (LINEAR_SIZES[array] - 1) // 256 * 256)) == pb.PA_ERR_INVALID_ARG


def alloc_code(**over):
    at = {n: FAKE + (i + 1) * FAR for i, n in enumerate(["bt", "free", "count", "new_count", "held", "ctx", "q", "loc", "lens",
                                                         "slots", "pos", "new_held"])}
    at.update({n: (at[x] if x else 0) + off for n, (x, off) in over.items()})
    new_held = at.pop("new_held")
    a = pb.pa_kv_alloc_args(*at.values(), 100, 4, 10, 8, 16, new_held)
    return pb.lib.pa_kv_alloc(ctypes.byref(a), None)


@pytest.mark.parametrize("array,size", [("bt", 128), ("free", 400), ("count", 4), ("new_count", 4), ("ctx", 16), ("q", 16),
                                        ("loc", 20), ("lens", 16), ("slots", 40), ("pos", 40), ("held", 16)])
def test_new_held_lens_over_other_arrays(array, size):
    if array != "held":
        assert alloc_code(new_held=(array, 0)) == pb.PA_ERR_INVALID_ARG
    assert alloc_code(new_held=(array, size - 4)) == pb.PA_ERR_INVALID_ARG
    assert alloc_code(new_held=(array, -12)) == pb.PA_ERR_INVALID_ARG
    assert alloc_code(new_held=("new_held", 2)) == pb.PA_ERR_INVALID_ARG
    # without held_lens, the context lengths are no place for it either
    assert alloc_code(held=(None, 0), new_held=("ctx", 0)) == pb.PA_ERR_INVALID_ARG
