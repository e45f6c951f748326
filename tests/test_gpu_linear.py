"""Linear attention with a decay a kv head on the GPU against the recurrence in float64."""
import math

import pytest
import torch

import step_helpers as S
from paged_kv_cache_308_gb300 import binding as pb

pytestmark = pytest.mark.gpu

SHAPES = [(24, 4, 256), (32, 8, 128), (8, 1, 64), (12, 12, 64), (10, 2, 128), (21, 3, 256), (3, 3, 256), (2, 1, 128)]


def status():
    torch.cuda.synchronize()
    return pb.pa_get_device_status()


def decode(c, **kw):
    B = len(c.new)
    pb.pa_linear_decode(c.out[:B], c.q[:B], c.k[:B], c.v[:B], c.states, c.slots, c.g, c.scale, **kw)


def prefix(c, max_new=None, **kw):
    pb.pa_linear_prefix(c.out, c.q, c.k, c.v, c.states, c.slots, c.g, c.ctx_lens, c.loc, c.scale,
                        max_query_len=max(c.new + [1]) if max_new is None else max_new, **kw)


@pytest.mark.parametrize("heads,hkv,dim", SHAPES)
@pytest.mark.parametrize("B", [1, 5, 70])
def test_decode(heads, hkv, dim, B):
    c = S.LinearCase([1] * B, heads, hkv, dim, seed=B + dim)
    decode(c)
    assert status() == 0
    c.check(c.out, c.states, chunked=False)


@pytest.mark.parametrize("g", [0.0, -1e-6, -0.4999, -0.5, -0.6, -30.0, -1e6, -math.inf])
def test_decode_decays(g):
    c = S.LinearCase([1] * 3, 8, 2, 128, g=[g, -0.1], seed=5)
    decode(c)
    assert status() == 0
    c.check(c.out, c.states, chunked=False)


@pytest.mark.parametrize("heads,hkv,dim", SHAPES)
@pytest.mark.parametrize("new,ctx", [
    ([1], None), ([2], [0]), ([17], None), ([64, 1, 0, 65], [5, 0, 3, 0]), ([127, 128, 129], [0, 7, 0]),
    ([255, 256, 257, 3], None), ([700, 30], [0, 1])])
def test_prefix(heads, hkv, dim, new, ctx):
    c = S.LinearCase(new, heads, hkv, dim, ctx=ctx, seed=sum(new) + dim)
    prefix(c)
    assert status() == 0
    c.check(c.out, c.states)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("g", [0.0, -1e-5, -0.3, -0.7, -6.0, -30.0, -1e6, -math.inf])
def test_prefix_decays(g, dim):
    c = S.LinearCase([300, 520], 4, 2, dim, ctx=[3, 0], g=[g, -0.02], seed=9)
    prefix(c)
    assert status() == 0
    c.check(c.out, c.states)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("size,scale", [(100.0, 1e-7), (1e-3, 1.0), (1e-3, 1e5), (1.0, 0.0), (1.0, -0.3)])
def test_prefix_magnitudes(size, scale, dim):
    """Scores and states beyond fp16's range on either side, and scales that bring the outputs back."""
    c = S.LinearCase([400, 33], 4, 2, dim, ctx=[3, 0], seed=11, size=size, scale=scale)
    prefix(c)
    assert status() == 0
    c.check(c.out, c.states)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prefix_columns_of_unlike_size(dim):
    """Entries of v and of k that differ by a factor of 2^20 between columns."""
    c = S.LinearCase([600], 2, 2, dim, ctx=[4], seed=12)
    col = 2.0 ** -(torch.arange(dim, device="cuda") % 21).float()
    c.v[:600] = (c.v[:600].float() * col).half()
    prefix(c)
    assert status() == 0
    c.check(c.out, c.states)


def test_prefix_long():
    c = S.LinearCase([5000, 2100], 8, 1, 128, ctx=[0, 9], g=[-1e-4], seed=13)
    prefix(c)
    assert status() == 0
    c.check(c.out, c.states)


def test_prefix_bound_above_the_lengths():
    c = S.LinearCase([3, 300, 0], 8, 2, 128, ctx=[0, 9, 2], seed=14)
    prefix(c, max_new=4000)
    assert status() == 0
    c.check(c.out, c.states)


def test_chunks_continue_as_one_prompt():
    """A prompt in three chunks and a token, against the whole."""
    sizes, heads, hkv, dim = [300, 1, 470, 1], 8, 2, 128
    c = S.LinearCase([sum(sizes)], heads, hkv, dim, ctx=[0], seed=15)
    at, states = 0, c.states
    for i, n in enumerate(sizes):
        rows = slice(at, at + n)
        out = torch.empty_like(c.q[rows])
        if i == len(sizes) - 1:
            pb.pa_linear_decode(out, c.q[rows].contiguous(), c.k[rows].contiguous(), c.v[rows].contiguous(), states, c.slots,
                                c.g, c.scale)
        else:
            pb.pa_linear_prefix(out, c.q[rows], c.k[rows], c.v[rows], states, c.slots, c.g,
                                torch.tensor([at], dtype=torch.int32, device="cuda"),
                                torch.tensor([0, n], dtype=torch.int32, device="cuda"), c.scale, max_query_len=n)
        c.out[rows] = out
        at += n
    assert status() == 0
    c.check(c.out, states)


@pytest.mark.parametrize("call,n", [("decode", 1), ("prefix", 1), ("prefix", 300)])
def test_slots_that_are_none_or_bad(call, n):
    c = S.LinearCase([n] * 4, 8, 2, 64, seed=16)
    c.slots[1] = -1
    c.out[n:2 * n] = 7.0
    before = c.before.clone()
    run = decode if call == "decode" else prefix
    run(c)
    assert status() == 0
    assert bool((c.out[n:2 * n] == 7.0).all())
    c.check(c.out, c.states, chunked=n > 1)
    c.states.copy_(before)
    c.out.fill_(7.0)
    c.slots[1] = c.states.shape[0]
    run(c)
    assert status() == pb.PA_DEV_BAD_BLOCK_ID
    assert bool((c.out[n:2 * n] == 7.0).all())
    c.slots[1] = -1
    c.check(c.out, c.states, chunked=n > 1)


@pytest.mark.parametrize("n", [1, 300])
def test_bad_decays_are_reported(n):
    c = S.LinearCase([n] * 2, 8, 2, 64, g=[0.1, -0.1], seed=17)
    prefix(c)
    assert status() == pb.PA_DEV_BAD_DECAY
    c.g[0] = math.nan
    prefix(c)
    assert status() == pb.PA_DEV_BAD_DECAY
    if n == 1:
        decode(c)
        assert status() == pb.PA_DEV_BAD_DECAY


@pytest.mark.parametrize("n", [7, 300])
def test_bad_lengths_skip_their_sequence(n):
    for loc, ctx, good in (([0, n, n + 5, n - 1, 3 * n], None, []), ([0, n, 2 * n, 3 * n + 9, 4 * n], None, [0, 1]),
                           ([0, n, 2 * n, 3 * n, 4 * n], [1, -1, 1, 1], [0, 2, 3])):
        c = S.LinearCase([n] * 4, 8, 2, 64, ctx=[1] * 4, seed=18, pad=2)
        c.loc.copy_(torch.tensor(loc, dtype=torch.int32))
        if ctx:
            c.ctx_lens.copy_(torch.tensor(ctx, dtype=torch.int32))
        prefix(c, max_new=n)
        assert status() == pb.PA_DEV_BAD_SEQ_LEN
        for b in good:
            rows = slice(b * n, (b + 1) * n)
            slot = int(c.slots[b])
            o, s, ob, sb = S.linear(c.q[rows], c.k[rows], c.v[rows], c.before[slot], c.g, c.scale)
            S.check(c.out[rows], o, ob)
            S.check(c.states[slot], s, sb)
        if ctx:
            assert torch.equal(c.states[int(c.slots[1])], c.before[int(c.slots[1])])


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n,at", [(5, 2), (300, 2), (300, 130), (600, 290)])
def test_non_finite_values_reach_only_later_tokens_of_their_column(n, at, dim):
    for bad in (math.nan, math.inf):
        c = S.LinearCase([n, n], 4, 2, dim, seed=19)
        clean = S.LinearCase([n, n], 4, 2, dim, seed=19)
        c.v[at, 1, 3] = bad
        prefix(c)
        clean.v[at, 1, 3] = 0
        prefix(clean)
        assert status() == 0
        touched = torch.zeros_like(c.out, dtype=torch.bool)
        touched[at:n, 2:4, 3] = True
        assert torch.equal(~torch.isfinite(c.out[:2 * n]), touched[:2 * n])
        clean.check(clean.out, clean.states)
        same = ~touched
        assert torch.equal(c.out[same], clean.out[same])
        slot = int(c.slots[0])
        assert not bool(torch.isfinite(c.states[slot, 1, :, 3]).any())
        other = torch.ones_like(c.states, dtype=torch.bool)
        other[slot, 1, :, 3] = False
        assert torch.equal(c.states[other].nan_to_num(nan=-9.0), clean.states[other].nan_to_num(nan=-9.0))


def test_non_finite_query_and_key():
    c = S.LinearCase([300], 4, 2, 64, seed=20)
    c.q[100, 0, 5] = math.inf
    c.k[200, 1, 7] = math.nan
    prefix(c)
    bad = ~torch.isfinite(c.out[:300])
    want = torch.zeros_like(bad)
    want[100, 0] = True
    want[200:, 2:] = True
    assert torch.equal(bad, want)


def test_states_past_32_bits():
    """A pool of more than 2^31 elements: the last slots are where they should be."""
    hkv, dim = 8, 256
    slots = (1 << 31) // (hkv * dim * dim) + 3
    c = S.LinearCase([1, 300], 8, 8, dim, seed=21)
    pool = torch.zeros(slots, hkv, dim, dim, device="cuda")
    at = [slots - 1, slots - 3]
    for b, s in enumerate(at):
        pool[s] = c.before[int(c.slots[b])]
    mine = torch.tensor(at, dtype=torch.int32, device="cuda")
    pb.pa_linear_prefix(c.out, c.q, c.k, c.v, pool, mine, c.g, c.ctx_lens, c.loc, c.scale, max_query_len=300)
    assert status() == 0
    for b, s in enumerate(at):
        c.states[int(c.slots[b])] = pool[s]
    c.check(c.out, c.states)
    assert bool((pool[:at[1]] == 0).all()) and bool((pool[at[1] + 1] == 0).all())


def test_repeats_give_the_same_bits():
    c = S.LinearCase([600, 40], 24, 4, 256, seed=22)
    prefix(c)
    out, states = c.out.clone(), c.states.clone()
    c.states.copy_(c.before)
    prefix(c)
    assert torch.equal(c.out.nan_to_num(), out.nan_to_num()) and torch.equal(c.states.nan_to_num(), states.nan_to_num())


def test_workspace_is_checked():
    c = S.LinearCase([600, 40], 8, 2, 128, seed=23)
    need = pb.pa_linear_prefix_workspace_size(2, c.q.shape[0], 600, 8, 2, 128)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
    if need:
        with pytest.raises(pb.PaDecodeError) as e:
            prefix(c, workspace=ws[:need - 1])
        assert e.value.code == pb.PA_ERR_WORKSPACE
        with pytest.raises(pb.PaDecodeError):
            prefix(c, workspace=ws[16:])
    prefix(c, workspace=ws[:need])
    assert status() == 0 and bool((ws[need:] == 255).all())
    c.check(c.out, c.states)


def test_binding_refusals():
    c = S.LinearCase([3, 2], 8, 2, 128, seed=24)
    with pytest.raises(TypeError):
        pb.pa_linear_decode(c.out, c.q, c.k, c.v, c.states.half(), c.slots, c.g, c.scale)
    with pytest.raises(ValueError):
        pb.pa_linear_decode(c.out, c.q, c.k, c.v, c.states, c.slots, c.g, c.scale)
    with pytest.raises(ValueError):
        pb.pa_linear_prefix(c.out, c.q, c.k[:, :1], c.v, c.states, c.slots, c.g, c.ctx_lens, c.loc, c.scale, max_query_len=3)
    with pytest.raises(ValueError):
        pb.pa_linear_prefix(c.out, c.q, c.k, c.v, c.states.transpose(2, 3), c.slots, c.g, c.ctx_lens, c.loc, c.scale,
                            max_query_len=3)
    with pytest.raises(pb.PaDecodeError):
        pb.pa_linear_prefix(c.out, c.q, c.k, c.v, c.states, c.slots, c.g, c.ctx_lens, c.loc, c.scale, max_query_len=-1)
