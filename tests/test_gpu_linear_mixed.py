"""Linear attention over batches of unlike lengths, streams, graphs, workspaces and alignments."""
import math
import random

import pytest
import torch

import step_helpers as S
from paged_kv_cache_308_gb300 import binding as pb

pytestmark = pytest.mark.gpu


def status():
    torch.cuda.synchronize()
    return pb.pa_get_device_status()


def prefix(c, max_new=None, **kw):
    pb.pa_linear_prefix(c.out, c.q, c.k, c.v, c.states, c.slots, c.g, c.ctx_lens, c.loc, c.scale,
                        max_query_len=max(c.new + [1]) if max_new is None else max_new, **kw)


@pytest.mark.parametrize("heads,hkv,dim", [(24, 4, 256), (32, 8, 128), (12, 12, 64), (7, 1, 64)])
def test_single_tokens_next_to_chunks(heads, hkv, dim):
    """A serving step: most sequences bring a token, some a chunk, one nothing; lengths around where the two forms meet."""
    new = [1] * 9 + [300, 0, 1, 9, 10, 14, 15, 24, 25, 1, 64, 513, 1]
    c = S.LinearCase(new, heads, hkv, dim, ctx=[(i * 7) % 3 for i in range(len(new))], seed=31)
    prefix(c)
    assert status() == 0
    c.check(c.out, c.states)


@pytest.mark.parametrize("seed", range(12))
def test_random_batches(seed):
    rng = random.Random(seed)
    heads, hkv, dim = rng.choice([(24, 4, 256), (32, 8, 128), (8, 1, 64), (12, 12, 64), (10, 2, 128), (21, 3, 256), (5, 1, 128)])
    new = [rng.choice([0, 1, 2, 9, 24, 63, 64, 65, 128, 200, 255, 256, 257, 384, 385, rng.randint(1, 900)])
           for _ in range(rng.choice([1, 2, 5, 33]))]
    if not sum(new):
        new[0] = 77
    g = [-rng.choice([0.0, 1e-3, 0.05, 1.0, 20.0]) for _ in range(hkv)]
    c = S.LinearCase(new, heads, hkv, dim, ctx=[rng.choice([0, 5]) for _ in new], g=g, seed=seed + 100,
                     size=rng.choice([0.1, 1.0, 10.0]), pad=rng.choice([0, 1, 200]))
    prefix(c, max_new=max(new) + rng.choice([0, 0, 1000]))
    assert status() == 0
    c.check(c.out, c.states)


def test_many_sequences():
    """More sequences than a round of the search for a block's has lanes, twice over."""
    rng = random.Random(3)
    new = [rng.choice([0, 1, 30, 40]) for _ in range(1500)]
    c = S.LinearCase(new, 1, 1, 64, ctx=[1] * 1500, g=[-0.01], seed=32)
    prefix(c)
    assert status() == 0
    picked = [i for i, n in enumerate(new) if n][::37]
    loc = c.loc.tolist()
    for b in picked:
        rows, slot = slice(loc[b], loc[b + 1]), int(c.slots[b])
        o, s, ob, sb = S.linear(c.q[rows], c.k[rows], c.v[rows], c.before[slot], c.g, c.scale)
        S.check(c.out[rows], o, ob, f"sequence {b}")
        S.check(c.states[slot], s, sb, f"state {b}")
    assert bool((c.out[loc[-1]:] == 7.0).all())


def test_more_units_than_the_device_holds_with_every_kind_of_tile():
    c = S.LinearCase([1300, 129, 700, 255, 1025], 16, 4, 64, ctx=[0, 3, 0, 1, 1], seed=33)
    prefix(c)
    assert status() == 0
    c.check(c.out, c.states)


@pytest.mark.parametrize("call", ["decode", "prefix"])
def test_another_stream(call):
    c = S.LinearCase([1] * 3 if call == "decode" else [300, 1, 20], 8, 2, 128, seed=34)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    if call == "decode":
        pb.pa_linear_decode(c.out[:3], c.q[:3], c.k[:3], c.v[:3], c.states, c.slots, c.g, c.scale, s)
    else:
        prefix(c, stream=s)
    s.synchronize()
    c.check(c.out, c.states, chunked=call == "prefix")


def test_two_streams_at_once():
    a, b = (S.LinearCase([600, 30], 24, 4, 256, seed=35 + i) for i in range(2))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for c, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                c.states.copy_(c.before)
                prefix(c)
    torch.cuda.synchronize()
    for c in (a, b):
        c.check(c.out, c.states)


@pytest.mark.parametrize("new", [[1, 1], [5, 9], [300, 1, 64]])
def test_captured_and_replayed(new):
    """Calls in a graph, replayed with other inputs, lengths and slots; two graphs have a workspace each."""
    c = S.LinearCase(new, 8, 2, 128, seed=37)
    d = S.LinearCase(new, 8, 2, 128, ctx=[0] * len(new), seed=38)
    need = pb.pa_linear_prefix_workspace_size(len(new), c.q.shape[0], 400, 8, 2, 128)
    for case in (c, d):
        prefix(case, max_new=400, workspace=torch.empty(max(need, 1), dtype=torch.uint8, device="cuda"))
    graphs = []
    for case in (c, d):
        ws = torch.full((max(need, 1),), 0xab, dtype=torch.uint8, device="cuda")
        case.out.fill_(7.0)
        case.states.copy_(case.before)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            prefix(case, max_new=400, workspace=ws)
        graphs.append((g, ws))
    for g, _ in graphs:
        g.replay()
    assert status() == 0
    for case in (c, d):
        case.check(case.out, case.states)
    # other contents in the same tensors
    e = S.LinearCase(new, 8, 2, 128, ctx=[0] * len(new), seed=39)
    for x, y in ((c.q, e.q), (c.k, e.k), (c.v, e.v), (c.states, e.before), (c.slots, e.slots), (c.ctx_lens, e.ctx_lens)):
        x.copy_(y)
    c.out.fill_(7.0)
    graphs[0][0].replay()
    assert status() == 0
    e.check(c.out, c.states)


@pytest.mark.parametrize("new", [[300, 20], [3]])
def test_tensors_off_by_16_bytes(new):
    c = S.LinearCase(new, 8, 2, 64, seed=40)
    for name in ("out", "q", "k", "v", "states"):
        x = getattr(c, name)
        extra = 16 // x.element_size()
        y = torch.empty(x.numel() + extra, dtype=x.dtype, device="cuda")[extra:].view(x.shape)
        y.copy_(x)
        setattr(c, name, y)
    prefix(c)
    assert status() == 0
    c.check(c.out, c.states)


def test_no_sequence_and_no_token():
    c = S.LinearCase([0, 0], 8, 2, 64, ctx=[3, 0], seed=41)
    prefix(c, max_new=500)
    assert status() == 0
    c.check(c.out, c.states)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_infinite_states_and_zero_inputs(dim):
    """A state with an infinity spoils its column of later outputs, and nothing else; zeros stay zeros."""
    c = S.LinearCase([300, 40], 2, 2, dim, seed=42)
    c.states[int(c.slots[0]), 1, 4, 6] = math.inf
    c.v[300:340] = 0
    c.k[300:340] = 0
    c.q[300:340] = 0
    before = c.states.clone()
    prefix(c)
    bad = ~torch.isfinite(c.out[:340])
    want = torch.zeros_like(bad)
    want[:300, 1, 6] = True
    assert not bool((bad & ~want).any())
    assert bool(bad[0, 1, 6]) and bool((c.out[300:340] == 0).all())
    slot = int(c.slots[1])
    whole = torch.exp(c.g.double() * 40)[:, None, None]
    S.check(c.states[slot], before[slot].double() * whole, before[slot].double().abs() * whole * 2.0 ** -20)


@pytest.mark.parametrize("n", [12, 300])
def test_values_behind_the_last_token_are_not_read(n):
    """NaN and infinities in the rows of the next sequence and in rows of padding."""
    for dim in (64, 128, 256):
        c = S.LinearCase([n, n + 1], 2, 2, dim, seed=43, pad=300)
        c.q[n:2 * n + 1] = math.inf
        c.k[n:2 * n + 1] = math.nan
        c.v[n:2 * n + 1] = math.inf
        prefix(c)
        slot = int(c.slots[0])
        o, s, ob, sb = S.linear(c.q[:n], c.k[:n], c.v[:n], c.before[slot], c.g, c.scale)
        S.check(c.out[:n], o, ob)
        S.check(c.states[slot], s, sb)
        assert bool((c.out[2 * n + 1:] == 7.0).all())


@pytest.mark.parametrize("n", [1, 3, 24, 25, 130])
def test_one_sequence_far_below_the_bound(n):
    for dim in (64, 128, 256):
        c = S.LinearCase([n], 4, 2, dim, seed=44 + n)
        prefix(c, max_new=5000)
        assert status() == 0
        c.check(c.out, c.states)


@pytest.mark.parametrize("heads,hkv,dim", [(24, 4, 256), (32, 8, 128), (12, 12, 64)])
def test_blocks_of_one_token_in_their_second_half_repeat(heads, hkv, dim):
    """Rows that do next to nothing in a block's first step run ahead of the products; the outputs stay the same."""
    c = S.LinearCase([129, 385, 128, 131, 257] * 6, heads, hkv, dim, ctx=[0, 5, 0, 0, 9] * 6, seed=dim)
    states = c.states.clone()
    first = None
    for _ in range(6):
        c.states.copy_(states)
        prefix(c)
        assert status() == 0
        if first is None:
            c.check(c.out, c.states)
            first = c.out.clone(), c.states.clone()
        assert torch.equal(c.out, first[0])
        assert torch.equal(c.states.nan_to_num(nan=-9.0), first[1].nan_to_num(nan=-9.0))
