"""Linear attention where decays, zeros and infinities leave little or nothing of a token: against the recurrence in
float64."""
import math

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


def check_out(c):
    """Every sequence's outputs against their reference."""
    loc = c.loc.tolist()
    for b in range(len(c.new)):
        rows, slot = slice(loc[b], loc[b + 1]), int(c.slots[b])
        s0 = c.before[slot] if c.ctx[b] > 0 else torch.zeros_like(c.before[slot])
        o, _, ob, _ = S.linear(c.q[rows], c.k[rows], c.v[rows], s0, c.g, c.scale)
        got = c.out[rows]
        # Half of fp16's last step beyond its largest value is 65520: what is within its bound of o and past that
        # on either side rounds to the infinity of that side (o itself may have the other sign, where the bound of a
        # difference of large products spans both).
        rounded = (got == math.inf) & (o + ob >= 65520.0) | (got == -math.inf) & (o - ob <= -65520.0)
        S.check(torch.where(rounded, 0.0, got), torch.where(rounded, 0.0, o), ob, f"sequence {b} out")


# Keys that are 0 from some token on: the rows behind have scores of 0 next to them and a largest one that falls by
# the decay down to 2^-126 and below, in a row's own 128 keys (g up to -0.7) and in those before (-0.5, -0.36).
# A scale of 2^96 brings what is 2^-112 into fp16; what is below 2^-126, which 32 bits may drop, stays below half of
# its smallest step.
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("g", [-6.0, -3.0, -1.0, -0.7, -0.5, -0.36])
@pytest.mark.parametrize("scale", [0.1, 2.0 ** 96])
def test_zero_keys_behind_others(g, dim, scale):
    new = [256, 250, 256, 250, 256, 130]
    c = S.LinearCase(new, 4, 2, dim, ctx=[0, 0, 0, 3, 3, 3], g=[g, g / 2], seed=51, scale=scale)
    loc = c.loc.tolist()
    for b, kept in enumerate([1, 70, 140, 1, 70, 2]):
        c.k[loc[b] + kept:loc[b + 1]] = 0
    prefix(c)
    assert status() == 0
    check_out(c)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("g", [-6.0, -1.0, -0.36])
def test_runs_of_zero_keys_between_others(g, dim):
    """Masked tokens, in runs that end and start anywhere, over several blocks."""
    c = S.LinearCase([700, 300], 4, 2, dim, ctx=[0, 3], g=[g, -0.01], seed=52)
    runs = [(0, 5), (9, 130), (140, 255), (258, 400), (401, 690), (700, 705), (710, 996)]
    for lo, hi in runs:
        c.k[lo:hi] = 0
    prefix(c)
    assert status() == 0
    check_out(c)


def linear_without(c, b, row, col):
    """Reference of sequence b whose state, of kv head 1, has a 0 at (row, col)."""
    loc, slot = c.loc.tolist(), int(c.slots[b])
    s0 = c.before[slot].clone()
    s0[1, row, col] = 0
    rows = slice(loc[b], loc[b + 1])
    return S.linear(c.q[rows], c.k[rows], c.v[rows], s0, c.g, c.scale, chunked=False)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("g", [0.0, -1e-9, -1e-6, -0.3, -0.4999, -0.5, -0.7, -30.0, -100.0])
@pytest.mark.parametrize("call,n", [("decode", 1), ("prefix", 1), ("prefix", 5)])
def test_infinite_states_stay_infinite_token_by_token(call, n, g, dim):
    c = S.LinearCase([n, n], 4, 2, dim, g=[-0.2, g], seed=53)
    row, col = 5, dim - 2
    for b, x in enumerate((math.inf, -math.inf)):
        c.states[int(c.slots[b]), 1, row, col] = x
    c.before = c.states.clone()
    if call == "decode":
        pb.pa_linear_decode(c.out[:2], c.q[:2], c.k[:2], c.v[:2], c.states, c.slots, c.g, c.scale)
    else:
        prefix(c)
    assert status() == 0
    for b, x in enumerate((math.inf, -math.inf)):
        o, s, ob, sb = linear_without(c, b, row, col)
        got, state = c.out[b * n:(b + 1) * n].clone(), c.states[int(c.slots[b])].clone()
        assert float(state[1, row, col]) == x
        want = torch.sign(c.q[b * n:(b + 1) * n, 2:, row].float()) * x
        assert torch.equal(got[:, 2:, col].float(), want)
        got[:, 2:, col], state[1, row, col] = 0, 0
        o[:, 2:, col], s[1, row, col] = 0, 0
        S.check(got, o, ob, "out")
        S.check(state, s, sb, "state")


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("g", [0.0, -1e-9, -1e-6, -0.01, -0.2])
def test_infinite_states_stay_infinite_in_chunks(g, dim):
    c = S.LinearCase([300, 300], 4, 2, dim, g=[-0.2, g], seed=54)
    row, col = 5, dim - 2
    for b, x in enumerate((math.inf, -math.inf)):
        c.states[int(c.slots[b]), 1, row, col] = x
    c.before = c.states.clone()
    prefix(c)
    assert status() == 0
    for b, x in enumerate((math.inf, -math.inf)):
        _, s, _, sb = linear_without(c, b, row, col)
        state = c.states[int(c.slots[b])].clone()
        assert float(state[1, row, col]) == x
        state[1, row, col] = s[1, row, col] = 0
        S.check(state, s, sb, "state")
        bad = ~torch.isfinite(c.out[b * 300:(b + 1) * 300])
        assert bool(bad[:, 2:, col].all())
        bad[:, 2:, col] = False
        assert not bool(bad.any())


# What tokens leave in the state does not depend on v of later tokens whose keys are 0, however small it has become
# by then (2^-133 for 256 tokens of -0.36).
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("g", [-6.0, -1.0, -0.36, -0.1])
def test_states_behind_zero_keys(g, dim):
    new = [256, 250, 40, 700, 130, 300]
    c = S.LinearCase(new, 4, 2, dim, ctx=[0, 3, 0, 0, 3, 0], g=[g, g / 2], seed=55)
    loc = c.loc.tolist()
    for b, (lo, hi) in enumerate([(1, 256), (70, 250), (3, 40), (280, 700), (5, 66), (256, 300)]):
        c.k[loc[b] + lo:loc[b] + hi] = 0
        if dim == 256:  # a half of the keys only
            c.k[loc[b] + lo - 1, 0, :128] = 0
    c.k[loc[3] + 600, 1, dim - 1] = -0.0
    prefix(c)
    assert status() == 0
    for b in range(len(new)):
        rows, slot = slice(loc[b], loc[b + 1]), int(c.slots[b])
        s0 = c.before[slot] if c.ctx[b] > 0 else torch.zeros_like(c.before[slot])
        _, s, _, sb = S.linear(c.q[rows], c.k[rows], c.v[rows], s0, c.g, c.scale)
        # Decayed values of v below 2^-110 become two halves after times 2^118, the largest factor that later
        # values up to 65504 can take back in one step: half of the second half's last step, 2^-24, is then 2^-143
        # for each |k|.  (Seen in states of 2^-130 only.)
        sb = sb + 2.0 ** -143 * c.k[rows].double().abs().sum(dim=0)[:, :, None]
        S.check(c.states[slot], s, sb, f"sequence {b} state")


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_non_finite_values_of_zero_keys(bad, dim):
    """0 times what is not a number is none: as for other keys, its column's state and later outputs."""
    c = S.LinearCase([300], 4, 2, dim, seed=56)
    c.k[20:200] = 0
    c.v[100, 1, 3] = bad
    prefix(c)
    assert status() == 0
    slot = int(c.slots[0])
    assert bool(c.states[slot, 1, :, 3].isnan().all())
    want = torch.zeros_like(c.out[:300], dtype=torch.bool)
    want[100:, 2:, 3] = True
    assert torch.equal(~torch.isfinite(c.out[:300]), want)
    c.states[slot, 1, :, 3] = 0
    assert bool(torch.isfinite(c.states[slot]).all())


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("ratio", [20, 24, 28, 30])
def test_columns_far_below_the_states_largest(ratio, dim):
    """Columns of v 2^-ratio of the others: their outputs are as exact as their own size, but for what the rounding of
    the state before a block leaves, 2^-33 of the state's largest entry for each |q|."""
    n, block = 700, 256
    c = S.LinearCase([n], 2, 2, dim, ctx=[4], g=[-0.004, -0.05], seed=57)
    col = torch.where(torch.arange(dim, device="cuda") % 2 == 0, 2.0 ** 10, 2.0 ** (10 - ratio))
    c.v[:n] = (c.v[:n].float() * col).half()
    slot = int(c.slots[0])
    c.states[slot] *= col
    c.before = c.states.clone()
    prefix(c)
    assert status() == 0
    q, k, v, g = (x.double() for x in (c.q[:n], c.k[:n], c.v[:n], c.g))
    for h in range(2):
        # of the state's largest entry before each block: the kernel's bound sums up the largest entries of the blocks'
        # sums, and rounds it up a little each time
        state, most = c.before[slot, h].double(), float(c.before[slot, h].abs().max())
        for lo in range(0, n, block):
            rows = slice(lo, min(n, lo + block))
            count = rows.stop - lo
            t = torch.arange(count, device="cuda", dtype=torch.float64)
            one = S.linear(c.q[rows, h:h + 1], c.k[rows, h:h + 1], c.v[rows, h:h + 1], state[None], c.g[h:h + 1], c.scale,
                           chunked=False)
            own = S.linear(c.q[rows, h:h + 1], c.k[rows, h:h + 1], c.v[rows, h:h + 1], torch.zeros_like(state)[None], c.g[h:h + 1],
                           c.scale, chunked=False)
            decay = torch.exp(g[h] * (t + 1))[:, None]
            # one rounding of each score and of each entry of the state, half a step each
            p = (q[rows, h] @ k[rows, h].T).abs() * torch.exp(g[h] * (t[:, None] - t).clamp(min=0)) * (t[:, None] >= t)
            lost = S.H16 * (1 + 2.0 ** -10) * (p @ v[rows, h].abs() + q[rows, h].abs() @ state.abs() * decay)
            # a row's scores below fp16's normals, of a largest that is brought to 2^-4 or more
            lost += 2.0 ** -21 * p.amax(dim=1, keepdim=True) * v[rows, h].abs().sum(dim=0)
            lost += 2.0 ** -33 * 1.01 * most * decay * q[rows, h].abs().sum(dim=1, keepdim=True)
            S.check(c.out[rows, h], one[0][:, 0], one[2][:, 0] + c.scale * lost, f"head {h} block {lo}")
            state = one[1][0]
            most = most * float(torch.exp(g[h] * count)) + float(own[1].abs().max())


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("small", ["k", "v"])
def test_states_of_subnormal_inputs(small, dim):
    """Keys, or values, that are subnormal numbers of fp16, next to others that are not."""
    c = S.LinearCase([300, 40], 4, 2, dim, ctx=[0, 0], g=[-1.0, -0.05], seed=58)
    x = c.k if small == "k" else c.v
    for lo, hi in ((100, 290), (305, 340)):
        x[lo:hi] = (x[lo:hi].float() * 2.0 ** -20).half()
    prefix(c)
    assert status() == 0
    loc = c.loc.tolist()
    for b in range(2):
        rows, slot = slice(loc[b], loc[b + 1]), int(c.slots[b])
        o, s, ob, sb = S.linear(c.q[rows], c.k[rows], c.v[rows], torch.zeros_like(c.before[slot]), c.g, c.scale)
        k, v = c.k[rows].double().abs(), c.v[rows].double().abs()
        left = torch.exp(c.g.double() * torch.arange(c.new[b] - 1, -1, -1, device="cuda")[:, None])
        most = (v * left[:, :, None]).amax(dim=0)[:, None]
        # the header's bounds: each product, and of the column's largest decayed v 2^-33 of |k| or 2^-37
        sb = sb + 2.0 ** -33 * most * k.sum(dim=0)[:, :, None] + 2.0 ** -37 * most
        S.check(c.states[slot], s, sb, f"sequence {b} state")
        # a row's scores to 2^-21 of its largest (256 keys at most)
        q = c.q[rows].double()
        for j in range(4):
            p = (q[:, j] @ c.k[rows, j // 2].double().T).abs()
            t = torch.arange(c.new[b], device="cuda", dtype=torch.float64)
            p = p * torch.exp(c.g[j // 2].double() * (t[:, None] - t).clamp(min=0)) * (t[:, None] >= t)
            ob[:, j] += c.scale * 2.0 ** -21 * p.amax(dim=1, keepdim=True) * v[:, j // 2].sum(dim=0)
        S.check(c.out[rows], o, ob, f"sequence {b} out")


@pytest.mark.parametrize("g", [0.0, -0.5, -0.7, -3.0, -40.0, -80.0])
def test_decays_are_one_rounding(g):
    """Behind a key of 0 a state is its product with exp(g), which an entry of 1 shows, rounded once."""
    c = S.LinearCase([1, 1], 4, 2, 128, g=[g, g], seed=59)
    c.k[:2] = 0
    c.states[c.slots.long(), :, 0, 0] = 1.0
    c.before = c.states.clone()
    pb.pa_linear_decode(c.out[:2], c.q[:2], c.k[:2], c.v[:2], c.states, c.slots, c.g, c.scale)
    assert status() == 0
    got, before = c.states[c.slots.long()], c.before[c.slots.long()]
    factor = got[0, 0, 0, 0]
    assert abs(float(factor) - math.exp(g)) <= 2.0 ** -22 * math.exp(g)
    if g > -59:
        assert torch.equal(got, before * factor)
    else:
        # 2^-64 of exp(-80), which keeps an infinite entry one, is less than the smallest number, 2^-149, that is added
        # in its place, times the entry; that product and the sum are rounded, the sum by half a unit, and each by half
        # of 2^-149 where it is subnormal
        exact = before.double() * float(factor)
        bound = before.double().abs() * 2.0 ** -149 + exact.abs() * 2.0 ** -24 + 2.0 ** -149
        assert bool(((got.double() - exact).abs() <= bound).all())


@pytest.mark.parametrize("g", [-88.0, -90.0, -97.0, -100.0])
def test_decays_below_the_normal_numbers(g):
    """exp(g) is then a number of units of 2^-149, off by half of one and as much of the function's own error."""
    c = S.LinearCase([1, 1], 4, 2, 64, g=[g, g], seed=60)
    c.k[:2] = 0
    c.states[c.slots.long(), :, 0, 0] = 1.0
    c.states[c.slots.long(), :, 0, 1] = 2.0 ** 20
    pb.pa_linear_decode(c.out[:2], c.q[:2], c.k[:2], c.v[:2], c.states, c.slots, c.g, c.scale)
    assert status() == 0
    got = c.states[c.slots.long()].double() * 2.0 ** 149
    for col, size in ((0, 1.0), (1, 2.0 ** 20)):
        assert bool(((got[:, :, 0, col] - math.exp(g) * 2.0 ** 149 * size).abs() <= size).all())
