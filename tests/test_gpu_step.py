"""Block allocation and rotary put on the GPU against their references."""
import math
import random

import pytest
import torch

import step_helpers as S
from paged_kv_cache_308_gb300 import binding as pb

pytestmark = pytest.mark.gpu


def ints(x, device="cuda"):
    return torch.tensor(x, dtype=torch.int32, device=device)


def status():
    torch.cuda.synchronize()
    return pb.pa_get_device_status()


class Step:
    """A pool whose sequences hold `held` tokens, the other blocks free."""

    def __init__(self, held, ctx, new, seed=0, extra=8, cols=0, pad=3, room=0):
        rng = random.Random(seed)
        self.held, self.ctx, self.new = list(held), list(ctx), list(new)
        need = [S.blocks(h) for h in held]
        most = max([1, cols] + [max(S.blocks(c + q), n) for c, q, n in zip(ctx, new, need)])
        take = sum(max(0, S.blocks(c + q) - n) for c, q, n in zip(ctx, new, need))
        total = sum(need) + max(0, take + extra) + room
        ids = list(range(total))
        rng.shuffle(ids)
        self.rows, at = [], 0
        for n in need:
            self.rows.append(ids[at:at + n] + [-1] * (most - n))
            at += n
        self.count = total - at - room
        self.stack = ids[at:at + self.count] + [-1] * (total - self.count)
        self.tokens = sum(new) + pad
        self.tables, self.free, self.free_count = ints(self.rows).view(len(held), most), ints(self.stack), ints([self.count])
        self.loc, self.lens = ints([-5] * (len(held) + 1)), ints([-5] * len(held))
        self.slots, self.positions = ints([-5] * self.tokens), ints([-5] * self.tokens)
        self.args = [ints(self.ctx), ints(self.new)]
        self.held_t = ints(self.held)

    def run(self, **kw):
        if "held_lens" not in kw:
            kw["held_lens"] = self.held_t
        pb.pa_kv_alloc(self.tables, self.free, self.free_count, *self.args, self.loc, self.lens, self.slots, self.positions,
                       **kw)
        return self

    def check(self):
        want, short = S.alloc(self.rows, self.stack, self.count, self.held, self.ctx, self.new, self.tokens)
        assert status() == (pb.PA_DEV_NO_BLOCKS if short else 0)
        got = dict(tables=self.tables.tolist(), free=self.free.tolist(), count=self.free_count.item(), loc=self.loc.tolist(),
                   lens=self.lens.tolist(), slots=self.slots.tolist(), positions=self.positions.tolist())
        for key in want:
            assert got[key] == want[key], key


@pytest.mark.parametrize("held,ctx,new", [
    ([], [], []), ([0], [0], [0]), ([0], [0], [1]), ([15], [15], [1]), ([16], [16], [1]), ([17], [16], [0]),
    ([17], [17], [0]), ([300], [0], [0]), ([0], [0], [300]), ([300], [300], [5000]), ([100], [3], [13]), ([100], [3], [14]),
    ([31, 40, 0, 16], [31, 0, 0, 16], [1, 0, 33, 1]), ([500, 500], [0, 500], [0, 700]),
    ([64] * 40, [64] * 40, [1] * 40), ([0, 0, 0], [0, 0, 0], [0, 5, 0])])
def test_alloc(held, ctx, new):
    Step(held, ctx, new).run().check()


@pytest.mark.parametrize("seqs,top,chunk,seed", [(1, 100, 20000, 1), (7, 300, 40, 2), (64, 2000, 1, 3), (513, 400, 70, 4),
                                                 (3000, 60, 9, 5), (65535, 40, 2, 6)])
def test_alloc_batches(seqs, top, chunk, seed):
    rng = random.Random(seed)
    held, ctx, new = [], [], []
    for _ in range(seqs):
        kind = rng.random()
        h = rng.randint(0, top)
        c, q = h, rng.randint(0, chunk)
        if kind < 0.1:
            c, q = 0, 0
        elif kind < 0.2:
            h = c = 0
        elif kind < 0.3:
            c = rng.randint(0, h)
        held.append(h), ctx.append(c), new.append(q)
    Step(held, ctx, new, seed).run().check()


# one and eight blocks of a cluster, tokens placed by it and by a launch of their own; blocks run out or not
@pytest.mark.parametrize("short", [False, True])
@pytest.mark.parametrize("seqs,top,chunk", [(64, 500, 60), (64, 500, 70), (65, 2000, 1), (100, 300, 200), (300, 300, 200),
                                            (2048, 100, 4), (2049, 100, 4)])
def test_alloc_batches_of_every_path(seqs, top, chunk, short):
    rng = random.Random(seqs + chunk)
    held = [rng.randint(0, top) for _ in range(seqs)]
    new = [rng.randint(0, chunk) for _ in range(seqs)]
    ctx = [0 if rng.random() < 0.1 else h for h in held]
    taken = sum(max(0, S.blocks(c + q) - S.blocks(h)) for h, c, q in zip(held, ctx, new))
    back = sum(max(0, S.blocks(h) - S.blocks(c + q)) for h, c, q in zip(held, ctx, new))
    Step(held, ctx, new, seqs, extra=-back - taken // 3 if short else 8).run().check()


@pytest.mark.parametrize("seqs", [6, 100])
@pytest.mark.parametrize("more", [100, 20000])
def test_alloc_bad_lengths_next_to_many_tokens(seqs, more):
    held = [20] * (seqs - 1) + [0]
    new = [1] * (seqs - 1) + [more]
    for h, c, q in [(-1, 0, 1), (16, 17, 1), (20, 20, -3), (20, -5, 5), (20, -5, 9), (1 << 30, 1 << 30, 1)]:
        a = Step(held, held, new)
        tables = a.tables.clone()
        a.held_t[2], a.args[0][2], a.args[1][2] = h, c, q
        a.slots, a.positions = ints([-5] * (sum(new) + 30)), ints([-5] * (sum(new) + 30))
        a.run()
        assert status() == pb.PA_DEV_BAD_SEQ_LEN
        lens, loc, slots = a.lens.tolist(), a.loc.tolist(), a.slots.tolist()
        assert lens == [21, 21, 0] + [21] * (seqs - 4) + [more] and torch.equal(a.tables[2], tables[2])
        assert [y - x for x, y in zip(loc, loc[1:])] == [1, 1, max(q, 0)] + [1] * (seqs - 4) + [more]
        table = a.tables.tolist()
        for b in range(seqs):
            at = range(loc[b], loc[b + 1])
            if b == 2:
                assert all(slots[i] == -1 for i in at)
                continue
            first = lens[b] - len(at)
            assert [slots[i] for i in at] == [table[b][p // 16] * 16 + p % 16 for p in range(first, lens[b])]
        assert all(x == -1 for x in slots[loc[-1]:])


@pytest.mark.parametrize("extra", [-1, -2, -5, -9, -1000])
def test_alloc_runs_out(extra):
    # later sequences that need nothing are served, earlier ones too; one that does not fit takes nothing
    held, ctx, new = [16, 40, 33, 0, 20, 16], [16, 40, 33, 0, 20, 16], [1, 60, 5, 100, 3, 1]
    Step(held, ctx, new, extra=extra).run().check()


def test_alloc_blocks_that_come_back_are_used():
    Step([160, 0, 16], [0, 0, 16], [0, 100, 1], extra=-8).run().check()


def test_alloc_without_held_lens_and_with_a_count_of_its_own():
    a = Step([31, 64], [31, 64], [2, 3])
    count, new_count = a.free_count, ints([-1])
    a.run(held_lens=None, new_free_count=new_count)
    assert count.item() == a.count
    a.free_count = new_count
    a.check()
    # the same call again finds the same blocks
    before = [x.clone() for x in (a.tables, a.free, a.slots)]
    a.free_count = count
    a.run(held_lens=None, new_free_count=new_count)
    assert all(torch.equal(x, y) for x, y in zip(before, (a.tables, a.free, a.slots)))


def test_alloc_bad_lengths_leave_the_others():
    good = Step([31, 16, 40, 40, 16], [31, 16, 40, 40, 16], [2, 1, 1, 9, 20])
    tables = good.tables.clone()
    for i, (h, c, q) in enumerate([(-1, 0, 1), (16, 17, 1), (40, 40, -3), (40, 40, 16 * tables.shape[1]), (1 << 30, 1 << 30, 1)]):
        a = Step([31, 16, 40, 40, 16], [31, 16, 40, 40, 16], [2, 1, 1, 9, 20])
        a.held_t[2], a.args[0][2], a.args[1][2] = h, c, q
        a.slots, a.positions = ints([-5] * 500), ints([-5] * 500)
        a.run()
        assert status() == pb.PA_DEV_BAD_SEQ_LEN
        assert torch.equal(a.tables[2], tables[2]) and a.lens.tolist() == [33, 17, 0, 49, 36]
        loc = a.loc.tolist()
        assert [y - x for x, y in zip(loc, loc[1:])] == [2, 1, min(max(q, 0), 497), min(9, max(0, 497 - max(q, 0))), min(
            20, max(0, 488 - max(q, 0)))]
        assert a.slots[loc[2]:loc[3]].tolist() == [-1] * (loc[3] - loc[2])
        ends = [(0, 31), (1, 16)] + ([(3, 40), (4, 16)] if q < 20 else [])
        for b, c0 in ends:
            row = a.tables[b].tolist()
            assert a.slots[loc[b]:loc[b + 1]].tolist() == [row[p // 16] * 16 + p % 16 for p in range(c0, c0 + loc[b + 1] - loc[b])]


@pytest.mark.parametrize("count", [-1, 1 << 20, -(1 << 31), (1 << 31) - 1])
def test_alloc_bad_count_moves_nothing(count):
    a = Step([31, 64], [31, 0], [2, 0], room=10)
    tables, free = a.tables.clone(), a.free.clone()
    a.free_count.fill_(count)
    a.run()
    assert status() == pb.PA_DEV_NO_BLOCKS
    assert torch.equal(a.tables, tables) and torch.equal(a.free, free) and a.free_count.item() == count


def test_alloc_more_back_than_there_are_blocks():
    a = Step([31, 64], [31, 0], [1, 0])
    a.free_count.fill_(a.free.shape[0] - 2)
    tables, free = a.tables.clone(), a.free.clone()
    a.run()
    assert status() == pb.PA_DEV_NO_BLOCKS
    assert torch.equal(a.tables, tables) and torch.equal(a.free, free)


def test_alloc_bad_blocks_are_reported():
    a = Step([16], [16], [40])
    a.free[a.count - 2] = 1 << 27
    a.run()
    assert status() == pb.PA_DEV_BAD_BLOCK_ID
    want = a.tables[0].tolist()
    assert a.slots[:40].tolist() == [-1 if want[p // 16] == 1 << 27 else want[p // 16] * 16 + p % 16 for p in range(16, 56)]


def test_alloc_too_few_rows_are_reported():
    a = Step([16, 16], [16, 16], [10, 20], pad=0)
    a.slots, a.positions = ints([-5] * 15), ints([-5] * 15)
    a.run()
    assert status() == pb.PA_DEV_BAD_SEQ_LEN
    assert a.loc.tolist() == [0, 10, 15] and a.positions.tolist() == list(range(16, 26)) + list(range(16, 21))


PUT_SHAPES = [(24, 4, 256, 64), (24, 4, 256, 256), (32, 8, 128, 128), (8, 1, 64, 64), (12, 12, 64, 24), (10, 2, 128, 2),
              (21, 3, 256, 126), (1, 1, 64, 0), (5, 5, 128, 32)]


def put_case(T, H, hkv, D, rot, top=50, seed=0, nblocks=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    half = lambda *s: torch.randn(*s, generator=g, device="cuda").half()
    nb = nblocks or S.blocks(T) + 2
    q, k, v = half(T, H, D), half(T, hkv, D), half(T, hkv, D)
    caches = [torch.full((nb, hkv, 16, D), 9.0, dtype=torch.float16, device="cuda") for _ in range(2)]
    order = torch.randperm(nb * 16, generator=torch.Generator().manual_seed(seed))[:T].to(torch.int32).cuda()
    pos = torch.randint(0, top, (T,), generator=torch.Generator().manual_seed(seed)).to(torch.int32).cuda()
    ang = torch.rand(top, rot // 2, generator=g, device="cuda") * 6.28
    return q, k, v, caches, order, pos, torch.cat([ang.cos(), ang.sin()], dim=1).contiguous()


def check_put(q, k, v, caches, slots, pos, table, pairs, q_out, k_out, q_in=None, k_in=None):
    on = pos >= 0
    at = pos.clamp(min=0).long()
    for x, out in ((q, q_out), (k, k_out)):
        y, bound = S.rotate(x, at, table, pairs)
        if out is not None:
            S.check(out[on], y[on], bound[on], "rotated")
            rot = table.shape[1]
            assert torch.equal(out[on][..., rot:], x[on][..., rot:])
    y, bound = S.rotate(k, at, table, pairs)
    used = torch.zeros(caches[0].shape[0] * 16, dtype=torch.bool, device="cuda")
    for t, slot in enumerate(slots.tolist()):
        if slot < 0 or int(pos[t]) < 0:
            continue
        used[slot] = True
        S.check(caches[0][slot // 16, :, slot % 16], y[t], bound[t], f"cache {t}")
        assert torch.equal(caches[1][slot // 16, :, slot % 16], v[t])
    for c in caches:
        assert bool((c.transpose(1, 2).flatten(0, 1)[~used] == 9.0).all())


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("H,hkv,D,rot", PUT_SHAPES)
@pytest.mark.parametrize("T", [1, 37])
def test_put(T, H, hkv, D, rot, pairs):
    q, k, v, caches, slots, pos, table = put_case(T, H, hkv, D, rot, seed=rot + T)
    slots[T // 2] = -1
    if T > 1:
        pos[T // 3] = -1
    q_out, k_out = torch.full_like(q, 5.0), torch.full_like(k, 5.0)
    pb.pa_kv_put(q_out, k_out, q, k, v, *caches, slots, pos, table, pairs=pairs)
    assert status() == 0
    check_put(q, k, v, caches, slots, pos, table, pairs, q_out, k_out)
    if T > 1:
        assert bool((q_out[T // 3] == 5.0).all()) and bool((k_out[T // 3] == 5.0).all())


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("rot", [128, 24, 64])
def test_put_in_place_and_from_a_joint_projection(rot, pairs):
    q, k, v, caches, slots, pos, table = put_case(50, 8, 2, 128, rot, seed=7)
    q2, k2 = q.clone(), k.clone()
    pb.pa_kv_put(q2, k2, q2, k2, v, *caches, slots, pos, table, pairs=pairs)
    assert status() == 0
    check_put(q, k, v, caches, slots, pos, table, pairs, q2, k2)
    joint = torch.cat([q, k, v], dim=1)
    other = [torch.full_like(c, 9.0) for c in caches]
    q3 = torch.empty_like(q)
    pb.pa_kv_put(q3, None, joint[:, :8], joint[:, 8:10], joint[:, 10:], *other, slots, pos, table, pairs=pairs)
    assert status() == 0
    assert torch.equal(q3, q2) and torch.equal(other[0], caches[0]) and torch.equal(other[1], caches[1])
    # without a cache
    q4, k4 = torch.empty_like(q), torch.empty_like(k)
    pb.pa_kv_put(q4, k4, q, k, None, None, None, None, pos, table, pairs=pairs)
    assert torch.equal(q4, q2) and torch.equal(k4, k2)


def test_put_non_finite_values_stay_in_their_pair():
    q, k, v, caches, slots, pos, table = put_case(4, 8, 2, 128, 64, seed=3)
    q[1, 2, 3], k[2, 1, 40], v[3, 0, 5] = math.nan, math.inf, -math.inf
    q_out, k_out = torch.empty_like(q), torch.empty_like(k)
    pb.pa_kv_put(q_out, k_out, q, k, v, *caches, slots, pos, table)
    bad = torch.zeros_like(q_out, dtype=torch.bool)
    bad[1, 2, 3] = bad[1, 2, 35] = True
    assert torch.equal(~torch.isfinite(q_out), bad)
    bad = torch.zeros_like(k_out, dtype=torch.bool)
    bad[2, 1, 8] = bad[2, 1, 40] = True
    assert torch.equal(~torch.isfinite(k_out), bad)
    assert caches[1][int(slots[3]) // 16, 0, int(slots[3]) % 16, 5].item() == -math.inf


def test_put_bad_slots_and_positions_are_reported():
    q, k, v, caches, slots, pos, table = put_case(6, 8, 2, 128, 128, seed=4)
    slots[2] = caches[0].shape[0] * 16
    q_out, k_out = torch.full_like(q, 5.0), torch.full_like(k, 5.0)
    pb.pa_kv_put(q_out, k_out, q, k, v, *caches, slots, pos, table)
    assert status() == pb.PA_DEV_BAD_BLOCK_ID
    slots[2] = -1
    check_put(q, k, v, caches, slots, pos, table, False, q_out, k_out)
    caches = [torch.full_like(c, 9.0) for c in caches]
    pos[4] = table.shape[0]
    q_out.fill_(5.0), k_out.fill_(5.0)
    pb.pa_kv_put(q_out, k_out, q, k, v, *caches, slots, pos, table)
    assert status() == pb.PA_DEV_BAD_SEQ_LEN
    assert bool((q_out[4] == 5.0).all())
    pos[4] = -1
    check_put(q, k, v, caches, slots, pos, table, False, q_out, k_out)


def test_put_offsets_past_32_bits():
    """A cache of more than 2^31 elements: the last blocks are where they should be."""
    hkv, D = 4, 256
    nb = (1 << 31) // (hkv * 16 * D) + 5
    q, k, v, _, _, pos, table = put_case(2, 4, hkv, D, 64, seed=5)
    caches = [torch.zeros(nb, hkv, 16, D, dtype=torch.float16, device="cuda") for _ in range(2)]
    slots = ints([nb * 16 - 1, nb * 16 - 18])
    q_out, k_out = torch.empty_like(q), torch.empty_like(k)
    pb.pa_kv_put(q_out, k_out, q, k, v, *caches, slots, pos, table)
    assert status() == 0
    for t, s in enumerate(slots.tolist()):
        assert torch.equal(caches[0][s // 16, :, s % 16], k_out[t]) and torch.equal(caches[1][s // 16, :, s % 16], v[t])


def test_put_binding_refusals():
    q, k, v, caches, slots, pos, table = put_case(4, 8, 2, 128, 64)
    with pytest.raises(TypeError):
        pb.pa_kv_put(q, k, q.float(), k, v, *caches, slots, pos, table)
    with pytest.raises(ValueError):
        pb.pa_kv_put(q, k, q, k, v, *caches, slots[:3], pos, table)
    with pytest.raises(ValueError):
        pb.pa_kv_put(q, k, q, k, v, caches[0], None, slots, pos, table)
    with pytest.raises(TypeError):
        pb.pa_kv_put(q, k, q, k, v, caches[0].to(torch.int8), caches[1].to(torch.int8), slots, pos, table)
    with pytest.raises(ValueError):
        pb.pa_kv_put(q, k, q.transpose(0, 1).contiguous().transpose(0, 1), k, v, *caches, slots, pos, table)
    with pytest.raises(ValueError):
        pb.pa_kv_alloc(ints([[0, 1]]), ints([1]), ints([0, 0]), ints([1]), ints([1]), ints([0, 0]), ints([0]), ints([0]), ints([0]))
