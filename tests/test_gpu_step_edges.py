"""Block allocation over several calls: no block is lost when blocks run out or lengths are bad."""
import random

import pytest
import torch

import step_helpers as S
from paged_kv_cache_308_gb300 import binding as pb

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def status():
    torch.cuda.synchronize()
    return pb.pa_get_device_status()


class Pool:
    """Sequences that hold `held` tokens, `spare` blocks free, in a stack with room for all."""

    def __init__(self, held, spare, cols):
        need = [S.blocks(h) for h in held]
        ids = list(range(sum(need) + spare))
        random.Random(len(held)).shuffle(ids)
        rows, at = [], 0
        for n in need:
            rows.append(ids[at:at + n] + [-1] * (cols - n))
            at += n
        self.total, self.held = len(ids), ints(held)
        self.tables, self.free, self.count = ints(rows), ints(ids[at:] + [-1] * at), ints([spare])

    def step(self, ctx, new, in_place, want, tokens=None):
        B, T = len(ctx), sum(max(n, 0) for n in new) + 3 if tokens is None else tokens
        held = self.held if in_place else torch.full_like(self.held, -7)
        lens = ints([-7] * B)
        pb.pa_kv_alloc(self.tables, self.free, self.count, ints(ctx), ints(new), ints([-7] * (B + 1)), lens, ints([-7] * T),
                       ints([-7] * T), held_lens=self.held, new_held_lens=held)
        assert status() == want
        self.held = held
        return lens.tolist()

    def check(self):
        """Every block is on the stack or in the part of a row that new_held_lens names."""
        rows, held = self.tables.tolist(), self.held.tolist()
        used = [x for row, h in zip(rows, held) for x in row[:S.blocks(h)]]
        assert sorted(used + self.free[:self.count.item()].tolist()) == list(range(self.total))

    def end(self):
        self.step([0] * len(self.held), [0] * len(self.held), True, 0)
        assert self.count.item() == self.total and self.held.tolist() == [0] * len(self.held)
        self.check()


@pytest.mark.parametrize("in_place", [False, True])
def test_held_lens_of_a_sequence_that_is_not_served(in_place):
    """It shrinks and grows in one step, finds no blocks, and ends: all of its blocks come back."""
    p = Pool([40, 20], 0, 8)
    assert p.step([3, 20], [60, 5], in_place, pb.PA_DEV_NO_BLOCKS) == [3, 25]
    assert p.held.tolist() == [40, 25]
    p.check()
    p.end()


# one and eight blocks of a cluster, all sequences kept or a share, tokens placed there or by a launch of their own
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("seqs,top,chunk", [(1, 90, 200), (64, 500, 60), (65, 300, 1), (300, 300, 200), (2049, 60, 20)])
def test_no_block_is_lost_when_blocks_run_out(seqs, top, chunk, in_place):
    rng = random.Random(seqs)
    held = [rng.randint(0, top) for _ in range(seqs)]
    p = Pool(held, seqs // 3, S.blocks(top + 4 * chunk))
    for _ in range(3):
        ctx = [rng.choice([h, h, rng.randint(0, h)]) for h in held]
        new = [rng.randint(0, chunk) for _ in ctx]
        before, count = p.held.tolist(), p.count.item()
        back = sum(max(0, S.blocks(h) - S.blocks(c + q)) for h, c, q in zip(before, ctx, new))
        wanted, ok = 0, []
        for h, c, q in zip(before, ctx, new):
            need = max(0, S.blocks(c + q) - S.blocks(h))
            wanted += need
            ok.append(need == 0 or wanted <= count + back)
        lens = p.step(ctx, new, in_place, 0 if all(ok) else pb.PA_DEV_NO_BLOCKS)
        held = p.held.tolist()
        assert held == [c + q if good else h for h, c, q, good in zip(before, ctx, new, ok)]
        assert lens == [c + q if good else c for c, q, good in zip(ctx, new, ok)]
        p.check()
    p.end()


@pytest.mark.parametrize("seqs", [5, 100])
@pytest.mark.parametrize("more", [10, 20000])
def test_held_lens_of_bad_lengths(seqs, more):
    for c, q in ((-1, 1), (41, 1), (40, -3), (40, 1 << 20)):
        p = Pool([40] * (seqs - 1) + [0], S.blocks(more) + seqs, S.blocks(more) + 3)
        ctx, new = [40] * (seqs - 1) + [0], [1] * (seqs - 1) + [more]
        ctx[2], new[2] = c, q
        p.step(ctx, new, True, pb.PA_DEV_BAD_SEQ_LEN, tokens=(1 << 20) + more + seqs)
        assert p.held.tolist() == [41, 41, 40] + [41] * (seqs - 4) + [more]
        p.check()
        p.end()


def test_held_lens_of_a_bad_count():
    """No block moves: who would have given some back, or got some, holds what it held."""
    p = Pool([40, 40, 40, 5], 3, 8)
    count = p.count.clone()
    p.count.fill_(-1)
    p.step([3, 40, 40, 5], [0, 30, 2, 0], True, pb.PA_DEV_NO_BLOCKS)
    assert p.held.tolist() == [40, 40, 42, 5]
    p.count = count
    p.check()
    p.end()


# 39 tokens are three blocks: more than a row of two has, and than are free
@pytest.mark.parametrize("cols,want,second", [(2, pb.PA_DEV_BAD_SEQ_LEN, 0), (3, pb.PA_DEV_NO_BLOCKS, 9)])
def test_held_lens_without_held_lens(cols, want, second):
    """Before the call a row holds the blocks of its context then."""
    tables, free, count = ints([[3, -1, -1][:cols], [4, -1, -1][:cols]]), ints([1, 2, -1, -1, -1]), ints([1])
    lens, held, slots = ints([0, 0]), ints([0, 0]), ints([0] * 40)
    pb.pa_kv_alloc(tables, free, count, ints([16, 9]), ints([2, 30]), ints([0, 0, 0]), lens, slots, torch.zeros_like(slots),
                   new_held_lens=held)
    assert status() == want
    assert held.tolist() == [18, 9] and lens.tolist() == [18, second]


def test_held_lens_in_a_captured_loop():
    """A sequence that waits for blocks step after step, in place in a graph, until another one ends."""
    p = Pool([16, 48, 20], 0, 8)
    ctx, new, loc, lens = ints([0, 48, 20]), ints([40, 0, 1]), ints([0] * 4), ints([0] * 3)
    slots, pos = ints([0] * 45), ints([0] * 45)

    def run():
        pb.pa_kv_alloc(p.tables, p.free, p.count, ctx, new, loc, lens, slots, pos, held_lens=p.held, new_held_lens=p.held)

    run()
    assert status() == pb.PA_DEV_NO_BLOCKS and p.held.tolist() == [16, 48, 21] and lens.tolist() == [0, 48, 21]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        run()
    ctx.copy_(ints([0, 48, 21]))
    g.replay()
    assert status() == pb.PA_DEV_NO_BLOCKS and p.held.tolist() == [16, 48, 22]
    p.check()
    ctx.copy_(ints([0, 0, 22]))
    g.replay()
    assert status() == 0 and p.held.tolist() == [40, 0, 23] and lens.tolist() == [40, 0, 23]
    p.check()
    p.end()
