"""Cases of the operators of a serving step around the paged cache, and of linear attention layers beside it.

Four operators:

* ``alloc``    block tables, slot map and positions from request lengths: sequences that shrank or ended give blocks
               back to a stack of free ones, sequences that grow take theirs from it;
* ``put``      the rotary embedding of new tokens' Q and K by position, and K and V written to the slot map's slots;
* ``ldecode``  linear attention with a decay a kv head, one new token a sequence: the state's update and its product
               with q;
* ``lprefix``  the same for packed chunks of new tokens, causal, going on from the sequences' states.

A state is S [head_dim (of K)][head_dim (of V)] in 32 bits for each (sequence, kv head), held in a pool of slots:
S_t = exp(g) S_(t-1) + k_t v_t^T and out_t = scale q_t S_t, with g <= 0 the kv head's log decay.
"""
import math
import random

import torch

own = False

BS = 16  # tokens per block
CHUNK = 128  # tokens of a chunk of the plain form


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a decoding step of a batch: every sequence one token more, a few ended and a few that start
        dict(name="alloc_step_b64", op="alloc", seqs=64, ctx=8192, chunk=1, spread="uniform", chunk_spread="full",
             lens_seed=1),
        # a large batch of prompt chunks of unlike lengths
        dict(name="alloc_prompt_b512", op="alloc", seqs=512, ctx=4096, chunk=512, spread="uniform",
             chunk_spread="uniform", lens_seed=2),
        # the projections' output of a decoding step
        dict(name="put_step_b64", op="put", tokens=64, heads=24, hkv=4, dim=256, rot=64, pairs=False, top=102400),
        # of prompt chunks
        dict(name="put_prompt_16k", op="put", tokens=16384, heads=32, hkv=8, dim=128, rot=128, pairs=False, top=16384),
        # a single request's step: the call's latency
        dict(name="ldecode_b1", op="ldecode", seqs=1, heads=24, hkv=4, dim=256, decay="slopes"),
        # a batch's step
        dict(name="ldecode_b64", op="ldecode", seqs=64, heads=24, hkv=4, dim=256, decay="slopes"),
        # a large batch, smaller heads
        dict(name="ldecode_b256", op="ldecode", seqs=256, heads=32, hkv=8, dim=128, decay="slopes"),
        # a short follow-up of one request
        dict(name="lprefix_b1_q37", op="lprefix", seqs=1, chunk=37, chunk_spread="full", heads=32, hkv=8, dim=128,
             decay="slopes", fresh="none", lens_seed=8),
        # prompt chunks of a batch, some of them the first
        dict(name="lprefix_b4_q512", op="lprefix", seqs=4, chunk=512, chunk_spread="full", heads=24, hkv=4, dim=256,
             decay="slopes", fresh="some", lens_seed=9),
        # one long prompt
        dict(name="lprefix_b1_q8192", op="lprefix", seqs=1, chunk=8192, chunk_spread="full", heads=24, hkv=4, dim=256,
             decay="slopes", fresh="all", lens_seed=10),
        # a ragged batch, small heads of their own keys, one of them without decay
        dict(name="lprefix_b16_u4096", op="lprefix", seqs=16, chunk=4096, chunk_spread="uniform", heads=12, hkv=12,
             dim=64, decay="mixed", fresh="some", lens_seed=11),
        # a batch of whole prompts
        dict(name="lprefix_b8_q8192", op="lprefix", seqs=8, chunk=8192, chunk_spread="full", heads=32, hkv=8, dim=128,
             decay="slopes", fresh="all", lens_seed=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["alloc", "put", "ldecode", "lprefix", "lprefix"])
    heads, hkv, dim = rng.choice([(24, 4, 256), (32, 8, 128), (8, 1, 64), (12, 12, 64), (10, 2, 128), (21, 3, 256)])
    case = dict(op=op)
    if op == "alloc":
        case.update(seqs=_log_int(rng, 1, 512), ctx=_log_int(rng, 1, 8192), spread=rng.choice(["full", "uniform"]),
                    chunk_spread=rng.choice(["full", "uniform"]), lens_seed=rng.randrange(1 << 30))
        case["chunk"] = _log_int(rng, 1, min(4096, 512 * 256 // case["seqs"]))
        return case
    case.update(heads=heads, hkv=hkv, dim=dim)
    if op == "put":
        case.update(tokens=_log_int(rng, 1, 16384 * 40 * 128 // ((heads + hkv) * dim)),
                    rot=rng.choice([dim, dim // 2, dim // 4, 24]), pairs=rng.random() < 0.5,
                    top=_log_int(rng, 16, 102400))
        return case
    case["decay"] = rng.choice(["slopes", "mixed", "none"])
    if op == "ldecode":
        case["seqs"] = _log_int(rng, 1, 256 * 8 * 128 * 128 // (hkv * dim * dim))
        return case
    case["seqs"] = _log_int(rng, 1, 16)
    most = 65536 * 32 * 128 // (heads * dim * case["seqs"]) * 128 // max(dim, 128)
    case.update(chunk=_log_int(rng, 1, min(8192, most)), chunk_spread=rng.choice(["full", "uniform"]),
                fresh=rng.choice(["all", "some", "none"]), lens_seed=rng.randrange(1 << 30))
    return case


def _lengths(case, key, spread, low):
    rng = random.Random(case["lens_seed"] * 2 + (key == "chunk"))
    top, n = case[key], case["seqs"]
    if spread == "full" or top <= low:
        return [top] * n
    return [rng.randint(low, top) for _ in range(n)]


def _requests(case):
    """(tokens that the table holds, tokens that stay, new tokens) of each sequence: one in 32 has ended, one in 32
    starts, one in 16 takes back tokens that were written ahead."""
    rng = random.Random(case["lens_seed"] * 2 + 7)
    held, ctx = _lengths(case, "ctx", case["spread"], 1), []
    new = _lengths(case, "chunk", case["chunk_spread"], 1)
    for b in range(case["seqs"]):
        kind = rng.random()
        ctx.append(held[b])
        if kind < 1 / 32:
            ctx[b], new[b] = 0, 0
        elif kind < 2 / 32:
            held[b] = ctx[b] = 0
        elif kind < 4 / 32:
            ctx[b] = max(0, held[b] - rng.randint(1, 40))
    return held, ctx, new


def _blocks(n):
    return -(-n // BS)


def work(case):
    op = case["op"]
    if op == "alloc":
        held, ctx, new = _requests(case)
        moved = sum(abs(_blocks(c + n) - _blocks(h)) for h, c, n in zip(held, ctx, new))
        return {"bytes": 4 * (5 * case["seqs"] + 3) + 8 * (sum(new) + moved), "flops": sum(new)}
    heads, hkv, dim = case["heads"], case["hkv"], case["dim"]
    if op == "put":
        t = case["tokens"]
        return {"bytes": 2 * t * dim * (2 * heads + 5 * hkv) + 8 * t + 4 * case["rot"] * min(t, case["top"]),
                "flops": 3 * t * (heads + hkv) * case["rot"]}
    if op == "ldecode":
        b = case["seqs"]
        return {"bytes": b * (8 * hkv * dim * dim + 4 * (heads + hkv) * dim),
                "flops": 2 * b * dim * dim * (heads + hkv)}
    t = sum(_lengths(case, "chunk", case["chunk_spread"], 1))
    states = sum(4 if f else 8 for f in _fresh(case))
    return {"bytes": 4 * t * dim * (heads + hkv) + states * hkv * dim * dim, "flops": 2 * t * dim * dim * (heads + hkv)}


# ---------------------------------------------------------------- inputs

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _fresh(case):
    """Which sequences start from no state."""
    rng = random.Random(case["lens_seed"] * 2 + 3)
    return [{"all": True, "none": False}.get(case["fresh"], rng.random() < 0.5) for _ in range(case["seqs"])]


def _log_decay(case):
    """Slopes that halve from head to head's share of eight octaves; "mixed" has heads that forget at once and never."""
    hkv = case["hkv"]
    g = [-(2.0 ** (-8.0 * (h + 1) / hkv)) for h in range(hkv)]
    if case["decay"] == "none":
        g = [0.0] * hkv
    if case["decay"] == "mixed":
        g[0], g[-1] = -6.0, 0.0
    return torch.tensor(g, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    half = lambda *s: torch.randn(*s, generator=gen, device="cuda").half()
    op = case["op"]
    st = {"case": case}
    if op == "alloc":
        held, ctx, new = _requests(case)
        need = [_blocks(h) for h in held]
        most = max(1, max(max(_blocks(c + n), h) for c, n, h in zip(ctx, new, need)))
        take = sum(max(0, _blocks(c + n) - h) for c, n, h in zip(ctx, new, need))
        total = sum(need) + take + 64
        perm = torch.randperm(total, generator=cpu).to(torch.int32)
        tables = torch.full((len(held), most), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            tables[b, :n] = perm[at:at + n]
            at += n
        free = torch.full((total,), -1, dtype=torch.int32)
        free[:total - at] = perm[at:]
        tokens = sum(new) + 5  # rows of padding
        st.update(held=_ints(held), ctx=_ints(ctx), new=_ints(new), tables=tables.cuda(), free=free.cuda(),
                  count=_ints([total - at]), new_count=_ints([0]), loc=_ints([0] * (len(held) + 1)),
                  lens=torch.zeros(len(held), dtype=torch.int32, device="cuda"), slots=_ints([0] * tokens),
                  positions=_ints([0] * tokens))
        return st
    heads, hkv, dim = case["heads"], case["hkv"], case["dim"]
    if op == "put":
        t, top, rot = case["tokens"], case["top"], case["rot"]
        blocks = _blocks(t) + 3
        angle = torch.arange(top, device="cuda").double()[:, None] * 1e6 ** (
            -torch.arange(rot // 2, device="cuda").double() / (rot // 2))
        st.update(table=torch.cat([angle.cos(), angle.sin()], dim=1).float(), q=half(t, heads, dim),
                  k=half(t, hkv, dim), v=half(t, hkv, dim), k_cache=half(blocks, hkv, BS, dim),
                  v_cache=half(blocks, hkv, BS, dim))
        slots = torch.randperm(blocks * BS, generator=cpu)[:t].to(torch.int32)
        slots[torch.rand(t, generator=cpu) < 0.01] = -1  # tokens that are kept elsewhere
        st.update(slots=slots.cuda(), positions=torch.randint(0, top, (t,), generator=cpu).to(torch.int32).cuda(),
                  q_out=torch.empty_like(st["q"]), k_out=torch.empty_like(st["k"]))
        return st
    b = case["seqs"]
    st["scale"] = 1.0 / math.sqrt(dim)
    st["g"] = _log_decay(case)
    # states as earlier tokens left them: larger where the decay is slow
    size = torch.rsqrt(1.0 - torch.exp(2.0 * st["g"]).clamp(max=1 - 1e-3))
    st["states"] = torch.randn(b + 3, hkv, dim, dim, generator=gen, device="cuda") * size[:, None, None]
    st["slots"] = torch.randperm(b + 3, generator=cpu)[:b].to(torch.int32).cuda()
    new = [1] * b if op == "ldecode" else _lengths(case, "chunk", case["chunk_spread"], 1)
    t = sum(new)
    st.update(q=half(t, heads, dim), k=half(t, hkv, dim), v=half(t, hkv, dim))
    st["out"] = torch.empty_like(st["q"])
    if op == "lprefix":
        st["ctx"] = _ints([0 if f else 100 for f in _fresh(case)])
        st["loc"] = torch.tensor([0] + new).cumsum(0).to(torch.int32).cuda()
        st["max_new"] = max(new)
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    op = st["case"]["op"]
    if own:
        return _run_own(st)
    if op == "alloc":
        return _alloc(st)
    if op == "put":
        return _put(st)
    return _ldecode(st) if op == "ldecode" else _lprefix(st)


def _run_own(st):
    from paged_kv_cache_308_gb300 import binding as pb
    case, op = st["case"], st["case"]["op"]
    if op == "alloc":
        pb.pa_kv_alloc(st["tables"], st["free"], st["count"], st["ctx"], st["new"], st["loc"], st["lens"], st["slots"],
                       st["positions"], held_lens=st["held"], new_free_count=st["new_count"])
        return _alloc_out(st)
    if op == "put":
        pb.pa_kv_put(st["q_out"], st["k_out"], st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"], st["slots"],
                     st["positions"], st["table"], pairs=case["pairs"])
        return _put_out(st)
    if op == "ldecode":
        pb.pa_linear_decode(st["out"], st["q"], st["k"], st["v"], st["states"], st["slots"], st["g"], st["scale"])
        return {"out": st["out"], "states": st["states"]}
    if "ws" not in st:
        st["ws"] = torch.empty(pb.pa_linear_prefix_workspace_size(
            case["seqs"], st["q"].shape[0], st["max_new"], case["heads"], case["hkv"], case["dim"]), dtype=torch.uint8,
            device="cuda")
    pb.pa_linear_prefix(st["out"], st["q"], st["k"], st["v"], st["states"], st["slots"], st["g"], st["ctx"], st["loc"],
                        st["scale"], max_query_len=st["max_new"], workspace=st["ws"])
    return {"out": st["out"], "states": st["states"]}


def _alloc_out(st):
    return {"tables": st["tables"], "free": st["free"], "count": st["new_count"], "loc": st["loc"], "lens": st["lens"],
            "slots": st["slots"], "positions": st["positions"]}


def _put_out(st):
    return {"q": st["q_out"], "k": st["k_out"], "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


# ---------------------------------------------------------------- the plain forms

def _alloc(st):
    held, ctx, new = st["held"].long(), st["ctx"].long(), st["new"].long()
    n0, n1 = (held + BS - 1) // BS, (ctx + new + BS - 1) // BS
    col = torch.arange(st["tables"].shape[1], device="cuda")
    tables, free, count = st["tables"], st["free"], st["count"].long()
    room = free.shape[0]
    # what is given back, onto the stack
    back = (col >= n1[:, None]) & (col < n0[:, None])
    rank = (torch.cumsum(back.flatten().long(), 0) - 1).view_as(back)
    stack = torch.cat([free, free[:1]])
    stack[torch.where(back, count + rank, torch.full_like(rank, room))] = tables
    top = count + back.sum()
    # what is taken, from its top
    need = (n1 - n0).clamp(min=0)
    total = torch.cumsum(need, 0)
    served = (need == 0) | (total <= top)
    need = torch.where(served, need, torch.zeros_like(need))
    k = (total - (n1 - n0).clamp(min=0))[:, None] + col - n0[:, None]
    mine = served[:, None] & (col >= n0[:, None]) & (col < n1[:, None])
    st["tables"].copy_(torch.where(mine, stack[torch.where(mine, top - 1 - k, torch.zeros_like(k))], tables))
    st["free"].copy_(stack[:room])
    st["new_count"].copy_(top - need.sum())
    loc = torch.cat([torch.zeros_like(new[:1]), torch.cumsum(new, 0)])
    st["loc"].copy_(loc)
    st["lens"].copy_(torch.where(served, ctx + new, ctx))
    # the tokens
    t = torch.arange(st["slots"].shape[0], device="cuda")
    b = torch.searchsorted(loc[1:].contiguous(), t, right=True)
    some = b < held.shape[0]
    b = torch.where(some, b, torch.zeros_like(b))
    pos = torch.where(some, ctx[b] + t - loc[b], torch.zeros_like(t))
    slot = st["tables"][b, pos // BS].long() * BS + pos % BS
    st["slots"].copy_(torch.where(some & served[b], slot, torch.full_like(slot, -1)))
    st["positions"].copy_(torch.where(some, pos, torch.full_like(pos, -1)))
    return _alloc_out(st)


def _rotated(x, cos, sin, rot, pairs):
    x = x.float()
    r = x[..., :rot]
    if pairs:
        a, b = r[..., 0::2], r[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([y, x[..., rot:]], dim=-1).half()


def _put(st):
    case = st["case"]
    rot = case["rot"]
    row = st["table"][st["positions"].long()][:, None]
    cos, sin = row[..., :rot // 2], row[..., rot // 2:]
    st["q_out"].copy_(_rotated(st["q"], cos, sin, rot, case["pairs"]))
    st["k_out"].copy_(_rotated(st["k"], cos, sin, rot, case["pairs"]))
    slot = st["slots"].long()
    kept = slot >= 0
    slot = slot[kept]
    st["k_cache"][slot // BS, :, slot % BS] = st["k_out"][kept]
    st["v_cache"][slot // BS, :, slot % BS] = st["v"][kept]
    return _put_out(st)


def _ldecode(st):
    slots = st["slots"].long()
    q, k, v = st["q"].float(), st["k"].float(), st["v"].float()
    b, hkv, d = k.shape
    s = st["states"][slots] * torch.exp(st["g"])[:, None, None] + k[..., :, None] * v[..., None, :]
    st["states"][slots] = s
    st["out"].copy_((torch.matmul(q.view(b, hkv, -1, d), s) * st["scale"]).view(b, -1, d))
    return {"out": st["out"], "states": st["states"]}


def _powers(g, n):
    """exp(g n) in 64 bits, 0 where n < 0; rounded to 32."""
    return torch.where(n >= 0, torch.exp(g.double() * n.clamp(min=0)), torch.zeros((), dtype=torch.float64,
                                                                                  device="cuda")).float()


def _lprefix(st):
    """Chunks of the sequences, which are padded in front so that they end with a chunk."""
    slots, loc, g = st["slots"].long(), st["loc"].long(), st["g"]
    t, heads, d = st["q"].shape
    hkv = st["k"].shape[1]
    b, c = slots.shape[0], CHUNK
    n = -(-st["max_new"] // c)
    size = loc[1:] - loc[:-1]
    i = torch.arange(n * c, device="cuda") - (n * c - size)[:, None]  # a token's place in its sequence
    some = i >= 0
    at = torch.where(some, loc[:-1, None] + i, torch.zeros_like(i))
    fill = lambda x: torch.where(some[..., None, None], x[at].float(), torch.zeros((), device="cuda"))
    q = fill(st["q"]).view(b, n, c, hkv, -1, d).permute(0, 3, 1, 4, 2, 5)  # [seqs, hkv, chunks, group, c, d]
    k = fill(st["k"]).view(b, n, c, hkv, d).permute(0, 3, 1, 2, 4)
    v = fill(st["v"]).view(b, n, c, hkv, d).permute(0, 3, 1, 2, 4)
    s0 = torch.where((st["ctx"] > 0)[:, None, None, None], st["states"][slots], torch.zeros((), device="cuda"))
    j = torch.arange(c, device="cuda")
    # inside a chunk
    p = torch.matmul(q, k[:, :, :, None].transpose(4, 5)) * _powers(g[:, None, None], j[:, None] - j)[:, None, None]
    o = torch.matmul(p, v[:, :, :, None])
    # from the chunks before it
    add = torch.matmul((k * _powers(g[:, None], c - 1 - j)[:, None, :, None]).transpose(3, 4), v)  # [seqs, hkv, chunks, d, d]
    m = torch.arange(n + 1, device="cuda")
    past = _powers(g[:, None, None], torch.where(m[:, None] > m[:n], (m[:, None] - 1 - m[:n]) * c, -1))
    s = torch.matmul(past, add.flatten(3)).view(b, hkv, n + 1, d, d)
    o = o + torch.matmul(q, s[:, :, :n, None]) * _powers(g[:, None], j + 1)[:, None, None, :, None]
    # from the state before the chunks
    then = _powers(g[:, None], i[:, None] + 1)  # [seqs, hkv, tokens]
    o = o + torch.matmul(q, s0[:, :, None, None]) * then.view(b, hkv, n, 1, c, 1)
    last = s[:, :, n] + s0 * _powers(g, size[:, None])[..., None, None]
    st["states"][slots] = torch.where((size > 0)[:, None, None, None], last, st["states"][slots])
    o = (o * st["scale"]).permute(0, 2, 4, 1, 3, 5).reshape(b, n * c, heads, d)
    st["out"].copy_(o[some])
    return {"out": st["out"], "states": st["states"]}


# ---------------------------------------------------------------- in 64 bits, from the definitions

def exact(case, seed):
    if case["op"] == "alloc":
        return None  # whole numbers
    st = prepare(case, seed)
    if case["op"] == "put":
        return _exact_put(st, case)
    return _exact_linear(st, case)


def _exact_put(st, case):
    rot, d = case["rot"], case["dim"]
    pos = st["positions"].long()
    # the rotation as a product of each pair, a complex number, with cos + i sin
    turn = torch.complex(st["table"][pos, :rot // 2].double(), st["table"][pos, rot // 2:].double())[:, None]
    first = torch.arange(0, rot, 2, device="cuda") if case["pairs"] else torch.arange(rot // 2, device="cuda")
    second = first + 1 if case["pairs"] else first + rot // 2
    res = {}
    for name in ("q", "k"):
        x = st[name].double()
        z = torch.complex(x[..., first], x[..., second]) * turn
        x[..., first], x[..., second] = z.real, z.imag
        res[name] = x
    for name, rows in (("k_cache", res["k"]), ("v_cache", st["v"].double())):
        flat = st[name].double().transpose(1, 2).reshape(-1, case["hkv"], d)  # by slot
        kept = st["slots"] >= 0
        flat[st["slots"][kept].long()] = rows[kept]
        res[name] = flat.view(-1, BS, case["hkv"], d).transpose(1, 2)
    return res


def _exact_linear(st, case):
    hkv = case["hkv"]
    group = case["heads"] // hkv
    states = st["states"].double()
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    b = case["seqs"]
    loc = st["loc"].tolist() if "loc" in st else list(range(b + 1))
    old = (st["ctx"] > 0).tolist() if "ctx" in st else [True] * b
    for x, slot in enumerate(st["slots"].tolist()):
        lo, hi = loc[x], loc[x + 1]
        if lo == hi:
            continue
        t = torch.arange(1.0, hi - lo + 1, dtype=torch.float64, device="cuda")
        for h in range(hkv):
            g = float(st["g"][h].double())
            s = states[slot, h].clone() if old[x] else torch.zeros_like(states[slot, h])
            k, v = st["k"][lo:hi, h].double(), st["v"][lo:hi, h].double()
            for j in range(h * group, (h + 1) * group):
                q = st["q"][lo:hi, j].double()
                o = (q @ s) * torch.exp(g * t)[:, None]
                for at in range(0, hi - lo, 1024):
                    end = min(hi - lo, at + 1024)
                    apart = t[at:end, None] - t[:end]
                    o[at:end] += ((q[at:end] @ k[:end].T) * torch.exp(g * apart.clamp(min=0)) * (apart >= 0)) @ v[:end]
                out[lo:hi, j] = o * st["scale"]
            states[slot, h] = s * math.exp(g * (hi - lo)) + (k * torch.exp(g * (hi - lo - t))[:, None]).T @ v
    return {"out": out, "states": states}
