"""Cases of the operators of the 8-bit paged cache and of eviction by accumulated attention weight.

Five operators over a block-tabled KV cache ([num_blocks][kv_heads][16 tokens][head_dim]):

* ``append``   new tokens' K and V written into the cache, in 8 bits with one scale per (block, kv head);
* ``decode``   one query token a sequence over an 8-bit cache;
* ``prefix``   a chunk of new tokens over an 8-bit cache, causal inside the chunk;
* ``weights``  decode that also adds each token's attention weight (summed over the query heads of its
               kv head) to an accumulator;
* ``evict``    the tokens with the largest accumulated weights (and the first and latest ones) move to other,
               fewer blocks.

The 8-bit formats: ``e4m3`` with block scales that are powers of two (the smallest with 448 s >= the block's
largest magnitude), ``int8`` with block scales of 8 significant bits (the smallest with 127 s >= it).  A scale
only grows while tokens join a block; the codes that are there are then rounded again to the new scale.
"""
import math
import random

import torch

own = False

BS = 16  # tokens per block
DTYPES = {"f16": torch.float16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step of a batch: each sequence's new token joins its last block
        dict(name="append_step_b64", op="append", fmt="e4m3", seqs=64, ctx=2048, chunk=1, spread="uniform",
             chunk_spread="full", hkv=4, dim=256, lens_seed=1),
        # prompts written chunk by chunk, ragged, behind cached prefixes of odd lengths
        dict(name="append_prompt_b16", op="append", fmt="int8", seqs=16, ctx=1000, chunk=4096, spread="uniform",
             chunk_spread="uniform", hkv=8, dim=128, lens_seed=2),
        # a short single request: the call's latency
        dict(name="decode_b1_l2048", op="decode", fmt="e4m3", seqs=1, len=2048, spread="full", heads=24, hkv=4,
             dim=256, lens_seed=3),
        # a small ragged batch
        dict(name="decode_b8_u8192", op="decode", fmt="int8", seqs=8, len=8192, spread="uniform", heads=24, hkv=4,
             dim=256, lens_seed=4),
        # one long document
        dict(name="decode_b1_l102400", op="decode", fmt="e4m3", seqs=1, len=102400, spread="full", heads=24, hkv=4,
             dim=256, lens_seed=5),
        # a large batch of very unlike lengths, smaller heads
        dict(name="decode_b64_loguniform", op="decode", fmt="e4m3", seqs=64, len=8192, spread="loguniform", heads=32,
             hkv=8, dim=128, lens_seed=6),
        # a short follow-up on a short cached prefix
        dict(name="prefix_b1_c500_q37", op="prefix", fmt="int8", seqs=1, ctx=500, chunk=37, spread="full",
             chunk_spread="full", heads=32, hkv=8, dim=128, lens_seed=7),
        # prompt chunks of a batch over long cached prefixes
        dict(name="prefix_b4_c8192_q512", op="prefix", fmt="e4m3", seqs=4, ctx=8192, chunk=512, spread="full",
             chunk_spread="full", heads=24, hkv=4, dim=256, lens_seed=8),
        # decoding that keeps the weights for a later eviction, 16-bit cache
        dict(name="weights_b8_u8192", op="weights", fmt="f16", seqs=8, len=8192, spread="uniform", heads=24, hkv=4,
             dim=256, lens_seed=9),
        # the same over an 8-bit cache, more heads
        dict(name="weights_b16_e4m3", op="weights", fmt="e4m3", seqs=16, len=16384, spread="uniform", heads=32, hkv=8,
             dim=128, lens_seed=10),
        # a batch over its budget: down to 1024 tokens a sequence, 16-bit cache
        dict(name="evict_b8_u8192", op="evict", fmt="f16", seqs=8, len=8192, spread="uniform", keep=1024, sinks=4,
             recent=256, hkv=4, dim=256, lens_seed=11),
        # one long document down to 16384 tokens, 8-bit cache
        dict(name="evict_b1_l102400", op="evict", fmt="e4m3", seqs=1, len=102400, spread="full", keep=16384, sinks=4,
             recent=1024, hkv=4, dim=256, lens_seed=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "prefix", "weights", "evict"])
    heads, hkv, dim = rng.choice([(24, 4, 256), (32, 8, 128), (8, 1, 64), (12, 12, 64), (10, 2, 128), (21, 3, 256)])
    case = dict(op=op, hkv=hkv, dim=dim, lens_seed=rng.randrange(1 << 30), seqs=_log_int(rng, 1, 64),
                spread=rng.choice(["full", "uniform", "loguniform"]))
    row = 2 * hkv * dim  # elements of K and V of one token
    if op == "append":
        case["fmt"] = rng.choice(["f16", "e4m3", "int8"])
        case["ctx"] = _log_int(rng, 1, 2048) - 1
        most = min(4096, 16 * 4096 * 2048 // (row * case["seqs"]))
        case["chunk"] = _log_int(rng, 1, max(1, most))
        case["chunk_spread"] = rng.choice(["full", "uniform"])
        return case
    if op == "prefix":
        case["fmt"] = rng.choice(["e4m3", "int8"])
        case["heads"] = heads
        case["seqs"] = _log_int(rng, 1, 16)
        case["chunk"] = _log_int(rng, 1, 512)
        most = 4 * 512 * 8192 * 24 * 256 // (case["seqs"] * case["chunk"] * heads * dim)
        case["ctx"] = _log_int(rng, 1, max(1, min(8192, most))) - 1
        case["chunk_spread"] = rng.choice(["full", "uniform"])
        return case
    top = 102400 if op in ("decode", "evict") else 32768
    case["len"] = _log_int(rng, 1, max(1, min(top, 102400 * 2048 // (row * case["seqs"]))))
    case["fmt"] = rng.choice(["e4m3", "int8"] if op == "decode" else ["f16", "e4m3", "int8"])
    if op == "evict":
        case["keep"] = _log_int(rng, 1, max(1, min(16384, case["len"])))
        case["sinks"] = rng.choice([0, 4, 16])
        case["recent"] = rng.choice([0, 1, 64, 500])
    else:
        case["heads"] = heads
    return case


def _lengths(case, key, spread, low):
    rng = random.Random(case["lens_seed"] * 2 + (key == "chunk"))
    top, n = case[key], case["seqs"]
    if spread == "full" or top <= low:
        return [top] * n
    if spread == "uniform":
        return [rng.randint(low, top) for _ in range(n)]
    return [_log_int(rng, max(1, low), top) for _ in range(n)]


def work(case):
    hkv, dim = case["hkv"], case["dim"]
    el = 2 if case["fmt"] == "f16" else 1
    scales = 0 if case["fmt"] == "f16" else 8 * hkv / BS  # both scales, a token's share of its block's
    if case["op"] == "append":
        t = sum(_lengths(case, "chunk", case["chunk_spread"], 1))
        return {"bytes": int(t * (2 * hkv * dim * (2 + el) + scales)), "flops": 4 * t * hkv * dim}
    if case["op"] == "prefix":
        c, q = _lengths(case, "ctx", case["spread"], 0), _lengths(case, "chunk", case["chunk_spread"], 1)
        keys = sum(a * b + b * (b + 1) // 2 for a, b in zip(c, q))
        io = sum(q) * dim * 2 * (2 * case["heads"] + 2 * hkv)
        return {"bytes": int(sum(c) * (2 * hkv * dim * el + scales) + io), "flops": 4 * keys * case["heads"] * dim}
    t = sum(_lengths(case, "len", case["spread"], 1))
    if case["op"] == "evict":
        k = sum(min(case["keep"], n) for n in _lengths(case, "len", case["spread"], 1))
        return {"bytes": int(4 * t * hkv + k * (2 * (2 * hkv * dim * el + scales) + 8 * hkv)), "flops": t * hkv}
    more = 8 * t * hkv if case["op"] == "weights" else 0
    return {"bytes": int(t * (2 * hkv * dim * el + scales) + more + 4 * case["seqs"] * case["heads"] * dim),
            "flops": 4 * t * case["heads"] * dim}


# ---------------------------------------------------------------- the 8-bit formats

def _scale_of(amax, fmt):
    """The block scale of a largest magnitude (32 bits; 0 for 0)."""
    if fmt == "e4m3":  # smallest 2^k with 448 2^k >= amax; 448 = 0.875 2^9
        m, e = torch.frexp(amax)
        s = torch.ldexp(torch.ones_like(amax), torch.where(m <= 0.875, e - 9, e - 8).to(torch.int32))
    else:  # amax / 127, rounded up to 8 significant bits
        # (a tensor divisor: by a number, torch multiplies by its rounded reciprocal)
        bits = (amax / torch.full_like(amax, 127.0)).contiguous().view(torch.int32)
        s = torch.bitwise_and(bits + 0xFFFF, -0x10000).view(torch.float32)
    return torch.where(amax > 0, s, torch.zeros_like(s))


def _codes(x, s, fmt):
    """Values x (32 bits) in units of s, rounded to the format's nearest (ties to even), saturated."""
    t = torch.where(s > 0, x / torch.where(s > 0, s, torch.ones_like(s)), x)
    if fmt == "e4m3":
        return t.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.nan_to_num(torch.round(t), nan=0.0).clamp(-127.0, 127.0).to(torch.int8).view(torch.uint8)


def _raw(cache):
    return cache.view(torch.uint8) if cache.element_size() == 1 else cache


def _values(raw, fmt):
    """The values of codes (taken from _raw) in 32 bits, without their scales."""
    return raw.float() if fmt == "f16" else raw.view(DTYPES[fmt]).float()


# ---------------------------------------------------------------- inputs

def _pool(case, blocks, gen):
    """A cache of `blocks` blocks as earlier appends left it, its last block unused: heads of unlike magnitude, 1 %
    of the tokens with larger keys."""
    hkv, dim, fmt = case["hkv"], case["dim"], case["fmt"]
    dev = "cuda"
    out = []
    heads = 0.5 + 1.5 * torch.rand(2, hkv, 1, 1, generator=gen, device=dev)
    for kv in range(2):
        cache = torch.empty(blocks, hkv, BS, dim, dtype=torch.float16 if fmt == "f16" else torch.uint8, device=dev)
        scales = torch.zeros(blocks, hkv, device=dev)
        step = max(1, (1 << 25) // (hkv * BS * dim))
        for at in range(0, blocks, step):
            n = min(step, blocks - at)
            x = torch.randn(n, hkv, BS, dim, generator=gen, device=dev) * heads[kv]
            if kv == 0:
                x = x * torch.where(torch.rand(n, 1, BS, 1, generator=gen, device=dev) < 0.01, 3.0, 1.0)
            x = x.half()
            if fmt == "f16":
                cache[at:at + n] = x
            else:
                x = x.float()
                s = _scale_of(x.abs().amax(dim=(2, 3)), fmt)
                cache[at:at + n] = _codes(x, s[:, :, None, None], fmt)
                scales[at:at + n] = s
        out.append((cache if fmt == "f16" else cache.view(DTYPES[fmt]), None if fmt == "f16" else scales))
    return out[0][0], out[1][0], out[0][1], out[1][1]


def _tables(lens, gen_cpu, spare=1):
    need = [-(-n // BS) for n in lens]
    total = sum(need) + spare
    perm = torch.randperm(total - spare, generator=gen_cpu).to(torch.int32)
    tables = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        tables[b, :n] = perm[at:at + n]
        at += n
    return tables.cuda(), total


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    hkv, dim, op = case["hkv"], case["dim"], case["op"]
    st = {"case": case, "scale": 1.0 / math.sqrt(dim)}
    half = lambda *s: torch.randn(*s, generator=gen, device="cuda").half()
    if op in ("append", "prefix"):
        ctx = _lengths(case, "ctx", case["spread"], 0)
        new = _lengths(case, "chunk", case["chunk_spread"], 1)
        loc = [0]
        for n in new:
            loc.append(loc[-1] + n)
        cover = [a + b for a, b in zip(ctx, new)] if op == "append" else ctx
        st["tables"], blocks = _tables(cover, cpu)
        st["k"], st["v"], st["ks"], st["vs"] = _pool(case, blocks, gen)
        # keys and values that now and then outgrow the scale of the block they join
        st["k_new"] = half(loc[-1], hkv, dim) * (1 + (torch.rand(loc[-1], 1, 1, generator=gen, device="cuda") < 0.1).half())
        st["v_new"] = half(loc[-1], hkv, dim)
        st["ctx"], st["loc"] = _ints(ctx), _ints(loc)
        st["max_ctx"], st["max_new"] = max(ctx), max(new)
        if op == "prefix":
            st["q"] = half(loc[-1], case["heads"], dim)
            st["out"] = torch.empty_like(st["q"])
        return st
    lens = _lengths(case, "len", case["spread"], 1)
    st["tables"], blocks = _tables(lens, cpu)
    st["k"], st["v"], st["ks"], st["vs"] = _pool(case, blocks, gen)
    st["lens"], st["max_len"] = _ints(lens), max(lens)
    if op in ("decode", "weights"):
        st["q"] = half(len(lens), case["heads"], dim)
        st["out"] = torch.empty_like(st["q"])
    if op != "decode":
        # the weight that earlier steps left: heavy-tailed, most of it on few tokens, some exactly equal
        w = torch.rand(len(lens), hkv, st["max_len"], generator=gen, device="cuda") ** 8
        st["w_in"] = torch.where(w < 1e-6, torch.zeros_like(w), w)
    if op == "weights":
        st["w_out"] = torch.zeros_like(st["w_in"])
    if op == "evict":
        kept = [min(n, case["keep"]) for n in lens]
        st["dst_tables"], blocks = _tables(kept, cpu)
        st["max_keep"] = max(kept)
        st["keep"] = _ints([case["keep"]] * len(lens)).clamp(max=st["max_keep"])
        shape = (blocks, hkv, BS, dim)
        st["dst_k"], st["dst_v"] = (torch.zeros(shape, dtype=torch.uint8 if st["ks"] is not None else torch.float16,
                                                device="cuda").view(st["k"].dtype) for _ in range(2))
        st["dst_ks"], st["dst_vs"] = ((torch.zeros(blocks, hkv, device="cuda") for _ in range(2))
                                      if st["ks"] is not None else (None, None))
        st["kept"] = torch.full((len(lens), hkv, st["max_keep"]), -1, dtype=torch.int32, device="cuda")
        st["new_lens"] = torch.zeros(len(lens), dtype=torch.int32, device="cuda")
        st["w_out"] = torch.zeros(len(lens), hkv, st["max_keep"], device="cuda")
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    op = st["case"]["op"]
    if own:
        return _run_own(st)
    if op == "append":
        return _append(st)
    if op == "prefix":
        return _prefix(st)
    if op == "evict":
        return _evict(st)
    return _decode(st, op == "weights")


def _run_own(st):
    from paged_kv_cache_308_gb300 import binding as pb
    case, op = st["case"], st["case"]["op"]
    cache = (st["k"], st["v"], st["ks"], st["vs"])
    if op == "append":
        pb.pa_kv_append(*cache, st["k_new"], st["v_new"], st["tables"], st["ctx"], st["loc"],
                        max_query_len=st["max_new"])
        return {"k": st["k"], "v": st["v"], "ks": st["ks"], "vs": st["vs"]}
    if op == "prefix":
        if "ws" not in st:
            st["ws"] = torch.empty(pb.pa_kv_prefix_workspace_size(
                case["seqs"], st["max_ctx"], case["hkv"], case["dim"], st["k"].dtype), dtype=torch.uint8, device="cuda")
        pb.pa_kv_prefix(st["out"], st["q"], st["k_new"], st["v_new"], *cache, st["tables"], st["ctx"], st["loc"],
                        st["scale"], max_context_len=st["max_ctx"], max_query_len=st["max_new"], workspace=st["ws"])
        return st["out"]
    if op == "evict":
        pb.pa_kv_evict(*cache, st["tables"], st["lens"], st["dst_k"], st["dst_v"], st["dst_ks"], st["dst_vs"],
                       st["dst_tables"], st["keep"], st["w_in"], st["kept"], st["new_lens"], st["w_out"],
                       max_seq_len=st["max_len"], max_keep_len=st["max_keep"], sinks=case["sinks"],
                       recent=case["recent"])
        return {"k": st["dst_k"], "v": st["dst_v"], "ks": st["dst_ks"], "vs": st["dst_vs"], "kept": st["kept"],
                "lens": st["new_lens"], "w": st["w_out"]}
    more = {"weights_in": st["w_in"], "weights_out": st["w_out"]} if op == "weights" else {}
    if "ws" not in st:
        st["ws"] = torch.empty(pb.pa_kv_decode_workspace_size(
            case["seqs"], st["max_len"], case["heads"], case["hkv"], case["dim"], st["k"].dtype,
            weights=op == "weights"), dtype=torch.uint8, device="cuda")
    pb.pa_kv_decode(st["out"], st["q"], *cache, st["tables"], st["lens"], st["scale"], max_seq_len=st["max_len"],
                    workspace=st["ws"], **more)
    return {"out": st["out"], "w": st["w_out"]} if op == "weights" else st["out"]


# ---------------------------------------------------------------- the plain forms

def _tokens(st, raw_scales):
    """The sequences' tokens [seqs, hkv, tokens of the table, dim] in 32 bits."""
    cache, scales = raw_scales
    ids = st["tables"].long().clamp(min=0)
    x = _values(_raw(cache)[ids], st["case"]["fmt"])
    if scales is not None:
        x = x * scales[ids][..., None, None]
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _softmax(s, mask):
    s = s.masked_fill(~mask, -math.inf)
    m = s.amax(dim=-1, keepdim=True)
    p = torch.exp(s - torch.where(m > -math.inf, m, torch.zeros_like(m))).masked_fill(~mask, 0.0)
    total = p.sum(dim=-1, keepdim=True)
    return p / torch.where(total > 0, total, torch.ones_like(total))


def _decode(st, weights):
    k, v = _tokens(st, (st["k"], st["ks"])), _tokens(st, (st["v"], st["vs"]))
    b, hkv, t, d = k.shape
    q = st["q"].float().view(b, hkv, -1, d)
    mask = (torch.arange(t, device="cuda") < st["lens"][:, None])[:, None, None]
    p = _softmax(torch.matmul(q, k.transpose(2, 3)) * st["scale"], mask)
    out = torch.matmul(p, v.masked_fill(~mask.squeeze(2)[..., None], 0.0)).view(b, -1, d).half()
    if not weights:
        return out
    n = st["max_len"]
    w = st["w_in"] + p.sum(dim=2)[..., :n]
    return {"out": out, "w": torch.where(mask[:, :, 0, :n], w, st["w_out"])}


def _prefix(st):
    case = st["case"]
    k, v = _tokens(st, (st["k"], st["ks"])), _tokens(st, (st["v"], st["vs"]))
    b, hkv, t, d = k.shape
    i = torch.arange(st["max_new"], device="cuda")
    loc = st["loc"].long()
    mine = i < (loc[1:] - loc[:-1])[:, None]
    at = torch.where(mine, loc[:-1, None] + i, torch.zeros_like(i))
    k = torch.cat([k, st["k_new"][at].float().transpose(1, 2)], dim=2)
    v = torch.cat([v, st["v_new"][at].float().transpose(1, 2)], dim=2)
    q = st["q"][at].float().view(b, -1, hkv, case["heads"] // hkv, d).permute(0, 2, 3, 1, 4)
    seen = torch.cat([(torch.arange(t, device="cuda") < st["ctx"][:, None])[:, None].expand(b, len(i), t),
                      (i[:, None] >= i)[None].expand(b, len(i), len(i))], dim=2)[:, None, None]
    p = _softmax(torch.matmul(q, k[:, :, None].transpose(3, 4)) * st["scale"], seen)
    v = v.masked_fill(~torch.cat([torch.arange(t, device="cuda") < st["ctx"][:, None], mine], dim=1)[:, None, :, None], 0.0)
    out = torch.matmul(p, v[:, :, None]).permute(0, 3, 1, 2, 4).reshape(b, len(i), -1, d).half()
    res = torch.empty(st["q"].shape[0] + 1, *st["q"].shape[1:], dtype=torch.float16, device="cuda")
    res[torch.where(mine, at, torch.full_like(at, st["q"].shape[0]))] = out
    return res[:-1]


def _append(st):
    case, fmt = st["case"], st["case"]["fmt"]
    ctx, loc = st["ctx"].long(), st["loc"].long()
    first = ctx // BS
    tiles = (st["max_new"] + BS - 2) // BS + 1
    blk = first[:, None] + torch.arange(tiles, device="cuda")
    pos = blk[..., None] * BS + torch.arange(BS, device="cuda")
    end = (ctx + loc[1:] - loc[:-1])[:, None, None]
    new = (pos >= ctx[:, None, None]) & (pos < end)
    old = (pos < ctx[:, None, None])[:, :, None, :]
    at = torch.where(new, loc[:-1, None, None] + pos - ctx[:, None, None], torch.zeros_like(pos))
    touched = new.any(dim=2)
    width = st["tables"].shape[1]
    spare = st["k"].shape[0] - 1
    phys = torch.gather(st["tables"].long(), 1, blk.clamp(max=width - 1))
    phys = torch.where(touched, phys, torch.full_like(phys, spare))
    new = new[:, :, None, :]
    res = {"k": st["k"], "v": st["v"], "ks": st["ks"], "vs": st["vs"]}
    res["k"], res["ks"] = _append_one(st["k"], st["ks"], st["k_new"], phys, at, new, old, touched, fmt)
    res["v"], res["vs"] = _append_one(st["v"], st["vs"], st["v_new"], phys, at, new, old, touched, fmt)
    return res


def _append_one(cache, scales, x, phys, at, new, old, touched, fmt):
    raw = _raw(cache)
    x = x[at].transpose(2, 3)  # [seqs, tiles, hkv, 16, dim]
    there = raw[phys]
    if fmt == "f16":
        raw[phys] = torch.where(new[..., None], x, there)
        return cache, scales
    x = x.float()
    amax = torch.where(new[..., None] & x.isfinite(), x.abs(), torch.zeros_like(x)).amax(dim=(3, 4))
    s0 = torch.where(old.any(dim=3), scales[phys], torch.zeros_like(amax))
    s1 = torch.maximum(s0, _scale_of(amax, fmt))
    s1e, s0e = s1[..., None, None], s0[..., None, None]
    again = torch.where(s1e > s0e, _codes(_values(there, fmt) * s0e, s1e, fmt), there)
    codes = torch.where(new[..., None], _codes(x, s1e, fmt), torch.where(old[..., None], again, there))
    raw[phys] = torch.where(touched[:, :, None, None, None], codes, there)
    scales[phys] = torch.where(touched[..., None], s1, scales[phys])
    return cache, scales


def _evict(st):
    case, fmt = st["case"], st["case"]["fmt"]
    w = st["w_in"]
    b, hkv, n = w.shape
    lens = st["lens"].long()[:, None, None]
    pos = torch.arange(n, device="cuda")
    k = torch.minimum(st["keep"].long()[:, None, None], lens)
    recent = k.clamp(max=case["recent"])
    sinks = torch.minimum(k - recent, torch.full_like(k, case["sinks"]))
    cls = (pos < lens).int() + ((pos < lens) & ((pos >= lens - recent) | (pos < sinks))).int()
    order = torch.sort(torch.where(w.isnan(), torch.full_like(w, -math.inf), w), dim=2, descending=True, stable=True)[1]
    again = torch.sort(torch.gather(cls.expand(b, hkv, n), 2, order), dim=2, descending=True, stable=True)[1]
    order = torch.gather(order, 2, again)
    i = torch.arange(st["max_keep"], device="cuda")
    take = torch.where(i < k, order[..., :st["max_keep"]], torch.full_like(order[..., :st["max_keep"]], n))
    kept = torch.sort(take, dim=2)[0]  # ascending positions, n past the last
    valid = i < k
    valid = valid.expand(b, hkv, -1)
    src = torch.where(valid, kept, torch.zeros_like(kept))
    blk = torch.gather(st["tables"].long()[:, None].expand(b, hkv, -1), 2, src // BS).clamp(min=0)
    head = torch.arange(hkv, device="cuda")[:, None].expand(b, hkv, st["max_keep"])
    spare = st["dst_k"].shape[0] - 1
    to = torch.gather(st["dst_tables"].long()[:, None].expand(b, hkv, -1), 2, (i // BS).expand(b, hkv, -1))
    to = torch.where(valid, to, torch.full_like(to, spare))
    res = {}
    for name in ("k", "v"):
        rows = _raw(st[name])[blk, head, src % BS]
        dst = _raw(st["dst_" + name])
        scales = st["dst_" + name + "s"]
        if scales is not None:
            s0 = torch.where(valid, st[name + "s"][blk, head], torch.zeros((), device="cuda"))
            pad = -s0.shape[2] % BS
            s1 = torch.nn.functional.pad(s0, (0, pad)).view(b, hkv, -1, BS).amax(dim=3)
            s1e = s1.repeat_interleave(BS, dim=2)[..., :s0.shape[2]]
            rows = _codes(_values(rows, fmt) * s0[..., None], s1e[..., None], fmt)
            scales[to, head] = torch.where(valid, s1e, torch.zeros_like(s1e))
        dst[to, head, (i % BS).expand(b, hkv, -1)] = torch.where(valid[..., None], rows, torch.zeros_like(rows))
        res[name], res[name + "s"] = st["dst_" + name], scales
    res["kept"] = torch.where(valid, kept, torch.full_like(kept, -1)).int()
    res["lens"] = k[:, 0, 0].int()
    res["w"] = torch.where(valid, torch.gather(w, 2, src), st["w_out"])
    return res


# ---------------------------------------------------------------- in 64 bits, from the definitions

def exact(case, seed):
    st = prepare(case, seed)
    f = {"append": _exact_append, "prefix": _exact_prefix, "evict": _exact_evict}.get(case["op"], _exact_decode)
    return f(st, case)


def _block64(cache, scales, fmt, ids):
    """Tokens of the blocks `ids` in order: [hkv, tokens, dim] in 64 bits."""
    x = (cache.view(torch.uint8)[ids].view(DTYPES[fmt]) if fmt != "f16" else cache[ids]).double()
    if scales is not None:
        x = x * scales[ids].double()[:, :, None, None]
    return x.transpose(0, 1).reshape(x.shape[1], -1, x.shape[3])


def _exact_decode(st, case):
    outs, w = [], st["w_out"].double() if case["op"] == "weights" else None
    for b, n in enumerate(st["lens"].tolist()):
        ids = st["tables"][b, :-(-n // BS)].long()
        k = _block64(st["k"], st["ks"], case["fmt"], ids)[:, :n]
        v = _block64(st["v"], st["vs"], case["fmt"], ids)[:, :n]
        q = st["q"][b].double().view(case["hkv"], -1, case["dim"])
        p = torch.softmax(q @ k.transpose(1, 2) * st["scale"], dim=2)
        outs.append((p @ v).reshape(-1, case["dim"]))
        if w is not None:
            w[b, :, :n] = st["w_in"][b, :, :n].double() + p.sum(dim=1)
    out = torch.stack(outs)
    return out if w is None else {"out": out, "w": w}


def _exact_prefix(st, case):
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    loc, g = st["loc"].tolist(), case["heads"] // case["hkv"]
    for b, c in enumerate(st["ctx"].tolist()):
        ids = st["tables"][b, :-(-c // BS)].long()
        new = slice(loc[b], loc[b + 1])
        n = loc[b + 1] - loc[b]
        causal = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
        mask = torch.cat([torch.ones(n, c, dtype=torch.bool, device="cuda"), causal], dim=1)
        for h in range(case["hkv"]):
            k = st["k_new"][new, h].double()
            v = st["v_new"][new, h].double()
            if c:
                one = lambda x, s: (x.view(torch.uint8)[ids, h].view(DTYPES[case["fmt"]]).double()
                                    * s[ids, h].double()[:, None, None]).reshape(-1, case["dim"])[:c]
                k, v = torch.cat([one(st["k"], st["ks"]), k]), torch.cat([one(st["v"], st["vs"]), v])
            for j in range(h * g, (h + 1) * g):
                s = (st["q"][new, j].double() @ k.T * st["scale"]).masked_fill(~mask, -math.inf)
                out[new, j] = torch.softmax(s, dim=1) @ v
    return out


def _scale64(amax, fmt):
    if amax == 0:
        return 0.0
    if fmt == "e4m3":
        k = math.floor(math.log2(amax / 448)) - 1
        while 448 * 2.0 ** k < amax:
            k += 1
        return 2.0 ** k
    e = math.frexp(amax / 127)[1] - 8
    return math.ceil(math.ldexp(amax / 127, -e)) * 2.0 ** e


def _round64(t, fmt):
    """The nearest number of the format (ties to even), saturated."""
    if fmt == "int8":
        return torch.round(t).clamp(-127, 127)
    e = torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6)))
    e = torch.where(2.0 ** (e + 1) <= t.abs(), e + 1, torch.where(2.0 ** e > t.abs().clamp(min=2.0 ** -6), e - 1, e))
    return (torch.round(t / 2.0 ** (e - 3)) * 2.0 ** (e - 3)).clamp(-448, 448)


def _exact_append(st, case):
    fmt = case["fmt"]
    if fmt == "f16" or st["k_new"].shape[0] > 4096:
        return None
    res, loc = {}, st["loc"].tolist()
    for name in ("k", "v"):
        codes = st[name].view(torch.uint8).view(DTYPES[fmt]).double()
        scales = st[name + "s"].double()
        for b, c in enumerate(st["ctx"].tolist()):
            at = c
            while at < c + loc[b + 1] - loc[b]:
                lo, hi = at % BS, min(BS, at % BS + c + loc[b + 1] - loc[b] - at)
                phys = int(st["tables"][b, at // BS])
                x = st[name + "_new"][loc[b] + at - c:loc[b] + at - c + hi - lo].double().transpose(0, 1)
                tops = x.abs().amax(dim=(1, 2)).tolist()
                for h, top in enumerate(tops):
                    s0 = float(scales[phys, h]) if lo else 0.0
                    s1 = max(s0, _scale64(top, fmt))
                    if s1 > s0 and lo:
                        codes[phys, h, :lo] = _round64(codes[phys, h, :lo] * s0 / x.new_tensor(s1), fmt)
                    codes[phys, h, lo:hi] = _round64(x[h] / x.new_tensor(s1), fmt) if s1 else 0.0
                    scales[phys, h] = s1
                at += hi - lo
        # codes in 8 whole bits have no rounding to be compared with
        res[name], res[name + "s"] = (codes if fmt == "e4m3" else None), scales
    return res


def _exact_evict(st, case):
    """The kept weights and the destination's scales; moved codes are compared as they are."""
    w64 = st["w_out"].double()
    w = st["w_in"].double().cpu()
    for b, n in enumerate(st["lens"].tolist()):
        k = min(int(st["keep"][b]), n)
        r = min(case["recent"], k)
        s = min(case["sinks"], k - r)
        for h in range(case["hkv"]):
            row = w[b, h, :n]
            mid = sorted(range(s, n - r), key=lambda t, v=row.tolist(): (-v[t], t))[:k - r - s]
            kept = sorted(list(range(s)) + mid + list(range(n - r, n)))
            w64[b, h, :k] = row[kept].cuda()
    return {"k": None, "v": None, "ks": None, "vs": None, "kept": None, "lens": None, "w": w64}
