"""Block allocation, rotary put and linear attention without a GPU: references against closed forms, argument
checks, workspace sizes, the binding's checks."""
import ctypes
import math

import pytest
import torch

import step_helpers as S
from paged_kv_cache_308_gb300 import binding as pb

FAKE = 0x100000  # an aligned non-null address that no call dereferences
BAD, UNSUP = pb.PA_ERR_INVALID_ARG, pb.PA_ERR_UNSUPPORTED


def alloc_args(nb=100, B=4, T=10, cols=8, bs=16, **p):
    at = {n: FAKE + 0x10000 * i for i, n in enumerate(["bt", "free", "count", "new_count", "held", "ctx", "q", "loc",
                                                        "lens", "slots", "pos"])}
    at.update(p)
    return pb.pa_kv_alloc_args(*at.values(), nb, B, T, cols, bs)


def apart(*names):
    """Addresses so far apart that no array of these tests reaches the next."""
    return {n: FAKE + (i + 1) * (1 << 28) for i, n in enumerate(names)}


def put_args(T=4, H=8, hkv=2, D=128, nb=10, bs=16, fmt=pb.PA_KV_F16, rot=128, top=100, pairs=0, strides=(0, 0, 0), **p):
    at = apart("kc", "vc", "q_out", "k_out", "q", "k", "v", "slots", "pos", "cs")
    at.update(p)
    cache = pb.pa_kv_cache(at["kc"], at["vc"], 0, 0, nb, hkv, D, bs, fmt)
    return pb.pa_kv_put_args(cache, at["q_out"], at["k_out"], at["q"], at["k"], at["v"], at["slots"], at["pos"], at["cs"],
                             *strides, T, H, rot, top, pairs)


def state(slots=5, hkv=4, D=128, states=FAKE):
    return pb.pa_linear_state(states, slots, hkv, D)


def ldecode_args(s=None, B=3, H=8, scale=0.1, **p):
    at = apart("out", "q", "k", "v", "g", "slots")
    at.update(p)
    return pb.pa_linear_decode_args(at["out"], at["q"], at["k"], at["v"], s or state(), at["g"], at["slots"], B, H, scale)


def lprefix_args(s=None, B=3, T=10, max_q=5, H=8, scale=0.1, **p):
    at = apart("out", "q", "k", "v", "g", "slots", "ctx", "loc")
    at.update(p)
    return pb.pa_linear_prefix_args(at["out"], at["q"], at["k"], at["v"], s or state(), at["g"], at["slots"], at["ctx"],
                                    at["loc"], B, T, max_q, H, scale)


def call(fn, a):
    if fn == "pa_linear_prefix":
        return pb.lib.pa_linear_prefix(ctypes.byref(a), None, 0, None)
    return getattr(pb.lib, fn)(ctypes.byref(a), None)


@pytest.mark.parametrize("fn", ["pa_kv_alloc", "pa_kv_put", "pa_linear_decode"])
def test_no_arguments_are_refused(fn):
    assert getattr(pb.lib, fn)(None, None) == BAD
    assert pb.lib.pa_linear_prefix(None, None, 0, None) == BAD


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), BAD), (dict(B=65536), BAD), (dict(T=-1), BAD), (dict(cols=-1), BAD), (dict(nb=-1), BAD),
    (dict(bs=0), BAD), (dict(bs=32), UNSUP), (dict(nb=1 << 27), UNSUP), (dict(T=(1 << 30) + 1), UNSUP),
    (dict(bt=0), BAD), (dict(free=0), BAD), (dict(count=0), BAD), (dict(new_count=0), BAD), (dict(ctx=0), BAD),
    (dict(q=0), BAD), (dict(loc=0), BAD), (dict(lens=0), BAD), (dict(slots=0), BAD), (dict(pos=0), BAD),
    (dict(held=FAKE + 2), BAD), (dict(lens=FAKE + 0x10000 * 8 + 1), BAD),
    # outputs over inputs and over each other
    (dict(lens=FAKE + 0x10000 * 5), BAD), (dict(lens=FAKE + 0x10000 * 4), BAD), (dict(loc=FAKE + 0x10000 * 6 + 12), BAD),
    (dict(slots=FAKE + 0x10000 * 10 + 36), BAD), (dict(new_count=FAKE + 0x10000 * 8 + 4), BAD),
    (dict(new_count=FAKE + 0x10000 * 5), BAD), (dict(free=FAKE + 0x10000 * 2 - 4), BAD), (dict(bt=FAKE + 0x10000), BAD),
    (dict(pos=FAKE + 0x10000 * 2), BAD)])
def test_alloc_refusals(kw, code):
    assert call("pa_kv_alloc", alloc_args(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), BAD), (dict(H=0), BAD), (dict(hkv=0), BAD), (dict(D=96), BAD), (dict(D=96, rot=96), UNSUP), (dict(bs=32), UNSUP),
    (dict(fmt=pb.PA_KV_E4M3), UNSUP), (dict(fmt=3), BAD), (dict(nb=-1), BAD), (dict(nb=1 << 27), UNSUP),
    (dict(rot=-2), BAD), (dict(rot=130), BAD), (dict(rot=33), BAD), (dict(top=-1), BAD), (dict(pairs=2), BAD),
    (dict(strides=(4, 0, 0)), BAD), (dict(strides=(0, 255, 0)), BAD), (dict(strides=(0, 0, 128)), BAD),
    (dict(strides=(-1024, 0, 0)), BAD), (dict(q=0), BAD), (dict(k=0), BAD), (dict(v=0), BAD), (dict(q_out=0), BAD),
    (dict(pos=0), BAD), (dict(slots=0), BAD), (dict(cs=0), BAD), (dict(cs=FAKE + 4), BAD), (dict(k_out=FAKE + 8), BAD),
    (dict(kc=0), BAD), (dict(vc=0), BAD), (dict(kc=FAKE + 8), BAD),
    (dict(q=FAKE, q_out=FAKE, strides=(2048, 0, 0)), BAD),
    (dict(k=FAKE, k_out=FAKE, strides=(0, 2048, 0)), BAD)])
def test_put_refusals(kw, code):
    assert call("pa_kv_put", put_args(**kw)) == code


LINEAR = [(dict(H=9), BAD), (dict(H=0), BAD), (dict(H=36), UNSUP), (dict(scale=math.nan), BAD), (dict(scale=math.inf), BAD),
          (dict(B=-1), BAD), (dict(B=65536), BAD), (dict(out=0), BAD), (dict(q=FAKE + 8), BAD), (dict(k=0), BAD),
          (dict(v=FAKE + 2), BAD), (dict(g=0), BAD), (dict(slots=FAKE + 1), BAD), (dict(s=state(D=96)), UNSUP),
          (dict(s=state(hkv=0)), BAD), (dict(s=state(slots=-1)), BAD), (dict(s=state(slots=1 << 31)), UNSUP),
          (dict(s=state(states=0)), BAD), (dict(s=state(states=FAKE + 4)), BAD)]


@pytest.mark.parametrize("kw,code", LINEAR)
def test_linear_refusals(kw, code):
    assert call("pa_linear_decode", ldecode_args(**kw)) == code
    assert call("pa_linear_prefix", lprefix_args(**kw)) == code


@pytest.mark.parametrize("kw,code", [(dict(T=-1), BAD), (dict(max_q=-1), BAD), (dict(max_q=0), BAD), (dict(ctx=0), BAD),
                                     (dict(loc=FAKE + 2), BAD), (dict(T=(1 << 30) + 1), UNSUP)])
def test_linear_prefix_refusals(kw, code):
    assert call("pa_linear_prefix", lprefix_args(**kw)) == code


Q, K, V, OUT = (apart("out", "q", "k", "v")[n] for n in ("q", "k", "v", "out"))


@pytest.mark.parametrize("fn,make", [("pa_linear_decode", ldecode_args), ("pa_linear_prefix", lprefix_args)])
def test_linear_arrays_that_overlap(fn, make):
    T = 3 if fn == "pa_linear_decode" else 10
    row = 128 * 2
    for kw in (dict(out=Q), dict(out=Q + T * 8 * row - 16), dict(q=OUT + T * 8 * row - 16), dict(out=K), dict(v=OUT),
               dict(s=state(states=OUT)), dict(s=state(states=K + 16)), dict(g=OUT), dict(slots=FAKE + 4),
               dict(s=state(slots=(1 << 31) - 1, hkv=1, D=256), H=8)):
        assert call(fn, make(**kw)) == BAD, kw
    # arrays next to each other are not refused for it
    if fn == "pa_linear_prefix":
        assert call(fn, make(out=Q - T * 8 * row, max_q=20)) == pb.PA_ERR_WORKSPACE
        assert call(fn, make(q=OUT + T * 8 * row, max_q=20)) == pb.PA_ERR_WORKSPACE


def test_put_arrays_that_overlap():
    at = apart("kc", "vc", "q_out", "k_out", "q", "k", "v", "slots", "pos", "cs")
    q_row, k_row = 8 * 128 * 2, 2 * 128 * 2
    for kw in (dict(q_out=at["q"] + q_row), dict(q_out=at["k"]), dict(k_out=at["v"]), dict(kc=at["k"]),
               dict(vc=at["v"] + 16), dict(k_out=at["kc"] + 10 * 16 * k_row - 16), dict(q_out=at["k_out"] - 16),
               dict(vc=at["kc"] + 16), dict(q_out=at["k"] + 4 * k_row - 16)):
        assert call("pa_kv_put", put_args(**kw)) == BAD, kw
    # a strided input reaches to its last token's row
    assert call("pa_kv_put", put_args(strides=(4096, 0, 0), q_out=at["q"] + 3 * 8192 + q_row - 16)) == BAD


# few new tokens a sequence go without a workspace: up to 9, 14 and 24 by head_dim
@pytest.mark.parametrize("dim,few", [(256, 9), (128, 14), (64, 24)])
def test_linear_prefix_workspace_size(dim, few):
    size = lambda B=3, T=1000, top=500, H=8, hkv=4, D=dim: pb.pa_linear_prefix_workspace_size(B, T, top, H, hkv, D)
    assert size(top=few) == 0 and size(top=few + 1) > 0 and size(top=1) == 0
    blocks = 3 + 1000 // 256  # one more for each sequence than whole blocks of 256 tokens
    states = blocks * 4 * dim * dim * 6
    assert states <= size() <= states * 1.02 + 16384
    assert size(T=1023) == size(T=1000) < size(T=1024) and size(B=4) > size() and size(hkv=8) > size()
    assert size(top=few + 1) == size()  # the sizes' sum counts, not the longest
    for bad in (dict(B=0), dict(B=-1), dict(B=65536), dict(T=0), dict(T=(1 << 30) + 1), dict(top=0), dict(H=0), dict(hkv=0),
                dict(hkv=65536), dict(D=96)):
        assert size(**bad) == 0, bad
    assert size(B=65535, T=1 << 30, top=1 << 30, H=8, hkv=8) > 1 << 32


def test_empty_calls_do_nothing():
    assert call("pa_kv_put", put_args(T=0, q=0, k=0, v=0)) == pb.PA_OK
    assert call("pa_linear_decode", ldecode_args(B=0, q=0)) == pb.PA_OK
    assert call("pa_linear_prefix", lprefix_args(B=0, q=0)) == pb.PA_OK
    assert call("pa_linear_prefix", lprefix_args(T=0, max_q=0, q=0)) == pb.PA_OK


def test_struct_sizes_match_the_header(tmp_path):
    """The ctypes structures have the C compiler's sizes."""
    import subprocess
    names = ["pa_kv_alloc_args", "pa_kv_put_args", "pa_linear_state", "pa_linear_decode_args", "pa_linear_prefix_args"]
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include "pa_decode.h"\nint main(){%s return 0;}' % "".join(
        'printf("%%zu\\n", sizeof(%s));' % n for n in names))
    import os
    subprocess.run(["gcc", "-I", os.path.dirname(pb.HEADER_PATH), str(src), "-o", str(tmp_path / "s")], check=True)
    sizes = [int(x) for x in subprocess.run([str(tmp_path / "s")], check=True, capture_output=True).stdout.split()]
    assert sizes == [ctypes.sizeof(getattr(pb, n)) for n in names]


def test_new_constants_match_the_header():
    text = open(pb.HEADER_PATH).read()
    for name in ("PA_DEV_NO_BLOCKS", "PA_DEV_BAD_DECAY"):
        assert f"{name} = {getattr(pb, name)}" in text


def test_linear_reference_is_the_recurrence():
    g = torch.Generator().manual_seed(1)
    T, H, hkv, D = 9, 4, 2, 8
    q, k, v = (torch.randn(T, n, D, generator=g).half() for n in (H, hkv, hkv))
    s0, decay = torch.randn(hkv, D, D, generator=g), torch.tensor([-0.3, -math.inf])
    out, st, ob, sb = S.linear(q, k, v, s0, decay, 0.25)
    s = s0.double().clone()
    for t in range(T):
        for h in range(hkv):
            s[h] = s[h] * math.exp(float(decay[h])) + k[t, h].double()[:, None] * v[t, h].double()
            for j in range(2 * h, 2 * h + 2):
                want = 0.25 * q[t, j].double() @ s[h]
                assert torch.allclose(out[t, j], want, rtol=1e-12, atol=1e-12)
    assert torch.allclose(st, s, rtol=1e-12, atol=1e-12)
    assert bool((ob > 0).all()) and bool((sb >= 0).all())


def test_alloc_reference():
    # two blocks come back (3 and 5), then one is taken: the last given back
    got, short = S.alloc([[1, 3], [5, -1], [7, -1]], [2, 9, -1, -1], 2, [30, 10, 16], [3, 0, 16], [0, 0, 2], 3)
    assert not short and got["count"] == 3 and got["free"] == [2, 9, 3, 5] and got["tables"][2] == [7, 5]
    assert got["slots"] == [80, 81, -1] and got["positions"] == [16, 17, -1] and got["lens"] == [3, 0, 18]
    _, short = S.alloc([[-1, -1]], [4, -1], 1, [0], [0], [17], 17)
    assert short


def test_rotate_reference():
    x = torch.tensor([[[1.0, 2.0, 3.0, 4.0]]]).half()
    table = torch.tensor([[0.0, 0.6, 1.0, 0.8]])  # cos 0, 0.6; sin 1, 0.8
    y, _ = S.rotate(x, torch.tensor([0]), table, False)
    assert torch.allclose(y, torch.tensor([[[-3.0, 2 * 0.6 - 4 * 0.8, 1.0, 4 * 0.6 + 2 * 0.8]]]).double(), atol=1e-6)
    y, _ = S.rotate(x, torch.tensor([0]), table, True)
    assert torch.allclose(y, torch.tensor([[[-2.0, 1.0, 3 * 0.6 - 4 * 0.8, 4 * 0.6 + 3 * 0.8]]]).double(), atol=1e-6)
