"""Rotary positions on the GPU, against the formula in 64 bits.

Tolerances: sine and cosine of an angle that is exact to 2^-34 of a turn carry fp32 errors of about 2^-23, each product and
the sum another 2^-24; bf16 outputs one rounding, 2^-9 of the value at most.  |x cos - y sin| has terms of size |x| + |y|, so
|out - exact| <= 4e-7 factor (|x| + |y|) + half a step of the output's type.
"""
import math

import pytest
import torch

from speculative_decoding_eagle_gb300 import binding as E

pytestmark = pytest.mark.gpu
DT = {"bf16": (E.ET_BF16, torch.bfloat16), "f32": (E.ET_F32, torch.float32)}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_eagle_gb300 import build_lib
    build_lib.build()
    E.load()


def exact(x, pos, freq, factor, rot, layout):
    t = x.double()
    a = pos.double()[:, None, None] * freq.double()
    c, s = torch.cos(a) * factor, torch.sin(a) * factor
    i = torch.arange(rot // 2, device=x.device)
    p, q = (i, i + rot // 2) if layout == E.ET_ROTARY_HALF else (2 * i, 2 * i + 1)
    y, size = t.clone(), torch.zeros_like(t)
    y[..., p] = t[..., p] * c - t[..., q] * s
    y[..., q] = t[..., q] * c + t[..., p] * s
    size[..., p] = size[..., q] = t[..., p].abs() + t[..., q].abs()
    return y, size


def check(out, x, pos, freq, factor, rot, layout):
    want, size = exact(x, pos, freq, factor, rot, layout)
    there = pos >= 0
    eps = torch.finfo(out.dtype).eps / 2
    err = (out.double() - want).abs()[there]
    bound = (4e-7 * factor * size + eps * want.abs())[there]
    assert bool((err <= bound).all()), float((err - bound).max())
    same = out[there][..., rot:] == x[there][..., rot:]
    assert bool(same.all())                               # the dims behind are copied bit by bit
    assert bool((out[~there] == 7).all())                 # rows without a token are left alone


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", [E.ET_ROTARY_HALF, E.ET_ROTARY_PAIRS])
@pytest.mark.parametrize("rows,Hq,Hkv,d,rot", [
    (1, 1, 0, 16, 16), (1, 4, 4, 64, 64), (61, 32, 32, 128, 128), (7, 5, 1, 128, 32), (33, 3, 2, 72, 48), (5, 2, 1, 40, 16),
    (13, 8, 8, 256, 64), (9, 1, 1, 512, 512), (2500, 3, 1, 128, 96)])
def test_matches_the_formula(rows, Hq, Hkv, d, rot, layout, dtype):
    et, dt = DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(rows + d)
    x = torch.randn(rows, Hq + 2 * Hkv + 1, d, generator=g, device="cuda").to(dt)  # a projection's output, q and k inside it
    q, k = x[:, :Hq], x[:, Hq:Hq + Hkv]
    pos = torch.randint(-1, 200000, (rows,), generator=g, device="cuda", dtype=torch.int32)
    freq, factor = E.et_rotary_frequencies(rot, 10000.0, E.ET_ROPE_RAMP, 8.0)
    freq = freq.cuda()
    qo = torch.full((rows, Hq, d), 7.0, dtype=dt, device="cuda")
    ko = torch.full((rows, Hkv, d), 7.0, dtype=dt, device="cuda")
    shape = E.RotaryShape(rows=rows, Hq=Hq, Hkv=Hkv, d=d, rot=rot, layout=layout, dtype=et, factor=factor)
    E.et_rotary(shape, pos, freq, q, qo, k=k if Hkv else None, k_out=ko if Hkv else None)
    torch.cuda.synchronize()
    check(qo, q, pos, freq, factor, rot, layout)
    if Hkv:
        check(ko, k, pos, freq, factor, rot, layout)


def test_far_positions_lose_nothing():
    pos = torch.tensor([0, 1, 2 ** 24 + 1, 2 ** 30 + 7, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    freq, _ = E.et_rotary_frequencies(64, 500000.0)
    freq = freq.cuda()
    x = torch.randn(5, 2, 64, device="cuda")
    out = torch.full_like(x, 7.0)
    E.et_rotary(E.RotaryShape(rows=5, Hq=2, d=64, dtype=E.ET_F32), pos, freq, x, out)
    torch.cuda.synchronize()
    # the angle in exact integers: freq as a multiple of 2^-80 of a turn, times the position, modulo a turn
    turn = [int(f * 2 ** 100 // 1) for f in freq.tolist()]
    two_pi = int(math.pi * 2 ** 60) * 2 ** 41 // 1  # 2 pi 2^100 to 53 bits: as the table's own products have it
    a = torch.tensor([[(t * p % two_pi) / two_pi for t in turn] for p in pos.tolist()], dtype=torch.float64, device="cuda")
    c, s = torch.cos(2 * math.pi * a)[:, None], torch.sin(2 * math.pi * a)[:, None]
    t = x.double()
    want = torch.cat([t[..., :32] * c - t[..., 32:] * s, t[..., 32:] * c + t[..., :32] * s], -1)
    size = (t[..., :32].abs() + t[..., 32:].abs()).repeat(1, 1, 2)
    # freq / 2 pi carries 2^-53 of itself, at most 2^-55 of a turn at freq = 1, 2^31 times: 2^-24 of a turn, 4e-7
    assert bool(((out.double() - want).abs() <= (4e-7 + 2 * math.pi * 2.0 ** -23) * size).all())


def test_in_place_and_inverse():
    x = torch.randn(40, 6, 128, device="cuda").to(torch.bfloat16)
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    freq = E.et_rotary_frequencies(128)[0].cuda()
    shape = E.RotaryShape(rows=40, Hq=6, d=128)
    apart, back = torch.empty_like(x), torch.empty_like(x)
    E.et_rotary(shape, pos, freq, x, apart)
    E.et_rotary(shape, pos, -freq, apart, back)          # the angles turned back
    y = x.clone()
    E.et_rotary(shape, pos, freq, y, y)
    torch.cuda.synchronize()
    assert torch.equal(y, apart)
    assert float((back.float() - x.float()).abs().max()) <= 3 * 2.0 ** -9 * float(x.abs().max()) * 2


def test_captured_on_a_side_stream():
    x, out = torch.randn(9, 4, 64, device="cuda"), torch.zeros(9, 4, 64, device="cuda")
    pos = torch.zeros(9, dtype=torch.int32, device="cuda")
    freq = E.et_rotary_frequencies(64)[0].cuda()
    shape = E.RotaryShape(rows=9, Hq=4, d=64, dtype=E.ET_F32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    E.et_rotary(shape, pos, freq, x, out, stream=s)
    s.synchronize()
    assert torch.equal(out, x)                            # position 0
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        E.et_rotary(shape, pos, freq, x, out)
    pos.copy_(torch.arange(100, 109, dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    check(out, x, pos, freq, 1.0, 64, E.ET_ROTARY_HALF)


def test_tree_rows_at_the_trees_positions():
    """posids of et_tree_mask_posids go straight in: siblings are turned alike."""
    B, n = 2, 8
    cfg = E.TreeCfg(B=B, V=100, depth=2, topk=4, m=4, n=n)
    tree = E.TreeBuffers.allocate(cfg)
    tree.flat_parent.copy_(torch.tensor([[-1, 0, 0, 0, 0, 1, 1, 2, 2]] * B, dtype=torch.int32))
    tree.flat_depth.copy_(torch.tensor([[0, 1, 1, 1, 1, 2, 2, 2, 2]] * B, dtype=torch.int32))
    plen = torch.tensor([100, 7], dtype=torch.int32, device="cuda")
    mask, posids = torch.zeros(B, 9, 1, dtype=torch.int64, device="cuda"), torch.zeros(B, 9, dtype=torch.int32, device="cuda")
    E.et_tree_mask_posids(cfg, tree, plen, mask, posids)
    x = torch.ones(B * 9, 1, 64, device="cuda")
    out = torch.zeros_like(x)
    freq = E.et_rotary_frequencies(64)[0].cuda()
    E.et_rotary(E.RotaryShape(rows=B * 9, Hq=1, d=64, dtype=E.ET_F32), posids.view(-1), freq, x, out)
    torch.cuda.synchronize()
    assert posids.tolist() == [[100, 101, 101, 101, 101, 102, 102, 102, 102], [7, 8, 8, 8, 8, 9, 9, 9, 9]]
    o = out.view(B, 9, 64)
    assert torch.equal(o[:, 1], o[:, 4]) and torch.equal(o[:, 5], o[:, 8]) and not torch.equal(o[:, 0], o[:, 1])
    check(out, x, posids.view(-1), freq, 1.0, 64, E.ET_ROTARY_HALF)
