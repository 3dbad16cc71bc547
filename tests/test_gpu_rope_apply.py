"""GPU tests of the scaled RoPE tables and of llama_rope_apply (marked gpu).

Tables against their rules in 64 bits; rotations against 64-bit pairs, over
both pair layouts, parts of the head, both types, strided inputs and outputs
and the transposed map, which is also checked as a gradient (by the adjoint
identity and by differences).

Tolerances.  A table entry is formed in fp64 and rounded once to fp32 (half a
step, 2^-24 of a value of at most `gain`); one more such step is left for a
reduced argument held in fp32, and the angle itself is good to 64 steps of
2^-53 of its size (the frequency's power, product and quotient).  A rotation
rounds two products and a sum in fp32 (2^-24 of |a c| + |z s| each, three at
most) and then once to the type (2^-8 of the value in bf16).
"""
import math

import numpy as np
import pytest
import torch

from llama_gqa_causal_b200 import api

pytestmark = pytest.mark.gpu

DEV = "cuda"
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def banded(D, theta, factor, original, low, high):
    out = []
    for i in range(D // 2):
        w = theta ** (-2.0 * i / D)
        turns = original * w / (2 * math.pi)
        keep = min(1.0, max(0.0, (turns - low) / (high - low)))
        out.append(w * keep + w / factor * (1 - keep))
    return np.array(out), 1.0


def yarn(D, theta, factor, original, fast, slow, gain):
    def d(beta):
        return D * math.log(original / (2 * math.pi * beta)) / (2 * math.log(theta))
    lo, hi = max(math.floor(d(fast)), 0), min(math.ceil(d(slow)), D - 1)
    out = []
    for i in range(D // 2):
        w = theta ** (-2.0 * i / D)
        ramp = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
        out.append(w / factor * ramp + w * (1 - ramp))
    return np.array(out), gain


def check_table(got, pos, freqs, gain):
    p = pos.cpu().double().numpy().reshape(-1, 1)
    angle = p * np.concatenate([freqs, freqs])
    tol = gain * 2 * 2.0 ** -24 + gain * np.abs(angle) * 64 * 2.0 ** -53
    for t, want in zip(got, (np.cos(angle) * gain, np.sin(angle) * gain)):
        assert t.dtype == torch.float32 and t.shape == pos.shape + (2 * len(freqs),)
        err = np.abs(t.cpu().double().numpy().reshape(want.shape) - want)
        assert (err <= tol).all(), float((err - tol).max())


POSITIONS = {
    "one": [0],
    "odd": [5, 0, 131071, 1, 77, 4096, 8191],
    "far": [1 << 20, (1 << 31) - 1, 1 << 33, -3],
}


@pytest.mark.parametrize("where", POSITIONS)
@pytest.mark.parametrize("D", [2, 20, 64, 96, 128, 512])
def test_tables_follow_their_rules(D, where):
    pos = torch.tensor(POSITIONS[where], device=DEV)
    for theta, factor, original in ((10000.0, 8.0, 8192), (500000.0, 1.0, 77), (1e6, 40.0, 4096)):
        got = api.rope_table_banded(pos, D, theta, factor=factor, original_len=original,
                                    low_freq_factor=1.0, high_freq_factor=4.0)
        check_table(got, pos, *banded(D, theta, factor, original, 1.0, 4.0))
        got = api.rope_table_yarn(pos, D, theta, factor=factor, original_len=original)
        check_table(got, pos, *yarn(D, theta, factor, original, 32.0, 1.0,
                                    0.1 * math.log(factor) + 1.0))
        got = api.rope_table_yarn(pos, D, theta, factor=factor, original_len=original,
                                  beta_fast=16.0, beta_slow=0.5, attn_factor=1.0)
        check_table(got, pos, *yarn(D, theta, factor, original, 16.0, 0.5, 1.0))


def test_tables_of_a_batch_of_prompts():
    pos = torch.arange(2 * 3001, device=DEV).view(2, 3001) * 21 - 5
    got = api.rope_table_yarn(pos, 128, 1e4, factor=16.0, original_len=4096)
    check_table(got, pos, *yarn(128, 1e4, 16.0, 4096, 32.0, 1.0, 0.1 * math.log(16.0) + 1.0))
    got = api.rope_table_banded(pos, 64, 1e4, factor=4.0, original_len=2048)
    check_table(got, pos, *banded(64, 1e4, 4.0, 2048, 1.0, 4.0))


def test_unscaled_banded_table_is_the_plain_one():
    pos = torch.randint(0, 40000, (513,), device=DEV)
    one = api.rope_table_banded(pos, 128, 1e4, factor=1.0, original_len=4096)
    plain = api.rope_table(pos, 128, 1e4)
    for a, b in zip(one, plain):  # each within a step of the same value
        assert (a - b).abs().max().item() <= 3 * 2.0 ** -24


# ---------------------------------------------------------------- rotation
def pairs(R, interleaved):
    i = torch.arange(R // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)


def expected(x, cos, sin, interleaved, transpose):
    """The rotation in 64 bits, and what its rounding may be off by."""
    R = cos.shape[-1]
    first, second = pairs(R, interleaved)
    c, s = (t[..., None, :R // 2].double() for t in (cos, sin))
    if transpose:
        s = -s
    y = x.double().clone()
    a, z = y[..., first].clone(), y[..., second].clone()
    y[..., first], y[..., second] = a * c - z * s, z * c + a * s
    tol = torch.zeros_like(y)
    tol[..., first] = 3 * 2.0 ** -24 * ((a * c).abs() + (z * s).abs())
    tol[..., second] = 3 * 2.0 ** -24 * ((z * c).abs() + (a * s).abs())
    return y, tol + HALF_STEP[x.dtype] * y.abs() * (y != x.double())


def tables(tokens, R, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    a = torch.rand(*tokens, R // 2, generator=g, device=DEV, dtype=torch.float64) * 400 - 200
    a = torch.cat([a, a], -1)
    return a.cos().float(), a.sin().float()


def check(x, y, cos, sin, interleaved, transpose):
    want, tol = expected(x, cos, sin, interleaved, transpose)
    assert y.dtype == x.dtype and y.shape == x.shape
    assert ((y.double() - want).abs() <= tol).all()


SHAPES = [
    # tokens, heads, kv heads, head_dim, rotary_dim
    ((1,), 1, 1, 2, 2),
    ((1,), 64, 8, 128, 128),
    ((7,), 5, 1, 64, 64),
    ((3, 11), 4, 2, 128, 64),
    ((2, 129), 9, 3, 96, 24),
    ((5, 1), 28, 4, 80, 80),
    ((1, 33), 3, 3, 80, 20),
    ((2, 17), 2, 2, 256, 128),
    ((130,), 8, 8, 72, 16),
    ((1, 2049), 32, 8, 128, 128),
    ((9,), 3, 1, 10, 6),
    ((3,), 7, 7, 576, 64),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[0])) + "h%dk%dd%dr%d" % s[1:])
def test_rotation_both_ways(shape, interleaved, dtype):
    tokens, H, Hkv, D, R = shape
    g = torch.Generator(device=DEV).manual_seed(D + R)
    q = torch.randn(*tokens, H, D, generator=g, device=DEV).to(dtype)
    k = torch.randn(*tokens, Hkv, D, generator=g, device=DEV).to(dtype)
    cos, sin = tables(tokens, R)
    kept = q.clone(), k.clone()
    for transpose in (False, True):
        yq, yk = api.rope_apply(q, k, cos, sin, interleaved=interleaved, transpose=transpose)
        check(q, yq, cos, sin, interleaved, transpose)
        check(k, yk, cos, sin, interleaved, transpose)
        alone, none = api.rope_apply(q, None, cos, sin, interleaved=interleaved, transpose=transpose)
        assert none is None and torch.equal(alone, yq)
    assert torch.equal(q, kept[0]) and torch.equal(k, kept[1])
    # in place
    api.rope_apply(q, k, cos, sin, interleaved=interleaved, out=(q, k))
    check(kept[0], q, cos, sin, interleaved, False)
    check(kept[1], k, cos, sin, interleaved, False)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("D,R,pad", [(128, 128, 0), (64, 32, 8), (128, 64, 3), (80, 40, 1)])
def test_strided_views_in_and_out(D, R, pad, interleaved, dtype):
    """q and k inside a fused projection's rows, k's output inside a cache; what lies
    between is left as it was."""
    b, s, H, Hkv, L = 2, 37, 6, 2, 50
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(b, s, (H + 2 * Hkv) * D + pad, generator=g, device=DEV).to(dtype)
    q = x[..., :H * D].unflatten(-1, (H, D))
    k = x[..., pad + H * D:pad + (H + Hkv) * D].unflatten(-1, (Hkv, D))
    cos, sin = tables((b, s), R)
    cache = torch.full((b, Hkv, L, D), 7.0, device=DEV, dtype=dtype)
    rows = cache[:, :, 5:5 + s].transpose(1, 2)
    before = x.clone()
    yq, yk = api.rope_apply(q, k, cos, sin, interleaved=interleaved, out=(torch.empty_like(q), rows))
    assert yk.data_ptr() == rows.data_ptr() and torch.equal(x, before)
    check(q, yq, cos, sin, interleaved, False)
    check(k, cache[:, :, 5:5 + s].transpose(1, 2), cos, sin, interleaved, False)
    assert (cache[:, :, :5] == 7).all() and (cache[:, :, 5 + s:] == 7).all()
    # in place inside the projection: v and the padding are left alone
    api.rope_apply(q, k, cos, sin, interleaved=interleaved, out=(q, k))
    check(before[..., :H * D].unflatten(-1, (H, D)), q, cos, sin, interleaved, False)
    assert torch.equal(x[..., pad + (H + Hkv) * D:], before[..., pad + (H + Hkv) * D:])
    assert torch.equal(x[..., H * D:H * D + pad], before[..., H * D:H * D + pad])


def test_unaligned_base():
    """A base pointer on an odd element: the vector path's alignment is not there."""
    for dtype in (torch.bfloat16, torch.float32):
        flat = torch.randn(3 + 9 * 4 * 64, device=DEV).to(dtype)
        q = flat[3:].view(9, 4, 64)
        cos, sin = tables((9,), 64)
        y, _ = api.rope_apply(q, None, cos, sin)
        check(q, y, cos, sin, False, False)


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
def test_transpose_is_the_gradient(interleaved):
    """<R x, y> = <x, R^T y> for a table with a gain, and directional differences."""
    pos = torch.arange(40, device=DEV) * 300
    cos, sin = api.rope_table_yarn(pos, 64, 1e4, factor=8.0, original_len=2048)
    g = torch.Generator(device=DEV).manual_seed(5)
    x, y, d = (torch.randn(40, 3, 96, generator=g, device=DEV) for _ in range(3))
    rx, _ = api.rope_apply(x, None, cos, sin, interleaved=interleaved)
    rty, _ = api.rope_apply(y, None, cos, sin, interleaved=interleaved, transpose=True)
    left, right = (rx.double() * y.double()).sum(), (x.double() * rty.double()).sum()
    # 11520 terms of order one, each product's factor within 3 fp32 half steps
    assert abs(left - right).item() <= 11520 * 2 * 3 * 2.0 ** -24 * 10
    # f(x) = <R x, y> is linear: a difference of any width is its derivative
    plus, _ = api.rope_apply(x + d, None, cos, sin, interleaved=interleaved)
    step = ((plus.double() - rx.double()) * y.double()).sum()
    slope = (rty.double() * d.double()).sum()
    assert abs(step - slope).item() <= 11520 * 4 * 3 * 2.0 ** -24 * 10


def test_offsets_past_32_bits():
    """A token stride of 2^27 elements: the last rows lie past 2^32 bytes and elements."""
    big = torch.zeros((1 << 31) + (1 << 27) + 4096, device=DEV, dtype=torch.bfloat16)
    q = big.as_strided((17, 2, 128), (1 << 27, 128, 1))
    x = torch.randn(17, 2, 128, device=DEV).bfloat16()
    q.copy_(x)
    cos, sin = tables((17,), 128)
    api.rope_apply(q, None, cos, sin, out=(q, None))
    check(x, q, cos, sin, False, False)
    del big, q
    torch.cuda.empty_cache()


def test_streams_and_graphs():
    g = torch.Generator(device=DEV).manual_seed(9)
    q = torch.randn(65, 8, 128, generator=g, device=DEV).bfloat16()
    k = torch.randn(65, 2, 128, generator=g, device=DEV).bfloat16()
    pos = torch.arange(65, device=DEV)
    cos, sin = api.rope_table_banded(pos, 128, 1e4, factor=8.0, original_len=8192)
    want = api.rope_apply(q, k, cos, sin)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = api.rope_apply(q, k, cos, sin, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c, s = api.rope_table_banded(pos, 128, 1e4, factor=8.0, original_len=8192)
        out = api.rope_apply(q, k, c, s)
    for shift in (1, 1000):
        pos += shift
        q.mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        check_table((c, s), pos, *banded(128, 1e4, 8.0, 8192, 1.0, 4.0))
        check(q, out[0], c, s, False, False)
        check(k, out[1], c, s, False, False)
