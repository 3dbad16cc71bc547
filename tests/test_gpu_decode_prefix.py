"""GPU tests of llama_attn_decode_prefix (marked gpu).

Against a softmax over prefix and own rows in 64 bits.  Everything that must
not be read holds NaN: cache rows past a sequence's length, and the rows around
the prefix in the buffer that it is a view of.

Tolerances.  With A = the attention-weighted mean of |v|: the probabilities
are rounded once to bf16 (at most 2^-8 of each, so 2^-8 A in the output), the
output once (2^-8 of its value), and fp32 sums, scores and exponentials are
left 2^-11 A (a score of size 30 out of 128 products is within 130 * 2^-24 * 30
= 2.3e-4 < 2^-12, and enters twice).
"""
import math

import pytest
import torch

from llama_gqa_causal_b200 import api

pytestmark = pytest.mark.gpu

DEV = "cuda"


def normal(g, *shape, gain=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * gain).to(torch.bfloat16)


def inputs(b, H, Hkv, D, P, L, lens, seed=0, gain=1.5, append=False, by_token=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = {"q": normal(g, b, H, D, gain=gain)}
    for name in ("k_prefix", "v_prefix"):
        if by_token:
            buf = torch.full((P + 3, Hkv, D), float("nan"), device=DEV, dtype=torch.bfloat16)
            view = buf[1:1 + P].transpose(0, 1)
        else:
            buf = torch.full((Hkv, P + 2, D), float("nan"), device=DEV, dtype=torch.bfloat16)
            view = buf[:, :P]
        view.copy_(normal(g, Hkv, P, D))
        x[name] = view
    x["k_cache"], x["v_cache"] = normal(g, b, Hkv, L, D), normal(g, b, Hkv, L, D)
    x["cache_lens"] = torch.tensor(lens, device=DEV, dtype=torch.int32)
    for i, n in enumerate(lens):
        for c in (x["k_cache"], x["v_cache"]):
            c[i, :, max(0, min(n, L)):] = float("nan")
    if append:
        x["k_new"], x["v_new"] = normal(g, b, Hkv, D), normal(g, b, Hkv, D)
    return x


def expected(x, scale=None):
    """(output, tolerance) in 64 bits, from copies of the caches with the new rows in place."""
    q, kc, vc = x["q"].double(), x["k_cache"].clone(), x["v_cache"].clone()
    b, H, D = q.shape
    Hkv, L = kc.shape[1], kc.shape[2]
    lens = x["cache_lens"].tolist()
    scale = D ** -0.5 if scale is None else scale
    out = torch.zeros(b, H, D, device=DEV, dtype=torch.float64)
    mean_abs = torch.zeros_like(out)
    for i in range(b):
        n = max(0, min(lens[i], L))
        if "k_new" in x:
            p = min(n, L - 1)
            kc[i, :, p], vc[i, :, p] = x["k_new"][i], x["v_new"][i]
            n = p + 1
        k = torch.cat([x["k_prefix"], kc[i, :, :n]], 1).double()
        v = torch.cat([x["v_prefix"], vc[i, :, :n]], 1).double()
        if k.shape[1] == 0:
            continue
        k, v = (t.repeat_interleave(H // Hkv, 0) for t in (k, v))
        p = torch.softmax(torch.einsum("hd,hjd->hj", q[i], k) * scale, -1)
        out[i] = torch.einsum("hj,hjd->hd", p, v)
        mean_abs[i] = torch.einsum("hj,hjd->hd", p, v.abs())
    tol = 2.0 ** -8 * out.abs() + (2.0 ** -8 + 2.0 ** -11) * mean_abs
    return out.view(b, H * D), tol.view(b, H * D), kc, vc


def run(x, **kw):
    args = {k: v for k, v in x.items() if k in ("k_new", "v_new")}
    out = api.decode_prefix(x["q"], x["k_prefix"], x["v_prefix"], x["k_cache"], x["v_cache"],
                            x["cache_lens"], **args, **kw)
    assert api.device_status() == api.LLAMA_OK
    return out


def check(x, out, scale=None, caches=None):
    want, tol, kc, vc = expected(x, scale)
    err = (out.double() - want).abs()
    assert torch.isfinite(out).all()
    assert (err <= tol).all(), f"off by {float((err - tol).max()):.3e} over the bound"
    # the roundings are independent: together a norm of 2^-8 sqrt(2 / 3) at most
    if want.norm() > 0:
        assert (err.norm() / want.norm()).item() <= 2.0 ** -8
    for got, was in ((x["k_cache"], kc), (x["v_cache"], vc)):
        assert torch.equal(got.view(torch.int16), was.view(torch.int16))


CASES = [
    # b, H, Hkv, D, prefix, L, lens
    (1, 1, 1, 64, 1, 1, [0]),
    (1, 8, 1, 128, 63, 4, [4]),
    (3, 16, 4, 64, 64, 16, [0, 16, 7]),
    (2, 4, 4, 128, 65, 70, [69, 1]),
    (5, 6, 3, 128, 127, 33, [0, 33, 32, 1, 100]),
    (4, 8, 2, 128, 128, 65, [0, 0, 0, 0]),
    (7, 28, 4, 128, 129, 20, [3, 0, 20, -5, 9, 1, 2]),
    (16, 8, 8, 64, 300, 40, list(range(16))),
    (17, 32, 8, 128, 1000, 64, [3 * i for i in range(17)]),
    (33, 16, 4, 128, 257, 9, [i % 10 for i in range(33)]),
    (32, 20, 1, 64, 513, 5, [i % 6 for i in range(32)]),
    (9, 160, 1, 128, 140, 8, [i % 9 for i in range(9)]),
    (40, 40, 5, 128, 700, 12, [i % 13 for i in range(40)]),
    (2, 300, 1, 64, 200, 3, [1, 3]),
    (129, 2, 2, 64, 390, 2, [i % 3 for i in range(129)]),
    (300, 8, 8, 64, 130, 3, [i % 4 for i in range(300)]),
    (70, 64, 8, 128, 2500, 30, [i % 31 for i in range(70)]),
    (4, 32, 32, 128, 4001, 33, [0, 33, 5, 20]),
    (1, 64, 8, 128, 20000, 100, [77]),
]


@pytest.mark.parametrize("by_token", [False, True], ids=["by_head", "by_token"])
@pytest.mark.parametrize("append", [False, True], ids=["plain", "append"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "b%dH%dK%dD%dP%dL%d" % c[:6])
def test_matches_64_bits(case, append, by_token):
    b, H, Hkv, D, P, L, lens = case
    x = inputs(b, H, Hkv, D, P, L, lens, seed=P, append=append, by_token=by_token)
    before = {k: v.clone() for k, v in x.items() if "cache" in k}
    out = run(x)
    after = dict(x, k_cache=before["k_cache"], v_cache=before["v_cache"])
    want, tol, kc, vc = expected(after)
    check(dict(x, k_cache=kc, v_cache=vc) if append else x, out)
    for name, was in (("k_cache", kc), ("v_cache", vc)):  # row p written, nothing else
        assert torch.equal(x[name].view(torch.int16), was.view(torch.int16))
    # nothing depends on what is left in the workspace, or on the order of a sum
    if append:
        x["k_cache"], x["v_cache"] = before["k_cache"], before["v_cache"]
    ws = torch.full((api.decode_prefix_workspace_bytes(b, H, Hkv, P, D),), 0xff, device=DEV,
                    dtype=torch.uint8)
    again = run(x, workspace=ws)
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("append", [False, True], ids=["plain", "append"])
def test_without_a_prefix(append):
    x = inputs(3, 8, 2, 128, 0, 40, [0, 40, 11], seed=1, append=append)
    before = x["k_cache"].clone(), x["v_cache"].clone()
    out = run(x)
    x["k_cache"], x["v_cache"] = before
    want, tol, _, _ = expected(x)
    assert ((out.double() - want).abs() <= tol).all()
    if not append:
        assert (out[0] == 0).all()


@pytest.mark.parametrize("P", [1, 77, 500])
def test_equals_decode_over_copies_of_the_prefix(P):
    """The batch with the prefix copied into every cache, through llama_attn_decode: two
    computations of one value, each within its bound."""
    b, H, Hkv, D, L = 6, 16, 4, 128, 90
    x = inputs(b, H, Hkv, D, P, L, [0, 90, 1, 64, 65, 30], seed=P)
    kc, vc = (torch.cat([p[None].expand(b, -1, -1, -1), c], 2).contiguous()
              for p, c in ((x["k_prefix"], x["k_cache"]), (x["v_prefix"], x["v_cache"])))
    whole = api.decode(x["q"], kc, vc, x["cache_lens"] + P)
    _, tol, _, _ = expected(x)
    assert ((run(x).double() - whole.double()).abs() <= 2 * tol).all()


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0])
def test_scales(scale):
    x = inputs(5, 8, 2, 64, 333, 20, [0, 20, 3, 7, 19], seed=2, gain=0.5)
    check(x, run(x, scale=scale), scale)


def test_peaked_scores():
    """Rows whose largest score is far from the others, in the prefix or the own rows, and
    grows along the keys, so that every running maximum moves."""
    x = inputs(9, 16, 2, 128, 1500, 200, [200, 0, 1, 64, 100, 128, 129, 199, 5], seed=3, gain=8.0)
    ramp = torch.linspace(0.2, 3.0, 1500, device=DEV)[None, :, None]
    x["k_prefix"].copy_((x["k_prefix"].float() * ramp).to(torch.bfloat16))
    want, _, _, _ = expected(x)
    err = (run(x).double() - want).abs()
    # scores reach some 400 here: 130 * 2^-24 * 400 * 2 = 2^-8 of A, beside the roundings
    k = x["v_prefix"].abs().amax().double()
    assert (err <= 2.0 ** -8 * want.abs() + (2.0 ** -7 + 2.0 ** -11) * k).all()
    assert (err.norm() / want.norm()).item() <= 2.0 ** -7


def test_infinities_and_nan_among_what_is_not_attended():
    b, P, L = 4, 200, 30
    x = inputs(b, 8, 2, 128, P, L, [0, 30, 7, 1], seed=4)
    for i, n in enumerate(x["cache_lens"].tolist()):
        x["k_cache"][i, :, n:] = float("inf")
        x["v_cache"][i, :, n:] = float("-inf")
    check(x, run(x))


def test_nan_that_is_attended_reaches_its_sequence_alone():
    x = inputs(4, 8, 2, 128, 150, 30, [3, 30, 7, 1], seed=5)
    clean = run(x)
    x["v_cache"][1, 0, 20, 5] = float("nan")
    x["q"][2, 6, 0] = float("nan")
    out = run(x).view(4, 8, 128)
    assert out[1, :4, 5].isnan().all() and out[2, 6].isnan().all()
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[1, :4, 5] = True
    bad[2, 6] = True
    assert torch.equal(out[~bad], clean.view(4, 8, 128)[~bad])


def test_nan_in_the_prefix_reaches_every_sequence():
    x = inputs(3, 8, 2, 64, 150, 30, [3, 30, 7], seed=6)
    x["k_prefix"][1, 140, 3] = float("nan")
    out = run(x).view(3, 8, 64)
    assert out[:, 4:].isnan().all() and torch.isfinite(out[:, :4]).all()


def test_buffers_given_and_streams():
    x = inputs(5, 16, 4, 128, 400, 50, [0, 50, 3, 7, 49], seed=7)
    want = run(x)
    out = torch.empty_like(want)
    ws = torch.empty(api.decode_prefix_workspace_bytes(5, 16, 4, 400, 128), device=DEV,
                     dtype=torch.uint8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        out.fill_(1)
        side.wait_stream(torch.cuda.current_stream())
        assert run(x, out=out, workspace=ws, stream=side) is out
        side.synchronize()
        assert torch.equal(out, want)
    with torch.cuda.stream(side):
        again = run(x)
    side.synchronize()
    assert torch.equal(again, want)


def test_back_to_back_calls_share_a_workspace():
    """Calls of one stream follow one another without a wait in between."""
    a = inputs(8, 16, 2, 128, 900, 70, [9 * i for i in range(8)], seed=8)
    c = inputs(40, 8, 8, 64, 300, 20, [i % 21 for i in range(40)], seed=9)
    sizes = [api.decode_prefix_workspace_bytes(8, 16, 2, 900, 128),
             api.decode_prefix_workspace_bytes(40, 8, 8, 300, 64)]
    ws = torch.empty(max(sizes), device=DEV, dtype=torch.uint8)
    want = [run(a), run(c)]
    outs = []
    for _ in range(20):
        for x in (a, c):
            outs.append(api.decode_prefix(x["q"], x["k_prefix"], x["v_prefix"], x["k_cache"],
                                          x["v_cache"], x["cache_lens"], workspace=ws))
            outs.append(api.decode(x["q"], x["k_cache"], x["v_cache"], x["cache_lens"]))
    for n in range(20):
        assert torch.equal(outs[4 * n], want[0]) and torch.equal(outs[4 * n + 2], want[1])


def test_decoding_loop_in_a_graph():
    """Prompt table, rotation of the prompt's keys, then captured steps: table, rotation of
    q and the new key, decode with append; lengths advance between replays."""
    b, H, Hkv, D, P, L = 6, 16, 4, 128, 333, 8
    g = torch.Generator(device=DEV).manual_seed(10)
    kw = dict(factor=8.0, original_len=256)
    cos, sin = api.rope_table_yarn(torch.arange(P, device=DEV), D, **kw)
    k_raw, v_prefix = normal(g, P, Hkv, D), normal(g, P, Hkv, D)
    _, k_prefix = api.rope_apply(k_raw.clone(), k_raw, cos, sin)
    q, k_new, v_new = normal(g, b, H, D), normal(g, b, Hkv, D), normal(g, b, Hkv, D)
    k_cache = torch.zeros(b, Hkv, L, D, device=DEV, dtype=torch.bfloat16)
    v_cache = torch.zeros_like(k_cache)
    lens = torch.zeros(b, device=DEV, dtype=torch.int32)
    pos = lens.long() + P

    def step():
        c, s = api.rope_table_yarn(pos, D, **kw)
        qr, kr = api.rope_apply(q, k_new, c, s)
        return qr, kr, api.decode_prefix(qr, k_prefix.transpose(0, 1), v_prefix.transpose(0, 1),
                                         k_cache, v_cache, lens, k_new=kr, v_new=v_new)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qr, kr, out = step()
    k_cache.zero_()
    v_cache.zero_()
    for n in range(L + 2):  # past the end: the last row is replaced
        for t in (q, k_new, v_new):
            t.copy_(normal(g, *t.shape))
        before = k_cache.clone(), v_cache.clone()
        graph.replay()
        torch.cuda.synchronize()
        x = {"q": qr, "k_prefix": k_prefix.transpose(0, 1), "v_prefix": v_prefix.transpose(0, 1),
             "k_cache": before[0], "v_cache": before[1], "cache_lens": lens, "k_new": kr,
             "v_new": v_new}
        want, tol, kc, vc = expected(x)
        assert ((out.double() - want).abs() <= tol).all()
        assert torch.equal(k_cache, kc) and torch.equal(v_cache, vc)
        lens += 1
        pos += 1
    assert api.device_status() == api.LLAMA_OK


def test_two_graphs_share_a_workspace():
    x = inputs(6, 16, 2, 128, 700, 40, [0, 40, 3, 9, 27, 11], seed=11)
    y = inputs(12, 8, 8, 64, 250, 30, [i for i in range(12)], seed=12)
    ws = torch.empty(max(api.decode_prefix_workspace_bytes(6, 16, 2, 700, 128),
                         api.decode_prefix_workspace_bytes(12, 8, 8, 250, 64)), device=DEV,
                     dtype=torch.uint8)
    want = [run(x), run(y)]
    graphs, outs = [], []
    for t in (x, y):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(api.decode_prefix(t["q"], t["k_prefix"], t["v_prefix"], t["k_cache"],
                                          t["v_cache"], t["cache_lens"], workspace=ws))
        graphs.append(graph)
    for _ in range(5):
        for o in outs:
            o.zero_()
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_offsets_past_32_bits():
    """A prefix whose K/V heads lie 2^31 elements apart."""
    b, H, Hkv, D, P = 2, 4, 2, 128, 150
    big = torch.empty((1 << 31) + P * D, device=DEV, dtype=torch.bfloat16)
    x = inputs(b, H, Hkv, D, P, 5, [5, 0], seed=13)
    view = big.as_strided((Hkv, P, D), (1 << 31, D, 1))
    view.copy_(x["k_prefix"])
    x["k_prefix"] = view
    check(x, run(x))
    del big, view
    x.clear()
    torch.cuda.empty_cache()
