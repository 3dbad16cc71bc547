"""GPU tests of the way llama_attn_decode_prefix splits a call over the SMs (marked gpu):
the tcgen05 kernel, the own rows' warps beside it, and the merge of their partials.

The library picks the way from the sizes.  Only the split writes the workspace, so every
test here reads from it which way ran, and fails if that is not the one it is for.  Bounds
as in test_gpu_decode_prefix.py where none is derived.
"""
import math

import pytest
import torch

from llama_gqa_causal_b200 import api
from test_gpu_decode_prefix import CASES as BLOCK_CASES
from test_gpu_decode_prefix import DEV, check, expected, inputs, normal, run

pytestmark = pytest.mark.gpu


def workspace(x, fill=0xff):
    (b, H, D), (Hkv, P, _) = x["q"].shape, x["k_prefix"].shape
    return torch.full((api.decode_prefix_workspace_bytes(b, H, Hkv, P, D),), fill, device=DEV,
                      dtype=torch.uint8)


def written(ws, fill=0xff):
    return bool((ws != fill).any())


def split(x, fill=0xff, **kw):
    """The output, of a call that is known to have been split."""
    ws = workspace(x, fill)
    out = run(x, workspace=ws, **kw)
    assert written(ws, fill), "the call was not split over the SMs"
    return out


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ---------------------------------------------------------------- which way
@pytest.mark.parametrize("case", BLOCK_CASES, ids=lambda c: "b%dH%dK%dD%dP%dL%d" % c[:6])
def test_which_way_the_smaller_cases_take(case):
    """Of test_gpu_decode_prefix.py's cases these are a block a sequence, three are split."""
    b, H, Hkv, D, P, L, lens = case
    x = inputs(b, H, Hkv, D, P, L, lens, seed=P)
    ws = workspace(x)
    run(x, workspace=ws)
    assert written(ws) == ((b, P) in ((300, 130), (70, 2500), (1, 20000)))


# ---------------------------------------------------------------- against 64 bits
SPLIT = [
    # b, H, Hkv, D, prefix, L, lens: groups of 1, 2, 3, 4, 7, 8, 20, 24 and 160 heads;
    # shared and full tile pairs; a last tile of 1, 127, 128 and other numbers of keys
    (1, 1, 1, 64, 6000, 1, [0]),
    (1, 8, 1, 128, 5001, 4, [4]),
    (3, 16, 4, 64, 4500, 16, [0, 16, 7]),
    (2, 4, 4, 128, 3001, 70, [69, 1]),
    (5, 6, 3, 128, 4095, 33, [0, 33, 32, 1, 100]),
    (4, 8, 2, 128, 4096, 65, [0, 0, 0, 0]),
    (7, 28, 4, 128, 4097, 20, [3, 0, 20, -5, 9, 1, 2]),
    (16, 8, 8, 64, 5000, 40, list(range(16))),
    (17, 32, 8, 128, 3001, 64, [3 * i for i in range(17)]),
    (33, 16, 4, 128, 2600, 9, [i % 10 for i in range(33)]),
    (32, 20, 1, 64, 3500, 600, [19 * i for i in range(32)]),
    (9, 160, 1, 128, 3300, 300, [0, 300, 37, 1, 16, 17, 128, 255, 299]),
    (40, 40, 5, 128, 2000, 100, [(7 * i) % 101 for i in range(40)]),
    (129, 2, 2, 64, 3900, 20, [i % 21 for i in range(129)]),
    (24, 96, 4, 128, 2500, 400, [(37 * i) % 401 for i in range(24)]),
    (12, 48, 2, 64, 5200, 700, [60 * i for i in range(12)]),
    (64, 64, 8, 128, 2500, 30, [i % 31 for i in range(64)]),
    # one key, and no prefix at all, before caches that are long and partly filled
    (5, 8, 8, 128, 1, 12000, [12000, 0, 1, 16, 700]),
    (8, 16, 1, 128, 0, 9000, [0, 9000, 11, 16, 17, 0, 1, 4000]),
    (6, 24, 3, 64, 0, 9000, [0, 0, 3, 0, 33, 9001]),
]


@pytest.mark.parametrize("append", [False, True], ids=["plain", "append"])
@pytest.mark.parametrize("case", SPLIT, ids=lambda c: "b%dH%dK%dD%dP%dL%d" % c[:6])
def test_matches_64_bits(case, append):
    b, H, Hkv, D, P, L, lens = case
    x = inputs(b, H, Hkv, D, P, L, lens, seed=P + 1, append=append, by_token=(b + append) % 2 == 0)
    before = {k: v.clone() for k, v in x.items() if "cache" in k}
    want, tol, kc, vc = expected(x)
    out = split(x)
    assert torch.isfinite(out).all()
    assert ((out.double() - want).abs() <= tol).all()
    assert ((out.double() - want).norm() <= 2.0 ** -8 * want.norm()).item()
    if not append:  # a sequence with nothing behind it
        for i, n in enumerate(lens):
            if P == 0 and n <= 0:
                assert (out[i] == 0).all()
    for name, was in (("k_cache", kc), ("v_cache", vc)):  # row p written, nothing else
        assert same(x[name], was)
    # nothing depends on what is left in the workspace, or on the order of a sum
    x.update(before)
    assert same(split(x, fill=0x3f), out)


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0])
@pytest.mark.parametrize("shape", [(40, 8, 1, 128, 3500), (40, 8, 1, 64, 3500), (4, 8, 2, 128, 4001),
                                   (60, 24, 3, 128, 3000)], ids=lambda s: "b%dH%dK%dD%dP%d" % s)
def test_scales(shape, scale):
    """A scale of zero or below is applied before the maximum is taken, in whole tiles too:
    in tile pairs that are full, shared, and both."""
    b, H, Hkv, D, P = shape
    x = inputs(b, H, Hkv, D, P, 20, [i % 21 for i in range(b)], seed=b, gain=0.5)
    check(x, split(x, scale=scale), scale)


# ---------------------------------------------------------------- the moving reference
@pytest.mark.parametrize("sign", [1.0, -1.0], ids=["scale_above_0", "scale_below_0"])
@pytest.mark.parametrize("D", [64, 128])
def test_outputs_corrected_when_the_maximum_moves(D, sign):
    """Scores that rise by 10 (log2 units) from tile to tile over six tiles, and start again:
    more than the reference is left behind by.  The values fall by 2^-10 a tile, so that for
    a row of weight one every tile gives as much to the output as the last, and a correction
    left out, made twice or made to the wrong rows shows.  Rows of weight 1/4, 1/2, 3/4 move
    their references at other tiles.  320 query rows: a full tile pair and a shared one,
    several tiles a segment.

    A score of n = D products, all of one sign but for noise, is off by (D + 2) 2^-24 of
    sum |q k| at most; the weight's exponent (up to 60) is rounded twice more, and ex2 and
    the scale's conversion add less: 2^-16 together.  An error e of every score moves
    numerator and denominator by e each: 2 e A beside the roundings.
    """
    b, H, P, L = 40, 8, 57637, 100
    x = inputs(b, H, 1, D, P, L, [(13 * i) % 101 for i in range(b)], seed=D)
    g = torch.Generator(device=DEV).manual_seed(D + 1)
    scale = sign * D ** -0.5
    per_unit = D * abs(scale) * math.log2(math.e)  # a weight of one, against a key of one
    u = torch.randn(D, generator=g, device=DEV).sign()
    weight = (torch.arange(b * H, device=DEV) % 4 + 1).view(b, H, 1) / 4.0
    x["q"] = (weight * u + 0.05 * torch.randn(b, H, D, generator=g, device=DEV)).to(torch.bfloat16)

    def fill(k, v, rows_a_level):
        rows = k.shape[-2]
        level = 10.0 * (torch.arange(rows, device=DEV) // rows_a_level % 6)
        noise = 0.1 * torch.randn(k.shape, generator=g, device=DEV)
        k.copy_((sign * (level / per_unit)[:, None] * u + noise).to(torch.bfloat16))
        v.copy_((torch.randn(v.shape, generator=g, device=DEV)
                 * torch.exp2(50.0 - level)[:, None]).to(torch.bfloat16))

    fill(x["k_prefix"], x["v_prefix"], 128)
    fill(x["k_cache"], x["v_cache"], 16)
    out = split(x, scale=scale)
    q, lens = x["q"].double(), x["cache_lens"].tolist()
    for i in range(b):
        k = torch.cat([x["k_prefix"][0], x["k_cache"][i, 0, :lens[i]]]).double()
        v = torch.cat([x["v_prefix"][0], x["v_cache"][i, 0, :lens[i]]]).double()
        p = torch.softmax(q[i] @ k.T * scale, -1)
        want, mean_abs = p @ v, p @ v.abs()
        e = (D + 2) * 2.0 ** -24 * abs(scale) * (q[i].abs() @ k.abs().T).amax(-1, keepdim=True)
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -11 + 2 * (e + 2.0 ** -16)) * mean_abs
        err = (out[i].view(H, D).double() - want).abs()
        assert torch.isfinite(out[i]).all() and (err <= tol).all(), (i, float((err / mean_abs).max()))


def test_a_row_of_queries_far_from_the_others():
    """Rows of one tile with references of very different size keep apart."""
    x = inputs(30, 8, 1, 64, 4000, 10, [i % 11 for i in range(30)], seed=5, gain=0.5)
    x["q"][7] *= 20.0
    x["q"][8] *= 0.0
    want, tol, _, _ = expected(x)
    err = (split(x).double() - want).abs().view(30, -1)
    tol = tol.view(30, -1)
    keep = [i for i in range(30) if i != 7]
    assert (err[keep] <= tol[keep]).all()
    # entry 7: a score is off by 66 2^-24 of sum |q k|, and enters twice
    q, k = x["q"][7].double().abs(), torch.cat([x["k_prefix"][0], x["k_cache"][7, 0, :7]]).double()
    e = 66 * 2.0 ** -24 * 64 ** -0.5 * (q @ k.abs().T).amax()
    assert (err[7] <= tol[7] + 2 * e * x["v_prefix"].abs().max().double()).all()


# ---------------------------------------------------------------- infinities and NaN
def test_infinities_among_what_is_not_attended():
    x = inputs(12, 16, 4, 128, 3500, 30, [(7 * i) % 31 for i in range(12)], seed=4)
    for i, n in enumerate(x["cache_lens"].tolist()):
        x["k_cache"][i, :, n:] = float("inf")
        x["v_cache"][i, :, n:] = float("-inf")
    check(x, split(x))


def test_an_infinite_value_reaches_its_column_alone():
    x = inputs(12, 16, 4, 128, 3500, 30, [(7 * i) % 31 for i in range(12)], seed=6)
    clean = split(x).view(12, 16, 128)
    x["v_prefix"][1, 7, 9] = float("inf")
    out = split(x).view(12, 16, 128)
    assert torch.isposinf(out[:, 4:8, 9]).all()
    out[:, 4:8, 9] = clean[:, 4:8, 9]
    assert same(out, clean)


@pytest.mark.parametrize("shape", [(12, 16, 4, 128, 3500), (40, 32, 4, 64, 4000)],
                         ids=["shared_pairs", "full_pairs"])
def test_nan_that_is_attended_reaches_its_rows_alone(shape):
    b, H, Hkv, D, P = shape
    g = H // Hkv
    x = inputs(b, H, Hkv, D, P, 30, [(7 * i) % 31 for i in range(b)], seed=7)
    clean = split(x).view(b, H, D)
    bad = torch.zeros_like(clean, dtype=torch.bool)
    n = int(x["cache_lens"][3])
    x["v_cache"][3, 2, n - 1, 5] = float("nan")
    x["q"][9, 1, 0] = float("nan")
    bad[3, 2 * g:3 * g, 5] = bad[9, 1] = True
    out = split(x).view(b, H, D)
    assert out[bad].isnan().all() and same(out[~bad], clean[~bad])
    for key in (0, 1500, P - 1):  # in any tile, the last, ragged one too
        was = x["k_prefix"][1, key, 3].clone()
        x["k_prefix"][1, key, 3] = float("nan")
        out = split(x).view(b, H, D)
        x["k_prefix"][1, key, 3] = was
        with_key = bad.clone()
        with_key[:, g:2 * g] = True
        assert out[with_key].isnan().all() and same(out[~with_key], clean[~with_key])


# ---------------------------------------------------------------- beside the other entry points
def test_equals_decode_over_copies_of_the_prefix():
    """Two computations of one value, each within its bound."""
    b, P = 6, 4000
    x = inputs(b, 16, 4, 128, P, 90, [0, 90, 1, 64, 65, 30], seed=8)
    kc, vc = (torch.cat([p[None].expand(b, -1, -1, -1), c], 2).contiguous()
              for p, c in ((x["k_prefix"], x["k_cache"]), (x["v_prefix"], x["v_cache"])))
    whole = api.decode(x["q"], kc, vc, x["cache_lens"] + P)
    _, tol, _, _ = expected(x)
    assert ((split(x).double() - whole.double()).abs() <= 2 * tol).all()


def test_offsets_past_32_bits():
    """A prefix whose K/V heads lie 2^31 elements apart."""
    P = 4000
    big = torch.empty((1 << 31) + P * 128, device=DEV, dtype=torch.bfloat16)
    x = inputs(2, 4, 2, 128, P, 5, [5, 0], seed=9)
    view = big.as_strided((2, P, 128), (1 << 31, 128, 1))
    view.copy_(x["k_prefix"])
    x["k_prefix"] = view
    check(x, split(x))
    del big, view
    x.clear()
    torch.cuda.empty_cache()


# ---------------------------------------------------------------- workspaces, streams, graphs
def two_batches():
    a = inputs(24, 16, 2, 128, 3000, 300, [12 * i for i in range(24)], seed=10)
    c = inputs(40, 8, 8, 64, 2500, 100, [i % 90 for i in range(40)], seed=11)
    return (a, c), [split(a), split(c)]


def plain_call(x, **kw):
    return api.decode_prefix(x["q"], x["k_prefix"], x["v_prefix"], x["k_cache"], x["v_cache"],
                             x["cache_lens"], **kw)


def test_back_to_back_calls_share_a_workspace():
    """Calls of one stream follow one another without a wait in between: the partials of one
    are merged before the next writes its own."""
    batches, want = two_batches()
    ws = max((workspace(x) for x in batches), key=torch.numel)
    outs = []
    for _ in range(20):
        for x in batches:
            outs.append(plain_call(x, workspace=ws))
            outs.append(api.decode(x["q"], x["k_cache"], x["v_cache"], x["cache_lens"]))
    torch.cuda.synchronize()
    assert api.device_status() == api.LLAMA_OK and written(ws)
    for n in range(20):
        assert same(outs[4 * n], want[0]) and same(outs[4 * n + 2], want[1])


def test_two_graphs_share_a_workspace():
    batches, want = two_batches()
    ws = max((workspace(x) for x in batches), key=torch.numel)
    graphs, outs = [], []
    for x in batches:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(plain_call(x, workspace=ws))
        graphs.append(graph)
    for _ in range(5):
        for o in outs:
            o.zero_()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert same(outs[0], want[0]) and same(outs[1], want[1])
    assert written(ws)


def test_buffers_given_and_streams():
    (x, _), (want, _) = two_batches()
    out, ws, side = torch.empty_like(want), workspace(x), torch.cuda.Stream()
    for _ in range(3):
        out.fill_(1)
        side.wait_stream(torch.cuda.current_stream())
        assert run(x, out=out, workspace=ws, stream=side) is out
        side.synchronize()
        assert same(out, want)
    with torch.cuda.stream(side):
        again = run(x)
    side.synchronize()
    assert same(again, want) and written(ws)


def test_scratch_belongs_to_the_stream_of_the_call():
    """A call enqueued behind other work on another stream keeps its scratch: memory that
    the current stream is handed meanwhile is not it."""
    (x, _), (want, _) = two_batches()
    out, side = torch.empty_like(want), torch.cuda.Stream()
    size = workspace(x).numel()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        busy = torch.ones(1 << 26, device=DEV)
        for _ in range(50):
            busy.mul_(1.0)
    plain_call(x, out=out, stream=side)
    held = [torch.empty(size, device=DEV, dtype=torch.uint8) for _ in range(4)]
    for _ in range(400):  # while the call waits, and while it runs
        for t in held:
            t.fill_(0xff)
    torch.cuda.synchronize()
    assert same(out, want)


def test_calls_side_by_side_with_scratch_of_their_own():
    batches, want = two_batches()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(30):
        for i, x in enumerate(batches):
            got[i].append(plain_call(x, stream=streams[i]))
    torch.cuda.synchronize()
    assert api.device_status() == api.LLAMA_OK
    for i in range(2):
        assert all(same(o, want[i]) for o in got[i])


def test_decoding_loop_in_a_graph():
    """Prompt table, rotation of the prompt's keys, then captured steps: table, rotation of
    q and the new key, decode with append in two launches; lengths advance between replays."""
    b, H, Hkv, D, P, L = 6, 16, 4, 128, 4096, 8
    g = torch.Generator(device=DEV).manual_seed(12)
    kw = dict(factor=8.0, original_len=1024)
    cos, sin = api.rope_table_yarn(torch.arange(P, device=DEV), D, **kw)
    k_raw, v_prefix = normal(g, P, Hkv, D), normal(g, P, Hkv, D).transpose(0, 1)
    k_prefix = api.rope_apply(k_raw.clone(), k_raw, cos, sin)[1].transpose(0, 1)
    q, k_new, v_new = normal(g, b, H, D), normal(g, b, Hkv, D), normal(g, b, Hkv, D)
    k_cache = torch.zeros(b, Hkv, L, D, device=DEV, dtype=torch.bfloat16)
    v_cache = torch.zeros_like(k_cache)
    lens = torch.zeros(b, device=DEV, dtype=torch.int32)
    pos = lens.long() + P
    ws = workspace({"q": q, "k_prefix": k_prefix})

    def step():
        c, s = api.rope_table_yarn(pos, D, **kw)
        qr, kr = api.rope_apply(q, k_new, c, s)
        return qr, kr, api.decode_prefix(qr, k_prefix, v_prefix, k_cache, v_cache, lens, k_new=kr,
                                         v_new=v_new, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qr, kr, out = step()
    k_cache.zero_()
    v_cache.zero_()
    for _ in range(L + 2):  # past the end: the last row is replaced
        for t in (q, k_new, v_new):
            t.copy_(normal(g, *t.shape))
        x = {"k_prefix": k_prefix, "v_prefix": v_prefix, "k_cache": k_cache.clone(),
             "v_cache": v_cache.clone(), "cache_lens": lens}
        ws.fill_(0xff)
        graph.replay()
        torch.cuda.synchronize()
        x.update(q=qr, k_new=kr, v_new=v_new)
        want, tol, kc, vc = expected(x)
        assert written(ws) and ((out.double() - want).abs() <= tol).all()
        assert same(k_cache, kc) and same(v_cache, vc)
        lens += 1
        pos += 1
    assert api.device_status() == api.LLAMA_OK
