"""GPU tests of llama_attn_decode_prefix (marked gpu): how its work is dealt out over the
SMs, streams, and calls side by side.  Bounds as in test_gpu_decode_prefix.py."""
import pytest
import torch

from llama_gqa_causal_b200 import api
from test_gpu_decode_prefix import DEV, check, expected, inputs, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("append", [False, True], ids=["plain", "append"])
@pytest.mark.parametrize("case", [
    # b, H, Hkv, D, prefix, L, lens: more blocks of 256 query rows than fit whole into the SMs
    (800, 32, 1, 64, 300, 3, [i % 4 for i in range(800)]),
    (2048, 32, 1, 64, 130, 2, [i % 3 for i in range(2048)]),
    (1300, 32, 1, 128, 260, 2, [0] * 1300),
    # the largest batch
    (4096, 4, 2, 64, 70, 2, [i % 3 for i in range(4096)]),
    # one long sequence among short and empty ones
    (64, 8, 8, 64, 140, 3000, [3000 if i == 40 else i % 2 for i in range(64)]),
    (9, 40, 2, 128, 20, 2500, [0, 1, 2500, 16, 17, 15, 0, 2499, 3]),
    # a prefix of one key before long sequences, and the other way round
    (3, 16, 2, 128, 1, 5000, [5000, 4999, 1]),
    (2, 8, 8, 64, 30000, 1, [0, 1]),
    (1, 1, 1, 128, 50001, 17, [17]),
], ids=lambda c: "b%dH%dK%dD%dP%dL%d" % c[:6])
def test_shares(case, append):
    b, H, Hkv, D, P, L, lens = case
    x = inputs(b, H, Hkv, D, P, L, lens, seed=b + P, append=append)
    before = {k: v.clone() for k, v in x.items() if "cache" in k}
    out = run(x)
    want, tol, kc, vc = expected(dict(x, k_cache=before["k_cache"], v_cache=before["v_cache"]))
    assert torch.isfinite(out).all()
    assert ((out.double() - want).abs() <= tol).all()
    for name, was in (("k_cache", kc), ("v_cache", vc)):
        assert torch.equal(x[name].view(torch.int16), was.view(torch.int16))


def test_scales_of_both_kinds_of_tile_pairs():
    """The scaled path of every tile, in a tile pair that is full and one that is shared."""
    for b, scale in ((40, -0.1), (40, 0.0), (60, -0.3)):
        x = inputs(b, 8, 1, 128, 500, 20, [i % 21 for i in range(b)], seed=b, gain=0.5)
        check(x, run(x, scale=scale), scale)


def test_calls_side_by_side():
    """Two streams, each with calls of its own one after another."""
    a = inputs(24, 16, 2, 128, 3000, 300, [12 * i for i in range(24)], seed=1)
    c = inputs(40, 8, 8, 64, 1500, 100, [i % 90 for i in range(40)], seed=2)
    want = [run(a), run(c)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(30):
        for i, x in enumerate((a, c)):
            with torch.cuda.stream(streams[i]):
                got[i].append(api.decode_prefix(x["q"], x["k_prefix"], x["v_prefix"], x["k_cache"],
                                                x["v_cache"], x["cache_lens"]))
    torch.cuda.synchronize()
    assert api.device_status() == api.LLAMA_OK
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])


def test_scratch_belongs_to_the_stream_of_the_call():
    """A call enqueued behind other work on another stream keeps its scratch: memory that
    the current stream is handed meanwhile is not it."""
    x = inputs(6, 16, 4, 128, 400, 50, [0, 50, 3, 7, 49, 20], seed=3)
    want = run(x)
    out = torch.empty_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    size = api.decode_prefix_workspace_bytes(6, 16, 4, 400, 128)
    with torch.cuda.stream(side):
        busy = torch.ones(1 << 26, device=DEV)
        for _ in range(50):
            busy.mul_(1.0)
    api.decode_prefix(x["q"], x["k_prefix"], x["v_prefix"], x["k_cache"], x["v_cache"],
                      x["cache_lens"], out=out, stream=side)
    for _ in range(4):  # would run while the call still waits
        torch.empty(size, device=DEV, dtype=torch.uint8).fill_(0xff)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_positions_of_another_type_on_another_stream():
    pos = torch.arange(3000, device=DEV, dtype=torch.int32)[::2]
    want = api.rope_table_yarn(pos.long(), 128, factor=8.0, original_len=4096)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = api.rope_table_yarn(pos, 128, factor=8.0, original_len=4096, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("rows", [1, 131, 65535, 65537])
def test_large_tables_equal_small_ones(rows):
    """Rows written past L2 (from 65536 rows of 128 on) and through it."""
    pos = torch.arange(rows, device=DEV)
    for make, kw in ((api.rope_table_yarn, dict(factor=32.0, original_len=4096)),
                     (api.rope_table_banded, dict(factor=8.0, original_len=8192))):
        whole = make(pos, 128, 1e6, **kw)
        for lo in (0, rows // 2, max(0, rows - 40)):
            part = make(pos[lo:lo + 40].clone(), 128, 1e6, **kw)
            assert torch.equal(whole[0][lo:lo + 40], part[0])
            assert torch.equal(whole[1][lo:lo + 40], part[1])


def test_infinities_that_are_attended():
    """An infinite value in the prefix reaches what has a weight on it, and only that column."""
    x = inputs(5, 8, 2, 128, 300, 20, [0, 20, 3, 7, 19], seed=4)
    clean = run(x).view(5, 8, 128)
    x["v_prefix"][1, 7, 9] = float("inf")
    out = run(x).view(5, 8, 128)
    assert torch.isposinf(out[:, 4:, 9]).all()
    out[:, 4:, 9] = clean[:, 4:, 9]
    assert torch.equal(out, clean)


def test_a_row_of_queries_far_from_the_others():
    """Rows of one tile with references of very different size keep apart."""
    x = inputs(30, 8, 1, 64, 700, 10, [i % 11 for i in range(30)], seed=5, gain=0.5)
    x["q"][7] *= 20.0
    x["q"][8] *= 0.0
    want, tol, _, _ = expected(x)
    err = (run(x).double() - want).abs().view(30, -1)
    tol = tol.view(30, -1)
    keep = [i for i in range(30) if i != 7]
    assert (err[keep] <= tol[keep]).all()
    # scores of entry 7 reach some 50: 66 products and sums of 2^-24 each of 50, twice in
    # numerator and denominator, 4e-4 relative: under 2^-11 of the mean of |v|, four times
    assert (err[7] <= tol[7] + 2.0 ** -9 * x["v_prefix"].abs().max().double()).all()


@pytest.mark.parametrize("append", [False, True], ids=["plain", "append"])
@pytest.mark.parametrize("P", [1, 63, 128, 129, 257])
@pytest.mark.parametrize("shape", [(40, 32, 32, 128), (40, 96, 32, 128), (64, 32, 32, 64),
                                   (70, 160, 8, 64), (150, 56, 8, 128), (90, 32, 32, 128),
                                   (100, 96, 32, 128), (160, 32, 32, 64), (300, 8, 8, 128)],
                         ids=lambda s: "b%dH%dK%dD%d" % s)
def test_many_sequences_behind_a_short_prefix(shape, P, append):
    """Several sequences a block's SM, and so many that they are split over the SMs with few
    tiles of the prefix: groups of 1, 3, 7 and 20 heads, tile pairs shared and full, segments
    of one tile."""
    b, H, Hkv, D = shape
    lens = [(0, 3, 1, 17, 16, 2)[i % 6] for i in range(b)]
    x = inputs(b, H, Hkv, D, P, 17, lens, seed=P + b, append=append)
    before = {k: v.clone() for k, v in x.items() if "cache" in k}
    out = run(x)
    want, tol, kc, vc = expected(dict(x, k_cache=before["k_cache"], v_cache=before["v_cache"]))
    assert ((out.double() - want).abs() <= tol).all()
    for name, was in (("k_cache", kc), ("v_cache", vc)):
        assert torch.equal(x[name].view(torch.int16), was.view(torch.int16))


def test_a_large_batch_with_nan_where_nothing_is_attended_and_where_it_is():
    b, Hkv = 40, 32
    x = inputs(b, 32, Hkv, 128, 200, 17, [i % 18 for i in range(b)], seed=9)
    clean = run(x).view(b, 32, 128)
    x["q"][11, 5, 0] = float("nan")
    x["v_cache"][17, 3, 16, 7] = float("nan")
    x["k_cache"][16, 2, 3, 1] = float("nan")
    out = run(x).view(b, 32, 128)
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[11, 5] = bad[16, 2] = True
    bad[17, 3, 7] = True
    assert out[bad].isnan().all() and torch.equal(out[~bad], clean[~bad])
    x["k_prefix"][4, 199, 3] = float("nan")
    out = run(x).view(b, 32, 128)
    bad[:, 4] = True
    assert out[bad].isnan().all() and torch.equal(out[~bad], clean[~bad])
