"""GPU tests (marked gpu) of outputs made for a call on another stream: they are not memory
that work still queued on the current stream reads, and they stay whole while work on the
current stream still reads them."""
import pytest
import torch

from llama_gqa_causal_b200 import api

pytestmark = pytest.mark.gpu

DEV = "cuda"


def bf(*shape, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).to(torch.bfloat16)


def inputs(seed):
    n, H, Hkv, D, P, L = 512, 16, 4, 128, 300, 20
    x = {"pos": torch.arange(n, device=DEV) + 1000 * seed, "q": bf(n, H, D, seed=seed),
         "k": bf(n, Hkv, D, seed=seed + 10), "kp": bf(Hkv, P, D, seed=seed + 20),
         "vp": bf(Hkv, P, D, seed=seed + 30), "kc": bf(n, Hkv, L, D, seed=seed + 40),
         "vc": bf(n, Hkv, L, D, seed=seed + 50),
         "lens": torch.arange(n, device=DEV, dtype=torch.int32) % (L + 1)}
    x["cos"], x["sin"] = api.rope_table(x["pos"], D)
    return x


YARN = dict(factor=8.0, original_len=4096)
CALLS = {
    "rope_table": lambda x, **kw: api.rope_table(x["pos"], 128, **kw),
    "rope_table_ntk": lambda x, **kw: api.rope_table_ntk(x["pos"], 128, alpha=2.0, **kw),
    "rope_table_banded": lambda x, **kw: api.rope_table_banded(x["pos"], 128, **YARN, **kw),
    "rope_table_yarn": lambda x, **kw: api.rope_table_yarn(x["pos"], 128, **YARN, **kw),
    "rope_apply": lambda x, **kw: api.rope_apply(x["q"], x["k"], x["cos"], x["sin"], **kw),
    "decode_prefix": lambda x, **kw: api.decode_prefix(x["q"], x["kp"], x["vp"], x["kc"], x["vc"],
                                                       x["lens"], **kw),
    "decode": lambda x, **kw: api.decode(x["q"], x["kc"], x["vc"], x["lens"], **kw),
    "prefill": lambda x, **kw: api.prefill(x["q"][None], x["k"][None], x["k"][None], **kw),
}


def tensors(result):
    return list(result) if isinstance(result, tuple) else [result]


def bits(t):
    return t.contiguous().view(torch.uint8)


def occupy():
    """Some milliseconds of work on the current stream."""
    busy = torch.ones(1 << 26, device=DEV)
    for _ in range(100):
        busy.mul_(1.0)


@pytest.mark.parametrize("name", CALLS)
def test_freed_memory_still_read_by_the_current_stream(name):
    call, x = CALLS[name], inputs(0)
    want = tensors(call(x))
    side = torch.cuda.Stream()
    victims = [torch.full((t.numel() * t.element_size(),), 7, device=DEV, dtype=torch.uint8)
               for t in want]
    kept = [torch.zeros_like(v) for v in victims]
    torch.cuda.synchronize()
    occupy()
    for k, v in zip(kept, victims):
        k.copy_(v)
    del v
    victims.clear()  # (back in the current stream's pool, and still to be read)
    got = tensors(call(x, stream=side))
    torch.cuda.synchronize()
    assert all((k == 7).all() for k in kept)
    assert all(torch.equal(bits(g), bits(w)) for g, w in zip(got, want))
    assert api.device_status() == api.LLAMA_OK


@pytest.mark.parametrize("name", CALLS)
def test_output_dropped_while_the_current_stream_still_reads_it(name):
    call, x, other = CALLS[name], inputs(0), inputs(1)
    want = tensors(call(x))
    side = torch.cuda.Stream()
    kept = [torch.zeros_like(bits(w)) for w in want]
    torch.cuda.synchronize()
    got = tensors(call(x, stream=side))
    torch.cuda.current_stream().wait_stream(side)
    occupy()
    for k, g in zip(kept, got):
        k.copy_(bits(g))
    del g
    got.clear()
    later = call(other, stream=side)  # would be handed the same memory
    torch.cuda.synchronize()
    assert all(torch.equal(k, bits(w)) for k, w in zip(kept, want))
    del later


@pytest.mark.parametrize("name", CALLS)
def test_calls_on_a_forked_stream_in_a_capture(name):
    """A captured fork and join: one output is dropped inside the capture, one is kept."""
    call, x = CALLS[name], inputs(2)
    want = tensors(call(x))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        call(x, stream=side)
        got = tensors(call(x, stream=side))
        torch.cuda.current_stream().wait_stream(side)
        copies = [g.clone() for g in got]
    for _ in range(3):
        for t in got + copies:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for g, c, w in zip(got, copies, want):
            assert torch.equal(bits(g), bits(w)) and torch.equal(bits(c), bits(w))
    again = tensors(call(x, stream=torch.cuda.current_stream()))  # (no other stream at all)
    torch.cuda.synchronize()
    assert all(torch.equal(bits(g), bits(w)) for g, w in zip(again, want))
