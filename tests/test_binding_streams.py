"""Whose memory a call on another stream takes: every tensor that the binding makes for a
call with ``stream=`` has to come from that stream's pool, since a block of the current
stream's pool may still be in use by work queued there, and an output has to be noted as
used by the current stream, which reads it.

Here on the CPU, with the library, the streams and the pointers' device stood in for: the
binding's own allocations are watched, nothing is launched.
"""
import contextlib

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from llama_gqa_causal_b200 import api

SIDE, CURRENT = object(), object()


class Library:
    """Every entry point succeeds; every workspace has 256 bytes."""

    def __getattr__(self, name):
        return (lambda *a: 256) if name.endswith("_bytes") else (lambda *a: api.LLAMA_OK)


class Watch(TorchDispatchMode):
    """Where each tensor was made: (operator, stream that was current)."""

    def __init__(self, under):
        super().__init__()
        self.under, self.made = under, []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        if func._schema.name.split("::")[1] in ("empty", "new_empty", "empty_like", "_to_copy",
                                                "clone", "empty_strided", "new_empty_strided"):
            self.made.append((func._schema.name, self.under[-1]))
        return func(*args, **(kwargs or {}))


@pytest.fixture
def streams(monkeypatch):
    """(stack of current streams, [(data pointer, stream)] noted by record_stream)"""
    under, noted = [CURRENT], []

    @contextlib.contextmanager
    def stream(s):
        under.append(under[-1] if s is None else s)
        try:
            yield
        finally:
            under.pop()

    def record(t, s):
        noted.append((t.data_ptr(), s))

    monkeypatch.setattr(api, "_lib", Library())
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: under[-1])
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True), raising=False)
    monkeypatch.setattr(torch.Tensor, "record_stream", record, raising=False)
    monkeypatch.setattr(api, "_stream", lambda stream=None: 0)
    monkeypatch.setattr(api, "_on", lambda device, where, fn, args, stream: None)
    api.decode_prefix_workspace_bytes.cache_clear()
    yield under, noted
    api.decode_prefix_workspace_bytes.cache_clear()


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def lens(n):
    return torch.ones(n, dtype=torch.int32)


# every entry point that makes a tensor, with inputs that it has to convert where it can
CALLS = {
    "rope_table": lambda s: api.rope_table(torch.arange(6, dtype=torch.int32), 64, stream=s),
    "rope_table_ntk": lambda s: api.rope_table_ntk(torch.arange(12)[::2], 64, stream=s),
    "rope_table_banded": lambda s: api.rope_table_banded(
        torch.arange(6, dtype=torch.int32), 64, factor=8.0, original_len=8192, stream=s),
    "rope_table_yarn": lambda s: api.rope_table_yarn(
        torch.arange(12)[::2], 64, factor=8.0, original_len=4096, stream=s),
    "rope_apply": lambda s: api.rope_apply(bf(5, 4, 64), bf(5, 2, 64), torch.zeros(5, 64),
                                           torch.zeros(5, 64), stream=s),
    "qkv_rope": lambda s: api.qkv_rope(bf(4, 128), bf(256, 128), 2, 1, 64, stream=s),
    "out_proj": lambda s: api.out_proj(bf(2, 4, 64).transpose(1, 2), bf(128, 256), stream=s),
    "prefill": lambda s: api.prefill(bf(1, 8, 2, 64), bf(1, 8, 1, 64), bf(1, 8, 1, 64), stream=s),
    "prefill_window": lambda s: api.prefill_window(
        bf(1, 8, 2, 64), bf(1, 8, 1, 64), bf(1, 8, 1, 64), window=3, stream=s),
    "prefill_varlen": lambda s: api.prefill_varlen(
        bf(1, 8, 2, 64), bf(1, 8, 1, 64), bf(1, 8, 1, 64), lens(1), stream=s),
    "prefill_packed": lambda s: api.prefill_packed(
        bf(8, 2, 64), bf(8, 1, 64), bf(8, 1, 64), lens(2), 8, stream=s),
    "decode": lambda s: api.decode(bf(3, 2, 64), bf(3, 1, 9, 64), bf(3, 1, 9, 64), lens(3), stream=s),
    "decode_append": lambda s: api.decode_append(
        bf(3, 2, 64), bf(3, 1, 64), bf(3, 1, 64), bf(3, 1, 9, 64), bf(3, 1, 9, 64), lens(3), stream=s),
    "decode_prefix": lambda s: api.decode_prefix(
        bf(3, 2, 64), bf(1, 7, 64), bf(1, 7, 64), bf(3, 1, 9, 64), bf(3, 1, 9, 64), lens(3), stream=s),
}


def outputs(result):
    return list(result) if isinstance(result, tuple) else [result]


@pytest.mark.parametrize("name", CALLS)
def test_memory_belongs_to_the_stream_of_the_call(name, streams):
    under, noted = streams
    inputs_made = Watch(under)
    with inputs_made:
        out = outputs(CALLS[name](SIDE))
    # (the inputs are made by the same call, by zeros, ones and arange)
    assert len(inputs_made.made) >= len(out)
    assert all(where is SIDE for _, where in inputs_made.made), inputs_made.made
    assert {(t.data_ptr(), CURRENT) for t in out} <= set(noted)


@pytest.mark.parametrize("name", CALLS)
def test_a_call_on_the_current_stream_notes_nothing(name, streams):
    under, noted = streams
    watch = Watch(under)
    with watch:
        outputs(CALLS[name](None))
    assert watch.made and all(where is CURRENT for _, where in watch.made) and not noted
