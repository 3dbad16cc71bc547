"""What the scaled tables, the rotation and the shared-prefix decode refuse.

Every call here carries an argument that the library or the binding rejects on
the host before anything is enqueued, so nothing needs a GPU.
"""
import ctypes
import math

import pytest
import torch

from llama_gqa_causal_b200 import api, build

FAKE = 0x10000  # 16-byte aligned, never dereferenced
INVALID, UNSUPPORTED = 1, 2
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.load()


def _call(fn, defaults, kw):
    assert set(kw) <= set(defaults)
    return fn(*{**defaults, **kw}.values())


BANDED = dict(pos=FAKE, bsz=1, seq=4, D=64, theta=1e4, factor=8.0, low=1.0, high=4.0,
              original=8192.0, cos=FAKE, sin=FAKE, stream=None)
YARN = dict(pos=FAKE, bsz=1, seq=4, D=64, theta=1e4, factor=8.0, fast=32.0, slow=1.0,
            original=4096.0, gain=1.2, cos=FAKE, sin=FAKE, stream=None)
TABLE = [(dict(pos=None), INVALID), (dict(cos=None), INVALID), (dict(sin=None), INVALID),
         (dict(bsz=0), INVALID), (dict(seq=0), INVALID), (dict(D=0), INVALID), (dict(D=7), INVALID),
         (dict(theta=0.0), INVALID), (dict(theta=NAN), INVALID), (dict(theta=INF), INVALID),
         (dict(factor=0.5), INVALID), (dict(factor=NAN), INVALID), (dict(factor=INF), INVALID),
         (dict(original=0.0), INVALID), (dict(original=NAN), INVALID), (dict(D=514), UNSUPPORTED)]


@pytest.mark.parametrize("kw,status", TABLE + [
    (dict(low=-1.0), INVALID), (dict(low=4.0), INVALID), (dict(high=INF), INVALID),
    (dict(high=NAN), INVALID), (dict(low=NAN), INVALID)])
def test_banded_table_refuses(lib, kw, status):
    assert _call(lib.llama_rope_table_banded, BANDED, kw) == status


@pytest.mark.parametrize("kw,status", TABLE + [
    (dict(theta=1.0), INVALID), (dict(slow=0.0), INVALID), (dict(slow=32.0), INVALID),
    (dict(fast=INF), INVALID), (dict(fast=NAN), INVALID), (dict(gain=0.0), INVALID),
    (dict(gain=NAN), INVALID), (dict(gain=INF), INVALID)])
def test_yarn_table_refuses(lib, kw, status):
    assert _call(lib.llama_rope_table_yarn, YARN, kw) == status


def strides(*s):
    return (ctypes.c_longlong * len(s))(*s)


APPLY = dict(q=FAKE, k=FAKE, cos=FAKE, sin=FAKE, bsz=2, seq=3, H=4, Hkv=2, D=64, R=64,
             interleaved=0, transpose=0, qs=None, ks=None, q_out=FAKE, k_out=FAKE, qos=None,
             kos=None, dtype=1, stream=None)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(cos=None), dict(sin=None), dict(q_out=None), dict(k=None), dict(k_out=None),
    dict(bsz=0), dict(seq=0), dict(H=0), dict(Hkv=0), dict(D=1, R=2), dict(R=0), dict(R=63),
    dict(R=66), dict(dtype=2), dict(dtype=-1), dict(q=FAKE + 1), dict(k_out=FAKE + 1),
    dict(q=FAKE + 2, dtype=0), dict(cos=FAKE + 4), dict(sin=FAKE + 8),
    dict(bsz=1 << 20, seq=1 << 20),
    dict(qs=strides(-1, 256, 64)), dict(kos=strides(384, 128, -64)),
    dict(qos=strides(0, 256, 64)),      # two batch entries written to one place
    dict(qos=strides(768, 256, 63)),    # heads that overlap
    dict(qos=strides(768, 255, 64)),    # tokens that overlap
    dict(kos=strides(1, 128, 64)),
    dict(qs=strides(768, 256, 128)),    # in place, but with other strides
], ids=str)
def test_rotation_refuses(lib, kw):
    assert _call(lib.llama_rope_apply, APPLY, kw) == INVALID


PREFIX = dict(q=FAKE, k_new=None, v_new=None, k_prefix=FAKE, v_prefix=FAKE, P=100, ks=None, vs=None,
              kc=FAKE, vc=FAKE, lens=FAKE, bsz=2, H=8, Hkv=2, L=10, D=128, scale=0.1, out=FAKE,
              ws=FAKE, ws_bytes=1 << 40, dtype=1, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(kc=None), INVALID), (dict(vc=None), INVALID),
    (dict(lens=None), INVALID), (dict(out=None), INVALID), (dict(k_prefix=None), INVALID),
    (dict(v_prefix=None), INVALID), (dict(k_new=FAKE), INVALID), (dict(v_new=FAKE), INVALID),
    (dict(P=-1), INVALID), (dict(L=0), INVALID), (dict(bsz=0), INVALID), (dict(H=0), INVALID),
    (dict(H=8, Hkv=3), INVALID), (dict(D=63), INVALID), (dict(scale=NAN), INVALID),
    (dict(scale=INF), INVALID), (dict(dtype=9), INVALID), (dict(q=FAKE + 8), INVALID),
    (dict(k_prefix=FAKE + 2), INVALID), (dict(v_new=FAKE + 8, k_new=FAKE), INVALID),
    (dict(lens=FAKE + 2), INVALID), (dict(ws=None), INVALID), (dict(ws=FAKE + 8), INVALID),
    (dict(ws_bytes=0), INVALID), (dict(ks=strides(12800, 127)), INVALID),
    (dict(vs=strides(12804, 128)), INVALID), (dict(ks=strides(0, 128)), INVALID),
    (dict(vs=strides(12800, 64)), INVALID), (dict(ks=strides(-12800, 128)), INVALID),
    (dict(D=96), UNSUPPORTED), (dict(dtype=0), UNSUPPORTED), (dict(bsz=4097), UNSUPPORTED),
], ids=str)
def test_prefix_decode_refuses(lib, kw, status):
    assert _call(lib.llama_attn_decode_prefix, PREFIX, kw) == status


def test_prefix_decode_refuses_a_workspace_one_byte_short(lib):
    for b, H, Hkv, P, D in ((1, 1, 1, 1, 64), (32, 64, 8, 8192, 128), (300, 8, 8, 5, 64)):
        need = lib.llama_attn_decode_prefix_workspace_bytes(b, H, Hkv, P, D)
        assert need > 0
        kw = dict(bsz=b, H=H, Hkv=Hkv, P=P, D=D, ws_bytes=need - 1)
        assert _call(lib.llama_attn_decode_prefix, PREFIX, kw) == INVALID
    for bad in ((0, 1, 1, 1, 64), (1, 0, 1, 1, 64), (1, 1, 0, 1, 64), (1, 1, 1, -1, 64)):
        assert lib.llama_attn_decode_prefix_workspace_bytes(*bad) == 0


# ---------------------------------------------------------------- the binding, on CPU tensors
def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def test_binding_takes_no_cpu_tensors(lib):
    t = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="CUDA device"):
        api.rope_table_banded(torch.arange(4), 64, factor=8.0, original_len=8192)
    with pytest.raises(ValueError, match="CUDA device"):
        api.rope_table_yarn(torch.arange(4), 64, factor=8.0, original_len=4096)
    with pytest.raises(ValueError, match="CUDA device"):
        api.rope_apply(torch.zeros(4, 2, 64), None, t, t)
    with pytest.raises(ValueError, match="CUDA device"):
        api.decode_prefix(bf(2, 4, 64), bf(2, 9, 64), bf(2, 9, 64), bf(2, 2, 5, 64), bf(2, 2, 5, 64),
                          torch.zeros(2, dtype=torch.int32))


@pytest.mark.parametrize("call,match", [
    (lambda t: api.rope_apply(torch.zeros(4, 64), None, t, t), "heads, head_dim"),
    (lambda t: api.rope_apply(torch.zeros(3, 2, 64), None, t, t), "elements"),
    (lambda t: api.rope_apply(torch.zeros(4, 2, 64), None, t, t[:, :32].contiguous()), "elements"),
    (lambda t: api.rope_apply(torch.zeros(4, 2, 64), None, t.double(), t), "float32"),
    (lambda t: api.rope_apply(torch.zeros(4, 2, 64), None, t, None), "both cos and sin"),
], ids=range(5))
def test_binding_checks_the_rotation(lib, call, match):
    with pytest.raises(ValueError, match=match):
        call(torch.zeros(4, 64))


@pytest.mark.parametrize("kw,match", [
    (dict(k_cache=bf(2, 2, 5, 128)), "k_cache must have shape"),
    (dict(v_cache=bf(2, 2, 6, 64)), "v_cache must have shape"),
    (dict(cache_lens=torch.zeros(3, dtype=torch.int32)), "2 elements"),
    (dict(cache_lens=torch.zeros(2, dtype=torch.int64)), "int32"),
    (dict(k_new=bf(2, 3, 64)), "k_new must have shape"),
    (dict(v_new=torch.zeros(2, 2, 64)), "v_new must be"),
    (dict(out=bf(2, 2, 64)), "out must hold"),
], ids=str)
def test_binding_checks_the_prefix_decode(lib, kw, match):
    args = dict(q=bf(2, 4, 64), k_prefix=bf(2, 9, 64), v_prefix=bf(2, 9, 64),
                k_cache=bf(2, 2, 5, 64), v_cache=bf(2, 2, 5, 64),
                cache_lens=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match=match):
        api.decode_prefix(**{**args, **kw})


def test_yarn_gain_of_the_rule(lib, monkeypatch):
    """attn_factor defaults to 0.1 ln(factor) + 1, whatever the other arguments."""
    seen = []
    monkeypatch.setattr(api, "_table_scaled", lambda where, pos, dim, args, stream: seen.append(args))
    api.rope_table_yarn(None, 64, factor=16.0, original_len=4096)
    api.rope_table_yarn(None, 64, factor=16.0, original_len=4096, attn_factor=1.0)
    assert seen[0][-1] == 0.1 * math.log(16.0) + 1.0 and seen[1][-1] == 1.0
