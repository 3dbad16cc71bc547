"""Sizes, inputs and plain forms of the shared-prefix decode and rotary-position operators.

Each case is one call as a serving or training program makes it: a cos/sin
table scaled for a long context (``rope_table_banded``, ``rope_table_yarn``),
the rotation of q and k by such a table (``rope_apply``), and a decode step of
a batch whose sequences all continue one prefix (``decode_prefix``).  ``run``
computes a case in elementary torch operations, or, with ``own`` set, through
the package's entry points; ``exact`` restates the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

LN2PI = math.log(2.0 * math.pi)


# ---------------------------------------------------------------- cases
def _table(name, kind, rows, dim, theta, factor, original, top):
    return {"name": name, "op": "table", "kind": kind, "rows": rows, "dim": dim, "theta": theta,
            "factor": factor, "original": original, "top": top}


def _apply(name, batch, seq, heads, kv_heads, dim, rotary, dtype, interleaved, transpose, fused):
    return {"name": name, "op": "apply", "batch": batch, "seq": seq, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "rotary": rotary, "dtype": dtype,
            "interleaved": interleaved, "transpose": transpose, "fused": fused}


def _prefix(name, batch, heads, kv_heads, dim, prefix, cache, lo, hi, append, by_token):
    return {"name": name, "op": "prefix", "batch": batch, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "prefix": prefix, "cache": cache, "lo": lo, "hi": hi, "append": append,
            "by_token": by_token}


def listed():
    return [
        # the table rows of one decode step: one position per sequence
        _table("table_banded_step", "banded", 32, 128, 10000.0, 8.0, 8192, 65536),
        # the table of a whole prompt, made once before its prefill
        _table("table_banded_prompt", "banded", 8192, 128, 500000.0, 4.0, 4096, 16384),
        # a few sequences with heads of 64
        _table("table_yarn_step", "yarn", 7, 64, 10000.0, 16.0, 4096, 65536),
        # the table of every position of a long context, kept by the program
        _table("table_yarn_context", "yarn", 131072, 128, 1000000.0, 32.0, 4096, 131072),
        # a decode step's queries and new keys, out of the fused projection
        _apply("apply_step", 32, 1, 64, 8, 128, 128, "bf16", False, False, True),
        # a prompt's queries and keys at the 70B shape, out of the fused projection
        _apply("apply_prompt", 1, 8192, 64, 8, 128, 128, "bf16", False, False, True),
        # the gradient through the rotation at the 7B training shape
        _apply("apply_gradient", 2, 4096, 32, 32, 128, 128, "bf16", False, True, False),
        # interleaved pairs, half of each head, in fp32, an odd length
        _apply("apply_interleaved_fp32", 1, 4097, 32, 8, 128, 64, "fp32", True, False, False),
        # a few short answers to one short prompt, heads of 64; the latency of one call
        _prefix("prefix_small", 3, 16, 4, 64, 77, 16, 0, 16, False, False),
        # the decode batch of the 70B shape behind a prompt of 8192 tokens
        _prefix("prefix_70b", 32, 64, 8, 128, 8192, 1024, 1, 1024, False, False),
        # multi-head attention at the 7B shape, odd lengths, the step's own row
        # appended; the prefix as the prefill leaves it, token by token
        _prefix("prefix_7b_append", 16, 32, 32, 128, 4001, 513, 0, 511, True, True),
        # many samples of one long prompt: bound by the products, not the reads
        _prefix("prefix_samples", 128, 64, 8, 128, 32768, 512, 0, 511, True, False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["table", "apply", "prefix", "prefix"])
    if op == "table":
        original = rng.choice([2048, 4096, 8192, 32768])
        factor = rng.choice([1.5, 2.0, 4.0, 8.0, 10.0, 32.0, 40.0])
        case = _table("", rng.choice(["banded", "yarn"]), _log_int(rng, 1, 131072),
                      rng.choice([32, 64, 80, 96, 128]),
                      rng.choice([10000.0, 100000.0, 500000.0, 1000000.0]), factor, original,
                      int(original * factor))
    elif op == "apply":
        dim = rng.choice([64, 80, 96, 128, 256])
        heads, kv_heads = rng.choice([(32, 32), (64, 8), (16, 4), (28, 4), (9, 3), (5, 1)])
        batch = _log_int(rng, 1, 64)
        room = 8192 * 72 * 128 // (batch * (heads + kv_heads) * dim)
        case = _apply("", batch, _log_int(rng, 1, max(1, min(8192, room))), heads, kv_heads, dim,
                      rng.choice([dim, dim, dim // 2, dim // 4]), "bf16", rng.random() < 0.4,
                      rng.random() < 0.4, rng.random() < 0.5)
        if rng.random() < 0.3:
            case["dtype"] = "fp32"
            case["seq"] = max(1, case["seq"] // 2)
    else:
        heads, kv_heads, dim = rng.choice([(32, 32, 128), (64, 8, 128), (32, 8, 128), (28, 4, 128),
                                           (16, 4, 64), (8, 1, 64), (6, 3, 128), (40, 8, 64)])
        batch, prefix = _log_int(rng, 1, 128), _log_int(rng, 1, 32768)
        cache = _log_int(rng, 1, 4096)
        while batch * heads * prefix > 128 * 64 * 32768 // 2:
            prefix = prefix // 2 + 1
        while batch * kv_heads * cache > 128 * 8 * 512:
            cache = cache // 2 + 1
        lo = rng.choice([0, 0, cache // 2])
        case = _prefix("", batch, heads, kv_heads, dim, prefix, cache, lo, cache,
                       rng.random() < 0.5, rng.random() < 0.3)
    del case["name"]
    return case


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    state = {"case": case}
    if case["op"] == "table":
        n = case["rows"]
        if n >= case["top"]:  # every position of the context, from a place of the seed's own
            state["pos"] = (torch.arange(n, device=dev) + seed % 1000).to(torch.int64)
        else:
            state["pos"] = torch.randint(0, case["top"], (n,), generator=g, device=dev)
        return state
    if case["op"] == "apply":
        dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        b, s, h, kv, d = (case[k] for k in ("batch", "seq", "heads", "kv_heads", "dim"))
        if case["fused"]:  # views of the projection's [b, s, (h + 2 kv) d]
            x = torch.randn(b, s, h + 2 * kv, d, generator=g, device=dev).to(dtype)
            state["q"], state["k"] = x[:, :, :h], x[:, :, h:h + kv]
        else:
            state["q"] = torch.randn(b, s, h, d, generator=g, device=dev).to(dtype)
            state["k"] = torch.randn(b, s, kv, d, generator=g, device=dev).to(dtype)
        r = case["rotary"]
        inv = 10000.0 ** (-torch.arange(0, r, 2, device=dev, dtype=torch.float64) / r)
        start = torch.randint(0, 4096, (b, 1), generator=g, device=dev)
        angle = (start + torch.arange(s, device=dev)).double()[..., None] * inv
        angle = torch.cat([angle, angle], -1)
        state["cos"], state["sin"] = angle.cos().float(), angle.sin().float()
        return state
    b, h, kv, d, n, m = (case[k] for k in ("batch", "heads", "kv_heads", "dim", "prefix", "cache"))

    def normal(*shape, gain=1.0):
        return torch.randn(*shape, generator=g, device=dev).mul_(gain).to(torch.bfloat16)

    # a gain of 2: scores as spread out as a trained head's, where some keys stand out
    state["q"] = normal(b, h, d, gain=2.0)
    if case["by_token"]:  # [tokens, kv heads, dim] as the projection leaves it
        state["k_prefix"] = normal(n, kv, d).transpose(0, 1)
        state["v_prefix"] = normal(n, kv, d).transpose(0, 1)
    else:
        state["k_prefix"], state["v_prefix"] = normal(kv, n, d), normal(kv, n, d)
    state["k_cache"], state["v_cache"] = normal(b, kv, m, d), normal(b, kv, m, d)
    state["lens"] = torch.randint(case["lo"], case["hi"] + 1, (b,), generator=g, device=dev,
                                  dtype=torch.int32)
    if case["append"]:
        state["k_new"], state["v_new"] = normal(b, kv, d), normal(b, kv, d)
    return state


# ---------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    if case["op"] == "table":
        return _own_table(state, case) if own else _plain_table(state, case)
    if case["op"] == "apply":
        return _own_apply(state, case) if own else _plain_apply(state, case)
    return _own_prefix(state, case) if own else _plain_prefix(state, case)


def _own_table(state, case):
    from llama_gqa_causal_b200 import api
    if case["kind"] == "banded":
        return api.rope_table_banded(state["pos"], case["dim"], case["theta"],
                                     factor=case["factor"], original_len=case["original"],
                                     low_freq_factor=1.0, high_freq_factor=4.0)
    return api.rope_table_yarn(state["pos"], case["dim"], case["theta"], factor=case["factor"],
                               original_len=case["original"])


def _own_apply(state, case):
    from llama_gqa_causal_b200 import api
    return api.rope_apply(state["q"], state["k"], state["cos"], state["sin"],
                          interleaved=case["interleaved"], transpose=case["transpose"])


def _own_prefix(state, case):
    from llama_gqa_causal_b200 import api
    out = api.decode_prefix(state["q"], state["k_prefix"], state["v_prefix"], state["k_cache"],
                            state["v_cache"], state["lens"], k_new=state.get("k_new"),
                            v_new=state.get("v_new"))
    return [out, state["k_cache"], state["v_cache"]] if case["append"] else out


def _plain_table(state, case):
    pos, dim, theta = state["pos"], case["dim"], case["theta"]
    i = torch.arange(dim // 2, device=pos.device, dtype=torch.float64)
    inv = theta ** (-2.0 * i / dim)
    gain = 1.0
    if case["kind"] == "banded":
        turns = case["original"] * inv / (2.0 * math.pi)
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
    else:
        at = [dim * (math.log(case["original"]) - LN2PI - math.log(beta)) / (2.0 * math.log(theta))
              for beta in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), dim - 1)
        keep = 1.0 - ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        gain = 0.1 * math.log(case["factor"]) + 1.0
    inv = inv * (keep + (1.0 - keep) / case["factor"])
    angle = pos.double()[:, None] * inv
    angle = torch.cat([angle, angle], -1)
    return (angle.cos() * gain).float(), (angle.sin() * gain).float()


def _plain_apply(state, case):
    r = case["rotary"]
    c = state["cos"][..., None, :r // 2]
    s = state["sin"][..., None, :r // 2]
    if case["transpose"]:
        s = -s

    def turn(x):
        y = x.float()
        if case["interleaved"]:
            a, z = y[..., 0:r:2], y[..., 1:r:2]
            t = torch.stack([a * c - z * s, z * c + a * s], -1).flatten(-2)
        else:
            a, z = y[..., :r // 2], y[..., r // 2:r]
            t = torch.cat([a * c - z * s, z * c + a * s], -1)
        return torch.cat([t, y[..., r:]], -1).to(x.dtype)

    return turn(state["q"]), turn(state["k"])


def _plain_prefix(state, case):
    b, h, kv, d, m = (case[k] for k in ("batch", "heads", "kv_heads", "dim", "cache"))
    g = h // kv
    k_cache, v_cache, lens = state["k_cache"], state["v_cache"], state["lens"].long()
    if case["append"]:
        rows, at = torch.arange(b, device=lens.device), lens.clamp(max=m - 1)
        k_cache[rows, :, at] = state["k_new"]
        v_cache[rows, :, at] = state["v_new"]
        lens = at + 1
    q = state["q"].float().view(b, kv, g, d) * d ** -0.5
    shared = torch.matmul(q.transpose(0, 1).reshape(kv, b * g, d),
                          state["k_prefix"].float().transpose(1, 2)).view(kv, b, g, -1)
    each = torch.matmul(q, k_cache.float().transpose(2, 3)).transpose(0, 1)  # kv, b, g, m
    seen = torch.arange(m, device=lens.device) < lens[:, None]
    each = each.masked_fill(~seen[None, :, None, :], float("-inf"))
    top = torch.maximum(shared.amax(-1), each.amax(-1))[..., None]
    shared, each = torch.exp(shared - top), torch.exp(each - top)
    total = shared.sum(-1) + each.sum(-1)
    out = torch.matmul(shared.reshape(kv, b * g, -1), state["v_prefix"].float()).view(kv, b, g, d)
    out = out + torch.matmul(each.transpose(0, 1), v_cache.float()).transpose(0, 1)
    out = (out / total[..., None]).transpose(0, 1).reshape(b, h * d).to(torch.bfloat16)
    return [out, k_cache, v_cache] if case["append"] else out


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "table":
        n = case["rows"] * case["dim"]
        return {"bytes": 8 * case["rows"] + 8 * n, "flops": 4 * n}
    if case["op"] == "apply":
        tokens = case["batch"] * case["seq"]
        size = 2 if case["dtype"] == "bf16" else 4
        x = tokens * (case["heads"] + case["kv_heads"])
        # of each table row one half is needed: the other repeats it
        return {"bytes": 2 * x * case["dim"] * size + tokens * case["rotary"] * 4,
                "flops": 3 * x * case["rotary"]}
    b, h, kv, d, n = (case[k] for k in ("batch", "heads", "kv_heads", "dim", "prefix"))
    rows = (case["lo"] + case["hi"]) / 2 + (1 if case["append"] else 0)  # of a sequence's own, on average
    return {"bytes": 4 * kv * d * (n + b * rows) + 4 * b * h * d + 4 * b
            + (4 * b * kv * d if case["append"] else 0),
            "flops": 4 * b * h * d * (n + rows)}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "table":
        dim, theta, original = case["dim"], case["theta"], case["original"]
        pos = state["pos"].cpu().numpy().astype(np.float64)
        inv, gain = [], 1.0
        if case["kind"] == "yarn":
            gain = 1.0 + 0.1 * math.log(case["factor"])
            first = max(0, math.floor(dim / 2 * math.log(original / (64 * math.pi), theta)))
            last = min(dim - 1, math.ceil(dim / 2 * math.log(original / (2 * math.pi), theta)))
        for j in range(dim // 2):
            w = theta ** (-j / (dim / 2))
            if case["kind"] == "banded":
                wavelength = 2 * math.pi / w
                if wavelength < original / 4.0:
                    inv.append(w)
                elif wavelength > original / 1.0:
                    inv.append(w / case["factor"])
                else:
                    mix = (original / wavelength - 1.0) / 3.0
                    inv.append((1 - mix) * w / case["factor"] + mix * w)
            else:
                ramp = min(1.0, max(0.0, (j - first) / max(last - first, 0.001)))
                inv.append(w / case["factor"] * ramp + w * (1 - ramp))
        angle = pos[:, None] * np.array(inv + inv)
        return gain * np.cos(angle), gain * np.sin(angle)
    if case["op"] == "apply":
        r = case["rotary"]
        half = r // 2
        i = torch.arange(half, device="cuda")
        first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
        # a pair as a complex number, turned by cos + i sin
        turn = torch.complex(state["cos"][..., :half].double(),
                             state["sin"][..., :half].double())[:, :, None]
        turn = turn.conj() if case["transpose"] else turn
        both = []
        for x in (state["q"], state["k"]):
            y = x.double().clone()
            z = torch.complex(y[..., first], y[..., second]) * turn
            y[..., first], y[..., second] = z.real, z.imag
            both.append(y)
        return both
    b, h, kv, d, m = (case[k] for k in ("batch", "heads", "kv_heads", "dim", "cache"))
    g = h // kv
    lens = state["lens"].long()
    kc, vc = state["k_cache"], state["v_cache"]
    if case["append"]:
        lens = torch.minimum(lens, torch.full_like(lens, m - 1))
        for x, new in ((kc, state["k_new"]), (vc, state["v_new"])):
            x.scatter_(2, lens.view(b, 1, 1, 1).expand(b, kv, 1, d), new[:, :, None])
        lens = lens + 1
    hidden = torch.arange(m, device="cuda")[None, :] >= lens[:, None]
    out = torch.empty(b, h, d, device="cuda", dtype=torch.float64)
    for j in range(kv):
        q = state["q"][:, j * g:(j + 1) * g].double()
        s = torch.cat([q @ state["k_prefix"][j].double().T, q @ kc[:, j].double().transpose(1, 2)],
                      -1) / math.sqrt(d)
        s[..., s.shape[-1] - m:].masked_fill_(hidden[:, None], -math.inf)
        p = torch.softmax(s, -1)
        out[:, j * g:(j + 1) * g] = (p[..., :-m] @ state["v_prefix"][j].double()
                                     + p[..., -m:] @ vc[:, j].double())
    out = out.view(b, h * d)
    return [out, None, None] if case["append"] else out
