"""bench.py's DRAM bytes per launch come from a committed record, and hold while the files
that a kernel is made of are as they were at its capture: the record has to name all of
them, and to be there for both kernels whose bytes the bench prints."""
import hashlib
import json
import os
import re

import pytest

import bench

CSRC = os.path.join(bench.ROOT, "llama_gqa_causal_b200", "csrc")
KERNELS = {"prefill_sm100_kernel<128>": "prefill_sm100.cuh", "decode_bf16_kernel<128>": "decode_bf16.cuh"}


def closure(name):
    """name and what it includes from the same folder."""
    src = open(os.path.join(CSRC, name)).read()
    found = {name}
    for inc in re.findall(r'#include "([^"]+)"', src):
        if os.path.exists(os.path.join(CSRC, inc)):
            found |= closure(inc)
    return found


@pytest.mark.parametrize("kernel", KERNELS)
def test_the_bench_has_the_bytes_of_its_kernels(kernel):
    rec = json.load(open(os.path.join(bench.ROOT, "profiles", "ncu_traffic.json")))[kernel]
    assert bench._traffic(kernel) == rec["dram_read_bytes"] + rec["dram_write_bytes"]


@pytest.mark.parametrize("kernel", KERNELS)
def test_the_record_names_every_file_of_the_kernel(kernel):
    rec = json.load(open(os.path.join(bench.ROOT, "profiles", "ncu_traffic.json")))[kernel]
    assert set(rec["sources"]) == closure(KERNELS[kernel])


def test_no_bytes_for_other_sources_or_other_kernels(tmp_path, monkeypatch):
    kernel, name = next(iter(KERNELS.items()))
    os.makedirs(tmp_path / "profiles")
    os.makedirs(tmp_path / "llama_gqa_causal_b200" / "csrc")
    source = tmp_path / "llama_gqa_causal_b200" / "csrc" / name
    source.write_text("a kernel")
    rec = {kernel: {"sources": [name], "dram_read_bytes": 2, "dram_write_bytes": 3,
                    "sources_sha256_16": hashlib.sha256(b"a kernel").hexdigest()[:16]}}
    (tmp_path / "profiles" / "ncu_traffic.json").write_text(json.dumps(rec))
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    assert bench._traffic(kernel) == 5
    assert bench._traffic("another") is None
    source.write_text("another kernel")
    assert bench._traffic(kernel) is None
    source.unlink()
    assert bench._traffic(kernel) is None
