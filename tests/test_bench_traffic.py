"""The bench's DRAM traffic records: each is valid for the sources that make its kernel, headers among them."""
import json
import os
import re
import shutil

import pytest

import bench

CSRC = os.path.join(bench.ROOT, "megatron_tensor_transformer_tp_gb300", "csrc")
KERNELS = ["mlp_b2_s2048_h4096_hp16384_N2/gemm_mlp_bwd", "mlp_b2_s2048_h4096_hp16384_N2/gemm_mlp_fwd",
           "embed_tied_V50257_h4096_T8192/embed_gather"]


def _includes(name):
    """The headers of csrc that a file includes, directly or through others."""
    seen, todo = set(), [name]
    while todo:
        with open(os.path.join(CSRC, todo.pop())) as f:
            found = re.findall(r'#include "([^"]+)"', f.read())
        new = {x for x in found if os.path.exists(os.path.join(CSRC, x))} - seen
        seen |= new
        todo += new
    return seen


@pytest.mark.parametrize("kind", sorted(bench.KERNEL_SOURCES))
def test_hashed_sources_hold_their_headers(kind):
    files = set(bench.KERNEL_SOURCES[kind])
    for name in files:
        assert _includes(name) <= files, name


@pytest.mark.parametrize("record", KERNELS)
def test_a_record_is_read_until_a_source_changes(tmp_path, monkeypatch, record):
    workload, kernel = record.split("/")
    shutil.copytree(CSRC, tmp_path / "megatron_tensor_transformer_tp_gb300" / "csrc")
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    (tmp_path / "profiles").mkdir()
    rec = {"kernels": {record: {"dram_bytes_per_call": 5, "source_hash": bench.kernel_source_hash(kernel)}}}
    (tmp_path / "profiles" / "dram_traffic.json").write_text(json.dumps(rec))
    assert bench.load_traffic(kernel, workload) == 5
    for name in bench.kernel_sources(kernel):
        p = tmp_path / "megatron_tensor_transformer_tp_gb300" / "csrc" / name
        text = p.read_text()
        p.write_text(text + "// changed\n")
        assert bench.load_traffic(kernel, workload) is None, name
        p.write_text(text)
    assert bench.load_traffic(kernel, workload) == 5


@pytest.mark.parametrize("record", KERNELS)
def test_the_committed_records_belong_to_these_sources(record):
    """What the bench line's `traffic` reports; after a change to a kernel's sources the counters are taken again."""
    workload, kernel = record.split("/")
    assert bench.load_traffic(kernel, workload) > 0
