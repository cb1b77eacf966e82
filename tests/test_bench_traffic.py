"""bench.py reports a recorded DRAM figure only for the sources that it was captured from."""
import importlib.util
import json
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture()
def bench(tmp_path, monkeypatch):
    spec = importlib.util.spec_from_file_location("bench_traffic", os.path.join(ROOT, "bench.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    monkeypatch.setattr(m, "ROOT", str(tmp_path))
    (tmp_path / "csrc").mkdir()
    (tmp_path / "profiles").mkdir()
    (tmp_path / "csrc" / "k.cu").write_text('#include <cstdint>\n#include "a.cuh"\n#include "api.h"\n')
    (tmp_path / "csrc" / "a.cuh").write_text('#pragma once\n  #  include "b.cuh"\nint a;\n')
    (tmp_path / "csrc" / "b.cuh").write_text('#include "a.cuh"\nint b;\n')
    return m


def test_a_changed_header_drops_the_recorded_figure(bench, tmp_path):
    src = tmp_path / "csrc" / "k.cu"
    heads = bench._headers(str(src))
    assert [os.path.basename(h) for h in heads] == ["a.cuh", "b.cuh"]  # not the API's, which lies elsewhere
    rec = {"k": {"source_sha": bench._sha(str(src)), "headers_sha": bench._sha(*sorted(heads)), "in_place": True,
                 "dram_bytes_per_launch": 7}}
    (tmp_path / "profiles" / "traffic.json").write_text(json.dumps(rec))
    assert bench._traffic("k", "csrc/k.cu", True) == 7
    assert bench._traffic("k", "csrc/k.cu", False) is None
    for name in ("b.cuh", "a.cuh", "k.cu"):
        old = (tmp_path / "csrc" / name).read_text()
        (tmp_path / "csrc" / name).write_text(old + "// changed\n")
        assert bench._traffic("k", "csrc/k.cu", True) is None
        (tmp_path / "csrc" / name).write_text(old)
    assert bench._traffic("k", "csrc/k.cu", True) == 7
    del rec["k"]["headers_sha"]
    (tmp_path / "profiles" / "traffic.json").write_text(json.dumps(rec))
    assert bench._traffic("k", "csrc/k.cu", True) is None


def test_the_record_names_its_headers():
    """Every record carries both hashes, so that neither can go stale unseen."""
    with open(os.path.join(ROOT, "profiles", "traffic.json")) as f:
        rec = json.load(f)
    assert rec and all({"source", "source_sha", "headers_sha"} <= set(v) for v in rec.values())
