"""bench.py's host-side bookkeeping, without a GPU: the kernel-source hash
that ties the committed DRAM-traffic figures to the sources they were taken
on, the lookup of those figures, the peak it divides by, and the pointer
offset the misaligned sweep entries use."""
import json
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402

STEP_OPS = ["bias_gelu_fwd", "bias_gelu_bwd", "bias_geglu_fwd", "bias_geglu_bwd", "bias_swiglu_fwd",
            "bias_swiglu_bwd", "bias_swiglu_w_fwd", "bias_swiglu_w_bwd", "bias_dropout_add_train",
            "bias_dropout_add_inference"]


def test_source_hash_is_stable_and_tracks_the_sources():
    h = bench.source_sha()
    assert h == bench.source_sha() and len(h) == 16 and int(h, 16) >= 0


def test_recorded_traffic_matches_the_current_sources_for_every_step_op():
    """When profiles/dram_traffic.txt holds figures for the current kernel
    sources, every step op has one and it lies within a few percent of the
    op's algorithmic bytes (no re-reads)."""
    alg = {"bias_gelu_fwd": 1073774592, "bias_gelu_bwd": 1610645504, "bias_geglu_fwd": 1409343488,
           "bias_geglu_bwd": 2348867584, "bias_swiglu_fwd": 1409343488, "bias_swiglu_bwd": 2348867584,
           "bias_swiglu_w_fwd": 1409409024, "bias_swiglu_w_bwd": 2348998656,
           "bias_dropout_add_train": 603987968, "bias_dropout_add_inference": 536879104}
    found = {op: bench.recorded_traffic(op) for op in STEP_OPS}
    if all(t is None for t in found.values()):
        pytest.skip("the committed DRAM-traffic figures predate the current kernel sources")
    for op, t in found.items():
        assert t is not None, op
        assert 0.9 * alg[op] <= t <= 1.02 * alg[op], (op, t / alg[op])
    assert bench.recorded_traffic("no_such_op") is None


def test_measured_peak_reads_the_peaks_file():
    peak, kind = bench.measured_peak()
    path = os.path.join(ROOT, "MEASURED_PEAKS.json")
    if os.path.exists(path):
        assert kind == "measured" and peak == pytest.approx(float(json.load(open(path))["hbm_gbs"]))
    else:
        assert kind == "fallback" and peak > 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.uint8])
def test_misalign_offsets_by_one_element(dtype):
    t = torch.arange(40, dtype=torch.float32).to(dtype).reshape(5, 8)
    m = bench.misalign(t)
    assert torch.equal(m, t) and m.shape == t.shape
    assert (m.data_ptr() - m.untyped_storage().data_ptr()) == m.element_size()


def test_result_line_is_short_enough_to_be_read_back():
    """A line with every table of a default run, the figures as wide as they
    get, stays below its limit and keeps its keys."""
    ops = lambda names: {n: {"ms": 123.4567, "ms_median": 123.4567, "gbs": 12345.6, "frac_measured": 1.2345,
                             "frac_nominal_8tbs": 1.2345, "elems_per_s": 1234567890123.4567, "bytes": 12345678901,
                             "l2": "flushed"} for n in names}
    beyond = [f"scaled_upper_triang_softmax_{i:02d}" for i in range(14)]
    family = STEP_OPS[:8] + [f"bias_dropout_add_train(p=0.{i},res=fp32)" for i in range(6)] + ["torch_copy_reference"]
    entry = ops(family)
    cells = [f"{d} T={t} H={h}" for d in ("bf16", "fp32") for t in (512, 4096, 32768, 65536)
             for h in (1024, 4096, 4099, 8192, 16384)]
    sweep = {"config": "c" * 600, "largest_bf16_min_frac_nominal_8tbs": 0.8192, "largest_bf16_min_frac_measured": 0.9786,
             "largest": {"bf16": entry, "fp32": entry}, "special": {"s" * 60 + str(i): entry for i in range(7)},
             "grid": {c: {o: [v["gbs"], v["frac_measured"]] for o, v in entry.items()} for c in cells},
             "grid_columns": ["GB/s", "fraction of the measured copy peak"]}
    head = {"metric": bench.METRIC, "value": 6644.4, "unit": "GB/s", "config": {"workload": bench.WORKLOAD},
            "cpu_baseline": {"sample": ", ".join(f"{o}:12345rows" for o in STEP_OPS)}, "rest": "r" * 1100}
    text = bench.result_text(head, ops(STEP_OPS), ops(STEP_OPS), ops(beyond), sweep, {"workload": "w" * 220})
    assert len(text) <= bench.LINE_BYTES and "\n" not in text
    d = json.loads(text)
    assert d["value"] == 6644.4 and list(d["per_op"]) == STEP_OPS and len(d["next_per_op"]) == 14
    assert set(d["sweep"]["grid"]) == set(cells)
    assert d["sweep"]["grid"][cells[0]] == {"torch_copy_reference": 12346, "ops": [12346, 12346]}
