"""bench.py's per-tensor workload with 8-bit moments times the list call beside the table's step: the same bits."""
import os
import sys

import pytest
import torch

from gpu_util import dev, needs_gpu

pytestmark = [pytest.mark.gpu, needs_gpu]
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_list_call_is_timed_and_equals_the_table():
    sys.path.insert(0, ROOT)
    import bench
    torch.cuda.set_device(0)
    wl = bench.RankWorkload("gpt2-small-fsdp2-pertensor", dev(), state_bits=8)
    phases, extra = dict(wl.phases), dict(wl.extra_phases)
    for name, fn in wl.phases:
        if name == "adamw":
            extra["adamw_list"]()
            fn()
            break
        fn()
    torch.cuda.synchronize()
    rs = wl.rs
    held = [rs.master_tensors, rs.exp_avg_tensors, rs.exp_avg_scale_tensors, rs.exp_avg_sq_tensors,
            rs.exp_avg_sq_scale_tensors]
    assert "adamw" in phases and len(wl._list_state) == len(held)
    assert any(int(torch.count_nonzero(t)) for t in rs.exp_avg_sq_tensors)
    for got, want in zip(wl._list_state, held):
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert wl.bytes_per_phase()["adamw_list"] == bench.adamw_bytes_per_element(wl) * wl.elems_per_step
