"""bench.py without flags: the end-to-end leg runs the warm-up steps of the timed leg."""

import os
import sys
import types

import pytest

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bench  # noqa: E402


@pytest.mark.parametrize("given,timed", [(None, 5), (1, 3), (7, 7)])
def test_end_to_end_leg_warms_up_as_the_timed_one(monkeypatch, given, timed):
    """The timed leg's steps: the flag's, at least 3, or the workload's own without a flag."""
    seen = {}
    monkeypatch.setattr(bench, "run_e2e", lambda *a, warmup: seen.update(warmup=warmup))
    args = types.SimpleNamespace(warmup=given, no_e2e=False, no_cpu_baseline=True)
    bench.finish_line(args, {"scaling": "strong", "warmup": timed}, None, types.SimpleNamespace(dplan=None),
                      2, 1, 0, None, None, None)
    assert seen == {"warmup": timed}
