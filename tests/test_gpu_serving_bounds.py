"""The debug library's index checks in the serving kernels: every serving call on ragged
shapes (tests/serving_bounds_battery.py), no check fails, and every result is
bit-identical to the release library's."""

import os
import subprocess
import sys

import pytest
import torch

from gpu_helpers import need_cuda
from test_gpu_debug_bounds import DEBUG_LIB, HERE, _equal

pytestmark = pytest.mark.gpu


def _run(tmp_path, debug):
    out = str(tmp_path / ("debug.pt" if debug else "release.pt"))
    env = {k: v for k, v in os.environ.items() if k != "AWQ_LIB"}
    if debug:
        env["AWQ_LIB"] = "debug"
    r = subprocess.run([sys.executable, os.path.join(HERE, "serving_bounds_battery.py"), out], env=env,
                       capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stderr[-3000:]
    return torch.load(out, weights_only=False)


def test_serving_calls_pass_the_index_checks_and_match_release(tmp_path):
    need_cuda()
    if not os.path.exists(DEBUG_LIB):
        pytest.skip("libawq_debug.so not built")
    dbg, rel = _run(tmp_path, True), _run(tmp_path, False)
    assert dbg["bounds"]["enabled"] and not rel["bounds"]["enabled"]
    assert dbg["bounds"]["ok"], dbg["bounds"]["message"]
    for k in rel:
        if k != "bounds":
            _equal(dbg[k], rel[k], k)
