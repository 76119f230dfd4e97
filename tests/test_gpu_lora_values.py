"""awq_w4a16_lora_gemm on values that a request may bring or a wait may leave:
what one adapter or token row holds stays with its own rows, and a wait that
runs out is never lost."""

import numpy as np
import pytest

import post_weight_quantization_awq_b200 as awq
from gpu_helpers import need_cuda
from test_gpu_lora import _case, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    need_cuda()


@pytest.mark.parametrize("T,rank", [(1, 8), (6, 64), (40, 16)])
def test_lora_wait_that_runs_out_is_never_lost(monkeypatch, T, rank):
    """Waits that give up after one poll, many calls: a call whose status is clean
    has the bits of the undisturbed one."""
    X, packed, A, B, c, ids = _case(T, 4096, 1056, rank, 4, 128, T)
    want = _run(X, packed, 128, A, B, c, ids).view(np.uint16)
    monkeypatch.setenv("AWQ_FAULT", "timeout")
    for _ in range(40):
        try:
            assert np.array_equal(_run(X, packed, 128, A, B, c, ids).view(np.uint16), want)
        except awq.AwqError as e:
            assert e.status_name == "AWQ_ERR_TIMEOUT"
    monkeypatch.delenv("AWQ_FAULT")
    assert np.array_equal(_run(X, packed, 128, A, B, c, ids).view(np.uint16), want)
