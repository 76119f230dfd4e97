"""What the binding's serving calls accept (no GPU: the library's entry points are
recorders, the current device that of CPU tensors): every tensor in the layout that
is read, and none that only has as many elements."""

import pytest
import torch

import post_weight_quantization_awq_b200 as awq
from post_weight_quantization_awq_b200 import abi


@pytest.fixture
def calls(monkeypatch):
    """The names of the library calls that were made."""
    made = []
    monkeypatch.setattr(abi, "_serving", (torch.float16, torch.int32, torch.float32, torch.uint8, lambda: -1,
                                          lambda dev: 0))
    for name in ("awq_w4a16_lora_gemm", "awq_w4a16_moe", "awq_block_norm"):
        monkeypatch.setattr(abi.LIB, name, lambda *a, n=name: made.append(n) or 0, raising=False)
    return made


def _h(*shape):
    return torch.zeros(shape, dtype=torch.float16)


def _i(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _lora(**kw):
    T, inn, out, n, r, g = 4, 256, 512, 3, 16, 64
    a = dict(X=_h(T, inn), q=_i(inn, out // 8), z=_i(inn // g, out // 8), s=_h(inn // g, out), A=_h(n, r, inn),
             B=_h(n, out, r), c=torch.zeros(n), ids=_i(T), Y=_h(T, out), ws=torch.zeros(4096, dtype=torch.uint8))
    a.update({k: f(a[k]) for k, f in kw.items()})
    awq.awq_w4a16_lora_gemm(a["X"], a["q"], a["z"], a["s"], awq.AwqConfig.make(group_size=g), a["A"], a["B"], a["c"],
                            a["ids"], a["Y"], a["ws"])


def _moe(**kw):
    T, h, i, E, k, g = 6, 256, 128, 8, 2, 64
    a = dict(X=_h(T, h), router=_h(E, h), gq=_i(E, h, i // 4), gz=_i(E, h // g, i // 4), gs=_h(E, h // g, 2 * i),
             dq=_i(E, i, h // 8), dz=_i(E, i // g, h // 8), ds=_h(E, i // g, h), mask=None, Y=_h(T, h), ids=_i(T, k),
             wt=torch.zeros(T, k), ws=torch.zeros(4096, dtype=torch.uint8))
    a.update({name: f(a[name]) for name, f in kw.items()})
    awq.awq_w4a16_moe(a["X"], a["router"], (a["gq"], a["gz"], a["gs"]), (a["dq"], a["dz"], a["ds"]),
                      awq.AwqConfig.make(group_size=g), True, a["mask"], a["Y"], a["ids"], a["wt"], a["ws"])


def _turned(t):
    """The last two axes exchanged, contiguous."""
    return t.transpose(-1, -2).contiguous()


def _every_other(t):
    return torch.zeros(2 * t.numel(), dtype=t.dtype)[::2]


def _wide(t):
    """Rows of the same width that lie further apart."""
    return torch.zeros(t.shape[0], t.shape[1] + 8, dtype=t.dtype)[:, :t.shape[1]]


@pytest.mark.parametrize("name", ["A", "B", "q", "z", "s", "Y"])
def test_lora_refuses_a_contiguous_transpose(calls, name):
    with pytest.raises(awq.AwqError) as e:
        _lora(**{name: _turned})
    assert e.value.status_name == "AWQ_ERR_INVALID_ARG" and not calls


@pytest.mark.parametrize("name", ["router", "gq", "gz", "gs", "dz", "ds", "Y", "ids", "wt"])
def test_moe_refuses_a_contiguous_transpose(calls, name):
    with pytest.raises(awq.AwqError) as e:
        _moe(**{name: _turned})
    assert e.value.status_name == "AWQ_ERR_INVALID_ARG" and not calls


@pytest.mark.parametrize("call", [_lora, _moe])
def test_a_workspace_that_is_not_contiguous_is_refused(calls, call):
    with pytest.raises(awq.AwqError) as e:
        call(ws=_every_other)
    assert e.value.status_name == "AWQ_ERR_INVALID_ARG" and "ws" in str(e.value) and not calls


def test_tensors_in_their_layout_are_accepted(calls):
    _lora()
    _lora(X=_wide, Y=_wide, c=lambda t: t.reshape(-1, 1), ids=lambda t: t.reshape(-1, 1),
          ws=lambda t: t.view(torch.int32).reshape(2, -1))
    _moe()
    _moe(X=_wide, Y=_wide, mask=lambda t: torch.ones(6, dtype=torch.uint8))
    R = _h(5, 64)
    awq.awq_block_norm(R, _h(5, 64), _h(64), _h(1, 64).expand(5, 64), 1.0, _h(64), 1e-6, R, _h(5, 64))
    assert calls == ["awq_w4a16_lora_gemm"] * 2 + ["awq_w4a16_moe"] * 2 + ["awq_block_norm"]
