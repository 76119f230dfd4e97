"""Host checks of the serving operators (no GPU): every refusal comes before
any CUDA work, with the status its cause has elsewhere in the library."""

import ctypes

import pytest

import post_weight_quantization_awq_b200 as awq
from post_weight_quantization_awq_b200 import abi

CFG = awq.AwqConfig.make()


def _name(st):
    return abi.STATUS[st]


def _lora(cfg=CFG, **kw):
    a = dict(X=16, T=4, inn=512, ldx=512, qw=16, qz=16, sc=16, out=256, A=16, B=16, c=16, n=2, rank=16, ids=16,
             Y=32, ldy=256, ws=256, nbytes=1 << 30)
    a.update(kw)
    return abi.LIB.awq_w4a16_lora_gemm(a["X"], a["T"], a["inn"], a["ldx"], a["qw"], a["qz"], a["sc"], a["out"],
                                       ctypes.byref(cfg), a["A"], a["B"], a["c"], a["n"], a["rank"], a["ids"],
                                       a["Y"], a["ldy"], a["ws"], a["nbytes"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), "AWQ_ERR_INVALID_ARG"), (dict(T=(1 << 22) + 1), "AWQ_ERR_INVALID_ARG"),
    (dict(inn=500), "AWQ_ERR_INVALID_ARG"), (dict(out=250), "AWQ_ERR_INVALID_ARG"),
    (dict(out=264, ldy=264), "AWQ_ERR_UNSUPPORTED"),
    (dict(ldx=511), "AWQ_ERR_INVALID_ARG"), (dict(ldx=516), "AWQ_ERR_INVALID_ARG"),
    (dict(ldy=248), "AWQ_ERR_INVALID_ARG"), (dict(ldy=260), "AWQ_ERR_INVALID_ARG"),
    (dict(X=None), "AWQ_ERR_INVALID_ARG"), (dict(X=18), "AWQ_ERR_INVALID_ARG"),
    (dict(qw=None), "AWQ_ERR_INVALID_ARG"), (dict(qz=8), "AWQ_ERR_INVALID_ARG"),
    (dict(sc=None), "AWQ_ERR_INVALID_ARG"), (dict(A=None), "AWQ_ERR_INVALID_ARG"),
    (dict(B=24), "AWQ_ERR_INVALID_ARG"), (dict(c=None), "AWQ_ERR_INVALID_ARG"),
    (dict(ids=18), "AWQ_ERR_INVALID_ARG"), (dict(Y=None), "AWQ_ERR_INVALID_ARG"),
    (dict(Y=16), "AWQ_ERR_INVALID_ARG"), (dict(n=65536, out=32768, ldy=32768), "AWQ_ERR_UNSUPPORTED"),
    (dict(n=0), "AWQ_ERR_INVALID_ARG"), (dict(n=65537), "AWQ_ERR_INVALID_ARG"),
    (dict(rank=0), "AWQ_ERR_INVALID_ARG"), (dict(rank=12), "AWQ_ERR_UNSUPPORTED"),
    (dict(rank=264), "AWQ_ERR_UNSUPPORTED"),
    (dict(ws=None), "AWQ_ERR_WORKSPACE"), (dict(ws=128), "AWQ_ERR_WORKSPACE"),
    (dict(nbytes=256), "AWQ_ERR_WORKSPACE")])
def test_lora_refusals(kw, status):
    assert _name(_lora(**kw)) == status, awq.last_error()
    assert awq.last_error()


def test_lora_refuses_bad_settings_and_sizes_its_workspace():
    assert _name(_lora(cfg=awq.AwqConfig.make(w_bit=5))) == "AWQ_ERR_UNSUPPORTED"
    g32 = awq.AwqConfig.make(group_size=32)
    assert _name(_lora(cfg=g32, inn=96, ldx=96)) == "AWQ_ERR_UNSUPPORTED"  # in % 64
    for shape in ((0, 512, 256, 16), (4, 512, 256, 0), (4, 512, 264, 16)):
        with pytest.raises(awq.AwqError):
            awq.awq_w4a16_lora_workspace_size(*shape, CFG)
    n = awq.awq_w4a16_lora_workspace_size(4, 512, 256, 16, CFG)
    assert 256 + 4 * 16 * 4 <= n < 1 << 20
    assert _name(_lora(nbytes=n - 1)) == "AWQ_ERR_WORKSPACE" and str(n) in awq.last_error()


def _norm(**kw):
    a = dict(R=16, ldr=64, V=16, ldv=64, T=3, d=64, post=None, gate=None, ldg=0, c=1.0, pre=None, eps=1e-6,
             Ro=32, ldro=64, No=48, ldno=64)
    a.update(kw)
    return abi.LIB.awq_block_norm(a["R"], a["ldr"], a["V"], a["ldv"], a["T"], a["d"], a["post"], a["gate"], a["ldg"],
                                  a["c"], a["pre"], a["eps"], a["Ro"], a["ldro"], a["No"], a["ldno"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), "AWQ_ERR_INVALID_ARG"), (dict(T=(1 << 22) + 1), "AWQ_ERR_INVALID_ARG"),
    (dict(d=0), "AWQ_ERR_INVALID_ARG"), (dict(d=60), "AWQ_ERR_INVALID_ARG"),
    (dict(d=32776, ldr=32776, ldv=32776, ldro=32776, ldno=32776), "AWQ_ERR_UNSUPPORTED"),
    (dict(R=None), "AWQ_ERR_INVALID_ARG"), (dict(R=24), "AWQ_ERR_INVALID_ARG"),
    (dict(Ro=16, ldr=64, ldro=72), "AWQ_ERR_INVALID_ARG"), (dict(V=80, No=80, ldno=72), "AWQ_ERR_INVALID_ARG"),
    (dict(ldr=56), "AWQ_ERR_INVALID_ARG"), (dict(ldv=68), "AWQ_ERR_INVALID_ARG"),
    (dict(V=None, post=16), "AWQ_ERR_INVALID_ARG"), (dict(V=None, gate=16), "AWQ_ERR_INVALID_ARG"),
    (dict(gate=16, ldg=32), "AWQ_ERR_INVALID_ARG"), (dict(gate=20), "AWQ_ERR_INVALID_ARG"),
    (dict(post=20), "AWQ_ERR_INVALID_ARG"), (dict(pre=20), "AWQ_ERR_INVALID_ARG"),
    (dict(eps=-1.0), "AWQ_ERR_INVALID_ARG"), (dict(eps=float("nan")), "AWQ_ERR_INVALID_ARG"),
    (dict(Ro=None, No=None), "AWQ_ERR_INVALID_ARG"), (dict(No=None, pre=16), "AWQ_ERR_INVALID_ARG"),
    (dict(Ro=48), "AWQ_ERR_INVALID_ARG"), (dict(ldno=32), "AWQ_ERR_INVALID_ARG")])
def test_norm_refusals(kw, status):
    assert _name(_norm(**kw)) == status, awq.last_error()
    assert awq.last_error()


def test_injected_launch_failure_reaches_the_serving_calls(monkeypatch):
    monkeypatch.setenv("AWQ_FAULT", "launch")
    assert _name(_lora()) == "AWQ_ERR_CUDA"
    assert _name(_norm()) == "AWQ_ERR_CUDA"
    monkeypatch.setenv("AWQ_FAULT", "alloc")
    assert _name(_lora()) == "AWQ_ERR_WORKSPACE"
    with pytest.raises(awq.AwqError):
        awq.awq_w4a16_lora_workspace_size(4, 512, 256, 16, CFG)


def _moe(cfg=CFG, **kw):
    a = dict(X=16, T=4, hidden=512, ldx=512, mask=None, router=16, E=8, k=2, ren=1, gq=16, gz=16, gs=16, inter=256,
             dq=16, dz=16, ds=16, Y=32, ldy=512, ids=16, wt=16, ws=256, nbytes=1 << 40)
    a.update(kw)
    return abi.LIB.awq_w4a16_moe(a["X"], a["T"], a["hidden"], a["ldx"], a["mask"], a["router"], a["E"], a["k"],
                                 a["ren"], a["gq"], a["gz"], a["gs"], a["inter"], a["dq"], a["dz"], a["ds"],
                                 ctypes.byref(cfg), a["Y"], a["ldy"], a["ids"], a["wt"], a["ws"], a["nbytes"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), "AWQ_ERR_INVALID_ARG"), (dict(T=65), "AWQ_ERR_UNSUPPORTED"),
    (dict(hidden=500, ldx=504, ldy=504), "AWQ_ERR_INVALID_ARG"), (dict(inter=200), "AWQ_ERR_INVALID_ARG"),
    (dict(hidden=16512, ldx=16512, ldy=16512), "AWQ_ERR_UNSUPPORTED"), (dict(inter=65664), "AWQ_ERR_UNSUPPORTED"),
    (dict(E=0), "AWQ_ERR_INVALID_ARG"), (dict(E=257), "AWQ_ERR_UNSUPPORTED"),
    (dict(k=0), "AWQ_ERR_INVALID_ARG"), (dict(k=9), "AWQ_ERR_INVALID_ARG"),
    (dict(E=64, k=17), "AWQ_ERR_UNSUPPORTED"), (dict(ren=2), "AWQ_ERR_INVALID_ARG"),
    (dict(X=None), "AWQ_ERR_INVALID_ARG"), (dict(X=24), "AWQ_ERR_INVALID_ARG"),
    (dict(ldx=504), "AWQ_ERR_INVALID_ARG"), (dict(ldy=516), "AWQ_ERR_INVALID_ARG"),
    (dict(router=None), "AWQ_ERR_INVALID_ARG"), (dict(gz=8), "AWQ_ERR_INVALID_ARG"),
    (dict(ds=None), "AWQ_ERR_INVALID_ARG"), (dict(Y=None), "AWQ_ERR_INVALID_ARG"),
    (dict(Y=16), "AWQ_ERR_INVALID_ARG"), (dict(ids=None), "AWQ_ERR_INVALID_ARG"),
    (dict(wt=18), "AWQ_ERR_INVALID_ARG"), (dict(ws=None), "AWQ_ERR_WORKSPACE"),
    (dict(nbytes=4096), "AWQ_ERR_WORKSPACE")])
def test_moe_refusals(kw, status):
    assert _name(_moe(**kw)) == status, awq.last_error()
    assert awq.last_error()


def test_moe_refuses_bad_settings_and_sizes_its_workspace():
    assert _name(_moe(cfg=awq.AwqConfig.make(group_size=96))) == "AWQ_ERR_UNSUPPORTED"
    assert _name(_moe(cfg=awq.AwqConfig.make(group_size=32), hidden=544, ldx=544, ldy=544)) == "AWQ_ERR_UNSUPPORTED"
    n = awq.awq_w4a16_moe_workspace_size(4, 512, 256, 8, 2, CFG)
    assert n < 64 << 20
    assert _name(_moe(nbytes=n - 1)) == "AWQ_ERR_WORKSPACE" and str(n) in awq.last_error()
    with pytest.raises(awq.AwqError):
        awq.awq_w4a16_moe_workspace_size(65, 512, 256, 8, 2, CFG)


def test_injected_launch_failure_reaches_the_moe_call(monkeypatch):
    monkeypatch.setenv("AWQ_FAULT", "launch")
    assert _name(_moe()) == "AWQ_ERR_CUDA"
    monkeypatch.setenv("AWQ_FAULT", "alloc")
    assert _name(_moe()) == "AWQ_ERR_WORKSPACE"


def test_library_exports_and_gates_every_serving_call(monkeypatch):
    names = set(abi.header_functions(abi.SERVING_HEADER_PATH)) - set(abi.header_functions())
    sizes = {n for n in names if n.endswith("_workspace_size")}
    assert names - sizes == {"awq_w4a16_lora_gemm", "awq_w4a16_moe", "awq_block_norm"}
    for n in names:
        assert abi.LIB[n] is not None and callable(getattr(awq, n))
    monkeypatch.setenv("AWQ_FAULT", "launch")
    for call in (_lora, _moe, _norm):
        assert _name(call()) == "AWQ_ERR_CUDA" and "injected launch failure" in awq.last_error()


def test_serving_header_is_plain_c(tmp_path):
    import os
    import shutil
    import subprocess
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    src = tmp_path / "h.c"
    src.write_text('#include "awq_serving.h"\nint main(void) { return awq_block_norm == 0; }\n')
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-Wno-address", "-fsyntax-only", "-I",
                    os.path.dirname(abi.SERVING_HEADER_PATH), str(src)], check=True)
