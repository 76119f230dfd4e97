"""The serving calls at their largest sizes, on layers that are narrow in the other
directions, against their definition in 64 bits on the GPU: 2^22 tokens, outputs and
norm rows, 2^20 inputs, 64 tokens of hidden 16384 and inter 65536, and packed experts
whose words pass 2^31."""

import pytest
import torch

import post_weight_quantization_awq_b200 as awq
from gpu_helpers import need_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    need_cuda()
    yield
    torch.cuda.empty_cache()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).half()


def _packed(g, lead, inn, out, group):
    """Random codes, zero points 7 or 8, steps around 0.005."""
    words = lambda *s: torch.randint(-2 ** 31, 2 ** 31, s, generator=g, device="cuda", dtype=torch.int32)  # noqa: E731
    z = 0x77777777 + (words(*lead, inn // group, out // 8) & 0x11111111)
    s = 0.004 + 0.003 * torch.rand((*lead, inn // group, out), generator=g, device="cuda")
    return words(*lead, inn, out // 8), z.to(torch.int32), s.half()


def _weights(packed, group, o0, o1):
    """((q - z) s, (q + z) s) of outputs [o0, o1) in 64 bits, [in, o1 - o0]."""
    q, z, s = packed
    sh = torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)
    nib = lambda w: ((w[:, o0 // 8:o1 // 8].unsqueeze(-1) >> sh) & 15).flatten(-2).double()  # noqa: E731
    qq, zz = nib(q), nib(z).repeat_interleave(group, 0)
    ss = s[:, o0:o1].double().repeat_interleave(group, 0)
    return (qq - zz) * ss, (qq + zz) * ss


def _ulp16(v):
    return torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -14))) - 10)


def _check_lora(X, w, group, A, B, c, ids, Y):
    """test_gpu_lora's bound: fp32 sums of n terms lose n 2^-23 of their magnitudes, W
    and U are rounded to fp16 past 64 tokens, and Y at the end."""
    T, inn = X.shape
    out, rank = Y.shape[1], A.shape[1]
    has = ids.long().clamp(min=0)
    for t0 in range(0, T, 1 << 18):
        x = X[t0:t0 + (1 << 18)].double()
        a = has[t0:t0 + (1 << 18)]
        on = (ids[t0:t0 + (1 << 18)] >= 0).double().unsqueeze(1)
        u = torch.stack([x @ Aa.double().T for Aa in A], 1)  # [t, n, rank]
        ua = torch.stack([x.abs() @ Aa.double().abs().T for Aa in A], 1)
        pick = a.reshape(-1, 1, 1).expand(-1, 1, rank)
        u = u.gather(1, pick).squeeze(1) * c[a].double().unsqueeze(1) * on
        ua = ua.gather(1, pick).squeeze(1) * c[a].double().unsqueeze(1) * on
        step = 1 << 14 if inn <= 64 else 32
        for o0 in range(0, out, step):
            o1 = min(out, o0 + step)
            W, mag = _weights(w, group, o0, o1)
            y, tol = x @ W, (inn + 8) * 2.0 ** -23 * (x.abs() @ mag)
            if T > 64:
                tol += 2.0 ** -11 * (x.abs() @ W.abs())
            for k in range(A.shape[0]):
                mine = (a == k).double().unsqueeze(1)
                Bk = B[k, o0:o1].double().T
                y += mine * (u @ Bk)
                tol += mine * ((inn + rank + 8) * 2.0 ** -23 * (ua @ Bk.abs()))
                if T > 64:
                    tol += mine * 2.0 ** -11 * (u.abs() @ Bk.abs())
            got = Y[t0:t0 + (1 << 18), o0:o1].double()
            assert bool(((got - y).abs() <= tol + 0.5 * _ulp16(y.abs() + tol)).all()), (t0, o0)


@pytest.mark.parametrize("T,inn,out,rank,n", [
    (1 << 22, 64, 32, 8, 3), (3, 64, 1 << 22, 8, 2), (66, 64, 1 << 22, 8, 2), (2, 1 << 20, 32, 8, 2),
    (40, 1 << 20, 32, 8, 2), (66, 1 << 20, 32, 8, 2), (66, 128, 32, 8, 65536), (5, 128, 32, 8, 65536)])
def test_lora_at_the_largest_sizes(T, inn, out, rank, n):
    g = _gen(T + out)
    X = _randn(g, T, inn)
    w = _packed(g, (), inn, out, 64)
    A, B = _randn(g, n, rank, inn, std=inn ** -0.5), _randn(g, n, out, rank, std=0.05)
    c = 0.5 + torch.rand(n, generator=g, device="cuda")
    ids = torch.randint(-1, n, (T,), generator=g, device="cuda", dtype=torch.int32)
    cfg = awq.AwqConfig.make(group_size=64)
    Y = torch.empty((T, out), dtype=torch.float16, device="cuda")
    ws = torch.empty(awq.awq_w4a16_lora_workspace_size(T, inn, out, rank, cfg), dtype=torch.uint8, device="cuda")
    awq.awq_w4a16_lora_gemm(X, *w, cfg, A, B, c, ids, Y, ws)
    awq.awq_device_status(ws)
    if n > 100:  # the adapters that are met
        few, ids = torch.unique(ids, return_inverse=True)
        ids = ids.to(torch.int32) - (few[0] == -1).int()
        few = few[few >= 0].long()
        A, B, c = A[few], B[few], c[few]
    _check_lora(X, w, 64, A, B, c, ids, Y)


@pytest.mark.parametrize("T,hidden,inter,E,k", [(2, 16384, 65536, 1, 1), (64, 16384, 65536, 1, 1),
                                                (64, 128, 65536, 4, 4), (5, 4096, 16384, 160, 2)])
def test_moe_at_the_largest_sizes(T, hidden, inter, E, k):
    """The rows' distance from the definition (serving_exact's bound)."""
    from serving_exact import ROW_BOUND, row_distance
    g = _gen(T + inter)
    X = _randn(g, T, hidden)
    router = _randn(g, E, hidden, std=0.02)
    if E > 100:  # the last experts, whose words begin past 2^31
        X[:, 0], router[:, 0] = 8.0, torch.linspace(0, 40, E, device="cuda").half()
    gu, dn = _packed(g, (E,), hidden, 2 * inter, 128), _packed(g, (E,), inter, hidden, 128)
    cfg = awq.AwqConfig.make(group_size=128)
    Y = torch.empty_like(X)
    ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
    wt = torch.empty((T, k), dtype=torch.float32, device="cuda")
    ws = torch.empty(awq.awq_w4a16_moe_workspace_size(T, hidden, inter, E, k, cfg), dtype=torch.uint8, device="cuda")
    awq.awq_w4a16_moe(X, router, gu, dn, cfg, True, None, Y, ids, wt, ws)
    awq.awq_device_status(ws)
    x = X.double()
    logits = x @ router.double().T
    top = torch.sort(logits, dim=1, descending=True, stable=True)
    assert torch.equal(ids.long(), top.indices[:, :k])
    p = torch.softmax(top.values[:, :k], 1)
    if E > 100:
        assert int(ids.min()) >= E - 20
    want = torch.zeros_like(x)
    for e in torch.unique(ids).tolist():
        rows, slot = (ids == e).nonzero(as_tuple=True)
        ge, de = [t[e] for t in gu], [t[e] for t in dn]
        y = torch.zeros((len(rows), hidden), dtype=torch.float64, device="cuda")
        for i0 in range(0, inter, 2048):
            i1 = min(inter, i0 + 2048)
            gate = x[rows] @ _weights(ge, 128, i0, i1)[0]
            up = x[rows] @ _weights(ge, 128, inter + i0, inter + i1)[0]
            h = gate * torch.sigmoid(gate) * up
            for o0 in range(0, hidden, 4096):
                o1 = min(hidden, o0 + 4096)
                part = [de[0][i0:i1], de[1][i0 // 128:i1 // 128], de[2][i0 // 128:i1 // 128]]
                y[:, o0:o1] += h @ _weights(part, 128, o0, o1)[0]
        want.index_add_(0, rows, p[rows, slot].unsqueeze(1) * y)
    d = row_distance(Y.cpu().numpy(), want.cpu().numpy())
    assert d.max() < ROW_BOUND, d


def test_norm_at_the_largest_token_count():
    g = _gen(9)
    T, d = 1 << 22, 264
    R, V = _randn(g, T, d), _randn(g, T, d)
    pre = _randn(g, d)
    r, n = torch.empty_like(R), torch.empty_like(R)
    awq.awq_block_norm(R, V, None, None, 0.5, pre, 1e-6, r, n)
    for t0 in range(0, T, 1 << 19):
        a, b = R[t0:t0 + (1 << 19)].double(), V[t0:t0 + (1 << 19)].double()
        want = a + 0.5 * b
        # sums of 264 squares in fp32, and two products: far below half a step of fp16
        tol = 64 * 2.0 ** -24 * (a.abs() + 0.5 * b.abs())
        assert bool(((r[t0:t0 + (1 << 19)].double() - want).abs() <= tol + 0.5 * _ulp16(want.abs() + tol)).all())
        h = 1 / torch.sqrt((want * want).mean(1, keepdim=True) + 1e-6)
        norm = want * h * pre.double()
        tol = tol * h * pre.double().abs() + 64 * 2.0 ** -24 * norm.abs()
        assert bool(((n[t0:t0 + (1 << 19)].double() - norm).abs() <= tol + 0.5 * _ulp16(norm.abs() + tol)).all())
