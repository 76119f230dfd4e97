"""Cases and plain forms of the operators that serve a layer packed by this
framework: what each call computes, on which sizes it is timed, and the 64-bit
definition its outputs are compared with.

lora   awq_w4a16_lora_gemm: a shared 4-bit projection with the low-rank
       adapter of each token's request beside it,
         y[t] = sum_j x[t,j] (q - z)[j,o] s[j/g,o]
                + c_a sum_r (sum_j x[t,j] A_a[r,j]) B_a[o,r],   a = adapter[t]
       (no second term where adapter[t] is -1).
moe    awq_w4a16_moe: a whole mixture-of-experts layer on packed experts for a
       few tokens: router, top-k, gate|up, SwiGLU, down, weighted sum.
norm   awq_block_norm: a block's exit and the next block's entrance,
         r' = r + c gate * (rmsnorm(v) post),   n = rmsnorm(r') pre.

Layouts are those of awq_quant_pack: the code of (output o, input j) is nibble
o % 8 of qweight[j][o/8], its zero point nibble o % 8 of qzeros[j/g][o/8] and
its step scales[j/g][o].
"""

import math

import torch

own = False  # set from outside: True makes run() call the framework


# ----------------------------------------------------------------- the cases
def listed():
    return [
        # one request, one token: a 4096 x 4096 projection of a 7B-shaped
        # decoder while a single user decodes; latency is all there is
        {"name": "lora decode 1", "op": "lora", "T": 1, "inn": 4096, "out": 4096, "rank": 16, "adapters": 4,
         "group": 128, "order": "mixed"},
        # sixteen requests, each with an adapter of its own or none
        {"name": "lora decode 16", "op": "lora", "T": 16, "inn": 4096, "out": 4096, "rank": 16, "adapters": 16,
         "group": 128, "order": "mixed"},
        # an odd batch on the fused q|k|v projection, finer groups, higher rank
        {"name": "lora batch 45 qkv", "op": "lora", "T": 45, "inn": 4096, "out": 12288, "rank": 64, "adapters": 8,
         "group": 64, "order": "mixed"},
        # a chunk of prompts of several requests, one after the other (ragged
        # runs of one adapter each), on the 4096 -> 11008 MLP projection
        {"name": "lora prompts 1531", "op": "lora", "T": 1531, "inn": 4096, "out": 11008, "rank": 32, "adapters": 5,
         "group": 128, "order": "runs"},
        # the largest prompt chunk, square projection
        {"name": "lora prompts 8192", "op": "lora", "T": 8192, "inn": 4096, "out": 4096, "rank": 16, "adapters": 12,
         "group": 128, "order": "runs"},
        # one token through eight 7B-shaped MLP experts, two of them chosen
        {"name": "moe decode 1 wide", "op": "moe", "T": 1, "hidden": 4096, "inter": 11008, "experts": 8, "top_k": 2,
         "group": 128, "renormalize": True, "padded": False},
        # a small batch over many narrow experts
        {"name": "moe decode 5 narrow", "op": "moe", "T": 5, "hidden": 2048, "inter": 1024, "experts": 64, "top_k": 8,
         "group": 128, "renormalize": False, "padded": False},
        # an odd, padded batch (a captured decode step whose last rows are
        # empty), finer groups
        {"name": "moe padded 37", "op": "moe", "T": 37, "hidden": 1024, "inter": 2816, "experts": 16, "top_k": 4,
         "group": 32, "renormalize": True, "padded": True},
        # the largest batch: every wide expert is met
        {"name": "moe batch 64 wide", "op": "moe", "T": 64, "hidden": 4096, "inter": 11008, "experts": 8, "top_k": 2,
         "group": 128, "renormalize": True, "padded": False},
        # one token between two blocks
        {"name": "norm decode 1", "op": "norm", "T": 1, "d": 4096, "post": False, "gate": "none"},
        # an odd batch with a norm after the block and a gate for each token
        {"name": "norm gated 333", "op": "norm", "T": 333, "d": 5120, "post": True, "gate": "token"},
        # a long prompt, residual scale for each channel
        {"name": "norm prompt 16384", "op": "norm", "T": 16384, "d": 4096, "post": True, "gate": "channel"},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["lora", "moe", "norm"])
    if op == "lora":
        group = rng.choice([32, 64, 128])
        while True:
            unit = max(64, group)
            c = {"op": op, "T": _log(rng, 1, 8192), "inn": unit * _log(rng, 1, 8192 // unit),
                 "out": 32 * _log(rng, 4, 384), "rank": 8 * rng.choice([1, 2, 3, 4, 8, 16]),
                 "adapters": _log(rng, 1, 48), "group": group, "order": rng.choice(["mixed", "runs"])}
            if c["T"] * c["inn"] * c["out"] <= 1531 * 4096 * 11008:
                return c
    if op == "moe":
        group = rng.choice([32, 64, 128])
        unit = max(64, group)
        while True:
            experts = _log(rng, 4, 64)
            c = {"op": op, "T": _log(rng, 1, 64), "hidden": unit * _log(rng, 256 // unit, 4096 // unit),
                 "inter": unit * _log(rng, 256 // unit, 11008 // unit), "experts": experts,
                 "top_k": rng.randint(1, min(8, experts)), "group": group, "renormalize": rng.random() < 0.5,
                 "padded": rng.random() < 0.3}
            if experts * c["hidden"] * c["inter"] <= 8 * 4096 * 11008:
                return c
    while True:
        c = {"op": op, "T": _log(rng, 1, 16384), "d": 8 * _log(rng, 8, 1024), "post": rng.random() < 0.5,
             "gate": rng.choice(["none", "channel", "token"])}
        if c["T"] * c["d"] <= 16384 * 4096:
            return c


# ----------------------------------------------------------------- the inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, T, d):
    """Heavy-tailed activations: one channel in a hundred is 20 to 50 times the others."""
    big = torch.rand(d, generator=g, device="cuda") < 0.01
    boost = 20 + 30 * torch.rand(d, generator=g, device="cuda")
    return (_randn(g, T, d) * torch.where(big, boost, torch.ones_like(boost))).half()


def _packed(g, lead, inn, out, group):
    """Random packed weights of [*lead] layers: codes over 0..15, zero points 7 or 8, steps around 0.005."""
    q = torch.randint(-2**31, 2**31, (*lead, inn, out // 8), generator=g, device="cuda", dtype=torch.int32)
    z = torch.randint(-2**31, 2**31, (*lead, inn // group, out // 8), generator=g, device="cuda", dtype=torch.int32)
    z = 0x77777777 + (z & 0x11111111)
    s = 0.004 + 0.003 * torch.rand(*lead, inn // group, out, generator=g, device="cuda")
    return q, z.to(torch.int32), s.half()


def prepare(case, seed):
    g = _generator(seed)
    st = {"case": case}
    if case["op"] == "lora":
        T, inn, out, r, n = (case[k] for k in ("T", "inn", "out", "rank", "adapters"))
        st["x"] = _activations(g, T, inn)
        st["w"] = _packed(g, (), inn, out, case["group"])
        st["A"] = (_randn(g, n, r, inn) / math.sqrt(inn)).half()
        st["B"] = (_randn(g, n, out, r) * 0.05).half()
        st["c"] = 0.5 + torch.rand(n, generator=g, device="cuda")
        if case["order"] == "runs":  # ragged runs of one request each, some without an adapter
            runs = 2 * n + 1
            ids = torch.randint(-1, n, (runs,), generator=g, device="cuda", dtype=torch.int32)
            cuts = torch.sort(torch.randint(0, T, (runs - 1,), generator=g, device="cuda")).values
            at = (torch.arange(T, device="cuda")[:, None] >= cuts[None, :]).sum(1)
            st["ids"] = ids[at].contiguous()
        else:
            st["ids"] = torch.randint(-1, n, (T,), generator=g, device="cuda", dtype=torch.int32)
        return st
    if case["op"] == "moe":
        T, h, i, e = (case[k] for k in ("T", "hidden", "inter", "experts"))
        st["x"] = _activations(g, T, h)
        st["router"] = (_randn(g, e, h) * 0.02).half()
        st["gate_up"] = _packed(g, (e,), h, 2 * i, case["group"])
        st["down"] = _packed(g, (e,), i, h, case["group"])
        st["mask"] = None
        if case["padded"]:  # the last quarter of the rows holds no request
            st["mask"] = (torch.arange(T, device="cuda") < T - T // 4).to(torch.uint8)
        return st
    T, d = case["T"], case["d"]
    st["r"] = (_randn(g, T, d) * 2).half()
    st["v"] = _activations(g, T, d)
    st["pre"] = (1 + 0.2 * _randn(g, d)).half()
    st["post"] = (1 + 0.2 * _randn(g, d)).half() if case["post"] else None
    st["gate"] = None
    if case["gate"] != "none":
        st["gate"] = torch.tanh(_randn(g, *((T, d) if case["gate"] == "token" else (d,)))).half()
    st["c"], st["eps"] = 0.75, 1e-6
    return st


# ------------------------------------------------------------ the plain forms
def _unpack(words):
    """Nibbles of [..., n] words as [..., 8 n] whole numbers."""
    shifts = torch.arange(0, 32, 4, device=words.device, dtype=torch.int32)
    return ((words.unsqueeze(-1) >> shifts) & 15).flatten(-2)


def _weights(w, group):
    """(q - z) scale as fp32 [..., in, out]: exact, 5 and 11 bits."""
    q, z, s = w
    d = _unpack(q).float().unflatten(-2, (-1, group)) - _unpack(z).float().unsqueeze(-2)
    return (d * s.float().unsqueeze(-2)).flatten(-3, -2)


def _plain_lora(st):
    x = st["x"].float()
    y = x @ _weights(st["w"], st["case"]["group"])
    n, r, inn = st["A"].shape
    u = (x @ st["A"].float().reshape(n * r, inn).T).reshape(-1, n, r)
    has = st["ids"].unsqueeze(1) == torch.arange(n, device=x.device, dtype=torch.int32)
    u = torch.where(has.unsqueeze(2), u * st["c"].reshape(1, n, 1), torch.zeros_like(u))
    y = y + u.reshape(-1, n * r) @ st["B"].float().permute(0, 2, 1).reshape(n * r, -1)
    return {"y": y.half()}


def _plain_moe(st):
    case, x = st["case"], st["x"].float()
    e, k, i = case["experts"], case["top_k"], case["inter"]
    # 64 bits: the choice of experts is made next to a border
    logits = st["x"].double() @ st["router"].double().T
    p = torch.exp(logits - logits.max(1, keepdim=True).values)
    p = p / p.sum(1, keepdim=True)
    a, b = logits.unsqueeze(2), logits.unsqueeze(1)  # rank of expert a: how many come before it
    index = torch.arange(e, device=x.device)
    before = (b > a) | ((b == a) & (index.reshape(1, 1, e) < index.reshape(1, e, 1)))
    rank = before.sum(2)
    ids = torch.argsort(rank, dim=1)[:, :k]
    wt = torch.gather(p, 1, ids)
    if case["renormalize"]:
        wt = wt / wt.sum(1, keepdim=True)
    dense = torch.zeros_like(p).scatter(1, ids, wt)
    if st["mask"] is not None:
        live = st["mask"].bool().unsqueeze(1)
        ids = torch.where(live, ids, torch.full_like(ids, -1))
        wt = torch.where(live, wt, torch.zeros_like(wt))
        dense = torch.where(live, dense, torch.zeros_like(dense))
    gu = torch.matmul(x.unsqueeze(0), _weights(st["gate_up"], case["group"]))  # [E, T, 2 i]
    gate, up = gu[..., :i], gu[..., i:]
    h = gate / (1 + torch.exp(-gate)) * up
    h = h * dense.T.float().unsqueeze(2)
    y = torch.matmul(h, _weights(st["down"], case["group"])).sum(0)
    return {"y": y.half(), "ids": ids.to(torch.int32), "weights": wt.float()}


def _plain_norm(st):
    r, v = st["r"].float(), st["v"].float()
    if st["post"] is not None:
        v = v * torch.rsqrt((v * v).mean(1, keepdim=True) + st["eps"]) * st["post"].float()
    if st["gate"] is not None:
        v = v * st["gate"].float()
    r = r + st["c"] * v
    n = r * torch.rsqrt((r * r).mean(1, keepdim=True) + st["eps"]) * st["pre"].float()
    return {"r": r.half(), "n": n.half()}


# ------------------------------------------------------ the framework's calls
def _own_lora(st):
    import post_weight_quantization_awq_b200 as awq
    x, out = st["x"], st["w"][2].shape[-1]
    if "cfg" not in st:  # what a program makes once for a layer and a batch size
        st["cfg"] = awq.AwqConfig.make(group_size=st["case"]["group"])
        need = awq.awq_w4a16_lora_workspace_size(x.shape[0], x.shape[1], out, st["A"].shape[1], st["cfg"])
        st["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
        st["y"] = torch.empty((x.shape[0], out), dtype=torch.float16, device="cuda")
    awq.awq_w4a16_lora_gemm(x, *st["w"], st["cfg"], st["A"], st["B"], st["c"], st["ids"], st["y"], st["ws"])
    return {"y": st["y"]}


def _own_moe(st):
    import post_weight_quantization_awq_b200 as awq
    case, x = st["case"], st["x"]
    if "cfg" not in st:
        st["cfg"] = awq.AwqConfig.make(group_size=case["group"])
        need = awq.awq_w4a16_moe_workspace_size(x.shape[0], case["hidden"], case["inter"], case["experts"],
                                                case["top_k"], st["cfg"])
        st["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
        st["y"] = torch.empty_like(x)
        st["ids"] = torch.empty((x.shape[0], case["top_k"]), dtype=torch.int32, device="cuda")
        st["weights"] = torch.empty((x.shape[0], case["top_k"]), dtype=torch.float32, device="cuda")
    awq.awq_w4a16_moe(x, st["router"], st["gate_up"], st["down"], st["cfg"], case["renormalize"], st["mask"],
                      st["y"], st["ids"], st["weights"], st["ws"])
    return {"y": st["y"], "ids": st["ids"], "weights": st["weights"]}


def _own_norm(st):
    import post_weight_quantization_awq_b200 as awq
    if "r_out" not in st:
        st["r_out"], st["n_out"] = torch.empty_like(st["r"]), torch.empty_like(st["r"])
    awq.awq_block_norm(st["r"], st["v"], st["post"], st["gate"], st["c"], st["pre"], st["eps"], st["r_out"],
                       st["n_out"])
    return {"r": st["r_out"], "n": st["n_out"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"lora": _own_lora, "moe": _own_moe, "norm": _own_norm}[op](state)
    return {"lora": _plain_lora, "moe": _plain_moe, "norm": _plain_norm}[op](state)


# ------------------------------------------------------------------- the work
def _packed_bytes(inn, out, group):
    return inn * out / 2 + inn // group * (out / 2 + 2 * out)


def work(case):
    """Bytes: each input read once (of the adapters and experts those that
    the tokens are expected to meet), each output written once."""
    if case["op"] == "lora":
        T, inn, out, r, n = (case[k] for k in ("T", "inn", "out", "rank", "adapters"))
        tries = min(T, 2 * n + 1) if case["order"] == "runs" else T
        met = n * (1 - (1 - 1 / (n + 1)) ** tries)
        size = 2 * T * (inn + out) + _packed_bytes(inn, out, case["group"]) + 2 * met * r * (inn + out)
        return {"bytes": size, "flops": 2.0 * T * inn * out + 2.0 * T * r * (inn + out) * n / (n + 1)}
    if case["op"] == "moe":
        T, h, i, e, k = (case[x] for x in ("T", "hidden", "inter", "experts", "top_k"))
        live = T - T // 4 if case["padded"] else T
        met = e * (1 - (1 - k / e) ** live)
        each = _packed_bytes(h, 2 * i, case["group"]) + _packed_bytes(i, h, case["group"])
        return {"bytes": met * each + 2 * e * h + 4 * T * h + 8 * T * k,
                "flops": live * (2.0 * e * h + 6.0 * k * h * i)}
    T, d = case["T"], case["d"]
    gate = {"none": 0, "channel": d, "token": T * d}[case["gate"]]
    return {"bytes": 8.0 * T * d + 2 * (gate + d + (d if case["post"] else 0)), "flops": 10.0 * T * d}


# ------------------------------------------------- the definitions in 64 bits
def _exact_weight(q, z, s, group):
    """W[o, j] in 64 bits of one packed layer, output by nibble."""
    inn, words = q.shape
    w = torch.empty((words, 8, inn), dtype=torch.float64, device=q.device)
    for p in range(8):
        code = ((q.long() >> (4 * p)) & 15).T
        zero = ((z.long() >> (4 * p)) & 15).T.repeat_interleave(group, dim=1)
        w[:, p] = (code - zero).double()
    return w.reshape(words * 8, inn) * s.double().T.repeat_interleave(group, dim=1)


def _exact_lora(st):
    x = st["x"].double()
    y = torch.einsum("tj,oj->to", x, _exact_weight(*st["w"], st["case"]["group"]))
    for a in range(st["A"].shape[0]):
        rows = (st["ids"] == a).nonzero().reshape(-1)
        if rows.numel():
            low = torch.einsum("tj,rj->tr", x[rows], st["A"][a].double())
            y[rows] += st["c"][a].double() * torch.einsum("tr,or->to", low, st["B"][a].double())
    return {"y": y}


def _exact_moe(st):
    case = st["case"]
    T, k, i = case["T"], case["top_k"], case["inter"]
    x = st["x"].double()
    logits = torch.einsum("th,eh->te", x, st["router"].double())
    order = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
    wt = torch.softmax(logits, 1).gather(1, order)
    if case["renormalize"]:
        wt = wt / wt.sum(1, keepdim=True)
    if st["mask"] is not None:
        order[st["mask"] == 0] = -1
        wt[st["mask"] == 0] = 0
    y = torch.zeros_like(x)
    for e in range(case["experts"]):
        rows, slot = (order == e).nonzero(as_tuple=True)
        if rows.numel():
            gu = torch.einsum("th,oh->to", x[rows], _exact_weight(*(v[e] for v in st["gate_up"]), case["group"]))
            act = gu[:, :i] * torch.sigmoid(gu[:, :i]) * gu[:, i:]
            part = torch.einsum("ti,oi->to", act, _exact_weight(*(v[e] for v in st["down"]), case["group"]))
            y.index_add_(0, rows, wt[rows, slot].unsqueeze(1) * part)
    return {"y": y, "ids": order.to(torch.int32), "weights": wt}


def _exact_norm(st):
    r, v, d = st["r"].double(), st["v"].double(), st["case"]["d"]
    if st["post"] is not None:
        v = v / torch.sqrt(v.pow(2).sum(1, keepdim=True) / d + st["eps"]) * st["post"].double()
    if st["gate"] is not None:
        v = v * st["gate"].double()
    r = r + st["c"] * v
    return {"r": r, "n": r / torch.sqrt(r.pow(2).sum(1, keepdim=True) / d + st["eps"]) * st["pre"].double()}


def exact(case, seed):
    st = prepare(case, seed)
    return {"lora": _exact_lora, "moe": _exact_moe, "norm": _exact_norm}[case["op"]](st)
