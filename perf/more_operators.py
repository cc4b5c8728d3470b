"""Cases of the gated feed-forward block, its gradients and the low-rank adapters, for timing and comparison.

``listed()`` gives the measured cases and ``draw(rng)`` further ones of the same ranges.  ``prepare`` makes a
case's inputs on the GPU, ``run`` passes them once through the operator: in elementary torch operations in
32 bits (``own = False``) or through fp8_block_scaled_x128_amd (``own = True``).  ``exact`` gives the same
outputs from the definitions in 64 bits.

Operators (``case["op"]``):
  gated           X [M,K], W [2I,K] (gate rows, then up rows) -> act(X Wg^T) * (X Wu^T), and the two products
                  themselves where a backward pass is to follow (keep)
  gated_backward  gradients of that with respect to X and W, from the kept products or without them
  lora            out[t] = Y[t] + s[a] B[a] (A[a] x[t]) with the adapter a = ids[t] of each row, -1 for none
"""
import math

import torch

own = False


def listed():
    return [
        # one token of a decode step through a shared expert's first layer (weights' bytes, latency)
        dict(name="gated_1", op="gated", M=1, I=2048, K=7168, act="silu", keep=False),
        # a decode batch through the same layer
        dict(name="gated_64", op="gated", M=64, I=2048, K=7168, act="silu", keep=False),
        # a prefill batch
        dict(name="gated_4096", op="gated", M=4096, I=2048, K=7168, act="silu", keep=False),
        # training's forward pass, products kept, sizes off every tile
        dict(name="gated_keep_1001", op="gated", M=1001, I=1416, K=2056, act="gelu_tanh", keep=True),
        # training's backward pass of the layer
        dict(name="gated_backward_4096", op="gated_backward", M=4096, I=2048, K=7168, act="silu", keep=True),
        # the same without kept products, sizes off every tile
        dict(name="gated_backward_1023", op="gated_backward", M=1023, I=1416, K=2056, act="gelu_tanh", keep=False),
        # a short sequence
        dict(name="gated_backward_77", op="gated_backward", M=77, I=512, K=1536, act="silu", keep=True),
        # one token's adapter beside a projection (latency)
        dict(name="lora_1", op="lora", T=1, L=64, R=16, K=7168, N=4096, mix="sorted", none=0),
        # a decode batch, every row a request of its own, some without an adapter
        dict(name="lora_decode_256", op="lora", T=256, L=64, R=16, K=7168, N=4096, mix="ordered", none=13),
        # a few requests' rows in arrival order, small rank, odd sizes
        dict(name="lora_mixed_45", op="lora", T=45, L=9, R=8, K=1544, N=2112, mix="any", none=5),
        # prefill of eight requests
        dict(name="lora_prefill_8192", op="lora", T=8192, L=8, R=32, K=7168, N=4096, mix="sorted", none=0),
        # prefill with a large rank
        dict(name="lora_prefill_2000", op="lora", T=2000, L=4, R=128, K=2048, N=7168, mix="sorted", none=100),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_backward", "lora", "lora"])
    if op != "lora":
        return dict(op=op, M=_log(rng, 1, 4096), I=8 * _log(rng, 8, 256), K=8 * _log(rng, 16, 896),
                    act=rng.choice(["silu", "gelu_tanh"]), keep=rng.random() < 0.5)
    R = 8 * _log(rng, 1, 16)
    T = _log(rng, 1, 8192)
    # rows in arrival order mix adapters freely only in batches of single tokens; longer ones come by request
    mix = rng.choice(["any", "ordered", "sorted"]) if T <= 512 else rng.choice(["ordered", "sorted"])
    return dict(op=op, T=T, L=_log(rng, 1, 1024 // R), R=R, K=8 * _log(rng, 16, 896), N=8 * _log(rng, 8, 512),
                mix=mix, none=rng.choice([0, T // 20]))


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(7000003 + int(seed))
    return g


def _normal(g, *shape, scale=1.0):
    """bfloat16 values, normal."""
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(torch.bfloat16)


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    K = c["K"]
    if c["op"] != "lora":
        M, I = c["M"], c["I"]
        s = dict(case=c, X=_normal(g, M, K), W=_normal(g, 2 * I, K, scale=K ** -0.5), pre=None)
        if c["keep"]:
            s["pre"] = torch.zeros((M, 2 * I), dtype=torch.bfloat16, device="cuda")
        if c["op"] == "gated":
            s["out"] = torch.zeros((M, I), dtype=torch.bfloat16, device="cuda")
            return s
        if c["keep"]:  # as the forward pass left them
            s["pre"] = (s["X"].float() @ s["W"].float().t()).to(torch.bfloat16)
        s.update(dH=_normal(g, M, I), dX=torch.zeros_like(s["X"]), dW=torch.zeros_like(s["W"]),
                 dpre=torch.zeros((M, 2 * I), dtype=torch.bfloat16, device="cuda"))
        return s
    T, L, R, N = c["T"], c["L"], c["R"], c["N"]
    ids = torch.randint(0, L, (T,), generator=g, device="cuda", dtype=torch.int32)
    ids[torch.randperm(T, generator=g, device="cuda")[: c["none"]]] = -1
    if c["mix"] == "sorted":  # a request's rows follow each other
        ids = ids.sort(stable=True).values
    # an order that brings a request's rows together, which a program finds once for a batch and all its layers
    order = ids.argsort(stable=True).to(torch.int32) if c["mix"] == "ordered" else None
    return dict(case=c, X=_normal(g, T, K), Y=_normal(g, T, N), A=_normal(g, L, R, K, scale=K ** -0.5),
                B=_normal(g, L, N, R, scale=R ** -0.5), ids=ids, order=order,
                scales=0.5 + torch.rand((L,), generator=g, device="cuda"),
                out=torch.zeros((T, N), dtype=torch.bfloat16, device="cuda"))


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import fp8_block_scaled_x128_amd as fg
    c = s["case"]
    if c["op"] == "gated":
        out = fg.gated_ffn(s["X"], s["W"], act=c["act"], pre=s["pre"], out=s["out"])
        return (out, s["pre"]) if c["keep"] else out
    if c["op"] == "gated_backward":
        return fg.gated_ffn_backward(s["dH"], s["X"], s["W"], pre=s["pre"], act=c["act"], dX=s["dX"], dW=s["dW"],
                                     dpre=s["dpre"])
    return fg.lora_add(s["Y"], s["X"], s["A"], s["B"], s["ids"], scales=s["scales"], order=s["order"], out=s["out"])


_GELU_A, _GELU_B = math.sqrt(2 / math.pi), 0.044715


def _plain_act(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        sg = 1 / (1 + torch.exp(-g))
        return g * sg, sg * (1 + g * (1 - sg))
    inner = 2 * _GELU_A * (g + _GELU_B * g * g * g)
    sg = 1 / (1 + torch.exp(-inner))
    return g * sg, sg + g * sg * (1 - sg) * 2 * _GELU_A * (1 + 3 * _GELU_B * g * g)


def _run_plain(s):
    c = s["case"]
    if c["op"] == "lora":
        return _plain_lora(s, c)
    x, w = s["X"].float(), s["W"].float()
    if c["op"] == "gated":
        p = x @ w.t()
        a, _ = _plain_act(p[:, : c["I"]], c["act"])
        out = (a * p[:, c["I"]:]).to(torch.bfloat16)
        return (out, p.to(torch.bfloat16)) if c["keep"] else out
    p = s["pre"].float() if c["keep"] else x @ w.t()
    a, da = _plain_act(p[:, : c["I"]], c["act"])
    d = s["dH"].float()
    dp = torch.cat((d * p[:, c["I"]:] * da, d * a), dim=1)
    return (dp @ w).to(torch.bfloat16), (dp.t() @ x).to(torch.bfloat16)


def _plain_lora(s, c):
    x, ids = s["X"].float(), s["ids"].long()
    there = ids >= 0
    at = ids.clamp(min=0)
    if c["T"] <= c["L"]:  # each row's own matrices
        v = torch.bmm(s["A"][at].float(), x.unsqueeze(2))
        d = torch.bmm(s["B"][at].float(), v).squeeze(2)
    else:  # all adapters' for all rows, the others' taken out
        v = (x @ s["A"].float().flatten(0, 1).t()).view(c["T"], c["L"], c["R"])
        mine = at.unsqueeze(1) == torch.arange(c["L"], device="cuda")
        v = torch.where(mine.unsqueeze(2), v, 0.0).flatten(1)
        d = v @ s["B"].float().transpose(1, 2).flatten(0, 1)
    d = d * s["scales"][at].unsqueeze(1)
    return (s["Y"].float() + torch.where(there.unsqueeze(1), d, 0.0)).to(torch.bfloat16)


def work(case):
    c = case
    K = c["K"]
    if c["op"] == "gated":
        M, I = c["M"], c["I"]
        return {"bytes": 2 * (M * K + 2 * I * K + M * I + (2 * M * I if c["keep"] else 0)), "flops": 4 * M * I * K}
    if c["op"] == "gated_backward":
        M, I = c["M"], c["I"]
        return {"bytes": 2 * (2 * M * K + 4 * I * K + M * I + (2 * M * I if c["keep"] else 0)),
                "flops": (8 if c["keep"] else 12) * M * I * K}
    T, L, R, N = c["T"], c["L"], c["R"], c["N"]
    used = L * (1 - (1 - 1 / L) ** (T - c["none"])) if L > 1 else 1  # adapters that at least one row has, on average
    return {"bytes": 2 * T * (K + 2 * N) + int(used * 2 * R * (K + N)) + 4 * T, "flops": 2 * (T - c["none"]) * R * (K + N)}


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "lora":
        out = s["Y"].double()
        for a in range(c["L"]):
            rows = (s["ids"] == a).nonzero().squeeze(1)
            low = s["X"][rows].double() @ s["A"][a].double().t()
            out[rows] += s["scales"][a].double() * (low @ s["B"][a].double().t())
        return out
    x, w = s["X"].double(), s["W"].double()
    wg, wu = w.chunk(2, dim=0)
    if c["keep"] and c["op"] == "gated_backward":
        g, u = s["pre"].double().chunk(2, dim=1)
    else:
        g, u = x @ wg.t(), x @ wu.t()
    # both activations are g times a logistic function of z(g), whose derivative is dz
    if c["act"] == "silu":
        z, dz = g, torch.ones_like(g)
    else:
        z = math.sqrt(8 / math.pi) * (g + 0.044715 * g ** 3)
        dz = math.sqrt(8 / math.pi) * (1 + 0.134145 * g ** 2)
    gate = torch.sigmoid(z)
    if c["op"] == "gated":
        out = g * gate * u
        return (out, torch.cat((g, u), dim=1)) if c["keep"] else out
    d = s["dH"].double()
    dg, du = d * u * gate * (1 + g * dz * torch.sigmoid(-z)), d * g * gate
    return dg @ wg + du @ wu, torch.cat((dg.t() @ x, du.t() @ x), dim=0)
