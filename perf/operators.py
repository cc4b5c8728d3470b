"""Cases of the MoE routing, token permutation and 4-bit matrix-vector operators, for timing and comparison.

``listed()`` gives the measured cases and ``draw(rng)`` further ones of the same ranges.  ``prepare`` makes a
case's inputs on the GPU, ``run`` passes them once through the operator: in elementary torch operations in
32 bits (``own = False``) or through fp8_block_scaled_x128_amd (``own = True``).  ``exact`` gives the same
outputs from the definitions in 64 bits.

Operators (``case["op"]``):
  route             logits [T,E] -> the k experts of each token and their weights (softmax or sigmoid scores,
                    a balance bias for the choice, expert groups, renormalised weights)
  route_backward    gradient of those weights with respect to the logits
  dispatch          token rows -> the grouped layouts' rows, quantised to E4M3 with 1x128 scales
  combine           the experts' rows back to tokens, weighted; combine_backward its gradients
  w4                Y = X . W^T for few rows of X, W in 4 bits with group scales
  w4_experts        the same with the matrix of each of a token's experts
"""
import math

import torch

own = False

_BIG = torch.finfo(torch.float32).max
_INF = float("inf")


def listed():
    return [
        # one token of a decode step: 256 experts in 8 groups, 8 picked from the best 4 groups (latency)
        dict(name="route_1", op="route", T=1, E=256, k=8, n_group=8, topk_group=4, group_top=2, score="sigmoid",
             bias=True, off=0, renorm=True, scale=2.5, dtype="float32"),
        # a whole prefill batch through the same router
        dict(name="route_32768", op="route", T=32768, E=256, k=8, n_group=8, topk_group=4, group_top=2,
             score="sigmoid", bias=True, off=3, renorm=True, scale=2.5, dtype="float32"),
        # training, softmax scores that are not renormalised, sizes off every power of two
        dict(name="route_backward_8191", op="route_backward", T=8191, E=160, k=6, score="softmax", renorm=False,
             scale=16.0, dtype="bfloat16"),
        # a decode batch into the masked layout
        dict(name="dispatch_masked_128", op="dispatch", layout="masked", T=128, k=8, G=16, H=7168, M_max=256),
        # a prefill batch into the contiguous layout, ragged groups
        dict(name="dispatch_contiguous_4095", op="dispatch", layout="contiguous", T=4095, k=8, G=64, H=7168, M_max=0),
        # a decode batch back to tokens
        dict(name="combine_128", op="combine", T=128, k=8, H=7168, R=4096, lost=0),
        # a prefill batch back to tokens, some pairs dropped for capacity
        dict(name="combine_4096", op="combine", T=4096, k=8, H=7168, R=33792, lost=100),
        # training: gradients of the rows and of the weights
        dict(name="combine_backward_1000", op="combine_backward", T=1000, k=6, H=2048, R=6400, lost=7),
        # a projection of one new token, INT4 weights
        dict(name="w4_int4_1", op="w4", M=1, N=4096, K=7168, fmt="int4", group=128, zeros=False),
        # the largest projection, a small decode batch, MXFP4 weights
        dict(name="w4_mxfp4_13", op="w4", M=13, N=7168, K=16384, fmt="mxfp4", group=32, zeros=False),
        # the first expert layer of one token (gate and up rows, SwiGLU), 256 experts' weights in memory
        dict(name="w4_experts_1", op="w4_experts", T=1, k=8, E=256, N=4096, K=7168, fmt="mxfp4", group=32,
             zeros=False, swiglu=True, per_pair=False),
        # the second expert layer of a decode batch, INT4 with zero points, several tokens on an expert
        dict(name="w4_experts_16", op="w4_experts", T=16, k=8, E=64, N=7168, K=2048, fmt="int4", group=64,
             zeros=True, swiglu=False, per_pair=True),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["route", "route", "route_backward", "dispatch", "dispatch", "combine", "combine_backward", "w4", "w4", "w4",
                     "w4_experts", "w4_experts"])
    if op == "route":
        n_group = rng.choice([1, 1, 2, 4, 8])
        E = n_group * _log(rng, 4, 512 // n_group)
        topk_group = rng.randint(1, n_group)
        room = E // n_group * topk_group
        off = rng.choice([0, 0, rng.randint(0, max(0, E // 8))])
        score = rng.choice(["softmax", "sigmoid"])
        return dict(op=op, T=_log(rng, 1, 32768), E=E, k=rng.randint(1, min(16, room)), n_group=n_group, topk_group=topk_group,
                    group_top=rng.choice([1, 2]), score=score, bias=rng.random() < 0.5 or off > 0, off=off,
                    renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5, 16.0]), dtype=rng.choice(["float32", "bfloat16"]))
    if op == "route_backward":
        E = _log(rng, 8, 512)
        return dict(op=op, T=_log(rng, 1, 32768), E=E, k=rng.randint(1, min(16, E)), score=rng.choice(["softmax", "sigmoid"]),
                    renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5, 16.0]), dtype=rng.choice(["float32", "bfloat16"]))
    H = 128 * _log(rng, 4, 56)
    if op == "dispatch":
        G = _log(rng, 4, 256)
        k = rng.randint(1, min(8, G))
        layout = rng.choice(["masked", "contiguous"])
        T = _log(rng, 1, 512 if layout == "masked" else 4096)
        # capacity of a group: twice its even share, so that a crowded one may overflow
        return dict(op=op, layout=layout, T=T, k=k, G=G, H=H, M_max=max(8, 2 * T * k // G) if layout == "masked" else 0)
    if op in ("combine", "combine_backward"):
        T, k = _log(rng, 1, 4096 if op == "combine" else 2048), rng.randint(1, 8)
        lost = rng.choice([0, min(T * k, _log(rng, 1, 64))])
        return dict(op=op, T=T, k=k, H=H, R=T * k + rng.randint(0, 500), lost=lost)
    fmt = rng.choice(["mxfp4", "int4"])
    group = 32 if fmt == "mxfp4" else rng.choice([32, 64, 128])
    zeros = fmt == "int4" and rng.random() < 0.5
    if op == "w4":
        return dict(op=op, M=_log(rng, 1, 16), N=_log(rng, 64, 16384), K=group * _log(rng, 256 // group, 7168 // group),
                    fmt=fmt, group=group, zeros=zeros)
    E = _log(rng, 4, 64)
    k = rng.randint(1, min(8, E))
    per_pair = rng.random() < 0.5
    return dict(op=op, T=_log(rng, 1, 16), k=k, E=E, N=2 * _log(rng, 64, 2048), K=group * _log(rng, 256 // group, 4096 // group),
                fmt=fmt, group=group, zeros=zeros, swiglu=not per_pair, per_pair=per_pair)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 + int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _distinct(g, T, E, k):
    """k distinct experts for each token, some experts more popular than others."""
    liking = _normal(g, 1, E) * 0.5 + _normal(g, T, E)
    return liking.sort(dim=1, descending=True, stable=True).indices[:, :k].to(torch.int32).contiguous()


def _weights4(g, lead, N, K, fmt, group, zeros):
    """4-bit codes (two a byte, the even element in the low nibble), group scales and zero points."""
    W = torch.randint(0, 256, (*lead, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    if fmt == "mxfp4":
        scales = torch.randint(117, 123, (*lead, N, K // 32), generator=g, device="cuda", dtype=torch.uint8)
        return W, scales, None
    scales = (0.004 + 0.004 * torch.rand((*lead, N, K // group), generator=g, device="cuda")).to(torch.bfloat16)
    z = torch.randint(4, 12, (*lead, N, K // group), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    return W, scales, z


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    op = c["op"]
    s = {"case": c}
    if op in ("route", "route_backward"):
        T, E, k = c["T"], c["E"], c["k"]
        dt = getattr(torch, c["dtype"])
        logits = (_normal(g, T, E) * 1.5).to(dt)
        if op == "route":
            bias = None
            if c["bias"]:
                bias = _normal(g, E) * 0.05
                if c["off"]:  # experts taken out of service
                    bias[torch.randperm(E, generator=g, device="cuda")[: c["off"]]] = -_INF
            # A row whose choice hangs on a difference below 32-bit rounding has no one answer: it gets other logits.
            rows = torch.arange(T, device="cuda")
            for _ in range(50):
                rows = rows[_hangs(logits[rows], bias, c)]
                if rows.numel() == 0:
                    break
                logits[rows] = (_normal(g, rows.numel(), E) * 1.5).to(dt)
            s.update(logits=logits, bias=bias, ids=torch.zeros((T, k), dtype=torch.int32, device="cuda"),
                     weights=torch.zeros((T, k), dtype=torch.float32, device="cuda"))
        else:
            s.update(logits=logits, ids=_distinct(g, T, E, k), dweights=_normal(g, T, k), dlogits=torch.zeros_like(logits))
        return s
    if op == "dispatch":
        T, k, G, H = c["T"], c["k"], c["G"], c["H"]
        X = (_normal(g, T, H) * (1 + 8 * (torch.rand((1, H), generator=g, device="cuda") < 0.01))).to(torch.bfloat16)
        rows = G * c["M_max"] if c["layout"] == "masked" else -(-(T * k + 127 * min(G, T * k)) // 128) * 128
        shape = (G, c["M_max"]) if c["layout"] == "masked" else (rows,)
        s.update(X=X, ids=_distinct(g, T, G, k), rows=rows,
                 codes=torch.zeros((*shape, H), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
                 scales=torch.zeros((*shape[:-1], H // 128, shape[-1]), dtype=torch.float32, device="cuda"),
                 where=torch.zeros((G if c["layout"] == "masked" else rows,), dtype=torch.int32, device="cuda"),
                 row_map=torch.zeros((T, k), dtype=torch.int32, device="cuda"))
        return s
    if op in ("combine", "combine_backward"):
        T, k, H, R = c["T"], c["k"], c["H"], c["R"]
        Y = _normal(g, R, H).to(torch.bfloat16)
        row_map = torch.randperm(R, generator=g, device="cuda")[: T * k].to(torch.int32)
        row_map[torch.randperm(T * k, generator=g, device="cuda")[: c["lost"]]] = -1
        w = torch.rand((T, k), generator=g, device="cuda")
        s.update(Y=Y, row_map=row_map.view(T, k), weights=w / w.sum(1, keepdim=True))
        if op == "combine":
            s.update(out=torch.zeros((T, H), dtype=torch.bfloat16, device="cuda"))
        else:
            s.update(dout=_normal(g, T, H).to(torch.bfloat16), dY=torch.zeros_like(Y), dweights=torch.zeros_like(w))
        return s
    N, K = c["N"], c["K"]
    if op == "w4":
        W, sc, z = _weights4(g, (), N, K, c["fmt"], c["group"], c["zeros"])
        X = _normal(g, c["M"], K).to(torch.bfloat16)
        s.update(W=W, scales=sc, zeros=z, X=X, out=torch.zeros((c["M"], N), dtype=torch.bfloat16, device="cuda"))
        return s
    W, sc, z = _weights4(g, (c["E"],), N, K, c["fmt"], c["group"], c["zeros"])
    pairs = c["T"] * c["k"]
    X = _normal(g, pairs if c["per_pair"] else c["T"], K).to(torch.bfloat16)
    s.update(W=W, scales=sc, zeros=z, X=X, ids=_distinct(g, c["T"], c["E"], c["k"]),
             out=torch.zeros((pairs, N // 2 if c["swiglu"] else N), dtype=torch.bfloat16, device="cuda"))
    return s


def _choice64(logits, bias, c):
    """Scores, choice values with the groups left out at -inf, and the groups' sorted scores, in 64 bits."""
    x = logits.double().nan_to_num(nan=-_INF, posinf=_BIG, neginf=-_INF)
    if c["score"] == "sigmoid":
        sc = 1 / (1 + torch.exp(-x))
    else:
        e = torch.exp(x - x.amax(1, keepdim=True))
        sc = e / e.sum(1, keepdim=True)
    ch = sc if bias is None else sc + bias.double()
    ch = torch.where(x == -_INF, -_INF, ch)
    if c["n_group"] == 1:
        return sc, ch, None
    T, E = ch.shape
    per = ch.view(T, c["n_group"], E // c["n_group"])
    gs = per.sort(dim=2, descending=True).values[:, :, : c["group_top"]].sum(2)
    by = gs.sort(dim=1, descending=True, stable=True)
    keep = torch.zeros_like(gs, dtype=torch.bool).scatter_(1, by.indices[:, : c["topk_group"]], True)
    return sc, torch.where(keep.unsqueeze(2), per, -_INF).reshape(T, E), by.values


def _hangs(logits, bias, c):
    """Rows where two neighbouring values that decide the choice differ, but by under 4e-6 of their size."""
    _, ch, gs = _choice64(logits, bias, c)

    def close(v):
        d = v[:, :-1] - v[:, 1:]
        return ((d > 0) & (d < 4e-6 * v[:, :-1].abs())).any(1)

    bad = close(ch.sort(dim=1, descending=True).values[:, : c["k"] + 1])
    if gs is not None and c["topk_group"] < c["n_group"]:
        bad |= close(gs[:, c["topk_group"] - 1: c["topk_group"] + 1])
    return bad


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import fp8_block_scaled_x128_amd as fg
    c = s["case"]
    op = c["op"]
    if op == "route":
        return fg.route_topk(s["logits"], c["k"], bias=s["bias"], score=c["score"], n_group=c["n_group"],
                             topk_group=c["topk_group"], group_top=c["group_top"], renorm=c["renorm"], scale=c["scale"],
                             ids=s["ids"], weights=s["weights"])
    if op == "route_backward":
        return fg.route_topk_backward(s["logits"], s["ids"], s["dweights"], score=c["score"], renorm=c["renorm"],
                                      scale=c["scale"], dlogits=s["dlogits"])
    if op == "dispatch":
        if c["layout"] == "masked":
            return fg.moe_dispatch_masked(s["X"], s["ids"], c["G"], c["M_max"], codes=s["codes"], scales=s["scales"],
                                          masked_m=s["where"], row_map=s["row_map"])
        return fg.moe_dispatch_contiguous(s["X"], s["ids"], c["G"], codes=s["codes"], scales=s["scales"],
                                          m_indices=s["where"], row_map=s["row_map"])
    if op == "combine":
        return fg.moe_combine(s["Y"], s["weights"], row_map=s["row_map"], out=s["out"])
    if op == "combine_backward":
        return fg.moe_combine_backward(s["dout"], s["Y"], s["weights"], row_map=s["row_map"], dY=s["dY"],
                                       dweights=s["dweights"])
    if op == "w4":
        return fg.w4_gemv(s["X"], s["W"], s["scales"], zeros=s["zeros"], out=s["out"])
    return fg.w4_gemv_experts(s["X"], s["W"], s["scales"], s["ids"], zeros=s["zeros"], swiglu=c["swiglu"], out=s["out"])


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "route":
        return _plain_route(s["logits"], s["bias"], c)
    if op == "route_backward":
        return _plain_route_backward(s["logits"], s["ids"], s["dweights"], c)
    if op == "dispatch":
        return _plain_dispatch(s["X"], s["ids"], s["rows"], c)
    if op == "combine":
        rows = s["row_map"].long()
        y = torch.where((rows >= 0).unsqueeze(2), s["Y"][rows.clamp(min=0)].float(), 0.0)
        return (s["weights"].unsqueeze(2) * y).sum(1).to(torch.bfloat16)
    if op == "combine_backward":
        rows, R = s["row_map"].long(), s["Y"].shape[0]
        d = s["dout"].float().unsqueeze(1)
        y = s["Y"][rows.clamp(min=0)].float()
        dw = torch.where(rows >= 0, (d * y).sum(2), 0.0)
        dY = torch.zeros((R + 1, s["Y"].shape[1]), dtype=torch.bfloat16, device="cuda")
        dY[torch.where(rows >= 0, rows, R).view(-1)] = (s["weights"].unsqueeze(2) * d).to(torch.bfloat16).flatten(0, 1)
        return dY[:R], dw
    if op == "w4":
        V = _plain_decode(s["W"], s["scales"], s["zeros"], c)
        return (s["X"].float() @ V.t()).to(torch.bfloat16)
    pick = s["ids"].long().view(-1)
    z = None if s["zeros"] is None else s["zeros"][pick]
    V = _plain_decode(s["W"][pick], s["scales"][pick], z, c)
    x = s["X"].float()
    x = x if c["per_pair"] else x.repeat_interleave(c["k"], dim=0)
    y = torch.bmm(V, x.unsqueeze(2)).squeeze(2)
    if c["swiglu"]:
        half = c["N"] // 2
        gate, up = y[:, :half], y[:, half:]
        y = gate / (1 + torch.exp(-gate)) * up
    return y.to(torch.bfloat16)


def _plain_scores(logits, c):
    x = logits.float()
    x = torch.where(torch.isnan(x), -_INF, x).clamp(max=_BIG)
    if c["score"] == "sigmoid":
        return x, 1 / (1 + torch.exp(-x))
    e = torch.exp(x - x.amax(1, keepdim=True))
    return x, e / e.sum(1, keepdim=True)


def _plain_route(logits, bias, c):
    T, E = logits.shape
    x, sc = _plain_scores(logits, c)
    ch = sc if bias is None else sc + torch.where(torch.isnan(bias), -_INF, bias).clamp(max=_BIG)
    ch = torch.where(x == -_INF, -_INF, ch)
    if c["n_group"] > 1:
        per = ch.view(T, c["n_group"], E // c["n_group"])
        gs = per.sort(dim=2, descending=True).values[:, :, : c["group_top"]].sum(2)
        best = gs.sort(dim=1, descending=True, stable=True).indices[:, : c["topk_group"]]
        keep = (torch.arange(c["n_group"], device="cuda") == best.unsqueeze(2)).any(1)
        ch = torch.where(keep.unsqueeze(2), per, -_INF).reshape(T, E)
    top = ch.sort(dim=1, descending=True, stable=True)
    ids = top.indices[:, : c["k"]]
    there = top.values[:, : c["k"]] > -_INF
    w = torch.where(there, sc.gather(1, ids), 0.0)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return torch.where(there, ids, -1).to(torch.int32), w * c["scale"]


def _plain_route_backward(logits, ids, dweights, c):
    _, sc = _plain_scores(logits, c)
    ids = ids.long()
    s = sc.gather(1, ids)
    ds = dweights * c["scale"]
    if c["renorm"]:
        total = s.sum(1, keepdim=True)
        ds = (ds - (ds * s).sum(1, keepdim=True) / total) / total
    if c["score"] == "sigmoid":
        dx = torch.zeros_like(sc).scatter(1, ids, ds * s * (1 - s))
    else:
        spread = torch.zeros_like(sc).scatter(1, ids, ds)
        dx = sc * (spread - (ds * s).sum(1, keepdim=True))
    return dx.to(logits.dtype)


def _plain_dispatch(X, ids, rows, c):
    T, k, G, H, cap = c["T"], c["k"], c["G"], c["H"], c["M_max"]
    flat = ids.long().view(-1)
    mine = flat.unsqueeze(1) == torch.arange(G, device="cuda")
    rank = (mine.to(torch.int32).cumsum(0).gather(1, flat.unsqueeze(1)) - 1).squeeze(1)
    count = mine.sum(0)
    blocks = X.float().view(T, H // 128, 128)
    scale = blocks.abs().amax(2).clamp(min=1e-4) / 448.0
    code = (blocks / scale.unsqueeze(2)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(T, H).view(torch.uint8)
    if c["layout"] == "masked":
        row = torch.where(rank < cap, flat * cap + rank, rows)
        where = count.clamp(max=cap).to(torch.int32)
    else:
        first = ((count + 127) // 128 * 128).cumsum(0) - (count + 127) // 128 * 128
        row = first[flat] + rank
        at = torch.arange(rows, device="cuda").unsqueeze(1)
        inside = (at >= first) & (at < first + count)
        where = torch.where(inside.any(1), inside.to(torch.int32).argmax(1), -1).to(torch.int32)
    codes = torch.zeros((rows + 1, H), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((rows + 1, H // 128), dtype=torch.float32, device="cuda")
    token = torch.arange(T, device="cuda").repeat_interleave(k)
    codes[row] = code[token]
    scales[row] = scale[token]
    row_map = torch.where(row < rows, row, -1).to(torch.int32).view(T, k)
    codes, scales = codes[:rows].view(torch.float8_e4m3fn), scales[:rows]
    if c["layout"] == "masked":
        return codes.view(G, cap, H), scales.view(G, cap, H // 128).transpose(1, 2).contiguous(), where, row_map
    return codes, scales.t().contiguous(), where, row_map


def _plain_decode(W, scales, zeros, c):
    """4-bit weights as 32-bit values."""
    q = torch.stack((W & 15, W >> 4), dim=-1).flatten(-2)
    if c["fmt"] == "mxfp4":
        table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device="cuda")
        v = torch.cat((table, -table))[q.int()]
        v = v.unflatten(-1, (-1, 32)) * torch.exp2(scales.float() - 127.0).unsqueeze(-1)
        return v.flatten(-2)
    z = 8.0 if zeros is None else zeros.float().unsqueeze(-1)
    return ((q.float().unflatten(-1, (-1, c["group"])) - z) * scales.float().unsqueeze(-1)).flatten(-2)


def work(case):
    c = case
    op = c["op"]
    if op in ("route", "route_backward"):
        size = 4 if c["dtype"] == "float32" else 2
        T, E, k = c["T"], c["E"], c["k"]
        if op == "route":
            return {"bytes": T * E * size + (4 * E if c["bias"] else 0) + 8 * T * k, "flops": 6 * T * E}
        dense = c["score"] == "softmax" and not c["renorm"]
        return {"bytes": T * E * size + (T * E if dense else T * k) * size + 8 * T * k, "flops": 6 * T * (E if dense else k)}
    if op == "dispatch":
        T, k, H = c["T"], c["k"], c["H"]
        pairs = T * k
        rows = c["G"] if c["layout"] == "masked" else pairs
        return {"bytes": T * H * 2 + pairs * (H + H // 32) + 8 * pairs + 4 * rows, "flops": 3 * T * H}
    if op in ("combine", "combine_backward"):
        T, k, H = c["T"], c["k"], c["H"]
        pairs = T * k - c["lost"]
        if op == "combine":
            return {"bytes": pairs * H * 2 + T * H * 2 + 8 * T * k, "flops": 2 * pairs * H}
        return {"bytes": 2 * pairs * H * 2 + T * H * 2 + 12 * T * k, "flops": 3 * pairs * H}
    N, K = c["N"], c["K"]
    matrix = N * K // 2 + N * (K // c["group"]) * (1 if c["fmt"] == "mxfp4" else 3 if c["zeros"] else 2)
    if op == "w4":
        return {"bytes": matrix + 2 * c["M"] * (K + N), "flops": 2 * c["M"] * N * K}
    pairs = c["T"] * c["k"]
    used = c["E"] * (1 - (1 - c["k"] / c["E"]) ** c["T"])  # experts that at least one token picks, on average
    return {"bytes": int(used * matrix) + 2 * K * (pairs if c["per_pair"] else c["T"]) + 2 * pairs * (N // 2 if c["swiglu"] else N),
            "flops": 2 * pairs * N * K}


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    op = c["op"]
    if op == "route":
        sc, ch, _ = _choice64(s["logits"], s["bias"], c)
        top = ch.sort(dim=1, descending=True, stable=True)
        w = sc.gather(1, top.indices[:, : c["k"]]) * (top.values[:, : c["k"]] > -_INF)
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
        return None, w * c["scale"]
    if op == "route_backward":
        x = s["logits"].double()
        ids = s["ids"].long()
        g = s["dweights"].double() * c["scale"]
        dx = torch.zeros_like(x)
        if c["score"] == "sigmoid":
            p = torch.sigmoid(x.gather(1, ids))
            if c["renorm"]:
                share = p / p.sum(1, keepdim=True)
                g = (g - (g * share).sum(1, keepdim=True)) / p.sum(1, keepdim=True)
            return dx.scatter_(1, ids, g * p * (1 - p))
        if c["renorm"]:  # the same as a softmax over the picked experts alone
            p = torch.softmax(x.gather(1, ids), 1)
            return dx.scatter_(1, ids, p * (g - (g * p).sum(1, keepdim=True)))
        p = torch.softmax(x, 1)
        dx.scatter_(1, ids, g)
        return p * (dx - (dx * p).sum(1, keepdim=True))
    if op == "dispatch":
        T, k, H = c["T"], c["k"], c["H"]
        amax = s["X"].double().view(T, H // 128, 128).abs().amax(2).clamp(min=1e-4) / 448
        shape = s["scales"].shape
        scales = torch.zeros((s["rows"], H // 128), dtype=torch.float64, device="cuda")
        ids = s["ids"].cpu().view(-1).tolist()
        count = [0] * c["G"]
        rank = []
        for e in ids:
            rank.append(count[e])
            count[e] += 1
        if c["layout"] == "masked":
            at = [(e * c["M_max"] + r, p // k) for p, (e, r) in enumerate(zip(ids, rank)) if r < c["M_max"]]
        else:
            first = [0]
            for n in count:
                first.append(first[-1] + (n + 127) // 128 * 128)
            at = [(first[e] + r, p // k) for p, (e, r) in enumerate(zip(ids, rank))]
        at = torch.tensor(at, device="cuda").t()
        scales[at[0]] = amax[at[1]]
        if c["layout"] == "masked":
            return None, scales.view(c["G"], c["M_max"], H // 128).transpose(1, 2).reshape(shape), None, None
        return None, scales.t().contiguous(), None, None
    if op == "combine":
        out = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device="cuda")
        for j in range(c["k"]):
            there = s["row_map"][:, j] >= 0
            out[there] += s["weights"][there, j].double().unsqueeze(1) * s["Y"][s["row_map"][there, j].long()].double()
        return out
    if op == "combine_backward":
        dY = torch.zeros(s["Y"].shape, dtype=torch.float64, device="cuda")
        dw = torch.zeros(s["weights"].shape, dtype=torch.float64, device="cuda")
        for j in range(c["k"]):
            there = s["row_map"][:, j] >= 0
            rows, d = s["row_map"][there, j].long(), s["dout"][there].double()
            dY[rows] = s["weights"][there, j].double().unsqueeze(1) * d
            dw[there, j] = (d * s["Y"][rows].double()).sum(1)
        return dY, dw
    if op == "w4":
        return s["X"].double() @ _value64(s["W"], s["scales"], s["zeros"], c).t()
    ids = s["ids"].view(-1)
    x = s["X"].double()
    x = x if c["per_pair"] else x[torch.arange(len(ids), device="cuda") // c["k"]]
    y = torch.zeros((len(ids), c["N"]), dtype=torch.float64, device="cuda")
    for e in sorted(set(ids.tolist())):
        on = ids == e
        z = None if s["zeros"] is None else s["zeros"][e]
        y[on] = x[on] @ _value64(s["W"][e], s["scales"][e], z, c).t()
    if c["swiglu"]:
        gate, up = y.chunk(2, dim=1)
        y = gate * torch.sigmoid(gate) * up
    return y


def _value64(W, scales, zeros, c):
    """The weights' values in 64 bits, from the bit fields."""
    N = W.shape[0]
    q = torch.zeros((N, c["K"]), dtype=torch.int32, device="cuda")
    q[:, 0::2] = (W % 16).int()
    q[:, 1::2] = torch.div(W, 16, rounding_mode="floor").int()
    step = scales.shape[1]
    if c["fmt"] == "mxfp4":
        power, bit = (q >> 1) & 3, q & 1
        size = torch.where(power == 0, bit * 0.5, (1 + 0.5 * bit) * 2.0 ** (power - 1.0)).double()
        v = size * (1 - 2 * (q >> 3)).double()
        return (v.view(N, step, 32) * 2.0 ** (scales.double() - 127).unsqueeze(2)).view(N, -1)
    z = 8.0 if zeros is None else zeros.double().unsqueeze(2)
    return ((q.double().view(N, step, -1) - z) * scales.double().unsqueeze(2)).view(N, -1)
