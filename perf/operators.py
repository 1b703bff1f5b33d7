"""Cases of the operators for rows that are routed to one of many weights.

* route: the k greatest router logits of a token and their softmax weights (and the logits' gradient)
* sort: the row of every (token, choice) among the experts' rows, in the layouts of the grouped products
* dispatch: tokens copied to their experts' rows, as bfloat16 or quantised 1x128 to FP8 (and the tokens' gradient)
* combine: the experts' rows weighted and summed back to tokens (and the rows' and weights' gradients)
* lora: a shared projection with a low-rank adapter per row, beside a BF16 or an FP8 base product

``own`` chooses who computes ``run``: elementary torch operations in 32 bits, or this repository's calls.
"""
import math

import torch

own = False


# ---- the cases ---------------------------------------------------------------------------------------------------

def listed():
    return [
        # one decode step of 16 sequences: latency alone
        dict(name="route_decode", op="route", T=16, E=256, k=8, dtype="f32", renorm=True, scale=2.5, grad=False),
        # a training step's router, forward and backward, weights of the softmax over all experts
        dict(name="route_train", op="route", T=16383, E=128, k=6, dtype="bf16", renorm=False, scale=1.0, grad=True),
        # decode into the masked layout (16 experts of 256 rows)
        dict(name="sort_decode", op="sort", T=64, k=8, G=16, layout="masked", cap=256),
        # prefill over many experts, contiguous layout
        dict(name="sort_prefill", op="sort", T=16384, k=8, G=256, layout="contiguous", cap=0),
        # prefill: the FP8 operand of the contiguous expert products, about 32768 rows of 7168
        dict(name="dispatch_prefill", op="dispatch", T=4096, k=8, H=7168, G=8, to="fp8", layout="contiguous", cap=0, grad=False),
        # a ragged training micro-batch: bfloat16 rows, and the tokens' gradient
        dict(name="dispatch_train", op="dispatch", T=1021, k=4, H=2112, G=16, to="bf16", layout="contiguous", cap=0, grad=True),
        # decode: the masked product's rows back to 64 tokens
        dict(name="combine_decode", op="combine", T=64, k=8, H=7168, G=16, layout="masked", cap=256, grad=False),
        # a training step: rows back to tokens, then both gradients
        dict(name="combine_train", op="combine", T=4095, k=8, H=4096, G=64, layout="contiguous", cap=0, grad=True),
        # one token of one request
        dict(name="lora_token", op="lora", base="bf16", M=1, N=4096, K=7168, G=8, R=16, requests=1),
        # a decode batch: every row a request with an adapter of its own choice (or none)
        dict(name="lora_decode", op="lora", base="fp8", M=64, N=7168, K=2048, G=64, R=16, requests=64),
        # ragged prefill of a few requests beside an FP8 projection
        dict(name="lora_ragged", op="lora", base="fp8", M=777, N=2112, K=7168, G=32, R=32, requests=5),
        # a large prefill beside a BF16 projection
        dict(name="lora_prefill", op="lora", base="bf16", M=4096, N=4096, K=7168, G=16, R=64, requests=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["route", "sort", "dispatch", "combine", "lora", "lora"])
    if op == "route":
        E = _log(rng, 8, 512)
        return dict(op=op, T=_log(rng, 1, 16384), E=E, k=rng.randint(1, min(E, 10)), dtype=rng.choice(["f32", "bf16"]),
                    renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]), grad=rng.random() < 0.5)
    layout = rng.choice(["contiguous", "masked"])
    if op == "sort":
        G, T = _log(rng, 2, 384), _log(rng, 1, 16384)
        k = rng.randint(1, min(G, 8))
        return dict(op=op, T=T, k=k, G=G, layout=layout, cap=0 if layout == "contiguous" else _cap(rng, T * k, G))
    if op in ("dispatch", "combine"):
        G, T = _log(rng, 2, 64), _log(rng, 1, 4096)
        k = rng.randint(1, min(G, 8))
        H = _log(rng, 64, 7168)
        c = dict(op=op, T=T, k=k, H=H, G=G, layout=layout, cap=0 if layout == "contiguous" else _cap(rng, T * k, G))
        if op == "combine":
            return dict(c, H=min(H, 4096), grad=rng.random() < 0.5)
        if rng.random() < 0.5:
            return dict(c, H=128 * max(1, H // 128), to="fp8", grad=False)
        return dict(c, H=min(H, 2112), to="bf16", grad=rng.random() < 0.7)
    base = rng.choice(["bf16", "fp8"])
    M = _log(rng, 1, 4096)
    return dict(op=op, base=base, M=M, N=_log(rng, 64, 4096), K=(64 if base == "bf16" else 128) * rng.randint(2, 56), G=_log(rng, 1, 64),
                R=8 * rng.randint(1, 8), requests=M if M <= 128 and rng.random() < 0.7 else min(M, rng.randint(1, 24)))


def _cap(rng, slots, G):
    """Rows an expert has room for: mostly enough, now and then not."""
    return max(1, round(rng.choice([0.9, 2.0, 2.0]) * slots / G) + rng.randint(0, 40))


def _rows(case):
    """Rows of the sorted layout: enough for every choice with each expert's run rounded up to 128 rows."""
    if case["layout"] == "masked":
        return case["G"] * case["cap"]
    S = case["T"] * case["k"]
    return (S + 127 * min(case["G"], S)) // 128 * 128


def work(case):
    op = case["op"]
    if op == "route":
        T, E, k, e = case["T"], case["E"], case["k"], 2 if case["dtype"] == "bf16" else 4
        b, f = T * E * e + T * k * 8, T * E * (4 + k)
        return {"bytes": b + (T * (2 * E * e + 3 * k * 4) if case["grad"] else 0), "flops": f + (T * E * 6 if case["grad"] else 0)}
    if op == "lora":
        M, N, K, G, R = (case[n] for n in ("M", "N", "K", "G", "R"))
        used = G * (1 - (1 - 1 / G) ** (case["requests"] * 7 / 8)) if G > 1 else 1.0
        adapters = used * R * (K + N) * 2 + M * 4 + G * 4
        if case["base"] == "bf16":
            b = 2 * (M * K + N * K + M * N)
        else:
            b = M * K + N * K + 4 * (K // 128) * (M + -(-N // 128)) + 2 * (M * K + M * N)
        return {"bytes": b + adapters, "flops": 2.0 * M * N * K + 2.0 * M * R * (K + N)}
    T, k, S = case["T"], case["k"], case["T"] * case["k"]
    if op == "sort":
        return {"bytes": 8 * S + 4 * case["G"] + (4 * _rows(case) if case["layout"] == "contiguous" else 0), "flops": 4.0 * S}
    H = case["H"]
    if op == "dispatch":
        if case["to"] == "fp8":
            return {"bytes": 2 * T * H + 4 * S + S * H + 4 * S * H // 128, "flops": 3.0 * T * H}
        b = 2 * T * H + 4 * S + 2 * S * H
        return {"bytes": b * (2 if case["grad"] else 1), "flops": float(S * H) if case["grad"] else float(T)}
    b = 2 * S * H + 8 * S + 2 * T * H
    if case["grad"]:
        b += 2 * T * H + 4 * S * H + 12 * S
    return {"bytes": b, "flops": (5.0 if case["grad"] else 2.0) * S * H}


# ---- inputs ------------------------------------------------------------------------------------------------------

def _choices(gen, T, k, G):
    """k different experts a token, some experts more popular than others; a few choices belong to no expert here."""
    score = torch.randn(T, G, generator=gen, device="cuda") + 0.5 * torch.randn(G, generator=gen, device="cuda")
    ids = torch.argsort(score, dim=1, descending=True)[:, :k].to(torch.int32)
    return torch.where(torch.rand(T, k, generator=gen, device="cuda") < 0.02, -1, ids).contiguous()


def _codes(x, rows):
    """e4m3 codes and scales of x in blocks of `rows` x 128."""
    M, K = x.shape
    pad = torch.nn.functional.pad(x.float(), (0, 0, 0, -M % rows)).view(-1, rows, K // 128, 128)
    amax = pad.abs().amax(dim=(1, 3))
    s = torch.where(amax > 0, amax / 448, 1.0)
    q = (pad / s[:, None, :, None]).clamp(-448, 448).view(-1, K)[:M]
    return q.to(torch.float8_e4m3fn).view(torch.uint8).contiguous(), s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device="cuda") * scale

    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        logits = normal(T, E, scale=1.5) + normal(E, scale=0.5)
        # one token in 16 may use half of the experts only, and one may use none
        half = (torch.arange(T, device="cuda") % 16 == 7)[:, None] & (torch.arange(E, device="cuda") < E // 2)
        logits = logits.masked_fill(half, -math.inf)
        if T > 16:
            logits[11] = -math.inf
        return dict(case=case, logits=logits.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32), dw=normal(T, k))
    if op == "lora":
        M, N, K, G, R, n = (case[x] for x in ("M", "N", "K", "G", "R", "requests"))
        x = normal(M, K).to(torch.bfloat16)
        w = normal(N, K, scale=K ** -0.5).to(torch.bfloat16)
        # requests of uneven lengths one after the other, each with an adapter of its own choice or, one in eight, none
        if n < M:
            ends = torch.sort(torch.randint(1, M, (n - 1,), generator=gen, device="cuda")).values
            request = torch.searchsorted(ends, torch.arange(M, device="cuda"), right=True)
        else:
            request = torch.arange(M, device="cuda")
        pick = torch.randint(0, G, (M,), generator=gen, device="cuda")
        none = torch.rand(M, generator=gen, device="cuda") < (0.125 if n > 1 else 0.0)
        ids = torch.where(none, -1, pick)[request].to(torch.int32)
        s = dict(case=case, x=x, ids=ids, la=normal(G, R, K, scale=K ** -0.5).to(torch.bfloat16), lb=normal(G, N, R, scale=0.5 * R ** -0.5).to(torch.bfloat16),
                 scale=torch.rand(G, generator=gen, device="cuda") + 0.5)
        if case["base"] == "bf16":
            return dict(s, w=w)
        a, sa = _codes(x, 1)
        b, sb = _codes(w, 128)
        return dict(s, a=a, sa=sa.t().contiguous(), b=b, sb=sb.contiguous())
    T, k, G = case["T"], case["k"], case["G"]
    ids = _choices(gen, T, k, G)
    if op == "sort":
        return dict(case=case, ids=ids)
    H, M = case["H"], _rows(case)
    row = _sorted(case, ids)[0]
    lead = (G, case["cap"]) if case["layout"] == "masked" else (M,)
    # buffers that a program keeps: rows that no token has stay as they are
    if op == "dispatch":
        s = dict(case=case, row=row, x=normal(T, H).to(torch.bfloat16))
        if case["to"] == "fp8":
            s["x"] = (s["x"] * torch.exp(normal(T, 1))).to(torch.bfloat16)
            return dict(s, a=torch.zeros(*lead, H, dtype=torch.uint8, device="cuda"), sa=torch.zeros(*lead[:-1], H // 128, lead[-1], device="cuda"))
        s["a"] = torch.zeros(*lead, H, dtype=torch.bfloat16, device="cuda")
        if case["grad"]:
            s["da"] = normal(M, H).to(torch.bfloat16).view(*lead, H)
        return s
    s = dict(case=case, row=row, y=normal(M, H).to(torch.bfloat16).view(*lead, H), w=torch.softmax(normal(T, k), 1))
    if case["grad"]:
        s |= dict(dout=normal(T, H).to(torch.bfloat16), dy=torch.zeros(*lead, H, dtype=torch.bfloat16, device="cuda"))
    return s


# ---- the plain forms ---------------------------------------------------------------------------------------------

def _sorted(case, ids):
    """(row [T,k], m_indices [M], counts [G]) of the contiguous layout, or (row [T,k], masked_m [G]) of the masked one."""
    T, k, G, flat = case["T"], case["k"], case["G"], ids.reshape(-1).long()
    upto = torch.cumsum(torch.arange(G, device=ids.device)[:, None] == flat, 1, dtype=torch.int32)
    counts = upto[:, -1]
    live, e = flat >= 0, flat.clamp(min=0)
    rank = upto.gather(0, e[None])[0] - 1
    if case["layout"] == "masked":
        row = torch.where(live & (rank < case["cap"]), e * case["cap"] + rank, -1)
        return row.to(torch.int32).view(T, k), counts.clamp(max=case["cap"]).contiguous()
    M = _rows(case)
    ends = torch.cumsum((counts + 127) // 128 * 128, 0)
    first = ends - (counts + 127) // 128 * 128
    row = torch.where(live, first[e] + rank, -1)
    at = torch.arange(M, device=ids.device)
    g = torch.searchsorted(ends, at, right=True).clamp(max=G - 1)
    m_indices = torch.where((at >= first[g]) & (at < first[g] + counts[g]), g, -1)
    return row.to(torch.int32).view(T, k), m_indices.to(torch.int32), counts.contiguous()


def _weights(logits, k, renorm, scale):
    """ids, weights and the softmax over all experts; an expert at -inf is not there, and fewer than k leave -1 and 0."""
    x = logits.float()
    order = torch.argsort(x, dim=1, descending=True, stable=True)[:, :k]
    top = x.gather(1, order)
    there = top > -math.inf
    m = x.amax(1, keepdim=True)
    p = torch.where(x > -math.inf, torch.exp(x - m), 0.0)
    q = p / p.sum(1, keepdim=True).clamp(min=1e-30)
    w = torch.where(there, q.gather(1, order), 0.0)
    if renorm:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-30)
    return torch.where(there, order, -1).to(torch.int32), w * scale, q


def _place(values, row, M):
    """values [T,k,...] or [T,1,...] at their rows of M, zeros elsewhere."""
    T, k = row.shape
    out = torch.zeros(M + 1, *values.shape[2:], dtype=values.dtype, device=values.device)
    out[torch.where(row < 0, M, row.long())] = values.expand(T, k, *values.shape[2:])
    return out[:M]


def _gathered(rows, row):
    """rows [M,H] at row [T,k] in 32 bits, zeros where there is none."""
    return torch.where(row[..., None] >= 0, rows[row.clamp(min=0).long()].float(), 0.0)


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "route":
        k, renorm, scale = case["k"], case["renorm"], case["scale"]
        ids, w, q = _weights(s["logits"], k, renorm, scale)
        if not case["grad"]:
            return ids, w
        there = ids >= 0
        at = ids.clamp(min=0).long()
        dw = torch.where(there, s["dw"], 0.0)
        mean = (w * dw).sum(1, keepdim=True)
        if renorm:
            d = torch.zeros_like(q).scatter_add_(1, at, w * (dw - mean / scale))
        else:
            d = torch.zeros_like(q).scatter_add_(1, at, w * dw) - q * mean
        return ids, w, d.to(s["logits"].dtype)
    if op == "sort":
        return _sorted(case, s["ids"])
    if op == "lora":
        M, N, K, G, R = (case[n] for n in ("M", "N", "K", "G", "R"))
        x, ids = s["x"].float(), s["ids"].long()
        if case["base"] == "bf16":
            d = x @ s["w"].float().t()
        else:
            a = s["a"].view(torch.float8_e4m3fn).float() * s["sa"].t().repeat_interleave(128, 1)
            b = s["b"].view(torch.float8_e4m3fn).float() * s["sb"].repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)
            d = a @ b.t()
        # every adapter's product with every row, the other adapters' columns then cleared
        mine = ids[:, None] == torch.arange(G, device=ids.device)
        h = (x @ s["la"].float().view(G * R, K).t()).view(M, G, R) * torch.where(mine, s["scale"], 0.0)[..., None]
        d = d + h.view(M, G * R) @ s["lb"].float().permute(0, 2, 1).reshape(G * R, N)
        return d.to(torch.bfloat16)
    row, H = s["row"], case["H"]
    M = _rows(case)
    T = row.shape[0]
    if op == "dispatch":
        if case["to"] == "fp8":
            x = s["x"].float().view(T, H // 128, 128)
            amax = x.abs().amax(2)
            sc = torch.where(amax > 0, amax / 448, 1.0)
            q = (x / sc[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(T, 1, H)
            a = _place(q, row, M).view(s["a"].shape).view(torch.float8_e4m3fn)
            sa = _place(sc[:, None], row, M)
            sa = sa.view(case["G"], case["cap"], -1).transpose(1, 2) if case["layout"] == "masked" else sa.t()
            return a, sa.contiguous()
        a = _place(s["x"][:, None], row, M).view(s["a"].shape)
        if not case["grad"]:
            return a
        return a, _gathered(s["da"].view(M, H), row).sum(1).to(torch.bfloat16)
    y = _gathered(s["y"].view(M, H), row)
    out = (y * s["w"][..., None]).sum(1).to(torch.bfloat16)
    if not case["grad"]:
        return out
    dout = s["dout"].float()[:, None]
    dw = (y * dout).sum(2)
    return out, _place((s["w"][..., None] * dout).to(torch.bfloat16), row, M).view(s["y"].shape), dw


# ---- one pass ----------------------------------------------------------------------------------------------------

def run(state):
    if not own:
        return _plain(state)
    import moe_grouped_gemm_act_amd as fg
    case = state["case"]
    op = case["op"]
    if op == "route":
        kw = dict(renormalize=case["renorm"], scale=case["scale"])
        ids, w = fg.moe_topk(state["logits"], case["k"], **kw)
        if not case["grad"]:
            return ids, w
        return ids, w, fg.moe_topk_backward(state["logits"], ids, w, state["dw"], **kw)
    if op == "sort":
        if case["layout"] == "masked":
            return fg.moe_sort_masked(state["ids"], case["G"], case["cap"])
        return fg.moe_sort_contiguous(state["ids"], case["G"], _rows(case))
    if op == "lora":
        if case["base"] == "bf16":
            return fg.gemm_bf16_nt_lora(state["x"], state["w"], state["la"], state["lb"], state["ids"], state["scale"])
        return fg.gemm_fp8_1x128_128x128_bf16_lora(state["a"], state["sa"], state["b"], state["sb"], state["x"], state["la"], state["lb"], state["ids"],
                                                   state["scale"])
    rows = (case["G"], case["cap"]) if case["layout"] == "masked" else _rows(case)
    if op == "dispatch":
        if case["to"] == "fp8":
            a, sa = fg.moe_dispatch_fp8(state["x"], state["row"], rows, A=state["a"], sa=state["sa"])
            return a.view(torch.float8_e4m3fn), sa
        a = fg.moe_dispatch_bf16(state["x"], state["row"], rows, A=state["a"])
        return (a, fg.moe_dispatch_backward(state["da"], state["row"])) if case["grad"] else a
    out = fg.moe_combine(state["y"], state["row"], state["w"])
    if not case["grad"]:
        return out
    return (out, *fg.moe_combine_backward(state["dout"], state["y"], state["row"], state["w"], dY=state["dy"]))


# ---- the definitions in 64 bits ----------------------------------------------------------------------------------

def _nearest_e4m3(v):
    """The e4m3 value next to v (ties to even), for |v| <= 448."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "sort":
        return None
    if op == "route":
        x = s["logits"].double()
        ids = _weights(s["logits"], case["k"], False, 1.0)[0].long()
        lse = torch.logsumexp(x, 1, keepdim=True)
        ok = ids >= 0
        chosen = torch.where(ok, x.gather(1, ids.clamp(min=0)), -math.inf)
        norm = torch.logsumexp(chosen, 1, keepdim=True) if case["renorm"] else lse
        w = case["scale"] * torch.where(ok, torch.exp(chosen - norm), 0.0)
        if not case["grad"]:
            return None, w
        # d w_j / d l_e = w_j ([e = e_j] - p_e), p the softmax that normalises w
        g = (w * torch.where(ok, s["dw"].double(), 0.0))
        p = torch.where(x > -math.inf, torch.exp(x - norm), 0.0)
        if case["renorm"]:
            chosen_at = torch.zeros_like(x).scatter_add_(1, ids.clamp(min=0), ok.double())
            p = p * chosen_at.clamp(max=1)
        d = torch.zeros_like(x).scatter_add_(1, ids.clamp(min=0), g)
        return None, w, d - p * g.sum(1, keepdim=True)
    if op == "lora":
        N, x = case["N"], s["x"].double()
        if case["base"] == "bf16":
            d = x @ s["w"].double().t()
        else:
            a = s["a"].view(torch.float8_e4m3fn).double().view(case["M"], -1, 128) * s["sa"].double().t()[..., None]
            b = s["b"].view(torch.float8_e4m3fn).double().view(N, -1, 128)
            b = b * s["sb"].double()[torch.arange(N, device="cuda") // 128][..., None]
            d = a.reshape(case["M"], -1) @ b.reshape(N, -1).t()
        for g in range(case["G"]):
            at = (s["ids"] == g).nonzero()[:, 0]
            if at.numel():
                d[at] += s["scale"][g].double() * (x[at] @ s["la"][g].double().t()) @ s["lb"][g].double().t()
        return d
    row, H, M = s["row"].long(), case["H"], _rows(case)
    token, choice = (row >= 0).nonzero(as_tuple=True)
    at = row[token, choice]
    if op == "dispatch":
        if case["to"] == "fp8":
            x = s["x"].double().view(case["T"], -1, 128)
            sc = x.abs().amax(2) / 448
            sc = torch.where(sc > 0, sc, 1.0)
            codes = torch.zeros(M, H, dtype=torch.float32, device="cuda")
            codes[at] = _nearest_e4m3((x / sc[..., None]).clamp(-448, 448)).view(case["T"], H).float()[token]
            scales = torch.zeros(M, H // 128, dtype=torch.float64, device="cuda")
            scales[at] = sc[token]
            if case["layout"] == "masked":
                return codes.view(s["a"].shape), scales.view(case["G"], case["cap"], -1).transpose(1, 2).contiguous()
            return codes, scales.t().contiguous()
        a = torch.zeros(M, H, dtype=torch.float64, device="cuda")
        a[at] = s["x"].double()[token]
        if not case["grad"]:
            return a.view(s["a"].shape)
        dx = torch.zeros(case["T"], H, dtype=torch.float64, device="cuda").index_add_(0, token, s["da"].view(M, H)[at].double())
        return a.view(s["a"].shape), dx
    y, w = s["y"].view(M, H)[at].double(), s["w"].double()[token, choice]
    out = torch.zeros(case["T"], H, dtype=torch.float64, device="cuda").index_add_(0, token, y * w[:, None])
    if not case["grad"]:
        return out
    d = s["dout"].double()[token]
    dy = torch.zeros(M, H, dtype=torch.float64, device="cuda")
    dy[at] = d * w[:, None]
    dw = torch.zeros(row.shape, dtype=torch.float64, device="cuda")
    dw[token, choice] = (y * d).sum(1)
    return out, dy.view(s["y"].shape), dw
