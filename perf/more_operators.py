"""The operators of expert layers: what is timed, and their plain forms.

  route      scores of E experts (softmax or sigmoid of the logits), the k best of a token by
             score + bias, within its best groups where there are groups; their weights
  route_bwd  the gradient of the logits from that of the weights
  gather     (token, expert) pairs sorted by expert, and the tokens' rows in that order,
             quantized in groups of 128 along the row (and along the rows of an expert)
  fwd        y[r] = x[r] W_e^T for the rows r of each expert e, FP8 operands with a scale for
             each 1x128 of x and 128x128 of W
  dgrad      dx[r] = dy[r] W_e
  wgrad      dW_e = sum over the rows r of e of dy[r]^T x[r], operands quantized 128x1
  combine    out[t] = residual[t] + sum over t's experts of weight * y[row of the pair]
  comb_bwd   its gradients: of y, quantized in expert order, and of the weights

Rows in expert order: expert e has the rows start[e] .. start[e] + count[e], in token order, and
start[e + 1] is the next multiple of `align` after them.  src[r] is the pair t k + j in row r, or
-1; pos[t, j] is the pair's row.  An 8-bit tensor is E4M3 codes with one scale s = amax / 448 per
group.  It is returned as its codes (float8) and its groups' maxima 448 s, which are BF16 numbers.
"""
import math

import torch

own = False

TINY = 1e-20    # added to the sum that the weights are divided by


def listed():
    return [
        # one new token of a rollout
        {"name": "route_one_token", "op": "route", "T": 1, "E": 64, "k": 8, "score": "softmax", "bias": False,
         "groups": 1, "top": 1, "rank": 1, "renorm": True, "scale": 1.0, "dtype": "fp32"},
        # a training batch of 16384 tokens on many experts, limited to 4 of 8 groups, with a balancing bias
        {"name": "route_groups_train", "op": "route", "T": 16384, "E": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "top": 4, "rank": 2, "renorm": True, "scale": 2.5, "dtype": "fp32"},
        # the backward of a softmax router on BF16 logits, whose gradient reaches every expert
        {"name": "route_bwd_train", "op": "route_bwd", "T": 16384, "E": 128, "k": 8, "score": "softmax",
         "renorm": False, "scale": 1.0, "dtype": "bf16"},
        # an odd number of sequences in a rollout, from the router's choice to the first product's operand
        {"name": "gather_rollout", "op": "gather", "T": 61, "K": 3584, "E": 64, "k": 6, "align": 1, "dual": False},
        # the training forward of a 4096-wide layer at 8192 tokens, both quantized layouts
        {"name": "gather_train", "op": "gather", "T": 8192, "K": 4096, "E": 64, "k": 8, "align": 128, "dual": True},
        # one new token through the gate_up weights of its 8 experts
        {"name": "fwd_one_token", "op": "fwd", "T": 1, "E": 64, "k": 8, "N": 2816, "K": 4096, "align": 1},
        # an odd number of sequences on the down weights
        {"name": "fwd_rollout", "op": "fwd", "T": 61, "E": 64, "k": 6, "N": 3584, "K": 1408, "align": 1},
        # training: the gate_up product at 8192 tokens
        {"name": "fwd_train", "op": "fwd", "T": 8192, "E": 64, "k": 8, "N": 2816, "K": 4096, "align": 128},
        # the input gradient of a small ragged batch, a reduction of 22 blocks
        {"name": "dgrad_ragged", "op": "dgrad", "T": 1111, "E": 32, "k": 4, "N": 2816, "K": 3584, "align": 128},
        # training: the weight gradient of the down product
        {"name": "wgrad_train", "op": "wgrad", "T": 8192, "E": 64, "k": 8, "N": 4096, "K": 1408, "align": 128},
        # a prefill's experts added to its residual stream
        {"name": "combine_ragged", "op": "combine", "T": 777, "E": 64, "k": 6, "N": 3584, "align": 1, "residual": True},
        # training: the backward of the weighted sum, both layouts of the gradient
        {"name": "comb_bwd_train", "op": "comb_bwd", "T": 8192, "E": 64, "k": 8, "N": 4096, "align": 128, "dual": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_bwd", "gather", "fwd", "fwd", "dgrad", "wgrad", "combine", "comb_bwd"])
    if op in ("route", "route_bwd"):
        E = rng.choice([8, 16, 32, 60, 64, 96, 128, 160, 256, 320, 384, 512])
        T = _log(rng, 1, min(16384, 16384 * 256 // E))
        c = {"op": op, "T": T, "E": E, "k": rng.randint(1, min(12, E)), "score": rng.choice(["softmax", "sigmoid"]),
             "renorm": rng.random() < 0.6, "scale": rng.choice([1.0, 2.5, 1.826]), "dtype": rng.choice(["fp32", "bf16"])}
        if op == "route_bwd":
            return c
        groups = rng.choice([1] + [g for g in (1, 2, 4, 8) if E % g == 0])
        rank = rng.choice([1, 2])
        need = -(-c["k"] * groups // E)     # groups that hold k experts
        top = rng.randint(need, groups)
        return {**c, "bias": rng.random() < 0.5, "groups": groups, "top": top, "rank": rank if groups > 1 else 1}
    E = rng.choice([4, 8, 16, 24, 32, 60, 64, 96, 128])
    k = rng.randint(1, min(8, E))
    if op in ("gather", "combine", "comb_bwd"):
        C = 128 * _log(rng, 1, 56)
        T = _log(rng, 1, min(16384, 65536 * 4096 // (C * k)))
        align = 128 if op == "comb_bwd" else rng.choice([1, 128])
        if align == 128:        # the padding's rows count too
            T = max(1, min(T, (65536 * 4096 // C - 128 * min(E, T * k)) // k))
        c = {"op": op, "T": T, "E": E, "k": k, "align": align}
        if op == "combine":
            return {**c, "N": C, "residual": rng.random() < 0.5}
        return {**c, ("K" if op == "gather" else "N"): C, "dual": align == 128 and rng.random() < 0.6}
    N, K = 128 * _log(rng, 2, 44), 128 * _log(rng, 2, 32)
    E = min(E, max(k, 64 * 2816 * 4096 // (N * K)))
    if op == "fwd" and rng.random() < 0.5:
        return {"op": op, "T": _log(rng, 1, 256), "E": E, "k": k, "N": N, "K": K, "align": 1}
    T = _log(rng, 64, min(8192, 65536 * 2816 * 4096 // (N * K * k)))
    return {"op": op, "T": T, "E": E, "k": k, "N": N, "K": K, "align": 128}


# ------------------------------------------------------------------ inputs

def _normal(gen, shape, std, outliers=0):
    x = torch.randn(shape, generator=gen, device="cuda") * std
    if outliers:
        x[:, torch.randperm(shape[1], generator=gen, device="cuda")[:outliers]] *= 30.0
    return x.to(torch.bfloat16)


def _index(gen, T, E, k):
    """k different experts a token, some experts more often than others: int32 [T,k]."""
    likes = 0.4 * torch.randn(E, generator=gen, device="cuda")
    return torch.topk(likes + torch.randn((T, E), generator=gen, device="cuda"), k, dim=1).indices.to(torch.int32)


def _rows(index, E, align):
    """The pairs in expert order, as the module's first lines say."""
    T, k = index.shape
    P, dev = T * k, index.device
    R = (P + min(E, P) * (align - 1)) // align * align
    e = index.reshape(-1).long()
    count = torch.zeros(E, dtype=torch.int64, device=dev).scatter_add_(0, e, torch.ones_like(e))
    start = torch.zeros(E + 1, dtype=torch.int64, device=dev)
    start[1:] = torch.cumsum((count + align - 1) // align * align, 0)
    order = torch.sort(e, stable=True).indices
    first = torch.cumsum(count, 0) - count
    row = start[e[order]] + torch.arange(P, device=dev) - first[e[order]]
    src = torch.full((R,), -1, dtype=torch.int32, device=dev)
    src[row] = order.to(torch.int32)
    pos = torch.empty(P, dtype=torch.int32, device=dev)
    pos[order] = row.to(torch.int32)
    return {"pos": pos.view(T, k), "src": src, "start": start.to(torch.int32), "count": count.to(torch.int32), "align": align}


def _take(x, rows, weight=None):
    """Row src[r] / k of x for each row r, times the pair's weight; zeros where src[r] is -1."""
    k = rows["pos"].shape[1]
    src = rows["src"].long()
    v = x[src.clamp(min=0) // k]
    if weight is not None:
        v = (v.float() * weight.reshape(-1)[src.clamp(min=0)][:, None]).to(torch.bfloat16)
    return torch.where((src >= 0)[:, None], v, torch.zeros_like(v[:1]))


def _grid(f, amax):
    s = amax / torch.full_like(amax, 448.0)      # by a tensor: a true division on the GPU
    return (f / torch.where(s > 0, s, 1.0)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), s


def _quant_rows(x):
    """Groups of 128 along the rows of BF16 x [M,C]: codes float8 [M,C], scales fp32 [C/128,M]."""
    M, C = x.shape
    f = x.float().view(M, C // 128, 128)
    q, s = _grid(f, f.abs().amax(2, keepdim=True))
    return q.view(M, C), s[:, :, 0].t().contiguous()


def _quant_cols(x):
    return _quant_rows(x.t().contiguous())


def _quant_weights(w, E):
    """FP32 [E N, K] -> codes uint8 [E N, K], scales [E N / 128, K / 128], codes transposed [K, E N]."""
    EN, K = w.shape
    f = w.view(EN // 128, 128, K // 128, 128)
    q, s = _grid(f, f.abs().amax((1, 3), keepdim=True))
    q = q.view(EN, K).view(torch.uint8)
    return q, s.view(EN // 128, K // 128).contiguous(), q.t().contiguous()


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    op, T, E, k = case["op"], case["T"], case["E"], case["k"]
    st = dict(case)
    if op in ("route", "route_bwd"):
        kind = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
        st["logits"] = (1.5 * torch.randn((T, E), generator=gen, device="cuda")).to(kind)
        if op == "route":
            # a balancing bias of the size that it reaches in training; None where there is none
            st["bias_v"] = 0.05 * torch.randn(E, generator=gen, device="cuda") if case["bias"] else None
        else:
            st["index"] = torch.topk(st["logits"].float(), k, dim=1).indices.to(torch.int32)
            st["dweight"] = 1e-2 * torch.randn((T, k), generator=gen, device="cuda")
        return st
    index = _index(gen, T, E, k)
    if op == "gather":
        st["index"] = index
        st["x"] = _normal(gen, (T, case["K"]), 1.0, max(1, case["K"] // 1000))
        return st
    rows = st["rows"] = _rows(index, E, case["align"])
    N = case["N"]
    if op in ("combine", "comb_bwd"):
        st["y"] = _normal(gen, (rows["src"].numel(), N), 0.7, max(1, N // 1000))
        st["weight"] = torch.softmax(torch.randn((T, k), generator=gen, device="cuda"), 1)
        if op == "comb_bwd":
            st["dout"] = _normal(gen, (T, N), 1e-3)
        else:
            st["res"] = _normal(gen, (T, N), 1.0, max(1, N // 1000)) if case["residual"] else None
        return st
    K, R = case["K"], rows["src"].numel()
    if op != "wgrad":
        w = 0.02 * torch.randn((E * N, K), generator=gen, device="cuda")
        q, st["sw"], qT = _quant_weights(w.to(torch.bfloat16).float(), E)
        st["qw"] = q if op == "fwd" else qT
        # outputs of rows that hold no token's row of any expert stay as they are
        st["out"] = torch.zeros((R, N if op == "fwd" else K), dtype=torch.bfloat16, device="cuda")
    if op != "dgrad":
        x = _take(_normal(gen, (T, K), 1.0, max(1, K // 1000)), rows)
        q, st["sx"] = _quant_rows(x) if op == "fwd" else _quant_cols(x)
        st["qx"] = q.view(torch.uint8)
    if op != "fwd":
        dy = _take(_normal(gen, (T, N), 1e-3), rows)
        q, st["sdy"] = _quant_rows(dy) if op == "dgrad" else _quant_cols(dy)
        st["qdy"] = q.view(torch.uint8)
    return st


# ------------------------------------------------------------------ plain forms

def _best(v, n):
    """Indices of the n largest of each row, the lowest index first among equals."""
    return torch.sort(v, dim=1, descending=True, stable=True).indices[:, :n]


def _scores(z, score):
    return torch.softmax(z, 1) if score == "softmax" else torch.sigmoid(z)


def _plain_route(st):
    T, E, G = st["T"], st["E"], st["groups"]
    z = st["logits"].double()        # two scores next to each other are told apart
    s = _scores(z, st["score"])
    v = z if st["bias_v"] is None and st["rank"] == 1 else s
    if st["bias_v"] is not None:
        v = s + st["bias_v"].double()
    if G > 1:
        g = torch.sort(v.view(T, G, E // G), dim=2, descending=True).values[:, :, :st["rank"]].sum(2)
        keep = torch.zeros((T, G), dtype=torch.bool, device=z.device).scatter_(1, _best(g, st["top"]), True)
        v = torch.where(keep.repeat_interleave(E // G, 1), v, -math.inf)
    index = _best(v, st["k"])
    w = s.gather(1, index).float()
    if st["renorm"]:
        w = w / (w.sum(1, keepdim=True) + TINY)
    return {"weight": w * st["scale"], "index": index.to(torch.int32)}


def _plain_route_bwd(st):
    s = _scores(st["logits"].float(), st["score"])
    index = st["index"].long()
    p, g = s.gather(1, index), st["dweight"] * st["scale"]
    if st["renorm"]:
        total = p.sum(1, keepdim=True) + TINY
        g = (g - (g * p).sum(1, keepdim=True) / total) / total
    ds = torch.zeros_like(s).scatter_(1, index, g)
    if st["score"] == "sigmoid":
        d = ds * s * (1.0 - s)
    else:
        inner = torch.zeros_like(g[:, :1]) if st["renorm"] else (g * p).sum(1, keepdim=True)
        d = s * (ds - inner)
    return {"dlogits": d.to(st["logits"].dtype)}


def _maxima(q, s):
    return q, (s * 448.0).to(torch.bfloat16)


def _quantized(v, dual):
    out = {"rows": _maxima(*_quant_rows(v))}
    if dual:
        out["cols"] = _maxima(*_quant_cols(v))
    return out


def _plain_gather(st):
    rows = _rows(st["index"], st["E"], st["align"])
    out = {n: rows[n] for n in ("pos", "src", "start", "count")}
    return {**out, **_quantized(_take(st["x"], rows), st["dual"])}


def _values(q, s):
    """FP32 values of codes [M,C] with scales [C/128,M]."""
    M, C = q.shape
    return (q.view(torch.float8_e4m3fn).float().view(M, C // 128, 128) * s.t()[:, :, None]).view(M, C)


def _slots(rows):
    """The experts that have rows, and for each the same number of row numbers, with which of them are its own."""
    used = rows["count"].nonzero()[:, 0]
    count, start = rows["count"][used].long(), rows["start"][used].long()
    c = torch.arange(int(count.max()), device=used.device)
    mine = c < count[:, None]
    return used, torch.where(mine, start[:, None] + c, 0), mine


def _plain_product(st):
    E, N, K = st["E"], st["N"], st["K"]
    used, row, mine = _slots(st["rows"])
    sw = st["sw"].view(E, N // 128, 1, K // 128, 1)[used]
    if st["op"] == "fwd":
        a = _values(st["qx"], st["sx"])
        w = st["qw"].view(torch.float8_e4m3fn).view(E, N // 128, 128, K // 128, 128)[used].float() * sw
        w = w.view(-1, N, K).transpose(1, 2)
    else:
        a = _values(st["qdy"], st["sdy"])
        w = st["qw"].view(torch.float8_e4m3fn).view(K, E, N).permute(1, 2, 0)[used].float()
        w = (w.reshape(-1, N // 128, 128, K // 128, 128) * sw).view(-1, N, K)
    out = torch.zeros_like(st["out"])
    out[row[mine]] = torch.bmm(a[row], w)[mine].to(torch.bfloat16)
    return {"y" if st["op"] == "fwd" else "dx": out}


def _plain_wgrad(st):
    used, row, mine = _slots(st["rows"])
    x = _values(st["qx"], st["sx"]).t()[row] * mine[:, :, None]
    dy = _values(st["qdy"], st["sdy"]).t()[row]
    dw = torch.zeros((st["E"], st["N"], st["K"]), dtype=torch.bfloat16, device=x.device)
    dw[used] = torch.bmm(dy.transpose(1, 2), x).to(torch.bfloat16)
    return {"dw": dw}


def _plain_combine(st):
    v = (st["y"][st["rows"]["pos"].long()].float() * st["weight"][:, :, None]).sum(1)
    if st["res"] is not None:
        v = v + st["res"].float()
    return {"out": v.to(torch.bfloat16)}


def _plain_comb_bwd(st):
    rows, dout = st["rows"], st["dout"]
    dweight = (st["y"][rows["pos"].long()].float() * dout.float()[:, None, :]).sum(2)
    return {"dweight": dweight, **_quantized(_take(dout, rows, st["weight"]), st["dual"])}


# ------------------------------------------------------------------ one pass

def _codes(q, s):
    return _maxima(q.view(torch.float8_e4m3fn), s)


def run(state):
    st, op = state, state["op"]
    if not own:
        return {"route": _plain_route, "route_bwd": _plain_route_bwd, "gather": _plain_gather, "fwd": _plain_product,
                "dgrad": _plain_product, "wgrad": _plain_wgrad, "combine": _plain_combine, "comb_bwd": _plain_comb_bwd}[op](st)
    import block_scaled_fp8_x1_gb300.ops as fp8
    if op == "route":
        r = fp8.route_topk(st["logits"], st["k"], score=st["score"], bias=st["bias_v"], n_groups=st["groups"],
                           top_groups=st["top"], group_rank=st["rank"], renormalize=st["renorm"], scale=st["scale"])
        return {"weight": r.weight, "index": r.index}
    if op == "route_bwd":
        return {"dlogits": fp8.route_topk_bwd(st["dweight"], st["logits"], st["index"], score=st["score"],
                                              renormalize=st["renorm"], scale=st["scale"])}
    if op == "gather":
        rows = fp8.expert_rows(st["index"], st["E"], align=st["align"])
        q, s, qT, sT = fp8.expert_gather_quant(st["x"], rows, dual=st["dual"])
        out = {"pos": rows.pos, "src": rows.src, "start": rows.start, "count": rows.count, "rows": _codes(q, s)}
        if st["dual"]:
            out["cols"] = _codes(qT, sT)
        return out
    rows = fp8.ExpertRows(**st["rows"])
    if op == "fwd":
        return {"y": fp8.gemm_experts_fwd(st["qx"], st["sx"], st["qw"], st["sw"], rows, out=st["out"])}
    if op == "dgrad":
        return {"dx": fp8.gemm_experts_dgrad(st["qdy"], st["sdy"], st["qw"], st["sw"], rows, out=st["out"])}
    if op == "wgrad":
        return {"dw": fp8.gemm_experts_wgrad(st["qdy"], st["sdy"], st["qx"], st["sx"], rows)}
    if op == "combine":
        return {"out": fp8.expert_combine(st["y"], rows, st["weight"], residual=st["res"])}
    q, s, qT, sT, dweight = fp8.expert_combine_bwd(st["dout"], st["y"], rows, st["weight"], dual=st["dual"])
    out = {"dweight": dweight, "rows": _codes(q, s)}
    if st["dual"]:
        out["cols"] = _codes(qT, sT)
    return out


def work(case):
    op, T, E, k = case["op"], case["T"], case["E"], case["k"]
    P = T * k
    if op in ("route", "route_bwd"):
        size = 4 if case["dtype"] == "fp32" else 2
        once = T * E * size + 8 * P
        return {"bytes": once + T * E * size if op == "route_bwd" else once + 4 * E * case["bias"], "flops": 8 * T * E}
    code = 1.0 + 4.0 / 128.0
    if op == "gather":
        C = case["K"]
        return {"bytes": 2 * T * C + P * C * code * (1 + case["dual"]) + 12 * P, "flops": 4 * P * C}
    N = case["N"]
    if op == "combine":
        return {"bytes": 2 * P * N + 2 * T * N * (1 + case["residual"]) + 8 * P, "flops": 2 * P * N}
    if op == "comb_bwd":
        return {"bytes": 2 * P * N + 2 * T * N + P * N * code * (1 + case["dual"]) + 12 * P, "flops": 8 * P * N}
    K = case["K"]
    w = min(E, P) * N * K
    if op == "wgrad":
        return {"bytes": P * (N + K) * code + 2 * E * N * K, "flops": 2 * P * N * K}
    a, b = (K, N) if op == "fwd" else (N, K)
    return {"bytes": P * a * code + 2 * P * b + w * (1.0 + 4.0 / 16384.0), "flops": 2 * P * N * K}


# ------------------------------------------------------------------ 64 bits

def _exact_route(st):
    T, E, G = st["T"], st["E"], st["groups"]
    parts = []
    for lo in range(0, T, 512):
        z = st["logits"][lo:lo + 512].double()
        if st["score"] == "softmax":
            e = torch.exp(z - z.max(1, keepdim=True).values)
            s = e / e.sum(1, keepdim=True)
        else:
            s = 1.0 / (1.0 + torch.exp(-z))
        rank_by = s if st["rank"] == 2 else z
        if st["bias_v"] is not None:
            rank_by = s + st["bias_v"].double()[None]

        def place(v):       # how many come before each, equal ones by their index
            n = torch.arange(v.shape[1], device=v.device)
            before = (v[:, None, :] > v[:, :, None]) | ((v[:, None, :] == v[:, :, None]) & (n[None, None, :] < n[None, :, None]))
            return before.sum(2)

        if G > 1:
            blocks = rank_by.reshape(-1, G, E // G)
            top = blocks.max(2).values
            if st["rank"] == 2:
                order = place(blocks.reshape(-1, E // G)).reshape(blocks.shape)
                top = top + torch.where(order == 1, blocks, 0.0).sum(2)
            allowed = place(top) < st["top"]
            rank_by = torch.where(allowed[:, :, None], blocks, -math.inf).reshape(-1, E)
        at = place(rank_by)
        index = torch.stack([(at == j).to(torch.int64).argmax(1) for j in range(st["k"])], 1)
        w = torch.stack([torch.where(at == j, s, 0.0).sum(1) for j in range(st["k"])], 1)
        if st["renorm"]:
            w = w / (w.sum(1)[:, None] + TINY)
        parts.append((w * st["scale"], index))
    return {"weight": torch.cat([p[0] for p in parts]), "index": torch.cat([p[1] for p in parts])}


def _exact_route_bwd(st):
    z = st["logits"].double().requires_grad_()
    with torch.enable_grad():
        if st["score"] == "softmax":
            e = torch.exp(z - z.detach().max(1, keepdim=True).values)
            s = e / e.sum(1, keepdim=True)
        else:
            s = 1.0 / (1.0 + torch.exp(-z))
        w = torch.take_along_dim(s, st["index"].long(), 1)
        if st["renorm"]:
            w = w / (w.sum(1, keepdim=True) + TINY)
        loss = (w * st["scale"] * st["dweight"].double()).sum()
    return {"dlogits": torch.autograd.grad(loss, z)[0]}


def _grid64(x):
    """E4M3 codes and group maxima of groups of 128 along the rows of the BF16 numbers x."""
    r, c = x.shape
    blocks = x.double().reshape(r, c // 128, 128)
    top = blocks.abs().max(-1).values
    unit = top / 448.0
    unit[unit == 0] = 1.0
    m = blocks / unit.unsqueeze(-1)
    # spacing of E4M3 at |m|: 2^(e - 3), e at least -6; round() goes to even
    e = torch.frexp(m.abs().clamp(min=2.0 ** -6)).exponent.double() - 1.0
    step = torch.exp2(e - 3.0)
    codes = (torch.round(m / step) * step).clamp(-448.0, 448.0)
    return codes.reshape(r, c).float(), top.T.contiguous()


def _both64(v, dual):
    """The layouts of BF16 v [R,C] (C the columns), a slice of columns at a time."""
    out = {}
    rows = [_grid64(v[lo:lo + 8192]) for lo in range(0, v.shape[0], 8192)]
    out["rows"] = [torch.cat([a for a, _ in rows], 0), torch.cat([b for _, b in rows], 1)]
    if dual:
        cols = [_grid64(v[:, lo:lo + 512].T.contiguous()) for lo in range(0, v.shape[1], 512)]
        out["cols"] = [torch.cat([a for a, _ in cols], 0), torch.cat([b for _, b in cols], 1)]
    return out


def _layout64(index, E, align):
    """Rows in expert order by counting, on the host."""
    T, k = index.shape
    e = index.cpu().reshape(-1).tolist()
    of = [[] for _ in range(E)]
    for p, x in enumerate(e):
        of[x].append(p)
    start = [0]
    for x in of:
        start.append(start[-1] + -(-len(x) // align) * align)
    R = (T * k + min(E, T * k) * (align - 1)) // align * align
    src, pos = [-1] * R, [0] * (T * k)
    for x, s in zip(of, start):
        src[s:s + len(x)] = x
        for i, p in enumerate(x):
            pos[p] = s + i
    t = lambda v: torch.tensor(v, dtype=torch.int64, device=index.device)  # noqa: E731
    return t(pos).view(T, k), t(src), t(start), t([len(x) for x in of])


def _scattered(x, src, k, factor=None):
    v = torch.zeros((src.numel(), x.shape[1]), dtype=torch.bfloat16, device=x.device)
    r = (src >= 0).nonzero()[:, 0]
    p = src[r].long()
    v[r] = x[p // k] if factor is None else (x[p // k].double() * factor.double().reshape(-1)[p][:, None]).to(torch.bfloat16)
    return v


def _saved64(q, s):
    """Values of codes [M,C] with scales [C/128,M]."""
    return q.view(torch.float8_e4m3fn).double() * s.double().T.repeat_interleave(128, dim=1)


def _exact_product(st):
    E, N, K = st["E"], st["N"], st["K"]
    first, n = st["rows"]["start"].tolist(), st["rows"]["count"].tolist()
    if st["op"] == "wgrad":
        dw = torch.zeros((E, N, K), dtype=torch.float32, device="cuda")
        for e in range(E):
            if n[e]:
                a, b = first[e], first[e + 1]
                dy = _saved64(st["qdy"][:, a:b].contiguous(), st["sdy"][a // 128:b // 128])
                x = _saved64(st["qx"][:, a:b].contiguous(), st["sx"][a // 128:b // 128])
                dw[e] = dy @ x.T
        return {"dw": dw}
    out = torch.zeros(st["out"].shape, dtype=torch.float32, device="cuda")
    for e in range(E):
        if n[e]:
            a, b = first[e], first[e] + n[e]
            sw = st["sw"][e * (N // 128):(e + 1) * (N // 128)].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
            if st["op"] == "fwd":
                w = st["qw"][e * N:(e + 1) * N].view(torch.float8_e4m3fn).double() * sw
                out[a:b] = _saved64(st["qx"][a:b], st["sx"][:, a:b]) @ w.T
            else:
                w = st["qw"][:, e * N:(e + 1) * N].contiguous().view(torch.float8_e4m3fn).double().T * sw
                out[a:b] = _saved64(st["qdy"][a:b], st["sdy"][:, a:b]) @ w
    return {"y" if st["op"] == "fwd" else "dx": out}


def _exact_rows_of(st):
    """(sum over a token's pairs, or None; the pairs' dot products, or None), a slice of tokens at a time."""
    pos, y = st["rows"]["pos"].long(), st["y"]
    sums, dots = [], []
    for lo in range(0, st["T"], 512):
        v = y[pos[lo:lo + 512]].double()
        if st["op"] == "combine":
            a = torch.einsum("tkn,tk->tn", v, st["weight"][lo:lo + 512].double())
            sums.append(a if st["res"] is None else a + st["res"][lo:lo + 512].double())
        else:
            dots.append(torch.einsum("tkn,tn->tk", v, st["dout"][lo:lo + 512].double()))
    return torch.cat(sums) if sums else None, torch.cat(dots) if dots else None


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(st)
    if op == "route_bwd":
        return _exact_route_bwd(st)
    if op == "gather":
        pos, src, start, count = _layout64(st["index"], case["E"], case["align"])
        out = {"pos": pos, "src": src, "start": start, "count": count}
        return {**out, **_both64(_scattered(st["x"], src, case["k"]), case["dual"])}
    if op in ("fwd", "dgrad", "wgrad"):
        return _exact_product(st)
    sums, dots = _exact_rows_of(st)
    if op == "combine":
        return {"out": sums}
    return {"dweight": dots, **_both64(_scattered(st["dout"], st["rows"]["src"], case["k"], st["weight"]), case["dual"])}
