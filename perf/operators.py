"""The INT8 expert path's operators, as they are timed and compared: cases, inputs,
plain forms and 64-bit values.

Four operators, in the order one mixture-of-experts layer runs them:

  topk     routing to experts: scores from the router's logits (softmax or sigmoid), an
           optional balance bias that steers the choice only, optional groups, top-k
           with ties to the lowest index, weights renormalised and scaled.
  quant    BF16 rows to INT8 with one scale per row (token), optionally written
           straight into the experts' row order.
  gemm     Y = BF16(sA[m] sW[n] sum_k a[m,k] w[n,k]) with INT8 codes a, w and one
           scale for each token and each output channel.
  experts  the same product with each expert's rows against its own weights.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# --- cases ------------------------------------------------------------------------

def _topk(T, E, k, score="softmax", bias=False, groups=1, top_groups=1, renorm=True, scale=1.0,
          dtype="fp32"):
    return dict(op="topk", T=T, E=E, k=k, score=score, bias=bias, groups=groups,
                top_groups=top_groups, renorm=renorm, scale=scale, dtype=dtype)


def _quant(rows, K, k=0):
    return dict(op="quant", rows=rows, K=K, k=k)  # k = 0: rows stay in place


def _gemm(M, N, K):
    return dict(op="gemm", M=M, N=N, K=K)


def _experts(T, k, E, N, K, zipf=0.0):
    return dict(op="experts", T=T, k=k, E=E, N=N, K=K, zipf=zipf)


def listed():
    cases = [
        # one decoding batch through a router of 8 experts: latency is all that counts
        dict(_topk(16, 8, 2, dtype="bf16"), name="topk_decode"),
        # an odd number of tokens and of experts, probabilities kept as they are
        dict(_topk(3001, 60, 4, renorm=False), name="topk_odd"),
        # a prefill batch through 256 experts in 8 groups, chosen with a balance bias
        dict(_topk(8192, 256, 8, score="sigmoid", bias=True, groups=8, top_groups=4, scale=2.5),
             name="topk_groups"),
        # one decoded token's activations ahead of a projection
        dict(_quant(1, 4096), name="quant_token"),
        # prefill activations ahead of the FFN down projection
        dict(_quant(4096, 14336), name="quant_prefill"),
        # a layer's tokens written twice each, into the experts' row order
        dict(_quant(8192, 4096, k=2), name="quant_routed"),
        # FFN down projection: one token, a ragged batch, a prefill
        dict(_gemm(1, 5376, 14336), name="gemm_token"),
        dict(_gemm(333, 5376, 14336), name="gemm_batch"),
        dict(_gemm(4096, 5376, 14336), name="gemm_prefill"),
        # decoding through 8 large experts: few rows, every weight of the experts hit is read
        dict(_experts(16, 2, 8, 14336, 4096), name="experts_decode"),
        # many small experts, some 64 ragged rows each
        dict(_experts(512, 8, 64, 2816, 2048, zipf=0.5), name="experts_small"),
        # prefill through 8 large experts with skewed popularity
        dict(_experts(8192, 1, 8, 14336, 4096, zipf=1.1), name="experts_prefill"),
    ]
    return cases


MAX_MACS = 4096 * 5376 * 14336     # the largest listed product
MAX_WEIGHTS = 8 * 14336 * 4096     # and the largest listed set of weights


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["topk", "quant", "gemm", "experts"])
    if op == "topk":
        groups = rng.choice([1, 1, 2, 4, 8])
        per = _log_int(rng, max(2, 8 // groups), 256 // groups)
        E = groups * per
        top_groups = rng.randint(1, groups)
        k = rng.randint(1, min(8, top_groups * per))
        return _topk(_log_int(rng, 1, 8192), E, k, score=rng.choice(["softmax", "sigmoid"]),
                     bias=rng.random() < 0.5, groups=groups, top_groups=top_groups,
                     renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]),
                     dtype=rng.choice(["fp32", "bf16"]))
    if op == "quant":
        K = 16 * _log_int(rng, 8, 896)
        k = rng.choice([0, 0, 1, 2, 4])
        top = 4096 * 14336 // (K * max(1, k))
        return _quant(_log_int(rng, 1, min(8192, top)), K, k)
    if op == "gemm":
        K = 16 * _log_int(rng, 8, 896)
        N = _log_int(rng, 64, 14336)
        return _gemm(_log_int(rng, 1, max(1, min(8192, MAX_MACS // (N * K)))), N, K)
    E = _log_int(rng, 2, 128)
    K = 16 * _log_int(rng, 16, 256)
    N = 8 * _log_int(rng, 16, max(16, min(1792, MAX_WEIGHTS // (E * K * 8))))
    k = rng.randint(1, min(8, E))
    T = _log_int(rng, 1, max(1, min(8192, MAX_MACS // (N * K * k))))
    return _experts(T, k, E, N, K, zipf=rng.choice([0.0, 0.5, 1.1]))


# --- inputs -----------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _int8_rows(x):
    """[rows, K] float -> INT8 codes and one scale per row (input preparation only)."""
    s = x.abs().amax(dim=1, keepdim=True).clamp_min(1e-20) / 127
    return torch.round(x / s).to(torch.int8), s[:, 0].contiguous()


def _pick_experts(g, T, k, E, zipf):
    """[T, k] distinct experts per token, popularity (e + 1)^-zipf (Gumbel top-k)."""
    pop = -zipf * torch.log(torch.arange(1, E + 1, device=DEV, dtype=torch.float32))
    u = torch.rand(T, E, generator=g, device=DEV).clamp_min(1e-20)
    return torch.topk(pop - torch.log(-torch.log(u)), k, dim=1).indices


def _dest_of(ids, E):
    """Row of each (token, slot) pair in the stable expert order, and the E+1 offsets."""
    flat = ids.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    dest = torch.empty_like(order)
    dest[order] = torch.arange(order.numel(), device=DEV)
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = torch.cumsum(counts, 0)
    return dest.to(torch.int32), offsets.to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    op = case["op"]
    if op == "topk":
        T, E = case["T"], case["E"]
        logits = 1.5 * _randn(g, T, E) + 0.5 * _randn(g, 1, E)
        st["logits"] = logits.to(torch.bfloat16) if case["dtype"] == "bf16" else logits
        st["bias_t"] = 0.1 * _randn(g, E) if case["bias"] else None
    elif op == "quant":
        rows, K, k = case["rows"], case["K"], case["k"]
        # tokens of different size, a few channels larger than the rest
        chan = torch.exp(0.5 * _randn(g, 1, K))
        st["x"] = (torch.exp(0.5 * _randn(g, rows, 1)) * chan * _randn(g, rows, K)).to(torch.bfloat16)
        if k:
            st["dest"], _ = _dest_of(_pick_experts(g, rows, k, max(8, k), 0.5), max(8, k))
    elif op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        st["A"], st["sA"] = _int8_rows(_randn(g, M, K))
        st["W"], st["sW"] = _int8_rows(0.02 * _randn(g, N, K))
    else:
        T, k, E, N, K = case["T"], case["k"], case["E"], case["N"], case["K"]
        _, st["offsets"] = _dest_of(_pick_experts(g, T, k, E, case["zipf"]), E)
        st["host_offsets"] = st["offsets"].tolist()
        st["A"], st["sA"] = _int8_rows(_randn(g, T * k, K))
        W = torch.empty(E, N, K, dtype=torch.int8, device=DEV)
        sW = torch.empty(E, N, dtype=torch.float32, device=DEV)
        for e in range(E):
            W[e], sW[e] = _int8_rows(0.02 * _randn(g, N, K))
        st["W"], st["sW"] = W, sW
    if own:
        import block_scaled_precision_nvfp4_b200 as nv
        nv.load_library()
        st["nv"] = nv
    return st


# --- one pass ---------------------------------------------------------------------

def _plain_topk(st):
    # in 64 bits: the choice between experts is a comparison of values next to each other
    T, E, k, G = st["T"], st["E"], st["k"], st["groups"]
    x = st["logits"].double()
    if st["score"] == "softmax":
        p = torch.exp(x - x.amax(dim=1, keepdim=True))
        score = p / p.sum(dim=1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-x))
    choice = score if st["bias_t"] is None else score + st["bias_t"].double()
    if G > 1:
        per = E // G
        member = torch.sort(choice.view(T, G, per), dim=2, descending=True).values
        gscore = member[:, :, :2].sum(dim=2)
        kept = torch.sort(gscore, dim=1, descending=True, stable=True).indices[:, :st["top_groups"]]
        inside = torch.zeros(T, G, dtype=torch.bool, device=x.device)
        inside.scatter_(1, kept, True)
        choice = choice.masked_fill(~inside.repeat_interleave(per, dim=1), -math.inf)
    ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.gather(score, 1, ids)
    if st["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return ids.to(torch.int32), (w * st["scale"]).float()


def _plain_quant(st):
    x = st["x"].float()
    amax = x.abs().amax(dim=1, keepdim=True)
    live = amax > 0
    codes = torch.round(127.0 * x / torch.where(live, amax, torch.ones_like(amax))).to(torch.int8)
    scales = torch.where(live, amax / 127.0, torch.ones_like(amax))[:, 0]
    k = st["k"]
    if not k:
        return codes, scales
    dest = st["dest"].long()
    gc = torch.empty(codes.shape[0] * k, codes.shape[1], dtype=torch.int8, device=codes.device)
    gs = torch.empty(codes.shape[0] * k, dtype=torch.float32, device=codes.device)
    gc[dest] = codes.repeat_interleave(k, dim=0)
    gs[dest] = scales.repeat_interleave(k, dim=0)
    return gc, gs


def _plain_gemm(A, sA, W, sW):
    acc = A.float() @ W.float().t()
    return (acc * sA[:, None] * sW[None, :]).to(torch.bfloat16)


def run(st):
    op = st["op"]
    if own:
        nv = st["nv"]
        if op == "topk":
            return nv.moe_topk(st["logits"], st["k"], score=st["score"], bias=st["bias_t"],
                               groups=st["groups"], top_groups=st["top_groups"],
                               renormalize=st["renorm"], scale=st["scale"])
        if op == "quant":
            if st["k"]:
                return nv.int8_quantize_bf16_routed(st["x"], st["dest"], st["k"])
            return nv.int8_quantize_bf16(st["x"])
        if op == "gemm":
            return nv.gemm_int8_w8a8(st["A"], st["sA"], st["W"], st["sW"])
        return nv.gemm_int8_w8a8_grouped(st["A"], st["sA"], st["W"], st["sW"], st["offsets"])
    if op == "topk":
        return _plain_topk(st)
    if op == "quant":
        return _plain_quant(st)
    if op == "gemm":
        return _plain_gemm(st["A"], st["sA"], st["W"], st["sW"])
    off = st["host_offsets"]
    Y = torch.empty(st["A"].shape[0], st["N"], dtype=torch.bfloat16, device=st["A"].device)
    for e in range(st["E"]):
        r0, r1 = off[e], off[e + 1]
        if r1 > r0:
            Y[r0:r1] = _plain_gemm(st["A"][r0:r1], st["sA"][r0:r1], st["W"][e], st["sW"][e])
    return Y


def work(case):
    op = case["op"]
    if op == "topk":
        T, E, k = case["T"], case["E"], case["k"]
        size = 2 if case["dtype"] == "bf16" else 4
        # a score and a comparison for each expert of each token
        return {"bytes": T * E * size + (4 * E if case["bias"] else 0) + T * k * 8,
                "flops": 8 * T * E}
    if op == "quant":
        rows, K, k = case["rows"], case["K"], case["k"]
        out = rows * max(1, k)
        return {"bytes": rows * K * 2 + out * (K + 4) + (4 * out if k else 0), "flops": 3 * rows * K}
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K + N * K + 4 * (M + N) + 2 * M * N, "flops": 2 * M * N * K}
    T, k, E, N, K = case["T"], case["k"], case["E"], case["N"], case["K"]
    P = T * k
    # the experts that rows are expected to reach (exact for even popularity)
    pop = np.arange(1, E + 1, dtype=np.float64) ** -case["zipf"]
    pop /= pop.sum()
    hit = float(np.sum(1.0 - (1.0 - np.minimum(1.0, k * pop)) ** T))
    hit = min(hit, E, P)
    return {"bytes": int(P * K + hit * N * (K + 4) + 4 * (P + E + 1) + 2 * P * N),
            "flops": 2 * P * N * K}


# --- 64-bit values ----------------------------------------------------------------

def _exact_topk(st):
    T, E, k, G = st["T"], st["E"], st["k"], st["groups"]
    x = st["logits"].double().cpu().numpy()
    if st["score"] == "softmax":
        z = x - np.log(np.sum(np.exp(x), axis=1, keepdims=True))
        score = np.exp(z)
    else:
        score = 0.5 * (1.0 + np.tanh(0.5 * x))
    b = np.zeros(E) if st["bias_t"] is None else st["bias_t"].double().cpu().numpy()
    choice = score + b
    if st["bias_t"] is None:
        # equal logits have equal scores; nothing else ties
        choice = np.where(np.isfinite(x), choice, -np.inf)
    ids = np.empty((T, k), dtype=np.int32)
    index = np.arange(E)
    per = E // G
    for t in range(T):
        c = choice[t]
        allowed = index
        if G > 1:
            gs = [math.fsum(sorted(c[g * per:(g + 1) * per], reverse=True)[:2]) for g in range(G)]
            kept = sorted(range(G), key=lambda g: (-gs[g], g))[:st["top_groups"]]
            allowed = np.concatenate([index[g * per:(g + 1) * per] for g in sorted(kept)])
        order = np.lexsort((allowed, -c[allowed]))[:k]
        ids[t] = allowed[order]
    w = np.take_along_axis(score, ids.astype(np.int64), axis=1)
    if st["renorm"]:
        w = w / w.sum(axis=1, keepdims=True)
    return (torch.from_numpy(ids).to(DEV), torch.from_numpy(w * st["scale"]).to(DEV))


def _exact_quant(st):
    x = st["x"].double()
    top = torch.maximum(x.amax(dim=1), -x.amin(dim=1))
    safe = torch.where(top == 0, torch.ones_like(top), top)
    codes = torch.round(x * 127.0 / safe[:, None])
    scales = torch.where(top == 0, torch.ones_like(top), top / 127.0)
    k = st["k"]
    if k:
        src = torch.empty(st["rows"] * k, dtype=torch.int64, device=x.device)
        src[st["dest"].long()] = torch.arange(st["rows"] * k, device=x.device) // k
        codes, scales = codes[src], scales[src]
    return codes.to(torch.int8), scales


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "topk":
        return _exact_topk(st)
    if op == "quant":
        return _exact_quant(st)
    if op == "gemm":
        return torch.einsum("mk,nk->mn", st["A"].double() * st["sA"].double()[:, None],
                            st["W"].double() * st["sW"].double()[:, None])
    off = st["host_offsets"]
    parts = [torch.einsum("mk,nk->mn", st["A"][off[e]:off[e + 1]].double(), st["W"][e].double())
             * (st["sA"][off[e]:off[e + 1]].double()[:, None] * st["sW"][e].double()[None, :])
             for e in range(st["E"])]
    return torch.cat(parts, dim=0)
