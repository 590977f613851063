"""The workloads of the router and of the 8-bit floating point operators.

Four operators: routing to experts, quantisation of activations to e4m3 with a
scale for each 128 of a row, the matrix product of such activations with
weights that have a scale for each block of 128 x 128, and the mixture-of-experts
layer made of them.  With ``own`` false ``run`` computes them in elementary
torch operations; with ``own`` true it calls this package.

Definitions.  quantise, per row and group of 128 columns with largest magnitude
A: scale A / 448 and codes e4m3(448 x / A), rounded to nearest even; a group
with A < 2**-100 is held as zeros with scale 0.  product: out = sum over groups
of (activation scale) (weight scale) (product of the codes), rounded to bf16.
layer: h = silu(gate) up from the quantised x, quantised again, the down
product, and the sum over a token's slots with its routing weights.  router:
choice = score + bias, the best groups by the sum of their two best choices
(one without a bias), then the k best choices, ties to the lowest index;
weights are the scores, divided by their sum if asked, times a factor.
"""

import math

import torch

own = False

F8 = torch.float8_e4m3fn
F8_MAX = 448.0
TINY = 2.0 ** -100
GROUP = 128


def listed():
    return [
        # One token of an interactive decode: only the latency of the call counts.
        dict(name="route_t1", op="route", T=1, E=384, k=8, scoring="softmax", bias=False, n_group=1,
             topk_group=1, renorm=True, scaling=1.0, dtype="float32", masked=False),
        # A decode batch with a balance bias and grouped experts, 16-bit logits
        # (ties are common), a few experts taken out of service.
        dict(name="route_t64_groups", op="route", T=64, E=256, k=8, scoring="sigmoid", bias=True,
             n_group=8, topk_group=4, renorm=True, scaling=2.5, dtype="bfloat16", masked=True),
        # A prefill batch, balance bias over all experts.
        dict(name="route_t8192", op="route", T=8192, E=384, k=8, scoring="sigmoid", bias=True,
             n_group=1, topk_group=1, renorm=True, scaling=2.5, dtype="float32", masked=False),
        # Activations of a decode batch in front of a product.
        dict(name="quantize_t32", op="quantize", T=32, K=7168),
        # Activations of a prefill batch; a width that ends inside a group.
        dict(name="quantize_t8192", op="quantize", T=8191, K=7112),
        # One token through a dense gate_up projection: the weights' bytes.
        dict(name="gemm_m1", op="gemm", M=1, N=4096, K=7168),
        # A decode batch through a projection whose output is no multiple of a block.
        dict(name="gemm_m100_ragged", op="gemm", M=100, N=2112, K=7168),
        # A prefill batch through the dense gate_up projection: the matrix rate.
        dict(name="gemm_m8192", op="gemm", M=8192, N=4096, K=7168),
        # One token of a tensor-parallel slice: eight thin experts, latency.
        dict(name="moe_t1_tp", op="moe", T=1, H=7168, I=256, E_g=384, E_l=384, k=8, first=0),
        # A decode batch on one of eight expert-parallel shares: the weights' bytes.
        dict(name="moe_t64_ep", op="moe", T=64, H=7168, I=2048, E_g=384, E_l=48, k=8, first=96),
        # A mixed batch on a tensor-parallel slice: many experts, few rows each.
        dict(name="moe_t512_tp", op="moe", T=512, H=7168, I=256, E_g=384, E_l=384, k=8, first=0),
        # A prefill batch on one of eight expert-parallel shares: the matrix rate.
        dict(name="moe_t8192_ep", op="moe", T=8192, H=7168, I=2048, E_g=384, E_l=48, k=8, first=0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "quantize", "gemm", "gemm", "moe", "moe"])
    if op == "route":
        n_group = rng.choice([1, 1, 2, 4, 8])
        E = n_group * _log_int(rng, 4 if n_group > 1 else 8, 1024 // n_group)
        topk_group = rng.randint(1, n_group)
        most = min(16, E // n_group * topk_group)
        return dict(op=op, T=_log_int(rng, 1, 16384), E=E, k=rng.randint(1, most),
                    scoring=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.6,
                    n_group=n_group, topk_group=topk_group, renorm=rng.random() < 0.7,
                    scaling=rng.choice([1.0, 2.5]), dtype=rng.choice(["float32", "bfloat16"]),
                    masked=rng.random() < 0.3)
    if op == "quantize":
        return dict(op=op, T=_log_int(rng, 1, 8192), K=_log_int(rng, 128, 8192))
    if op == "gemm":
        return dict(op=op, M=_log_int(rng, 1, 8192), N=_log_int(rng, 64, 8192),
                    K=_log_int(rng, 256, 7168))
    E_g = rng.choice([8, 16, 40, 64, 128, 256, 384])
    E_l = rng.choice([e for e in range(1, E_g + 1) if E_g % e == 0 and e * 8 >= E_g])
    H = 128 * _log_int(rng, 4, 56)
    I = 128 * rng.randint(1, 16)
    while E_l * 3 * H * I > 2.1e9:  # the weights of the largest listed case
        I = max(128, I // 2 // 128 * 128)
    k = rng.randint(1, 8)
    most = min(8192, 8192 * 7168 * 2048 * E_g // (k * E_l * H * I))
    return dict(op=op, T=_log_int(rng, 1, max(1, most)), H=H, I=I, E_g=E_g, E_l=E_l, k=k,
                first=rng.randrange(E_g // E_l) * E_l)


def work(case):
    op = case["op"]
    if op == "route":
        size = 4 if case["dtype"] == "float32" else 2
        return {"bytes": case["T"] * (case["E"] * size + case["k"] * 8) + 4 * case["E"] * case["bias"],
                "flops": case["T"] * case["E"] * 4}
    if op == "quantize":
        groups = -(-case["K"] // GROUP)
        return {"bytes": case["T"] * (2 * case["K"] + groups * (GROUP + 4)),
                "flops": case["T"] * case["K"] * 4}
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        groups = -(-K // GROUP)
        return {"bytes": M * groups * (GROUP + 4) + N * K + 4 * groups * -(-N // GROUP) + 2 * M * N,
                "flops": 2 * M * N * K}
    T, H, I, k = case["T"], case["H"], case["I"], case["k"]
    rows = T * k * case["E_l"] / case["E_g"]
    active = case["E_l"] * (1 - (1 - k / case["E_g"]) ** T)  # expected over uniform routing
    weights = active * 3 * H * I * (1 + 4 / GROUP ** 2)
    return {"bytes": int(weights + 4 * T * H + 8 * T * k), "flops": int(6 * rows * H * I)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _weights(g, E, N, K):
    """Codes e4m3 [E, N, K] and scales fp32 [E, ceil(N/128), ceil(K/128)] of
    normal weights whose rows have unit gain, each block with its own spread."""
    nb, kb = -(-N // GROUP), -(-K // GROUP)
    codes = torch.empty((E, N, K), dtype=F8, device="cuda")
    scales = torch.empty((E, nb, kb), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 28) // (nb * kb * GROUP * GROUP))
    for e in range(0, E, step):
        n = min(step, E - e)
        w = torch.randn((n, nb, GROUP, kb, GROUP), generator=g, device="cuda")
        spread = 0.5 + torch.rand((n, nb, 1, kb, 1), generator=g, device="cuda")
        top = w.abs().amax(dim=(2, 4), keepdim=True)
        codes[e:e + n] = (w * (F8_MAX / top)).to(F8).reshape(n, nb * GROUP, kb * GROUP)[:, :N, :K]
        scales[e:e + n] = (top * spread / (F8_MAX * math.sqrt(K))).reshape(n, nb, kb)
    return codes, scales


def _activations(g, T, K):
    """Unit normal rows, a few channels ten times as large, as activations are."""
    x = torch.randn((T, K), generator=g, device="cuda")
    return (x * torch.where(torch.rand(K, generator=g, device="cuda") < 0.01, 10.0, 1.0)).bfloat16()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    state = {"case": case}
    if op == "route":
        T, E = case["T"], case["E"]
        logits = 1.5 * torch.randn((T, E), generator=g, device="cuda")
        if case["masked"]:
            logits[:, torch.rand(E, generator=g, device="cuda") < 0.05] = -math.inf
        state["logits"] = logits.to(getattr(torch, case["dtype"]))
        state["bias"] = 0.1 * torch.randn(E, generator=g, device="cuda") if case["bias"] else None
        return state
    if op == "quantize":
        state["x"] = _activations(g, case["T"], case["K"])
        return state
    if op == "gemm":
        state["q"], state["s"] = _quantize(_activations(g, case["M"], case["K"]))
        state["wq"], state["ws"] = _weights(g, 1, case["N"], case["K"])
        if own:
            from quantized_moe_amd import chord as C
            state["w"] = C.chord_f8_pack(C.ROLE_PLAIN, state["wq"], state["ws"])
        return state
    T, H, I, E_l = case["T"], case["H"], case["I"], case["E_l"]
    state["x"] = _activations(g, T, H)
    state["w13"] = _weights(g, E_l, 2 * I, H)
    state["w2"] = _weights(g, E_l, H, I)
    scores = torch.randn((T, case["E_g"]), generator=g, device="cuda").softmax(dim=1)
    w, ids = scores.topk(case["k"], dim=1)
    state["ids"] = ids.to(torch.int32)
    state["weights"] = w / w.sum(dim=1, keepdim=True)
    if own:
        from quantized_moe_amd.moe import W8A8MoE
        state["layer"] = W8A8MoE(*state["w13"], *state["w2"])
    return state


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _grouped(x):
    """[T, K] -> fp32 [T, groups, 128], the last group filled up with zeros."""
    T, K = x.shape
    groups = -(-K // GROUP)
    x = torch.nn.functional.pad(x.float(), (0, groups * GROUP - K))
    return x.reshape(T, groups, GROUP)


def _quantize(x):
    v = _grouped(x)
    top = v.abs().amax(dim=2, keepdim=True)
    live = top >= TINY
    # 448 x / A with factors that neither overflow nor round: 0.875 = 448 / 512
    q = (v * 0.875) / torch.where(live, top * 2.0 ** -9, 1.0)
    q = torch.where(live, q, 0.0).to(F8)
    s = torch.where(live, top / F8_MAX, 0.0)
    return q.reshape(x.shape[0], -1), s.squeeze(2)


def _dequantize(q, s):
    T = q.shape[0]
    return (q.float().reshape(T, -1, GROUP) * s.unsqueeze(2)).reshape(T, -1)


def _dequantize_weight(q, s):
    """fp32 [E, N, K] from codes and block scales."""
    E, N, K = q.shape
    wide = s.repeat_interleave(GROUP, dim=1)[:, :N].repeat_interleave(GROUP, dim=2)[:, :, :K]
    return q.float() * wide


def _route(logits, bias, k, scoring, n_group, topk_group, renorm, scaling):
    v = logits.double()  # 64 bits: scores next to each other decide the order
    off = ~(v > -math.inf)
    if bias is not None:
        off = off | ~(bias > -math.inf)
    if scoring == "softmax":
        top = torch.where(off, -math.inf, v).amax(dim=1, keepdim=True)
        e = torch.where(off, 0.0, (v - top).exp())
        score = e / e.sum(dim=1, keepdim=True)
    else:
        score = torch.where(off, 0.0, 1.0 / (1.0 + (-v).exp()))
    choice = score if bias is None else score + bias.double()
    choice = torch.where(off, -math.inf, choice)
    if n_group > 1:
        T, E = v.shape
        best = choice.reshape(T, n_group, -1).sort(dim=2, descending=True).values[:, :, :2]
        if bias is None:
            of_group = best[:, :, 0]
        else:
            of_group = torch.where(best > -math.inf, best, 0.0).sum(dim=2)
            of_group = torch.where(best[:, :, 0] > -math.inf, of_group, -math.inf)
        order = of_group.sort(dim=1, descending=True, stable=True).indices[:, :topk_group]
        keep = torch.zeros_like(of_group, dtype=torch.bool).scatter_(1, order, True)
        choice = torch.where(keep.repeat_interleave(E // n_group, dim=1), choice, -math.inf)
    value, ids = choice.sort(dim=1, descending=True, stable=True)
    found = value[:, :k] > -math.inf
    ids = ids[:, :k]
    w = torch.where(found, score.gather(1, ids), 0.0)
    if renorm:
        w = w / (w.sum(dim=1, keepdim=True) + 1e-20)
    return torch.where(found, ids, -1).to(torch.int32), (w * scaling).float()


def _moe(x, w13, w2, ids, weights, first):
    T, H = x.shape
    k = ids.shape[1]
    E, I = w13[0].shape[0], w2[0].shape[2]
    flat = ids.reshape(-1).long() - first
    flat = torch.where((flat >= 0) & (flat < E), flat, E)
    order = flat.sort(stable=True).indices
    count = torch.bincount(flat, minlength=E + 1)
    start = count.cumsum(0) - count
    rank = torch.empty_like(flat)
    rank[order] = torch.arange(T * k, device=x.device) - start[flat[order]]
    cap = max(1, int(count[:E].max()))
    local = (flat < E).nonzero().squeeze(1)  # the slots that have an expert here
    e, r, t = flat[local], rank[local], local // k
    a = torch.zeros((E, cap, H), dtype=torch.float32, device=x.device)
    a[e, r] = _dequantize(*_quantize(x))[t]
    gu = torch.bmm(a, _dequantize_weight(*w13).transpose(1, 2))
    h = torch.nn.functional.silu(gu[:, :, :I]) * gu[:, :, I:]
    h = _dequantize(*_quantize(h.reshape(E * cap, I))).reshape(E, cap, I)
    y = torch.bmm(h, _dequantize_weight(*w2).transpose(1, 2))
    slots = torch.zeros((T * k, H), dtype=torch.float32, device=x.device)
    slots[local] = y[e, r] * weights.reshape(-1, 1)[local]
    return slots.reshape(T, k, H).sum(dim=1).bfloat16()


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        from quantized_moe_amd import chord as C
        if op == "route":
            scoring = C.SCORE_SOFTMAX if case["scoring"] == "softmax" else C.SCORE_SIGMOID
            ids, w = C.chord_moe_route(state["logits"], case["k"], scoring=scoring, bias=state["bias"],
                                       n_group=case["n_group"], topk_group=case["topk_group"],
                                       renormalize=case["renorm"], scaling=case["scaling"])
            return {"ids": ids, "weights": w}
        if op == "quantize":
            q, s = C.chord_f8_quantize(state["x"])
            return {"q": q, "s": s}
        if op == "gemm":
            return {"out": C.chord_f8_gemm(state["q"], state["s"], state["w"])}
        return {"out": state["layer"].indexed(state["x"], state["ids"], state["weights"],
                                              case["first"], case["E_g"])}
    if op == "route":
        ids, w = _route(state["logits"], state["bias"], case["k"], case["scoring"], case["n_group"],
                        case["topk_group"], case["renorm"], case["scaling"])
        return {"ids": ids, "weights": w}
    if op == "quantize":
        q, s = _quantize(state["x"])
        return {"q": q, "s": s}
    if op == "gemm":
        w = _dequantize_weight(state["wq"], state["ws"])[0]
        a = _dequantize(state["q"], state["s"])[:, :w.shape[1]]
        return {"out": (a @ w.t()).bfloat16()}
    return {"out": _moe(state["x"], state["w13"], state["w2"], state["ids"], state["weights"],
                        case["first"])}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _nearest_e4m3(v):
    """Nearest e4m3 value of each |v| <= 448, ties to even: 3 fraction bits, the
    spacing of the smallest normal (2**-6) below it."""
    _, e = torch.frexp(v)  # |v| in [2**(e - 1), 2**e)
    spacing = torch.tensor([2.0 ** i for i in range(-9, 6)], dtype=torch.float64, device=v.device)
    step = spacing[torch.clamp(e - 1, min=-6) + 6]
    return torch.round(v / step) * step


def _exact_quantize(x):
    """Values of the codes [T, groups * 128] and the scales, in 64 bits."""
    T, K = x.shape
    groups = -(-K // GROUP)
    v = torch.zeros((T, groups * GROUP), dtype=torch.float64, device=x.device)
    v[:, :K] = x
    v = v.view(T, groups, GROUP)
    top = v.abs().max(dim=2).values
    top[top < TINY] = 0
    q = _nearest_e4m3((v * F8_MAX / top.unsqueeze(2)).nan_to_num(0.0, 0.0, 0.0) * (top > 0).unsqueeze(2))
    return q.view(T, -1), top / F8_MAX


def _exact_rows(q, s):
    return (q.view(q.shape[0], -1, GROUP) * s.unsqueeze(2)).view(q.shape[0], -1)


def _exact_weight(q, s):
    N, K = q.shape
    w = q.double()
    n = torch.arange(N, device=q.device) // GROUP
    c = torch.arange(K, device=q.device) // GROUP
    return w * s.double()[n][:, c]


def _exact_route(case, logits, bias):
    import numpy as np
    v = logits.double().cpu().numpy()
    b = None if bias is None else bias.double().cpu().numpy()
    T, E = v.shape
    k, G, keep = case["k"], case["n_group"], case["topk_group"]
    ok = v > -np.inf
    if b is not None:
        ok = ok & (b > -np.inf)
    with np.errstate(all="ignore"):
        if case["scoring"] == "softmax":
            e = np.exp(v - np.where(ok, v, -np.inf).max(axis=1, keepdims=True))
            e = np.where(ok, e, 0.0)
            score = e / e.sum(axis=1, keepdims=True)
        else:
            score = np.where(ok, 1.0 / (1.0 + np.exp(-v)), 0.0)
    choice = np.where(ok, score if b is None else score + b, -np.inf)
    if G > 1:
        per = np.sort(choice.reshape(T, G, E // G), axis=2)[:, :, ::-1]
        total = per[:, :, 0].copy()
        if b is not None and E // G > 1:
            total += np.where(np.isfinite(per[:, :, 1]), per[:, :, 1], 0.0)
        chosen = np.argsort(-total, axis=1, kind="stable")[:, :keep]
        mask = np.zeros((T, G), bool)
        np.put_along_axis(mask, chosen, True, axis=1)
        choice = np.where(np.repeat(mask, E // G, axis=1), choice, -np.inf)
    ids = np.argsort(-choice, axis=1, kind="stable")[:, :k]
    there = np.isfinite(np.take_along_axis(choice, ids, axis=1))
    w = np.where(there, np.take_along_axis(score, ids, axis=1), 0.0)
    if case["renorm"]:
        w = w / (w.sum(axis=1, keepdims=True) + 1e-20)
    return {"ids": torch.from_numpy(np.where(there, ids, -1).astype(np.int32)),
            "weights": torch.from_numpy(w * case["scaling"])}


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(case, state["logits"], state["bias"])
    if op == "quantize":
        q, s = _exact_quantize(state["x"])
        return {"q": q, "s": s}
    if op == "gemm":
        a = _exact_rows(state["q"].double(), state["s"].double())[:, :case["K"]]
        return {"out": a @ _exact_weight(state["wq"][0], state["ws"][0]).t()}
    x = _exact_rows(*_exact_quantize(state["x"]))
    I = case["I"]
    out = torch.zeros_like(x)
    ids = state["ids"].cpu()
    for e in range(case["E_l"]):
        t, j = (ids == e + case["first"]).nonzero(as_tuple=True)
        if not len(t):
            continue
        t, j = t.cuda(), j.cuda()
        gu = x[t] @ _exact_weight(state["w13"][0][e], state["w13"][1][e]).t()
        h = gu[:, :I] / (1 + (-gu[:, :I]).exp()) * gu[:, I:]
        y = _exact_rows(*_exact_quantize(h)) @ _exact_weight(state["w2"][0][e], state["w2"][1][e]).t()
        out.index_add_(0, t, y * state["weights"][t, j].double().unsqueeze(1))
    return {"out": out}
