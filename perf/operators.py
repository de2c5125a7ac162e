"""The router, the token permutation and the expert products' gradient, measured.

A layer of routed experts needs more than its forward products.  The router
turns logits into the top-k ids and weights that the sort and the combine take,
and a layer that is trained through (its 4-bit experts frozen, the router and
everything before them learning) runs the permutation, the activation and the
products backwards.  This file lists calls of those operators, makes their
inputs, and computes them either in plain torch (own False) or through the
library (own True).

    gate          logits [T, E] -> the k chosen experts of each token and their weights
    gate_grad     gradient of the weights -> gradient of the logits
    dispatch      token rows -> band order (one copy per chosen expert)
    dispatch_grad band-ordered gradient -> token order, summed over a token's copies
    combine_grad  gradient of the combined output -> gradients of the band rows and of the weights
    product_grad  gradient of a 4-bit grouped product's output -> gradient of its input, with
                  "act" through the SiLU-gated activation whose output that input was
    gated         the SiLU-gated activation of kept gate/up sums
"""

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "bf16": 2}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a batch of 64: sigmoid scores, chosen with a load-balancing bias
        dict(name="gate_decode_64", op="gate", T=64, E=256, k=6, dtype="f32", score="sigmoid", bias=True,
             renorm=True, scale=2.5, masked=0, pad=0),
        # a prefill batch padded to its length, logits straight from a bf16 router, 32 experts out of service
        dict(name="gate_prefill_4096", op="gate", T=4096, E=256, k=6, dtype="bf16", score="softmax", bias=False,
             renorm=True, scale=1.0, masked=32, pad=61),
        # the router's share of a training step
        dict(name="gate_grad_4096", op="gate_grad", T=4096, E=256, k=6, dtype="f32", score="softmax", bias=False,
             renorm=False, scale=1.0, masked=0, pad=0),
        # rows laid out per expert, as an exchange between expert-parallel ranks sends them
        dict(name="dispatch_prefill_4096", op="dispatch", T=4096, k=6, E=256, N=4096, dtype="bf16"),
        # the way back in training, an odd batch
        dict(name="dispatch_grad_1237", op="dispatch_grad", T=1237, k=8, E=64, N=2560, dtype="f32", out="bf16"),
        # gradient of the weighted sum over a token's experts
        dict(name="combine_grad_4096", op="combine_grad", T=4096, k=6, E=256, N=4096, dtype="bf16", out="bf16"),
        # gradient through the fused gate/up weights, 4,096 tokens
        dict(name="w13_grad_4096", op="product_grad", T=4096, k=6, E=256, N=4096, K=4096, fmt="mxfp4",
             routing="uniform", out="bf16", act=False),
        # gradient through the down weights and the activation that feeds them, 4,096 tokens
        dict(name="w2_act_grad_4096", op="product_grad", T=4096, k=6, E=256, N=4096, K=2048, fmt="mxfp4",
             routing="uniform", out="bf16", act=True),
        # a short step (64 tokens): bound by the weights it streams
        dict(name="w13_grad_64", op="product_grad", T=64, k=6, E=256, N=4096, K=4096, fmt="mxfp4",
             routing="uniform", out="f32", act=False),
        # skewed routing, NVFP4 weights with calibrated (general E4M3) block scales
        dict(name="w2_grad_nvfp4_256", op="product_grad", T=256, k=6, E=256, N=4096, K=2048, fmt="nvfp4",
             routing="zipf", out="f32", act=False),
        # the activation of a training step's kept gate/up sums
        dict(name="gated_24576", op="gated", M=24576, N=4096, dtype="bf16", out="bf16"),
        # the same for a handful of rows of an odd width, f32
        dict(name="gated_100", op="gated", M=100, N=1416, dtype="f32", out="f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gate", "gate", "gate_grad", "dispatch", "dispatch_grad", "combine_grad", "product_grad",
                     "product_grad", "product_grad", "product_grad", "gated"])
    dt = lambda: rng.choice(["f32", "bf16"])  # noqa: E731
    if op in ("gate", "gate_grad"):
        E = _log_int(rng, 8, 1024)
        T = _log_int(rng, 1, 16384)
        score = rng.choice(["softmax", "sigmoid"])
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(E, 16)), dtype=dt(), score=score,
                    bias=op == "gate" and rng.random() < 0.5, renorm=rng.random() < 0.5,
                    scale=rng.choice([1.0, 2.5]), masked=rng.choice([0, 0, E // 8]),
                    pad=rng.choice([0, 0, T // 10]))
    if op in ("dispatch", "dispatch_grad", "combine_grad"):
        E = _log_int(rng, 8, 256)
        c = dict(op=op, T=_log_int(rng, 1, 4096), k=rng.randint(1, 8), E=E, N=4 * _log_int(rng, 64, 1024), dtype=dt())
        if op != "dispatch":
            c["out"] = dt()
        return c
    if op == "product_grad":
        return dict(op=op, T=_log_int(rng, 1, 4096), k=rng.randint(1, 6), E=_log_int(rng, 8, 256),
                    N=64 * _log_int(rng, 2, 64), K=128 * _log_int(rng, 1, 32),
                    fmt=rng.choice(["mxfp4", "mxfp4", "nvfp4", "nvfp4_pow2"]), routing=rng.choice(["uniform", "zipf"]),
                    out=dt(), act=rng.random() < 0.4)
    return dict(op=op, M=_log_int(rng, 1, 24576), N=8 * _log_int(rng, 16, 512), dtype=dt(), out=dt())


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _normal(g, shape, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dtype)


def _routes(g, T, k, E, routing="uniform"):
    """Top-k routing without replacement and the band order it gives."""
    keys = torch.rand((T, E), generator=g, device=DEV).clamp_(1e-7, 1 - 1e-7)
    if routing == "zipf":
        keys = -torch.log(-torch.log(keys)) - 1.1 * torch.log(torch.arange(1, E + 1, device=DEV, dtype=torch.float32))
    ids = torch.sort(keys, dim=1, descending=True, stable=True).indices[:, :k].contiguous()
    flat = ids.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    pair_row = torch.empty(T * k, dtype=torch.int32, device=DEV)
    pair_row[order] = torch.arange(T * k, dtype=torch.int32, device=DEV)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.cumsum(torch.bincount(flat, minlength=E), 0).int()
    return dict(topk_ids=ids.int(), sorted_token=(order // k).int(), pair_row=pair_row, offsets=offsets)


def _pack(fmt, codes, scales, tensor_scale):
    """The library's packed weights: 1 KiB chunks of 16 columns x 128 K, then the scale words, then (NVFP4) the
    tensor scales and a word per 16 columns that says whether some block scale is not a power of two."""
    E, N, K2 = codes.shape
    NT, KC = N // 16, K2 // 64
    parts = [codes.view(E, NT, 16, KC, 4, 16).permute(0, 1, 3, 4, 2, 5).reshape(-1)]
    per = 4 if fmt == "mxfp4" else 2
    groups = -(-KC // per)
    s = scales.view(E, NT, 16, KC, 4, -1)
    s = torch.nn.functional.pad(s, (0, 0, 0, 0, 0, groups * per - KC))
    s = s.view(E, NT, 16, groups, per, 4, -1).permute(0, 1, 3, 5, 2, 4, 6)
    parts.append(s.reshape(-1))
    if fmt != "mxfp4":
        exps = torch.frexp(scales.view(torch.float8_e4m3fn).float())
        odd = (exps.mantissa != 0.5).view(E, NT, -1).any(-1).int()
        for t in (tensor_scale, odd.reshape(-1)):
            b = t.contiguous().view(torch.uint8)
            parts.append(torch.nn.functional.pad(b, (0, -b.numel() % 256)))
    return torch.cat(parts)


def _gate_inputs(case, g):
    T, E = case["T"], case["E"]
    logits = _normal(g, (T, E), std=1.5)
    if case["masked"]:
        logits[:, torch.randperm(E, generator=g, device=DEV)[: case["masked"]]] = -math.inf
    if case["pad"]:
        logits[T - case["pad"]:] = -math.inf
    logits = logits.to(DTYPES[case["dtype"]])
    bias = _normal(g, (E,), std=0.1) if case["bias"] else None
    return dict(logits=logits, bias=bias)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op = case["op"]
    st = dict(case)
    if op in ("gate", "gate_grad"):
        st.update(_gate_inputs(case, g))
        if op == "gate_grad":
            st["ids"] = _choose(st)[0]
            st["dweights"] = _normal(g, (case["T"], case["k"]))
    elif op in ("dispatch", "dispatch_grad", "combine_grad"):
        T, k, E, N = (case[n] for n in ("T", "k", "E", "N"))
        st.update(_routes(g, T, k, E) if k <= E else {})
        dt = DTYPES[case["dtype"]]
        if op == "dispatch":
            st["x"] = _normal(g, (T, N), dt)
        elif op == "dispatch_grad":
            st["dxs"] = _normal(g, (T * k, N), dt)
        else:
            st["dout"] = _normal(g, (T, N), dt)
            st["y"] = _normal(g, (T * k, N), dt)
            st["weights"] = torch.softmax(_normal(g, (T, k)), dim=1)
    elif op == "product_grad":
        T, k, E, N, K = (case[n] for n in ("T", "k", "E", "N", "K"))
        M = T * k
        st.update(_routes(g, T, k, E, case["routing"]))
        st["M"] = M
        st["band_rows"] = int((st["offsets"][1:] - st["offsets"][:-1]).max())
        st["codes"] = torch.randint(0, 256, (E, N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
        st["tensor_scale"] = None
        if case["fmt"] == "mxfp4":
            st["scales"] = torch.randint(119, 125, (E, N, K // 32), generator=g, device=DEV, dtype=torch.uint8)
        else:
            # normal E4M3 bytes of exponents -3 .. 4, every mantissa or (the lossless cast) none
            st["scales"] = torch.randint(32, 96, (E, N, K // 16), generator=g, device=DEV, dtype=torch.uint8)
            if case["fmt"] == "nvfp4_pow2":
                st["scales"] &= 0x78
            st["tensor_scale"] = torch.exp2(torch.randint(-9, -5, (E,), generator=g, device=DEV).float()) * (
                1 + torch.rand(E, generator=g, device=DEV) / 8)
        st["packed"] = _pack(case["fmt"], st["codes"], st["scales"], st["tensor_scale"])
        m = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=DEV)
        values = torch.cat((m, -m))
        b = torch.arange(256, device=DEV)
        st["code_pairs"] = torch.stack((values[b & 15], values[b >> 4]), 1)   # a byte's two weights
        st["dy"] = _normal(g, (M, N), torch.bfloat16, std=0.1)
        st["preact"] = _normal(g, (M, 2 * K), torch.bfloat16) if case["act"] else None
    else:
        st["y"] = _normal(g, (case["M"], case["N"]), DTYPES[case["dtype"]], std=2.0)
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _choose(st):
    """Chosen ids (descending, ties to the lowest index, -1 where nothing is left) and the scores' logits."""
    x = st["logits"].double()
    if st["bias"] is None:
        key = x
    else:
        p = torch.softmax(x, 1).nan_to_num(0.0) if st["score"] == "softmax" else torch.sigmoid(x)
        key = torch.where(x > -math.inf, p + st["bias"].double(), -math.inf)
    top = torch.sort(key, dim=1, descending=True, stable=True)
    ids = top.indices[:, : st["k"]]
    return torch.where(top.values[:, : st["k"]] > -math.inf, ids, -1).int(), x


def _shares(st, ids, x):
    """Scores of the chosen experts, as f32 weights before the scale, and the logits they come from."""
    live = ids >= 0
    chosen = torch.gather(x, 1, ids.clamp_min(0).long()).float()
    chosen = torch.where(live, chosen, -math.inf)
    if st["score"] == "softmax":
        top = (chosen if st["renorm"] else x.float()).amax(1, keepdim=True).clamp_min(-3.0e38)
        s = torch.exp(chosen - top)
        total = s.sum(1, keepdim=True) if st["renorm"] else torch.exp(x.float() - top).sum(1, keepdim=True)
    else:
        s = torch.sigmoid(chosen)
        total = s.sum(1, keepdim=True) if st["renorm"] else torch.ones_like(s[:, :1])
    return torch.where(live, s / torch.where(total > 0, total, 1.0), 0.0), chosen


def _gate(st):
    ids, x = _choose(st)
    return ids, _shares(st, ids, x)[0] * st["scale"]


def _gate_grad(st):
    ids = st["ids"]
    x = st["logits"].double()
    w, chosen = _shares(st, ids, x)
    live = (ids >= 0).float()
    gs = st["dweights"] * st["scale"] * live
    common = (gs * w).sum(1, keepdim=True) if st["score"] == "softmax" or st["renorm"] else 0.0
    d = w * (gs - common)
    if st["score"] == "sigmoid":
        d = d * torch.sigmoid(-chosen)
    full = torch.zeros(st["logits"].shape, device=DEV)
    if st["score"] == "softmax" and not st["renorm"]:
        xf = x.float()
        e = torch.exp(xf - xf.amax(1, keepdim=True).clamp_min(-3.0e38))
        total = e.sum(1, keepdim=True)
        full = -common * e / torch.where(total > 0, total, 1.0)
        d = w * gs
    full.scatter_add_(1, ids.clamp_min(0).long(), d * live)
    return full.to(st["logits"].dtype)


def _dispatch(st):
    return st["x"][st["sorted_token"].long()]


def _dispatch_grad(st):
    rows = st["dxs"][st["pair_row"].long()].float()
    return rows.view(st["T"], st["k"], st["N"]).sum(1).to(DTYPES[st["out"]])


def _combine_grad(st):
    dout = st["dout"].float()
    tok = st["sorted_token"].long()
    pair = torch.empty_like(tok)
    rows = torch.arange(tok.numel(), device=DEV)
    pair[st["pair_row"].long()] = rows
    dy = dout[tok] * st["weights"].reshape(-1)[pair][:, None]
    dw = (dout[tok] * st["y"].float()).sum(1)
    return dy.to(DTYPES[st["out"]]), dw[st["pair_row"].long()].view(st["T"], st["k"])


def _weights(st):
    E, N, K = st["E"], st["N"], st["K"]
    w = st["code_pairs"][st["codes"].int()].view(E, N, -1, 32 if st["fmt"] == "mxfp4" else 16)
    if st["fmt"] == "mxfp4":
        s = (st["scales"].int() << 23).view(torch.float32)
    else:
        s = st["scales"].view(torch.float8_e4m3fn).float()
    return w.mul_(s[..., None]).view(E, N, K)


def _silu_grads(pre, dh):
    g, u = pre.float().chunk(2, dim=1)
    s = torch.sigmoid(g)
    return torch.cat((dh * u * s * (1 + g * (1 - s)), dh * g * s), 1)


def _product_grad(st):
    E, M, N, R = st["E"], st["M"], st["N"], st["band_rows"]
    off = st["offsets"].long()
    slot = torch.arange(R, device=DEV)
    rows = off[:-1, None] + slot
    rows = torch.where(rows < off[1:, None], rows, M)
    dy = torch.cat((st["dy"].float(), torch.zeros((1, N), device=DEV)))
    d = torch.bmm(dy[rows], _weights(st))
    if st["tensor_scale"] is not None:
        d = d * st["tensor_scale"][:, None, None]
    r = torch.arange(M, device=DEV)
    e = torch.searchsorted(off, r, right=True) - 1
    d = d.view(E * R, -1)[e * R + r - off[e]]
    if st["act"]:
        d = _silu_grads(st["preact"], d)
    return d.to(DTYPES[st["out"]])


def _gated(st):
    g, u = st["y"].float().chunk(2, dim=1)
    return (g * torch.sigmoid(g) * u).to(DTYPES[st["out"]])


PLAIN = dict(gate=_gate, gate_grad=_gate_grad, dispatch=_dispatch, dispatch_grad=_dispatch_grad,
             combine_grad=_combine_grad, product_grad=_product_grad, gated=_gated)


def _library(st):
    import moe_grouped_gemm_route_amd as moe
    op = st["op"]
    dt = {"f32": moe.F32, "bf16": moe.BF16}
    if op in ("gate", "gate_grad"):
        score = moe.GATE_SOFTMAX if st["score"] == "softmax" else moe.GATE_SIGMOID
        if op == "gate":
            return moe.topk_gate(st["logits"], st["k"], score=score, bias=st["bias"], renormalize=st["renorm"],
                                 scale=st["scale"])
        return moe.topk_gate_bwd(st["logits"], st["ids"], st["dweights"], score=score, renormalize=st["renorm"],
                                 scale=st["scale"])
    if op == "dispatch":
        return moe.moe_dispatch(st["x"], st["pair_row"], st["k"])
    if op == "dispatch_grad":
        return moe.moe_dispatch_bwd(st["dxs"], st["pair_row"], st["k"], out_dtype=dt[st["out"]])
    if op == "combine_grad":
        return moe.moe_combine_bwd(st["dout"], st["y"], st["weights"], st["pair_row"], out_dtype=dt[st["out"]])
    if op == "product_grad":
        return moe.moe_gmm_dgrad(st["packed"], moe.MXFP4 if st["fmt"] == "mxfp4" else moe.NVFP4, st["E"], st["N"],
                                 st["K"], st["dy"], st["offsets"], st["M"], out_dtype=dt[st["out"]],
                                 act=moe.ACT_SILU_MUL if st["act"] else moe.ACT_NONE, preact=st["preact"])
    return moe.silu_mul(st["y"], out_dtype=dt[st["out"]])


def run(state):
    return _library(state) if own else PLAIN[state["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its values in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    s = SIZES.get(case.get("dtype"), 2)
    o = SIZES.get(case.get("out"), 2)
    if op == "gate":
        return {"bytes": case["T"] * (case["E"] * s + case["k"] * 8), "flops": 4 * case["T"] * case["E"]}
    if op == "gate_grad":
        return {"bytes": case["T"] * (2 * case["E"] * s + case["k"] * 8), "flops": 6 * case["T"] * case["E"]}
    if op == "gated":
        return {"bytes": case["M"] * case["N"] * (s + o / 2), "flops": 5 * case["M"] * case["N"] / 2}
    T, k, N = case["T"], case["k"], case["N"]
    M = T * k
    if op == "dispatch":
        return {"bytes": (T + M) * N * s + 4 * M, "flops": 0}
    if op == "dispatch_grad":
        return {"bytes": M * N * s + T * N * o + 4 * M, "flops": M * N}
    if op == "combine_grad":
        return {"bytes": (T + M) * N * s + M * N * o + 12 * M, "flops": 3 * M * N}
    K = case["K"]
    # experts that some row reaches, as uniform or Zipf routing leaves them
    E = case["E"]
    p = [(e + 1) ** -1.1 for e in range(E)] if case["routing"] == "zipf" else [1.0] * E
    total = sum(p)
    used = sum(1 - (1 - min(1.0, k * q / total)) ** T for q in p)
    weights = used * N * K * (0.5 + (1 / 32 if case["fmt"] == "mxfp4" else 1 / 16))
    out = M * K * ((2 * o + 4) if case["act"] else o)
    return {"bytes": weights + 2 * M * N + out, "flops": 2 * M * N * K}


def _exact_gate(st):
    x = st["logits"].double().cpu()
    k = st["k"]
    neg = x == -math.inf
    if st["score"] == "softmax":
        top = x.max(1, keepdim=True).values
        e = torch.where(neg, 0.0, (x - torch.where(top == -math.inf, 0.0, top)).exp())
        z = e.sum(1, keepdim=True)
        p = e / torch.where(z == 0, 1.0, z)
    else:
        p = torch.where(neg, 0.0, 1 / (1 + (-x).exp()))
    return x, neg, p, k


def _exact_weights(st, ids, p):
    w = torch.where(ids < 0, 0.0, p.gather(1, ids.clamp(min=0)))
    if st["renorm"]:
        z = w.sum(1, keepdim=True)
        w = w / torch.where(z == 0, 1.0, z)
    return w


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "gate":
        x, neg, p, k = _exact_gate(st)
        b = 0.0 if st["bias"] is None else st["bias"].double().cpu()
        key = torch.where(neg, -math.inf, x if st["bias"] is None else p + b)
        order = torch.argsort(-key, dim=1, stable=True)[:, :k]
        ids = torch.where(key.gather(1, order) == -math.inf, -1, order)
        return ids.int(), _exact_weights(st, ids, p) * st["scale"]
    if op == "gate_grad":
        x, neg, p, k = _exact_gate(st)
        ids = st["ids"].long().cpu()
        slot = torch.nn.functional.one_hot(ids.clamp(min=0), case["E"]).double() * (ids >= 0)[..., None]
        gs = (slot * (st["dweights"].double().cpu() * st["scale"])[..., None]).sum(1)   # by expert
        on = slot.sum(1)
        if st["renorm"]:                       # w = p / sum of the chosen p
            z = (on * p).sum(1, keepdim=True)
            z = torch.where(z == 0, 1.0, z)
            gs = on * (gs - (gs * p).sum(1, keepdim=True) / z) / z
        d = p * (gs - (gs * p).sum(1, keepdim=True)) if st["score"] == "softmax" else gs * p * (1 - p)
        return d
    if op == "dispatch":
        return st["x"].double()[st["sorted_token"].long()]
    if op == "dispatch_grad":
        out = torch.zeros((case["T"], case["N"]), dtype=torch.float64, device=DEV)
        return out.index_add_(0, torch.arange(case["T"] * case["k"], device=DEV) // case["k"],
                              st["dxs"].double()[st["pair_row"].long()])
    if op == "combine_grad":
        T, k = case["T"], case["k"]
        rows = st["pair_row"].long().view(T, k)
        dy = torch.empty((T * k, case["N"]), dtype=torch.float64, device=DEV)
        dw = torch.empty((T, k), dtype=torch.float64, device=DEV)
        dout = st["dout"].double()
        for j in range(k):
            dy[rows[:, j]] = st["weights"].double()[:, j, None] * dout
            dw[:, j] = (dout * st["y"][rows[:, j]].double()).sum(1)
        return dy, dw
    if op == "gated":
        h = case["N"] // 2
        g = st["y"][:, :h].double()
        return g / (1 + (-g).exp()) * st["y"][:, h:].double()
    E, N, K, M = case["E"], case["N"], case["K"], st["M"]
    off = st["offsets"].tolist()
    d = torch.zeros((M, K), dtype=torch.float64, device=DEV)
    block = 32 if case["fmt"] == "mxfp4" else 16
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        c = torch.stack((st["codes"][e] & 15, st["codes"][e] >> 4), -1).view(N, K).long()
        exponent, fraction = (c >> 1) & 3, (c & 1).double()
        v = torch.where(exponent == 0, fraction / 2, (1 + fraction / 2) * (1 << exponent.clamp(min=1)).double() / 2)
        v = torch.where(c >= 8, -v, v)
        sb = st["scales"][e].long()
        if case["fmt"] == "mxfp4":
            s = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=DEV), (sb - 127).double())
        else:
            s = (1 + (sb & 7).double() / 8) * torch.pow(torch.tensor(2.0, dtype=torch.float64, device=DEV),
                                                        (((sb >> 3) & 15) - 7).double())
        w = (v.view(N, K // block, block) * s[..., None]).view(N, K)
        d[a:b] = st["dy"][a:b].double() @ w
        if st["tensor_scale"] is not None:
            d[a:b] *= st["tensor_scale"][e].double()
    if case["act"]:
        g, u = st["preact"][:, :K].double(), st["preact"][:, K:].double()
        q = 1 / (1 + (-g).exp())
        d = torch.cat((d * u * (q + g * q * (1 - q)), d * g * q), 1)
    return d
