"""The dense half of the layer, measured: a gated feed-forward block and 4-bit integer weights.

Beside its routed experts a layer has a gated block that every token passes
(the shared expert), trained in bf16 and often served with 4-bit integer
weights that carry a scale per group along K.  Routed experts come in that
format too; for a handful of tokens they are multiplied without a sort.  This
file lists calls of those operators, makes their inputs, and computes them
either in plain torch (own False) or through the library (own True).

    w4        rows times 4-bit integer weights, group scales, optional zero points:
              dense, per chosen expert of a token, or those summed with the router's weights;
              with "act" the SiLU-gated product of the two column halves
    gate_up   bf16 gate and up projections and the SiLU-gated product, with "keep" also the sums
    gate_up_grad   gradient of that block: of its input and of its weights
"""

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "bf16": 2, None: 0}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # a dense projection at one token: the smallest call of a decode step
        dict(name="w4_dense_1", op="w4", E=0, T=1, k=0, N=4096, K=4096, G=128, scale="bf16", zeros=False,
             weighted=False, act=False, pad=0, out="bf16"),
        # the shared expert's gate and up weights for a batch of 16, zero points
        dict(name="w4_gate_up_16", op="w4", E=0, T=16, k=0, N=4096, K=4096, G=64, scale="bf16", zeros=True,
             weighted=False, act=True, pad=0, out="bf16"),
        # one token through the gate and up weights of its six experts
        dict(name="w4_experts_1", op="w4", E=256, T=1, k=6, N=4096, K=4096, G=32, scale="bf16", zeros=False,
             weighted=False, act=True, pad=0, out="bf16"),
        # the down weights of a batch of 8, summed with the router's weights; one token is padding
        dict(name="w4_down_8", op="w4", E=64, T=8, k=6, N=4096, K=2048, G=32, scale="f32", zeros=True,
             weighted=True, act=False, pad=1, out="f32"),
        # an output head over a vocabulary, five rows
        dict(name="w4_head_5", op="w4", E=0, T=5, k=0, N=131072, K=4096, G=128, scale="bf16", zeros=False,
             weighted=False, act=False, pad=0, out="f32"),
        # one token through the block's bf16 gate and up weights
        dict(name="gate_up_1", op="gate_up", M=1, N=4096, K=4096, keep=None, out="bf16"),
        # an odd batch through a block of odd widths
        dict(name="gate_up_237", op="gate_up", M=237, N=2832, K=1416, keep=None, out="f32"),
        # a training step's forward pass, sums kept for the gradient
        dict(name="gate_up_4096", op="gate_up", M=4096, N=4096, K=4096, keep="bf16", out="bf16"),
        # a long prompt's prefill
        dict(name="gate_up_16384", op="gate_up", M=16384, N=4096, K=4096, keep=None, out="bf16"),
        # the training step's gradients
        dict(name="gate_up_grad_4096", op="gate_up_grad", M=4096, N=4096, K=4096, keep="bf16", dh="bf16",
             dx="bf16", dw="bf16"),
        # a ragged micro-batch whose weight gradient stays in f32, for a sum over micro-batches
        dict(name="gate_up_grad_1237", op="gate_up_grad", M=1237, N=2832, K=2560, keep="bf16", dh="bf16",
             dx="bf16", dw="f32"),
        # a few rows with frozen weights, everything in f32
        dict(name="gate_up_grad_64", op="gate_up_grad", M=64, N=4096, K=4096, keep="f32", dh="f32",
             dx="f32", dw=None),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["w4", "w4", "gate_up", "gate_up_grad"])
    dt = lambda: rng.choice(["f32", "bf16"])  # noqa: E731
    if op == "w4":
        G = rng.choice([32, 64, 128, 256])
        K = G * _log_int(rng, 1, 8192 // G)
        c = dict(op=op, E=0, T=_log_int(rng, 1, 64), k=0, N=2 * _log_int(rng, 32, 8192), K=K, G=G, scale=dt(),
                 zeros=rng.random() < 0.5, weighted=False, act=rng.random() < 0.4, pad=0, out=dt())
        if rng.random() < 0.5:
            c.update(E=_log_int(rng, 8, 256), T=_log_int(rng, 1, 16), k=rng.randint(1, 8))
            c["pad"] = rng.choice([0, c["T"] // 4])
            c["weighted"] = not c["act"] and rng.random() < 0.5
            while c["E"] * c["N"] * K > 1 << 31:
                c["E"] = max(8, c["E"] // 2)
                c["N"] = c["N"] // 4 * 2
            while c["T"] * c["k"] * c["N"] * K > 1 << 29:
                c["T"] = (c["T"] + 1) // 2
                c["N"] = c["N"] // 4 * 2
            c["pad"] = min(c["pad"], c["T"] - 1)
        return c
    c = dict(op=op, M=_log_int(rng, 1, 8192), N=16 * _log_int(rng, 8, 512), K=8 * _log_int(rng, 16, 1024),
             keep=dt() if op == "gate_up_grad" else rng.choice([None, "f32", "bf16"]))
    if op == "gate_up":
        c["out"] = dt()
    else:
        c["dh"] = dt()
        c["dx"], c["dw"] = rng.choice([("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("bf16", None),
                                       (None, "bf16")])
    while c["M"] * c["N"] * c["K"] > 1 << 36:
        c["M"] = (c["M"] + 1) // 2
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _normal(g, shape, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dtype)


def _w4_inputs(case, g):
    E, T, k, N, K, G = (case[n] for n in ("E", "T", "k", "N", "K", "G"))
    lead = (E, N) if E else (N,)
    st = dict(codes=torch.randint(0, 256, lead + (K // 2,), generator=g, device=DEV, dtype=torch.uint8),
              scales=((0.5 + torch.rand(lead + (K // G,), generator=g, device=DEV)) / (8 * math.sqrt(K))).to(
                  DTYPES[case["scale"]]), zeros=None, ids=None, weights=None)
    if case["zeros"]:
        st["zeros"] = torch.randint(4, 13, lead + (K // G,), generator=g, device=DEV, dtype=torch.uint8)
    rows = T
    if E:
        keys = torch.rand((T, E), generator=g, device=DEV)
        st["ids"] = torch.sort(keys, dim=1, descending=True, stable=True).indices[:, :k].int().contiguous()
        if case["pad"]:
            st["ids"][T - case["pad"]:] = -1       # what the router leaves where every expert is masked
        if case["weighted"]:
            st["weights"] = torch.softmax(_normal(g, (T, k)), dim=1)
            rows = T * k                           # a row per expert: the gated products of the layer's first half
    st["x"] = _normal(g, (rows, K), torch.bfloat16)
    return st


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    st = dict(case)
    if case["op"] == "w4":
        st.update(_w4_inputs(case, g))
        return st
    M, N, K = case["M"], case["N"], case["K"]
    st["x"] = _normal(g, (M, K), torch.bfloat16)
    st["w13"] = _normal(g, (N, K), torch.bfloat16, std=1 / math.sqrt(K))
    if case["op"] == "gate_up_grad":
        st["preact"] = _normal(g, (M, N), DTYPES[case["keep"]])
        st["dh_t"] = _normal(g, (M, N // 2), DTYPES[case["dh"]], std=0.1)
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _silu_mul(y):
    g, u = y.chunk(2, dim=-1)
    return g * torch.sigmoid(g) * u


def _w4_weights(codes, scales, zeros, G):
    """Integer codes minus their zero points, times the group scales, in f32."""
    c = torch.stack((codes & 15, codes >> 4), -1).view(scales.shape + (G,)).float()
    z = 8.0 if zeros is None else zeros.float()[..., None]
    return ((c - z) * scales.float()[..., None]).flatten(-2)


def _w4(st):
    G, x = st["G"], st["x"].float()
    if st["ids"] is None:
        y = x @ _w4_weights(st["codes"], st["scales"], st["zeros"], G).t()
    else:
        ids = st["ids"].reshape(-1)
        live = ids >= 0
        e = ids.clamp_min(0).long()
        w = _w4_weights(st["codes"][e], st["scales"][e], None if st["zeros"] is None else st["zeros"][e], G)
        rows = x if x.shape[0] == ids.numel() else x.repeat_interleave(st["k"], 0)
        y = torch.where(live[:, None], torch.bmm(w, rows[:, :, None])[:, :, 0], 0.0)
        if st["weighted"]:
            y = (y.view(st["T"], st["k"], -1) * st["weights"][:, :, None]).sum(1)
    return (_silu_mul(y) if st["act"] else y).to(DTYPES[st["out"]])


def _gate_up(st):
    y = st["x"].float() @ st["w13"].float().t()
    h = _silu_mul(y).to(DTYPES[st["out"]])
    return h if st["keep"] is None else (h, y.to(DTYPES[st["keep"]]))


def _gate_up_grad(st):
    g, u = st["preact"].float().chunk(2, dim=1)
    dh, s = st["dh_t"].float(), torch.sigmoid(g)
    d = torch.cat((dh * u * s * (1 + g * (1 - s)), dh * g * s), 1)
    dx = None if st["dx"] is None else (d @ st["w13"].float()).to(DTYPES[st["dx"]])
    dw = None if st["dw"] is None else (d.t() @ st["x"].float()).to(DTYPES[st["dw"]])
    return dict(dx=dx, dw=dw)


PLAIN = dict(w4=_w4, gate_up=_gate_up, gate_up_grad=_gate_up_grad)


def _library(st):
    import moe_grouped_gemm_route_amd as moe
    dt = {"f32": moe.F32, "bf16": moe.BF16, None: None}
    if st["op"] == "w4":
        return moe.w4_gemv(st["codes"], st["scales"], st["x"], zeros=st["zeros"], topk_ids=st["ids"],
                           topk_weights=st["weights"], out_dtype=dt[st["out"]],
                           act=moe.ACT_SILU_MUL if st["act"] else moe.ACT_NONE)
    if st["op"] == "gate_up":
        return moe.gate_up(st["x"], st["w13"], out_dtype=dt[st["out"]], preact_dtype=dt[st["keep"]])
    dx, dw = moe.gate_up_bwd(st["dh_t"], st["x"], st["w13"], st["preact"], dx_dtype=dt[st["dx"]],
                             dw_dtype=dt[st["dw"]])
    return dict(dx=dx, dw=dw)


def run(state):
    return _library(state) if own else PLAIN[state["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its values in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    N, K = case["N"], case["K"]
    if case["op"] == "w4":
        T, E, k = case["T"], case["E"], case["k"]
        live = T - case["pad"]
        used = 1 if not E else E * (1 - (1 - k / E) ** live)      # experts that some token reaches
        per = N * K / 2 + N * (K // case["G"]) * (SIZES[case["scale"]] + case["zeros"])
        rows_in = T * k if case["weighted"] else T
        rows_out = T if case["weighted"] or not E else T * k
        out = rows_out * (N // 2 if case["act"] else N) * SIZES[case["out"]]
        return {"bytes": used * per + rows_in * K * 2 + out, "flops": 2 * live * max(k, 1) * N * K}
    M = case["M"]
    if case["op"] == "gate_up":
        return {"bytes": 2 * (M + N) * K + M * N * (SIZES[case["out"]] / 2 + SIZES[case["keep"]]),
                "flops": 2 * M * N * K}
    wants = [n for n in ("dx", "dw") if case[n]]
    moved = M * N * (SIZES[case["keep"]] + SIZES[case["dh"]] / 2)
    moved += N * K * 2 + M * K * SIZES[case["dx"]] if case["dx"] else 0
    moved += M * K * 2 + N * K * SIZES[case["dw"]] if case["dw"] else 0
    return {"bytes": moved, "flops": 2 * M * N * K * len(wants)}


def _sigmoid64(x):
    return 1 / (1 + (-x).exp())


def _exact_rows(st, e, x):
    """x [r, K] in 64 bits times the weights of expert e (None: the dense ones), a block of columns at a time."""
    pick = (lambda t: t) if e is None else (lambda t: t[e])
    codes, scales = pick(st["codes"]), pick(st["scales"])
    K, G = st["K"], st["G"]
    out = torch.empty((x.shape[0], st["N"]), dtype=torch.float64, device=DEV)
    for a in range(0, st["N"], 8192):
        c = codes[a:a + 8192].long()
        w = torch.empty((c.shape[0], K), dtype=torch.float64, device=DEV)
        w[:, 0::2] = (c % 16).double()
        w[:, 1::2] = (c // 16).double()
        z = pick(st["zeros"])[a:a + 8192].double() if st["zeros"] is not None else torch.full_like(scales[a:a + 8192], 8).double()
        w -= z.repeat_interleave(G, 1)
        w *= scales[a:a + 8192].double().repeat_interleave(G, 1)
        out[:, a:a + 8192] = x @ w.t()
    return out


def exact(case, seed):
    st = prepare(case, seed)
    N = case["N"]
    h = N // 2
    if case["op"] == "w4":
        x = st["x"].double()
        if st["ids"] is None:
            y = _exact_rows(st, None, x)
        else:
            T, k = case["T"], case["k"]
            y = torch.zeros((T, N) if case["weighted"] else (T * k, N), dtype=torch.float64, device=DEV)
            for t, chosen in enumerate(st["ids"].tolist()):
                for j, e in enumerate(chosen):
                    if e < 0:
                        continue
                    p = t * k + j
                    row = p if case["weighted"] else t
                    v = _exact_rows(st, e, x[row:row + 1])[0]
                    if case["weighted"]:
                        y[t] += st["weights"][t, j].double() * v
                    else:
                        y[p] = v
        return y[:, :h] * _sigmoid64(y[:, :h]) * y[:, h:] if case["act"] else y
    x, w = st["x"].double(), st["w13"].double()
    if case["op"] == "gate_up":
        g, u = x @ w[:h].t(), x @ w[h:].t()
        out = g * _sigmoid64(g) * u
        return out if case["keep"] is None else (out, torch.cat((g, u), 1))
    g, u, dh = st["preact"][:, :h].double(), st["preact"][:, h:].double(), st["dh_t"].double()
    q = _sigmoid64(g)
    dg, du = dh * u * (q + g * q * (1 - q)), dh * (g * q)
    dx = dg @ w[:h] + du @ w[h:] if case["dx"] else None
    dw = torch.cat((dg.t() @ x, du.t() @ x)) if case["dw"] else None
    return dict(dx=dx, dw=dw)
