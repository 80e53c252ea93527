"""Measured cases of the mixture-of-experts block's operators: the RMS norm with the
residual's addition and MXFP8 output (forward and backward), the token routing (gates,
row plan and gradient) and the expert layer for a few tokens.

``run`` computes each operator in plain torch operations in fp32 where ``own`` is false,
and through the package's entry points where it is true.
"""
import math

import torch

own = False

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
TYPES = {"bf16": BF16, "f16": F16, "f32": F32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "mx": 1 + 1 / 32}
EPS = 1e-6
DEV = "cuda"


def listed():
    norm, norm_b = dict(op="norm"), dict(op="norm_backward")
    route, moe = dict(op="route"), dict(op="moe")
    return [
        # one decode step of 4 sequences: the norm before the experts, new residual and normalised rows
        dict(norm, name="norm_decode_4", T=4, C=4096, dtype="bf16", gamma="bf16", residual=True, h=True, y=True, mx=False),
        # training / prefill of 16384 tokens: residual stream, normalised rows and the MXFP8 codes of the experts' product
        dict(norm, name="norm_prefill_mx", T=16384, C=4096, dtype="bf16", gamma="f32", residual=True, h=True, y=True,
             mx=True),
        # a ragged batch of an fp16 model, a norm without a residual and of an odd width
        dict(norm, name="norm_ragged_f16", T=4099, C=1992, dtype="f16", gamma="f16", residual=False, h=False, y=True,
             mx=False),
        # backward of the training batch, with the gradient that arrives through the residual stream
        dict(norm_b, name="norm_backward_train", T=16384, C=4096, dtype="bf16", gamma="f32", dh=True),
        # backward of a short ragged batch in fp32, wide rows
        dict(norm_b, name="norm_backward_f32", T=333, C=7168, dtype="f32", gamma="f32", dh=False),
        # one decode step of 32 sequences over 64 experts, with the row plan
        dict(route, name="route_decode_32", T=32, E=64, k=8, dtype="f32", score="softmax", renorm=True, masked=False),
        # prefill of 32768 tokens over 256 experts, some experts masked per token and some padding tokens
        dict(route, name="route_prefill", T=32768, E=256, k=8, dtype="bf16", score="sigmoid", renorm=True, masked=True),
        # the gates' gradient over a training batch
        dict(op="route_backward", name="route_backward_train", T=16384, E=64, k=4, dtype="f32", score="softmax",
             renorm=False, masked=False),
        # one token through a layer of 64 small experts: the least a decode step can ask for
        dict(moe, name="moe_one_token", T=1, E=64, k=8, K=2048, F=768, N=2048, w="bf16", bias=False, residual=True,
             absent=False),
        # five tokens of an fp16 model with 8 large experts and biases
        dict(moe, name="moe_f16_5_tokens", T=5, E=8, k=2, K=4096, F=14336, N=4096, w="f16", bias=True, residual=False,
             absent=False),
        # 17 tokens, experts held as MXFP8 codes, a part of them on another device
        dict(moe, name="moe_mx_17_tokens", T=17, E=32, k=4, K=4096, F=2048, N=4096, w="mx", bias=False, residual=True,
             absent=True),
        # the most tokens the layer takes, 256 experts of a large model
        dict(moe, name="moe_64_tokens", T=64, E=256, k=8, K=7168, F=2048, N=7168, w="bf16", bias=False, residual=True,
             absent=False),
    ]


def draw(rng):
    def size(lo, hi, step=1):
        v = max(step, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)
        return v + step if v in (1536, 3072) else v

    op = rng.choice(["norm", "norm", "norm_backward", "route", "route_backward", "moe", "moe", "moe"])
    yes = lambda: rng.random() < 0.5  # noqa: E731
    if op in ("norm", "norm_backward"):
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        gamma = rng.choice([dtype, "f32"])
        mx = op == "norm" and yes()
        T, C = size(1, 16384), size(64, 8192, 32 if mx else 8)
        T = max(1, min(T, 16384 * 4096 // (C * SIZE[dtype] // 2)))
        if op == "norm_backward":
            return dict(op=op, T=T, C=C, dtype=dtype, gamma=gamma, dh=yes())
        residual = yes()
        return dict(op=op, T=T, C=C, dtype=dtype, gamma=gamma, residual=residual, h=residual, y=not mx or yes(), mx=mx)
    if op in ("route", "route_backward"):
        E = size(2, 512)
        T = size(1, 32768)
        k = min(E, size(1, 16))
        return dict(op=op, T=min(T, 32768 * 256 // E), E=E, k=k, dtype=rng.choice(["f32", "f32", "bf16", "f16"]),
                    score=rng.choice(["softmax", "sigmoid"]), renorm=k > 1 and yes(), masked=yes())
    w = rng.choice(["bf16", "bf16", "f16", "f32", "mx"])
    K, F = size(256, 7168, 32), size(128, 8192, 32)
    N = rng.choice([K, size(256, 7168, 8)])
    E = min(size(2, 256), max(2, int(5e9 / SIZE[w] / (2 * F * K + N * F))))
    T, k = size(1, 64), min(E, size(1, 12))
    return dict(op=op, T=T, E=E, k=k, K=K, F=F, N=N, w=w, bias=yes(), residual=yes(), absent=T * k >= 8 and yes())


# ------------------------------------------------------------------------ inputs


def _logits(case, rand):
    logits = rand(case["T"], case["E"]) * 1.5
    if case["masked"]:  # a tenth of the experts per token, and one token in fifty is padding: all of its experts
        u = torch.rand(case["T"], case["E"] + 1, device=DEV, generator=rand.gen)
        logits = logits.masked_fill((u[:, 1:] < 0.1) | (u[:, :1] < 0.02), -math.inf)
    return logits.to(TYPES[case["dtype"]])


def _mx_matrix(w):
    """E4M3 codes [rows, cols] and E8M0 scales [rows, cols / 32] of one expert's matrix."""
    v = w.view(w.shape[0], -1, 32)
    x = torch.floor(torch.log2(v.abs().amax(-1))) - 8
    q = (v * torch.exp2(-x)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).view(w.shape), (x + 127).to(torch.uint8)


class _Rand:
    def __init__(self, seed):
        self.gen = torch.Generator(device=DEV).manual_seed(int(seed))

    def __call__(self, *shape, dtype=F32):
        return torch.randn(*shape, generator=self.gen, device=DEV, dtype=dtype)


def prepare(case, seed):
    rand = _Rand(seed)
    s = {"case": case, "kept": {}}  # kept: the workspace, made by the first call as a program's would be
    op = case["op"]
    if op in ("norm", "norm_backward"):
        T, C, dt = case["T"], case["C"], TYPES[case["dtype"]]
        new = lambda dtype=dt: torch.empty(T, C, dtype=dtype, device=DEV)  # noqa: E731
        outliers = 1 + 9 * (torch.rand(C, device=DEV, generator=rand.gen) < 0.01)  # a few large channels
        s["gamma"] = (1 + 0.2 * rand(C)).to(TYPES[case["gamma"]])
        if op == "norm":
            s["x"] = (rand(T, C) * outliers).to(dt)
            s["residual"] = (3 * rand(T, C) * outliers).to(dt) if case["residual"] else None
            s["h"] = new() if case["h"] else None
            s["y"] = new() if case["y"] else None
            if case["mx"]:
                s["data"] = new(torch.uint8)
                s["scale"] = torch.empty(T, C // 32, dtype=torch.uint8, device=DEV)
        else:
            s["h"] = (3 * rand(T, C) * outliers).to(dt)
            s["dy"] = (0.1 * rand(T, C)).to(dt)
            s["dh"] = (0.1 * rand(T, C)).to(dt) if case["dh"] else None
            s["dx"] = new()
            s["dgamma"] = torch.empty(C, dtype=F32, device=DEV)
    elif op in ("route", "route_backward"):
        T, E, k = case["T"], case["E"], case["k"]
        s["logits"] = _logits(case, rand)
        s["ids"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
        if op == "route":
            s["weights"] = torch.empty(T, k, dtype=F32, device=DEV)
            s["m_splits"] = torch.empty(E, dtype=torch.int64, device=DEV)
            s["row_index"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
            s["slot_index"] = torch.empty(T * k, dtype=torch.int32, device=DEV)
        else:
            s["ids"] = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True)[1][:, :k].to(torch.int32)
            s["ids"] = s["ids"].contiguous()
            s["dweights"] = rand(T, k)
            s["dlogits"] = torch.empty_like(s["logits"])
    else:
        T, E, k, K, F, N = (case[n] for n in ("T", "E", "k", "K", "F", "N"))
        dt = BF16 if case["w"] == "mx" else TYPES[case["w"]]
        s["x"] = rand(T, K).to(dt)
        top, ids = torch.topk(rand(T, E) * 1.5, k, dim=1)
        s["weights"] = torch.softmax(top, 1)
        if case["absent"]:  # experts of the upper quarter are held elsewhere: their slots name none
            ids = ids.masked_fill(ids >= E - E // 4, -1)
        s["ids"] = ids.to(torch.int32)
        w1_std, w2_std = K ** -0.5, F ** -0.5
        if case["w"] == "mx":
            for name, rows, cols, std in (("w1", 2 * F, K, w1_std), ("w2", N, F, w2_std)):
                s[name] = torch.empty(E, rows, cols, dtype=torch.uint8, device=DEV)
                s[name + "_scale"] = torch.empty(E, rows, cols // 32, dtype=torch.uint8, device=DEV)
                for e in range(E):
                    s[name][e], s[name + "_scale"][e] = _mx_matrix(rand(rows, cols) * std)
        else:
            s["w1"] = rand(E, 2 * F, K, dtype=dt).mul_(w1_std)
            s["w2"] = rand(E, N, F, dtype=dt).mul_(w2_std)
            s["w1_scale"] = s["w2_scale"] = None
        s["b1"] = (0.1 * rand(E, 2 * F)).to(dt) if case["bias"] else None
        s["b2"] = (0.1 * rand(E, N)).to(dt) if case["bias"] else None
        s["residual"] = rand(T, N).to(dt) if case["residual"] else None
        s["y"] = torch.empty(T, N, dtype=dt, device=DEV)
    return s


# ------------------------------------------------------------------- plain forms


def _mx_codes(y):
    """The E4M3 values and E8M0 scales of y's blocks of 32 along each row."""
    T, C = y.shape
    v = y.view(T, C // 32, 32)
    amax = v.abs().amax(-1)
    e = torch.floor(torch.log2(amax)) - 8
    e = torch.where(torch.exp2(e + 8) > amax, e - 1, e)  # log2 rounded up to the next whole number
    e = torch.where(torch.exp2(e + 9) <= amax, e + 1, e)  # or down
    e = torch.where(amax == 0, -127.0, e).clamp(-127, 127)
    q = (v * torch.exp2(-e)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(T, C), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _plain_norm(s):
    case, dt = s["case"], s["x"].dtype
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    rstd = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)
    y = h * rstd * s["gamma"].float()
    out = {}
    if case["h"]:
        out["h"] = h.to(dt)
    if case["y"]:
        out["y"] = y.to(dt)
    if case["mx"]:
        out["data"], out["scale"] = _mx_codes(y)
    return out


def _plain_norm_backward(s):
    h, dy = s["h"].float(), s["dy"].float()
    rstd = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)
    xh = h * rstd
    v = dy * s["gamma"].float()
    dx = rstd * (v - xh * (v * xh).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["h"].dtype), "dgamma": (dy * xh).sum(0)}


def _plain_scores(case, logits):
    """Scores of all experts, zero where the logit is masked, and the masked logits."""
    l = torch.where(torch.isnan(logits), -math.inf, logits.float())
    if case["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-l)), l
    top = l.amax(1, keepdim=True)
    p = torch.where(l == -math.inf, 0.0, torch.exp(l - top))
    total = p.sum(1, keepdim=True)
    return torch.where(total > 0, p / total, 0.0), l


def _plain_route(s):
    case = s["case"]
    E, k = case["E"], case["k"]
    scores, l = _plain_scores(case, s["logits"])
    ids = torch.sort(l, dim=1, descending=True, stable=True)[1][:, :k]  # stable: ties go to the lowest expert
    w = scores.gather(1, ids)
    if case["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    flat = ids.reshape(-1)
    slots = torch.sort(flat, stable=True)[1]
    rows = torch.empty_like(slots)
    rows[slots] = torch.arange(flat.numel(), device=flat.device)
    splits = torch.zeros(E, dtype=torch.int64, device=flat.device).scatter_add_(0, flat, torch.ones_like(flat))
    return {"ids": ids.to(torch.int32), "weights": w, "m_splits": splits, "row_index": rows.view_as(ids).to(torch.int32),
            "slot_index": slots.to(torch.int32)}


def _plain_route_backward(s):
    case = s["case"]
    ids, dw = s["ids"].long(), s["dweights"]
    scores, l = _plain_scores(case, s["logits"])
    w = scores.gather(1, ids)
    total = w.sum(1, keepdim=True)
    if case["renorm"]:  # to the gradient of the scores before they were divided
        w = torch.where(total > 0, w / total, 0.0)
        dw = torch.where(total > 0, (dw - (dw * w).sum(1, keepdim=True)) / total, 0.0)
    ds = torch.zeros_like(scores).scatter_(1, ids, dw)
    if case["score"] == "sigmoid":
        return {"dlogits": (ds * scores * (1 - scores)).to(s["logits"].dtype)}
    return {"dlogits": (scores * (ds - (ds * scores).sum(1, keepdim=True))).to(s["logits"].dtype)}


def _weights32(w, scale):
    if scale is None:
        return w.float()
    q = w.view(torch.float8_e4m3fn).float()
    return (q.view(*scale.shape, 32) * torch.exp2(scale.float() - 127)[..., None]).view(w.shape)


def _plain_moe(s):
    case = s["case"]
    T, E, k, F, N = (case[n] for n in ("T", "E", "k", "F", "N"))
    x, here = s["x"].float(), s["ids"] >= 0
    gates = torch.where(here, s["weights"], 0.0)
    ids = torch.where(here, s["ids"], 0).long()
    pick = lambda t, at: t if t is None or at is None else t[at]  # noqa: E731
    few = T * k <= E  # a slot's own experts, or every expert on all tokens, whichever reads less
    at = ids.reshape(-1) if few else None
    w1 = _weights32(pick(s["w1"], at), pick(s["w1_scale"], at))
    w2 = _weights32(pick(s["w2"], at), pick(s["w2_scale"], at))
    rows = x[:, None].expand(T, k, x.shape[1]).reshape(T * k, 1, -1) if few else x.expand(E, *x.shape)
    h = torch.matmul(rows, w1.transpose(1, 2))
    if s["b1"] is not None:
        h = h + pick(s["b1"], at).float()[:, None]
    g, u = h[..., :F], h[..., F:]
    z = torch.matmul(g / (1 + torch.exp(-g)) * u, w2.transpose(1, 2))
    if s["b2"] is not None:
        z = z + pick(s["b2"], at).float()[:, None]
    if few:
        y = (z.view(T, k, N) * gates[..., None]).sum(1)
    else:
        dense = torch.zeros(T, E, device=x.device).scatter_add_(1, ids, gates)
        y = (z * dense.t()[..., None]).sum(0)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": y.to(s["y"].dtype)}


PLAIN = {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "route": _plain_route,
         "route_backward": _plain_route_backward, "moe": _plain_moe}


# -------------------------------------------------------------- the entry points


def _workspace(s, size):
    if "ws" not in s["kept"]:
        s["kept"]["ws"] = torch.empty(size(), dtype=torch.uint8, device=DEV)
    return s["kept"]["ws"]


def _own(s):
    import grouped_gemm_gl_amd as gl

    case, op = s["case"], s["case"]["op"]
    if op == "norm":
        data, scale = s.get("data"), s.get("scale")
        gl.gl_rmsnorm_forward(s["x"], s["gamma"], EPS, residual=s["residual"], h=s["h"], y=s["y"], data=data, scale=scale)
        out = {n: s[n] for n in ("h", "y") if s[n] is not None}
        if case["mx"]:
            out["data"], out["scale"] = data.view(torch.float8_e4m3fn), scale.view(torch.float8_e8m0fnu)
        return out
    if op == "norm_backward":
        ws = _workspace(s, lambda: gl.gl_rmsnorm_workspace_size(case["T"], case["C"]))
        gl.gl_rmsnorm_backward(s["dy"], s["h"], s["gamma"], EPS, s["dx"], dh=s["dh"], dgamma=s["dgamma"], workspace=ws)
        return {"dx": s["dx"], "dgamma": s["dgamma"]}
    if op in ("route", "route_backward"):
        score = gl.GL_SCORE_SIGMOID if case["score"] == "sigmoid" else gl.GL_SCORE_SOFTMAX
        if op == "route_backward":
            gl.gl_route_backward(s["logits"], s["ids"], s["dweights"], s["dlogits"], score=score, renormalize=case["renorm"])
            return {"dlogits": s["dlogits"]}
        ws = _workspace(s, lambda: gl.gl_route_workspace_size(case["T"], case["E"]))
        gl.gl_route_forward(s["logits"], s["ids"], s["weights"], score=score, renormalize=case["renorm"],
                            m_splits=s["m_splits"], row_index=s["row_index"], slot_index=s["slot_index"], workspace=ws)
        return {n: s[n] for n in ("ids", "weights", "m_splits", "row_index", "slot_index")}
    ws = _workspace(s, lambda: gl.gl_moe_few_tokens_workspace_size(case["T"], case["k"], case["E"], case["F"]))
    gl.gl_moe_few_tokens(s["x"], s["ids"], s["weights"], s["w1"], s["w2"], s["y"], ws, w1_scale=s["w1_scale"],
                         w2_scale=s["w2_scale"], b1=s["b1"], b2=s["b2"], residual=s["residual"])
    return {"y": s["y"]}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ----------------------------------------------------------------- work and exact


def work(case):
    op = case["op"]
    if op in ("norm", "norm_backward"):
        n, b = case["T"] * case["C"], SIZE[case["dtype"]]
        if op == "norm":
            moved = n * (b * (1 + case["residual"] + case["h"] + case["y"]) + case["mx"] * SIZE["mx"])
            return {"bytes": moved + case["C"] * SIZE[case["gamma"]], "flops": 5 * n}
        return {"bytes": n * b * (3 + case["dh"]) + case["C"] * (SIZE[case["gamma"]] + 4), "flops": 10 * n}
    if op in ("route", "route_backward"):
        n, slots = case["T"] * case["E"], case["T"] * case["k"]
        if op == "route":
            return {"bytes": n * SIZE[case["dtype"]] + slots * 16 + case["E"] * 8, "flops": 6 * n}
        return {"bytes": 2 * n * SIZE[case["dtype"]] + slots * 8, "flops": 8 * n}
    T, E, k, K, F, N = (case[n] for n in ("T", "E", "k", "K", "F", "N"))
    share = (E - E // 4) / E if case["absent"] else 1.0
    used = share * E * (1 - (1 - k / E) ** T)  # the experts that T tokens' draws name, on average
    per_expert = 2 * F * K + N * F
    act = 4 if case["w"] == "f32" else 2
    moved = used * (per_expert * SIZE[case["w"]] + case["bias"] * act * (2 * F + N))
    moved += T * (act * (K + N * (1 + case["residual"])) + 8 * k)
    return {"bytes": moved, "flops": 2 * share * T * k * per_expert}


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    f64 = lambda t: t.to(torch.float64)  # noqa: E731
    if op == "norm":
        h = f64(s["x"]) if s["residual"] is None else f64(s["x"]) + f64(s["residual"])
        norm = torch.linalg.vector_norm(h, dim=1, keepdim=True)
        y = h / torch.sqrt(norm.square() / case["C"] + EPS) * f64(s["gamma"])
        out = {n: v for n, v in (("h", h), ("y", y)) if case[n]}
        if case["mx"]:  # what the codes stand for before their rounding, in the scale of their block
            blocks = y.reshape(case["T"], -1, 32)
            top = torch.frexp(blocks.abs().amax(-1, keepdim=True))[1] - 1
            out["data"] = torch.ldexp(blocks, 8 - top).reshape(y.shape)
            out["scale"] = None
        return out
    if op == "norm_backward":
        h, dy, C = f64(s["h"]), f64(s["dy"]), case["C"]
        r = torch.sqrt(h.square().sum(1) / C + EPS)
        gdy = dy * f64(s["gamma"])
        dx = gdy / r[:, None] - h * ((gdy * h).sum(1) / (C * r ** 3))[:, None]
        if s["dh"] is not None:
            dx = dx + f64(s["dh"])
        return {"dx": dx, "dgamma": torch.mv((dy * h).t(), 1 / r)}
    if op in ("route", "route_backward"):
        l = f64(s["logits"])
        k, masked = case["k"], torch.isinf(l)
        chosen = torch.argsort(l, dim=1, descending=True, stable=True)[:, :k]
        keep = torch.zeros_like(masked).scatter_(1, chosen, torch.ones_like(chosen, dtype=torch.bool))
        if case["score"] == "softmax":
            over = l.masked_fill(~keep, -math.inf) if case["renorm"] else l
            scores = torch.nan_to_num(torch.softmax(over, 1), nan=0.0)
        else:
            scores = torch.sigmoid(l)
            if case["renorm"]:
                scores = torch.nan_to_num(scores / (scores * keep).sum(1, keepdim=True), nan=0.0)
        if op == "route":
            return {"ids": None, "weights": scores.gather(1, chosen), "m_splits": None, "row_index": None, "slot_index": None}
        d = torch.zeros_like(l).scatter_(1, chosen, f64(s["dweights"]))
        mean = (d * scores * keep).sum(1, keepdim=True)
        if case["score"] == "softmax":
            return {"dlogits": scores * (d - mean)}
        slope = 1 - torch.sigmoid(l)
        return {"dlogits": keep * scores * slope * ((d - mean) if case["renorm"] else d)}
    y = torch.zeros(case["T"], case["N"], dtype=torch.float64, device=DEV)
    if s["residual"] is not None:
        y += s["residual"]
    ids, F = s["ids"].long(), case["F"]

    def matrix(name, e):
        w, sc = s[name][e], s[name + "_scale"]
        if sc is None:
            return f64(w)
        return torch.ldexp(f64(w.view(torch.float8_e4m3fn)), sc[e].int().repeat_interleave(32, dim=1) - 127)

    for e in range(case["E"]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if not t.numel():
            continue
        h = f64(s["x"][t]) @ matrix("w1", e).t()
        if s["b1"] is not None:
            h = h + f64(s["b1"][e])
        z = (h[:, :F] * torch.sigmoid(h[:, :F]) * h[:, F:]) @ matrix("w2", e).t()
        if s["b2"] is not None:
            z = z + f64(s["b2"][e])
        y[t] += z * f64(s["weights"][t, j])[:, None]  # an expert names a token once
    return {"y": y}
