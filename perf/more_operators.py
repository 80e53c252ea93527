"""Measured cases of the experts' gated first layer (both projections, the activation and their
product, forward and backward) and of the grouped product in 8-bit integers (rows quantized with a
scale for each token, the product with scales for each token and channel, plain or gated).

``run`` computes each operator in plain torch operations in fp32 where ``own`` is false,
and through the package's entry points where it is true.
"""
import math

import torch

own = False

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
TYPES = {"bf16": BF16, "f16": F16, "f32": F32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
LEAST = 2.0 ** -100  # a row's largest magnitude counts as at least this when it is quantized
DEV = "cuda"


def listed():
    glu, glu_b = dict(op="glu", bias=False, h=False), dict(op="glu_backward", bias=False)
    quant, prod = dict(op="quantize_int8"), dict(op="int8", bias=False)
    return [
        # one token through 8 of 64 small experts: the least a decode step can ask for
        dict(glu, name="glu_one_token", G=64, T=8, K=2048, F=768, dtype="bf16", act="silu"),
        # training or prefill of 16384 token rows over 8 large experts, the values before the activation kept
        dict(glu, name="glu_train", G=8, T=16384, K=4096, F=7168, dtype="bf16", act="silu", h=True),
        # a ragged batch over 64 experts of an fp16 model with biases, and an odd width
        dict(glu, name="glu_ragged_f16", G=64, T=4099, K=2048, F=1400, dtype="f16", act="gelu", bias=True),
        # a small fp32 model
        dict(glu, name="glu_f32", G=4, T=333, K=1024, F=2048, dtype="f32", act="gelu_tanh"),
        # backward of the training batch from the tokens alone (nothing of the forward was kept)
        dict(glu_b, name="glu_backward_train", G=8, T=16384, K=4096, F=7168, dtype="bf16", act="silu", kept=False),
        # backward of a ragged batch over 64 experts with biases, from the kept values
        dict(glu_b, name="glu_backward_ragged_f16", G=64, T=4099, K=2048, F=1400, dtype="f16", act="gelu", bias=True,
             kept=True),
        # backward of a small fp32 model
        dict(glu_b, name="glu_backward_f32", G=4, T=333, K=1024, F=1024, dtype="f32", act="silu", kept=True),
        # the tokens of one decode step of 4 sequences
        dict(quant, name="quantize_decode_4", T=4, K=4096, dtype="bf16"),
        # the tokens of a prefill
        dict(quant, name="quantize_prefill", T=16384, K=4096, dtype="bf16"),
        # 4 tokens of a decode step through 8 of 64 experts each: second layer of the experts
        dict(prod, name="int8_decode", G=64, T=32, K=1408, F=2048, dtype="bf16", act="none"),
        # prefill of 16384 token rows over 8 large experts
        dict(prod, name="int8_prefill", G=8, T=16384, K=4096, F=14336, dtype="bf16", act="none"),
        # gated first layer of a ragged batch over 64 experts, with biases
        dict(prod, name="int8_glu_ragged", G=64, T=4099, K=2048, F=1408, dtype="f16", act="silu", bias=True),
    ]


MOST_FLOPS = 3 * 4 * 16384 * 4096 * 7168  # of the largest listed case


def draw(rng):
    def size(lo, hi, step=1):
        v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
        return max(step, int(round(v / step)) * step)

    yes = lambda: rng.random() < 0.5  # noqa: E731
    op = rng.choice(["glu", "glu", "glu_backward", "glu_backward", "quantize_int8", "int8", "int8"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "quantize_int8":
        K = size(64, 16384, 16)
        return dict(op=op, T=max(1, min(size(1, 16384), 16384 * 4096 // K)), K=K, dtype=dtype)
    G = size(1, 256)
    K, F = size(128, 7168, 16), size(64, 14336, 8)
    G = max(1, min(G, int(8 * 14336 * 4096 / (2 * F * K))))
    rows = 16384 if dtype != "f32" or op == "int8" else 2048
    T = size(1, rows)
    T = max(1, min(T, int(MOST_FLOPS / 3 / (4 * F * K))))
    case = dict(op=op, G=G, T=T, K=K, F=F, dtype=dtype, act=rng.choice(["silu", "silu", "gelu", "gelu_tanh"]), bias=yes())
    if op == "glu":
        case["h"] = yes()
    elif op == "glu_backward":
        case["kept"] = yes()
    elif yes():
        case["act"] = "none"
    return case


# ------------------------------------------------------------------------ inputs


class _Rand:
    def __init__(self, seed):
        self.gen = torch.Generator(device=DEV).manual_seed(int(seed))

    def __call__(self, *shape, dtype=F32):
        return torch.randn(*shape, generator=self.gen, device=DEV, dtype=dtype)

    def tokens(self, T, K):
        """Normalised rows: a few channels are large in all of them."""
        return self(T, K).mul_(1 + 9 * (torch.rand(K, device=DEV, generator=self.gen) < 0.01))

    def splits(self, G, T):
        """Rows of each expert: some are asked for more often than others, some not at all."""
        p = torch.softmax(0.5 * self(G), 0)
        return torch.bincount(torch.multinomial(p, T, replacement=True, generator=self.gen), minlength=G)


def _int8(v):
    """Codes and scale of each row of v (in fp32)."""
    top = v.abs().amax(-1).clamp_min(LEAST)
    return torch.round(v * (127.0 / top)[..., None]).to(torch.int8), top / 127.0


def prepare(case, seed):
    rand, op = _Rand(seed), case["op"]
    T, K, dt = case["T"], case["K"], TYPES[case["dtype"]]
    s = {"case": case, "kept": {}}  # kept: the workspace, made by the first call as a program's would be
    new = lambda *shape, dtype=dt: torch.empty(*shape, dtype=dtype, device=DEV)  # noqa: E731
    if op == "quantize_int8":
        s.update(x=rand.tokens(T, K).to(dt), data=new(T, K, dtype=torch.int8), scale=new(T, dtype=F32))
        return s
    G, F = case["G"], case["F"]
    N = F if case["act"] == "none" else 2 * F
    s["m_splits"] = rand.splits(G, T)
    s["most"] = int(s["m_splits"].max())  # rows of the largest expert
    x = rand.tokens(T, K)
    w = rand(G, N, K, dtype=BF16 if op == "int8" else dt).mul_(K ** -0.5)
    s["bias"] = (0.1 * rand(G, N)).to(dt) if case["bias"] else None
    if op == "int8":
        s["x"], s["x_scale"] = _int8(x)
        s["w"], s["w_scale"] = new(G, N, K, dtype=torch.int8), new(G, N, dtype=F32)
        for g in range(G):
            s["w"][g], s["w_scale"][g] = _int8(w[g].float())
        s["y"] = new(T, F)
        return s
    s["x"], s["w"] = x.to(dt), w
    if op == "glu":
        s["a"], s["h"] = new(T, F), new(T, N) if case["h"] else None
    else:
        s["da"] = (0.1 * rand(T, F)).to(dt)
        # about what x and w would give
        s["h"] = rand(T, N).to(dt) if case["kept"] else None
        s["dh"], s["dx"], s["dw"] = new(T, N), new(T, K), new(G, N, K)
        s["db"] = new(G, N) if case["bias"] else None
    return s


# ------------------------------------------------------------------- plain forms


def _where(s):
    """The expert of each row and the row's place among the expert's."""
    ends = torch.cumsum(s["m_splits"], 0)
    at = torch.arange(s["case"]["T"], device=ends.device)
    g = torch.searchsorted(ends, at, right=True)
    return g, at - (ends - s["m_splits"])[g]


def _by_expert(s, rows, g, place):
    """The rows as [G, most, C], zeros behind an expert's last."""
    out = torch.zeros(s["case"]["G"], s["most"], rows.shape[1], device=rows.device)
    out[g, place] = rows.float()
    return out


def _grouped_product(s, x, w):
    """x [T, K] times each row's expert's w [G, N, K], fp32 [T, N]."""
    g, place = _where(s)
    if s["case"]["T"] <= s["case"]["G"]:  # fewer rows than experts: only the named experts' weights are read
        return torch.matmul(x.float()[:, None], w[g].float().transpose(1, 2))[:, 0]
    return torch.matmul(_by_expert(s, x, g, place), w.float().transpose(1, 2))[g, place]


def _act(name, v):
    """The activation and its slope."""
    if name == "silu":
        q = 1 / (1 + torch.exp(-v))
        return v * q, q * (1 + v * (1 - q))
    if name == "gelu":
        q = 0.5 * (1 + torch.erf(v * math.sqrt(0.5)))
        return v * q, q + v * torch.exp(-0.5 * v * v) * (1 / math.sqrt(2 * math.pi))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (v + 0.044715 * v * v * v))
    return 0.5 * v * (1 + t), 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * c * (1 + 3 * 0.044715 * v * v)


def _with_bias(s, h):
    return h if s["bias"] is None else h + s["bias"].float()[_where(s)[0]]


def _plain_glu(s):
    F, dt = s["case"]["F"], s["x"].dtype
    h = _with_bias(s, _grouped_product(s, s["x"], s["w"]))
    out = {"a": (_act(s["case"]["act"], h[:, :F])[0] * h[:, F:]).to(dt)}
    if s["case"]["h"]:
        out["h"] = h.to(dt)
    return out


def _plain_glu_backward(s):
    case, dt, w = s["case"], s["x"].dtype, s["w"].float()
    F, (g, place) = case["F"], _where(s)
    x = _by_expert(s, s["x"], g, place)
    if case["kept"]:
        h = s["h"].float()
    else:
        h = _with_bias(s, torch.matmul(x, w.transpose(1, 2))[g, place])
    y, slope = _act(case["act"], h[:, :F])
    da = s["da"].float()
    dh = _by_expert(s, torch.cat([da * h[:, F:] * slope, da * y], 1), g, place)
    out = {"dx": torch.matmul(dh, w)[g, place].to(dt), "dw": torch.matmul(dh.transpose(1, 2), x).to(dt)}
    if case["bias"]:
        out["db"] = dh.sum(1).to(dt)
    return out


def _plain_quantize(s):
    data, scale = _int8(s["x"].float())
    return {"data": data, "scale": scale}


def _plain_int8(s):
    F, act = s["case"]["F"], s["case"]["act"]
    h = _grouped_product(s, s["x"], s["w"]) * s["x_scale"][:, None] * s["w_scale"][_where(s)[0]]
    h = _with_bias(s, h)
    return {"y": (h if act == "none" else _act(act, h[:, :F])[0] * h[:, F:]).to(s["y"].dtype)}


PLAIN = {"glu": _plain_glu, "glu_backward": _plain_glu_backward, "quantize_int8": _plain_quantize, "int8": _plain_int8}


# -------------------------------------------------------------- the entry points


def _own(s):
    import grouped_gemm_gl_amd as gl

    case, op = s["case"], s["case"]["op"]
    if op == "quantize_int8":
        gl.gl_quantize_int8(s["x"], s["data"], s["scale"])
        return {"data": s["data"], "scale": s["scale"]}
    if "ws" not in s["kept"]:
        s["kept"]["ws"] = gl.new_workspace(case["G"])
    ws = s["kept"]["ws"]
    act = {"silu": gl.GL_GLU_SILU, "gelu": gl.GL_GLU_GELU, "gelu_tanh": gl.GL_GLU_GELU_TANH, "none": None}[case["act"]]
    gl.gl_offsets(s["m_splits"], case["T"], ws)  # the rows of each expert are new with every step
    if op == "glu":
        gl.gl_glu_forward(s["x"], s["w"], s["a"], ws, bias=s["bias"], h=s["h"], act=act)
        return {n: s[n] for n in ("a", "h") if s[n] is not None}
    if op == "glu_backward":
        gl.gl_glu_backward(s["x"], s["w"], s["da"], s["dh"], s["dx"], s["dw"], ws, h=s["h"], bias=s["bias"], db=s["db"],
                           act=act)
        return {n: s[n] for n in ("dx", "dw", "db") if s[n] is not None}
    if act is None:
        gl.gl_forward_int8(s["x"], s["x_scale"], s["w"], s["w_scale"], s["y"], ws, bias=s["bias"])
    else:
        gl.gl_glu_forward_int8(s["x"], s["x_scale"], s["w"], s["w_scale"], s["y"], ws, bias=s["bias"], act=act)
    return {"y": s["y"]}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ----------------------------------------------------------------- work and exact


def work(case):
    T, K, b = case["T"], case["K"], SIZE[case["dtype"]]
    if case["op"] == "quantize_int8":
        return {"bytes": T * K * (b + 1) + 4 * T, "flops": 3 * T * K}
    G, F = case["G"], case["F"]
    N = F if case["act"] == "none" else 2 * F
    used = G * (1 - (1 - 1 / G) ** T)  # the experts that T rows name, about
    wide = 1 if case["op"] == "int8" else b
    moved = used * N * (K * wide + b * case["bias"]) + 8 * G
    if case["op"] == "glu_backward":
        moved += G * N * b * (K + case["bias"]) + T * b * (2 * K + F + N * case["kept"])
        return {"bytes": moved, "flops": 2 * T * K * N * (2 if case["kept"] else 3)}
    moved += T * (K * wide + F * b)
    if case["op"] == "int8":
        moved += 4 * (T + used * N)
    elif case["h"]:
        moved += T * N * b
    return {"bytes": moved, "flops": 2 * T * K * N}


def _exact_act(name, v):
    if name == "silu":
        p = torch.sigmoid(v)
        return v * p, p + v * p * torch.sigmoid(-v)
    if name == "gelu":
        p = 0.5 * torch.special.erfc(-v / math.sqrt(2))
        return v * p, p + v * torch.exp(-v.square() / 2) / math.sqrt(2 * math.pi)
    z = 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)  # (1 + tanh(z / 2)) / 2 is the sigmoid of z
    p = torch.sigmoid(z)
    return v * p, p + v * p * torch.sigmoid(-z) * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * v.square())


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    f64 = lambda t: t.to(torch.float64)  # noqa: E731
    if op == "quantize_int8":
        top = f64(s["x"]).abs().max(1).values
        return {"data": None, "scale": torch.clamp(top, min=LEAST) / 127}
    F, act, first = case["F"], case["act"], 0
    parts = []
    for e, rows in enumerate(s["m_splits"].tolist()):
        r = slice(first, first + rows)
        first += rows
        x, w = f64(s["x"][r]), f64(s["w"][e])
        if op == "glu_backward" and case["kept"]:
            h = f64(s["h"][r])
        else:
            h = x @ w.t()
            if op == "int8":
                h = h * torch.outer(f64(s["x_scale"][r]), f64(s["w_scale"][e]))
            if s["bias"] is not None:
                h = h + f64(s["bias"][e])
        if act == "none":
            parts.append((h,))
            continue
        gate, slope = _exact_act(act, h[:, :F])
        if op == "glu_backward":
            da = f64(s["da"][r])
            dh = torch.cat([da * slope * h[:, F:], da * gate], 1)
            parts.append((dh @ w, dh.t() @ x, dh.sum(0)))
        else:
            parts.append((gate * h[:, F:], h if op == "glu" and case["h"] else None))
    if op == "glu_backward":
        dx, dw, db = zip(*parts)
        out = {"dx": torch.cat(dx), "dw": torch.stack(dw)}
        return dict(out, db=torch.stack(db)) if case["bias"] else out
    if op == "int8":
        return {"y": torch.cat([p[0] for p in parts])}
    out = {"a": torch.cat([p[0] for p in parts])}
    return dict(out, h=torch.cat([p[1] for p in parts])) if case["h"] else out
