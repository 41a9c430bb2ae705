"""The operators around a layer's routed experts, as cases to measure: the
norm in front of the layer, its routing with biased and grouped scores, and
the always-on expert in 8-bit integers (row quantisation, integer product,
SwiGLU).

Each case is one operator at one size; run(state) computes it in its plain
form (elementary torch operations), or, with `own` set, by the library's
entry point.  Codes of 8 bits are returned as the values they stand for, in
bf16 (code x scale of the row), next to the rows' scales.
"""
import functools
import math

import torch

own = False

# the hidden size, expert widths and expert counts of the benchmark's decode, coder and prefill layers are
# among the sizes below (H 2048; I 512 and 768; E 128 and 512 with k 8 and 10); the others are generic
ROUTE, NORM, SWIGLU, QUANT, MATMUL = "route", "norm", "swiglu", "quant", "matmul"
EPS = 1e-6


def listed():
    return [
        # one decode token of a layer of 512 experts: latency is all that counts
        dict(name="route_decode", op=ROUTE, T=1, E=512, k=10, score="sigmoid", bias=True, G=8, top=4, gtop=2,
             renorm=True, scale=2.5, L=0.125),
        # a prefill chunk, sigmoid scores with the balancing bias, half of the groups kept
        dict(name="route_chunk", op=ROUTE, T=4096, E=256, k=8, score="sigmoid", bias=True, G=8, top=4, gtop=2,
             renorm=True, scale=2.5, L=0.0),
        # the longest chunk: softmax scores, no groups, weights left as they are
        dict(name="route_long", op=ROUTE, T=16384, E=512, k=10, score="softmax", bias=False, G=1, top=1, gtop=1,
             renorm=False, scale=1.0, L=0.0),
        # one decode token: the previous layer's fp32 FFN output joins the bf16 residual stream
        dict(name="norm_decode", op=NORM, T=1, H=2048, h="bf16", delta="f32"),
        # a long prefill chunk of a wide model
        dict(name="norm_long", op=NORM, T=16384, H=4096, h="bf16", delta="bf16"),
        # a few decode requests at once through a shared expert of 768 columns
        dict(name="swiglu_batch", op=SWIGLU, T=6, I=768, gu="bf16"),
        # a prefill chunk of a wide shared expert, rows of an odd number of 8-column pieces
        dict(name="swiglu_chunk", op=SWIGLU, T=4000, I=8200, gu="bf16"),
        # a shared expert's gate and up rows when the model is loaded
        dict(name="quant_weights", op=QUANT, T=1536, H=2048, h="f32"),
        # a chunk of bf16 activations that come without a norm
        dict(name="quant_chunk", op=QUANT, T=8191, H=4096, h="bf16"),
        # one decode token against a shared expert's down projection, added to the routed experts' sum
        dict(name="matmul_decode", op=MATMUL, T=1, N=4096, K=8192, y="f32", add=True, row_w=True),
        # 48 decode requests, an odd number of outputs
        dict(name="matmul_batch", op=MATMUL, T=48, N=5003, K=2048, y="bf16", add=False, row_w=False),
        # a prefill chunk: arithmetic bounds it
        dict(name="matmul_chunk", op=MATMUL, T=4096, N=8192, K=4096, y="bf16", add=False, row_w=False),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice([ROUTE, NORM, SWIGLU, QUANT, MATMUL, MATMUL])
    if op == ROUTE:
        G = rng.choice([1, 1, 2, 4, 8])
        m = _log(rng, 8, 1024 // G)  # experts of a group
        E = G * m
        top = rng.randint(1, G)
        k = rng.randint(1, min(16, top * m))
        T = _log(rng, 1, min(16384, 16384 * 512 // E))
        return dict(op=op, T=T, E=E, k=k, score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.7, G=G,
                    top=top, gtop=rng.randint(1, 2), renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]),
                    L=rng.choice([0.0, 0.0, 0.125]))
    if op in (NORM, QUANT):
        H, h, delta = 8 * _log(rng, 2, 1024), rng.choice(["bf16", "f32"]), rng.choice(["none", "bf16", "f32"])
        wide = (h == "f32") + (op == NORM and delta == "f32")  # rows of fp32: fewer of them
        T = _log(rng, 1, min(16384, (16384 * 4096 if op == NORM else 8191 * 4096) // (H * (1 + wide))))
        return dict(op=op, T=T, H=H, h=h, **({"delta": delta} if op == NORM else {}))
    if op == SWIGLU:
        inner, gu = 8 * _log(rng, 2, 1536), rng.choice(["bf16", "f32"])
        return dict(op=op, T=_log(rng, 1, min(16384, 4000 * 8200 // (inner * (1 + (gu == "f32"))))), I=inner, gu=gu)
    K = 16 * _log(rng, 4, 512)
    N = _log(rng, 16, min(16384, 33554432 // K))
    T = _log(rng, 1, max(1, min(8192, 33554432 // N, 4096 * 8192 * 4096 // (N * K))))
    f32 = rng.random() < 0.5
    return dict(op=op, T=T, N=N, K=K, y="f32" if f32 else "bf16", add=f32 and rng.random() < 0.7,
                row_w=f32 and rng.random() < 0.5)


_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) & 0x7FFFFFFFFFFF)

    def rnd(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    def new(*shape, dt=torch.float32):
        return torch.empty(shape, device=dev, dtype=dt)

    s = {"case": c, "stream": torch.cuda.current_stream()}
    T, op = c["T"], c["op"]
    if op == ROUTE:
        E, k = c["E"], c["k"]
        # N(0, 1) scores over a popularity of the experts that falls off with their rank
        rank = torch.argsort(torch.rand(E, generator=g, device=dev)) + 1
        s["logits"] = rnd(T, E) - 0.6 * torch.log(rank.float())
        s["bias"] = 0.1 * rnd(E) if c["bias"] else None
        # three eighths of the experts resident
        slots = torch.argsort(torch.rand(E, generator=g, device=dev)).to(torch.int32)
        s["table"] = torch.where(slots < max(1, 3 * E // 8), slots, torch.full_like(slots, -1))
        s["ids"], s["w"] = new(T, k, dt=torch.int32), new(T, k)
    elif op in (NORM, QUANT):
        H = c["H"]
        s["h"] = rnd(T, H).to(_DT[c["h"]]) if op == NORM else (0.02 * rnd(T, H)).to(_DT[c["h"]])
        if op == NORM:
            s["delta"] = (0.5 * rnd(T, H)).to(_DT[c["delta"]]) if c["delta"] != "none" else None
            s["gamma"] = (1.0 + 0.2 * rnd(H)).to(torch.bfloat16)
            # with nothing to add the residual stream stays as it is
            s["h_out"] = new(T, H, dt=_DT[c["h"]]) if s["delta"] is not None else None
            s["x"] = new(T, H, dt=torch.bfloat16)
        s["q"], s["scale"], s["values"] = new(T, H, dt=torch.int8), new(T), new(T, H, dt=torch.bfloat16)
    elif op == SWIGLU:
        s["gu"] = rnd(T, 2 * c["I"]).to(_DT[c["gu"]])
        s["q"], s["scale"] = new(T, c["I"], dt=torch.int8), new(T)
        s["values"] = new(T, c["I"], dt=torch.bfloat16)
    else:
        N, K = c["N"], c["K"]
        s["xq"] = (32.0 * rnd(T, K)).round().clamp(-127, 127).to(torch.int8)
        s["wq"] = (32.0 * rnd(N, K)).round().clamp(-127, 127).to(torch.int8)
        s["xs"] = 0.02 + 0.01 * torch.rand(T, generator=g, device=dev)
        s["wsc"] = 0.0005 + 0.0005 * torch.rand(N, generator=g, device=dev)
        s["add"] = rnd(T, N) if c["add"] else None
        s["row_w"] = torch.rand(T, generator=g, device=dev) if c["row_w"] else None
        s["y"] = new(T, N, dt=_DT[c["y"]])
        s["err"] = torch.zeros(1, device=dev, dtype=torch.int32)
    return s


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
@functools.lru_cache(maxsize=None)
def _layer(E, k):
    from streamed_quantized_expert_b200 import ops
    return ops.desc(E, k, 64, 32, 32, 4)


@functools.lru_cache(maxsize=None)
def _routing(score, G, top, gtop, renorm, scale):
    from streamed_quantized_expert_b200 import ops
    return ops.route_config(score, G, top, gtop, renorm, scale)


def _run_own(s):
    from streamed_quantized_expert_b200 import ops
    c, st = s["case"], s["stream"]
    T, op = c["T"], c["op"]
    if op == ROUTE:
        ops.moe_route_grouped(s["logits"], T, _layer(c["E"], c["k"]),
                              _routing(c["score"], c["G"], c["top"], c["gtop"], c["renorm"], c["scale"]), s["bias"],
                              c["L"], s["table"], 0, None, s["ids"], s["w"], st)
        return {"ids": s["ids"], "w": s["w"]}
    if op == MATMUL:
        ops.moe_int_matmul(s["xq"], s["xs"], T, s["wq"], s["wsc"], c["N"], c["K"], s["add"], s["row_w"], s["y"],
                           ops.MOE_F32 if c["y"] == "f32" else ops.MOE_BF16, s["err"], st)
        return {"y": s["y"]}
    out = {"scale": s["scale"], "values": s["values"]}
    if op == NORM:
        ops.moe_add_norm_quant(s["h"], ops.MOE_F32 if c["h"] == "f32" else ops.MOE_BF16, s["delta"],
                               ops.MOE_F32 if c["delta"] == "f32" else ops.MOE_BF16, s["gamma"], EPS, T, c["H"],
                               s["h_out"], s["x"], s["q"], s["scale"], st)
        out["x"] = s["x"]
        if s["delta"] is not None:
            out["h"] = s["h_out"]
    elif op == QUANT:
        ops.moe_quantize_channels(s["h"], ops.MOE_F32 if c["h"] == "f32" else ops.MOE_BF16, T, c["H"], s["q"],
                                  s["scale"], st)
    else:
        ops.moe_swiglu_quant(s["gu"], ops.MOE_F32 if c["gu"] == "f32" else ops.MOE_BF16, T, c["I"], s["q"],
                             s["scale"], st)
    torch.mul(s["q"], s["scale"].unsqueeze(1), out=s["values"])  # the values the codes stand for
    return out


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _route_plain(s):
    """In 64 bits: the choice goes by differences between scores that 32 bits round away."""
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["G"]
    l = s["logits"].double()
    if c["score"] == "sigmoid":
        sc = 1.0 / (1.0 + torch.exp(-l))
    else:
        u = torch.exp(l - l.amax(dim=1, keepdim=True))
        sc = u / u.sum(dim=1, keepdim=True)
    key = sc if s["bias"] is None else sc + s["bias"].double()
    if c["L"] > 0:
        span = key.amax(dim=1, keepdim=True) - key.amin(dim=1, keepdim=True)
        key = torch.where(s["table"] >= 0, key + c["L"] * span, key)
    if c["top"] < G:
        best = torch.sort(key.view(T, G, E // G), dim=2, descending=True)[0][:, :, :c["gtop"]].sum(dim=2)
        order = torch.sort(best, dim=1, descending=True, stable=True)[1][:, :c["top"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter_(1, order, True)
        key = torch.where(keep.unsqueeze(2).expand(T, G, E // G).reshape(T, E), key, -math.inf)
    ids = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :k]
    w = torch.gather(sc, 1, ids)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return {"ids": ids.to(torch.int32), "w": (c["scale"] * w).float()}


def _quant_plain(p):
    """Codes of the rows of p (32 bits), and the rows' largest absolute values."""
    most = p.abs().amax(dim=1, keepdim=True)
    codes = torch.round(p / torch.where(most > 0, most, 1.0) * 127.0).to(torch.int8)
    return codes, most


def _run_plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == ROUTE:
        return _route_plain(s)
    if op == MATMUL:
        y = s["xq"].float() @ s["wq"].float().t()
        y = y * s["xs"].unsqueeze(1) * s["wsc"]
        if s["row_w"] is not None:
            y = y * s["row_w"].unsqueeze(1)
        if s["add"] is not None:
            y = y + s["add"]
        return {"y": y.to(_DT[c["y"]])}
    out = {}
    if op == NORM:
        h = s["h"].float()
        if s["delta"] is not None:
            out["h"] = (h + s["delta"].float()).to(_DT[c["h"]])
            h = out["h"].float()
        r = 1.0 / torch.sqrt(h.square().mean(dim=1, keepdim=True) + EPS)
        gamma = s["gamma"].float()
        out["x"] = (h * r * gamma).to(torch.bfloat16)
        codes, most = _quant_plain(h * gamma)
        scale = most * r / 127.0
    elif op == QUANT:
        codes, most = _quant_plain(s["h"].float())
        scale = most / 127.0
    else:
        a, b = s["gu"][:, :c["I"]].float(), s["gu"][:, c["I"]:].float()
        codes, most = _quant_plain(a / (1.0 + torch.exp(-a)) * b)
        scale = most / 127.0
    out["scale"], out["values"] = scale.squeeze(1), (codes.float() * scale).to(torch.bfloat16)
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------
# work, and the results in 64 bits
# ---------------------------------------------------------------------------
def work(case):
    c, T, op = case, case["T"], case["op"]
    size = {"bf16": 2, "f32": 4, "none": 0}
    if op == ROUTE:  # the logits once, ids and weights once; the scores' exponentials and comparisons
        return {"bytes": T * (4 * c["E"] + 8 * c["k"]) + (4 * c["E"] if c["bias"] else 0), "flops": 8 * T * c["E"]}
    if op == MATMUL:
        y = size[c["y"]] + (4 if c["add"] else 0)
        return {"bytes": (T + c["N"]) * (c["K"] + 4) + T * c["N"] * y, "flops": 2 * T * c["N"] * c["K"]}
    if op == NORM:  # both inputs, the new residual, x and the codes
        per = size[c["h"]] + size[c["delta"]] + (size[c["h"]] if c["delta"] != "none" else 0) + 2 + 1
        return {"bytes": T * (c["H"] * per + 4) + 2 * c["H"], "flops": 9 * T * c["H"]}
    if op == QUANT:
        return {"bytes": T * (c["H"] * (size[c["h"]] + 1) + 4), "flops": 3 * T * c["H"]}
    return {"bytes": T * (c["I"] * (2 * size[c["gu"]] + 1) + 4), "flops": 8 * T * c["I"]}


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op == ROUTE:
        import numpy as np
        l = s["logits"].cpu().numpy().astype(np.float64)
        T, E, G, k = c["T"], c["E"], c["G"], c["k"]
        if c["score"] == "sigmoid":
            sc = 0.5 + 0.5 * np.tanh(0.5 * l)
        else:
            top = l.max(axis=1, keepdims=True)
            sc = np.exp(l - (top + np.log(np.exp(l - top).sum(axis=1, keepdims=True))))
        key = sc.copy()
        if s["bias"] is not None:
            key += s["bias"].cpu().numpy().astype(np.float64)
        if c["L"] > 0:
            lift = c["L"] * np.ptp(key, axis=1)
            key += np.outer(lift, s["table"].cpu().numpy() >= 0)
        if c["top"] < G:
            parts = np.sort(key.reshape(T, G, -1), axis=2)[:, :, -c["gtop"]:].sum(axis=2)
            out = np.argsort(-parts, axis=1, kind="stable")[:, c["top"]:]
            key = key.reshape(T, G, -1)
            key[np.arange(T)[:, None], out] = -np.inf
            key = key.reshape(T, E)
        ids = np.argsort(-key, axis=1, kind="stable")[:, :k]
        w = np.take_along_axis(sc, ids, axis=1)
        if c["renorm"]:
            w = w / w.sum(axis=1, keepdims=True)
        return {"ids": None, "w": c["scale"] * w}
    if op == MATMUL:
        x = s["xq"].double() * s["xs"].double()[:, None]
        if s["row_w"] is not None:
            x = x * s["row_w"].double()[:, None]
        y = torch.matmul(x, (s["wq"].double() * s["wsc"].double()[:, None]).T)
        return {"y": y if s["add"] is None else y.add_(s["add"])}
    out = {}
    if op == NORM:
        h = s["h"].double()
        if s["delta"] is not None:
            # the residual stream is kept in its own type, and what is kept is what is normalised
            h = (h + s["delta"].double()).to(_DT[c["h"]]).double()
            out["h"] = h
        v = h * torch.rsqrt(torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / c["H"] + EPS) * s["gamma"].double()
        out["x"] = v
    elif op == QUANT:
        v = s["h"].double()
    else:
        v = torch.sigmoid(s["gu"][:, :c["I"]].double()) * s["gu"][:, :c["I"]].double() * s["gu"][:, c["I"]:].double()
    step = v.abs().max(dim=1).values / 127.0
    out["scale"] = step
    out["values"] = torch.round(v / step.clamp_min(1e-300)[:, None]) * step[:, None]
    return out
