"""Measured cases of the operators between a decoder layer's attention and
expert halves: the residual's addition with the root-mean-square norm and its
8-bit output, the matrix product with bias, activation and residual in its
epilogue, and routing to experts by softmax or sigmoid scores.

Each has a plain form in elementary torch operations (32 bits, rounded once at
the end; the router's scores in 64) and the call a user makes of the library;
``own`` says which of the two ``run`` takes.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
F8_MAX = 448.0                 # largest e4m3 value
EPS = 1e-6                     # of the RMS norm
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step: sum and norm in front of the experts, which take 8 bits, and the router, which takes bf16
        dict(name="norm decode", op="norm", T=64, H=7168, dtype="bf16", res="bf16", out=1, codes="f32", pad=0),
        # a prefill wave in front of an 8-bit projection
        dict(name="norm prefill", op="norm", T=16384, H=7168, dtype="bf16", res="bf16", out=0, codes="pow2", pad=0),
        # the norm of a part of each token's row, ragged batch, fp32, no residual
        dict(name="norm part f32", op="norm", T=1087, H=1536, dtype="f32", res="", out=1, codes="", pad=576),
        # one user's decode step: a query/key/value projection with bias for a single token
        dict(name="linear one", op="linear", T=1, N=10240, K=7168, dtype="bf16", out="bf16", act="none", bias=1, res=0),
        # a decode batch in 8 bits, first matrix of a dense block
        dict(name="linear decode e8m0", op="linear", T=64, N=18432, K=7168, dtype="e8m0", out="bf16", act="silu", bias=0,
             res=0),
        # the router's product over a prefill wave: few outputs, kept in fp32
        dict(name="linear router", op="linear", T=4096, N=256, K=7168, dtype="bf16", out="f32", act="none", bias=0, res=0),
        # a prefill wave's output projection onto the residual stream
        dict(name="linear prefill", op="linear", T=8192, N=7168, K=8192, dtype="bf16", out="bf16", act="none", bias=0,
             res=1),
        # the same in 8 bits with fp32 scales, a ragged wave into a dense block
        dict(name="linear prefill fp8", op="linear", T=4001, N=18432, K=7168, dtype="fp8", out="bf16", act="gelu_tanh",
             bias=1, res=0),
        # a small fp32 layer, everything in the epilogue
        dict(name="linear f32", op="linear", T=301, N=1536, K=512, dtype="f32", out="f32", act="gelu", bias=1, res=1),
        # one decode step's routing: softmax scores, balance bias, renormalised
        dict(name="route decode", op="route", B=128, N=256, K=8, score="softmax", group=1, keep=1, best=1, bias=1, renorm=1,
             dtype="f32", masked=0),
        # a prefill wave: groups ranked by their best expert, weights left as they are, odd expert count
        dict(name="route groups", op="route", B=16384, N=160, K=6, score="softmax", group=8, keep=3, best=1, bias=0, renorm=0,
             dtype="bf16", masked=0),
        # few experts, many tokens
        dict(name="route few", op="route", B=32768, N=8, K=2, score="softmax", group=1, keep=1, best=1, bias=0, renorm=1,
             dtype="f32", masked=0),
    ]


def _log_int(rng, lo, hi):
    """An int of [lo, hi], spread over the logarithm where that spans more than a factor of ten."""
    if hi <= 10 * max(lo, 1):
        return rng.randint(lo, hi)
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return min(hi, max(lo, int(v)))


def draw(rng):
    op = rng.choice(["norm", "linear", "linear", "route"])
    if op == "norm":
        codes = rng.choice(["", "f32", "pow2"])
        H = 128 * _log_int(rng, 1, 128) if codes else 8 * _log_int(rng, 1, 2048)
        return dict(op=op, T=_log_int(rng, 1, max(1, min(32768, 100_000_000 // H))), H=H, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    res=rng.choice(["", "bf16", "f32"]), out=1 if not codes else rng.randrange(2), codes=codes,
                    pad=rng.choice([0, 0, 8 * rng.randint(1, 200)]))
    if op == "linear":
        dtype = rng.choice(["bf16", "bf16", "fp8", "e8m0", "f32"])
        N, K = 16 * _log_int(rng, 1, 1152), 128 * _log_int(rng, 1, 144)
        T = _log_int(rng, 1, max(1, min(8192, (3 if dtype == "f32" else 400) * 1_000_000_000 // (N * K))))
        return dict(op=op, T=T, N=N, K=K, dtype=dtype, out="f32" if dtype == "f32" else rng.choice(["bf16", "bf16", "f32"]),
                    act=rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]), bias=rng.randrange(2), res=rng.randrange(2))
    group, each = rng.choice([1, 1, 2, 4, 8, 16]), _log_int(rng, 2, 64)
    if group == 1:
        each = _log_int(rng, 4, 1024)
    N = group * each
    keep = rng.randint(1, group)
    return dict(op=op, B=_log_int(rng, 1, 32768), N=N, K=rng.randint(1, min(10, keep * each)),
                score=rng.choice(["softmax", "sigmoid"]), group=group, keep=keep, best=rng.choice([1, 2]),
                bias=rng.randrange(2), renorm=rng.randrange(2), dtype=rng.choice(["f32", "bf16"]),
                masked=rng.choice([0, 0, each // 8]))


# ---------------------------------------------------------------- inputs
def _randn(gen, *shape):
    return torch.randn(*shape, device=DEV, generator=gen)


def _scale_of(amax, kind):
    """fp32 block scales of e4m3 codes: amax / 448, or the least power of two not below it; 1 for an empty block."""
    if kind == "pow2":
        mant, exp = torch.frexp(amax)                                  # amax = mant 2^exp, mant in [0.5, 1)
        s = torch.exp2((exp - 9 + (mant > 0.875)).float().clamp(-126, 127))
    else:
        s = amax / F8_MAX
    return torch.where(amax > 0, s, 1.0)


def _blocks(x, rows, kind):
    """e4m3 codes of x [n, k] and the scales of its rows x 128 blocks."""
    n, k = x.shape
    full = torch.zeros(-(-n // rows) * rows, k, device=DEV)
    full[:n] = x
    full = full.view(-1, rows, k // 128, 128)
    s = _scale_of(full.abs().amax((1, 3)), kind)
    q = (full / s[:, None, :, None]).clamp_(-F8_MAX, F8_MAX).to(torch.float8_e4m3fn)
    return q.view(-1, k)[:n].contiguous(), s


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case=case)
    {"norm": _prepare_norm, "linear": _prepare_linear, "route": _prepare_route}[case["op"]](case, gen, s)
    if own:
        import routing_dispatch_grouped_amd as rdg
        s["rdg"] = rdg
        _prepare_own(case, s, rdg)
    return s


def _prepare_norm(case, gen, s):
    T, H = case["T"], case["H"]
    # activations with a few strong channels, as a residual stream has them
    gain = torch.exp(0.7 * _randn(gen, 1, H + case["pad"]))
    s["x"] = (_randn(gen, T, H + case["pad"]) * gain).to(DTYPES[case["dtype"]])[:, :H]
    s["res"] = (3 * _randn(gen, T, H) * gain[:, :H]).to(DTYPES[case["res"]]) if case["res"] else None
    s["w"] = 1 + 0.2 * _randn(gen, H)


def _prepare_linear(case, gen, s):
    T, N, K, dtype = case["T"], case["N"], case["K"], case["dtype"]
    x = _randn(gen, T, K) * torch.exp(0.7 * _randn(gen, 1, K))
    w = _randn(gen, N, K) * K ** -0.5
    if dtype in DTYPES:
        s["x"], s["W"], s["xs"], s["Ws"] = x.to(DTYPES[dtype]), w.to(DTYPES[dtype]), None, None
    else:
        kind = "pow2" if dtype == "e8m0" else "f32"
        s["x"], s["xs"] = _blocks(x, 1, kind)
        s["W"], s["Ws"] = _blocks(w, 128, kind)
    s["bias"] = 0.3 * _randn(gen, N) if case["bias"] else None
    s["res"] = (2 * _randn(gen, T, N)).to(DTYPES[case["out"]]) if case["res"] else None


def _prepare_route(case, gen, s):
    logits = 1.5 * _randn(gen, case["B"], case["N"]) + 0.7 * _randn(gen, 1, case["N"])
    # experts that are switched off
    logits[:, torch.randperm(case["N"], device=DEV, generator=gen)[:case["masked"]]] = -math.inf
    s["logits"] = logits.to(DTYPES[case["dtype"]])
    s["bias"] = 0.05 * _randn(gen, case["N"]) if case["bias"] else None


def _prepare_own(case, s, rdg):
    """The outputs and laid-out weights that a program keeps from call to call."""
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        s["out"] = torch.empty(T, H, dtype=s["x"].dtype, device=DEV) if case["out"] else None
        s["res_out"] = torch.empty_like(s["res"]) if case["res"] else None
        s["q"] = torch.empty(T, H, dtype=torch.uint8, device=DEV) if case["codes"] else None
        s["qs"] = torch.empty(T, H // 128, device=DEV) if case["codes"] else None
        s["kind"] = rdg.RDG_FP8_E4M3_UE8M0 if case["codes"] == "pow2" else rdg.RDG_FP8_E4M3
    elif case["op"] == "linear":
        T, N, K = case["T"], case["N"], case["K"]
        s["kind"] = dict(bf16=rdg.RDG_BF16, f32=rdg.RDG_F32, fp8=rdg.RDG_FP8_E4M3, e8m0=rdg.RDG_FP8_E4M3_UE8M0)[case["dtype"]]
        s["act"] = dict(none=rdg.RDG_ACT_NONE, relu=rdg.RDG_ACT_RELU, silu=rdg.RDG_ACT_SILU, gelu=rdg.RDG_ACT_GELU,
                        gelu_tanh=rdg.RDG_ACT_GELU_TANH)[case["act"]]
        s["packed"] = torch.empty_like(s["W"])
        rdg.rdg_pack_weights(s["W"], s["kind"], s["packed"])
        s["out"] = torch.empty(T, N, dtype=DTYPES[case["out"]], device=DEV)
        s["work"] = torch.empty(rdg.rdg_linear_workspace_bytes(T, N, K, s["kind"]), dtype=torch.uint8, device=DEV)
    else:
        s["ids"] = torch.empty(case["B"], case["K"], dtype=torch.int32, device=DEV)
        s["topk_w"] = torch.empty(case["B"], case["K"], device=DEV)
        s["kind"] = rdg.RDG_SCORE_SOFTMAX if case["score"] == "softmax" else rdg.RDG_SCORE_SIGMOID


# ---------------------------------------------------------------- one pass
def run(s):
    return {"norm": _norm, "linear": _linear, "route": _route}[s["case"]["op"]](s)


def _norm(s):
    c = s["case"]
    if own:
        s["rdg"].rdg_add_norm(s["x"], s["w"], EPS, out=s["out"], residual=s["res"], residual_out=s["res_out"], q=s["q"],
                              q_scales=s["qs"], q_dtype=s["kind"])
        return dict(out=s["out"], res=s["res_out"], q=None if s["q"] is None else s["q"].view(torch.float8_e4m3fn),
                    qs=s["qs"])
    x = s["x"].float()
    got = dict(out=None, res=None, q=None, qs=None)
    if c["res"]:
        x = x + s["res"].float()
        got["res"] = x.to(s["res"].dtype)
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["w"]
    if c["out"]:
        got["out"] = y.to(s["x"].dtype)
    if c["codes"]:
        y = y.view(c["T"], -1, 128)
        got["qs"] = _scale_of(y.abs().amax(-1), c["codes"])
        q = (y / got["qs"][..., None]).clamp(-F8_MAX, F8_MAX).to(torch.float8_e4m3fn)
        got["q"] = q.view(c["T"], -1)
    return got


def _linear(s):
    c = s["case"]
    if own:
        s["rdg"].rdg_linear(s["x"], s["xs"], s["kind"], s["packed"], s["Ws"], s["out"], bias=s["bias"], act=s["act"],
                            residual=s["res"], work=s["work"])
        return s["out"]
    x, w = s["x"].float(), s["W"].float()
    if s["xs"] is not None:
        x = (x.view(c["T"], -1, 128) * s["xs"].view(c["T"], -1, 1)).view(c["T"], -1)
        # scales of 128 x 128 blocks, spread over their rows
        w = (w.view(c["N"], -1, 128) * s["Ws"].repeat_interleave(128, 0)[:c["N"], :, None]).view(c["N"], -1)
    y = x @ w.T
    if s["bias"] is not None:
        y = y + s["bias"]
    if c["act"] == "relu":
        y = y.clamp(min=0)
    elif c["act"] == "silu":
        y = y / (1 + torch.exp(-y))
    elif c["act"] == "gelu":
        y = 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    elif c["act"] == "gelu_tanh":
        y = 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    if s["res"] is not None:
        y = y + s["res"].float()
    return y.to(DTYPES[c["out"]])


def _route(s):
    c = s["case"]
    if own:
        s["rdg"].rdg_route_topk(s["logits"], s["kind"], c["group"], c["keep"], c["best"], c["K"], c["renorm"], 2.5, s["ids"],
                                s["topk_w"], bias=s["bias"])
        return dict(ids=s["ids"], w=s["topk_w"])
    x = s["logits"].double()
    if c["score"] == "softmax":
        e = torch.exp(x - x.amax(-1, keepdim=True))
        p = (e / e.sum(-1, keepdim=True)).float()
    else:
        p = (1 / (1 + torch.exp(-x.clamp(-87, 87)))).float()
    choice = p if s["bias"] is None else p + s["bias"]
    if c["group"] > 1:
        g = choice.view(c["B"], c["group"], -1)
        rank = g.amax(-1) if c["best"] == 1 else g.topk(2, -1).values.sum(-1)
        kept = torch.sort(rank, dim=-1, descending=True, stable=True).indices[:, :c["keep"]]
        out = torch.ones(c["B"], c["group"], dtype=torch.bool, device=DEV).scatter_(1, kept, False)
        choice = g.masked_fill(out[..., None], -math.inf).view(c["B"], -1)
    ids = torch.sort(choice, dim=-1, descending=True, stable=True).indices[:, :c["K"]]
    w = p.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return dict(ids=ids.int(), w=w * 2.5)


# ---------------------------------------------------------------- work of one pass
def work(case):
    size = dict(bf16=2, f32=4, fp8=1, e8m0=1)
    if case["op"] == "norm":
        n = case["T"] * case["H"]
        e = size[case["dtype"]]
        per = e + (2 * size[case["res"]] if case["res"] else 0) + (e if case["out"] else 0)
        return dict(bytes=n * per + (n + n // 32 if case["codes"] else 0) + 4 * case["H"], flops=n * (5 + 3 * bool(case["codes"])))
    if case["op"] == "linear":
        T, N, K, e = case["T"], case["N"], case["K"], size[case["dtype"]]
        scales = (T + -(-N // 128)) * (K // 128) * 4 if case["dtype"] in ("fp8", "e8m0") else 0
        return dict(bytes=(T + N) * K * e + scales + T * N * size[case["out"]] * (1 + case["res"]) + 4 * N * case["bias"],
                    flops=2 * T * N * K)
    B, N, K = case["B"], case["N"], case["K"]
    return dict(bytes=B * N * size[case["dtype"]] + 8 * B * K + 4 * N * case["bias"], flops=B * N * (30 + K))


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "linear": _exact_linear, "route": _exact_route}[case["op"]](case, s)


def _exact_norm(c, s):
    total = s["x"].double()
    if c["res"]:
        total = total + s["res"].double()
    length = torch.sqrt((total ** 2).sum(1) / c["H"] + EPS)
    y = total / length[:, None] * s["w"].double()[None]
    got = dict(out=y if c["out"] else None, res=total if c["res"] else None, q=None, qs=None)
    if c["codes"]:
        top = y.abs().reshape(c["T"], -1, 128).max(2).values / F8_MAX
        got["qs"] = top if c["codes"] == "f32" else torch.exp2(torch.ceil(torch.log2(top)))
        got["q"] = y / got["qs"].repeat_interleave(128, 1)
    return got


def _exact_linear(c, s):
    a, b = s["x"].double(), s["W"].double()
    if s["xs"] is not None:
        a = a * s["xs"].double().view(c["T"], -1).repeat_interleave(128, 1)
        b = b * s["Ws"].double().repeat_interleave(128, 1).repeat_interleave(128, 0)[:c["N"]]
    z = torch.zeros(c["T"], c["N"], dtype=torch.float64, device=DEV)
    if s["bias"] is not None:
        z += s["bias"].double()
    z.addmm_(a, b.t())
    if c["act"] == "relu":
        z = torch.maximum(z, torch.zeros_like(z))
    elif c["act"] == "silu":
        z = z * torch.sigmoid(z)
    elif c["act"] == "gelu":
        z = z * 0.5 * torch.erfc(-z / math.sqrt(2))
    elif c["act"] == "gelu_tanh":
        z = z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))
    return z if s["res"] is None else z + s["res"].double()


def _exact_route(c, s):
    x = s["logits"].double().cpu().numpy()
    if c["score"] == "softmax":
        p = np.exp(x - np.logaddexp.reduce(x, axis=1, keepdims=True))
    else:
        p = np.reciprocal(1.0 + np.exp(-np.clip(x, -87.0, 87.0)))
    # scores count as rounded to 32 bits where they are compared
    choice = p.astype(np.float32)
    if s["bias"] is not None:
        choice = choice + s["bias"].cpu().numpy()
    if c["group"] > 1:
        g = np.sort(choice.reshape(c["B"], c["group"], -1), axis=2)
        rank = g[..., -1] if c["best"] == 1 else g[..., -1] + g[..., -2]
        order = np.argsort(-rank, axis=1, kind="stable")
        place = np.argsort(order, axis=1, kind="stable")             # of each group
        choice = np.where(np.repeat(place < c["keep"], c["N"] // c["group"], axis=1), choice, -np.inf)
    ids = np.argsort(-choice, axis=1, kind="stable")[:, :c["K"]]
    w = np.take_along_axis(p, ids, axis=1)
    if c["renorm"]:
        w = w / w.sum(1, keepdims=True)
    return dict(ids=torch.from_numpy(ids.astype(np.int32)), w=torch.from_numpy(2.5 * w))
