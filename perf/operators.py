"""Operators around the MoE layer, as cases to be timed and compared.

A serving step of a W8A8 model runs, next to the MoE layer itself, three kinds
of operator that this file describes in elementary form:

``linear``       y = dequant(quant(x / s) Wq^T) + b: the dense products of the
                 model (attention projections, the LM head) in 8-bit integers,
                 one scale per token and one per output channel.  From float
                 activations (``codes`` false) or from codes that a producer
                 has already formed (``codes`` true).
``norm``         the RMS norms after and before a block with what lies between
                 them: r = a x + c g * norm(b), n = norm(r), and the 8-bit
                 codes of n for the next product.
``norm_linear``  the two together, as a decode step runs them: the norm writes
                 codes and scales, the product reads them.
``sample``       the next token of each row of logits from given random
                 numbers, with temperature, top-k, top-p and min-p.

Where ``own`` is false, ``run`` computes them with elementary torch operations;
where it is true, with the library's entry points.
"""
import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of one user: the output projection of an attention block
        dict(name="linear token", op="linear", T=1, K=4096, N=4096, inp="bf16", out="bf16", bias=False, smooth=True,
             codes=False),
        # a decode batch of 32 users: the joined query, key and value projection with grouped heads
        dict(name="linear decode", op="linear", T=32, K=4096, N=6144, inp="bf16", out="bf16", bias=True, smooth=True,
             codes=False),
        # the LM head of a decode batch: a vocabulary of 32000 and logits in fp32
        dict(name="linear head", op="linear", T=64, K=4096, N=32000, inp="bf16", out="f32", bias=False, smooth=False,
             codes=False),
        # ragged sizes: a short prompt through a small adapter whose sizes divide by nothing
        dict(name="linear ragged", op="linear", T=517, K=1000, N=1111, inp="f32", out="f32", bias=True, smooth=True,
             codes=True),
        # prefill of 32 prompts of 512 tokens through an attention projection of twice the hidden size
        dict(name="linear prefill", op="linear", T=16384, K=4096, N=8192, inp="bf16", out="bf16", bias=False,
             smooth=True, codes=False),
        # decode of one token: residual add, norm, codes, and the projection that reads them
        dict(name="norm linear token", op="norm_linear", T=1, K=4096, N=6144, inp="bf16", out="bf16"),
        # ragged sizes in fp32: a token gate (a shared expert's) and codes for the next product
        dict(name="norm ragged", op="norm", T=777, d=1001, stream="f32", out="f32", post=True, gate="token", sigmoid=True,
             codes=True),
        # a prompt of 4096 tokens: norms on both sides of a block and a learnt scale per channel
        dict(name="norm prefill", op="norm", T=4096, d=4096, stream="bf16", out="bf16", post=True, gate="channel",
             sigmoid=False, codes=False),
        # prefill of 32 x 512 tokens at the large hidden size: residual add and norm before a block
        dict(name="norm large", op="norm", T=16384, d=8192, stream="bf16", out="bf16", post=False, gate="none",
             sigmoid=False, codes=False),
        # one user, a vocabulary of 32000, the usual top-k and top-p
        dict(name="sample one", op="sample", T=1, V=32000, inp="f32", peak=18.0, top_k=50, top_p=0.95, min_p=0.0,
             greedy=False, mask=False),
        # 64 users with settings of their own, some greedy, bf16 logits (many equal ones), part of the tokens allowed
        dict(name="sample mixed", op="sample", T=64, V=131072, inp="bf16", peak=17.0, top_k=200, top_p=0.9, min_p=0.02,
             greedy=True, mask=True),
        # a full decode batch, top-p alone: every token's probability counts
        dict(name="sample batch", op="sample", T=256, V=131072, inp="f32", peak=15.0, top_k=0, top_p=0.95, min_p=0.0,
             greedy=False, mask=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("linear", "linear", "norm", "norm", "norm_linear", "sample", "sample"))
    typ = lambda: rng.choice(("bf16", "bf16", "f32"))  # noqa: E731
    if op == "linear":
        T, K, N = _log(rng, 1, 16384), _log(rng, 64, 8192), _log(rng, 64, 65536)
        while T * K * N > 16384 * 4096 * 8192 or T * N > 16384 * 8192:
            T = max(1, T // 2)
        return dict(op=op, T=T, K=K, N=N, inp=typ(), out=typ(), bias=rng.random() < 0.5, smooth=rng.random() < 0.5,
                    codes=rng.random() < 0.4)
    if op == "norm_linear":
        return dict(op=op, T=_log(rng, 1, 512), K=_log(rng, 64, 8192), N=_log(rng, 64, 16384), inp=typ(), out=typ())
    if op == "norm":
        T, d = _log(rng, 1, 16384), _log(rng, 64, 16384)
        while T * d > 16384 * 8192:
            T = max(1, T // 2)
        return dict(op=op, T=T, d=d, stream=typ(), out=typ(), post=rng.random() < 0.5,
                    gate=rng.choice(("none", "token", "channel", "element")), sigmoid=rng.random() < 0.5,
                    codes=rng.random() < 0.4)
    T, V = _log(rng, 1, 256), _log(rng, 1000, 262144)
    while T * V > 256 * 131072:
        T = max(1, T // 2)
    return dict(op=op, T=T, V=V, inp=typ(), peak=round(rng.uniform(8.0, 20.0), 2),
                top_k=rng.choice((0, 0, _log(rng, 1, 2000))), top_p=rng.choice((1.0, round(rng.uniform(0.3, 0.999), 3))),
                min_p=rng.choice((0.0, 0.0, round(rng.uniform(0.001, 0.2), 4))), greedy=rng.random() < 0.3,
                mask=rng.random() < 0.3)


def work(case):
    """Each input read once, each output written once; the arithmetic of the formulas."""
    op, T = case["op"], case["T"]
    size = {"f32": 4, "bf16": 2}
    if op in ("linear", "norm_linear"):
        K, N = case["K"], case["N"]
        b = N * K + 4 * N + T * N * size[case["out"]]
        if op == "norm_linear":
            b += 3 * T * K * size[case["inp"]] + 4 * K
        elif case["codes"]:
            b += T * K + 4 * T
        else:
            b += T * K * size[case["inp"]]
        return {"bytes": b, "flops": 2 * T * N * K}
    if op == "norm":
        n = T * case["d"]
        b = 3 * n * size[case["stream"]] + n * size[case["out"]] + (n + 4 * T if case["codes"] else 0)
        b += n * size[case["stream"]] if case["gate"] == "element" else 0
        return {"bytes": b, "flops": 12 * n}
    n = T * case["V"]
    return {"bytes": n * size[case["inp"]] + (T * case["V"] // 8 if case["mask"] else 0) + 32 * T, "flops": 4 * n}


# ------------------------------------------------------------------ inputs

def _pad16(n):
    return (n + 15) // 16 * 16


def _activations(g, T, d, dtype):
    """Hidden states: about unit scale, a few channels that are an order of magnitude larger."""
    x = torch.randn(T, d, generator=g, device="cuda")
    big = torch.randint(0, d, (max(1, d // 256),), generator=g, device="cuda")
    x[:, big] *= 12.0
    return x.to(dtype)


def _weights(g, N, K):
    """Codes and scales of a product of N channels over K inputs, and its smoothing."""
    wq = (torch.randn(N, K, generator=g, device="cuda") * 32).round_().clamp_(-127, 127).to(torch.int8)
    sw = (torch.rand(N, generator=g, device="cuda") + 0.5) / (32 * math.sqrt(K))
    inv_s = torch.rand(K, generator=g, device="cuda") + 0.5
    return wq, sw, inv_s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case=case)
    op, T = case["op"], case["T"]
    if op == "linear":
        K, N = case["K"], case["N"]
        s["wq"], s["sw"], inv_s = _weights(g, N, K)
        s["inv_s"] = inv_s if case["smooth"] and not case["codes"] else None
        s["bias"] = torch.randn(N, generator=g, device="cuda") * 0.1 if case["bias"] else None
        if case["codes"]:
            s["xq"] = torch.zeros(T, _pad16(K), dtype=torch.int8, device="cuda")
            s["xq"][:, :K] = (torch.randn(T, K, generator=g, device="cuda") * 36).round_().clamp_(-127, 127).to(torch.int8)
            s["sx"] = (torch.rand(T, generator=g, device="cuda") + 0.5) / 36
        else:
            s["x"] = _activations(g, T, K, DT[case["inp"]])
        s["y"] = torch.empty(T, N, dtype=DT[case["out"]], device="cuda")
    elif op == "norm_linear":
        K, N = case["K"], case["N"]
        dt = DT[case["inp"]]
        s["wq"], s["sw"], s["inv_s"] = _weights(g, N, K)
        s["b"], s["x"] = _activations(g, T, K, dt), (torch.randn(T, K, generator=g, device="cuda") * 3).to(dt)
        s["w_pre"] = torch.rand(K, generator=g, device="cuda") + 0.5
        s["x_out"] = torch.empty_like(s["x"])
        s["xq"] = torch.zeros(T, _pad16(K), dtype=torch.int8, device="cuda")
        s["sx"] = torch.empty(T, device="cuda")
        s["y"] = torch.empty(T, N, dtype=DT[case["out"]], device="cuda")
    elif op == "norm":
        d, dt = case["d"], DT[case["stream"]]
        s["b"], s["x"] = _activations(g, T, d, dt), (torch.randn(T, d, generator=g, device="cuda") * 3).to(dt)
        s["w_pre"] = torch.rand(d, generator=g, device="cuda") + 0.5
        s["w_post"] = torch.rand(d, generator=g, device="cuda") + 0.5 if case["post"] else None
        gate = {"none": None, "token": (T,), "channel": (d,), "element": (T, d)}[case["gate"]]
        s["gate"] = None if gate is None else torch.randn(gate, generator=g, device="cuda")
        if case["gate"] == "element":
            s["gate"] = s["gate"].to(dt)
        s["inv_s"] = torch.rand(d, generator=g, device="cuda") + 0.5
        s["x_out"], s["n_out"] = torch.empty_like(s["x"]), torch.empty(T, d, dtype=DT[case["out"]], device="cuda")
        s["xq"] = torch.zeros(T, _pad16(d), dtype=torch.int8, device="cuda") if case["codes"] else None
        s["sx"] = torch.empty(T, device="cuda") if case["codes"] else None
    else:
        V = case["V"]
        # a broad tail and a head whose probabilities fall as a power of the rank
        x = torch.randn(T, V, generator=g, device="cuda") * 1.5
        n = min(V // 4, 400)
        at = torch.randint(0, V // n, (T, n), generator=g, device="cuda") + torch.arange(n, device="cuda") * (V // n)
        rank = torch.rand(T, n, generator=g, device="cuda").argsort(1) + 1.0
        head = case["peak"] - 1.5 * torch.log(rank) + 0.3 * torch.randn(T, n, generator=g, device="cuda")
        s["logits"] = x.scatter_(1, at, head).to(DT[case["inp"]])
        r = lambda: torch.rand(T, generator=g, device="cuda")  # noqa: E731
        s["u"] = r()
        s["temperature"] = 0.6 + 0.6 * r()
        if case["greedy"]:
            s["temperature"][torch.arange(T, device="cuda") % 8 == 3] = 0.0
        s["top_k"] = (case["top_k"] * (0.5 + r())).to(torch.int32).clamp_(min=1) if case["top_k"] else None
        s["top_p"] = (case["top_p"] * (0.9 + 0.1 * r())) if case["top_p"] < 1.0 else None
        s["min_p"] = (case["min_p"] * (0.5 + r())) if case["min_p"] > 0.0 else None
        # bit i of word j of a row: token 32 j + i may be chosen
        words = (V + 31) // 32
        s["allowed"] = torch.randint(-2 ** 31, 2 ** 31, (T, words), generator=g, device="cuda",
                                     dtype=torch.int64).to(torch.int32) if case["mask"] else None
        s["token"] = torch.empty(T, dtype=torch.int32, device="cuda")
        s["prob"] = torch.empty(T, dtype=torch.float32, device="cuda")
    if own:
        _keep(s)
    return s


def _keep(s):
    """What a program that uses the library keeps besides its inputs: handles, workspaces, settings."""
    import w8a8_quantized_moe_b200 as M
    c = s["case"]
    code = {"f32": M.MOE_F32, "bf16": M.MOE_BF16}
    s["M"] = M
    if c["op"] in ("linear", "norm_linear"):
        cfg = M.make_linear_config(c["N"], c["K"], in_dtype=code[c["inp"]], out_dtype=code[c["out"]])
        s["lin"] = M.moe_w8a8_linear_prepare_codes(cfg, s["wq"], s["sw"], s.get("bias"), s["inv_s"])
        size = M.moe_w8a8_linear_workspace_size(s["lin"], c["T"])
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    if c["op"] == "norm_linear":
        s["cfg"] = M.make_norm_config(c["K"], in_dtype=code[c["inp"]], res_dtype=code[c["inp"]],
                                      out_dtype=code[c["inp"]])
    if c["op"] == "norm":
        gate = {"none": M.MOE_GATE_NONE, "token": M.MOE_GATE_TOKEN, "channel": M.MOE_GATE_CHANNEL,
                "element": M.MOE_GATE_ELEMENT}[c["gate"]]
        s["cfg"] = M.make_norm_config(c["d"], in_dtype=code[c["stream"]], res_dtype=code[c["stream"]],
                                      out_dtype=code[c["out"]], gate=gate, gate_sigmoid=c["sigmoid"], eps=1e-6,
                                      residual_scale=0.9, branch_scale=1.25)


# ------------------------------------------------------------------ the plain forms

def _quantize(v):
    """Codes (as fp32 whole numbers) and scales of rows: scale = amax / 127, codes rint(v / scale)."""
    amax = v.abs().amax(1, keepdim=True)
    scale = amax / torch.full_like(amax, 127.0)
    codes = torch.where(scale > 0, torch.round(v / scale), torch.zeros_like(v)).clamp(-127, 127)
    return codes, scale


def _product(codes, wq):
    """Exact sums of products of codes: 1024 products of at most 127^2 stay below 2^24."""
    pad = -codes.shape[1] % 1024
    a = torch.nn.functional.pad(codes, (0, pad)).reshape(codes.shape[0], -1, 1024).transpose(0, 1)
    b = torch.nn.functional.pad(wq.float(), (0, pad)).reshape(wq.shape[0], -1, 1024).permute(1, 2, 0)
    return torch.matmul(a, b).sum(0, dtype=torch.float64).float()


def _linear(s, codes, scale, out):
    y = _product(codes, s["wq"]) * scale * s["sw"]
    if s.get("bias") is not None:
        y = y + s["bias"]
    return y.to(out)


def _rms(v, w):
    return v * torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-6) * w


def _block(s, residual_scale, branch_scale):
    """r (rounded to the stream's type, as it is kept) in fp32."""
    c = s["case"]
    p = s["b"].float()
    if s.get("w_post") is not None:
        p = _rms(p, s["w_post"])
    g = s.get("gate")
    if g is not None:
        g = g.float()
        g = torch.sigmoid(g) if c["sigmoid"] else g
        p = p * (g[:, None] if c["gate"] == "token" else g)
    return (residual_scale * s["x"].float() + branch_scale * p).to(s["x"].dtype)


def _norm_codes(r, w, inv_s):
    """Codes of norm(r) w inv_s: the row's rms cancels in v / scale, so it enters the scale alone."""
    codes, scale = _quantize(r * w * inv_s)
    return codes, scale * torch.rsqrt((r * r).mean(1, keepdim=True) + 1e-6)


def _sample(s):
    c = s["case"]
    l = s["logits"].double()
    T, V = l.shape
    low = torch.full_like(l, -math.inf)
    l = torch.where(torch.isnan(l), low, l)
    if s["allowed"] is not None:
        i = torch.arange(V, device=l.device)
        l = torch.where((s["allowed"][:, i // 32] >> (i % 32)) & 1 != 0, l, low)
    l, order = torch.sort(l, dim=1, descending=True, stable=True)
    t = s["temperature"].double()[:, None]
    greedy = t <= 0
    e = torch.exp((l - l[:, :1]) / torch.where(greedy, torch.ones_like(t), t))
    rank = torch.arange(V, device=l.device)[None]
    keep = torch.isfinite(l)
    if s["top_k"] is not None:
        k = s["top_k"][:, None]
        keep &= (rank < k) | (k <= 0)
    keep &= ~greedy | (rank == 0)
    e = torch.where(keep, e, torch.zeros_like(e))
    if s["top_p"] is not None:
        before = torch.cumsum(e, 1) - e
        keep &= (rank == 0) | (before < s["top_p"].double()[:, None] * e.sum(1, keepdim=True))
    if s["min_p"] is not None:
        keep &= (rank == 0) | (e >= s["min_p"].double()[:, None])
    e = torch.where(keep, e, torch.zeros_like(e))
    p = torch.zeros_like(e).scatter_(1, order, e)          # in the order of the tokens
    cum = torch.cumsum(p, 1)
    total = cum[:, -1:]
    token = (cum <= s["u"].double()[:, None] * total).sum(1, keepdim=True).clamp(max=V - 1)
    prob = p.gather(1, token) / total
    some = total > 0
    s["token"].copy_(torch.where(some, token, torch.full_like(token, -1))[:, 0])
    s["prob"].copy_(torch.where(some, prob, torch.zeros_like(prob))[:, 0])
    return s["token"], s["prob"]


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        return _own(s)
    if op == "linear":
        if c["codes"]:
            return _linear(s, s["xq"][:, :c["K"]].float(), s["sx"][:, None], s["y"].dtype)
        v = s["x"].float()
        codes, scale = _quantize(v if s["inv_s"] is None else v * s["inv_s"])
        return _linear(s, codes, scale, s["y"].dtype)
    if op == "norm_linear":
        r = _block(s, 1.0, 1.0)
        codes, scale = _norm_codes(r.float(), s["w_pre"], s["inv_s"])
        return r, _linear(s, codes, scale, s["y"].dtype)
    if op == "norm":
        r = _block(s, 0.9, 1.25)
        out = [r, _rms(r.float(), s["w_pre"]).to(s["n_out"].dtype)]
        if c["codes"]:
            codes, scale = _norm_codes(r.float(), s["w_pre"], s["inv_s"])
            out += [(codes * scale).to(torch.bfloat16), scale[:, 0]]
        return out
    return _sample(s)


def _own(s):
    c, M = s["case"], s["M"]
    op = c["op"]
    if op == "linear":
        if c["codes"]:
            M.moe_w8a8_linear_forward_codes(s["lin"], s["xq"], s["sx"], c["T"], s["y"])
        else:
            M.moe_w8a8_linear_forward(s["lin"], s["x"], c["T"], s["y"], s["workspace"])
        return s["y"]
    if op == "norm_linear":
        M.moe_w8a8_block_norm(s["cfg"], c["T"], b=s["b"], x=s["x"], w_pre=s["w_pre"], inv_s=s["inv_s"],
                              x_out=s["x_out"], xq=s["xq"], sx=s["sx"])
        M.moe_w8a8_linear_forward_codes(s["lin"], s["xq"], s["sx"], c["T"], s["y"])
        return s["x_out"], s["y"]
    if op == "norm":
        M.moe_w8a8_block_norm(s["cfg"], c["T"], b=s["b"], x=s["x"], gate=s["gate"], w_post=s["w_post"],
                              w_pre=s["w_pre"], inv_s=s["inv_s"] if c["codes"] else None, x_out=s["x_out"],
                              n_out=s["n_out"], xq=s["xq"], sx=s["sx"])
        out = [s["x_out"], s["n_out"]]
        if c["codes"]:
            out += [(s["xq"][:, :c["d"]] * s["sx"][:, None]).to(torch.bfloat16), s["sx"]]
        return out
    M.moe_w8a8_sample(s["logits"], s["u"], s["token"], temperature=s["temperature"], top_k=s["top_k"],
                      top_p=s["top_p"], min_p=s["min_p"], allowed=s["allowed"], prob=s["prob"])
    return s["token"], s["prob"]


# ------------------------------------------------------------------ the definitions in 64 bits

def _codes64(v32):
    """The codes' definition, whose steps are single roundings to fp32 (a product, quotient or conversion of fp32
    numbers formed in 64 bits and rounded once is that step)."""
    v = v32.double()
    scale = (v.abs().max(1, keepdim=True).values / 127.0).float().double()
    q = (v / scale.clamp(min=1e-300)).float().double().round()
    return torch.where(scale > 0, q, torch.zeros_like(q)).clamp(-127, 127), scale


def _exact_norm(s, residual_scale, branch_scale):
    c = s["case"]
    p = s["b"].double()
    if s.get("w_post") is not None:
        p = p / torch.sqrt((p ** 2).mean(1, keepdim=True) + 1e-6) * s["w_post"].double()
    g = s.get("gate")
    if g is not None:
        g = g.double()
        g = 1.0 / (1.0 + torch.exp(-g)) if c["sigmoid"] else g
        p = p * (g.unsqueeze(1) if c["gate"] == "token" else g)
    r = residual_scale * s["x"].double() + branch_scale * p
    return r, r.to(s["x"].dtype).double()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "sample":
        return _exact_sample(s)
    bias = s["bias"].double() if s.get("bias") is not None else 0.0
    if op == "linear":
        if case["codes"]:
            q, scale = s["xq"][:, :case["K"]].double(), s["sx"].double().unsqueeze(1)
        else:
            v = s["x"].double()
            q, scale = _codes64(v.float() if s["inv_s"] is None else (v * s["inv_s"].double()).float())
        return (q @ s["wq"].double().T) * scale * s["sw"].double() + bias
    r, kept = _exact_norm(s, 0.9 if op == "norm" else 1.0, 1.25 if op == "norm" else 1.0)
    inv_rms = 1.0 / torch.sqrt((kept ** 2).mean(1, keepdim=True) + 1e-6)
    q, scale = _codes64(((kept * s["w_pre"].double()).float().double() * s["inv_s"].double()).float())
    if op == "norm_linear":
        return r, (q @ s["wq"].double().T) * (scale * inv_rms) * s["sw"].double()
    out = [r, kept * inv_rms * s["w_pre"].double()]
    if case["codes"]:
        out += [q * scale * inv_rms, (scale * inv_rms)[:, 0]]
    return out


def _exact_sample(s):
    l = s["logits"].double().cpu().numpy()
    T, V = l.shape
    get = lambda k: None if s[k] is None else s[k].cpu().numpy()  # noqa: E731
    u, temp, top_k, top_p, min_p, allowed = (get(k) for k in ("u", "temperature", "top_k", "top_p", "min_p", "allowed"))
    token, prob = np.full(T, -1, np.int32), np.zeros(T)
    for t in range(T):
        ok = ~np.isnan(l[t]) & (l[t] > -np.inf)
        if allowed is not None:
            ok &= np.unpackbits(np.ascontiguousarray(allowed[t]).view(np.uint8), bitorder="little")[:V].astype(bool)
        ids = np.flatnonzero(ok)
        if ids.size == 0:
            continue
        z = l[t, ids]
        if temp[t] <= 0:
            token[t], prob[t] = ids[np.argmax(z)], 1.0
            continue
        ids = ids[np.argsort(-z, kind="stable")]
        if top_k is not None and top_k[t] > 0:
            ids = ids[:top_k[t]]
        e = np.exp((l[t, ids] - l[t, ids[0]]) / float(temp[t]))
        n = ids.size
        if top_p is not None:
            before = np.concatenate([[0.0], np.cumsum(e)[:-1]])
            n = max(1, int(np.searchsorted(before, float(top_p[t]) * e.sum(), side="left")))
        if min_p is not None:
            n = max(1, min(n, int(np.count_nonzero(e >= float(min_p[t])))))
        by = np.argsort(ids[:n], kind="stable")
        ids, e = ids[:n][by], e[:n][by]
        cum = np.cumsum(e)
        at = min(n - 1, int(np.searchsorted(cum, float(u[t]) * cum[-1], side="right")))
        token[t], prob[t] = ids[at], e[at] / cum[-1]
    return token, prob
