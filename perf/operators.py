"""Workloads of the operators around the quantized linear layers: the norm
that feeds them (residual sum, root-mean-square norm and 8-bit activations in
one pass), the linear layer with its epilogue (bias, activation, residual),
the gated feed-forward projection (activation of one product times another),
and the token log probabilities that are read off the vocabulary
projection's logits.

`run` computes an operator in plain torch operations; with `own` set it makes
the library's calls instead.  `exact` computes the same outputs from the
definitions in 64 bits."""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
CODES = {"f32": 0, "bf16": 1, "f16": 2}                                  # QLL_DTYPE_*
ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}      # QLL_ACT_*


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decoded token enters a layer of an 8B-class model: residual sum, norm, Q8_0 row
        {"name": "norm q8_0 decode", "op": "norm", "form": "q8_0", "m": 1, "k": 4096, "dtype": "f32", "residual": True},
        # a long prompt through the same step
        {"name": "norm q8_0 prompt", "op": "norm", "form": "q8_0", "m": 8192, "k": 4096, "dtype": "f32",
         "residual": True},
        # a decode batch entering a BitNet layer: no residual, half-precision stream
        {"name": "norm i8 batch", "op": "norm", "form": "i8", "m": 64, "k": 2560, "dtype": "f16", "residual": False},
        # a prompt entering the BitNet down projection's width, bf16 stream
        {"name": "norm i8 prompt", "op": "norm", "form": "i8", "m": 4096, "k": 6912, "dtype": "bf16",
         "residual": True},
        # one token's down projection, added to the residual stream
        {"name": "linear down decode", "op": "linear", "layout": "blocks", "m": 1, "n": 4096, "k": 14336,
         "act": "none", "bias": False, "residual": True},
        # a short prompt on an odd-sized layer with every part of the epilogue
        {"name": "linear ragged", "op": "linear", "layout": "blocks", "m": 37, "n": 4099, "k": 1440, "act": "gelu",
         "bias": True, "residual": True},
        # a prompt's up projection of a non-gated model, weights repacked at load time
        {"name": "linear up prompt", "op": "linear", "layout": "repacked", "m": 512, "n": 14336, "k": 4096,
         "act": "gelu_tanh", "bias": True, "residual": False},
        # one token's gate and up projections
        {"name": "gated decode", "op": "gated", "layout": "blocks", "m": 1, "n": 14336, "k": 4096, "act": "silu"},
        # a decode batch
        {"name": "gated batch", "op": "gated", "layout": "blocks", "m": 16, "n": 14336, "k": 4096,
         "act": "gelu_tanh"},
        # a prompt, weights repacked at load time
        {"name": "gated prompt", "op": "gated", "layout": "repacked", "m": 512, "n": 14336, "k": 4096,
         "act": "silu"},
        # the sampled token's log probability with twenty alternatives
        {"name": "logprobs decode", "op": "logprobs", "m": 1, "v": 128256, "tokens": 1, "top": 20, "dtype": "f32",
         "masked": False},
        # scoring a prompt
        {"name": "logprobs prompt", "op": "logprobs", "m": 512, "v": 128256, "tokens": 1, "top": 5, "dtype": "f32",
         "masked": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["norm", "linear", "gated", "logprobs"])
    if op == "norm":
        form = rng.choice(["q8_0", "i8"])
        k = 32 * _log_int(rng, 1, 512) if form == "q8_0" else _log_int(rng, 1, 16384)
        m = _log_int(rng, 1, min(8192, 8192 * 4096 // k))
        return {"op": op, "form": form, "m": m, "k": k, "dtype": rng.choice(list(DTYPES)),
                "residual": rng.random() < 0.5}
    if op == "logprobs":
        v = _log_int(rng, 2, 160000)
        m = _log_int(rng, 1, min(512, 512 * 128256 // v))
        return {"op": op, "m": m, "v": v, "tokens": rng.randint(1, 4), "top": min(v, rng.randint(0, 32)),
                "dtype": rng.choice(list(DTYPES)), "masked": rng.random() < 0.5}
    while True:
        m, n, k = _log_int(rng, 1, 512), _log_int(rng, 1, 16384), 32 * _log_int(rng, 1, 480)
        if m * n * k <= 512 * 14336 * 4096:
            break
    layout = rng.choice(["blocks", "repacked"])
    act = rng.choice(list(ACTS))
    if op == "gated":
        return {"op": op, "layout": layout, "m": m, "n": n, "k": k, "act": act}
    return {"op": op, "layout": layout, "m": m, "n": n, "k": k, "act": act, "bias": rng.random() < 0.5,
            "residual": rng.random() < 0.5}


def work(case):
    op = case["op"]
    if op == "norm":
        m, k = case["m"], case["k"]
        e = 4 if case["dtype"] == "f32" else 2
        out = m * k // 32 * 34 if case["form"] == "q8_0" else m * (k + 8)
        # the norm of each row, its codes; the sum is read twice over and written once
        return {"bytes": m * k * e * (3 if case["residual"] else 1) + 4 * k + out, "flops": 6.0 * m * k}
    if op == "logprobs":
        m, v = case["m"], case["v"]
        e = 4 if case["dtype"] == "f32" else 2
        return {"bytes": m * v * e + m * (8 * case["tokens"] + 4 + 8 * case["top"]), "flops": 5.0 * m * v}
    m, n, k = case["m"], case["n"], case["k"]
    mats = 2 if op == "gated" else 1
    bytes_ = mats * n * (k // 32) * 18 + m * (k // 32) * 34 + 4 * m * n
    if op == "linear":
        bytes_ += (4 * n if case["bias"] else 0) + (4 * m * n if case["residual"] else 0)
    return {"bytes": bytes_, "flops": 2.0 * mats * m * n * k}


# ------------------------------------------------------------------ inputs

def _inputs(case, seed):
    """What both the plain form and the library start from."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    op = case["op"]
    if op == "norm":
        m, k = case["m"], case["k"]
        dt = DTYPES[case["dtype"]]
        # a residual stream: most channels near one, a few that are large in every row
        spread = torch.ones(k, device=DEV)
        spread[torch.randint(0, k, (1 + k // 512,), generator=g, device=DEV)] = 20.0
        st = {"x": (normal(m, k) * spread).to(dt),
              "weight": 0.5 + torch.rand(k, generator=g, device=DEV)}
        st["residual"] = (normal(m, k) * spread).to(dt) if case["residual"] else None
        return st
    if op == "logprobs":
        m, v = case["m"], case["v"]
        x = normal(m, v) * 3.0
        if case["masked"]:  # a constrained vocabulary; in a batch also a row with nothing left
            x.masked_fill_(torch.rand(m, v, generator=g, device=DEV) < 0.1, float("-inf"))
            if m > 1:
                x[m // 2] = float("-inf")
        return {"logits": x.to(DTYPES[case["dtype"]]),
                "tokens": torch.randint(0, v, (m, case["tokens"]), generator=g, device=DEV, dtype=torch.int32)}
    m, n, k = case["m"], case["n"], case["k"]
    nb = k // 32

    def weights():
        w = torch.randint(0, 256, (n, nb, 18), generator=g, device=DEV, dtype=torch.uint8)
        # the scale: 0.001 .. 0.01 times what keeps outputs near one
        d = (0.1 + 0.9 * torch.rand(n, nb, generator=g, device=DEV)) * (0.3 / math.sqrt(k))
        w[..., :2] = d.half().unsqueeze(-1).view(torch.uint8)
        return w

    x = normal(m, nb, 32)
    d = x.abs().amax(-1, keepdim=True) / 127.0
    xq = torch.empty(m, nb, 34, device=DEV, dtype=torch.uint8)
    xq[..., :2] = d.half().view(torch.uint8)
    xq[..., 2:] = torch.round(x / d).clamp(-127, 127).to(torch.int8).view(torch.uint8)
    st = {"w": weights(), "xq": xq}
    if op == "gated":
        st["wu"] = weights()
    else:
        st["bias"] = normal(n) if case["bias"] else None
        st["residual"] = normal(m, n) if case["residual"] else None
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"] = case
    op = case["op"]
    if op == "norm":
        m, k = case["m"], case["k"]
        st["h"] = torch.empty_like(st["x"]) if case["residual"] else None
        if case["form"] == "q8_0":
            st["xq"] = torch.empty(m, k // 32, 34, device=DEV, dtype=torch.uint8)
            st["scale"], st["codes"] = st["xq"][..., :2].view(torch.float16), st["xq"][..., 2:].view(torch.int8)
            st["values"] = torch.empty(m, k // 32, 32, device=DEV, dtype=torch.float16)
        else:
            st["xq"] = torch.empty(m, k, device=DEV, dtype=torch.int8)
            st["act_scale"] = torch.empty(m, device=DEV)
            st["act_sum"] = torch.empty(m, device=DEV, dtype=torch.int32)
            st["scale"] = st["act_scale"].unsqueeze(-1)
            st["values"] = torch.empty(m, k, device=DEV)
    elif op == "logprobs":
        m, t = case["m"], case["top"]
        st["logprob"] = torch.empty(m, case["tokens"], device=DEV)
        st["entropy"] = torch.empty(m, device=DEV)
        st["top_ids"] = torch.empty(m, t, device=DEV, dtype=torch.int32)
        st["top_logprob"] = torch.empty(m, t, device=DEV)
    else:
        st["y"] = torch.empty(case["m"], case["n"], device=DEV)
    if own:
        import quantized_linear_layer_amd as qll
        st["qll"] = qll
        need = 0
        if op == "logprobs":
            need = qll.qll_workspace_bytes(qll.QLL_OP_TOKEN_LOGPROBS, case["m"], case["v"], case["top"])
        elif op != "norm":
            m, n, k = case["m"], case["n"], case["k"]
            if case["layout"] == "blocks":
                kind = qll.QLL_OP_Q4_0_GATED if op == "gated" else qll.QLL_OP_Q4_0_LINEAR
            else:  # the load-time repack of a program that keeps its weights so
                kind = qll.QLL_OP_Q4_0_REPACKED_GATED if op == "gated" else qll.QLL_OP_Q4_0_REPACKED_GEMM
                if op == "gated":
                    st["wp"] = torch.empty(qll.qll_q4_0_repacked_gated_bytes(n, k), device=DEV, dtype=torch.uint8)
                    qll.qll_q4_0_repack_gated(st["w"], st["wu"], st["wp"], n, k)
                else:
                    st["wp"] = torch.empty(qll.qll_q4_0_repacked_bytes(n, k), device=DEV, dtype=torch.uint8)
                    qll.qll_q4_0_repack(st["w"], st["wp"], n, k)
            need = qll.qll_workspace_bytes(kind, m, n, k)
        st["ws"] = torch.empty(need, device=DEV, dtype=torch.uint8) if need else None
    return st


# ------------------------------------------------------------------ the library's calls

def _own(st):
    qll, case = st["qll"], st["case"]
    op = case["op"]
    if op == "norm":
        m, k, code = case["m"], case["k"], CODES[case["dtype"]]
        if case["form"] == "q8_0":
            qll.qll_rmsnorm_q8_0(st["x"], code, st["residual"], st["weight"], EPS, st["h"], st["xq"], m, k)
            out = {"values": torch.mul(st["codes"], st["scale"], out=st["values"])}
        else:
            qll.qll_rmsnorm_i8_rows(st["x"], code, st["residual"], st["weight"], EPS, st["h"], st["xq"],
                                    st["act_scale"], st["act_sum"], m, k)
            out = {"values": torch.div(st["xq"], st["scale"], out=st["values"]), "act_scale": st["act_scale"],
                   "act_sum": st["act_sum"]}
        if st["h"] is not None:
            out["h"] = st["h"]
        return out
    if op == "logprobs":
        m, v, t, top = case["m"], case["v"], case["tokens"], case["top"]
        qll.qll_token_logprobs(st["logits"], CODES[case["dtype"]], st["tokens"], t, st["logprob"], st["entropy"], top,
                               st["top_ids"], st["top_logprob"], m, v, ws=st["ws"])
        return {"logprob": st["logprob"], "entropy": st["entropy"], "top_ids": st["top_ids"],
                "top_logprob": st["top_logprob"]}
    m, n, k, act = case["m"], case["n"], case["k"], ACTS[case["act"]]
    if op == "gated":
        if case["layout"] == "blocks":
            qll.qll_q4_0_q8_0_gated(st["w"], st["wu"], st["xq"], act, st["y"], m, n, k, ws=st["ws"])
        else:
            qll.qll_q4_0_repacked_q8_0_gated(st["wp"], st["xq"], act, st["y"], m, n, k, ws=st["ws"])
    elif case["layout"] == "blocks":
        qll.qll_q4_0_q8_0_linear(st["w"], st["xq"], st["bias"], act, st["residual"], st["y"], m, n, k, ws=st["ws"])
    else:
        qll.qll_q4_0_repacked_q8_0_linear(st["wp"], st["xq"], st["bias"], act, st["residual"], st["y"], m, n, k,
                                          ws=st["ws"])
    return {"y": st["y"]}


# ------------------------------------------------------------------ the plain forms

def _activate(x, act):
    if act == "relu":
        return torch.clamp_min(x, 0.0)
    if act == "gelu":
        return 0.5 * x * (1.0 + torch.erf(x * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))
    if act == "silu":
        return x / (1.0 + torch.exp(-x))
    return x


def _q4_0_values(w):
    n, nb, _ = w.shape
    d = w[..., :2].contiguous().view(torch.float16).float()
    qs = w[..., 2:]
    codes = torch.cat((qs & 15, qs >> 4), -1).float() - 8.0
    return (codes * d).view(n, nb * 32)


def _q8_0_values(xq):
    m, nb, _ = xq.shape
    d = xq[..., :2].contiguous().view(torch.float16).float()
    return (xq[..., 2:].contiguous().view(torch.int8).float() * d).view(m, nb * 32)


def _plain_norm(st):
    case = st["case"]
    m, k = case["m"], case["k"]
    h = st["x"]
    if case["residual"]:
        h = (st["x"].float() + st["residual"].float()).to(h.dtype)
    # the codes round values next to a border: in 64 bits
    hd = h.double()
    rstd = 1.0 / torch.sqrt((hd * hd).mean(-1, keepdim=True) + EPS)
    p = hd * st["weight"].double()
    if case["form"] == "q8_0":
        p, rstd = p.view(m, k // 32, 32), rstd.unsqueeze(-1)
    amax = p.abs().amax(-1, keepdim=True)
    q = torch.where(amax > 0, 127.0 * p / amax, 0.0)
    q = torch.sign(q) * torch.floor(q.abs() + 0.5)
    if case["form"] == "q8_0":
        d = (amax * rstd / 127.0).float().half()
        out = {"values": (q.float() * d.float()).half()}
    else:
        s = (127.0 / (amax * rstd)).float()
        out = {"values": q.float() / s, "act_scale": s.squeeze(-1), "act_sum": q.sum(-1).to(torch.int32)}
    if case["residual"]:
        out["h"] = h
    return out


def _plain_logprobs(st):
    case = st["case"]
    x = st["logits"].float()
    mx = x.amax(-1, keepdim=True)
    e = torch.exp(x - mx)
    s = e.sum(-1, keepdim=True)
    log_s = torch.log(s)
    t = torch.where(e != 0, (x - mx) * e, 0.0).sum(-1, keepdim=True)
    best, ids = torch.sort(x, dim=-1, descending=True, stable=True)
    best, ids = best[:, :case["top"]], ids[:, :case["top"]]
    return {"logprob": torch.gather(x, 1, st["tokens"].long()) - mx - log_s, "entropy": (log_s - t / s).squeeze(-1),
            "top_ids": ids.to(torch.int32), "top_logprob": best - mx - log_s}


def _plain(st):
    case = st["case"]
    if case["op"] == "norm":
        return _plain_norm(st)
    if case["op"] == "logprobs":
        return _plain_logprobs(st)
    x = _q8_0_values(st["xq"])
    y = torch.matmul(x, _q4_0_values(st["w"]).t())
    if case["op"] == "gated":
        return {"y": _activate(y, case["act"]) * torch.matmul(x, _q4_0_values(st["wu"]).t())}
    if case["bias"]:
        y = y + st["bias"]
    y = _activate(y, case["act"])
    if case["residual"]:
        y = y + st["residual"]
    return {"y": y}


def run(st):
    return _own(st) if own else _plain(st)


# ------------------------------------------------------------------ 64 bits

def _half64(b):
    """Little-endian binary16 byte pairs [..., 2] as float64, from their bits."""
    bits = b[..., 0].to(torch.int64) | (b[..., 1].to(torch.int64) << 8)
    e, f = (bits >> 10) & 31, (bits & 1023).double()
    mag = torch.where(e > 0, (1024.0 + f) * torch.exp2((e - 25).double()), f * 2.0 ** -24)
    return torch.where(bits >= 32768, -mag, mag)


def _rows64(blocks, four_bit):
    out = torch.empty(blocks.shape[0], blocks.shape[1], 32, device=blocks.device, dtype=torch.float64)
    d = _half64(blocks[..., :2]).unsqueeze(-1)
    q = blocks[..., 2:].to(torch.int16)
    if four_bit:
        out[..., :16] = (q % 16 - 8).double() * d
        out[..., 16:] = (q // 16 - 8).double() * d
    else:
        out[...] = torch.where(q > 127, q - 256, q).double() * d
    return out.flatten(1)


def _act64(x, act):
    if act == "relu":
        return torch.where(x > 0, x, torch.zeros_like(x))
    if act == "gelu":
        return x * torch.special.ndtr(x)
    if act == "gelu_tanh":
        return x * torch.special.expit(2.0 * math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3))
    if act == "silu":
        return x * torch.special.expit(x)
    return x


def exact(case, seed):
    st = _inputs(case, seed)
    op = case["op"]
    if op == "norm":
        m, k, q8 = case["m"], case["k"], case["form"] == "q8_0"
        h = st["x"].double()
        if st["residual"] is not None:  # the stream keeps its type: the sum, rounded, is what is normed
            h = (h + st["residual"].double()).float().to(st["x"].dtype).double()
        v = h * st["weight"].double()
        groups = v.reshape(m, k // 32, 32) if q8 else v.reshape(m, 1, k)
        top = groups.abs().amax(-1)
        rms = torch.sqrt(torch.linalg.vector_norm(h, dim=-1) ** 2 / k + EPS).reshape(m, 1)
        steps = groups * 127.0 / top.unsqueeze(-1)
        codes = torch.where(steps < 0, torch.ceil(steps - 0.5), torch.floor(steps + 0.5))
        if q8:
            d = (top / (127.0 * rms)).float().half().double().unsqueeze(-1)
            out = {"values": codes * d}
        else:
            s = (127.0 * rms / top).float().double()
            out = {"values": (codes / s.unsqueeze(-1)).reshape(m, k), "act_scale": s.reshape(m),
                   "act_sum": codes.sum((1, 2)).to(torch.int32)}
        if st["residual"] is not None:
            out["h"] = h
        return out
    if op == "logprobs":
        x = st["logits"].double()
        lse = torch.logsumexp(x, -1, keepdim=True)
        lp = x - lse
        p = torch.exp(lp)
        entropy = -(torch.where(p == 0, torch.zeros_like(p), p * lp)).sum(-1)
        ids = []
        left = x.clone()
        taken = torch.zeros_like(x, dtype=torch.bool)
        for _ in range(case["top"]):  # the largest that is left, the first of equal ones
            best = torch.where(taken, float("-inf"), left).amax(-1, keepdim=True)
            hit = (left == best) & ~taken
            i = torch.argmax(hit.to(torch.uint8), -1, keepdim=True)
            taken.scatter_(1, i, True)
            ids.append(i)
        ids = torch.cat(ids, 1) if ids else torch.empty(case["m"], 0, device=DEV, dtype=torch.int64)
        empty = torch.isinf(lse) & (lse < 0)
        nan = float("nan")
        return {"logprob": torch.gather(lp, 1, st["tokens"].long()).masked_fill(empty, nan),
                "entropy": entropy.masked_fill(empty[:, 0], nan), "top_ids": ids.to(torch.int32),
                "top_logprob": torch.gather(lp, 1, ids).masked_fill(empty, nan)}
    x = _rows64(st["xq"], False)
    y = x @ _rows64(st["w"], True).T
    if op == "gated":
        return {"y": _act64(y, case["act"]) * (x @ _rows64(st["wu"], True).T)}
    if st["bias"] is not None:
        y += st["bias"].double()
    y = _act64(y, case["act"])
    return {"y": y if st["residual"] is None else y + st["residual"].double()}
