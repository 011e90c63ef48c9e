"""Workloads of the products with 4-bit weights that carry one scale, and where
wanted one zero point, per group of 32, 64 or 128 weights, on activations as
they are (f32, bf16 or f16): the linear layer with its epilogue, the router
that chooses experts, and the mixture-of-experts layer for a few tokens whose
experts are such weights.

`run` computes an operator in plain torch operations; with `own` set it makes
the library's calls instead.  `exact` computes the same outputs from the
definitions in 64 bits."""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
CODES = {"f32": 0, "bf16": 1, "f16": 2}                                  # QLL_DTYPE_*
ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}      # QLL_ACT_*
SCORES = {"softmax": 0, "sigmoid": 1}                                    # QLL_SCORE_*


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token through a small layer, f32 stream: a call's latency
        {"name": "linear small token", "op": "linear", "m": 1, "n": 512, "k": 512, "group": 32, "scales": "f16",
         "zeros": False, "x": "f32", "y": "f32", "act": "none", "bias": False, "residual": False},
        # one decoded token through an 8B-class up projection
        {"name": "linear up token", "op": "linear", "m": 1, "n": 14336, "k": 4096, "group": 128, "scales": "f16",
         "zeros": True, "x": "bf16", "y": "bf16", "act": "none", "bias": False, "residual": False},
        # a decode batch's down projection, added to the residual stream
        {"name": "linear down batch", "op": "linear", "m": 16, "n": 4096, "k": 14336, "group": 64, "scales": "bf16",
         "zeros": True, "x": "bf16", "y": "bf16", "act": "none", "bias": False, "residual": True},
        # a short prompt on an odd-sized layer with every part of the epilogue
        {"name": "linear ragged", "op": "linear", "m": 37, "n": 4099, "k": 1440, "group": 32, "scales": "f16",
         "zeros": True, "x": "f32", "y": "f32", "act": "gelu", "bias": True, "residual": True},
        # a prompt
        {"name": "linear prompt", "op": "linear", "m": 512, "n": 14336, "k": 4096, "group": 128, "scales": "f16",
         "zeros": False, "x": "f16", "y": "f16", "act": "silu", "bias": False, "residual": False},
        # one token's choice of experts
        {"name": "route token", "op": "route", "m": 1, "experts": 128, "top": 8, "k": 4096, "x": "bf16",
         "router": "bf16", "score": "softmax", "bias": False, "renorm": True},
        # a decode batch's, with the scores of each expert on their own and a bias that balances the load
        {"name": "route batch", "op": "route", "m": 64, "experts": 256, "top": 8, "k": 4096, "x": "bf16",
         "router": "f32", "score": "sigmoid", "bias": True, "renorm": True},
        # one token, a few experts of an 8B-class feed-forward block's size
        {"name": "moe token large", "op": "moe", "m": 1, "experts": 8, "top": 2, "n": 14336, "k": 4096, "group": 128,
         "scales": "f16", "zeros": True, "x": "bf16", "router": "bf16", "score": "softmax", "bias": False,
         "renorm": True, "act": "silu", "residual": True},
        # one token, many small experts
        {"name": "moe token", "op": "moe", "m": 1, "experts": 128, "top": 8, "n": 1024, "k": 2048, "group": 64,
         "scales": "bf16", "zeros": False, "x": "bf16", "router": "bf16", "score": "softmax", "bias": False,
         "renorm": True, "act": "silu", "residual": False},
        # a decode batch on the same experts
        {"name": "moe batch", "op": "moe", "m": 16, "experts": 128, "top": 8, "n": 1024, "k": 2048, "group": 64,
         "scales": "f16", "zeros": False, "x": "f16", "router": "f16", "score": "softmax", "bias": False,
         "renorm": True, "act": "silu", "residual": True},
        # odd sizes, f32 stream
        {"name": "moe ragged", "op": "moe", "m": 37, "experts": 23, "top": 3, "n": 1440, "k": 2592, "group": 32,
         "scales": "f16", "zeros": True, "x": "f32", "router": "f32", "score": "softmax", "bias": False,
         "renorm": False, "act": "gelu_tanh", "residual": True},
        # the largest decode batch: nearly every expert is read
        {"name": "moe large batch", "op": "moe", "m": 64, "experts": 64, "top": 6, "n": 1536, "k": 4096, "group": 128,
         "scales": "f16", "zeros": True, "x": "bf16", "router": "f32", "score": "sigmoid", "bias": True,
         "renorm": True, "act": "silu", "residual": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "route", "moe", "moe"])
    dtype = rng.choice(list(DTYPES))
    if op == "linear":
        group = rng.choice([32, 64, 128])
        while True:
            m, n, k = _log_int(rng, 1, 512), _log_int(rng, 1, 16384), group * _log_int(rng, 1, 15360 // group)
            if m * n * k <= 512 * 14336 * 4096:
                break
        return {"op": op, "m": m, "n": n, "k": k, "group": group, "scales": rng.choice(["f16", "bf16"]),
                "zeros": rng.random() < 0.5, "x": dtype, "y": rng.choice([dtype, "f32"]),
                "act": rng.choice(list(ACTS)), "bias": rng.random() < 0.5, "residual": rng.random() < 0.5}
    e = _log_int(rng, 2, 256)
    case = {"op": op, "m": _log_int(rng, 1, 64), "experts": e, "top": rng.randint(1, min(8, e)), "x": dtype,
            "router": rng.choice([dtype, "f32"]), "score": rng.choice(list(SCORES)), "bias": rng.random() < 0.5,
            "renorm": rng.random() < 0.5}
    if op == "route":
        return dict(case, k=_log_int(rng, 1, 8192))
    group = rng.choice([32, 64, 128])
    while True:
        n, k = group * _log_int(rng, 1, 14336 // group), group * _log_int(rng, 1, 4096 // group)
        if e * n * k <= 64 * 1536 * 4096:
            break
    return dict(case, n=n, k=k, group=group, scales=rng.choice(["f16", "bf16"]), zeros=rng.random() < 0.5,
                act=rng.choice(list(ACTS)), residual=rng.random() < 0.5)


def _size(dtype):
    return 4 if dtype == "f32" else 2


def _weight_bytes(case, n, k):
    return n * k // 2 + n * (k // case["group"]) * (2.5 if case["zeros"] else 2)


def work(case):
    m, k = case["m"], case["k"]
    e = _size(case["x"])
    if case["op"] == "linear":
        n, ey = case["n"], _size(case["y"])
        return {"bytes": _weight_bytes(case, n, k) + m * k * e + m * n * ey * (2 if case["residual"] else 1)
                + (4 * n if case["bias"] else 0), "flops": 2.0 * m * n * k}
    experts, top = case["experts"], case["top"]
    nbytes = experts * k * _size(case["router"]) + m * k * e + 8 * m * top + (4 * experts if case["bias"] else 0)
    flops = 2.0 * m * experts * k
    if case["op"] == "moe":
        # the weights of those experts that m tokens choose, each token independently of the others
        active = experts * (1.0 - (1.0 - top / experts) ** m)
        nbytes += active * 3 * _weight_bytes(case, case["n"], k) + m * k * e * (2 if case["residual"] else 1)
        flops += 6.0 * m * top * case["n"] * k
    return {"bytes": nbytes, "flops": flops}


# ------------------------------------------------------------------ inputs

def _inputs(case, seed):
    """What both the plain form and the library start from."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    def weights(*shape):
        """Codes [.., n, k], scales [.., n, k / group] that keep outputs near one, zero points around the middle."""
        n, k = shape[-2:]
        groups = (*shape[:-1], k // case["group"])
        codes = torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8).bitwise_and_(15)
        scales = (0.1 + 0.9 * torch.rand(groups, generator=g, device=DEV)) * (0.3 / math.sqrt(k))
        zeros = torch.randint(5, 12, groups, generator=g, device=DEV, dtype=torch.uint8) if case["zeros"] else None
        return codes, scales.to(DTYPES[case["scales"]]), zeros

    op, m, k = case["op"], case["m"], case["k"]
    st = {"x": normal(m, k).to(DTYPES[case["x"]])}
    if op == "linear":
        n, ydt = case["n"], DTYPES[case["y"]]
        st["w"] = weights(n, k)
        st["bias"] = normal(n) if case["bias"] else None
        st["residual"] = normal(m, n).to(ydt) if case["residual"] else None
        return st
    e = case["experts"]
    st["router"] = (normal(e, k) * (1.5 / math.sqrt(k))).to(DTYPES[case["router"]])
    st["router_bias"] = 0.1 * normal(e) if case["bias"] else None
    if op == "moe":
        n = case["n"]
        st["wg"], st["wu"], st["wd"] = weights(e, n, k), weights(e, n, k), weights(e, k, n)
        st["residual"] = normal(m, k).to(st["x"].dtype) if case["residual"] else None
    return st


def _scale(case):
    return 2.5 if case["score"] == "sigmoid" else 1.0


def _pack(qll, case, w):
    """The load-time packing of a program that keeps its weights so; experts one after another."""
    codes, scales, zeros = w
    n, k = codes.shape[-2:]
    count = codes.numel() // (n * k)
    fmt = _format(qll, case)
    size = qll.qll_q4g_packed_bytes(n, k, case["group"], fmt)
    wp = torch.empty(count, size, device=DEV, dtype=torch.uint8)
    codes, scales = codes.view(count, n, k), scales.view(count, n, -1)
    zeros = None if zeros is None else zeros.view(count, n, -1)
    for i in range(count):
        qll.qll_q4g_pack(codes[i], scales[i], None if zeros is None else zeros[i], case["group"], fmt, wp[i], n, k)
    return wp


def _format(qll, case):
    return (qll.QLL_Q4G_BF16 if case["scales"] == "bf16" else 0) | (qll.QLL_Q4G_ZEROS if case["zeros"] else 0)


def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"] = case
    op, m, k = case["op"], case["m"], case["k"]
    if not own:
        return st
    import quantized_linear_layer_amd as qll
    st["qll"] = qll
    if op == "linear":
        st["wp"] = _pack(qll, case, st.pop("w"))
        st["y"] = torch.empty(m, case["n"], device=DEV, dtype=DTYPES[case["y"]])
        need = qll.qll_workspace_bytes(qll.QLL_OP_Q4G_LINEAR, m, case["n"], k)
    else:
        e, top = case["experts"], case["top"]
        st["ids"] = torch.empty(m, top, device=DEV, dtype=torch.int32)
        st["weights"] = torch.empty(m, top, device=DEV)
        need = qll.qll_workspace_bytes(qll.QLL_OP_MOE_ROUTE, m, e, top)
        if op == "moe":
            for name in ("wg", "wu", "wd"):
                st[name] = _pack(qll, case, st[name])
            st["y"] = torch.empty(m, k, device=DEV, dtype=st["x"].dtype)
            need += qll.qll_workspace_bytes(qll.QLL_OP_Q4G_MOE, m, case["n"], top)
    st["ws"] = torch.empty(need, device=DEV, dtype=torch.uint8) if need else None
    return st


# ------------------------------------------------------------------ the library's calls

def _own(st):
    qll, case = st["qll"], st["case"]
    op, m, k, dtype = case["op"], case["m"], case["k"], CODES[case["x"]]
    if op == "linear":
        qll.qll_q4g_linear(st["wp"], case["group"], _format(qll, case), st["x"], dtype, st["bias"], ACTS[case["act"]],
                           st["residual"], st["y"], CODES[case["y"]], m, case["n"], k, ws=st["ws"])
        return {"y": st["y"]}
    e, top = case["experts"], case["top"]
    route = (st["x"], dtype, st["router"], CODES[case["router"]], st["router_bias"], SCORES[case["score"]],
             case["renorm"], _scale(case), st["ids"], st["weights"], top)
    out = {"ids": st["ids"], "weights": st["weights"]}
    if op == "route":
        qll.qll_moe_route(*route, m, e, k, ws=st["ws"])
        return out
    qll.qll_q4g_moe_layer(*route, st["wg"], st["wu"], st["wd"], case["group"], _format(qll, case), ACTS[case["act"]],
                          st["residual"], st["y"], m, case["n"], k, e, ws=st["ws"])
    return dict(out, y=st["y"])


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


def _values(w, group):
    """f32 values of codes [n, k] with their scales and zero points."""
    codes, scales, zeros = w
    n, k = codes.shape
    q = codes.view(n, k // group, group).float()
    q = q - (8.0 if zeros is None else zeros.float().unsqueeze(-1))
    return (q * scales.float().unsqueeze(-1)).view(n, k)


def _plain_route(st):
    case = st["case"]
    # the choice is between values next to each other: in 64 bits
    logits = torch.matmul(st["x"].double(), st["router"].double().t())
    if case["score"] == "softmax":
        e = torch.exp(logits - logits.amax(-1, keepdim=True))
        score = e / e.sum(-1, keepdim=True)
        by = logits
    else:
        score = 1.0 / (1.0 + torch.exp(-logits))
        by = logits
    if case["bias"]:
        by = score + st["router_bias"].double()
    _, ids = torch.sort(by, dim=-1, descending=True, stable=True)
    ids = ids[:, :case["top"]]
    w = torch.gather(score, 1, ids)
    if case["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return ids, (w * _scale(case)).float()


def _slot(w, expert):
    """One expert's weights, chosen by an index on the device."""
    return tuple(None if t is None else torch.index_select(t, 0, expert)[0] for t in w)


def _plain_moe(st, ids, weights):
    case = st["case"]
    m, e, top, group, act = case["m"], case["experts"], case["top"], case["group"], case["act"]
    x = st["x"].float()
    y = torch.zeros_like(x)

    def expert(rows, wg, wu, wd):
        h = _activate(torch.matmul(rows, _values(wg, group).t()), act) * torch.matmul(rows, _values(wu, group).t())
        return torch.matmul(h, _values(wd, group).t())

    if m * top <= e:  # few choices: each one's expert
        for i in range(m):
            for j in range(top):
                at = ids[i, j:j + 1]
                y[i] += weights[i, j] * expert(x[i:i + 1], *(_slot(st[w], at) for w in ("wg", "wu", "wd")))[0]
    else:  # every expert on every token, with weight 0 where it was not chosen
        dense = torch.zeros(m, e, device=DEV).scatter_(1, ids, weights)
        for i in range(e):
            one = [tuple(None if t is None else t[i] for t in st[w]) for w in ("wg", "wu", "wd")]
            y += dense[:, i:i + 1] * expert(x, *one)
    if case["residual"]:
        y = y + st["residual"].float()
    return y.to(st["x"].dtype)


def _plain(st):
    case = st["case"]
    if case["op"] == "linear":
        y = torch.matmul(st["x"].float(), _values(st["w"], case["group"]).t())
        if case["bias"]:
            y = y + st["bias"]
        y = _activate(y, case["act"])
        if case["residual"]:
            y = y + st["residual"].float()
        return {"y": y.to(DTYPES[case["y"]])}
    ids, weights = _plain_route(st)
    out = {"ids": ids.to(torch.int32), "weights": weights}
    if case["op"] == "moe":
        out["y"] = _plain_moe(st, ids, weights)
    return out


def run(st):
    return _own(st) if own else _plain(st)


# ------------------------------------------------------------------ 64 bits

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


def _times64(x, w, group):
    """x [m, k] times the rows of w, group by group: what the scale multiplies is the group's own sum."""
    codes, scales, zeros = w
    n, k = codes.shape
    out = torch.zeros(x.shape[0], n, device=DEV, dtype=torch.float64)
    step = max(group, group * ((1 << 27) // (n * group)))  # the codes of some 2^27 weights at a time
    for at in range(0, k, step):
        c = codes[:, at:at + step].to(torch.float64)
        s = scales[:, at // group:(at + step) // group].to(torch.float64)
        z = torch.full_like(s, 8.0) if zeros is None else zeros[:, at // group:(at + step) // group].to(torch.float64)
        s, z = s.repeat_interleave(group, 1), z.repeat_interleave(group, 1)
        out += x[:, at:at + step] @ (s * c - s * z).T
    return out


def exact(case, seed):
    st = _inputs(case, seed)
    x = st["x"].to(torch.float64)
    if case["op"] == "linear":
        y = _times64(x, st["w"], case["group"])
        if st["bias"] is not None:
            y += st["bias"].double()
        y = _act64(y, case["act"])
        return {"y": y if st["residual"] is None else y + st["residual"].double()}
    logits = x @ st["router"].to(torch.float64).T
    p = torch.softmax(logits, -1) if case["score"] == "softmax" else torch.sigmoid(logits)
    left = logits.clone() if st["router_bias"] is None else p + st["router_bias"].double()
    ids = []
    for _ in range(case["top"]):  # the largest that is left, the first of equal ones
        best = left.amax(-1, keepdim=True)
        i = torch.argmax((left == best).to(torch.uint8), -1, keepdim=True)
        left.scatter_(1, i, float("-inf"))
        ids.append(i)
    ids = torch.cat(ids, 1)
    weights = torch.take_along_dim(p, ids, 1)
    if case["renorm"]:
        weights = weights / weights.sum(1, keepdim=True)
    weights = weights * _scale(case)
    out = {"ids": ids.to(torch.int32), "weights": weights}
    if case["op"] == "moe":
        y = torch.zeros_like(x) if st["residual"] is None else st["residual"].to(torch.float64)
        for i in ids.unique().tolist():
            token, slot = torch.nonzero(ids == i, as_tuple=True)
            wg, wu, wd = ([None if t is None else t[i] for t in st[w]] for w in ("wg", "wu", "wd"))
            h = _act64(_times64(x[token], wg, case["group"]), case["act"]) * _times64(x[token], wu, case["group"])
            y.index_add_(0, token, weights[token, slot].unsqueeze(1) * _times64(h, wd, case["group"]))
        out["y"] = y
    return out
