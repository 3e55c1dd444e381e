"""The measured cases of the layer's front-end operators.

Three operators that stand between a block's residual stream and its experts:

* route   -- picks and weights from router logits by a routing rule: softmax or
             sigmoid scores, a balance bias that only selects, group-limited
             top-k, renormalised and scaled weights
             (strata_moe_route_logits);
* norm    -- residual addition, weighted RMSNorm, and the normalised row also
             in 8 bits with scales (strata_moe_add_rmsnorm);
* dequant -- rows of such an 8-bit matrix, picked by index, back in bf16: what
             an expert's owner runs on after an exchange in 8 bits
             (strata_moe_dequant_rows).

Where `own` is false, `run` computes them with elementary torch operations.
"""
import torch

own = False

E4M3_MAX = 448.0
INT8_MAX = 127.0


def listed():
    return [
        # one token of a decode step, 256 experts in 8 groups of which 4 stay,
        # sigmoid scores with a balance bias
        {"name": "route-t1-groups", "op": "route", "T": 1, "E": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "top_groups": 4, "group_sum": True, "renorm": True, "dtype": "f32"},
        # a full decode batch of the 512-expert layer, softmax renormalised over its 10 picks
        {"name": "route-t64-softmax", "op": "route", "T": 64, "E": 512, "k": 10, "score": "softmax", "bias": False,
         "groups": 1, "top_groups": 1, "group_sum": False, "renorm": True, "dtype": "f32"},
        # a ragged chunk with bf16 logits (many equal ones), groups of 20 by their best expert, plain softmax weights
        {"name": "route-t1037-bf16", "op": "route", "T": 1037, "E": 160, "k": 6, "score": "softmax", "bias": True,
         "groups": 8, "top_groups": 3, "group_sum": False, "renorm": False, "dtype": "bf16"},
        # a prompt chunk of the 512-expert layer under sigmoid scores and a balance bias
        {"name": "route-t8192-sigmoid", "op": "route", "T": 8192, "E": 512, "k": 10, "score": "sigmoid", "bias": True,
         "groups": 1, "top_groups": 1, "group_sum": False, "renorm": True, "dtype": "f32"},
        # the largest batch a layer takes
        {"name": "route-t65536-groups", "op": "route", "T": 65536, "E": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "top_groups": 4, "group_sum": True, "renorm": True, "dtype": "f32"},
        # one token of a decode step, a scale for every 128 columns
        {"name": "norm-t1-e4m3", "op": "norm", "T": 1, "H": 2560, "q8": "e4m3", "group": 128, "weight": "bf16"},
        # a ragged batch of the widest row, a scale for every 32 columns
        {"name": "norm-t333-wide", "op": "norm", "T": 333, "H": 6144, "q8": "e4m3", "group": 32, "weight": "f32"},
        # a prompt chunk
        {"name": "norm-t8192-e4m3", "op": "norm", "T": 8192, "H": 2560, "q8": "e4m3", "group": 128, "weight": "bf16"},
        # a prompt chunk in int8 with a scale for a row, read back by the receiving side
        {"name": "norm-t4001-int8-read", "op": "norm", "T": 4001, "H": 2560, "q8": "int8", "group": 0, "weight": "f32"},
        # the picks of a decode batch of 4 tokens
        {"name": "dequant-n40", "op": "dequant", "n": 40, "src": 4, "H": 2560, "q8": "e4m3", "group": 128},
        # what one of four ranks receives of a prompt chunk's picks, int8 rows with one scale
        {"name": "dequant-n20483-int8", "op": "dequant", "n": 20483, "src": 8192, "H": 2560, "q8": "int8", "group": 0},
        # every pick of a prompt chunk
        {"name": "dequant-n81920", "op": "dequant", "n": 81920, "src": 8192, "H": 2560, "q8": "e4m3", "group": 128},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(("route", "route", "norm", "norm", "dequant"))
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 8, 16))
        E = groups * rng.randint(-(-16 // groups), 1024 // groups)
        top_groups = rng.randint(1, groups)
        k = rng.randint(1, min(16, top_groups * (E // groups)))
        return {"op": op, "T": _log(rng, 1, min(65536, 65536 * 256 // E)), "E": E, "k": k, "score": rng.choice(("softmax", "sigmoid")),
                "bias": rng.random() < 0.7, "groups": groups, "top_groups": top_groups,
                "group_sum": rng.random() < 0.5 and E // groups >= 2, "renorm": rng.random() < 0.7,
                "dtype": rng.choice(("f32", "f32", "bf16"))}
    H = 128 * rng.randint(1, 48)
    q8, group = rng.choice(("e4m3", "int8")), rng.choice((0, 32, 64, 128))
    if op == "norm":
        return {"op": op, "T": _log(rng, 1, 8192 * 2560 // H), "H": H, "q8": q8, "group": group,
                "weight": rng.choice(("bf16", "f32"))}
    n = _log(rng, 1, 81920 * 2560 // H)
    return {"op": op, "n": n, "src": max(1, n // rng.choice((1, 4, 10))), "H": H, "q8": q8, "group": group}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    f32, bf16, i32 = torch.float32, torch.bfloat16, torch.int32

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=f32)

    def empty(shape, dtype):
        return torch.empty(shape, device="cuda", dtype=dtype)

    s = dict(case)
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        # a trained router's logits: spread about 1.5, some experts popular (Zipf over a random rank)
        rank = torch.argsort(torch.rand(E, generator=g, device="cuda")).to(f32) + 1
        logits = 1.5 * normal(T, E) - 0.5 * 1.1 * rank.log()
        s["logits"] = logits.to(bf16) if case["dtype"] == "bf16" else logits
        # the balance bias leans against the popular experts
        size = 0.02 if case["score"] == "sigmoid" else 0.2 / E
        s["select_bias"] = size * (normal(E) + 0.5 * rank.log() - 2) if case["bias"] else None
        s["idx"], s["w"] = empty((T, k), i32), empty((T, k), f32)
        return s
    H = case["H"]
    code = torch.int8 if case["q8"] == "int8" else torch.float8_e4m3fn
    n_scales = H // case["group"] if case["group"] else 1
    if case["op"] == "norm":
        T = case["T"]
        # a residual stream has a few channels far above the others
        channel = torch.where(torch.rand(H, generator=g, device="cuda") < 0.01, 25.0, 1.0)
        s["x"] = (normal(T, H) * channel).to(bf16)
        s["delta"] = (0.5 * normal(T, H)).to(bf16)
        s["weight"] = (1 + 0.2 * normal(H)).to(bf16 if case["weight"] == "bf16" else f32)
        s["h"], s["xn"] = empty((T, H), bf16), empty((T, H), bf16)
        s["q"], s["scale"] = empty((T, H), code), empty((T, n_scales), f32)
        s["out"] = empty((T, H), bf16) if case["q8"] == "int8" else None
        return s
    n, src = case["n"], case["src"]
    step = INT8_MAX if case["q8"] == "int8" else E4M3_MAX
    s["q"] = (step / 4 * normal(src, H)).clamp(-step, step).to(code)
    s["scale"] = (4 / step) * (0.3 * normal(src, n_scales)).exp()
    s["rows"] = torch.randint(0, src, (n,), generator=g, device="cuda", dtype=i32)
    s["out"] = empty((n, H), bf16)
    return s


# ------------------------------------------------------------------ plain forms
def _plain_route(s):
    T, E, k, G = s["T"], s["E"], s["k"], s["groups"]
    low = -float("inf")
    # 64 bits: the order of near-equal scores decides whole numbers
    l = s["logits"].double()
    if s["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-l))
    else:
        score = torch.exp(l - l.max(1, keepdim=True).values)
        score = score / score.sum(1, keepdim=True)
    # without a bias the scores are in the logits' order
    value = l if s["select_bias"] is None else score + s["select_bias"].double()
    if G > 1:
        by_group = (score if s["select_bias"] is None and s["group_sum"] else value).view(T, G, E // G)
        if s["group_sum"]:
            best = by_group.sort(dim=2, descending=True).values[:, :, :2].sum(2)
        else:
            best = by_group.max(2).values
        kept = best.sort(dim=1, descending=True, stable=True).indices[:, : s["top_groups"]]
        out = torch.ones(T, G, dtype=torch.bool, device=l.device).scatter_(1, kept, False)
        value = value.masked_fill(out.repeat_interleave(E // G, 1), low)
    idx = value.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, idx)
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"idx": idx.int(), "w": (w * s_scale(s)).float()}


def s_scale(s):
    """The factor on the weights: such a rule scales renormalised sigmoid scores up."""
    return 2.5 if s["score"] == "sigmoid" and s["renorm"] else 1.0


def _plain_codes(y, s):
    """(codes as the values of their type, scales) of fp32 rows y."""
    T, H = y.shape
    blocks = y.view(T, -1, s["group"] or H)
    top = INT8_MAX if s["q8"] == "int8" else E4M3_MAX
    scale = blocks.abs().amax(2) / top
    a = blocks / torch.where(scale > 0, scale, 1.0).unsqueeze(2)
    q = a.round().clamp(-top, top) if s["q8"] == "int8" else a.clamp(-top, top)
    return q.to(s["q"].dtype).view(T, H), scale


def _plain_values(q, scale, s):
    n, H = q.shape
    return (q.float().view(n, -1, s["group"] or H) * scale.unsqueeze(2)).view(n, H).to(torch.bfloat16)


def _plain_norm(s):
    h = (s["x"].float() + s["delta"].float()).to(torch.bfloat16)
    v = h.float()
    y = v / (v.square().mean(1, keepdim=True) + 1e-6).sqrt() * s["weight"].float()
    q, scale = _plain_codes(y, s)
    if s["out"] is not None:
        return {"h": h, "xn": y.to(torch.bfloat16), "read": _plain_values(q, scale, s), "scale": scale}
    return {"h": h, "xn": y.to(torch.bfloat16), "q": q, "scale": scale}


def _plain_dequant(s):
    rows = s["rows"].long()
    q = s["q"].view(torch.int8)[rows].view(s["q"].dtype)
    return {"out": _plain_values(q, s["scale"][rows], s)}


# ------------------------------------------------------------------ the framework's calls
def _own_route(s):
    import quantized_expert_ffn_04_b200 as qe

    rule = s.get("rule")  # a program keeps its rule
    if rule is None:
        rule = s["rule"] = qe.make_routing(score=s["score"], n_groups=s["groups"], top_groups=s["top_groups"],
                                           group_score="sum2" if s["group_sum"] else "best", renorm=s["renorm"],
                                           scale=s_scale(s))
    bias = s["select_bias"]
    qe.strata_moe_route_logits(rule, s["logits"].data_ptr(), qe.STRATA_BF16 if s["dtype"] == "bf16" else qe.STRATA_F32,
                               s["E"], None if bias is None else bias.data_ptr(), s["T"], s["E"], s["k"],
                               s["idx"].data_ptr(), s["w"].data_ptr())
    return {"idx": s["idx"], "w": s["w"]}


def _own_norm(s):
    import quantized_expert_ffn_04_b200 as qe

    T, H, scale = s["T"], s["H"], s["scale"]
    q8 = qe.STRATA_Q8_INT8 if s["q8"] == "int8" else qe.STRATA_Q8_E4M3
    qe.strata_moe_add_rmsnorm(s["x"].data_ptr(), s["delta"].data_ptr(), s["weight"].data_ptr(),
                              qe.STRATA_BF16 if s["weight"].dtype == torch.bfloat16 else qe.STRATA_F32, 1e-6, T, H,
                              s["h"].data_ptr(), s["xn"].data_ptr(), q8, s["group"], s["q"].data_ptr(), H,
                              scale.data_ptr(), scale.shape[1])
    if s["out"] is not None:
        qe.strata_moe_dequant_rows(s["q"].data_ptr(), q8, H, scale.data_ptr(), scale.shape[1], s["group"], None, T, T, H,
                                   s["out"].data_ptr())
        return {"h": s["h"], "xn": s["xn"], "read": s["out"], "scale": scale}
    return {"h": s["h"], "xn": s["xn"], "q": s["q"], "scale": scale}


def _own_dequant(s):
    import quantized_expert_ffn_04_b200 as qe

    qe.strata_moe_dequant_rows(s["q"].data_ptr(), qe.STRATA_Q8_INT8 if s["q8"] == "int8" else qe.STRATA_Q8_E4M3, s["H"],
                               s["scale"].data_ptr(), s["scale"].shape[1], s["group"], s["rows"].data_ptr(), s["n"],
                               s["src"], s["H"], s["out"].data_ptr())
    return {"out": s["out"]}


def run(state):
    if own:
        return {"route": _own_route, "norm": _own_norm, "dequant": _own_dequant}[state["op"]](state)
    return {"route": _plain_route, "norm": _plain_norm, "dequant": _plain_dequant}[state["op"]](state)


def work(case):
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        size = 2 if case["dtype"] == "bf16" else 4
        # a score (exp, add, divide) and a comparison for each logit
        return {"bytes": T * E * size + T * k * 8 + (E * 4 if case["bias"] else 0), "flops": 4 * T * E}
    H = case["H"]
    n_scales = H // case["group"] if case["group"] else 1
    if case["op"] == "norm":
        T = case["T"]
        weight = H * (2 if case["weight"] == "bf16" else 4)
        # x, delta and weight in; h, xn, codes and scales out
        row = H * (2 + 2) + H * (2 + 2 + 1) + n_scales * 4
        read = H * (1 + 2) + n_scales * 4 if case["q8"] == "int8" else 0
        return {"bytes": T * (row + read) + weight, "flops": 8 * T * H}
    n, src = case["n"], case["src"]
    return {"bytes": min(n, src) * (H + 4 * n_scales) + n * (H * 2 + 4), "flops": n * H}


# ------------------------------------------------------------------ 64 bits
def _exact_route(s):
    import numpy as np

    l = s["logits"].float().cpu().numpy().astype(np.float64)
    bias = None if s["select_bias"] is None else s["select_bias"].cpu().numpy().astype(np.float64)
    T, E = l.shape
    G, k = s["groups"], s["k"]
    if s["score"] == "sigmoid":
        p = np.where(l >= 0, 1 / (1 + np.exp(-np.abs(l))), np.exp(-np.abs(l)) / (1 + np.exp(-np.abs(l))))
    else:
        p = np.exp(l - np.logaddexp.reduce(l, axis=1)[:, None])
    key = l if bias is None else p + bias
    if G > 1:
        m = (p if bias is None and s["group_sum"] else key).reshape(T, G, -1)
        if s["group_sum"]:
            two = np.partition(m, m.shape[2] - 2, axis=2)[:, :, -2:]
            rank = two[:, :, 0] + two[:, :, 1]
        else:
            rank = m.max(axis=2)
        order = np.argsort(-rank, axis=1, kind="stable")
        place = np.argsort(order, axis=1)
        key = np.where((place < s["top_groups"])[:, :, None], key.reshape(T, G, -1), -np.inf).reshape(T, E)
    idx = np.argsort(-key, axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(p, idx, axis=1)
    if s["renorm"]:
        w = w / w.sum(axis=1, keepdims=True)
    return {"idx": torch.from_numpy(idx.astype(np.int32)), "w": torch.from_numpy(w * s_scale(s))}


def _near(a, steps, least):
    """a (64 bits) at the nearest value of a binary format with `steps` values a power of two, ties to even;
    `least`: its smallest normal exponent."""
    e = torch.frexp(a.abs()).exponent.double() - 1
    unit = torch.exp2(e.clamp(min=least)) / steps
    return torch.round(a / unit) * unit


def _exact_norm(s):
    h = _near(s["x"].double() + s["delta"].double(), 128, -126)
    mean = (h * h).sum(1) / s["H"]
    y = h * s["weight"].double() * torch.rsqrt(mean + 1e-6)[:, None]
    top = INT8_MAX if s["q8"] == "int8" else E4M3_MAX
    width = s["group"] or s["H"]
    blocks = y.reshape(y.shape[0], s["H"] // width, width)
    scale = blocks.abs().max(2).values / top
    a = blocks / scale[:, :, None]
    q = torch.round(a) if s["q8"] == "int8" else _near(a, 8, -6)
    if s["out"] is not None:
        return {"h": h, "xn": y, "read": (q * scale[:, :, None]).reshape(y.shape), "scale": scale}
    return {"h": h, "xn": y, "q": q.reshape(y.shape), "scale": scale}


def _exact_dequant(s):
    width = s["group"] or s["H"]
    rows = s["rows"].long()
    v = s["q"].double().reshape(s["src"], -1, width) * s["scale"].double()[:, :, None]
    return {"out": v.reshape(s["src"], s["H"])[rows]}


def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "norm": _exact_norm, "dequant": _exact_dequant}[case["op"]](s)
