"""Plain 64-bit forms of the routing rules and the 8-bit rows (test-only)."""
import numpy as np

F32_MAX = float(np.finfo(np.float32).max)


def route_rule(logits, k, score="softmax", bias=None, n_groups=1, top_groups=None,
               group_score="best", renorm=True, scale=1.0):
    """Picks [T][k] and float64 weights of a routing rule, one token at a time."""
    T, E = logits.shape
    gs = E // n_groups
    top_groups = n_groups if top_groups is None else top_groups
    idx, w = np.zeros((T, k), np.int32), np.zeros((T, k))
    for t in range(T):
        l = logits[t].astype(np.float64)
        l = np.where(np.isnan(l), -np.inf, np.minimum(l, F32_MAX))
        ok = l > -np.inf
        with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
            if score == "sigmoid":
                s = np.where(ok, 1 / (1 + np.exp(-l)), 0.0)
            else:
                m = l.max() if ok.any() else 0.0
                s = np.where(ok, np.exp(l - m), 0.0)
                s = s / s.sum() if ok.any() else s
            v = l.copy()
            if bias is not None:
                b = bias.astype(np.float64)
                v = np.where(ok & ~np.isnan(b), s + b, -np.inf)
        ok &= v > -np.inf
        stay = np.ones(E, bool)
        if top_groups < n_groups:
            gv = np.full(n_groups, -np.inf)
            for g in range(n_groups):
                sel = slice(g * gs, (g + 1) * gs)
                x = (s if bias is None and group_score == "sum2" else v)[sel][ok[sel]]
                if x.size:
                    x = np.sort(x)[::-1]
                    gv[g] = x[:2].sum() if group_score == "sum2" else x[0]
            kept = np.lexsort((np.arange(n_groups), -gv))[:top_groups]
            stay = np.isin(np.arange(E) // gs, kept)
        v = np.where(ok & stay, v, -np.inf)
        pick = np.lexsort((np.arange(E), -v))[:k]
        live = v[pick] > -np.inf
        if renorm and live.any():
            # relative to the largest pick's logit, so that tiny scores keep their ratios
            lp = l[pick][live]
            if score == "sigmoid":  # exp(min(l, 0)) / (1 + exp(-|l|)), without its common factor
                x = np.exp(np.minimum(lp, 0) - min(0.0, lp.max())) / (1 + np.exp(-np.abs(lp)))
            else:
                x = np.exp(lp - lp.max())
            w[t, :live.sum()] = x / x.sum() * scale
        else:
            w[t] = np.where(live, s[pick], 0.0) * scale
        idx[t] = pick
    return idx, w


def round_to(a, steps, least):
    """a at the nearest value of a binary format with `steps` values a power of
    two and the smallest normal exponent `least`; ties to even."""
    _, e = np.frexp(np.abs(a))
    unit = np.exp2(np.maximum(e - 1.0, least)) / steps
    return np.round(a / unit) * unit


def norm_rows(x, delta, weight, eps):
    """(h, y) of float64 arrays x and delta that hold bf16 values: h rounded to bf16."""
    h = x if delta is None else round_to((x.astype(np.float32) + delta.astype(np.float32))
                                         .astype(np.float64), 128, -126)
    y = h / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)
    return h, y * (1.0 if weight is None else weight)
