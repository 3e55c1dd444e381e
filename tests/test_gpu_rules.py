"""Routing rules on the GPU: strata_moe_route_logits against a plain 64-bit
form, and layers whose rule is set (strata_moe_set_routing) through route,
forward, the stack and expert parallelism's steps.

Picks are compared bit for bit.  Weights: the kernel computes a pick's score
from its fp32 logit with expf (2 ulp of 2^-23), a subtraction, an addition and
a division (2^-24 each, the subtraction's rounding of |l - c| <= 32 times
larger in the exponent), a sum of at most 32 of them (5 roundings) and one
division and one product: (4 + 32 + 2) on either side of the quotient + 7
roundings of 2^-24 = 5e-6 for renormalised weights (and plain sigmoid ones);
plain softmax weights divide by a sum of __expf terms, within 6.2e-6 of it
(select.cuh), so 1.2e-5.
"""
import numpy as np
import pytest

import gen
import oracle
from tests import npref
from tests.front_ref import route_rule
from tests.gpu_util import THREADS, check_output, from_dev_bf16, to_dev_bf16

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import quantized_expert_ffn_04_b200 as qe  # noqa: E402

W_TOL, W_TOL_PLAIN_SOFTMAX = 5e-6, 1.2e-5


def call(logits, k, bias=None, stream=None, pad=None, **kw):
    """route_logits of a numpy [T][E] (or a cuda tensor), into buffers with a guard row."""
    t = torch.from_numpy(logits).cuda() if isinstance(logits, np.ndarray) else logits
    T, E = logits.shape
    idx = torch.full((T + 1, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, k), -7.0, dtype=torch.float32, device="cuda")
    b = None if bias is None else torch.from_numpy(bias).cuda()
    qe.strata_moe_route_logits(qe.make_routing(**kw), t.data_ptr(),
                               qe.STRATA_BF16 if t.dtype == torch.bfloat16 else qe.STRATA_F32,
                               t.stride(0) if T > 1 else max(E, t.stride(0)),
                               None if b is None else b.data_ptr(), T, E, k, idx.data_ptr(),
                               w.data_ptr(), stream)
    torch.cuda.synchronize()
    assert (idx[T] == -7).all() and (w[T] == -7).all(), "wrote past the last token"
    return idx[:T].cpu().numpy(), w[:T].cpu().numpy()


def check(logits, k, bias=None, **kw):
    host = logits if isinstance(logits, np.ndarray) else logits.float().cpu().numpy()
    idx, w = call(logits, k, bias, **kw)
    ridx, rw = route_rule(host, k, bias=bias, **kw)
    assert np.array_equal(idx, ridx), np.argwhere(idx != ridx)[:5]
    plain = kw.get("score", "softmax") == "softmax" and not kw.get("renorm", True)
    np.testing.assert_allclose(w, rw, rtol=W_TOL_PLAIN_SOFTMAX if plain else W_TOL, atol=1e-37)


def logits_of(T, E, seed, scale=1.5):
    return (scale * np.random.default_rng(seed).standard_normal((T, E))).astype(np.float32)


def bias_of(E, seed, scale=0.05):
    return (scale * np.random.default_rng(seed + 1000).standard_normal(E)).astype(np.float32)


RULES = [dict(score="softmax"), dict(score="softmax", renorm=False, scale=0.5), dict(score="sigmoid", scale=2.5),
         dict(score="sigmoid", renorm=False)]
GROUPS = [(1, 1, "best"), (8, 4, "sum2"), (4, 1, "best"), (8, 3, "best"), (2, 1, "sum2"), (8, 8, "sum2")]


@pytest.mark.parametrize("rule", RULES, ids=["softmax", "softmax-plain", "sigmoid", "sigmoid-plain"])
@pytest.mark.parametrize("groups", GROUPS, ids=lambda g: "%dof%d-%s" % (g[1], g[0], g[2]))
@pytest.mark.parametrize("bias", [False, True], ids=["nobias", "bias"])
def test_rules_match_the_plain_form(rule, groups, bias):
    n, top, gsc = groups
    for T, E, k, seed in [(1, 256, 8, 0), (5, 16, 2, 1), (130, 160, 6, 2), (64, 512, 10, 3), (33, 1024, 16, 4), (7, 1000, 5, 5)]:
        if k <= top * (E // n):
            check(logits_of(T, E, seed), k, bias_of(E, seed) if bias else None, n_groups=n, top_groups=top,
                  group_score=gsc, **rule)


@pytest.mark.parametrize("E,k,n,top", [(1, 1, 1, 1), (2, 2, 1, 1), (3, 2, 1, 1), (31, 31, 1, 1), (33, 32, 1, 1), (32, 32, 1, 1),
                                       (1020, 32, 17, 3), (1024, 32, 32, 1), (990, 7, 30, 2), (62, 4, 31, 2), (64, 2, 32, 1),
                                       (1023, 32, 1, 1), (1024, 32, 1, 1), (513, 9, 3, 1), (96, 32, 3, 2),
                                       (16, 4, 16, 5), (32, 7, 32, 9), (32, 16, 4, 2), (128, 32, 4, 1)])
def test_odd_sizes(E, k, n, top):
    for score in ("softmax", "sigmoid"):
        for bias in (None, bias_of(E, E)):
            gs = "sum2" if E // n >= 2 and k % 2 else "best"
            check(logits_of(19, E, E + k), k, bias, score=score, n_groups=n, top_groups=top, group_score=gs)


@pytest.mark.parametrize("E,k,n,top", [(256, 8, 8, 4), (256, 10, 1, 1), (512, 10, 1, 1), (512, 16, 4, 2), (160, 6, 8, 3), (64, 16, 2, 1),
                                       (16, 2, 1, 1), (1024, 16, 16, 1), (480, 15, 16, 3), (768, 4, 1, 1), (250, 7, 5, 2), (31, 16, 1, 1),
                                       (1000, 12, 8, 8), (60, 1, 15, 1), (256, 16, 1, 1)])
def test_large_batches(E, k, n, top):
    """Batches large enough for several tokens a warp: every token against the
    call of few, and a sample (with masked and equal rows) against the plain form."""
    T = 17001 if k % 2 == 0 else 9001
    rng = np.random.default_rng(E + k)
    l = logits_of(T, E, E)
    odd = rng.choice(T, 60, replace=False)
    l[odd[:10], : E // 2] = -np.inf
    l[odd[10:20]] = 0.25
    l[odd[20:30], ::3] = np.nan
    l[odd[30:40]] = -np.inf
    l[odd[40:50]] = np.round(l[odd[40:50]])
    l[odd[50:], rng.integers(0, E)] = np.inf
    sample = np.concatenate([odd, [0, 1, 2, 3, 4, T - 5, T - 4, T - 3, T - 2, T - 1], rng.choice(T, 60)])
    for dt in (torch.float32, torch.bfloat16):
        t = torch.from_numpy(l).cuda().to(dt)
        host = t.float().cpu().numpy()
        for kw in [dict(score="sigmoid", scale=2.5), dict(score="softmax", renorm=False)]:
            for bias in (None, bias_of(E, 3, 0.05 if kw["score"] == "sigmoid" else 0.2 / E)):
                kw.update(n_groups=n, top_groups=top, group_score="sum2" if E // n >= 2 and bias is not None else "best")
                idx, w = call(t, k, bias, **kw)
                ridx, rw = route_rule(host[sample], k, bias=bias, **kw)
                assert np.array_equal(idx[sample], ridx)
                np.testing.assert_allclose(w[sample], rw, rtol=W_TOL if kw["score"] == "sigmoid" else W_TOL_PLAIN_SOFTMAX, atol=1e-37)
                for t0 in range(0, T, 1000):
                    part = t[t0:t0 + 1000].contiguous()
                    i2, w2 = call(part, k, bias, **kw)
                    assert np.array_equal(idx[t0:t0 + 1000], i2)
                    np.testing.assert_allclose(w[t0:t0 + 1000], w2, rtol=2 * W_TOL_PLAIN_SOFTMAX, atol=1e-37)


@pytest.mark.parametrize("T", [9000, 20000])
def test_large_batches_with_odd_biases(T):
    """Biases that are not finite, and rows masked with the type's lowest value."""
    E, k = 128, 6
    l = logits_of(T, E, T)
    l[::7, 40:] = np.finfo(np.float32).min
    bias = bias_of(E, 9)
    bias[[3, 8, 50]] = [np.nan, -np.inf, np.inf]
    sample = np.r_[0:64, T - 40:T]
    for kw in [dict(score="sigmoid"), dict(score="softmax"), dict(score="sigmoid", n_groups=8, top_groups=3, group_score="sum2")]:
        idx, w = call(l, k, bias, **kw)
        ridx, rw = route_rule(l[sample], k, bias=bias, **kw)
        assert np.array_equal(idx[sample], ridx)
        np.testing.assert_allclose(w[sample], rw, rtol=W_TOL, atol=1e-37)


def test_bf16_logits_with_many_ties():
    for E, k, kw in [(160, 6, dict(n_groups=8, top_groups=3)), (512, 10, {}), (256, 8, dict(n_groups=8, top_groups=4, group_score="sum2"))]:
        t = torch.from_numpy(logits_of(400, E, 9)).cuda().to(torch.bfloat16)
        coarse = (t * 2).round() / 2  # a handful of values: hundreds of ties, and more of them than lanes
        for l in (t, coarse):
            for score in ("softmax", "sigmoid"):
                check(l, k, None, score=score, **kw)
                check(l, k, bias_of(E, 3), score=score, **kw)
                check(l, k, np.zeros(E, np.float32), score=score, **kw)


def test_row_strides_and_unaligned_rows():
    for dt in (torch.float32, torch.bfloat16):
        for ld, off in [(300, 0), (301, 0), (300, 1), (304, 3)]:
            base = torch.from_numpy(logits_of(40, ld + 8, 11)).cuda().to(dt)
            view = base.flatten()[off:off + 39 * ld + 256].as_strided((39, 256), (ld, 1))
            check(view, 8, bias_of(256, 2), score="sigmoid", n_groups=8, top_groups=4, group_score="sum2")


def test_masked_and_extreme_logits():
    """Rows whose mask leaves nothing, or fewer than k; the type's lowest value as
    a mask; infinities and NaN; scores that underflow; equal rows."""
    E, k = 64, 6
    base = logits_of(16, E, 21)
    rows = base.copy()
    rows[0] = -np.inf
    rows[1] = np.nan
    rows[2, 3:] = -np.inf
    rows[3] = -np.inf
    rows[3, [60, 2, 33]] = [0.5, -3.0, 0.5]
    rows[4, 5:] = np.finfo(np.float32).min
    rows[5] = np.finfo(np.float32).min
    rows[6, 7] = np.inf
    rows[7, [9, 4]] = np.inf
    rows[7, 2] = np.finfo(np.float32).max
    rows[8, ::2] = np.nan
    rows[9] = 0.0
    rows[10] = -200 + base[10]   # every sigmoid below fp32's smallest
    rows[11] = 60 + base[11]     # every sigmoid rounds to one
    rows[12] = 1e30 * base[12]
    rows[13, 10:] = -1e9
    rows[14] = -88.5 + 0.01 * base[14]
    for kw in [dict(), dict(n_groups=8, top_groups=2), dict(n_groups=8, top_groups=4, group_score="sum2")]:
        for score in ("softmax", "sigmoid"):
            for renorm in (True, False):
                check(rows, k, None, score=score, renorm=renorm, **kw)
                # with a bias the 64-bit scores decide; the rows whose scores it
                # cannot tell apart tie there too
                check(np.delete(rows, [10, 11, 12, 14], axis=0), k, bias_of(E, 5), score=score, renorm=renorm, **kw)
    bias = bias_of(E, 6)
    bias[[3, 8, 9]] = [np.nan, -np.inf, np.inf]
    check(base, k, bias, score="sigmoid")
    bias[11] = np.inf
    check(base, k, bias, score="softmax", n_groups=8, top_groups=4, group_score="sum2")
    rows[15, 20:] = -np.inf
    rows[15, :3] = np.nan
    check(rows[15:], k, None, score="sigmoid", n_groups=8, top_groups=4, group_score="sum2")
    check(rows[15:], k, None, score="softmax", n_groups=8, top_groups=4, group_score="sum2")
    huge = np.zeros(E, np.float32)
    huge[::3] = 3e38
    check(base, k, huge, score="sigmoid")


def test_zeros_of_either_sign_tie():
    l = np.full((3, 64), -1.0, np.float32)
    l[:, [3, 10, 11, 40]] = [0.0, -0.0, 0.0, -0.0]
    l[1] = -l[1] * 0
    for bias in (None, np.zeros(64, np.float32)):
        check(l, 4, bias)
        check(l, 2, bias, score="sigmoid", n_groups=4, top_groups=2)


def test_near_ties_are_decided_in_64_bits():
    """Values that differ by less than fp32 can tell: sigmoid scores of large
    logits and biases that cancel them, inside a group's boundary too."""
    rng = np.random.default_rng(31)
    E, T = 128, 200
    l = (6 + 6 * rng.random((T, E))).astype(np.float32)  # scores 1 - 2e-3 .. 1 - 6e-6
    check(l, 8, bias_of(E, 1, 1e-7), score="sigmoid")
    check(l, 8, bias_of(E, 1, 1e-7), score="sigmoid", n_groups=8, top_groups=3, group_score="sum2")
    check(l, 8, None, score="sigmoid", n_groups=8, top_groups=3, group_score="sum2")
    # pairs one ulp apart, the bias the same
    l2 = logits_of(T, E, 32)
    l2[:, 1::2] = np.nextafter(l2[:, ::2], np.float32(np.inf))
    for kw in [dict(score="sigmoid"), dict(score="softmax"), dict(score="softmax", n_groups=4, top_groups=2, group_score="sum2")]:
        check(l2, 9, np.full(E, 0.125, np.float32), **kw)
        check(l2, 9, None, **kw)


def test_softmax_pairs_that_only_their_own_bound_tells_apart():
    """Softmax values a few units of 2^-24 apart: with equal biases (the sum's
    error is common and tells nothing), with biases that cancel the scores, with
    large biases."""
    rng = np.random.default_rng(33)
    T, E = 400, 64
    l = logits_of(T, E, 34, 1.0)
    top = np.argsort(-l, 1)[:, :2]
    rows = np.arange(T)
    for ulps in (1, 2, 5, 20):  # the two largest logits of a row, some units apart
        x = l.copy()
        x[rows, top[:, 1]] = x[rows, top[:, 0]] * (1 - ulps * np.float32(2.0 ** -23))
        check(x, 8, np.zeros(E, np.float32))
        check(x, 8, np.full(E, 3.0, np.float32))
        check(x, 8, (1e-7 * rng.standard_normal(E)).astype(np.float32), renorm=False)
    p = np.exp(l[0].astype(np.float64) - l[0].max())
    p /= p.sum()
    b = (0.25 - p + 1e-9 * rng.standard_normal(E)).astype(np.float32)  # row 0: all values near 1/4
    check(l, 8, b)
    check(np.tile(l[:1], (9000, 1)) + 1e-6 * rng.standard_normal((9000, 1)).astype(np.float32), 8, b)


def test_bias_cancels_the_score():
    """A bias that turns every value into nearly the same number: more close
    candidates than lanes."""
    E = 256
    l = np.tile(logits_of(1, E, 41), (3, 1))
    s = 1 / (1 + np.exp(-l[0].astype(np.float64)))
    check(l, 8, (0.5 - s).astype(np.float32), score="sigmoid")
    check(l, 8, (0.5 - s).astype(np.float32), score="sigmoid", n_groups=8, top_groups=4, group_score="sum2")


@pytest.mark.parametrize("T", [0, 1, 2, 3, 5, 127, 4096])
def test_token_counts(T):
    check(logits_of(T, 256, 50 + T), 8, bias_of(256, 7), score="sigmoid", n_groups=8, top_groups=4, group_score="sum2")


def test_streams_graph_and_two_calls_at_once():
    E, k, T = 256, 8, 300
    kw = dict(score="sigmoid", n_groups=8, top_groups=4, group_score="sum2", scale=2.5)
    rule = qe.make_routing(**kw)
    bias = bias_of(E, 60)
    b = torch.from_numpy(bias).cuda()
    ins = [torch.from_numpy(logits_of(T, E, 61 + i)).cuda() for i in range(2)]
    outs = [(torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()

    def go(i, s):
        qe.strata_moe_route_logits(rule, ins[i].data_ptr(), qe.STRATA_F32, E, b.data_ptr(), T, E, k,
                                   outs[i][0].data_ptr(), outs[i][1].data_ptr(), s.cuda_stream)

    for _ in range(20):
        for i in range(2):
            go(i, streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        ridx, rw = route_rule(ins[i].cpu().numpy(), k, bias=bias, **kw)
        assert np.array_equal(outs[i][0].cpu().numpy(), ridx)
        np.testing.assert_allclose(outs[i][1].cpu().numpy(), rw, rtol=W_TOL)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go(0, torch.cuda.current_stream())
    ins[0].copy_(torch.from_numpy(logits_of(T, E, 70)))
    g.replay()
    torch.cuda.synchronize()
    ridx, _ = route_rule(ins[0].cpu().numpy(), k, bias=bias, **kw)
    assert np.array_equal(outs[0][0].cpu().numpy(), ridx)


# ------------------------------------------------------------------ layers
LAYER_RULES = [dict(score="sigmoid", n_groups=8, top_groups=4, group_score="sum2", scale=2.5),
               dict(score="softmax", renorm=False, n_groups=4, top_groups=3)]


def layer_with_rule(shape, T, kw, seed=0, bias=True):
    layer = gen.layer_weights(shape, seed=seed)
    L = qe.Layer(layer, max_tokens=T)
    sb = bias_of(shape.n_experts, seed, 0.05 if kw["score"] == "sigmoid" else 0.2 / shape.n_experts) if bias else None
    L.set_routing(qe.make_routing(**kw), sb)
    return layer, L, sb


def rule_reference(layer, x_bits, kw, sb):
    logits = oracle.router_logits(x_bits, layer.router_w, layer.router_b, threads=THREADS)
    return route_rule(logits, layer.shape.top_k, bias=sb, **kw)


@pytest.mark.parametrize("kw", LAYER_RULES, ids=["sigmoid-groups", "softmax-plain"])
@pytest.mark.parametrize("shape,T", [(gen.TINY, 1), (gen.TINY, 8), (gen.TINY, 70), (gen.TINY, 1025), (gen.FLASH2, 4), (gen.FLASH2, 300), (gen.FLASH2, 1100),
                                     (gen.LayerShape(hidden=384, n_experts=40, top_k=3, inter=32, router_bias=True), 1031)],
                         ids=["tiny-1", "tiny-8", "tiny-70", "tiny-1025", "flash-4", "flash-300", "flash-1100", "odd-1031"])
def test_layer_routes_by_its_rule(shape, T, kw):
    layer, L, sb = layer_with_rule(shape, T, kw)
    x = gen.hidden(T, shape.hidden, seed=5)
    idx, w, off, lst = L.route(to_dev_bf16(x))
    ridx, rw = rule_reference(layer, x, kw, sb)
    assert np.array_equal(idx.cpu().numpy(), ridx)
    np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=W_TOL if kw.get("renorm", True) else W_TOL_PLAIN_SOFTMAX)
    _, roff, rlst, _ = oracle.dispatch(ridx, shape.n_experts)
    assert np.array_equal(off.cpu().numpy(), roff) and np.array_equal(lst.cpu().numpy(), rlst)
    # back to the default rule
    L.set_routing(None)
    oidx, ow = oracle.route(oracle.router_logits(x, layer.router_w, layer.router_b, threads=THREADS), shape.top_k)
    idx, w, _, _ = L.route(to_dev_bf16(x))
    assert np.array_equal(idx.cpu().numpy(), oidx)
    L.sync_status()
    L.close()


def forward_reference(layer, x_bits, idx, w, tokens):
    s = layer.shape
    xf = npref.bf16_bits_to_f64(x_bits)
    cb, sb = 3 * s.mat_code_bytes, 3 * s.mat_scales
    shared = npref.expert_mats(s, layer.shared_codes, layer.shared_scales)
    mats = {}
    out = []
    for t in tokens:
        y = npref.swiglu(shared, xf[t])
        for j in np.argsort(idx[t], kind="stable"):
            e = int(idx[t, j])
            if e not in mats:
                mats[e] = npref.expert_mats(s, layer.codes[e * cb:(e + 1) * cb], layer.scales[e * sb:(e + 1) * sb])
            y = y + w[t, j] * npref.swiglu(mats[e], xf[t])
        out.append(y)
    return np.array(out)


@pytest.mark.parametrize("kw", LAYER_RULES, ids=["sigmoid-groups", "softmax-plain"])
@pytest.mark.parametrize("shape,T", [(gen.TINY, 1), (gen.TINY, 9), (gen.TINY, 70), (gen.TINY, 300), (gen.TINY, 1100), (gen.FLASH2, 4)],
                         ids=["tiny-1", "tiny-9", "tiny-70", "tiny-300", "tiny-1100", "flash-4"])
def test_layer_forward_by_its_rule(shape, T, kw):
    layer, L, sb = layer_with_rule(shape, T, kw, seed=2)
    x = gen.hidden(T, shape.hidden, seed=6)
    xd = to_dev_bf16(x)
    y = L.forward(xd)
    ridx, rw = rule_reference(layer, x, kw, sb)
    tokens = list(range(T))[::max(1, T // 100)] if shape is gen.TINY else [0, T - 1]
    check_output(from_dev_bf16(y)[tokens], forward_reference(layer, x, ridx, rw, tokens))
    assert torch.equal(L.forward(xd), y), "two forwards differ"
    # a captured forward keeps working on new tokens
    g = torch.cuda.CUDAGraph()
    out = torch.empty_like(xd)
    with torch.cuda.graph(g):
        L.forward(xd, out=out, stream=torch.cuda.current_stream())
    x2 = gen.hidden(T, shape.hidden, seed=7)
    xd.copy_(to_dev_bf16(x2))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, L.forward(xd))
    L.sync_status()
    del g
    L.close()


@pytest.mark.parametrize("kw", LAYER_RULES + [dict(score="sigmoid", renorm=False), dict(score="softmax", n_groups=8, top_groups=2)],
                         ids=["sigmoid-groups", "softmax-plain", "sigmoid-plain", "softmax-groups"])
@pytest.mark.parametrize("shape,T", [(gen.TINY, 3), (gen.TINY, 9), (gen.TINY, 17), (gen.TINY, 64), (gen.FLASH2, 1), (gen.FLASH2, 4),
                                     (gen.FLASH2, 16), (gen.FLASH2, 64), (gen.FLASH3, 8), (gen.CODER1, 5)],
                         ids=["tiny-3", "tiny-9", "tiny-17", "tiny-64", "flash2-1", "flash2-4", "flash2-16", "flash2-64", "flash3-8", "coder1-5"])
def test_single_launch_decode_by_rule(shape, T, kw):
    """The fused decode kernel picks by the rule too: one launch, and the kernel
    chain's output on the same routing within the layer tolerance."""
    for bias in (True, False):
        layer, L, sb = layer_with_rule(shape, T, kw, seed=4, bias=bias)
        x = to_dev_bf16(gen.hidden(T, shape.hidden, seed=12))
        L.set_option(qe.STRATA_OPT_PATH, 3)
        assert qe.strata_moe_launch_count(L.handle, T) == 1
        y = L.forward(x)
        assert torch.equal(L.forward(x), y)
        L.sync_status()
        L.set_option(qe.STRATA_OPT_PATH, 1)
        ref = npref.bf16_bits_to_f64(from_dev_bf16(L.forward(x)))
        check_output(from_dev_bf16(y), ref)
        L.sync_status()
        L.close()


def test_rules_the_fused_kernel_does_not_hold_take_the_chain():
    shape = gen.LayerShape(hidden=256, n_experts=510, top_k=3, inter=128)
    kw = dict(score="sigmoid", n_groups=17, top_groups=3, group_score="sum2")
    layer, L, sb = layer_with_rule(shape, 5, kw, seed=1)
    x = gen.hidden(5, shape.hidden, seed=3)
    xd = to_dev_bf16(x)
    assert qe.strata_moe_launch_count(L.handle, 5) == 9
    y = L.forward(xd)
    ridx, rw = rule_reference(layer, x, kw, sb)
    check_output(from_dev_bf16(y), forward_reference(layer, x, ridx, rw, range(5)))
    L.set_option(qe.STRATA_OPT_PATH, 3)
    with pytest.raises(qe.StrataError) as e:
        L.forward(xd)
    assert e.value.status == qe.STRATA_ERR_INVALID_ARG
    # a stack refuses before it touches its rows
    first = qe.Layer(layer, max_tokens=5)
    first.set_option(qe.STRATA_OPT_PATH, 3)
    h = xd.clone()
    with pytest.raises(qe.StrataError) as e:
        qe.strata_moe_stack_forward([first.handle, L.handle], h.data_ptr(), 5)
    assert e.value.status == qe.STRATA_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert torch.equal(h, xd)
    first.close()
    L.set_option(qe.STRATA_OPT_PATH, 0)
    assert torch.equal(L.forward(xd), y)
    L.sync_status()
    L.close()


def test_default_rule_given_explicitly_matches_the_default():
    """softmax, no groups, renormalised: the same picks as without a rule."""
    shape, T = gen.FLASH2, 64
    layer = gen.layer_weights(shape, seed=3)
    L = qe.Layer(layer, max_tokens=T)
    x = to_dev_bf16(gen.hidden(T, shape.hidden, seed=8))
    idx0, w0, off0, lst0 = L.route(x)
    L.set_routing(qe.make_routing())
    idx1, w1, off1, lst1 = L.route(x)
    assert torch.equal(idx0, idx1) and torch.equal(off0, off1) and torch.equal(lst0, lst1)
    np.testing.assert_allclose(w1.cpu().numpy(), w0.cpu().numpy(), rtol=2 * W_TOL)
    L.close()


def test_stack_uses_every_layer_s_own_rule():
    shape, T = gen.TINY, 12
    layers, Ls, sbs = [], [], []
    kws = [LAYER_RULES[0], None, LAYER_RULES[1]]
    for i, kw in enumerate(kws):
        if kw is None:
            layers.append(gen.layer_weights(shape, seed=10 + i))
            Ls.append(qe.Layer(layers[-1], max_tokens=T))
            sbs.append(None)
        else:
            layer, L, sb = layer_with_rule(shape, T, kw, seed=10 + i)
            layers.append(layer), Ls.append(L), sbs.append(sb)
    h0 = gen.hidden(T, shape.hidden, seed=9)
    h = to_dev_bf16(h0)
    trace = torch.empty((3, T, shape.hidden), dtype=torch.bfloat16, device="cuda")
    qe.strata_moe_stack_forward([L.handle for L in Ls], h.data_ptr(), T, trace.data_ptr())
    Ls[0].sync_status()
    ins = [from_dev_bf16(trace[i]) for i in range(3)] + [from_dev_bf16(h)]
    for i, kw in enumerate(kws):
        xn = oracle.rmsnorm(ins[i])
        if kw is None:
            logits = oracle.router_logits(xn, layers[i].router_w, layers[i].router_b)
            idx, w = oracle.route(logits, shape.top_k)
        else:
            idx, w = rule_reference(layers[i], xn, kw, sbs[i])
        y = forward_reference(layers[i], xn, idx, w, range(T))
        ref = npref.bf16_bits_to_f64(ins[i]) + y
        # the residual addition rounds twice more (bf16, half a step of 2^-8 each)
        got = npref.bf16_bits_to_f64(ins[i + 1])
        assert np.abs(got - ref).max() <= 2e-2 * np.abs(y).max() + 2 * 2.0 ** -8 * np.abs(ref).max()
    for L in Ls:
        L.close()


def test_set_routing_keeps_the_old_rule_when_refused_and_counts_launches():
    shape = gen.TINY
    layer, L, sb = layer_with_rule(shape, 8, LAYER_RULES[0])
    x = to_dev_bf16(gen.hidden(8, shape.hidden, seed=1))
    before = L.route(x)
    for bad in (qe.make_routing(n_groups=3, top_groups=1), qe.make_routing(n_groups=16, top_groups=1)):
        with pytest.raises(qe.StrataError) as e:
            L.set_routing(bad)
        assert e.value.status == qe.STRATA_ERR_INVALID_ARG
    with pytest.raises(qe.StrataError):
        L.set_routing(None, np.zeros(shape.n_experts, np.float32))
    after = L.route(x)
    assert all(torch.equal(a, b) for a, b in zip(before, after))
    L.close()
    live = qe.strata_moe_debug_live_allocs()
    layer, L, sb = layer_with_rule(shape, 8, LAYER_RULES[0])
    L.set_routing(qe.make_routing(), sb)  # a second bias reuses the first one's memory
    L.close()
    assert qe.strata_moe_debug_live_allocs() == live
    L = qe.Layer(layer, max_tokens=8)
    qe.strata_moe_debug_fail_alloc(0)
    with pytest.raises(qe.StrataError) as e:
        L.set_routing(qe.make_routing(), sb)
    qe.strata_moe_debug_fail_alloc(-1)
    assert e.value.status == qe.STRATA_ERR_OOM
    L.close()


def triples(T, E, share, unit_gap, seed):
    """Rows and a bias with three values next to each other: experts 7 and 11 with
    scores near 0, `unit_gap` units of 2^-24 of the largest score apart, and
    expert 3, the row's most likely one (score about `share`) with a bias that
    cancels it, whose value lies above both by less than half a unit."""
    rng = np.random.default_rng(seed)
    unit = share * 2.0 ** -24
    l = rng.standard_normal((T, E))
    l[:, [7, 11]] = -200
    rest = np.delete(np.arange(E), [3, 7, 11])
    odds = np.exp(0.35) * (1 - share) / share  # sum of the others' exp for a logit of 0.35
    l[:, rest] += np.log(odds) - np.log(np.exp(l[:, rest]).sum(1, keepdims=True))
    l = l.astype(np.float32)
    l = np.minimum(l, np.float32(0.2))
    bias = np.full(E, -4.0, np.float32)
    low = np.float32(2.0 ** -9)
    bias[3] = np.float32(low - share)
    bias[7] = low
    bias[11] = np.float32(low - unit_gap * unit)
    others = l.astype(np.float64)
    others[:, 3] = -np.inf
    s = np.exp(others).sum(1)
    want = np.float64(low) - np.float64(bias[3]) + 0.02 * unit  # expert 3's score
    l[:, 3] = np.log(want * s / (1 - want))
    p = lambda: np.exp(l[:, 3].astype(np.float64)) / (s + np.exp(l[:, 3].astype(np.float64)))  # noqa: E731
    for _ in range(3):  # the first float at or above it
        under = p() < want
        l[under, 3] = np.nextafter(l[under, 3], np.float32(np.inf))
    ok = (p() >= want) & (p() - want < 0.4 * unit) & (l[:, 3] > l[:, rest].max(1))
    return l[ok], bias


@pytest.mark.parametrize("E,share", [(512, 0.4), (1024, 0.3), (512, 0.2), (160, 0.4)])
def test_softmax_values_behind_the_first_one_left_out(E, share):
    """A value that lies two places behind the last pick in fp32 and is the pick
    in 64 bits: its score's error is larger than that of the two before it."""
    for gap in (2.14, 2.2, 2.5, 3.0):
        l, bias = triples(20000, E, share, gap, E)
        T = l.shape[0]
        assert T > 8192
        for n in (T, 8191):  # several tokens a warp, and one
            idx, _ = call(l[:n], 1, bias)
            assert (idx == 3).all(), (n, gap, (idx != 3).sum())
            idx, _ = call(l[:n], 2, bias)
            assert (idx == [3, 7]).all(), (n, gap, (idx != [3, 7]).any(1).sum())
            idx, _ = call(l[:n], 3, bias)
            assert (idx == [3, 7, 11]).all(), (n, gap)


@pytest.mark.parametrize("T", [1, 9001, 17001])
def test_infinite_and_largest_logits_tie_between_groups(T):
    """+inf counts as the largest finite float in the choice of groups as well: a
    tie there goes to the lower group."""
    E, big = 64, np.finfo(np.float32).max
    l = logits_of(T, E, 80)
    l[::2, 10] = big            # group 1 of 8
    l[::2, 45] = np.inf         # group 5
    l[1::2, 3] = np.inf
    l[1::2, 60] = big
    sample = np.unique(np.r_[0:min(T, 40), max(0, T - 40):T])
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            for top in (1, 2):
                for gsc in ("best", "sum2"):
                    kw = dict(score=score, renorm=renorm, n_groups=8, top_groups=top, group_score=gsc)
                    idx, w = call(l, 3, None, **kw)
                    ridx, rw = route_rule(l[sample], 3, **kw)
                    assert np.array_equal(idx[sample], ridx), kw
                    np.testing.assert_allclose(w[sample], rw, rtol=W_TOL_PLAIN_SOFTMAX, atol=1e-37)


@pytest.mark.parametrize("E", [64, 256])
def test_a_token_s_weights_do_not_depend_on_its_neighbours(E):
    """Tokens with scores near fp32's smallest next to ordinary ones, several
    tokens a warp: the ordinary ones keep their bits."""
    k = 6
    for T in (9001, 17001):
        l = logits_of(T, E, 90)
        odd = l.copy()
        odd[::3] -= 95
        for score in ("sigmoid", "softmax"):
            for bias in (None, bias_of(E, 8, 0.2 / E)):
                for renorm in (True, False):
                    kw = dict(score=score, renorm=renorm)
                    if score == "softmax" and bias is not None:
                        # one expert takes all, and the bias picks others
                        odd = l.copy()
                        odd[::3, 5] += 120
                        bias[5] = -2
                    idx, w = call(l, k, bias, **kw)
                    i2, w2 = call(odd, k, bias, **kw)
                    keep = np.arange(T) % 3 != 0
                    assert np.array_equal(idx[keep], i2[keep]) and np.array_equal(w[keep], w2[keep]), kw


@pytest.mark.parametrize("T", [16, 9001, 17001])
def test_extreme_logits_with_a_bias(T):
    """Scores that underflow, that all round to one, or of which one takes all,
    where the bias then decides."""
    E, k = 64, 6
    rows = logits_of(T, E, 21)
    for i, t in enumerate((0, 1, 2, 3, 4, 5, 6, T - 2, T - 1)):
        base = rows[t].copy()
        rows[t] = [-200 + base, 60 + base, np.float32(1e30) * base, -88.5 + np.float32(0.01) * base, 17 + base, -17 + base,
                   np.float32(-1e30) * np.abs(base), np.full(E, 5.0), 1e-30 * base][i]
    sample = np.unique(np.r_[0:14, T - 12:T])
    sizes = {"large": bias_of(E, 5, 0.05), "equal": np.full(E, 0.25, np.float32), "none": np.zeros(E, np.float32),
             "tiny": bias_of(E, 6, 1e-9)}
    for groups in [dict(), dict(n_groups=8, top_groups=2), dict(n_groups=8, top_groups=4, group_score="sum2")]:
        for score in ("softmax", "sigmoid"):
            for renorm in (True, False):
                for name, bias in sizes.items():
                    kw = dict(score=score, renorm=renorm, **groups)
                    idx, w = call(rows, k, bias, **kw)
                    ridx, rw = route_rule(rows[sample], k, bias=bias, **kw)
                    assert np.array_equal(idx[sample], ridx), (kw, name, sample[np.any(idx[sample] != ridx, axis=1)])
                    np.testing.assert_allclose(w[sample], rw, rtol=W_TOL if score == "sigmoid" or renorm else W_TOL_PLAIN_SOFTMAX,
                                               atol=1e-37)


@pytest.mark.parametrize("T", [5, 9001, 17001])
def test_any_scale(T):
    """Factors near either end of fp32's range, with scores that sum to little."""
    E, k = 64, 4
    l = logits_of(T, E, 95)
    l[1::2] -= 40
    sample = np.unique(np.r_[0:min(T, 30), max(0, T - 30):T])
    for score in ("softmax", "sigmoid"):
        for bias in (None, bias_of(E, 96, 0.2 / E)):
            for scale in (3e38, 1e25, -1e25, 1e-30, 0.0):
                kw = dict(score=score, scale=scale)
                idx, w = call(l, k, bias, **kw)
                ridx, rw = route_rule(l[sample], k, bias=bias, **dict(kw, scale=float(np.float32(scale))))
                assert np.array_equal(idx[sample], ridx)
                np.testing.assert_allclose(w[sample], rw, rtol=W_TOL, atol=1e-37)


@pytest.mark.parametrize("T", [1100, 8200])
def test_logits_past_32_bits(T):
    """Rows of logits that lie further than 2^32 bytes from the first."""
    E, k = 64, 6
    ld = (1 << 30) // (T - 20) // 4 * 4 + 4
    l = logits_of(T, E, 99)
    flat = torch.zeros((T - 1) * ld + E, device="cuda")
    view = flat.as_strided((T, E), (ld, 1))
    view.copy_(torch.from_numpy(l))
    assert (T - 1) * ld * 4 > 1 << 32
    idx, w = call(view, k, bias_of(E, 4), score="sigmoid")
    i2, w2 = call(l, k, bias_of(E, 4), score="sigmoid")
    assert np.array_equal(idx, i2) and np.array_equal(w, w2)


@pytest.mark.parametrize("T", [3, 9001, 17001])
def test_small_weights_next_to_small_sums(T):
    """Renormalised weights keep their relative accuracy where the picks' scores sum
    to little and differ by many powers of two (down to 2^-106 of the sum, where
    scores leave fp32's normal range: 1e-31 covers it)."""
    E, k = 64, 5
    l = np.full((T, E), -300, np.float32)
    rng = np.random.default_rng(98)
    step = np.log(2) * np.array([0, -25, -50, -70, -85])
    for t in range(T):
        l[t, 10:15] = step - (t % 62) * np.log(2) - rng.random(5)
    bias = np.full(E, -4.0, np.float32)
    bias[10:15] = [0.5, 0.4, 0.3, 0.2, 0.1]
    soft = l.copy()
    soft[:, 40] = 0.5  # takes nearly all of the softmax and is not picked
    sample = np.unique(np.r_[0:min(T, 62), max(0, T - 62):T])
    for score, rows, b in (("softmax", soft, bias), ("sigmoid", l, bias), ("sigmoid", l, None)):
        idx, w = call(rows, k, b, score=score)
        ridx, rw = route_rule(rows[sample], k, bias=b, score=score)
        assert np.array_equal(idx[sample], ridx)
        np.testing.assert_allclose(w[sample], rw, rtol=2 * W_TOL, atol=1e-31)
