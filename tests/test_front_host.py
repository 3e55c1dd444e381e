"""Refusals of the routing-rule and 8-bit-row entry points (no GPU needed):
every bad argument comes back as an error before the device is touched, and
host memory is refused where device memory is due."""
import ctypes as C

import numpy as np
import pytest

import quantized_expert_ffn_04_b200 as qe

INV = qe.STRATA_ERR_INVALID_ARG
P = 1 << 20  # an aligned pointer that is never dereferenced: each call below is refused


def refused(fn, *args):
    with pytest.raises(qe.StrataError) as e:
        fn(*args)
    assert e.value.status == INV
    assert str(e.value).count("strata_moe_") == 1  # the message names the call


def rule(**kw):
    return qe.make_routing(**kw)


def route(r, logits=P, typ=qe.STRATA_F32, ld=64, bias=None, T=4, E=64, k=4, idx=8 * P, w=9 * P):
    qe.strata_moe_route_logits(r, logits, typ, ld, bias, T, E, k, idx, w)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(E=0, ld=64), dict(E=1025, ld=1025), dict(k=0), dict(k=33), dict(E=4, k=5),
    dict(typ=2), dict(ld=63), dict(logits=None), dict(idx=None), dict(w=None),
    dict(logits=P + 2), dict(logits=P + 1, typ=qe.STRATA_BF16), dict(bias=P + 2), dict(idx=P + 1),
    dict(w=P + 3), dict(ld=1 << 61), dict(idx=P + 64), dict(w=P + 960), dict(idx=8 * P, w=8 * P + 60), dict(bias=16 * P, w=16 * P),
    dict(bias=8 * P + 60),
], ids=str)
def test_route_logits_refuses(kw):
    refused(lambda: route(rule(), **kw))


@pytest.mark.parametrize("r", [
    dict(n_groups=0, top_groups=1), dict(n_groups=33, top_groups=1), dict(n_groups=3, top_groups=1),
    dict(n_groups=4, top_groups=5), dict(n_groups=4, top_groups=0), dict(n_groups=32, top_groups=1),
    dict(scale=float("nan")), dict(scale=float("inf")),
], ids=str)
def test_route_logits_refuses_rules(r):
    refused(lambda: route(rule(**r)))


def test_route_logits_refuses_unknown_fields():
    for field, v in [("score", 2), ("score", -1), ("group_score", 2), ("renorm", 2)]:
        r = rule()
        setattr(r, field, v)
        refused(lambda: route(r))
    r = rule(n_groups=32, top_groups=32, group_score="sum2")
    refused(lambda: route(r, E=32, ld=32))  # groups of one
    refused(lambda: route(None))


def test_no_tokens_is_a_no_op_and_host_memory_is_refused():
    route(rule(), T=0, logits=None, idx=None, w=None)
    a = np.zeros(1024, np.float32)
    p = a.ctypes.data + (-a.ctypes.data) % 16
    refused(lambda: route(rule(), logits=p, T=1))


def test_make_routing_and_struct_layout():
    assert C.sizeof(qe.strata_moe_routing) == 24
    r = qe.make_routing("sigmoid", 8, 4, "sum2", renorm=True, scale=2.5)
    assert (r.score, r.n_groups, r.top_groups, r.group_score, r.renorm, r.scale) == (1, 8, 4, 1, 1, 2.5)
    assert qe.make_routing(n_groups=4).top_groups == 4
    with pytest.raises(ValueError):
        qe.make_routing("tanh")
    with pytest.raises(ValueError):
        qe.make_routing(group_score="mean")


def test_set_routing_refuses_null_handle():
    assert qe._lib.strata_moe_set_routing(None, None, None) == INV


def norm(x=P, delta=None, weight=None, wt=qe.STRATA_F32, eps=1e-6, T=2, H=256, h=None, xn=8 * P,
         q8=qe.STRATA_Q8_E4M3, group=128, q=None, qs=256, scale=None, ss=2):
    qe.strata_moe_add_rmsnorm(x, delta, weight, wt, eps, T, H, h, xn, q8, group, q, qs, scale, ss)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(H=0), dict(H=48), dict(H=16416), dict(wt=2), dict(eps=-1e-6),
    dict(eps=float("nan")), dict(eps=float("inf")), dict(x=None), dict(xn=None),
    dict(delta=2 * P), dict(x=P + 8), dict(weight=P // 2 + 4), dict(xn=8 * P + 2),
    dict(q=4 * P), dict(q=4 * P, scale=5 * P, q8=2), dict(q=4 * P, scale=5 * P, group=16),
    dict(q=4 * P, scale=5 * P, group=-32), dict(q=4 * P, scale=5 * P, H=288, group=64, qs=288, ss=8),
    dict(q=4 * P, scale=5 * P, qs=240), dict(q=4 * P, scale=5 * P, qs=264),
    dict(q=4 * P, scale=5 * P, ss=1), dict(q=4 * P + 8, scale=5 * P), dict(q=4 * P, scale=5 * P + 4),
    dict(q=4 * P, scale=5 * P, qs=1 << 60), dict(q=4 * P, scale=5 * P, ss=1 << 60),
    # overlaps: xn on x, h half on x, q on xn, scales on codes without a packed row
    dict(xn=P), dict(h=P + 512, delta=2 * P), dict(q=8 * P + 512, scale=5 * P),
    dict(q=4 * P, scale=4 * P + 256, qs=256), dict(h=8 * P, delta=2 * P),
], ids=str)
def test_add_rmsnorm_refuses(kw):
    refused(lambda: norm(**kw))


def test_add_rmsnorm_host_memory():
    norm(T=0, x=None, xn=None)
    a = np.zeros(8192, np.float32)
    p = a.ctypes.data + (-a.ctypes.data) % 16
    # in place and a packed row (scales behind the codes) pass every check but this last one
    with pytest.raises(qe.StrataError, match="not device memory"):
        norm(x=p, delta=2 * P, h=p)
    with pytest.raises(qe.StrataError, match="not device memory"):
        norm(x=p, q=4 * P, qs=272, scale=4 * P + 256, ss=68)


def dequant(q=P, q8=qe.STRATA_Q8_INT8, qs=256, scale=2 * P, ss=2, group=128, rows=None, n=2, n_src=2,
            H=256, out=3 * P):
    qe.strata_moe_dequant_rows(q, q8, qs, scale, ss, group, rows, n, n_src, H, out)


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(n_src=-1), dict(H=0), dict(H=40), dict(H=65568, qs=65568, ss=600), dict(q8=2),
    dict(group=8), dict(H=288, qs=288, ss=8, group=64), dict(qs=240), dict(qs=260), dict(ss=1), dict(n=3),
    dict(q=None), dict(scale=None), dict(out=None), dict(q=P + 4), dict(out=3 * P + 8),
    dict(scale=2 * P + 2), dict(rows=4 * P + 2), dict(out=P + 256), dict(out=2 * P),
    dict(rows=3 * P), dict(qs=1 << 60), dict(ss=1 << 61),
], ids=str)
def test_dequant_rows_refuses(kw):
    refused(lambda: dequant(**kw))


def test_dequant_rows_no_ops_and_host_memory():
    dequant(n=0, q=None, scale=None, out=None)
    dequant(n_src=0, n=5, rows=4 * P)  # every row is outside
    a = np.zeros(1024, np.float32)
    p = a.ctypes.data + (-a.ctypes.data) % 16
    with pytest.raises(qe.StrataError, match="not device memory"):
        dequant(q=p)


def test_tensor_functions_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    for bad in [lambda: qe.add_rmsnorm(x), lambda: qe.route_logits(torch.zeros(2, 64), rule(), 4),
                lambda: qe.dequant_rows(torch.zeros(2, 272, dtype=torch.uint8), 256)]:
        with pytest.raises(ValueError):
            bad()
    assert qe.packed_row_bytes(2560) == 2640 and qe.packed_row_bytes(256, 0) == 272 and qe.packed_row_bytes(6144, 32) == 6912


def test_layer_set_routing_refuses_a_bias_of_another_length(monkeypatch):
    """The C call copies n_experts floats from the host: fewer would be read past
    their end."""
    import gen
    L = object.__new__(qe.Layer)
    L.handle, L.shape = None, gen.TINY
    seen = []
    monkeypatch.setattr(qe, "strata_moe_set_routing", lambda *a: seen.append(a))
    E = gen.TINY.n_experts
    for bad in (np.zeros(E - 1), np.zeros(E + 1), np.zeros((E, 2)), np.zeros((1, E)), 0.5, np.zeros(0)):
        with pytest.raises(ValueError, match=f"{E} values"):
            L.set_routing(rule(), bad)
    assert not seen
    L.set_routing(rule(), [0.0] * E)
    L.set_routing(rule(), np.zeros(E, np.float64)[::-1])
    L.set_routing(rule())
    L.set_routing()
    assert len(seen) == 4 and seen[1][2].shape == (E,) and seen[2][2] is None
