"""A block's front half on the GPU as it is used: pre-norm, routing by a rule,
8-bit rows, experts and combine, through the torch-tensor functions and through
ExpertParallel.forward_block (one rank, NCCL)."""
import datetime
import socket

import numpy as np
import pytest

import gen
import oracle
from tests import npref
from tests.front_ref import norm_rows, route_rule
from tests.gpu_util import check_output, from_dev_bf16, to_dev_bf16
from tests.test_gpu_rules import bias_of, forward_reference

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import quantized_expert_ffn_04_b200 as qe  # noqa: E402
from quantized_expert_ffn_04_b200.ep import ExpertParallel, GpuBackend  # noqa: E402

RULE = dict(score="sigmoid", n_groups=8, top_groups=4, group_score="sum2", scale=2.5)


def block_inputs(shape, T, seed):
    rng = np.random.default_rng(seed)
    h = to_dev_bf16(gen.hidden(T, shape.hidden, seed=seed))
    delta = torch.from_numpy((0.5 * rng.standard_normal((T, shape.hidden))).astype(np.float32)).cuda().to(torch.bfloat16)
    weight = torch.from_numpy((1 + 0.2 * rng.standard_normal(shape.hidden)).astype(np.float32)).cuda()
    return h, delta, weight


def rule_layer(shape, max_tokens, seed=0):
    layer = gen.layer_weights(shape, seed=seed)
    L = qe.Layer(layer, max_tokens=max_tokens)
    sb = bias_of(shape.n_experts, seed)
    L.set_routing(qe.make_routing(**RULE), sb)
    return layer, L, sb


@pytest.mark.parametrize("shape,T", [(gen.TINY, 1), (gen.TINY, 40), (gen.TINY, 130), (gen.FLASH2, 4)],
                         ids=["tiny-1", "tiny-40", "tiny-130", "flash-4"])
def test_pre_norm_then_layer(shape, T):
    """h + delta -> pre-norm -> the layer under its rule, against the 64-bit steps."""
    layer, L, sb = rule_layer(shape, T)
    h, delta, weight = block_inputs(shape, T, 3)
    h2, xn, packed = qe.add_rmsnorm(h, delta, weight, 1e-6, "e4m3", 128)
    y = L.forward(xn)
    L.sync_status()
    rh, ry = norm_rows(h.double().cpu().numpy(), delta.double().cpu().numpy(), weight.double().cpu().numpy(), 1e-6)
    assert np.array_equal(h2.double().cpu().numpy(), rh)
    xb = from_dev_bf16(xn)  # the layer is held to its own input
    assert (np.abs(npref.bf16_bits_to_f64(xb) - ry) <= (2.0 ** -8 + 4.7e-6) * np.abs(ry)).all()
    idx, w = route_rule(oracle.router_logits(xb, layer.router_w, layer.router_b), shape.top_k, bias=sb, **RULE)
    gi, gw = qe.route_logits(torch.from_numpy(oracle.router_logits(xb, layer.router_w, layer.router_b)).cuda(),
                             qe.make_routing(**RULE), shape.top_k, torch.from_numpy(sb).cuda())
    assert np.array_equal(gi.cpu().numpy(), idx)
    tokens = list(range(T)) if shape is gen.TINY else [0, T - 1]
    check_output(from_dev_bf16(y)[tokens], forward_reference(layer, xb, idx, w, tokens))
    # the packed rows read back: within e4m3's half step of the normalised rows
    back = qe.dequant_rows(packed, shape.hidden).double().cpu().numpy()
    scale = np.repeat(np.abs(ry.reshape(T, -1, 128)).max(2) / 448, 128, 1)
    assert (np.abs(back - ry) <= (2.0 ** -4 + 2.0 ** -8) * np.abs(ry) + scale * 2.0 ** -9).all()
    L.close()


@pytest.fixture(scope="module")
def one_rank():
    import torch.distributed as dist
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    dist.init_process_group("nccl", init_method=f"tcp://127.0.0.1:{port}", rank=0, world_size=1,
                            timeout=datetime.timedelta(seconds=60))
    yield
    dist.destroy_process_group()


@pytest.mark.parametrize("shape,T", [(gen.TINY, 5), (gen.TINY, 100), (gen.FLASH2, 4)], ids=["tiny-5", "tiny-100", "flash-4"])
def test_forward_block_equals_its_steps(one_rank, shape, T):
    k, H = shape.top_k, shape.hidden
    layer, L, sb = rule_layer(shape, T + T * k, seed=1)
    h, delta, weight = block_inputs(shape, T, 5)
    ep = ExpertParallel(GpuBackend(L), shape.n_experts, k, H)
    h2, y = ep.forward_block(h, delta, weight)
    L.sync_status()
    # the same steps through the entry points, without an exchange
    rh, xn, packed = qe.add_rmsnorm(h, delta, weight, 1e-6, "e4m3", 128)
    assert torch.equal(h2, rh)
    idx, w, _, _ = L.route(xn)
    ridx, _ = route_rule(oracle.router_logits(from_dev_bf16(xn), layer.router_w, layer.router_b), k, bias=sb, **RULE)
    assert np.array_equal(idx.cpu().numpy(), ridx)
    x = qe.dequant_rows(packed, H)
    prefill = T > 64
    yd = torch.float16 if prefill else torch.float32
    order = torch.arange(T, dtype=torch.int32, device="cuda").repeat_interleave(k)
    rows = torch.cat([x, qe.dequant_rows(packed, H, rows=order)])
    ids = torch.cat([torch.full((T,), -1, dtype=torch.int32, device="cuda"), idx.reshape(-1)])
    out = torch.empty((T + T * k, H), dtype=yd, device="cuda")
    Y = torch.empty((T * k + T, H), dtype=yd, device="cuda")
    qe.strata_moe_expert_rows(L.handle, rows.data_ptr(), ids.data_ptr(), T + T * k, T, prefill, out.data_ptr(), Y[T * k:].data_ptr())
    Y[:T * k] = out[T:]
    slot = torch.arange(T * k, dtype=torch.int32, device="cuda")
    ref = torch.empty_like(x)
    qe.strata_moe_combine_rows(L.handle, x.data_ptr(), T, idx.data_ptr(), w.data_ptr(), slot.data_ptr(), Y.data_ptr(), prefill, ref.data_ptr())
    L.sync_status()
    assert torch.equal(y, ref)
    tokens = list(range(T)) if shape is gen.TINY else [0, T - 1]
    check_output(from_dev_bf16(y)[tokens], forward_reference(layer, from_dev_bf16(x), idx.cpu().numpy(), w.double().cpu().numpy(), tokens))
    # the plain forward still sends bf16 rows
    assert torch.equal(ep.forward(xn), ep.forward(xn))
    L.sync_status()
    L.close()


def test_tensor_functions_refuse():
    x = torch.randn(4, 256, device="cuda").to(torch.bfloat16)
    r = qe.make_routing()
    l = torch.randn(4, 64, device="cuda")
    for bad in [lambda: qe.add_rmsnorm(x.float()), lambda: qe.add_rmsnorm(x.cpu()), lambda: qe.add_rmsnorm(x[:, ::2]),
                lambda: qe.add_rmsnorm(x, x[:2].contiguous()), lambda: qe.add_rmsnorm(x, weight=torch.ones(128, device="cuda")),
                lambda: qe.add_rmsnorm(x, weight=torch.ones(256)), lambda: qe.add_rmsnorm(x, quant="e5m2"),
                lambda: qe.route_logits(l.double(), r, 4), lambda: qe.route_logits(l.t(), r, 2),
                lambda: qe.route_logits(l[:1].expand(4, 64), r, 4), lambda: qe.route_logits(l, r, 4, torch.zeros(64)),
                lambda: qe.route_logits(l, r, 4, torch.zeros(63, device="cuda")),
                lambda: qe.dequant_rows(torch.zeros(4, 256, dtype=torch.uint8, device="cuda"), 256),
                lambda: qe.dequant_rows(torch.zeros(4, 272, dtype=torch.uint8, device="cuda"), 256, rows=torch.zeros(2, dtype=torch.int64, device="cuda"))]:
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(qe.StrataError):
        qe.route_logits(l, r, 65)
    # rows of a wider tensor are taken as they lie
    wide = torch.randn(5, 100, device="cuda")
    a, b = qe.route_logits(wide[:, :64], r, 4), qe.route_logits(wide[:, :64].contiguous(), r, 4)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    one = qe.route_logits(wide[:1, 3:67], r, 4)
    assert torch.equal(one[0], qe.route_logits(wide[:1, 3:67].contiguous(), r, 4)[0])
    e = qe.route_logits(torch.empty(0, 64, device="cuda"), r, 4)
    assert e[0].shape == (0, 4)
    h, xn, packed = qe.add_rmsnorm(torch.empty(0, 256, device="cuda", dtype=torch.bfloat16), quant="int8", group=0)
    assert packed.shape == (0, 272) and qe.dequant_rows(packed, 256, "int8", 0).shape == (0, 256)


@pytest.mark.parametrize("shape,T", [(gen.TINY, 5), (gen.TINY, 100), (gen.FLASH2, 4)], ids=["tiny-5", "tiny-100", "flash-4"])
def test_plain_forward_equals_its_steps_on_bf16_rows(one_rank, shape, T):
    """ExpertParallel.forward sends its rows as they are: bit for bit the same steps
    without an exchange, and the layer's own output on the same kernels."""
    k, H = shape.top_k, shape.hidden
    layer, L, sb = rule_layer(shape, T + T * k, seed=1)
    x = to_dev_bf16(gen.hidden(T, H, seed=15))
    sent = []

    class Watched(GpuBackend):
        def gather_rows(self, src, rows):
            sent.append((src.dtype, tuple(src.shape)))
            return super().gather_rows(src, rows)

    y = ExpertParallel(Watched(L), shape.n_experts, k, H).forward(x)
    L.sync_status()
    assert sent == [(torch.bfloat16, (T, H))]
    idx, w, _, _ = L.route(x)
    prefill = T > 64
    yd = torch.float16 if prefill else torch.float32
    rows = torch.cat([x, x.repeat_interleave(k, dim=0)])
    ids = torch.cat([torch.full((T,), -1, dtype=torch.int32, device="cuda"), idx.reshape(-1)])
    out = torch.empty((T + T * k, H), dtype=yd, device="cuda")
    Y = torch.empty((T * k + T, H), dtype=yd, device="cuda")
    qe.strata_moe_expert_rows(L.handle, rows.data_ptr(), ids.data_ptr(), T + T * k, T, prefill, out.data_ptr(), Y[T * k:].data_ptr())
    Y[:T * k] = out[T:]
    slot = torch.arange(T * k, dtype=torch.int32, device="cuda")
    ref = torch.empty_like(x)
    qe.strata_moe_combine_rows(L.handle, x.data_ptr(), T, idx.data_ptr(), w.data_ptr(), slot.data_ptr(), Y.data_ptr(), prefill, ref.data_ptr())
    L.sync_status()
    assert torch.equal(y, ref)
    L.set_option(qe.STRATA_OPT_PATH, 2 if prefill else 1)
    assert torch.equal(y, L.forward(x))
    L.sync_status()
    L.close()


class Late:
    """A stream whose inputs arrive late: what the calls read is written behind a
    long wait, so a call on any other stream reads the old values."""

    def __init__(self):
        torch.cuda.synchronize()
        self.stream = torch.cuda.Stream()

    def fill(self, pairs):
        torch.cuda._sleep(40_000_000)  # about 20 ms
        for dst, src in pairs:
            dst.copy_(src)


def test_tensor_functions_follow_the_current_stream():
    """Norm, read, routing and the layer under `torch.cuda.stream`, without a
    stream argument: on the current stream, like the copies around them."""
    shape, T = gen.TINY, 40
    layer, L, sb = rule_layer(shape, T)
    h, delta, weight = block_inputs(shape, T, 21)
    bias = torch.from_numpy(sb).cuda()
    rule = qe.make_routing(**RULE)
    logits = torch.randn(T, shape.n_experts, device="cuda")

    def steps(h, delta, logits):
        h2, xn, packed = qe.add_rmsnorm(h, delta, weight, 1e-6, "e4m3", 128)
        x = qe.dequant_rows(packed, shape.hidden)
        idx, w = qe.route_logits(logits, rule, shape.top_k, bias)
        y = L.forward(xn)
        li, lw, off, lst = L.route(xn)
        return [t.clone() for t in (h2, xn, x, idx, w, y, li, lw, off, lst)]

    want = steps(h, delta, logits)
    torch.cuda.synchronize()
    late = Late()
    ins = [torch.zeros_like(t) for t in (h, delta, logits)]
    torch.cuda.synchronize()
    with torch.cuda.stream(late.stream):
        late.fill(zip(ins, (h, delta, logits)))
        got = steps(*ins)
        L.sync_status()  # waits for the current stream, too
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    # a given stream, from another current one
    for t in ins:
        t.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(late.stream):
        late.fill(zip(ins, (h, delta, logits)))
    s = late.stream
    h2, xn, packed = qe.add_rmsnorm(ins[0], ins[1], weight, 1e-6, "e4m3", 128, stream=s)
    x = qe.dequant_rows(packed, shape.hidden, stream=s)
    idx, w = qe.route_logits(ins[2], rule, shape.top_k, bias, stream=s)
    y = L.forward(xn, stream=s)
    outs = [h2, xn, x, idx, w, y, *L.route(xn, stream=s)]
    L.sync_status(s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    L.close()


def test_tensor_functions_join_a_capture():
    """Inside torch.cuda.graph the calls without a stream argument are captured."""
    shape, T = gen.TINY, 24
    layer, L, sb = rule_layer(shape, T)
    h, delta, weight = block_inputs(shape, T, 22)
    ih, idl = torch.zeros_like(h), torch.zeros_like(delta)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        h2, xn, packed = qe.add_rmsnorm(ih, idl, weight, 1e-6, "int8", 32)
        x = qe.dequant_rows(packed, shape.hidden, "int8", 32)
        y = L.forward(xn)
    for seed in (22, 23):
        a, b, _ = block_inputs(shape, T, seed)
        ih.copy_(a), idl.copy_(b)
        g.replay()
        rh, rxn, rp = qe.add_rmsnorm(a, b, weight, 1e-6, "int8", 32)
        assert torch.equal(h2, rh) and torch.equal(xn, rxn) and torch.equal(x, qe.dequant_rows(rp, shape.hidden, "int8", 32))
        assert torch.equal(y, L.forward(rxn))
    L.sync_status()
    del g
    L.close()


@pytest.mark.parametrize("T", [5, 100])
def test_forward_block_on_a_side_stream(one_rank, T):
    """ExpertParallel under `torch.cuda.stream`: its kernels, copies and exchange
    stay on that stream."""
    shape = gen.TINY
    layer, L, sb = rule_layer(shape, T + T * shape.top_k, seed=1)
    h, delta, weight = block_inputs(shape, T, 25)
    ep = ExpertParallel(GpuBackend(L), shape.n_experts, shape.top_k, shape.hidden)
    want = ep.forward_block(h, delta, weight) + (ep.forward(h),)
    torch.cuda.synchronize()
    ih, idl = torch.zeros_like(h), torch.zeros_like(delta)
    for _ in range(3):
        ih.zero_(), idl.zero_()
        late = Late()
        with torch.cuda.stream(late.stream):
            late.fill([(ih, h), (idl, delta)])
            got = ep.forward_block(ih, idl, weight) + (ep.forward(ih),)
            L.sync_status()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    L.close()


def test_forward_block_without_tokens(one_rank):
    shape = gen.TINY
    layer, L, sb = rule_layer(shape, 8, seed=1)
    ep = ExpertParallel(GpuBackend(L), shape.n_experts, shape.top_k, shape.hidden)
    none = torch.empty(0, shape.hidden, dtype=torch.bfloat16, device="cuda")
    h, y = ep.forward_block(none, none, None)
    assert h.shape == y.shape == none.shape and ep.forward(none).shape == none.shape
    L.sync_status()
    L.close()
