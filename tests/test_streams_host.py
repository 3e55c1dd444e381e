"""The torch-tensor functions and the layer run on torch's current stream of
their tensors' device unless a stream is given, and what they allocate belongs
to the stream they run on (no GPU: the C calls and torch's streams are stand-ins
that record what they get)."""
import contextlib
import inspect
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")

import gen  # noqa: E402
import quantized_expert_ffn_04_b200 as qe  # noqa: E402
from quantized_expert_ffn_04_b200 import ep  # noqa: E402

CURRENT, GIVEN = SimpleNamespace(cuda_stream=0x510), SimpleNamespace(cuda_stream=0x77)


class OnGpu(torch.Tensor):
    """A host tensor that says it is on a GPU; the C calls never see it."""
    is_cuda = property(lambda self: True)


def tensor(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


@pytest.fixture
def calls(monkeypatch):
    """Every C call's name and stream, and the stream that torch allocates on."""
    seen, on = [], []

    for name in ("strata_moe_route_logits", "strata_moe_add_rmsnorm", "strata_moe_dequant_rows", "strata_moe_forward",
                 "strata_moe_route", "strata_moe_sync_status", "strata_ep_gather_rows", "strata_moe_expert_rows",
                 "strata_moe_combine_rows"):
        at = list(inspect.signature(getattr(qe, name)).parameters).index("stream")

        def stand_in(*args, stream=None, name=name, at=at):  # the stream by position or by keyword
            seen.append((name, args[at] if len(args) > at else stream))
        monkeypatch.setattr(qe, name, stand_in)
        if hasattr(ep, name):
            monkeypatch.setattr(ep, name, stand_in)

    def current(device=None):
        seen.append(("device", device))
        return CURRENT

    @contextlib.contextmanager
    def stream(s):
        on.append(s)
        yield
        on.pop()

    empty, empty_like = torch.empty, torch.empty_like
    monkeypatch.setattr(torch.cuda, "current_stream", current)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: seen.append(("kept for", s)))
    monkeypatch.setattr(torch, "empty", lambda *a, **k: (seen.append(("empty", on[-1] if on else None)), empty(*a, **k))[1])
    monkeypatch.setattr(torch, "empty_like", lambda *a, **k: (seen.append(("empty", on[-1] if on else None)), empty_like(*a, **k))[1])
    return seen


def layer():
    L = object.__new__(qe.Layer)
    L.handle, L.shape, L.device = None, gen.TINY, 3
    return L


H = gen.TINY.hidden
ENTRIES = {
    "route_logits": lambda s: qe.route_logits(tensor(2, 64), qe.make_routing(), 4, **s),
    "add_rmsnorm": lambda s: qe.add_rmsnorm(tensor(2, 256, dtype=torch.bfloat16), tensor(2, 256, dtype=torch.bfloat16), quant="e4m3", **s),
    "dequant_rows": lambda s: qe.dequant_rows(tensor(2, 272, dtype=torch.uint8), 256, out=tensor(2, 256, dtype=torch.bfloat16), **s),
    "forward": lambda s: layer().forward(tensor(2, H, dtype=torch.bfloat16), **s),
    "route": lambda s: layer().route(tensor(2, H, dtype=torch.bfloat16), **s),
    "sync_status": lambda s: layer().sync_status(**s),
}


@pytest.mark.parametrize("entry", ENTRIES)
def test_without_a_stream_the_current_one_of_the_device(calls, entry):
    ENTRIES[entry]({})
    ran = [s for name, s in calls if name.startswith("strata")]
    assert ran == [CURRENT.cuda_stream]
    # of the tensors' (the layer's) device, not of whichever is current
    assert {d for name, d in calls if name == "device"} == {3 if entry == "sync_status" else torch.device("cpu")}
    assert all(s is None for name, s in calls if name == "empty")


@pytest.mark.parametrize("entry", ENTRIES)
def test_a_given_stream_runs_the_call_and_owns_its_outputs(calls, entry):
    ENTRIES[entry](dict(stream=GIVEN))
    assert [s for name, s in calls if name.startswith("strata")] == [GIVEN.cuda_stream]
    made = [s for name, s in calls if name == "empty"]
    assert all(s is GIVEN for s in made)
    # and the stream of whoever reads them is known to the allocator
    assert [s for name, s in calls if name == "kept for"] == [CURRENT] * len(made)


def test_the_expert_parallel_backend_runs_on_the_current_stream(calls):
    be = ep.GpuBackend(layer())
    x = tensor(4, H, dtype=torch.bfloat16)
    idx, w = be.route(x)
    be.gather_rows(x, tensor(3, dtype=torch.int32))
    be.expert_rows(x, tensor(4, dtype=torch.int32), 2, False, tensor(4, H), tensor(2, H))
    be.combine(x, idx, w, tensor(4, 2, dtype=torch.int32), tensor(4, H), False)
    _, _, packed = be.pre_norm(x, None, None, 1e-6)
    be.unpack_rows(packed.as_subclass(OnGpu), tensor(4, H, dtype=torch.bfloat16))
    ran = [(name, s) for name, s in calls if name.startswith("strata")]
    assert [n for n, _ in ran] == ["strata_moe_route", "strata_ep_gather_rows", "strata_moe_expert_rows", "strata_moe_combine_rows",
                                   "strata_moe_add_rmsnorm", "strata_moe_dequant_rows"]
    assert all(s == CURRENT.cuda_stream for _, s in ran)
