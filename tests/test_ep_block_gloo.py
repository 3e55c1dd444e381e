"""ExpertParallel.forward_block on CPU ranks (gloo, world size 2 and 3): the
pre-norm, the exchange of 8-bit rows and the experts, driven by a float64 numpy
backend.  Each rank's output must be the same bits as the same steps without
any exchange, the exchanged rows must be half as large as bf16 ones, and the
layer's output close to the one of unquantised rows."""
import os

import numpy as np
import pytest
import torch
import torch.distributed as dist
import torch.multiprocessing as mp

import gen
from tests import npref
from tests.front_ref import norm_rows
from tests.test_ep_gloo import NumpyBackend, _bits, _free_port, _tokens

EPS = 1e-6


class BlockBackend(NumpyBackend):
    """The 8-bit rows of the numpy backend: e4m3 codes, a scale for 128 columns."""

    wire_bytes = 0

    def y_dtype(self, prefill):
        self.prefill = prefill
        return super().y_dtype(prefill)

    def gather_rows(self, src, rows):
        if src.dtype == torch.uint8:
            self.wire_bytes += rows.numel() * src.shape[1]
        return super().gather_rows(src, rows)

    def pre_norm(self, h, delta, weight, eps):
        h, y = norm_rows(npref.bf16_bits_to_f64(_bits(h)), None if delta is None else npref.bf16_bits_to_f64(_bits(delta)),
                         weight.numpy().astype(np.float64), eps)
        T, H = y.shape
        scale = np.abs(y.reshape(T, H // 128, 128)).max(2) / 448
        codes = torch.from_numpy((y / np.repeat(scale, 128, 1)).astype(np.float32)).to(torch.float8_e4m3fn)
        pad = (-4 * scale.shape[1]) % 16
        packed = torch.cat([codes.view(torch.uint8), torch.from_numpy(scale.astype(np.float32).view(np.uint8)),
                            torch.zeros((T, pad), dtype=torch.uint8)], 1)
        return (torch.from_numpy(h).to(torch.bfloat16), torch.from_numpy(y.astype(np.float32)).to(torch.bfloat16), packed)

    def unpack_rows(self, packed, out):
        H = self.s.hidden
        scale = packed[:, H:H + 4 * (H // 128)].contiguous().view(torch.float32)
        q = packed[:, :H].contiguous().view(torch.float8_e4m3fn).float()
        out.copy_((q * scale.repeat_interleave(128, 1)).to(torch.bfloat16))

    def block_local(self, h, delta, weight):
        """The same steps on one rank, no exchange."""
        h, xn, packed = self.pre_norm(h, delta, weight, EPS)
        idx, w = self.route(xn)
        x = torch.empty_like(xn)
        self.unpack_rows(packed, x)
        T, k = x.shape[0], self.s.top_k
        Y = torch.empty((T * k + T, self.s.hidden), dtype=torch.float64)
        self.expert_rows(x.repeat_interleave(k, dim=0), torch.from_numpy(idx.numpy().reshape(-1).astype(np.int32)), 0, False, Y[:T * k], None)
        self.expert_rows(x, torch.full((T,), -1, dtype=torch.int32), T, False,
                         torch.empty((T, self.s.hidden), dtype=torch.float64), Y[T * k:])
        slot = torch.arange(T * k, dtype=torch.int32)
        return h, self.combine(x, idx, w, slot, Y, False), xn


def _inputs(shape, T, rank):
    g = torch.Generator().manual_seed(90 + rank)
    h = _tokens(shape, T, rank)
    delta = (0.5 * torch.randn((T, shape.hidden), generator=g)).to(torch.bfloat16)
    weight = 1 + 0.2 * torch.randn(shape.hidden, generator=torch.Generator().manual_seed(1))
    return h, delta, weight


def _worker(rank, world, port, Ts, out):
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port), RANK=str(rank), WORLD_SIZE=str(world))
    import datetime
    from quantized_expert_ffn_04_b200.ep import ExpertParallel
    dist.init_process_group("gloo", rank=rank, world_size=world, timeout=datetime.timedelta(seconds=120))
    try:
        be = BlockBackend(gen.layer_weights(gen.TINY, seed=0))
        ep = ExpertParallel(be, gen.TINY.n_experts, gen.TINY.top_k, gen.TINY.hidden)
        h, y = ep.forward_block(*_inputs(gen.TINY, Ts[rank], rank))
        out[rank] = (_bits(h).copy(), _bits(y).copy(), be.wire_bytes, be.prefill)
        dist.barrier()
    finally:
        dist.destroy_process_group()


@pytest.mark.parametrize("world,Ts", [(2, (8, 8)), (3, (5, 1, 9)), (2, (3, 0)), (2, (70, 3))], ids=["2x8", "5-1-9", "3-0", "70-3"])
def test_block_matches_one_rank(world, Ts):
    port = _free_port()
    with mp.Manager() as m:
        out = m.dict()
        mp.spawn(_worker, args=(world, port, Ts, out), nprocs=world, join=True)
        res = dict(out)
    be = BlockBackend(gen.layer_weights(gen.TINY, seed=0))
    # one path everywhere: the outputs that travel have its type
    assert all(res[r][3] == (max(Ts) > 64) for r in range(world))
    for r in range(world):
        if not Ts[r]:
            assert res[r][1].size == 0
            continue
        h, y, xn = be.block_local(*_inputs(gen.TINY, Ts[r], r))
        assert np.array_equal(res[r][0], _bits(h)) and np.array_equal(res[r][1], _bits(y)), f"rank {r}"
        # one copy of every picked row: H codes and H / 128 scales (16 bytes here) against 2 H
        assert res[r][2] == Ts[r] * gen.TINY.top_k * (gen.TINY.hidden + 16)
        # e4m3 moves a value by at most 2^-4: the outputs stay near the bf16 rows' ones
        ref = npref.bf16_bits_to_f64(_bits(be.forward_local(xn)))
        got = npref.bf16_bits_to_f64(res[r][1])
        assert np.linalg.norm(got - ref) <= 2 * 2.0 ** -4 * np.linalg.norm(ref)
