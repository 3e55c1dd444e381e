"""The pre-norm with 8-bit rows and their read on the GPU
(strata_moe_add_rmsnorm, strata_moe_dequant_rows) against plain 64-bit forms.

Tolerances, from the arithmetic: the sum of squares takes at most 8 ceil(H /
1024) + 16 roundings of 2^-24 (halved by the square root), the mean, eps, root
and quotient four, y two products, a scale one quotient: for H <= 16384 below
(72 + 4 + 3) 2^-24 = 4.7e-6 = FP32_TOL.  bf16 rounds by half a step, 2^-8 of
the value; e4m3 by 2^-4 of the value, or 2^-10 of the scale where codes are
subnormal; int8 by half a scale.
"""
import numpy as np
import pytest

from tests.front_ref import norm_rows, round_to

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import quantized_expert_ffn_04_b200 as qe  # noqa: E402

FP32_TOL = 4.7e-6
Q8 = {"e4m3": (qe.STRATA_Q8_E4M3, torch.float8_e4m3fn, 448.0), "int8": (qe.STRATA_Q8_INT8, torch.int8, 127.0)}


def bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).cuda().to(torch.bfloat16)


def f64(t):
    return t.double().cpu().numpy()


class Norm:
    """One call's buffers, with guards behind them."""

    def __init__(self, x, delta=None, weight=None, eps=1e-6, q8=None, group=0, xn=True, h=None, in_place=False, packed=False):
        T, H = x.shape
        self.T, self.H, self.eps, self.q8, self.group = T, H, eps, q8, group
        self.x, self.delta, self.weight = x, delta, weight
        self.h = x if in_place else (torch.full((T + 1, H), 7.0, dtype=torch.bfloat16, device="cuda")
                                     if (h if h is not None else delta is not None) else None)
        self.in_place = in_place
        self.xn = torch.full((T + 1, H), 7.0, dtype=torch.bfloat16, device="cuda") if xn else None
        self.ns = H // group if group else 1
        self.q = self.scale = None
        if q8:
            if packed:
                self.stride = H + (4 * self.ns + 15) // 16 * 16 + 16
                self.buf = torch.full((T + 1, self.stride), 99, dtype=torch.uint8, device="cuda")
                self.q = self.buf[:, :H]
                self.scale = self.buf.view(torch.float32)[:, H // 4:H // 4 + self.ns]
            else:
                self.stride = H + 32
                self.buf = torch.full((T + 1, self.stride), 99, dtype=torch.uint8, device="cuda")
                self.q = self.buf[:, :H]
                self.scale_buf = torch.full((T + 1, self.ns + 3), 7.0, device="cuda")
                self.scale = self.scale_buf[:, :self.ns]

    def go(self, stream=None):
        p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        wt = qe.STRATA_BF16 if self.weight is not None and self.weight.dtype == torch.bfloat16 else qe.STRATA_F32
        qe.strata_moe_add_rmsnorm(p(self.x), p(self.delta), p(self.weight), wt, self.eps, self.T, self.H, p(self.h), p(self.xn),
                                  Q8[self.q8][0] if self.q8 else 0, self.group, p(self.q), self.stride if self.q8 else 0,
                                  p(self.scale), self.scale.stride(0) if self.q8 else 0, stream)

    def codes(self):
        """The values of the codes and their scales for every column, in 64 bits."""
        c = self.q[:self.T].contiguous().view(Q8[self.q8][1]).float()
        s = self.scale[:self.T].repeat_interleave(self.H // self.ns, 1)
        return f64(c), f64(s)

    def check(self, x, delta, weight):
        """Against the 64-bit form of the float64 inputs."""
        T = self.T
        h, y = norm_rows(x, delta, weight, self.eps)
        if self.h is not None:
            assert np.array_equal(f64(self.h[:T]), h)
            if not self.in_place:
                assert (self.h[T] == 7.0).all()
        if self.xn is not None:
            got = f64(self.xn[:T])
            assert (np.abs(got - y) <= (2.0 ** -8 + FP32_TOL) * np.abs(y) + 1e-38).all()
            assert (self.xn[T] == 7.0).all()
        if self.q8:
            top = Q8[self.q8][2]
            blocks = np.abs(y).reshape(T, self.ns, -1)
            np.testing.assert_allclose(f64(self.scale[:T]), blocks.max(2) / top, rtol=FP32_TOL, atol=0)
            c, s = self.codes()
            err = np.abs(c * s - y)
            if self.q8 == "e4m3":
                assert (err <= (2.0 ** -4 + 3 * FP32_TOL) * np.abs(y) + s * (2.0 ** -10 + 1e-9)).all()
            else:  # half a step, and y's error of up to 127 steps times FP32_TOL
                assert (err <= s * (0.5 + 2 * 127 * FP32_TOL)).all()
            assert (np.abs(c).reshape(T, self.ns, -1).max(2) == top).all(), "a group's largest value has the largest code"
            assert (self.buf[T] == 99).all() and (self.buf[:T, self.H + 4 * self.ns:] == 99).all(), "padding was written"


def inputs(T, H, seed, wt=None):
    rng = np.random.default_rng(seed)
    x = bf16(rng.standard_normal((T, H)) * np.where(rng.random(H) < 0.02, 30.0, 1.0))
    d = bf16(0.5 * rng.standard_normal((T, H)))
    w = None if wt is None else torch.from_numpy((1 + 0.3 * rng.standard_normal(H)).astype(np.float32)).cuda().to(wt)
    return x, d, w


@pytest.mark.parametrize("q8", ["e4m3", "int8"])
@pytest.mark.parametrize("T,H,group", [(1, 2560, 128), (3, 128, 0), (5, 32, 32), (2, 96, 32), (1, 6144, 64), (7, 2560, 0),
                                       (4, 2592, 32), (37, 1024, 128), (2, 16384, 128), (2, 16352, 32), (300, 640, 64), (9, 4160, 64), (3, 8192, 0)])
def test_norm_matches_the_plain_form(T, H, group, q8):
    for i, wt in enumerate((None, torch.float32, torch.bfloat16)):
        x, d, w = inputs(T, H, 100 * i + T + H, wt)
        n = Norm(x, d, w, q8=q8, group=group, packed=i == 1)
        n.go()
        torch.cuda.synchronize()
        n.check(f64(x), f64(d), None if w is None else f64(w))


def test_norm_options():
    """Every combination of outputs; without a residual; in place."""
    T, H = 6, 384
    for delta in (False, True):
        for xn in (False, True):
            for q8 in (None, "e4m3"):
                if not delta and not xn and q8 is None:
                    continue
                x, d, w = inputs(T, H, 7, torch.float32)
                n = Norm(x, d if delta else None, w, q8=q8, group=128, xn=xn)
                n.go()
                torch.cuda.synchronize()
                n.check(f64(x), f64(d) if delta else None, f64(w))
    x, d, w = inputs(T, H, 8, torch.bfloat16)
    keep = f64(x)
    n = Norm(x, d, w, q8="int8", group=32, in_place=True)
    n.go()
    torch.cuda.synchronize()
    n.check(keep, f64(d), f64(w))
    # h without a residual is a copy of x
    x, d, w = inputs(T, H, 9)
    n = Norm(x, h=True, xn=False)
    n.go()
    torch.cuda.synchronize()
    assert torch.equal(n.h[:T], x)


def test_the_residual_sum_is_the_fp32_sum_rounded_once():
    """bf16(f32(x) + f32(delta)) bit for bit over all exponents, subnormal values
    and overflow to infinity included."""
    T, H = 64, 4096
    rng = np.random.default_rng(5)
    bits = rng.integers(0, 1 << 16, (2, T, H)).astype(np.uint16)
    near = rng.integers(-1200, 1200, (T // 2, H))  # delta's exponent near x's, and nine below it
    bits[1, :T // 2] = np.clip(bits[0, :T // 2].astype(np.int64) + near, 0, 0xFFFF)
    x, d = (torch.from_numpy(b.view(np.int16).copy()).view(torch.bfloat16).cuda() for b in bits)
    x, d = (torch.where(torch.isfinite(t), t, torch.ones_like(t)) for t in (x, d))
    n = Norm(x, d, xn=False)
    n.go()
    torch.cuda.synchronize()
    assert torch.equal(n.h[:T].view(torch.int16), (x.float() + d.float()).to(torch.bfloat16).view(torch.int16))


def test_rows_do_not_depend_on_their_batch():
    """The same row alone, in a small and in a large batch: the same bits."""
    H = 2592
    x, d, w = inputs(400, H, 6, torch.float32)
    outs = []
    for T in (400, 148, 1):
        n = Norm(x[:T], d[:T], w, q8="e4m3", group=32)
        n.go()
        torch.cuda.synchronize()
        outs.append((n.xn[0].clone(), n.q[0].clone(), n.scale[0].clone()))
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))


def test_codes_of_bf16_weights_are_the_64_bit_ones():
    """Every code as 64-bit arithmetic gives it, exact halves going to the even one."""
    for q8, group in (("e4m3", 128), ("e4m3", 0), ("int8", 64)):
        x, d, w = inputs(200, 1024, 17, torch.bfloat16)
        x[:, ::3] = x[:, :1] * 0.25  # many equal values and exact ratios
        n = Norm(x, d, w, q8=q8, group=group)
        n.go()
        torch.cuda.synchronize()
        h, _ = norm_rows(f64(x), f64(d), None, 1e-6)
        t = (h * f64(w)).reshape(200, n.ns, -1)
        # the product is exact, so the one rounded quotient is a half only where the exact one is
        a = t * Q8[q8][2] / np.abs(t).max(2, keepdims=True)
        want = round_to(a, 8, -6) if q8 == "e4m3" else np.round(a)
        assert np.array_equal(n.codes()[0], want.reshape(200, -1))


@pytest.mark.parametrize("eps", [0.0, 1e-35, 1e-6, 1.0])
def test_norm_range(eps):
    """Rows whose squares overflow or underflow fp32, and zero rows."""
    rng = np.random.default_rng(3)
    H = 256
    scales = [3e38 / 6, 1e30, 1e19, 1.0, 1e-15, 1e-19, 1e-25, 1e-37]
    x = bf16(np.stack([np.clip(rng.standard_normal(H), -5, 5) * s for s in scales]))
    n = Norm(x, eps=eps)
    n.go()
    torch.cuda.synchronize()
    h, y = norm_rows(f64(x), None, None, eps)
    got = f64(n.xn[:len(scales)])
    # outputs below bf16's normal range round by half its smallest step, 2^-134
    assert (np.abs(got - y) <= (2.0 ** -8 + FP32_TOL) * np.abs(y) + 2.0 ** -133).all()
    if eps > 0:
        z = Norm(bf16(np.zeros((2, H))), eps=eps, q8="e4m3", group=128)
        z.go()
        torch.cuda.synchronize()
        assert (z.xn[:2] == 0).all() and (z.scale[:2] == 0).all() and (z.q[:2] == 0).all()


@pytest.mark.parametrize("q8", ["e4m3", "int8"])
def test_norm_keeps_what_is_not_finite_in_its_row_or_group(q8):
    T, H = 4, 512
    x, d, w = inputs(T, H, 11, torch.float32)
    x[1, 200] = float("nan")
    x[2, 3] = float("inf")
    w2 = w.clone()
    w2[130] = float("inf")
    n = Norm(x, None, w, q8=q8, group=128)
    n.go()
    torch.cuda.synchronize()
    xn = n.xn[:T].float()
    assert torch.isnan(xn[1]).all() and torch.isnan(n.scale[1]).all() and (n.q[1] == 0).all()
    assert torch.isnan(xn[2, 3]) and (xn[2, 4:] == 0).all()
    assert torch.isnan(n.scale[2, 0]) and (n.scale[2, 1:] == 0).all() and (n.q[2] == 0).all()
    assert torch.isfinite(xn[[0, 3]]).all() and torch.isfinite(n.scale[[0, 3]]).all()
    out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    qe.strata_moe_dequant_rows(n.q.data_ptr(), Q8[q8][0], n.stride, n.scale.data_ptr(), n.scale.stride(0), 128, None, T, T, H,
                               out.data_ptr())
    torch.cuda.synchronize()
    assert torch.isnan(out[1]).all() and torch.isnan(out[2, :128]).all() and (out[2, 128:] == 0).all()
    m = Norm(x[3:], None, w2, q8=q8, group=128)
    m.go()
    torch.cuda.synchronize()
    assert torch.isinf(m.xn[0, 130].float()) and torch.isnan(m.scale[0, 1]) and (m.q[0, 128:256] == 0).all()
    assert torch.isfinite(m.scale[0, [0, 2, 3]]).all()


def test_tiny_groups_store_zeros():
    T, H = 2, 128
    x = bf16(np.ones((T, H)))
    w = torch.ones(H, device="cuda")
    w[:32] = 1e-36  # below 2^-116
    w[32:64] = 1e-34
    n = Norm(x, None, w, eps=0.0, q8="e4m3", group=32, xn=False)
    n.go()
    torch.cuda.synchronize()
    assert (n.q[:T, :32] == 0).all() and (n.scale[:T, 0] == 0).all()
    c, s = n.codes()
    assert (c[:, 32:] == 448).all()
    np.testing.assert_allclose(s[:, 32] * 448, np.float64(np.float32(1e-34)), rtol=FP32_TOL)


def all_codes(q8, n, H, rng):
    c = rng.integers(0, 256, (n, H)).astype(np.uint8)
    c.reshape(-1)[:256] = np.arange(256)[:c.size]
    return torch.from_numpy(c).cuda()


@pytest.mark.parametrize("q8", ["e4m3", "int8"])
@pytest.mark.parametrize("n,src,H,group", [(1, 1, 32, 0), (7, 3, 2560, 128), (100, 20, 96, 32), (33, 33, 640, 64), (1025, 64, 6144, 0),
                                           (5, 9, 1056, 32), (64, 8, 128, 128), (3, 2, 16384, 64)])
def test_dequant_rows_exactly(n, src, H, group, q8):
    """bf16(f32(code) * scale) bit for bit, any byte a code (e4m3's two NaN too)."""
    rng = np.random.default_rng(n + H)
    code = all_codes(q8, src, H + 16, rng)
    ns = H // group if group else 1
    scale = torch.from_numpy(np.exp(rng.standard_normal((src, ns + 1))).astype(np.float32)).cuda()
    rows = torch.from_numpy(rng.integers(0, src, n).astype(np.int32)).cuda()
    if n > 4:
        rows[1], rows[3] = -1, src  # outside: skipped
    out = torch.full((n + 1, H), 7.0, dtype=torch.bfloat16, device="cuda")
    qe.strata_moe_dequant_rows(code.data_ptr(), Q8[q8][0], H + 16, scale.data_ptr(), ns + 1, group, rows.data_ptr(), n, src, H,
                               out.data_ptr())
    torch.cuda.synchronize()
    ref = code[:, :H].contiguous().view(Q8[q8][1]).float() * scale[:, :ns].repeat_interleave(H // ns, 1)
    ref = ref.to(torch.bfloat16)[rows.long().clamp(0, src - 1)]
    ok = (rows >= 0) & (rows < src)
    got = out[:n]
    same = (got == ref) | (torch.isnan(got) & torch.isnan(ref))
    assert same[ok].all() and (got[~ok] == 7.0).all() and (out[n] == 7.0).all()
    if n <= src:  # without an index
        qe.strata_moe_dequant_rows(code.data_ptr(), Q8[q8][0], H + 16, scale.data_ptr(), ns + 1, group, None, n, src, H,
                                   out.data_ptr())
        torch.cuda.synchronize()
        ref = (code[:n, :H].contiguous().view(Q8[q8][1]).float() * scale[:n, :ns].repeat_interleave(H // ns, 1)).to(torch.bfloat16)
        assert ((out[:n] == ref) | (torch.isnan(out[:n]) & torch.isnan(ref))).all()


@pytest.mark.parametrize("q8", ["e4m3", "int8"])
def test_dequant_to_rows_on_16_bytes_only(q8):
    """An output that starts between two 32-byte lines."""
    rng = np.random.default_rng(4)
    H, n = 96, 37
    code = all_codes(q8, n, H, rng)
    scale = torch.from_numpy(np.exp(rng.standard_normal((n, 3))).astype(np.float32)).cuda()
    buf = torch.full((n * H + 24,), 7.0, dtype=torch.bfloat16, device="cuda")
    assert buf.data_ptr() % 32 == 0
    for off in (0, 8):
        buf.fill_(7.0)
        out = buf[off:off + n * H].view(n, H)
        qe.strata_moe_dequant_rows(code.data_ptr(), Q8[q8][0], H, scale.data_ptr(), 3, 32, None, n, n, H, out.data_ptr())
        torch.cuda.synchronize()
        ref = (code.view(Q8[q8][1]).float() * scale.repeat_interleave(32, 1)).to(torch.bfloat16)
        assert ((out == ref) | (torch.isnan(out) & torch.isnan(ref))).all()
        assert (buf[:off] == 7.0).all() and (buf[off + n * H:] == 7.0).all()


def test_offsets_past_32_bits():
    """Rows further than 2^32 bytes into the codes and the output."""
    H, group = 65536, 0
    src = (1 << 32) // H + 3
    q = torch.zeros((src, H), dtype=torch.int8, device="cuda")
    q[-1] = 5
    q[-3] = -3
    scale = torch.full((src, 1), 0.5, device="cuda")
    n = (1 << 31) // H + 2  # 2^32 bytes of bf16 and two rows
    rows = torch.zeros(n, dtype=torch.int32, device="cuda")
    rows[-1], rows[-2] = src - 1, src - 3
    out = torch.full((n, H), 7.0, dtype=torch.bfloat16, device="cuda")
    qe.strata_moe_dequant_rows(q.data_ptr(), qe.STRATA_Q8_INT8, H, scale.data_ptr(), 1, group, rows.data_ptr(), n, src, H, out.data_ptr())
    torch.cuda.synchronize()
    assert (out[-1] == 2.5).all() and (out[-2] == -1.5).all() and (out[:-2] == 0).all()


def test_streams_and_graph():
    T, H = 64, 2560
    x, d, w = inputs(T, H, 21, torch.bfloat16)
    n = Norm(x, d, w, q8="e4m3", group=128)
    out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")

    def go(s):
        n.go(s.cuda_stream)
        qe.strata_moe_dequant_rows(n.q.data_ptr(), qe.STRATA_Q8_E4M3, n.stride, n.scale.data_ptr(), n.scale.stride(0), 128, None,
                                   T, T, H, out.data_ptr(), s.cuda_stream)

    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(10):
        go(s)
    torch.cuda.synchronize()
    n.check(f64(x), f64(d), f64(w))
    c, sc = n.codes()
    assert np.array_equal(f64(out), f64(torch.from_numpy(c * sc).float().to(torch.bfloat16)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go(torch.cuda.current_stream())
    x2, d2, _ = inputs(T, H, 22)
    x.copy_(x2), d.copy_(d2)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    n.check(f64(x2), f64(d2), f64(w))


def range_rows(H, rng):
    """Rows whose norm's factor runs from 2^-127 to 2^70, and rows with parts far
    below their mean, where another part's squares decide the factor."""
    z = rng.standard_normal((16, H))
    level = np.exp2([2, 0, -3, -6, -10, -20, -29, -31, -60, -70, 29, 31, 64, 100, 123, 0])
    x = np.clip(z, -5, 5) * level[:, None]
    part = np.arange(H) // 128
    for row in (10, 13, 14):
        for p in range(8):  # from the row's own level down to 2^-140 of it
            x[row, part == p] *= np.exp2(-20.0 * p)
    x[15, 128:] *= 2.0 ** -40
    return bf16(x)


@pytest.mark.parametrize("eps", [0.0, 1e-6])
@pytest.mark.parametrize("wt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("q8", ["e4m3", "int8"])
def test_rows_over_the_whole_range(q8, group, wt, eps):
    """bf16 rows, codes and scales of rows of any size under weights of any size:
    products of a row's value and a weight that leave fp32's normal range on
    either side while their normalised value is well inside it."""
    H = 1024
    rng = np.random.default_rng(97)
    x = range_rows(H, rng)
    T = x.shape[0]
    sizes = np.array([[1.0, 1e-34, 1.5e-36, 2.0 ** -115, 2.0 ** -119, 1e-38, 3e-40, 1.0],  # the last three: no codes
                      [2.0 ** 95] * 8, [1e-34] * 8, [2.0 ** -112] * 8, [1.0, 2.0 ** 95, 1e-30, 2.0 ** 60, 1e-20, 2.0 ** 90, 1e-3, 1e-36]])
    for size in sizes:
        w = (np.repeat(size, 128) * rng.uniform(0.5, 1.0, H)).astype(np.float32)
        w = torch.from_numpy(w).cuda().to(wt)
        n = Norm(x, None, w, eps=eps, q8=q8, group=group)
        n.go()
        torch.cuda.synchronize()
        _, y = norm_rows(f64(x), None, f64(w), eps)
        # below the normal range fp32 and bf16 round by half their smallest steps, 2^-150 (twice) and 2^-134
        err = np.abs(f64(n.xn[:T]) - y)
        assert (err <= (2.0 ** -8 + FP32_TOL) * np.abs(y) + 2.0 ** -134 + 2.0 ** -149).all()
        top = Q8[q8][2]
        big = np.abs(y).reshape(T, n.ns, -1).max(2)
        c, s = n.codes()
        c, s = c.reshape(T, n.ns, -1), s.reshape(T, n.ns, -1)[:, :, 0]
        none, some = big < 2.0 ** -116 * (1 - FP32_TOL), big > 2.0 ** -116 * (1 + FP32_TOL)
        assert (s[none] == 0).all() and (c[none] == 0).all()
        np.testing.assert_allclose(s[some], big[some] / top, rtol=FP32_TOL)
        assert (np.abs(c).max(2)[some] == top).all()
        e, s = np.abs(c * s[:, :, None] - y.reshape(c.shape))[some], s[some][:, None]
        if q8 == "e4m3":
            assert (e <= (2.0 ** -4 + 3 * FP32_TOL) * np.abs(y.reshape(c.shape)[some]) + s * (2.0 ** -10 + 1e-9)).all()
        else:
            assert (e <= s * (0.5 + 2 * 127 * FP32_TOL)).all()
    # without a weight
    n = Norm(x, None, None, eps=eps)
    n.go()
    torch.cuda.synchronize()
    _, y = norm_rows(f64(x), None, None, eps)
    assert (np.abs(f64(n.xn[:T]) - y) <= (2.0 ** -8 + FP32_TOL) * np.abs(y) + 2.0 ** -134 + 2.0 ** -149).all()


def test_norm_rows_past_32_bits():
    """Rows further than 2^32 bytes into x, xn and the codes: as in a call of their own."""
    H = 16384
    T = (1 << 32) // H + 5  # one byte a code
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    tail, _, w = inputs(5, H, 41, torch.float32)
    x[-5:] = tail
    xn = torch.empty_like(x)
    q = torch.empty((T, H), dtype=torch.uint8, device="cuda")
    scale = torch.empty((T, H // 32), device="cuda")

    def go(x, n, xn, q, scale):
        qe.strata_moe_add_rmsnorm(x.data_ptr(), None, w.data_ptr(), qe.STRATA_F32, 1e-6, n, H, None, xn.data_ptr(), qe.STRATA_Q8_E4M3, 32,
                                  q.data_ptr(), H, scale.data_ptr(), H // 32)

    go(x, T, xn, q, scale)
    few = [torch.empty_like(t[:5]) for t in (xn, q, scale)]
    go(tail, 5, *few)
    torch.cuda.synchronize()
    assert all(torch.equal(a[-5:], b) for a, b in zip((xn, q, scale), few))
    assert (xn[:-5] == 0).all() and (q[:-5] == 0).all() and (scale[:-5] == 0).all()
