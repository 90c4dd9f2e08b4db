"""The operators on 8-bit rows where a call can go wrong without its numbers being
hard: streams, graphs, handles side by side, places that allow no vectors, rows
past 32-bit offsets, nothing to do.  Tolerances as in test_gpu_rows.py."""
from __future__ import annotations

import pytest
import torch

import dense_tiled_gemm_02_gb300 as pkg
from gpu_helpers import forced_plan
from test_gpu_rows import (BF16, EPS, F16, F32, U, backward_ref, blocks_ref, done, held, i8_check, ints,
                           near, norm_ref, offsets_of, rnd)

pytestmark = pytest.mark.gpu


class Set:
    """Every operator once, on buffers that stay: the inputs may be refilled."""

    def __init__(self, T, H, F, seed):
        self.T, self.H, self.F = T, H, F
        self.x, self.res, self.dy, self.dres = (torch.empty((T, H), dtype=BF16, device="cuda")
                                                for _ in range(4))
        self.w = torch.empty(H, dtype=BF16, device="cuda")
        self.W, self.ws = ints((1, F, H), 9), rnd((1, F), F32, 10).abs() / 900
        self.h, self.y, self.dx = (torch.empty_like(self.x) for _ in range(3))
        self.y8, self.s = torch.empty((T, H), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
        self.rstd, self.dw = torch.empty(T, device="cuda"), torch.empty(H, device="cuda")
        self.q, self.e = pkg.Rows8.empty(self.x)
        self.back = torch.empty_like(self.x)
        self.D = torch.empty((T, F), dtype=BF16, device="cuda")
        self.dD = torch.empty((T, F), dtype=BF16, device="cuda")
        self.dW = torch.empty((1, H, F), device="cuda")
        self.norm = pkg.RmsNorm.like(self.x, self.w, self.y, residual=self.res, h=self.h, eps=EPS)
        self.norm8 = pkg.RmsNorm.like(self.x, self.w, self.y8, scales=self.s, eps=EPS)
        self.rows = pkg.Rows8.like(self.x, self.q, self.e)
        self.product = pkg.I8Gemm.like(self.y8, self.s, self.W, self.ws, None, self.D)
        self.grad = pkg.Rows8Grad.like(self.q, self.e, self.dD, None, None, self.dW)
        self.fill(seed)

    def fill(self, seed):
        for i, t in enumerate((self.x, self.res, self.dy, self.dres, self.w, self.dD)):
            t.copy_(rnd(t.shape, BF16, seed + i))

    def run(self, stream=None):
        self.norm.run(self.x, self.w, self.y, residual=self.res, h=self.h, rstd=self.rstd, stream=stream)
        self.rows.pack(self.h, self.q, self.e, stream=stream)
        self.rows.unpack(self.q, self.e, self.back, stream=stream)
        self.norm.backward(self.dy, self.q, self.w, self.rstd, self.dx, self.dw, self.dres, self.e,
                           stream=stream)
        self.norm8.run(self.x, self.w, self.y8, scales=self.s, stream=stream)
        self.product.run(self.y8, self.s, self.W, self.ws, None, self.D, stream=stream)
        self.grad.run(self.q, self.e, self.dD, None, None, self.dW, stream=stream)

    def check(self):
        H, T = self.H, self.T
        h, r, y = norm_ref(self.x, self.res, self.w)
        assert torch.equal(self.h, h)
        near(self.y, y, (H + 8) * U * y.abs())
        q, e, v = blocks_ref(h)
        assert torch.equal(self.q.cpu(), q) and torch.equal(self.e.cpu(), e)
        assert torch.equal(self.back.cpu(), v)
        v = v.double().cuda()
        dx, size, dw, dw_size = backward_ref(self.dy, v, self.w, self.rstd, self.dres)
        near(self.dx, dx, (H + 12) * U * size)
        near(self.dw, dw, (T + 4) * U * dw_size)
        # (integers first: scaled ones would not cancel exactly in 64 bits either)
        D = self.y8.double() @ self.W[0].double().t() * self.s.double()[:, None] * self.ws[0].double()
        near(self.D, D, 4 * U * D.abs())
        dD = self.dD.double()
        near(self.dW[0], v.t() @ dD, 2 * T * U * (v.abs().t() @ dD.abs()))

    def status(self):
        for op in (self.norm, self.norm8, self.rows, self.product, self.grad):
            assert op.status() == pkg.GEMM_OK


@pytest.mark.parametrize("T,H,F", [(1, 256, 128), (64, 512, 320), (300, 1024, 264), (130, 200, 72)])
def test_captured_and_replayed_with_other_inputs(T, H, F):
    s = Set(T, H, F, 1)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        s.run()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for seed in (20, 40, 60):
        s.fill(seed)
        for t in (s.D, s.dW, s.dx, s.back, s.y):
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        s.check()
    s.status()


def test_two_sets_on_two_streams():
    """Handles of their own overlap; each stream's results are its own."""
    sets, streams = [Set(200, 768, 392, 1), Set(200, 768, 392, 50)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, stream in zip(sets, streams):
            s.run(stream=stream)
    torch.cuda.synchronize()
    for s in sets:
        s.check()
        s.status()


def test_inputs_made_on_the_given_stream():
    s, stream = Set(64, 512, 256, 1), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(20_000_000)
        s.fill(30)
    s.run(stream=stream)
    stream.synchronize()
    s.check()


def test_a_function_makes_its_result_for_a_given_stream():
    X, W = ints((40, 256), 1), ints((1, 128, 256), 2)
    xs, ws = rnd((40,), F32, 3).abs(), rnd((1, 128), F32, 4).abs()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    D = pkg.i8_matmul(X, xs, W, ws, out_dtype=F32, stream=stream)
    stream.synchronize()
    ref = X.double() @ W[0].double().t() * xs.double()[:, None] * ws[0].double()
    near(D, ref, 4 * U * ref.abs())


def test_equal_calls_give_equal_bits():
    s = Set(777, 1000, 520, 3)
    s.run()
    first = [t.clone() for t in (s.y, s.dx, s.dw, s.D, s.dW, s.s)]
    for _ in range(5):
        s.run()
        for a, b in zip(first, (s.y, s.dx, s.dw, s.D, s.dW, s.s)):
            assert torch.equal(a, b)


# ---------------------------------------------------------------- places
def at(t, offset):
    """t's values in rows of the same length that begin `offset` elements on."""
    flat = torch.empty(t.numel() + offset, dtype=t.dtype, device=t.device)
    out = flat[offset:].view(t.shape)
    out.copy_(t)
    return out


@pytest.mark.parametrize("offset", [1, 3, 8])
@pytest.mark.parametrize("H", [64, 1024])
def test_norm_from_any_element(offset, H):
    T = 9
    x, res, dy, dres = (at(rnd((T, H), BF16, i), offset) for i in range(4))
    w = at(rnd((H,), BF16, 7), offset)
    h, y, dx = (at(torch.zeros((T, H), dtype=BF16, device="cuda"), offset) for _ in range(3))
    rstd, dw = torch.empty(T, device="cuda"), torch.empty(H, device="cuda")
    op = pkg.RmsNorm.like(x, w, y, residual=res, h=h, eps=EPS)
    op.run(x, w, y, residual=res, h=h, rstd=rstd)
    h_ref, r, y_ref = norm_ref(x, res, w)
    assert torch.equal(h, h_ref)
    near(y, y_ref, (H + 8) * U * y_ref.abs())
    op.backward(dy, h, w, rstd, dx, dw, dres)
    dx_ref, size, dw_ref, dw_size = backward_ref(dy, h, w, rstd, dres)
    near(dx, dx_ref, (H + 12) * U * size)
    near(dw, dw_ref, (T + 4) * U * dw_size)
    q, e, v = held(T, H, 11)
    op.backward(dy, at(q, offset), w, rstd, dx, dw, dres, at(e, offset))
    dx_ref, size, dw_ref, dw_size = backward_ref(dy, v, w, rstd, dres)
    near(dx, dx_ref, (H + 12) * U * size)
    near(dw, dw_ref, (T + 4) * U * dw_size)
    y8 = at(torch.zeros((T, H), dtype=torch.int8, device="cuda"), offset)
    op8 = pkg.RmsNorm.like(x, w, y8, scales=rstd, eps=EPS)
    op8.run(x, w, y8, scales=rstd)
    hw = x.double() * w.double()
    ratio = 127 * hw / hw.abs().amax(1, keepdim=True)
    assert float((y8.double() - ratio).abs().max()) <= 0.5 + 127 * 6 * U
    done(op)
    done(op8)


@pytest.mark.parametrize("offset", [1, 4, 16])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows8_from_any_element(offset, dtype):
    X = at(rnd((33, 96), dtype, 1), offset)
    q, e = pkg.Rows8.empty(X)
    q, e, back = at(q, offset), at(e, offset), at(torch.zeros_like(X), offset)
    op = pkg.Rows8.like(X, q, e)
    op.pack(X, q, e)
    op.unpack(q, e, back)
    done(op)
    q_ref, e_ref, v = blocks_ref(X)
    assert torch.equal(q.cpu(), q_ref) and torch.equal(e.cpu(), e_ref) and torch.equal(back.cpu(), v)


@pytest.mark.parametrize("R", [3, 40, 150])
@pytest.mark.parametrize("plan", [None, "wide=1"])
def test_i8_from_any_element(R, plan):
    K, N = 144, 88
    X, W = at(ints((R, K), 1), 5), ints((1, N, K), 2)
    xs, ws = at(rnd((R,), F32, 3).abs(), 1), at(rnd((1, N), F32, 4).abs(), 3)
    D = at(torch.zeros((R, N), dtype=F16, device="cuda"), 1)
    with forced_plan(plan):
        op = pkg.I8Gemm.like(X, xs, W, ws, None, D)
    op.run(X, xs, W, ws, None, D)
    ref = X.double() @ W[0].double().t() * xs.double()[:, None] * ws[0].double()
    fits = ref.abs() < 65504  # others round to infinity, or to the largest number
    near(D[fits], ref[fits], 4 * U * ref[fits].abs())
    assert bool((D[~fits].abs() >= 65504).all()) and torch.equal(D[~fits] > 0, ref[~fits] > 0)
    # rows of W that the TMA unit could read, did they start where it can
    odd = at(W, 1)
    with pytest.raises(pkg.GemmError) as err:
        op.run(X, xs, odd, ws, None, D)
    assert err.value.code == pkg.GEMM_ERR_MISALIGNED
    done(op)


def test_i8_rows_of_weights_from_any_element():
    """Rows off the 16-byte grid may start anywhere."""
    R, K, N = 40, 131, 50
    X, W = ints((R, K), 1), at(ints((2, N, K), 2), 7)
    xs, ws = rnd((R,), F32, 3).abs(), rnd((2, N), F32, 4).abs() / 100
    off = offsets_of([15, 25])
    for plan in (None, "tiles=1", "wide=1"):
        with forced_plan(plan):
            D = pkg.i8_matmul(X, xs, W, ws, off, out_dtype=F32)
        for e, r in ((0, slice(0, 15)), (1, slice(15, 40))):
            ref = X[r].double() @ W[e].double().t() * xs[r, None].double() * ws[e].double()
            near(D[r], ref, 4 * U * ref.abs())


# ---------------------------------------------------------------- sizes
def test_rows_past_32_bit_offsets():
    """2.2 thousand million values: the last rows are as right as the first."""
    T, H = 540_000, 4096
    x = torch.empty((T, H), dtype=BF16, device="cuda")
    x.normal_(generator=torch.Generator("cuda").manual_seed(1))
    w = rnd((H,), BF16, 2)
    q, e = pkg.Rows8.empty(x)
    y, rstd, dw = torch.empty_like(x), torch.empty(T, device="cuda"), torch.empty(H, device="cuda")
    rows, norm = pkg.Rows8.like(x, q, e), pkg.RmsNorm.like(x, w, y, eps=EPS)
    rows.pack(x, q, e)
    norm.run(x, w, y, rstd=rstd)
    some = torch.tensor([0, 1, T // 2, T - 2, T - 1], device="cuda")
    q_ref, e_ref, v_ref = blocks_ref(x[some])
    assert torch.equal(q[some].cpu(), q_ref) and torch.equal(e[some].cpu(), e_ref)
    _, r, y_ref = norm_ref(x[some], None, w)
    near(y[some], y_ref, (H + 8) * U * y_ref.abs())
    # the gradient over y's buffer, of the gradient y itself
    norm.backward(y, q, w, rstd, y, dw, exponents=e)
    dx_ref, size, _, _ = backward_ref(y_ref.to(BF16), v_ref.cuda(), w, rstd[some], None)
    # y as the kernel rounded it is off by half a step of what it is here
    near(y[some], dx_ref, ((H + 12) * U + 2.0 ** -7) * size)
    rows.unpack(q, e, y)
    assert torch.equal(y[some].cpu(), v_ref)
    s = torch.empty(T, device="cuda")
    rows8 = pkg.Rows8.like(x, q, s)
    rows8.pack(x, q, s)
    top = x[some].float().abs().amax(1)
    assert torch.equal(s[some], (top.double() / 127).float())
    for op in (rows, norm, rows8):
        done(op)


@pytest.mark.parametrize("R", [4, 2000])
def test_weights_past_32_bit_offsets(R):
    """64 experts of 8192 x 8192: the last one's weights begin past 2^32."""
    E, K, N = 66, 8192, 8192
    W = torch.empty((E, N, K), dtype=torch.int8, device="cuda")
    W.random_(-127, 128, generator=torch.Generator("cuda").manual_seed(1))
    X, xs, ws = ints((R, K), 1), rnd((R,), F32, 2).abs(), rnd((E, N), F32, 3).abs() / 1e4
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:] = R // 2
    off[E] = R
    D = torch.empty((R, N), device="cuda")
    op = pkg.I8Gemm.like(X, xs, W, ws, off, D)
    op.run(X, xs, W, ws, off, D)
    done(op)
    for e, r in ((0, slice(0, R // 2)), (E - 1, slice(R // 2, R))):
        a, b, s = X[r].double(), W[e].double(), xs[r, None].double() * ws[e].double()
        ref = a @ b.t() * s
        near(D[r], ref, (4 * ref.abs() + K * (a.abs() @ b.abs().t()) * s) * U)


@pytest.mark.parametrize("T,H", [(0, 64), (4, 0), (0, 0)])
def test_nothing_to_do(T, H):
    x, w = torch.empty((T, H), dtype=BF16, device="cuda"), torch.empty(H, dtype=BF16, device="cuda")
    y, dw, rstd = torch.empty_like(x), torch.full((H,), 7.0, device="cuda"), torch.empty(T, device="cuda")
    op = pkg.RmsNorm.like(x, w, y, residual=x, h=y, eps=EPS)
    op.run(x, w, y, residual=x, h=y, rstd=rstd)
    op.backward(y, y, w, rstd, y, dw)
    done(op)
    assert not dw.any()  # the sum over no rows
    q, e = pkg.Rows8.empty(x)
    rows = pkg.Rows8.like(x, q, e)
    rows.pack(x, q, e)
    rows.unpack(q, e, x)
    done(rows)
    D = torch.empty((T, 16), device="cuda")
    W = torch.empty((1, 16, H), dtype=torch.int8, device="cuda")
    product = pkg.I8Gemm.like(q, rstd, W, torch.ones((1, 16), device="cuda"), None, D)
    product.run(q, rstd, W, torch.ones((1, 16), device="cuda"), None, D)
    done(product)
    B, dW = torch.empty((T, 16), dtype=BF16, device="cuda"), torch.full((1, H, 16), 7.0, device="cuda")
    grad = pkg.Rows8Grad.like(q, e, B, None, None, dW)
    grad.run(q, e, B, None, None, dW)
    done(grad)
    assert not dW.any() if T == 0 else True


def test_tensors_other_than_planned_are_refused():
    s = Set(8, 128, 64, 1)
    with pytest.raises(ValueError, match="x: planned"):
        s.norm.run(s.x[:7], s.w, s.y, residual=s.res, h=s.h)
    with pytest.raises(ValueError, match="planned with residual"):
        s.norm.run(s.x, s.w, s.y, h=s.h)
    with pytest.raises(ValueError, match="planned without scales"):
        s.norm.run(s.x, s.w, s.y, scales=s.s, residual=s.res, h=s.h)
    with pytest.raises(ValueError, match="no gradient"):
        s.norm8.backward(s.dy, s.x, s.w, s.rstd, s.dx, s.dw)
    with pytest.raises(ValueError, match="h: planned"):
        s.norm.backward(s.dy, s.q, s.w, s.rstd, s.dx, s.dw)  # 8 bits without exponents
    with pytest.raises(ValueError, match="exponents: planned"):
        s.norm.backward(s.dy, s.q, s.w, s.rstd, s.dx, s.dw, exponents=s.e[:, :3])
    with pytest.raises(ValueError, match="scales: planned"):
        s.rows.pack(s.x, s.q, s.s)
    with pytest.raises(ValueError, match="W: planned"):
        s.product.run(s.y8, s.s, s.W.view(torch.uint8), s.ws, None, s.D)
    with pytest.raises(ValueError, match="planned without offsets"):
        s.product.run(s.y8, s.s, s.W, s.ws, offsets_of([8]), s.D)
    with pytest.raises(ValueError, match="planned without C"):
        s.grad.run(s.q, s.e, s.dD, None, s.dW, s.dW)


WIDTHS = [1, 2, 5, 7, 8, 9, 15, 17, 23, 31, 33, 40, 47, 255, 257, 511, 1023, 2047, 2051, 4099, 8191]


def framed(shape, dtype, offset):
    """A tensor from element `offset` of a buffer of 77s, and that buffer."""
    n = shape[0] * shape[1]
    buf = torch.full((n + offset + 40,), 77, device="cuda").to(dtype)
    return buf[offset:offset + n].view(shape), buf


def kept(t, buf, offset):
    """Whether the buffer around the tensor is as it was."""
    return bool((buf[:offset] == 77).all()) and bool((buf[offset + t.numel():] == 77).all())


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,offset", [(1, 0), (2, 3), (9, 1), (40, 6)])
def test_rows8_of_any_width(H, dtype, T, offset):
    X, _ = framed((T, H), dtype, offset)
    X.copy_(rnd((T, H), dtype, H, 3.0))
    q, qbuf = framed((T, H), torch.int8, offset + 5)
    back, bbuf = framed((T, H), dtype, offset + 1)
    E = torch.empty((T, -(-H // 32)), dtype=torch.uint8, device="cuda")
    q_ref, e_ref, v_ref = (t.cuda() for t in blocks_ref(X))
    op = pkg.Rows8.like(X, q, E)
    op.pack(X, q, E)
    assert torch.equal(q, q_ref) and torch.equal(E, e_ref) and kept(q, qbuf, offset + 5)
    op2 = pkg.Rows8.like(back, q, E)
    op2.unpack(q, E, back)
    assert torch.equal(back.double(), v_ref) and kept(back, bbuf, offset + 1)
    s = torch.empty(T, device="cuda")
    op3 = pkg.Rows8.like(X, q, s)
    op3.pack(X, q, s)
    top = X.double().abs().amax(1)
    # two roundings of a scale; five of a ratio of at most 127
    near(s, top / 127, 2 * U * top / 127)
    ratio = 127 * X.double() / top[:, None]
    assert float((q.double() - ratio).abs().max()) <= 0.5 + 127 * 6 * U
    assert kept(q, qbuf, offset + 5)
    for o in (op, op2, op3):
        done(o)


@pytest.mark.parametrize("H", WIDTHS + [16385, 33333])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,offset", [(1, 0), (3, 5), (50, 1)])
@pytest.mark.parametrize("in_8_bits", [False, True])
def test_norm_of_any_width(H, dtype, T, offset, in_8_bits):
    """Forward and backward, h over x and dx over dresidual."""
    x, xbuf = framed((T, H), dtype, offset)
    x.copy_(rnd((T, H), dtype, 1, 2.0))
    res, _ = framed((T, H), dtype, offset + 2)
    res.copy_(rnd((T, H), dtype, 2))
    w = rnd((H,), dtype, 3)
    y, ybuf = framed((T, H), dtype, offset + 3)
    rstd, dw = torch.empty(T, device="cuda"), torch.empty(H, device="cuda")
    h_ref, r_ref, y_ref = norm_ref(x, res, w)
    op = pkg.RmsNorm.like(x, w, y, residual=res, h=x, eps=EPS)
    op.run(x, w, y, residual=res, h=x, rstd=rstd)
    assert torch.equal(x, h_ref) and kept(x, xbuf, offset) and kept(y, ybuf, offset + 3)
    near(rstd, r_ref, (H + 5) * U * r_ref)
    near(y, y_ref, (H + 8) * U * y_ref.abs())
    dy = rnd((T, H), dtype, 4)
    dx, dbuf = framed((T, H), dtype, offset + 1)
    dx.copy_(rnd((T, H), dtype, 5))
    dres = dx.clone()
    if in_8_bits:
        q, e, h = held(T, H, 7)
        q8, _ = framed((T, H), torch.int8, offset)
        q8.copy_(q)
        op.backward(dy, q8, w, rstd, dx, dw, dresidual=dx, exponents=e)
    else:
        h = h_ref
        op.backward(dy, x, w, rstd, dx, dw, dresidual=dx)
    dx_ref, size, dw_ref, dw_size = backward_ref(dy, h, w, rstd, dres)
    near(dx, dx_ref, (H + 12) * U * size, "dx")
    near(dw, dw_ref, (T + 4) * U * dw_size, "dweight")
    assert kept(dx, dbuf, offset + 1)
    done(op)


@pytest.mark.parametrize("H", [7, 257, 1001, 16385])
def test_norm_to_8_bits_of_any_width(H):
    T, offset = 40, 3
    x, _ = framed((T, H), F16, offset)
    x.copy_(rnd((T, H), F16, 1, 2.0))
    w = rnd((H,), F16, 3)
    y, ybuf = framed((T, H), torch.int8, offset)
    s = torch.empty(T, device="cuda")
    op = pkg.RmsNorm.like(x, w, y, scales=s, eps=EPS)
    op.run(x, w, y, scales=s)
    done(op)
    _, _, y_ref = norm_ref(x, None, w)
    top = y_ref.abs().amax(1)
    near(s, top / 127, (H + 9) * U * top / 127)
    hw = x.double() * w.double()
    ratio = 127 * hw / hw.abs().amax(1, keepdim=True)
    assert float((y.double() - ratio).abs().max()) <= 0.5 + 127 * 6 * U
    assert kept(y, ybuf, offset)


@pytest.mark.parametrize("H", [64, 1024, 1028, 2048, 4096, 8192, 8200, 16384, 16392])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("offset", [0, 1])
def test_norm_backward_of_as_many_rows_as_blocks_take(H, dtype, offset):
    """More rows than blocks, so that every block's partial sums are in use, and
    those of a handle beside it stay what they are."""
    T = 2000
    x, _ = framed((T, H), dtype, offset)
    x.copy_(rnd((T, H), dtype, 1))
    w, dy = rnd((H,), dtype, 2), rnd((T, H), dtype, 3)
    rstd = rnd((T,), F32, 4).abs() + 0.5
    dx, dw, dw2 = torch.empty_like(dy), torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    ops = [pkg.RmsNorm.like(x, w, torch.empty_like(x), eps=EPS) for _ in range(2)]
    ops[0].backward(dy, x, w, rstd, dx, dw)
    ops[1].backward(dy, x, w, rstd, dx, dw2)
    for o in ops:
        done(o)
    dx_ref, size, dw_ref, dw_size = backward_ref(dy, x, w, rstd, None)
    near(dx, dx_ref, (H + 12) * U * size, "dx")
    near(dw, dw_ref, (T + 4) * U * dw_size, "dweight")
    assert torch.equal(dw, dw2)


@pytest.mark.parametrize("H", [64, 1001, 1024, 40000])
@pytest.mark.parametrize("dtype,low,high", [(BF16, 225, 249), (F32, 225, 249), (BF16, 1, 12), (F16, 100, 130)])
def test_norm_backward_from_steps_at_the_ends_of_the_range(H, dtype, low, high):
    """Block rows whose exponents lie near the ends: with h r of about 1, as the
    forward pass leaves it, no intermediate value may leave fp32's range."""
    T = 5
    q = ints((T, H), 1, -127, 128)
    E = ints((T, -(-H // 32)), 2, 0, 4).to(torch.uint8)
    E += torch.linspace(low, high - 4, T, device="cuda").round().to(torch.uint8)[:, None]
    h = q.double() * torch.exp2(E.cpu().double() - 127).cuda().repeat_interleave(32, 1)[:, :H]
    rstd = (1 / torch.sqrt((h * h).mean(1))).float()
    w, dy = rnd((H,), dtype, 3), rnd((T, H), dtype, 4, 2.0 ** -10)
    dx, dw = torch.empty_like(dy), torch.empty(H, device="cuda")
    op = pkg.RmsNorm.like(dy, w, torch.empty_like(dy), eps=EPS)
    op.backward(dy, q, w, rstd, dx, dw, exponents=E)
    done(op)
    dx_ref, size, dw_ref, dw_size = backward_ref(dy, h, w, rstd, None)
    # (where values are below fp32's normal range, a rounding is 2^-150 instead
    # of relative: 12 of them, times r at most 2^126 where h is that small)
    tiny = 12 * 2.0 ** -150 * rstd.double()[:, None].clamp_min(1.0) * (1 + h.abs())
    inf = torch.finfo(dtype).max
    fits = dx_ref.abs() < inf
    near(torch.where(fits, dx, torch.zeros_like(dx)), torch.where(fits, dx_ref, 0.0),
         torch.where(fits, (H + 12) * U * size + tiny, 0.0), "dx")
    # a term's dy h may be below the normal range, too: off by at most 2^-150
    # there, which r then multiplies (of h of about 2^-118 and r of 2^118, 2^-32)
    near(dw, dw_ref, (T + 4) * U * dw_size + float(rstd.double().sum()) * 2.0 ** -150, "dweight")
