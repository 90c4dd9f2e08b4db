"""An expert (mixture-of-experts) layer made of the library's operators.

    Y[t] = sum_j g[t, j] W2[e] relu(W1[e] X[t]),   e = the j-th expert of t,

the gates g being the softmax of the k largest of the router's logits X R^T.

``ExpertLayer`` is the training form, forward and backward: routing, rows into
expert order, two grouped products, the gated sum, and the gradients of all
of them.  ``ExpertDecoder`` is the serving form: the experts' weights in 4 bits,
or in 8 with the rows rounded to 8 as well, and the step recorded once as a CUDA
graph, because at a few tokens the calls cost more than the kernels.  Both are
planned for a fixed number of tokens and hold every buffer, so a step allocates
nothing of theirs.

With a `norm` (its weights) the layer is a block of a residual stream: it takes
the block before it and the stream, h = X + residual is the new stream, and the
experts see h normalised, Y = experts(rmsnorm(h)).  With `keep8` the training
form keeps what its backward pass reads of rows (the stream, the normalised and
the sorted rows) in 8 bits, 33 bytes for 32 values, and puts the gradients into the
16-bit buffers that this frees: of a row's H values it holds 3.03 bytes instead of
4 for each of the k sorted rows, and, with a norm, 4.06 instead of 4 for the token,
whose h (2 bytes) the caller then need not keep.

    python -m dense_tiled_gemm_02_gb300.expert_layer [--tokens 4096 ...]

trains a layer for some steps towards another one's outputs, then serves it
in 4 (or 8) bits, and prints the losses, the times and that form's error.
"""
from __future__ import annotations

import argparse

import torch

import dense_tiled_gemm_02_gb300 as gemm
from dense_tiled_gemm_02_gb300.experts import (GroupedGemm, Permute, Route, W4Gemm, _on_one_device,
                                               _Planned, pack_w4)
from dense_tiled_gemm_02_gb300.rows import I8Gemm, RmsNorm, Rows8, Rows8Grad


def quantize_w4(w: torch.Tensor, group: int):
    """Weights (..., N, K) as 4-bit values with a scale and zero point for each
    `group` along K: (packed, scales, zeros), (q - zero) * scale nearest to w.
    The scales have w's type."""
    K = w.shape[-1]
    G = -(-K // group)
    x = torch.nn.functional.pad(w.float(), (0, G * group - K)).unflatten(-1, (G, group))
    lo, hi = x.amin(-1).clamp(max=0), x.amax(-1).clamp(min=0)  # 0 stays a value
    scales = ((hi - lo) / 15).to(w.dtype)
    s = scales.float().clamp(min=1e-30)
    zeros = (-lo / s).round().clamp(0, 15)
    q = (x / s.unsqueeze(-1) + zeros.unsqueeze(-1)).round().clamp(0, 15)
    return pack_w4(q.flatten(-2)[..., :K]), scales, zeros.to(torch.uint8)


def quantize_w8(w: torch.Tensor):
    """Weights (E, N, K) as 8-bit integers with a scale for each output: (q,
    scales (E, N) fp32), q * scale nearest to w."""
    E, N, K = w.shape
    rows = w.reshape(E * N, K)
    q, scales = Rows8.empty(rows, block=False)
    op = Rows8.like(rows, q, scales)
    op.pack(rows, q, scales)
    op.close()
    return q.view(E, N, K), scales.view(E, N)


def _sizes(router, W1, W2, norm=None):
    """(E, F, H) of a layer's weights, which must agree."""
    E, F, H = W1.shape
    if tuple(router.shape) != (E, H) or tuple(W2.shape) != (E, H, F):
        raise ValueError(f"router {tuple(router.shape)} and W2 {tuple(W2.shape)} do not go with W1 "
                         f"{tuple(W1.shape)}: {(E, H)} and {(E, H, F)} do")
    for name, t in (("router", router), ("W1", W1), ("W2", W2)):
        if t.dtype != W1.dtype or t.dtype not in (torch.float16, torch.bfloat16):
            raise ValueError(f"{name} is {t.dtype}: the weights are of one 16-bit type")
    if norm is not None and (tuple(norm.shape) != (H,) or
                             norm.dtype not in (W1.dtype, torch.float32)):
        raise ValueError(f"norm must be {H} weights of {W1.dtype} or float32, got "
                         f"{tuple(norm.shape)} {norm.dtype}")
    _on_one_device(W1.device, router=router, W2=W2, norm=norm)
    return E, F, H


def _check(ops, what: str) -> None:
    """Synchronise; raise if a kernel of these handles reported an error."""
    stream = torch.cuda.current_stream()
    for rc in [op.status(stream) for op in ops]:
        if rc != gemm.GEMM_OK:
            raise gemm.GemmError(rc, what)


class ExpertLayer:
    """The layer for T tokens in training.  router is E x H, W1 E x F x H and
    W2 E x H x F, of one 16-bit type; `grads` holds the gradients of all three
    after `backward`, and that of `norm`.  norm, keep8: see the module."""

    def __init__(self, tokens: int, router, W1, W2, k: int, norm=None, eps: float = 1e-6,
                 keep8: bool = False):
        E, F, H = _sizes(router, W1, W2, norm)
        T, R, dtype, dev = tokens, tokens * k, W1.dtype, W1.device
        self.router, self.W1, self.W2, self.norm, self.keep8 = router, W1, W2, norm, keep8

        def new(*shape, dtype=dtype):
            return torch.empty(shape, dtype=dtype, device=dev)

        X, Y = new(T, H), new(T, H)
        # the dense products do not look at what they are given: checked here
        self._tokens = {name: _Planned(name, X)
                        for name in ("X", "Y", "dY", "dX", "residual", "h", "dh")}
        self.logits = new(T, E, dtype=torch.float32)
        self.route = Route.like(self.logits, k)
        self.experts, self.gates, self.offsets, self.row_slot, self.slot_row = self.route.outputs()
        self.permute = Permute.like(X, self.slot_row)
        self.Xs, self.hid, self.Ys = new(R, H), new(R, F), new(R, H)
        self.dYs, self.dhid = new(R, H), new(R, F)
        # kept in 8 bits, rows leave their 16-bit buffer free for their gradient
        self.dXs = self.Xs if keep8 else new(R, H)
        self.dgates, self.dlogits = torch.empty_like(self.gates), torch.empty_like(self.logits)
        self.grads = {"router": torch.empty_like(router), "W1": torch.empty_like(W1),
                      "W2": torch.empty_like(W2)}
        g, off = self.grads, self.offsets
        # forward: rows times the transposed weights, which are K-contiguous
        self.logit_gemm = gemm.Gemm.like(X, router.T, None, self.logits)
        self.up = GroupedGemm.like(self.Xs, W1.transpose(1, 2), off, None, self.hid)
        self.down = GroupedGemm.like(self.hid, W2.transpose(1, 2), off, None, self.Ys)
        # backward: the weights as they lie, and the rows' outer products
        self.down_dx = GroupedGemm.like(self.dYs, W2, off, None, self.dhid)
        self.up_dx = GroupedGemm.like(self.dhid, W1, off, None, self.dXs)
        self.down_dw = GroupedGemm.like(self.dYs, self.hid, off, None, g["W2"])
        self.dlog = new(T, E)
        self.router_dx = gemm.Gemm.like(self.dlog, router, Y, Y)
        self._ops = [self.logit_gemm, self.route, self.permute, self.up, self.down, self.down_dx,
                     self.up_dx, self.down_dw, self.router_dx]
        if keep8:
            # the product's 8-bit operand is its first: the gradient comes transposed
            self._dW1 = new(E, H, F)
            g["W1"] = self._dW1.transpose(1, 2)
            self.Xs8 = Rows8.empty(self.Xs)
            self.keep_rows = Rows8.like(self.Xs, *self.Xs8)
            self.up_dw = Rows8Grad.like(*self.Xs8, self.dhid, off, None, self._dW1)
            self._ops.append(self.keep_rows)
        else:
            self.up_dw = GroupedGemm.like(self.dhid, self.Xs, off, None, g["W1"])
        if norm is not None:
            g["norm"] = new(H, dtype=torch.float32)
            self.Xn, self.rstd = new(T, H), new(T, dtype=torch.float32)
            self.dXn = self.Xn if keep8 else new(T, H)
            self.norm_op = RmsNorm.like(X, norm, self.Xn, residual=X, h=X, eps=eps)
            self._ops.append(self.norm_op)
        if norm is not None and keep8:
            self.h8, self.Xn8 = Rows8.empty(X), Rows8.empty(X)
            self.keep = Rows8.like(X, *self.h8)
            self._drouter = new(1, H, E)
            g["router"] = self._drouter[0].T
            self.router_dw = Rows8Grad.like(*self.Xn8, self.dlog, None, None, self._drouter)
            self._ops.append(self.keep)
        else:
            self.router_dw = gemm.Gemm.like(self.dlog.T, X, None, g["router"])
        self._ops += [self.up_dw, self.router_dw]

    def _check_tokens(self, **tensors) -> None:
        for name, t in tensors.items():
            self._tokens[name].pointer(t)

    def _stream(self, residual, what: str, **others) -> None:
        """The residual stream's operands, which go with a norm."""
        given = [residual, *others.values()]
        if any((t is None) != (self.norm is None) for t in given):
            raise ValueError(f"{what} go with a norm, and only with one")
        if self.norm is not None:
            self._check_tokens(**others)

    def forward(self, X: torch.Tensor, Y: torch.Tensor, residual=None, h=None) -> None:
        """Enqueue Y = layer(X), both T x H; with a norm also the new stream h =
        X + residual, which may be either of them, and Y of its normalised rows."""
        self._check_tokens(X=X, Y=Y)
        self._stream(residual, "residual and h", h=h)
        if self.norm is not None:
            self._check_tokens(residual=residual)
            self.norm_op.run(X, self.norm, self.Xn, residual=residual, h=h, rstd=self.rstd)
            if self.keep8:
                self.keep.pack(h, *self.h8)
                self.keep.pack(self.Xn, *self.Xn8)
            X = self.Xn
        self.logit_gemm.run(X, self.router.T, None, self.logits)
        self.route.run(self.logits, self.experts, self.gates, self.offsets, self.row_slot,
                       self.slot_row)
        self.permute.gather(X, self.row_slot, self.slot_row, self.Xs)
        self.up.run(self.Xs, self.W1.transpose(1, 2), self.offsets, None, self.hid)
        if self.keep8:
            self.keep_rows.pack(self.Xs, *self.Xs8)
        self.hid.clamp_(min=0)
        self.down.run(self.hid, self.W2.transpose(1, 2), self.offsets, None, self.Ys)
        self.permute.combine(self.Ys, self.slot_row, self.gates, Y)

    def backward(self, X: torch.Tensor, dY: torch.Tensor, dX: torch.Tensor, h=None,
                 dh=None) -> None:
        """Enqueue the gradients for dY, after `forward` with this X: dX and
        `grads`.  With a norm: for dh, too, which comes to h by the stream (h as
        `forward` made it, or None where keep8 keeps it), and dX is the gradient
        of X and of residual; X itself is then not looked at."""
        self._check_tokens(X=X, dY=dY, dX=dX)
        if self.norm is None or not self.keep8:
            self._stream(dh, "h and dh", h=h)
        elif dh is None or h is not None:
            raise ValueError("dh goes with a norm; h is kept by the layer")
        if self.norm is not None:
            self._check_tokens(dh=dh)
        off, g = self.offsets, self.grads
        self.permute.combine_backward(dY, self.Ys, self.row_slot, self.slot_row, self.gates,
                                      self.dYs, self.dgates)
        self.down_dw.run(self.dYs, self.hid, off, None, g["W2"])
        self.down_dx.run(self.dYs, self.W2, off, None, self.dhid)
        # rows of no expert hold anything: chosen away, not multiplied away
        self.dhid.masked_fill_(self.hid <= 0, 0)
        if self.keep8:
            self.up_dw.run(*self.Xs8, self.dhid, off, None, self._dW1)
        else:
            self.up_dw.run(self.dhid, self.Xs, off, None, g["W1"])
        self.up_dx.run(self.dhid, self.W1, off, None, self.dXs)
        dXn = dX if self.norm is None else self.dXn
        self.permute.combine(self.dXs, self.slot_row, None, dXn)
        self.route.backward(self.logits, self.experts, self.gates, self.dgates, self.dlogits)
        self.dlog.copy_(self.dlogits)
        self.router_dx.run(self.dlog, self.router, dXn, dXn)  # dXn + dlogits R
        if self.norm is None:
            self.router_dw.run(self.dlog.T, X, None, g["router"])
            return
        if self.keep8:
            self.router_dw.run(*self.Xn8, self.dlog, None, None, self._drouter)
            h, exponents = self.h8
        else:
            self.router_dw.run(self.dlog.T, self.Xn, None, g["router"])
            exponents = None
        self.norm_op.backward(dXn, h, self.norm, self.rstd, dX, g["norm"], dresidual=dh,
                              exponents=exponents)

    def check(self) -> None:
        """Synchronise; raise if a kernel reported an error."""
        _check(self._ops, "expert layer")


class ExpertDecoder:
    """The layer for T tokens in serving, its experts' weights in 4 bits, or in 8
    (`bits`) with the rows they meet in 8 bits.  `step` works on the buffers X and
    Y (and residual and h, with a norm); the graph is recorded by the first."""

    def __init__(self, tokens: int, router, W1, W2, k: int, group: int = 128, bits: int = 4,
                 norm=None, eps: float = 1e-6):
        E, F, H = _sizes(router, W1, W2, norm)
        if bits not in (4, 8):
            raise ValueError(f"weights are of 4 or 8 bits, not {bits}")
        dtype, dev = W1.dtype, W1.device
        self.router, self.norm, self.bits = router, norm, bits
        self.X = torch.zeros(tokens, H, dtype=dtype, device=dev)
        self.Y = torch.empty_like(self.X)
        self.logits = torch.empty(tokens, E, dtype=torch.float32, device=dev)
        self.route = Route.like(self.logits, k)
        self.experts, self.gates, self.offsets, self.row_slot, self.slot_row = self.route.outputs()
        self.permute = Permute.like(self.X, self.slot_row)
        self.Xs = torch.empty(tokens * k, H, dtype=dtype, device=dev)
        self.hid = torch.empty(tokens * k, F, dtype=dtype, device=dev)
        self.Ys = torch.empty_like(self.Xs)
        self.logit_gemm = gemm.Gemm.like(self.X, router.T, None, self.logits)
        self._ops = [self.logit_gemm, self.route, self.permute]
        if bits == 4:
            self.w1, self.w2 = quantize_w4(W1, group), quantize_w4(W2, group)
            self.up = W4Gemm.like(self.Xs, *self.w1, self.offsets, self.hid, group)
            self.down = W4Gemm.like(self.hid, *self.w2, self.offsets, self.Ys, group)
        else:
            self.w1, self.w2 = quantize_w8(W1), quantize_w8(W2)
            self.Xs8, self.hid8 = Rows8.empty(self.Xs, False), Rows8.empty(self.hid, False)
            self.round_x = Rows8.like(self.Xs, *self.Xs8)
            self.round_hid = Rows8.like(self.hid, *self.hid8)
            self.up = I8Gemm.like(*self.Xs8, *self.w1, self.offsets, self.hid)
            self.down = I8Gemm.like(*self.hid8, *self.w2, self.offsets, self.Ys)
            self._ops += [self.round_x, self.round_hid]
        self._ops += [self.up, self.down]
        if norm is not None:
            self.residual, self.h = torch.zeros_like(self.X), torch.empty_like(self.X)
            self.Xn = torch.empty_like(self.X)
            self.norm_op = RmsNorm.like(self.X, norm, self.Xn, residual=self.residual, h=self.h,
                                        eps=eps)
            self._ops.append(self.norm_op)
        self._graph = None

    def _enqueue(self) -> None:
        X = self.X
        if self.norm is not None:
            self.norm_op.run(X, self.norm, self.Xn, residual=self.residual, h=self.h)
            X = self.Xn
        self.logit_gemm.run(X, self.router.T, None, self.logits)
        self.route.run(self.logits, self.experts, self.gates, self.offsets, self.row_slot,
                       self.slot_row)
        self.permute.gather(X, self.row_slot, self.slot_row, self.Xs)
        if self.bits == 4:
            self.up.run(self.Xs, *self.w1, self.offsets, self.hid)
            self.hid.clamp_(min=0)
            self.down.run(self.hid, *self.w2, self.offsets, self.Ys)
        else:
            self.round_x.pack(self.Xs, *self.Xs8)
            self.up.run(*self.Xs8, *self.w1, self.offsets, self.hid)
            self.hid.clamp_(min=0)
            self.round_hid.pack(self.hid, *self.hid8)
            self.down.run(*self.hid8, *self.w2, self.offsets, self.Ys)
        self.permute.combine(self.Ys, self.slot_row, self.gates, self.Y)

    def step(self, X: torch.Tensor, residual=None) -> torch.Tensor:
        """Enqueue Y = layer(X) for T x H tokens; returns the buffer Y, which
        the next step overwrites.  With a norm, the new stream is the buffer h."""
        if X.shape != self.X.shape:
            raise ValueError(f"X: planned for {tuple(self.X.shape)}, got {tuple(X.shape)}")
        if (residual is None) != (self.norm is None):
            raise ValueError("residual goes with a norm, and only with one")
        if residual is not None:
            if residual.shape != X.shape:
                raise ValueError(f"residual: planned for {tuple(X.shape)}, got "
                                 f"{tuple(residual.shape)}")
            self.residual.copy_(residual)
        self.X.copy_(X)
        if self._graph is None:
            side = torch.cuda.Stream(self.X.device)  # loads the kernels
            side.wait_stream(torch.cuda.current_stream(self.X.device))
            with torch.cuda.stream(side):
                self._enqueue()
            torch.cuda.current_stream(self.X.device).wait_stream(side)
            torch.cuda.synchronize(self.X.device)
            self._graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self._graph):
                self._enqueue()
        self._graph.replay()
        return self.Y

    def check(self) -> None:
        """Synchronise; raise if a kernel reported an error."""
        _check(self._ops, "expert decoder")


def random_weights(E: int, H: int, F: int, dtype=torch.bfloat16, device="cuda", seed: int = 0):
    """(router, W1, W2) with rows of unit length, so values stay near one."""
    g = torch.Generator(device=device).manual_seed(seed)

    def draw(*shape):
        w = torch.randn(shape, generator=g, device=device) / shape[-1] ** 0.5
        return w.to(dtype)

    return draw(E, H), draw(E, F, H), draw(E, H, F)


def _milliseconds(call, n: int) -> float:
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for _ in range(3):
        call()
    torch.cuda.synchronize()
    a.record()
    for _ in range(n):
        call()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / n


def arguments(argv=None) -> argparse.Namespace:
    p = argparse.ArgumentParser(description=__doc__,
                                formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--tokens", type=int, default=4096, help="of a training step")
    p.add_argument("--decode-tokens", type=int, default=16, help="of a serving step")
    p.add_argument("--hidden", type=int, default=2048)
    p.add_argument("--inner", type=int, default=1024, help="width inside an expert")
    p.add_argument("--experts", type=int, default=64)
    p.add_argument("-k", type=int, default=4, help="experts of a token")
    p.add_argument("--norm", action="store_true", help="a residual stream and its norm before it")
    p.add_argument("--keep8", action="store_true", help="train from rows kept in 8 bits")
    p.add_argument("--bits", type=int, choices=(4, 8), default=4, help="of the served weights")
    p.add_argument("--steps", type=int, default=8)
    p.add_argument("--rate", type=float, default=0.03,
                   help="learning rate, for a token's squared distance")
    return p.parse_args(argv)


def main(argv=None) -> None:
    a = arguments(argv)
    if not torch.cuda.is_available():
        raise SystemExit("a CUDA device is needed")
    # the goal is the layer itself with other second matrices
    router, W1, W2 = random_weights(a.experts, a.hidden, a.inner)
    norm = torch.ones(a.hidden, device="cuda") if a.norm else None
    goal = ExpertLayer(a.tokens, router, W1, random_weights(a.experts, a.hidden, a.inner, seed=1)[2],
                       a.k, norm)
    layer = ExpertLayer(a.tokens, router, W1, W2, a.k, norm, keep8=a.keep8)
    X = torch.randn(a.tokens, a.hidden, device="cuda").to(W1.dtype)
    Y, want, dX = (torch.empty_like(X) for _ in range(3))
    # the stream starts as zeros, and what comes back by it as well
    stream = {"residual": torch.zeros_like(X), "h": torch.empty_like(X)} if a.norm else {}
    back = {"h": None if a.keep8 else stream["h"], "dh": stream["residual"]} if a.norm else {}
    goal.forward(X, want, **stream)
    for step in range(a.steps):
        layer.forward(X, Y, **stream)
        diff = Y.float() - want.float()
        print(f"step {step}: loss {diff.square().mean().item():.5f}")
        layer.backward(X, (diff * (2 / a.tokens)).to(Y.dtype), dX, **back)
        for name in ("router", "W1", "W2"):
            getattr(layer, name).sub_(layer.grads[name], alpha=a.rate)
    layer.check()
    dY = torch.randn_like(Y)
    print(f"training step, {a.tokens} tokens: forward "
          f"{_milliseconds(lambda: layer.forward(X, Y, **stream), 10):.3f} ms, backward "
          f"{_milliseconds(lambda: layer.backward(X, dY, dX, **back), 10):.3f} ms")
    few = ExpertLayer(a.decode_tokens, router, W1, W2, a.k, norm)
    decoder = ExpertDecoder(a.decode_tokens, router, W1, W2, a.k, bits=a.bits, norm=norm)
    x, y = X[:a.decode_tokens], Y[:a.decode_tokens].clone()
    stream = {name: t[:a.decode_tokens] for name, t in stream.items()}
    residual = (stream["residual"],) if a.norm else ()
    few.forward(x, y, **stream)
    error = (decoder.step(x, *residual).float() - y.float()).norm() / y.float().norm()
    decoder.check()
    print(f"serving step, {a.decode_tokens} tokens: {a.bits}-bit weights "
          f"{_milliseconds(lambda: decoder.step(x, *residual), 50) * 1e3:.1f} us, 16-bit weights "
          f"{_milliseconds(lambda: few.forward(x, y, **stream), 50) * 1e3:.1f} us, "
          f"{a.bits}-bit output off by {error:.3f}")


if __name__ == "__main__":
    main()
