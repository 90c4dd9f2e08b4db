"""An expert (mixture-of-experts) layer made of the library's operators.

    Y[t] = sum_j g[t, j] W2[e] relu(W1[e] X[t]),   e = the j-th expert of t,

the gates g being the softmax of the k largest of the router's logits X R^T.

``ExpertLayer`` is the training form, forward and backward: routing, rows into
expert order, two grouped products, the gated sum, and the gradients of all
of them.  ``ExpertDecoder`` is the serving form: the experts' weights in 4 bits
and the step recorded once as a CUDA graph, because at a few tokens the calls
cost more than the kernels.  Both are planned for a fixed number of tokens and
hold every buffer, so a step allocates nothing of theirs.

    python -m dense_tiled_gemm_02_gb300.expert_layer [--tokens 4096 ...]

trains a layer for some steps towards another one's outputs, then serves it
in 4 bits, and prints the losses, the times and the 4-bit form's error.
"""
from __future__ import annotations

import argparse

import torch

import dense_tiled_gemm_02_gb300 as gemm
from dense_tiled_gemm_02_gb300.experts import (GroupedGemm, Permute, Route, W4Gemm, _on_one_device,
                                               _Planned, pack_w4)


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


def _sizes(router, W1, W2):
    """(E, F, H) of a layer's weights, which must agree."""
    E, F, H = W1.shape
    if tuple(router.shape) != (E, H) or tuple(W2.shape) != (E, H, F):
        raise ValueError(f"router {tuple(router.shape)} and W2 {tuple(W2.shape)} do not go with W1 "
                         f"{tuple(W1.shape)}: {(E, H)} and {(E, H, F)} do")
    for name, t in (("router", router), ("W1", W1), ("W2", W2)):
        if t.dtype != W1.dtype or t.dtype not in (torch.float16, torch.bfloat16):
            raise ValueError(f"{name} is {t.dtype}: the weights are of one 16-bit type")
    _on_one_device(W1.device, router=router, W2=W2)
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
    after `backward`."""

    def __init__(self, tokens: int, router, W1, W2, k: int):
        E, F, H = _sizes(router, W1, W2)
        T, R, dtype, dev = tokens, tokens * k, W1.dtype, W1.device
        self.router, self.W1, self.W2 = router, W1, W2

        def new(*shape, dtype=dtype):
            return torch.empty(shape, dtype=dtype, device=dev)

        X, Y = new(T, H), new(T, H)
        # the dense products do not look at what they are given: checked here
        self._tokens = {name: _Planned(name, X) for name in ("X", "Y", "dY", "dX")}
        self.logits = new(T, E, dtype=torch.float32)
        self.route = Route.like(self.logits, k)
        self.experts, self.gates, self.offsets, self.row_slot, self.slot_row = self.route.outputs()
        self.permute = Permute.like(X, self.slot_row)
        self.Xs, self.hid, self.Ys = new(R, H), new(R, F), new(R, H)
        self.dYs, self.dhid, self.dXs = new(R, H), new(R, F), new(R, H)
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
        self.up_dw = GroupedGemm.like(self.dhid, self.Xs, off, None, g["W1"])
        self.dlog = new(T, E)
        self.router_dx = gemm.Gemm.like(self.dlog, router, Y, Y)
        self.router_dw = gemm.Gemm.like(self.dlog.T, X, None, g["router"])

    def _check_tokens(self, **tensors) -> None:
        for name, t in tensors.items():
            self._tokens[name].pointer(t)

    def forward(self, X: torch.Tensor, Y: torch.Tensor) -> None:
        """Enqueue Y = layer(X), both T x H."""
        self._check_tokens(X=X, Y=Y)
        self.logit_gemm.run(X, self.router.T, None, self.logits)
        self.route.run(self.logits, self.experts, self.gates, self.offsets, self.row_slot,
                       self.slot_row)
        self.permute.gather(X, self.row_slot, self.slot_row, self.Xs)
        self.up.run(self.Xs, self.W1.transpose(1, 2), self.offsets, None, self.hid)
        self.hid.clamp_(min=0)
        self.down.run(self.hid, self.W2.transpose(1, 2), self.offsets, None, self.Ys)
        self.permute.combine(self.Ys, self.slot_row, self.gates, Y)

    def backward(self, X: torch.Tensor, dY: torch.Tensor, dX: torch.Tensor) -> None:
        """Enqueue the gradients for dY, after `forward` with this X: dX and
        `grads`."""
        self._check_tokens(X=X, dY=dY, dX=dX)
        off, g = self.offsets, self.grads
        self.permute.combine_backward(dY, self.Ys, self.row_slot, self.slot_row, self.gates,
                                      self.dYs, self.dgates)
        self.down_dw.run(self.dYs, self.hid, off, None, g["W2"])
        self.down_dx.run(self.dYs, self.W2, off, None, self.dhid)
        # rows of no expert hold anything: chosen away, not multiplied away
        self.dhid.masked_fill_(self.hid <= 0, 0)
        self.up_dw.run(self.dhid, self.Xs, off, None, g["W1"])
        self.up_dx.run(self.dhid, self.W1, off, None, self.dXs)
        self.permute.combine(self.dXs, self.slot_row, None, dX)
        self.route.backward(self.logits, self.experts, self.gates, self.dgates, self.dlogits)
        self.dlog.copy_(self.dlogits)
        self.router_dx.run(self.dlog, self.router, dX, dX)  # dX + dlogits R
        self.router_dw.run(self.dlog.T, X, None, g["router"])

    def check(self) -> None:
        """Synchronise; raise if a kernel reported an error."""
        _check((self.logit_gemm, self.route, self.permute, self.up, self.down, self.down_dx,
                self.up_dx, self.down_dw, self.up_dw, self.router_dx, self.router_dw),
               "expert layer")


class ExpertDecoder:
    """The layer for T tokens in serving, its experts' weights in 4 bits.
    `step` works on the buffers X and Y; the graph is recorded by the first."""

    def __init__(self, tokens: int, router, W1, W2, k: int, group: int = 128):
        E, F, H = _sizes(router, W1, W2)
        dtype, dev = W1.dtype, W1.device
        self.router = router
        self.w1, self.w2 = quantize_w4(W1, group), quantize_w4(W2, group)
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
        self.up = W4Gemm.like(self.Xs, *self.w1, self.offsets, self.hid, group)
        self.down = W4Gemm.like(self.hid, *self.w2, self.offsets, self.Ys, group)
        self._graph = None

    def _enqueue(self) -> None:
        self.logit_gemm.run(self.X, self.router.T, None, self.logits)
        self.route.run(self.logits, self.experts, self.gates, self.offsets, self.row_slot,
                       self.slot_row)
        self.permute.gather(self.X, self.row_slot, self.slot_row, self.Xs)
        self.up.run(self.Xs, *self.w1, self.offsets, self.hid)
        self.hid.clamp_(min=0)
        self.down.run(self.hid, *self.w2, self.offsets, self.Ys)
        self.permute.combine(self.Ys, self.slot_row, self.gates, self.Y)

    def step(self, X: torch.Tensor) -> torch.Tensor:
        """Enqueue Y = layer(X) for T x H tokens; returns the buffer Y, which
        the next step overwrites."""
        if X.shape != self.X.shape:
            raise ValueError(f"X: planned for {tuple(self.X.shape)}, got {tuple(X.shape)}")
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
        _check((self.logit_gemm, self.route, self.permute, self.up, self.down), "expert decoder")


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
    goal = ExpertLayer(a.tokens, router, W1, random_weights(a.experts, a.hidden, a.inner, seed=1)[2],
                       a.k)
    layer = ExpertLayer(a.tokens, router, W1, W2, a.k)
    X = torch.randn(a.tokens, a.hidden, device="cuda").to(W1.dtype)
    Y, want, dX = (torch.empty_like(X) for _ in range(3))
    goal.forward(X, want)
    for step in range(a.steps):
        layer.forward(X, Y)
        diff = Y.float() - want.float()
        print(f"step {step}: loss {diff.square().mean().item():.5f}")
        layer.backward(X, (diff * (2 / a.tokens)).to(Y.dtype), dX)
        for name in ("router", "W1", "W2"):
            getattr(layer, name).sub_(layer.grads[name], alpha=a.rate)
    layer.check()
    dY = torch.randn_like(Y)
    print(f"training step, {a.tokens} tokens: forward "
          f"{_milliseconds(lambda: layer.forward(X, Y), 10):.3f} ms, backward "
          f"{_milliseconds(lambda: layer.backward(X, dY, dX), 10):.3f} ms")
    few = ExpertLayer(a.decode_tokens, router, W1, W2, a.k)
    decoder = ExpertDecoder(a.decode_tokens, router, W1, W2, a.k)
    x, y = X[:a.decode_tokens], Y[:a.decode_tokens].clone()
    few.forward(x, y)
    error = (decoder.step(x).float() - y.float()).norm() / y.float().norm()
    decoder.check()
    print(f"serving step, {a.decode_tokens} tokens: 4-bit weights "
          f"{_milliseconds(lambda: decoder.step(x), 50) * 1e3:.1f} us, 16-bit weights "
          f"{_milliseconds(lambda: few.forward(x, y), 50) * 1e3:.1f} us, "
          f"4-bit output off by {error:.3f}")


if __name__ == "__main__":
    main()
