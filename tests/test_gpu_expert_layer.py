"""The expert layer made of the operators, against 64-bit autograd on the CPU.

Bounds.  The kernels sum 16-bit products in 32 bits and round each stored
matrix once to 16 bits (u = 2^-9 for bf16, relative).  Forward, the roundings
of Xs (none), hid, Ys and Y follow each other, and backward those of dYs, dhid,
dXs and of the gradient itself, over hid and Ys that carry their own: at most
eight roundings on a path.  Errors of rounding are independent of one another,
so the norm of the whole error stays well below 8 u of the norm of the
result; a cancellation in a gradient can double it: 16 u = 2^-5.  relu's
kink: a hidden value whose sign the rounding turns is smaller than u, and so
is what it adds.

The residual stream's norm adds the roundings of h and of its rows, within the
same bound.  Rows in 8 bits: the largest of n <= 1024 normal values is below 4.2
of their standard deviations, a step of it at most 1 / 63.5 (block rows) or 1 /
127 (scaled rows), and the error, spread evenly over a step, 1 / sqrt(12) of
one: at most 2^-6 of the norm for block rows (32 values, below 2.7 deviations on
average), 2^-6 for scaled rows, for each such rounding on a path.
"""
import pytest
import torch

from dense_tiled_gemm_02_gb300 import expert_layer as el


def dense_layer(X, router, W1, W2, experts, k):
    """The formula in the arguments' precision, for the given choices."""
    logits = X @ router.T
    gates = logits.gather(1, experts.clamp(min=0)).softmax(1)
    Y = torch.zeros_like(X)
    for t in range(X.shape[0]):
        for j in range(k):
            e = int(experts[t, j])
            Y[t] = Y[t] + gates[t, j] * (W2[e] @ (W1[e] @ X[t]).relu())
    return Y


def far(got, want):
    return float((got.double().cpu() - want).norm() / want.norm())


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("K", [32, 96, 256])
def test_quantize_w4_rounds_to_the_nearest_step(group, K):
    g = torch.Generator().manual_seed(K + group)
    w = torch.randn(3, 5, K, generator=g)
    packed, scales, zeros = el.quantize_w4(w, group)
    G = -(-K // group)
    assert packed.shape == (3, 5, K // 2) and scales.shape == zeros.shape == (3, 5, G)
    q = torch.stack((packed & 15, packed >> 4), -1).flatten(-2).float()
    per_k = torch.arange(K) // group
    back = (q - zeros.float()[..., per_k]) * scales[..., per_k]
    # a value lies in the range, off by half a step, and the rounded zero point
    # moves the range's ends by up to half a step more
    assert ((back - w).abs() <= 1.001 * scales[..., per_k]).all()


def test_quantize_w4_keeps_zeros():
    packed, scales, zeros = el.quantize_w4(torch.zeros(1, 2, 64), 32)
    assert (scales == 0).all() and (packed == 0).all() and (zeros == 0).all()


def test_arguments_have_a_default_for_everything():
    a = el.arguments([])
    assert a.tokens > a.decode_tokens > 0 and a.k <= a.experts


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,H,F", [(1, 4, 2, 64, 32), (37, 8, 2, 128, 96), (200, 16, 4, 64, 64)])
def test_layer_and_gradients(T, E, k, H, F):
    router, W1, W2 = el.random_weights(E, H, F, seed=T)
    g = torch.Generator(device="cuda").manual_seed(T + 1)
    X = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    dY = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    layer = el.ExpertLayer(T, router, W1, W2, k)
    Y, dX = torch.empty_like(X), torch.empty_like(X)
    layer.forward(X, Y)
    layer.backward(X, dY, dX)
    layer.check()
    leaves = [t.detach().double().cpu().requires_grad_() for t in (X, router, W1, W2)]
    want = dense_layer(*leaves, layer.experts.cpu().long(), k)
    want.backward(dY.double().cpu())
    bound = 2.0 ** -5
    assert far(Y, want.detach()) < bound
    for got, leaf in zip((dX, *(layer.grads[n] for n in ("router", "W1", "W2"))), leaves):
        assert far(got, leaf.grad) < bound


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,H,F,group", [(1, 8, 2, 256, 128, 128), (5, 4, 4, 128, 96, 32)])
def test_decoder(T, E, k, H, F, group):
    router, W1, W2 = el.random_weights(E, H, F, seed=T)
    decoder = el.ExpertDecoder(T, router, W1, W2, k, group)

    def widened(w4, K):
        packed, scales, zeros = (t.cpu() for t in w4)
        q = torch.stack((packed & 15, packed >> 4), -1).flatten(-2).double()
        per_k = torch.arange(K) // group
        return (q - zeros.double()[..., per_k]) * scales.double()[..., per_k]

    w1, w2 = widened(decoder.w1, H), widened(decoder.w2, F)
    for step in range(3):  # recorded, then replayed with other tokens
        g = torch.Generator(device="cuda").manual_seed(step)
        X = torch.randn(T, H, generator=g, device="cuda").bfloat16()
        got = decoder.step(X).clone()
        decoder.check()
        want = dense_layer(X.double().cpu(), router.double().cpu(), w1, w2,
                           decoder.experts.cpu().long(), k)
        assert far(got, want) < 2.0 ** -5


def signed_layer(X, router, W1, W2, experts, k, positive):
    """dense_layer with relu's side given, too: (T, k, F) truth values.  The norm's
    rounding of a row turns the sign of one in some thousand hidden values near
    zero, and the gradient of such a value comes or goes as a whole."""
    gates = (X @ router.T).gather(1, experts.clamp(min=0)).softmax(1)
    Y = torch.zeros_like(X)
    for t in range(X.shape[0]):
        for j in range(k):
            e = int(experts[t, j])
            Y[t] = Y[t] + gates[t, j] * (W2[e] @ (W1[e] @ X[t] * positive[t, j]))
    return Y


def normed(X, residual, w, eps=1e-6):
    h = X + residual
    return h, h / (h.square().mean(1, keepdim=True) + eps).sqrt() * w


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,H,F", [(1, 4, 2, 64, 32), (37, 8, 2, 128, 96), (200, 16, 4, 64, 64)])
@pytest.mark.parametrize("keep8", [False, True])
@pytest.mark.parametrize("with_norm", [False, True])
def test_layer_of_a_stream_and_rows_kept_in_8_bits(T, E, k, H, F, keep8, with_norm):
    router, W1, W2 = el.random_weights(E, H, F, seed=T)
    g = torch.Generator(device="cuda").manual_seed(T + 1)

    def rows():
        return torch.randn(T, H, generator=g, device="cuda").bfloat16()

    X, dY = rows(), rows()
    norm = 1 + 0.1 * torch.randn(H, generator=g, device="cuda") if with_norm else None
    layer = el.ExpertLayer(T, router, W1, W2, k, norm, keep8=keep8)
    Y, dX = torch.empty_like(X), torch.empty_like(X)
    leaves = [t.detach().double().cpu().requires_grad_() for t in (X, router, W1, W2)]
    names = ["router", "W1", "W2"]
    if with_norm:
        residual, dh, h = rows(), rows(), torch.empty_like(X)
        layer.forward(X, Y, residual=residual, h=h)
        layer.backward(X, dY, dX, h=None if keep8 else h, dh=dh)
        leaves.append(norm.double().cpu().requires_grad_())
        names.append("norm")
        stream, seen = normed(leaves[0], residual.double().cpu(), leaves[-1])
    else:
        layer.forward(X, Y)
        layer.backward(X, dY, dX)
        stream, seen = None, leaves[0]
    layer.check()
    positive = (layer.hid > 0)[layer.slot_row.long()].cpu()
    want = signed_layer(seen, *leaves[1:4], layer.experts.cpu().long(), k, positive)
    loss = (want * dY.double().cpu()).sum()
    if with_norm:
        loss = loss + (stream * dh.double().cpu()).sum()
        assert far(h, stream.detach()) < 2.0 ** -8
    loss.backward()
    assert far(Y, want.detach()) < 2.0 ** -5
    bound = 2.0 ** -5 + (2.0 ** -6 if keep8 else 0)
    assert far(dX, leaves[0].grad) < bound
    for name, leaf in zip(names, leaves[1:]):
        assert far(layer.grads[name], leaf.grad) < bound, name


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,H,F", [(1, 8, 2, 256, 128), (5, 4, 4, 128, 96), (64, 4, 2, 64, 80)])
@pytest.mark.parametrize("with_norm", [False, True])
def test_decoder_of_8_bits(T, E, k, H, F, with_norm):
    router, W1, W2 = el.random_weights(E, H, F, seed=T)
    norm = torch.rand(H, device="cuda") + 0.5 if with_norm else None
    decoder = el.ExpertDecoder(T, router, W1, W2, k, bits=8, norm=norm)
    w1, w2 = (q.double().cpu() * s.double().cpu()[..., None] for q, s in (decoder.w1, decoder.w2))
    for w, W in ((w1, W1), (w2, W2)):
        assert far(W, w) < 2.0 ** -6
    for step in range(3):  # recorded, then replayed with other tokens
        g = torch.Generator(device="cuda").manual_seed(step)
        X = torch.randn(T, H, generator=g, device="cuda").bfloat16()
        residual = torch.randn(T, H, generator=g, device="cuda").bfloat16() if with_norm else None
        got = decoder.step(X, *([residual] if with_norm else [])).clone()
        decoder.check()
        seen = X.double().cpu()
        if with_norm:
            h, seen = normed(seen, residual.double().cpu(), norm.double().cpu())
            assert far(decoder.h, h) < 2.0 ** -8
        want = dense_layer(seen, router.double().cpu(), w1, w2, decoder.experts.cpu().long(), k)
        assert far(got, want) < 2.0 ** -5 + 2 * 2.0 ** -6


@pytest.mark.gpu
def test_command_runs_with_every_option(capsys):
    el.main(["--tokens", "256", "--hidden", "128", "--inner", "64", "--experts", "8", "-k", "2",
             "--steps", "2", "--norm", "--keep8", "--bits", "8"])
    out = capsys.readouterr().out
    assert "8-bit weights" in out and "training step" in out


@pytest.mark.gpu
def test_command_learns(capsys):
    el.main(["--tokens", "256", "--hidden", "128", "--inner", "64", "--experts", "8", "-k", "2",
             "--steps", "4", "--rate", "0.1"])
    losses = [float(line.split()[-1]) for line in capsys.readouterr().out.splitlines()
              if line.startswith("step")]
    assert len(losses) == 4 and losses[-1] < losses[0]
