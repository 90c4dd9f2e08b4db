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


@pytest.mark.gpu
def test_command_learns(capsys):
    el.main(["--tokens", "256", "--hidden", "128", "--inner", "64", "--experts", "8", "-k", "2",
             "--steps", "4", "--rate", "0.1"])
    losses = [float(line.split()[-1]) for line in capsys.readouterr().out.splitlines()
              if line.startswith("step")]
    assert len(losses) == 4 and losses[-1] < losses[0]
