"""What a training layer holds of its rows, with and without keeping them in 8 bits."""
import pytest
import torch

from dense_tiled_gemm_02_gb300 import expert_layer as el


def held_bytes(layer, names):
    """Of the named tensors (or pairs of them), each storage once."""
    sizes = {}
    for name in names:
        value = getattr(layer, name, ())
        for t in value if isinstance(value, tuple) else (value,):
            sizes[t.untyped_storage().data_ptr()] = t.untyped_storage().nbytes()
    return sum(sizes.values())


@pytest.mark.gpu
@pytest.mark.parametrize("with_norm", [False, True])
def test_rows_in_8_bits_take_the_place_of_buffers(with_norm):
    T, E, k, H, F = 64, 8, 2, 256, 96
    router, W1, W2 = el.random_weights(E, H, F)
    norm = torch.ones(H, device="cuda") if with_norm else None
    plain = el.ExpertLayer(T, router, W1, W2, k, norm)
    kept = el.ExpertLayer(T, router, W1, W2, k, norm, keep8=True)
    sorted_rows, tokens = ("Xs", "dXs", "Xs8"), ("Xn", "dXn", "Xn8", "h8")
    assert held_bytes(plain, sorted_rows) == T * k * H * 4
    assert held_bytes(kept, sorted_rows) == T * k * (H * 2 + H + H // 32)
    if with_norm:
        assert held_bytes(plain, tokens) == T * H * 4
        assert held_bytes(kept, tokens) == T * (H * 2 + 2 * (H + H // 32))


@pytest.mark.gpu
@pytest.mark.parametrize("with_norm", [False, True])
def test_a_second_backward_pass_gives_the_same_bits(with_norm):
    """The buffers that it shares hold nothing that the next one reads."""
    T, E, k, H, F = 40, 8, 2, 128, 96
    router, W1, W2 = el.random_weights(E, H, F)
    norm = torch.rand(H, device="cuda") + 0.5 if with_norm else None
    layer = el.ExpertLayer(T, router, W1, W2, k, norm, keep8=True)
    X, dY, residual, dh = (torch.randn(T, H, device="cuda").bfloat16() for _ in range(4))
    Y, h = torch.empty_like(X), torch.empty_like(X)
    forward = dict(residual=residual, h=h) if with_norm else {}
    backward = dict(dh=dh) if with_norm else {}
    layer.forward(X, Y, **forward)
    seen = []
    for _ in range(2):
        dX = torch.empty_like(X)
        layer.backward(X, dY, dX, **backward)
        seen.append([dX] + [g.clone() for g in layer.grads.values()])
    layer.check()
    assert all(torch.equal(a, b) for a, b in zip(*seen))
