"""What the expert layer refuses before anything is planned or enqueued."""
import pytest
import torch

from dense_tiled_gemm_02_gb300 import expert_layer as el

BF16 = torch.bfloat16


def weights(E=4, H=64, F=32):
    return dict(router=torch.zeros(E, H, dtype=BF16), W1=torch.zeros(E, F, H, dtype=BF16),
                W2=torch.zeros(E, H, F, dtype=BF16))


@pytest.mark.parametrize("cls", [el.ExpertLayer, el.ExpertDecoder])
@pytest.mark.parametrize("name,change,match", [
    ("router", lambda t: t.float(), "router is torch.float32"),     # would be read as 16 bits
    ("W2", lambda t: t.half(), "W2 is torch.float16"),
    ("W1", lambda t: t.float(), "one 16-bit type"),
    ("router", lambda t: t[:3], "do not go with W1"),
    ("W2", lambda t: t.transpose(1, 2).contiguous(), "do not go with W1"),
    ("W2", lambda t: t.to("meta"), "W2 is on meta"),
])
def test_weights_agree(cls, name, change, match):
    w = weights()
    w[name] = change(w[name])
    with pytest.raises(ValueError, match=match):
        cls(8, k=2, **w)


@pytest.mark.gpu
def test_tokens_of_another_shape_are_refused():
    w = {name: t.cuda() for name, t in weights().items()}
    layer = el.ExpertLayer(8, k=2, **w)
    X = torch.zeros(8, 64, dtype=BF16, device="cuda")
    others = (X[:7], X.float(), torch.zeros(8, 72, dtype=BF16, device="cuda")[:, :64],
              torch.zeros(8, 64, dtype=BF16))
    for bad in others:
        with pytest.raises(ValueError, match="X: planned"):
            layer.forward(bad, X)
        with pytest.raises(ValueError, match="Y: planned"):
            layer.forward(X, bad)
        with pytest.raises(ValueError, match="X: planned"):
            layer.backward(bad, X, X)
        with pytest.raises(ValueError, match="dX: planned"):
            layer.backward(X, X, bad)
    layer.check()
    decoder = el.ExpertDecoder(8, k=2, group=32, **w)
    with pytest.raises(ValueError, match="X: planned"):
        decoder.step(X[:1])  # copy_ would have repeated it


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["logit_gemm", "router_dx", "router_dw", "up", "down_dw"])
def test_check_reports_every_product(name):
    """A wait that runs out in any product of the layer reaches check()."""
    w = el.random_weights(16, 128, 64)
    layer = el.ExpertLayer(256, *w, 2)
    X = torch.randn(256, 128, device="cuda").bfloat16()
    Y, dX = torch.empty_like(X), torch.empty_like(X)
    op = getattr(layer, name)
    hook = op.debug_set if hasattr(op, "debug_set") else (
        lambda flags, ns: el.gemm.gemm_debug_set(op.handle, flags, ns))
    hook(el.gemm.GEMM_DEBUG_SKIP_FIRST_FILL, 20_000_000)
    layer.forward(X, Y)
    layer.backward(X, Y, dX)
    with pytest.raises(el.gemm.GemmError) as e:
        layer.check()
    assert e.value.code == el.gemm.GEMM_ERR_DEVICE_TIMEOUT
    hook(0, 0)
    layer.forward(X, Y)
    layer.backward(X, Y, dX)
    layer.check()


def norm_of(H=64, dtype=torch.float32, device="cpu"):
    return torch.ones(H, dtype=dtype, device=device)


@pytest.mark.parametrize("cls", [el.ExpertLayer, el.ExpertDecoder])
@pytest.mark.parametrize("norm,match", [
    (norm_of(63), "norm must be 64 weights"),
    (norm_of(dtype=torch.float16), "norm must be 64 weights"),   # neither the weights' nor fp32
    (norm_of(device="meta"), "norm is on meta"),
])
def test_norm_agrees_with_the_weights(cls, norm, match):
    with pytest.raises(ValueError, match=match):
        cls(8, k=2, norm=norm, **weights())


def test_decoder_bits():
    with pytest.raises(ValueError, match="4 or 8 bits, not 6"):
        el.ExpertDecoder(8, k=2, bits=6, **weights())


@pytest.mark.gpu
def test_the_stream_goes_with_a_norm():
    w = {name: t.cuda() for name, t in weights().items()}
    X = torch.zeros(8, 64, dtype=BF16, device="cuda")
    plain = el.ExpertLayer(8, k=2, **w)
    with pytest.raises(ValueError, match="go with a norm"):
        plain.forward(X, X, residual=X, h=X)
    with pytest.raises(ValueError, match="go with a norm"):
        plain.backward(X, X, X, dh=X)
    normed = el.ExpertLayer(8, k=2, norm=norm_of(device="cuda"), **w)
    for kw in ({}, {"residual": X}, {"h": X}):
        with pytest.raises(ValueError, match="go with a norm"):
            normed.forward(X, X, **kw)
    with pytest.raises(ValueError, match="residual: planned"):
        normed.forward(X, X, residual=X[:7], h=X)
    with pytest.raises(ValueError, match="h: planned"):
        normed.forward(X, X, residual=X, h=X.float())
    with pytest.raises(ValueError, match="go with a norm"):
        normed.backward(X, X, X, h=X)
    kept = el.ExpertLayer(8, k=2, norm=norm_of(device="cuda"), keep8=True, **w)
    with pytest.raises(ValueError, match="h is kept"):
        kept.backward(X, X, X, h=X, dh=X)
    decoder = el.ExpertDecoder(8, k=2, bits=8, norm=norm_of(device="cuda"), **w)
    with pytest.raises(ValueError, match="residual goes with a norm"):
        decoder.step(X)
    with pytest.raises(ValueError, match="residual: planned"):
        decoder.step(X, X[:1])
