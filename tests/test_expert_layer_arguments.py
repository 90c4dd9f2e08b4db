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
