"""What the Python classes of the expert and 4-bit-weight operators refuse
before anything is planned or launched, and what they accept: on the CPU, where
the next error of an accepted call is the missing CUDA device."""
from __future__ import annotations

import pytest
import torch

import dense_tiled_gemm_02_gb300 as pkg

BF16 = torch.bfloat16


def grouped_operands(E=2, R=4, K=8, N=16, with_c=False):
    return dict(A=torch.zeros(R, K, dtype=BF16), B=torch.zeros(E, K, N, dtype=BF16),
                offsets=torch.zeros(E + 1, dtype=torch.int32),
                C=torch.zeros(R, N, dtype=BF16) if with_c else None,
                D=torch.zeros(R, N, dtype=BF16))


def w4_operands(E=2, R=4, K=64, N=16, group=32):
    G = -(-K // group)
    return dict(X=torch.zeros(R, K, dtype=BF16), W=torch.zeros(E, N, K // 2, dtype=torch.uint8),
                scales=torch.zeros(E, N, G, dtype=BF16),
                zeros=torch.zeros(E, N, G, dtype=torch.uint8),
                offsets=torch.zeros(E + 1, dtype=torch.int32), D=torch.zeros(R, N, dtype=BF16),
                group=group)


@pytest.mark.parametrize("name", ["B", "offsets", "C", "D"])
def test_grouped_operands_are_on_one_device(name):
    t = grouped_operands(with_c=True)
    t[name] = t[name].to("meta")
    with pytest.raises(ValueError, match=f"{name} is on meta, not on cpu"):
        pkg.GroupedGemm.like(**t)


@pytest.mark.parametrize("name", ["W", "scales", "zeros", "offsets", "D"])
def test_w4_operands_are_on_one_device(name):
    t = w4_operands()
    t[name] = t[name].to("meta")
    with pytest.raises(ValueError, match=f"{name} is on meta, not on cpu"):
        pkg.W4Gemm.like(**t)


def test_operands_on_the_host_need_a_device():
    with pytest.raises(ValueError, match="CUDA"):
        pkg.GroupedGemm.like(**grouped_operands(with_c=True))
    with pytest.raises(ValueError, match="CUDA"):
        pkg.W4Gemm.like(**w4_operands())


@pytest.mark.gpu
def test_operands_on_the_host_are_refused_beside_others_on_the_gpu():
    t = grouped_operands()
    t.update(A=t["A"].cuda(), D=t["D"].cuda(), offsets=t["offsets"].cuda())
    with pytest.raises(ValueError, match="B is on cpu, not on cuda:0"):
        pkg.GroupedGemm.like(**t)
    t = w4_operands()
    t.update(X=t["X"].cuda(), W=t["W"].cuda(), D=t["D"].cuda(), offsets=t["offsets"].cuda())
    with pytest.raises(ValueError, match="scales is on cpu, not on cuda:0"):
        pkg.W4Gemm.like(**t)


@pytest.mark.parametrize("dtype", [torch.uint8, torch.int8, torch.int32, torch.int64,
                                   torch.float32, torch.bfloat16])
def test_pack_w4_takes_four_bits(dtype):
    q = torch.arange(16).reshape(2, 8).to(dtype)
    assert pkg.pack_w4(q).tolist() == [[0x10, 0x32, 0x54, 0x76], [0x98, 0xBA, 0xDC, 0xFE]]
    assert pkg.pack_w4(torch.zeros(3, 0, 4, dtype=dtype)).shape == (3, 0, 2)


@pytest.mark.parametrize("q,match", [
    (torch.tensor([[1, 16]]), "0..15, not 1..16"),       # would spill into its neighbour
    (torch.tensor([[-1, 3]]), "0..15, not -1..3"),
    (torch.tensor([[16.0, 3.0]]), "0..15"),
    (torch.tensor([[float("nan"), 3.0]]), "0..15"),
    (torch.tensor([[1, 2, 3]]), "K = 3 is odd"),         # would pair 1 and 3 with the one 2
    (torch.tensor([[1]]), "K = 1 is odd"),
])
def test_pack_w4_refuses_other_values(q, match):
    with pytest.raises(ValueError, match=match):
        pkg.pack_w4(q)


@pytest.mark.parametrize("E,K,ld", [(3, 24, 32), (3, 24, 24), (1, 24, 32), (3, 1, 8), (1, 1, 1)])
def test_grouped_takes_a_single_column_with_padding(E, K, ld):
    """B of one column, stored along K with a gap after each expert's."""
    t = grouped_operands(E=E, K=K, N=1)
    t["B"] = torch.zeros(E, 1, ld, dtype=BF16)[:, :, :K].transpose(1, 2)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.GroupedGemm.like(**t)
    t["B"] = torch.zeros(E, K, ld, dtype=BF16)[:, :, :1]  # or across it
    with pytest.raises(ValueError, match="CUDA"):
        pkg.GroupedGemm.like(**t)


@pytest.mark.parametrize("group", [0, -32])
def test_w4_group_is_positive(group):
    t = w4_operands()
    t["group"] = group
    with pytest.raises(ValueError, match="group"):
        pkg.W4Gemm.like(**t)
