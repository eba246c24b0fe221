"""The forward's workspace on MXFP4 weights holds its pieces side by side: routing, h
as codes and scales, y, x as codes and scales, the list of row tiles, each at a
multiple of 256 bytes.  Checked through the sizes that the library gives out."""
import pytest
import torch

from moe_layer_zero_amd import zcmoe

BF = torch.bfloat16


def a256(n):
    return -(-n // 256) * 256


def size(op=zcmoe.ZC_OP_EXPERTS, **kw):
    n = zcmoe.zc_moe_workspace_size(zcmoe.LayerDesc(dtype=BF, **kw), op)
    assert n > 0
    return n


def check(T, K, N, Z, d, I, a):
    sizes = dict(T=T, K=K, N=N, Z=Z, d=d, I=I)
    rows = T * K
    # the layer on 4-bit integer weights: routing, h in bf16, y in fp32, the same list
    route = size(zcmoe.ZC_OP_ROUTE, **sizes)
    tiles = size(weight_layout=zcmoe.int4_layout(32), **sizes) - route - a256(2 * rows * I) - a256(4 * rows * d)
    codes = lambda n: a256(n if a == 8 else n // 2) + a256(n // 32)  # noqa: E731
    y = a256((2 if many(T, K, N, Z, d, I) else 4) * rows * d)
    need = route + codes(rows * I) + y + codes(T * d) + tiles
    assert size(weight_layout=zcmoe.mxfp4_layout(a), **sizes) >= need, sizes


def many(T, K, N, Z, d, I):
    return T * K // (N + Z) > 10 and d % 512 == 0 and I % 512 == 0


@pytest.mark.parametrize("a", [8, 4])
def test_pieces_of_small_layers(a):
    for I in (128, 256, 384, 512, 640):
        for T, K in ((1, 1), (1, 2), (1, 3), (2, 1), (3, 1), (5, 2), (40, 1)):
            for d in (128, 512, 4096):
                check(T, K, 3, 1, d, I, a)


@pytest.mark.parametrize("a", [8, 4])
def test_pieces_of_one_row(a):
    # 128 values of h: their codes and their scales take 256 bytes each
    check(1, 1, 1, 0, 128, 128, a)
