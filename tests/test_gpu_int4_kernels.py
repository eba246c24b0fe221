"""The 4-bit expert kernels that a launch rule picks only at other sizes than
those of test_gpu_int4: each tile shape with reductions long enough that every
wavefront's loop runs round, and the 64-row kernel past the reuse of its LDS ring
(a slot takes new rows from the fifth slab of 128 on).  Against the reference and
with the tolerances of test_gpu_int4.

rows = T K; rows / (N + Z) on average an expert: to 13 16-row tiles, to 20
32-row tiles, else 64-row tiles.  For 16 rows, with tiles = rows / 16 + min(rows,
N), gate/up takes 16 columns of h where tiles * I / 32 < 1024, else 64 with more
than 8 rows an FFN expert and 32 with fewer; down takes 128 columns of y from
tiles * d / 128 = 4096 on, else 64.
"""
import pytest
import torch

from moe_layer_zero_amd import zcmoe
from tests import test_gpu_int4 as X

pytestmark = pytest.mark.gpu


def shape_of(T, d, N, Z, I, K):
    """(row tile, columns of h, columns of y) of a call."""
    rows = T * K
    avg = rows // (N + Z)
    if avg > 20:
        return 64, 128, 256
    if avg > 13:
        return 32, 32, 64
    tiles = rows // 16 + min(rows, N)
    gate_up = 16 if tiles * (I // 32) < 1024 else 64 if rows > 8 * N else 32
    return 16, gate_up, 64 if tiles * (d // 128) < 4096 else 128


def run(case, G, want, skew=None):
    print(f"[int4 kernels] {case} G={G} {want}", flush=True)
    assert shape_of(*case) == want
    X.check(*X.make(*case, G, seed=200 + case[0], skew=skew), G)


CASES = [
    # T, d, N, Z, I, K
    ((67, 640, 64, 3, 512, 2), (16, 32, 64)),     # few rows an expert; 5 and 4 slabs
    ((3, 1152, 64, 0, 1024, 16), (16, 32, 64)),   # 9 and 8 slabs, experts with one row
    ((97, 640, 32, 4, 640, 4), (16, 64, 64)),     # more than 8 rows an FFN expert, 5 slabs
    ((79, 1280, 8, 2, 1152, 2), (32, 32, 64)),    # 32-row tiles; 10 and 9 slabs
    ((81, 1408, 7, 1, 1024, 2), (32, 32, 64)),    # 11 and 8 slabs, ragged counts
    ((307, 640, 4, 1, 896, 2), (64, 128, 256)),   # 64-row tiles: 5 and 7 slabs, half a last tile of y
    ((503, 1152, 4, 1, 1024, 2), (64, 128, 256)), # 9 and 8 slabs, four row tiles an expert
    ((260, 1280, 3, 0, 640, 1), (64, 128, 256)),  # 10 and 5 slabs
    ((130, 768, 2, 1, 1536, 1), (64, 128, 256)),  # 6 and 12 slabs
]


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("case,want", CASES, ids=["x".join(map(str, c[0])) for c in CASES])
def test_parity(case, want, G):
    run(case, G, want)


# 128 columns of y a workgroup: wide rows and many experts
@pytest.mark.parametrize("case,want,G", [
    ((104, 4608, 64, 0, 128, 8), (16, 16, 128), 64),
    ((128, 1664, 256, 0, 128, 8), (16, 32, 128), 128),
    ((103, 4736, 60, 4, 384, 8), (16, 64, 128), 32),
])
def test_parity_of_wide_layers(case, want, G):
    run(case, G, want)


@pytest.mark.parametrize("G", [32, 128])
@pytest.mark.parametrize("case,want", [
    ((150, 640, 40, 8, 640, 4), (16, 64, 64)),
    ((90, 1152, 10, 0, 640, 2), (32, 32, 64)),
    ((400, 640, 8, 2, 896, 2), (64, 128, 256)),
])
def test_one_expert_takes_every_token(case, want, G):
    run(case, G, want, skew=1)


@pytest.mark.parametrize("G", [32, 64, 128])
def test_groups_of_rows_do_not_meet(G):
    """The 64-row kernel on a long reduction: a token's row does not depend on the
    others' values (ring slots, sums left in LDS and rows past the tile)."""
    case = (311, 1152, 4, 1, 1024, 2)
    desc, x, w, route, packed = X.make(*case, G, seed=77)
    a, b = torch.empty((311, 1152), dtype=X.BF, device="cuda"), torch.empty((311, 1152), dtype=X.BF, device="cuda")
    zcmoe.zc_moe_experts(desc, x.cuda(), route, *packed, a)
    y = x.clone()
    y[::2] = 100.0 * torch.randn(y[::2].shape, generator=X.gen(5)).to(X.BF)
    zcmoe.zc_moe_experts(desc, y.cuda(), route, *packed, b)
    assert torch.equal(a[1::2], b[1::2]) and not torch.equal(a[::2], b[::2])
