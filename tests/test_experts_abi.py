"""zc_moe_experts refuses an output or a workspace over its weights, whatever
their layout, before any work is queued."""
import ctypes as C

import pytest
import torch

from moe_layer_zero_amd import zcmoe

A = [(i + 1) << 40 for i in range(20)]  # distinct, aligned, never dereferenced
BF, F32 = torch.bfloat16, torch.float32
N, I, d = 8, 512, 1024

# layout, dtype, bytes of one weight set
SETS = [(zcmoe.ZC_WEIGHTS_ROWMAJOR, BF, N * I * d * 2), (zcmoe.ZC_WEIGHTS_ROWMAJOR, F32, N * I * d * 4),
        (zcmoe.ZC_WEIGHTS_PACKED, BF, N * I * d * 2), (zcmoe.ZC_WEIGHTS_MXFP8, BF, N * I * d * 33 // 32),
        (zcmoe.ZC_WEIGHTS_INT4_G32, BF, N * I * d // 2 + N * I * d // 32 * 2),
        (zcmoe.ZC_WEIGHTS_INT4_G128, BF, N * I * d // 2 + N * I * d // 128 * 2)]


def experts(desc, **over):
    a = dict(x=A[0], w_gate=A[1], w_up=A[2], w_down=A[3], out=A[4], ws=A[5])
    a.update(over)
    r = zcmoe.zc_route_buf(topk_idx=A[6], topk_gate=A[7], offsets=A[8], perm=A[9], inv=A[10])
    c = desc.c()
    return zcmoe.lib().zc_moe_experts(C.byref(c), a["x"], C.byref(r), a["w_gate"], a["w_up"], a["w_down"],
                                      None, None, a["out"], a["ws"], 1 << 30, None)


@pytest.mark.parametrize("layout,dtype,size", SETS)
@pytest.mark.parametrize("w", ["w_gate", "w_up", "w_down"])
def test_outputs_over_weights_are_refused(layout, dtype, size, w):
    desc = zcmoe.LayerDesc(16, d, N, 4, I, 2, dtype, weight_layout=layout)
    need = zcmoe.zc_moe_workspace_size(desc, zcmoe.ZC_OP_EXPERTS)
    es = 2 if dtype == BF else 4
    for name, own in (("out", 16 * d * es), ("ws", need)):
        # the set's first bytes under the output's last, and its last under the output's first
        for at in (A[12] + (own - 1) // 256 * 256, A[12] - (size - 1) // 256 * 256):
            assert experts(desc, **{name: A[12], w: at}) == zcmoe.ZC_ERR_INVALID, (name, at)
            assert f"{name} overlaps {w}" in zcmoe.lib().zc_last_error().decode()
