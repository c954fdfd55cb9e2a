"""GPU parity of the layer operators where their dispatch and their arithmetic
change: few CTAs a slab, fast decays, saturated gates, scales at the ends of
fp32.  Bounds as in tests/layer_cases.py, or derived beside the test."""
import numpy as np
import pytest
import torch

from oracle import layer_ops as O
from tests import layer_cases as C
from tests.test_gpu_layer_ops import BF16, E4M3, F32, P, check_adjoint, check_scan, near

pytestmark = pytest.mark.gpu

# rows of a tile (scan, adjoint)
TILE = {BF16: (120, 40), F32: (60, 30)}


def ends(T, packed):
    return [1, T // 3, T // 3, T // 3 + 1, T - 3] if packed else [0, T]


# CTAs a slab on 148 SMs: 1, 2, 3, 4
@pytest.mark.parametrize("D,ctas", [(4800, 1), (4096, 2), (3000, 3), (2048, 4)])
@pytest.mark.parametrize("tiles", [1, 2, 3, 4, 5, 6])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_recurrence_few_ctas_a_slab(cuda, D, ctas, tiles, dtype):
    """`tiles` tiles a CTA, the last one short; one sequence or several."""
    packed = tiles % 2 == 0
    for k, check in enumerate((check_scan, check_adjoint)):
        T = TILE[dtype][k] * ctas * tiles - 7
        starts = ends(T, packed)
        u, rate, h0, _ = C.glr_inputs(T, len(starts) - 1, D, dtype, seed=D + tiles, starts=starts, fast=tiles < 4)
        if k == 0:
            check_scan(cuda, u, rate, h0, starts, True)
        else:
            check_adjoint(cuda, u, rate, h0, starts, u.to(cuda), torch.tensor(starts, dtype=torch.int32, device=cuda), D)


@pytest.mark.parametrize("D,T", [(4800, 233), (4800, 1201), (2048, 957), (64, 9000)])
def test_adjoint_repeats_bit_for_bit(cuda, D, T):
    u, rate, h0, _ = C.glr_inputs(T, 1, D, BF16, 1)
    ud, rd, hd = u[None].to(cuda), rate.to(cuda), h0.to(cuda)
    h, dh = torch.randn(1, T, D, device=cuda), torch.randn(1, T, D, device=cuda)
    first = P().pararnn_glr_adjoint(ud, rd, hd, h, dh)
    for _ in range(30):
        assert all(torch.equal(x, y) for x, y in zip(first, P().pararnn_glr_adjoint(ud, rd, hd, h, dh)))
