"""Rotary tables of pairs that hardly turn: their small sines by relative error."""
import numpy as np
import pytest
import torch

import tree_util as U

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("theta,n_rot,scaling,factor,orig", [
    (500000.0, 128, 0, 1.0, 0),
    (500000.0, 128, 1, 32.0, 0),
    (1e7, 64, 3, 32.0, 4096),
    (1e13, 128, 0, 1.0, 0),                       # the slowest pair takes 4e13 positions a turn
    (1e12, 64, 1, 1000.0, 0),
])
def test_sines_of_slow_pairs(theta, n_rot, scaling, factor, orig):
    import llama_decoder_forward_02_gb300 as L
    r = L.rope(theta, n_rot, scaling=scaling, factor=factor, n_ctx_orig=orig)
    f, m = U.frequencies(np.float32(theta).astype(np.float64), n_rot, scaling, factor, 1.0, 32.0, orig)
    seen = 0
    for pos0 in (1, 4000, 100000, 1 << 20):
        out = torch.empty((500, n_rot // 2, 2), device="cuda")
        assert L.llm_op_rope_table(r, pos0, 500, out.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
        pos = np.arange(pos0, pos0 + 500, dtype=np.float64)[:, None]
        slow = pos * f < 1e-3                     # one direction and the short series
        ref = np.sin(pos * f) * m
        got = out.cpu().double().numpy()[..., 1]
        # relative: the constant that takes turns to radians, its product, the series, the factor and the result, five
        # roundings of 2^-24; and the angle: a frequency to 2^-65 of a turn a position, what the series takes of it
        # to 2^-55 of a turn
        tol = 5 * 2.0 ** -24 * np.abs(ref) + m * 2 * np.pi * (pos * 2.0 ** -65 * (1 + 1e-9) + 2.0 ** -55)
        seen += slow.sum()
        assert np.all(np.abs(got - ref)[slow] <= tol[slow])
    assert seen
