"""Products with Q4_0 weights, held to the precision the kernel has: c - 8 and x are
multiplied exactly, a block's 32 products are summed in two steps of 2^-23 of their
magnitudes, and blocks in fp32: at most K / 512 + 24 roundings of 2^-24 in a chain
(a sixteenth of K's blocks a warp and the joins of 16 warps, with room for smaller
splits of K).  Errors of different blocks have no common sign: in the mean square
two truncations of 2^-23 and such a chain's share stay below 3e-7 of y."""
import numpy as np
import pytest
import torch

from oracle import llama as O
from q4_util import pack_weights
from test_gpu_q4 import dev, stream

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    import llama_decoder_forward_02_gb300 as L
    return L


@pytest.mark.parametrize("N,K,T,ws,xs,mean", [
    (4096, 4096, 1, 0.02, 1.0, 0.0), (2049, 4096, 8, 0.02, 1.0, 0.0), (1024, 14336, 8, 0.02, 1.0, 0.0),
    (4096, 14336, 1, 0.02, 1.0, 0.0), (700, 2816, 3, 30.0, 100.0, 0.0), (513, 1024, 5, 1e-4, 1e-2, 0.0),
    (2000, 4096, 2, 0.02, 1.0, 3.0),                                        # x with a large mean, which an offset summed apart magnifies
])
def test_precision(lib, N, K, T, ws, xs, mean):
    rng = np.random.default_rng(N + K + T)
    c, d = O.quantize_q4_0(rng.standard_normal((N, K)) * ws)
    d = d.astype(np.float16)
    x = ((rng.standard_normal((T, K)) + mean) * xs).astype(np.float16)
    W = O.dequantize_q4_0(c, d)
    ref = x.astype(np.float64) @ W.T
    mag = np.abs(x.astype(np.float64)) @ np.abs(W).T
    Wd, xd, y = dev(pack_weights(c, d)), dev(x), torch.zeros((T, N), device="cuda")
    assert lib.llm_op_gemv_q4_0(Wd.data_ptr(), xd.data_ptr(), y.data_ptr(), N, K, T, K, N, stream()) == 0
    off = np.abs(y.cpu().double().numpy() - ref)
    units = 16 if K >= 4096 else 1                                          # the launcher may give a short K fewer warps
    assert np.all(off <= mag * (2 * 2.0 ** -23 + (K / 32 / units + 24) * 2.0 ** -24)), (off / mag).max()
    if not mean:
        assert np.linalg.norm(off) <= 3e-7 * np.linalg.norm(ref), np.linalg.norm(off) / np.linalg.norm(ref)
