"""Refusals of the latent attention that need no GPU."""
import ctypes

import pytest

from long_context_sparse_indexer_b200 import lsa


@pytest.mark.parametrize("dtype", [lsa.BF16, lsa.FP8_E4M3])
def test_softmax_scales_beyond_the_fp8_range(dtype):
    """An FP8 cache's weights carry 2^60 sm_scale and its results 2^60 / (sm_scale log2 e), which are finite in 32 bits
    from 2^-68 to 2^67 only, and exact enough well inside.  Calls of no token: nothing is launched."""
    lib = lsa.library()
    b = lsa.CBatch(2, 0, 1, 100, 16, 16, 16)
    c = lsa.CCache(4096, 16 if dtype == lsa.FP8_E4M3 else None, dtype, 576, 57600, 576, 100)
    for sm, ok in ((2.0 ** -30, True), (1 / 24, True), (2.0 ** 30, True), (2.0 ** -31, False), (2.0 ** -70, False),
                   (2.0 ** 31, False), (2.0 ** 70, False)):
        got = lib.lsa_latent_attn(ctypes.byref(b), 4096, 128, ctypes.byref(c), None, sm, 8192, lsa.BF16, None, 1 << 20, 0,
                                  None, None)
        assert got == (lsa.OK if ok or dtype == lsa.BF16 else lsa.ERR_UNSUPPORTED), sm
