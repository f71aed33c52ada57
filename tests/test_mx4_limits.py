"""Sizes that lmoe_mx4_gemm's 32-bit indices do not reach are refused before anything is launched.  No GPU."""
import pytest

import latent_space_routed_b200 as lm
from test_mx4_abi import A, UNS, _gemm

TOP = 2 ** 31 - 1


@pytest.mark.parametrize("kw", [
    dict(N=TOP, ldo=TOP), dict(N=TOP - 190, ldo=TOP), dict(N=TOP - 255, ldo=TOP),
    dict(off=A, E=1, N=TOP - 255, ldo=TOP), dict(off=A, E=1023, N=2099202, ldo=TOP),         # E N = TOP - 1
    dict(off=A, E=3, N=(TOP - 100) // 3, ldo=TOP)])
def test_row_indices_past_the_last_tile_fit(kw):
    """The last tile's 192 rows of W are indexed in 32 bits: E N and N stop 256 short of 2^31."""
    assert _gemm(**kw) == UNS
    assert "2^31" in lm.lmoe_last_error()


@pytest.mark.parametrize("K", [2 ** 31 - 64, 2 ** 31 - 128, 2 ** 31 - 256])
def test_columns_past_the_last_stage_fit(K):
    """K is taken in stages of 256 values, counted in 32 bits."""
    assert _gemm(K=K, M=1, N=1, ldo=1) == UNS
    assert "2^31" in lm.lmoe_last_error()


@pytest.mark.parametrize("at", [1, 2, 3])
def test_offsets_are_words(at):
    assert _gemm(off=A + at, E=2) == UNS
    assert "offsets" in lm.lmoe_last_error()
