"""GPU tests of ``paged_sparse_decode_fp8`` on rows of far apart magnitudes, against 64 bits.

A key is k' 2^a and a value v' 2^b with e4m3 numbers k', v'; a and b may be any exponents the cache holds,
-127 to 119 (and higher from other writers), and q any bf16 number.
"""
import numpy as np
import pytest
import torch

import block_sparse_attention_msa_gb300 as msa
import test_gpu_fp8_cache as base
from test_gpu_fp8_cache import D, DEV, F8, PAGE, check, i32, reference, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_sparse_attention_msa_gb300 import build
    build.build()
    msa.load()
    assert msa.device_error() == 0


@pytest.fixture(autouse=True)
def no_error_left():
    yield
    assert msa.device_error() == 0


# A power of the keys and one of the queries that cancels it; where the queries' reach ends (bf16's subnormals
# below 2^-126, its largest number 2^127 or so) the scores are small or large, but finite and told apart.
@pytest.mark.parametrize("R,Hq", [(1, 8), (40, 8), (1, 32), (40, 32)])
@pytest.mark.parametrize("a,c", [(119, -119), (110, -112), (97, -97), (80, -78), (-127, 120), (-120, 118), (-90, 90),
                                 (126, -126)])
def test_scores_of_large_keys_and_small_queries_and_the_reverse(R, Hq, a, c):
    Hkv = 2
    w = base.make(base._lens(R * Hkv, a & 7, 6, 200), 6, Hq, Hkv, seed=a & 31, spread=0.0)
    # the keys' powers, near -7, moved by a and the queries' by c
    w["ks"] = (w["ks"].int() + a).clamp(0, 253).to(torch.uint8)
    w["q"] = (w["q"].double() * 2.0 ** c).to(torch.bfloat16)
    ref = reference(w)
    assert torch.isfinite(ref[0]).all()
    check(run(w), ref)
