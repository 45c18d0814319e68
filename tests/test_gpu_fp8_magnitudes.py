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


@pytest.mark.parametrize("R,Hq", [(1, 8), (24, 8), (1, 32), (24, 32)])
@pytest.mark.parametrize("power", [12, 18, 22, 25])
@pytest.mark.parametrize("n", [2, 3, 40, 700])
def test_values_beside_one_token_of_far_larger_values(R, Hq, power, n):
    """One token's values are 2^power larger, in channel 0 alone: the other channels' outputs are the other
    tokens', whose weights (with their values' powers of two) lie as far below the largest.

    Tolerance: each weight is rounded to fp16 at 2^-11 of its value or at 2^-32 of the row's largest, whichever
    is more; the rest as in the other decode tests."""
    Hkv, topk = 2, 6
    w = base.make([n] * (R * Hkv), topk, Hq, Hkv, seed=power + n, spread=0.0, pages=64)
    first = w["fpt"][:, 0].long()
    page, g = first // (PAGE * Hkv), first % (PAGE * Hkv)
    code, e = base.ref_quantise(np.concatenate([[2.0 ** power], np.zeros(D - 1)])[None])
    at = n // 2 if n < PAGE else 77
    w["vc"][page, g, at], w["vs"][page, g, at] = torch.from_numpy(code), torch.from_numpy(e)
    o, lse, to, tl = reference(w)
    fpt = w["fpt"].long()
    tight = torch.zeros_like(to)
    G = Hq // Hkv
    for f in range(R * Hkv):
        r, h = f // Hkv, slice(f % Hkv * G, (f % Hkv + 1) * G)
        vp = fpt[f, :(n + PAGE - 1) // PAGE]
        pg, gg = vp // (PAGE * Hkv), vp % (PAGE * Hkv)
        k, v = (torch.from_numpy(base.ref_values(w[x + "c"][pg, gg].numpy(), w[x + "s"][pg, gg].numpy())).flatten(0, 1)[:n]
                for x in "kv")
        b = torch.exp2(w["vs"][pg, gg].double().flatten()[:n] - 127)
        qi = w["q"][r, h].double()
        s = qi @ k.T
        p = torch.softmax(s, -1)
        big = (p * b).amax(-1, keepdim=True)
        step = torch.maximum(2.0 ** -11 * (1 + 2.0 ** -7) * p, 2.0 ** -32 * (1 + 2.0 ** -7) * big / b)   # of a weight
        ds = 2.0 ** -23 * 128 * (qi.abs() @ k.abs().T).amax(-1, keepdim=True) + 2.0 ** -21 * s.abs().amax(-1, keepdim=True) \
            + 2.0 ** -39 * qi.abs().amax(-1, keepdim=True) * k.abs().sum(-1).max()
        A = p @ v.abs()
        tight[r, h] = 2.0 ** -8 * (p @ v).abs() * (1 + 2.0 ** -7) + step @ v.abs() + (2 * ds + 2.0 ** -20 + n * 2.0 ** -24) * A
    check(run(w), (o, lse, tight, tl))
