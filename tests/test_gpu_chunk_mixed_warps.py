"""GPU tests of ``chunk_attention`` where the rows of one warp take different ways: rows of padding beside live
ones, rows that see a later token's non-finite values, rows without a finite score beside rows whose scores lie
beyond 2^24. Tensor memory is accessed by whole warps, so each of these has to end before the next access."""
import pytest
import torch

import block_sparse_attention_msa_gb300 as msa
from test_gpu_chunk_attention import D, DEV, NAN, PAGE, check, make, reference, run

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


@pytest.mark.parametrize("Hq,Hkv,new", [(8, 8, 7), (8, 4, 3), (16, 2, 3), (16, 1, 2), (32, 2, 3), (4, 1, 13)])
@pytest.mark.parametrize("held", [0, 61, 900])
def test_rows_of_padding_beside_rows_that_see_a_later_nan(Hq, Hkv, new, held):
    # live rows end inside a warp; of these, the last token's alone sees its own values, of which every 16 channels
    # hold something that is not finite
    w = make([new, new], [held, 3], Hq, Hkv, seed=held + new)
    clean = reference(w)
    pos = held + new - 1
    for c in range(0, D, 16):
        w["vc"][w["table"][0, pos // PAGE], pos % PAGE, :, c + c // 16] = (NAN, float("inf"))[c // 16 & 1]
    o, lse = run(w)
    bad = o[new - 1].float().cpu()
    for c in range(0, D, 16):
        at = c + c // 16
        assert not torch.isfinite(bad[:, at]).any()
        o[new - 1, :, at] = clean[0][new - 1, :, at].to(torch.bfloat16).to(DEV)
    check((o, lse), clean)


@pytest.mark.parametrize("Hq,Hkv,held", [(8, 2, 40), (8, 1, 200), (32, 2, 64), (16, 16, 300)])
def test_rows_without_a_finite_score_beside_rows_of_far_scores(Hq, Hkv, held):
    """Keys hold -3e38 in channel 0: a query of 4 there has no finite score, one of 2^-80 scores near -2.5e14,
    beyond 2^24, with one key far above the others."""
    new = 5
    w = make([new], [held], Hq, Hkv, seed=held)
    n = held + new
    w["kc"] = torch.where(torch.isnan(w["kc"]), NAN, 0.0).to(torch.bfloat16)
    w["kc"][..., 0] = torch.where(torch.isnan(w["kc"][..., 0]), NAN, -3e38).to(torch.bfloat16)
    best = held // 2
    w["kc"][w["table"][0, best // PAGE], best % PAGE, :, 0] = -2.5e38
    w["q"][:] = 0
    w["q"][:, :, 0] = 2.0 ** -80
    w["q"][1::2, ::3, 0] = 4.0
    none = torch.zeros((new, Hq), dtype=torch.bool)
    none[1::2, ::3] = True
    o, lse = run(w)
    o, lse = o.cpu(), lse.cpu()
    assert (o[none] == 0).all() and torch.isneginf(lse[none]).all()
    v = w["vc"][w["table"][0, best // PAGE], best % PAGE].repeat_interleave(Hq // Hkv, 0)
    assert torch.equal(o[~none], v.expand(new, -1, -1)[~none])       # all weight on one key
    score = float(torch.tensor(-2.5e38).to(torch.bfloat16)) * 2.0 ** -80
    assert ((lse[~none].double() - score).abs() <= 2.0 ** -22 * abs(score)).all()
    assert n <= w["table"].shape[1] * PAGE


@pytest.mark.parametrize("Hq,Hkv,N", [(8, 8, 7), (8, 4, 3), (16, 1, 2), (32, 2, 3), (64, 8, 1)])
@pytest.mark.parametrize("held", [0, 900])
def test_the_same_rows_in_the_shared_prefix_decode(Hq, Hkv, N, held):
    w = make([N, N], [held, 3], Hq, Hkv, seed=held + N)
    clean = reference(w)
    pos = held + N - 1
    w["vc"][w["table"][0, pos // PAGE], pos % PAGE, :, 17] = NAN
    d = {k: x.to(DEV) for k, x in w.items()}
    o, lse = msa.shared_prefix_decode(d["q"], d["kc"], d["vc"], d["table"], d["seq"],
                                      torch.zeros(1, dtype=torch.int32, device=DEV), N=N)
    assert torch.isnan(o[N - 1, :, 17]).all()
    o[N - 1, :, 17] = clean[0][N - 1, :, 17].to(torch.bfloat16).to(DEV)
    check((o, lse), clean)
