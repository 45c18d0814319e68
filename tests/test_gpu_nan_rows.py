"""GPU tests: a row that sees a NaN gives NaN, in o and in lse, whatever form of a kernel takes it: one
cluster per row or partials with a merge, whole rows or halves of their keys. An lse of -inf says that a row
saw no key, and a later merge drops such a row."""
import numpy as np
import pytest
import torch

import block_sparse_attention_msa_gb300 as msa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
PAGE = 128
D = 128
NAN = float("nan")
F8 = torch.float8_e4m3fn


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


def i32(x):
    return torch.from_numpy(np.array(x, dtype=np.int32))


def sparse_rows(R, Hq, Hkv, n, topk, seed):
    """R rows of n visible tokens, every row on pages of its own."""
    g = torch.Generator().manual_seed(seed)
    m = (n + PAGE - 1) // PAGE
    pages = R * m
    fpt = torch.full((R * Hkv, topk), -1, dtype=torch.int64)
    for f in range(R * Hkv):
        fpt[f, :m] = (f // Hkv * m + torch.arange(m)) * PAGE * Hkv + f % Hkv
    return dict(q=(torch.randn((R, Hq, D), generator=g) * D ** -0.5).to(torch.bfloat16).to(DEV),
                k=torch.randn((pages, PAGE, Hkv, D), generator=g).to(torch.bfloat16).to(DEV),
                v=torch.randn((pages, PAGE, Hkv, D), generator=g).to(torch.bfloat16).to(DEV),
                fpt=fpt.to(torch.int32).to(DEV), lens=torch.full((R * Hkv,), n, dtype=torch.int32, device=DEV), m=m)


def decode_fp8(w):
    P, _, Hkv, _ = w["k"].shape
    c = [torch.zeros((P, Hkv, PAGE, D), dtype=torch.uint8, device=DEV).view(F8) for _ in range(2)]
    c += [torch.zeros((P, Hkv, PAGE), dtype=torch.uint8, device=DEV) for _ in range(2)]
    slots = torch.arange(P * PAGE, dtype=torch.int32, device=DEV)
    msa.append_kv_fp8(w["k"].view(-1, Hkv, D), w["v"].view(-1, Hkv, D), slots, *c)
    return msa.paged_sparse_decode_fp8(w["q"], *c, w["fpt"], w["lens"])


def decode_bf16(w):
    return msa.paged_sparse_decode(w["q"], w["k"], w["v"], w["fpt"], w["lens"])


DECODES = [pytest.param(decode_fp8, id="e4m3"), pytest.param(decode_bf16, id="bf16")]


# rows: one cluster each where there are few, else partials and a merge kernel
@pytest.mark.parametrize("decode", DECODES)
@pytest.mark.parametrize("R", [1, 40])
@pytest.mark.parametrize("n,topk", [(1, 2), (100, 4), (128, 4), (500, 4), (700, 40)])
@pytest.mark.parametrize("what", ["query", "key"])
def test_decode_rows_that_see_a_nan(decode, R, n, topk, what):
    Hq, Hkv = 16, 2
    w = sparse_rows(R, Hq, Hkv, n, topk, seed=n)
    clean = decode(w)
    r = R // 2
    if what == "query":
        w["q"][r, 9, 77] = NAN                      # one head of group 1
        heads = slice(9, 10)
    else:
        for page in range(w["m"]):                  # one visible key of every page of group 1
            w["k"][r * w["m"] + page, min(PAGE, n - page * PAGE) // 2, 1, 5] = NAN
        heads = slice(8, 16)
    o, lse = decode(w)
    assert torch.isnan(o[r, heads]).all() and torch.isnan(lse[r, heads]).all()
    o[r, heads], lse[r, heads] = clean[0][r, heads], clean[1][r, heads]
    assert torch.equal(o, clean[0]) and torch.equal(lse, clean[1])


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("S", [1, 3, 40])
def test_a_merge_of_parts_one_of_which_is_nan(bf16, S):
    g = torch.Generator().manual_seed(S)
    U, G = 5, 4
    parts = torch.randn((U, S, G, D), generator=g).to(torch.bfloat16 if bf16 else torch.float32).to(DEV)
    lse = torch.randn((U, S, G), generator=g).to(DEV)
    lse[1, 1:] = lse[3] = -float("inf")       # one part; none
    clean = msa.lse_merge(parts, lse)
    assert (clean[0][3] == 0).all() and torch.isneginf(clean[1][3]).all()
    lse[1, 0, 2] = lse[2, S // 2, 1] = NAN
    lse[4, :, 0] = -float("inf")
    lse[4, S - 1, 0] = NAN                    # beside empty parts
    o, z = msa.lse_merge(parts, lse)
    for u, e in ((1, 2), (2, 1), (4, 0)):
        assert torch.isnan(o[u, e]).all() and torch.isnan(z[u, e])
        o[u, e], z[u, e] = clean[0][u, e], clean[1][u, e]
    assert torch.equal(o, clean[0]) and torch.equal(z, clean[1])


@pytest.mark.parametrize("n,at", [(65, 64), (33, 32), (129, 128), (200, 64)])
@pytest.mark.parametrize("what", ["k", "v"])
def test_a_nan_in_the_later_half_of_a_single_group_s_keys(n, at, what):
    """One KV group: the keys of a tile are halved between two lanes. The NaN key is the only one that the row
    sees in the later half, or its values are NaN and its weight vanishes beside the earlier half's."""
    Hq = 8
    g = torch.Generator().manual_seed(n)
    bf = torch.bfloat16
    P = (n + PAGE - 1) // PAGE
    kc, vc = (torch.randn((P, PAGE, 1, D), generator=g).to(bf).to(DEV) for _ in range(2))
    q = torch.ones((1, Hq, D), dtype=bf, device=DEV)
    table = torch.arange(P, dtype=torch.int32, device=DEV)[None]
    call = lambda: msa.chunk_attention(q, kc, vc, table, i32([n]).to(DEV), i32([0, 1]).to(DEV))
    page, off = at // PAGE, at % PAGE
    if what == "k":
        kc[page, off] = NAN
        o, lse = call()
        assert torch.isnan(o).all() and torch.isnan(lse).all()
    else:
        vc[page, off] = NAN
        kc[page, off] = -200.0        # a score of -25600: no weight is left of it in fp32
        if n == 200:                  # every key of the later half
            kc.view(-1, 1, D)[at:n] = -200.0
        o, lse = call()
        assert torch.isnan(o).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("new,held,Hq,Hkv", [([40, 1], [700, 90], 32, 4), ([9, 2], [0, 400], 8, 1), ([1, 1, 1], [5, 64, 900], 8, 2)])
@pytest.mark.parametrize("junk", [NAN, float("inf")])
def test_queries_that_are_not_finite_beside_others_in_a_tile(new, held, Hq, Hkv, junk):
    from test_gpu_chunk_attention import make, reference, run, check
    w = make(new, held, Hq, Hkv, seed=Hq + len(new))
    clean = reference(w)
    T = sum(new)
    bad = torch.zeros((T, Hq), dtype=torch.bool)
    bad[::3, 1::4] = True
    w["q"][:T][bad] = junk              # infinity: scores of both signs, or infinity times 0
    o, lse = run(w)
    assert torch.isnan(o.cpu()[bad]).all() and torch.isnan(lse.cpu()[bad]).all()
    o[bad.to(DEV)], lse[bad.to(DEV)] = clean[0][bad].to(torch.bfloat16).to(DEV), clean[1][bad].float().to(DEV)
    check((o, lse), clean)
