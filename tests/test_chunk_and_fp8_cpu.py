"""Chunk attention and the quantised cache without a GPU: every refusal happens on the host, before any
device work, through the C ABI and through the Python binding."""
import ctypes
import math

import pytest
import torch

import block_sparse_attention_msa_gb300 as msa

at = ctypes.c_void_p
FAKE = at(0x1000)  # never dereferenced: every call below fails host validation
ARG, SHAPE, UNSUPPORTED, WORKSPACE = -1, -2, -3, -4


@pytest.fixture(scope="module")
def lib():
    from block_sparse_attention_msa_gb300 import build
    build.build()
    return msa.load()


def chunk(lib, **kw):
    a = dict(q=FAKE, qs=8192, k=FAKE, v=FAKE, table=FAKE, seq=FAKE, cu=FAKE, B=4, T=100, Hq=64, Hkv=8, D=128, mb=16,
             pages=64, o=FAKE, lse=None, ws=at(0x10000), nbytes=1 << 40)
    a.update(kw)
    return lib.msa_chunk_attention(*a.values(), None)


@pytest.mark.parametrize("change,code", [
    (dict(q=None), ARG), (dict(k=None), ARG), (dict(v=None), ARG), (dict(table=None), ARG), (dict(seq=None), ARG),
    (dict(cu=None), ARG), (dict(o=None), ARG), (dict(B=-1), ARG), (dict(T=-1), ARG), (dict(mb=0), ARG),
    (dict(pages=0), ARG), (dict(q=at(0x1008)), ARG), (dict(o=at(0x1002)), ARG), (dict(qs=8196), ARG),
    (dict(qs=8184), ARG), (dict(qs=-8192), ARG), (dict(qs=1 << 40), ARG),
    (dict(D=64), UNSUPPORTED), (dict(Hkv=3, Hq=24), UNSUPPORTED), (dict(Hq=60), UNSUPPORTED),
    (dict(Hq=256), UNSUPPORTED), (dict(Hq=0), UNSUPPORTED), (dict(Hkv=0), UNSUPPORTED),
    (dict(pages=1 << 24), UNSUPPORTED), (dict(pages=1 << 62), UNSUPPORTED), (dict(mb=1 << 24), UNSUPPORTED),
    (dict(B=16385), UNSUPPORTED), (dict(T=1 << 30), UNSUPPORTED), (dict(T=1 << 21, Hq=256, Hkv=16, qs=1 << 15), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(nbytes=1024), WORKSPACE), (dict(ws=at(0x10010)), WORKSPACE),
])
def test_chunk_refuses(lib, change, code):
    assert chunk(lib, **change) == code
    assert lib.msa_last_error()


def append(lib, **kw):
    a = dict(k=FAKE, ks=1024, v=FAKE, vs=1024, slots=FAKE, T=4, Hkv=8, D=128, pages=16, kc=FAKE, vc=FAKE, ksc=FAKE,
             vsc=FAKE)
    a.update(kw)
    return lib.msa_append_kv_fp8(*a.values(), None)


def gather(lib, **kw):
    a = dict(kc=FAKE, vc=FAKE, ksc=FAKE, vsc=FAKE, pages=16, slots=FAKE, T=4, Hkv=8, D=128, k=FAKE, v=FAKE)
    a.update(kw)
    return lib.msa_gather_kv_fp8(*a.values(), None)


def decode(lib, **kw):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, ksc=FAKE, vsc=FAKE, fpt=FAKE, lens=FAKE, R=4, Hq=64, Hkv=8, D=128, topk=16,
             pages=16, o=FAKE, lse=None, ws=at(0x10000), nbytes=1 << 40)
    a.update(kw)
    return lib.msa_paged_sparse_decode_fp8(*a.values(), None)


CACHES = [
    (dict(kc=None), ARG), (dict(vc=None), ARG), (dict(ksc=None), ARG), (dict(vsc=None), ARG), (dict(kc=at(0x1008)), ARG),
    (dict(vsc=at(0x1004)), ARG), (dict(pages=0), ARG), (dict(D=64), UNSUPPORTED), (dict(Hkv=3), UNSUPPORTED),
    (dict(Hkv=32), UNSUPPORTED), (dict(pages=1 << 21), UNSUPPORTED), (dict(pages=1 << 60), UNSUPPORTED),
]


@pytest.mark.parametrize("change,code", CACHES + [
    (dict(k=None), ARG), (dict(v=None), ARG), (dict(slots=None), ARG), (dict(T=-1), ARG), (dict(ks=1028), ARG),
    (dict(vs=-8), ARG), (dict(k=at(0x1008)), ARG), (dict(v=at(0x1002)), ARG),
])
def test_append_refuses(lib, change, code):
    assert append(lib, **change) == code
    assert lib.msa_last_error()


@pytest.mark.parametrize("change,code", CACHES + [
    (dict(k=None), ARG), (dict(v=None), ARG), (dict(slots=None), ARG), (dict(T=-1), ARG), (dict(k=at(0x1008)), ARG),
])
def test_gather_refuses(lib, change, code):
    assert gather(lib, **change) == code
    assert lib.msa_last_error()


@pytest.mark.parametrize("change,code", CACHES + [
    (dict(q=None), ARG), (dict(fpt=None), ARG), (dict(lens=None), ARG), (dict(o=None), ARG), (dict(R=-1), ARG),
    (dict(topk=0), ARG), (dict(topk=65), ARG), (dict(q=at(0x1008)), ARG), (dict(o=at(0x1008)), ARG),
    (dict(Hq=60), UNSUPPORTED), (dict(Hq=256), UNSUPPORTED), (dict(Hq=0), UNSUPPORTED), (dict(R=1 << 26), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(nbytes=1024), WORKSPACE), (dict(ws=at(0x10010)), WORKSPACE),
])
def test_decode_refuses(lib, change, code):
    assert decode(lib, **change) == code
    assert lib.msa_last_error()


def test_empty_calls_are_no_ops(lib):
    assert chunk(lib, B=0) == 0 and chunk(lib, T=0) == 0
    assert append(lib, T=0) == 0 and gather(lib, T=0) == 0 and decode(lib, R=0) == 0


def test_chunk_workspace_size(lib):
    size = lib.msa_chunk_attention_workspace_size
    assert size(1, 2048, 64, 8, 485) > size(1, 2048, 64, 8, 64) > size(1, 1, 64, 8, 64) > 0
    # few rows need small partials
    assert size(1, 1, 8, 1, 128) < size(1, 16, 8, 1, 128)
    # the stated number of pieces, 520 bytes a row, 2 * 128 rows a piece
    for mb in (485, 1024):
        stated = 456 * (1 + math.log(mb / 8)) * 2 * 128 * 520
        assert 0.95 * stated < size(1, 2048, 64, 8, mb) < 1.05 * stated
    for bad in ((0, 4, 64, 8, 4), (4, 0, 64, 8, 4), (4, 4, 60, 8, 4), (4, 4, 0, 8, 4), (4, 4, 96, 3, 4), (4, 4, 64, 8, 0),
                (16385, 4, 64, 8, 4), (4, 1 << 30, 64, 8, 4)):
        assert size(*bad) == 0


def test_binding_refuses_cpu_tensors(lib):
    i = torch.zeros(2, dtype=torch.int32)
    b = torch.zeros((2, 8, 128), dtype=torch.bfloat16)
    c = torch.zeros((1, 128, 8, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        msa.chunk_attention(b, c, c, torch.zeros((1, 1), dtype=torch.int32), i[:1], i)
    f = torch.zeros((1, 8, 128, 128), dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.zeros((1, 8, 128), dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        msa.append_kv_fp8(b, b, i, f, f, s, s)
    with pytest.raises(ValueError, match="CUDA"):
        msa.gather_kv_fp8(f, f, s, s, i)
    with pytest.raises(ValueError, match="CUDA"):
        msa.paged_sparse_decode_fp8(b, f, f, s, s, torch.zeros((16, 4), dtype=torch.int32), torch.zeros(16, dtype=torch.int32))
