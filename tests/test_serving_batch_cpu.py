"""The serving-batch entry points without a GPU: every refusal happens on the host, before any
device work, through the C ABI and through the Python binding."""
import ctypes

import pytest
import torch

import block_sparse_attention_msa_gb300 as msa

FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: every call below fails host validation
OUT = [ctypes.c_void_p(0x2000 + 0x100 * i) for i in range(6)]
ARG, SHAPE, UNSUPPORTED, WORKSPACE = -1, -2, -3, -4


@pytest.fixture(scope="module")
def lib():
    from block_sparse_attention_msa_gb300 import build
    build.build()
    return msa.load()


def tables(lib, **kw):
    a = dict(prev=FAKE, new=FAKE, B=4, mb=8, table=OUT[5], free=FAKE, nfree=10, used=FAKE, shared=None,
             nshared=0, pages=64, T=16, seq=OUT[0], cu=OUT[1], slots=OUT[2], pos=OUT[3], out=OUT[4])
    a.update(kw)
    return lib.msa_build_page_tables(*a.values(), None)


@pytest.mark.parametrize("change,code", [
    (dict(prev=None), ARG), (dict(new=None), ARG), (dict(table=None), ARG), (dict(free=None), ARG),
    (dict(used=None), ARG), (dict(nshared=2), ARG), (dict(seq=None), ARG), (dict(cu=None), ARG),
    (dict(slots=None), ARG), (dict(pos=None), ARG), (dict(out=None), ARG),
    (dict(B=-1), ARG), (dict(B=0), ARG), (dict(T=-1), ARG), (dict(mb=0), ARG), (dict(nfree=-1), ARG),
    (dict(nshared=-1), ARG), (dict(pages=0), ARG),
    (dict(seq=FAKE), ARG), (dict(out=FAKE), ARG), (dict(table=FAKE), ARG),    # an output is an input
    (dict(shared=FAKE, nshared=9), SHAPE),
    (dict(B=16385), UNSUPPORTED), (dict(pages=1 << 24), UNSUPPORTED),
    (dict(mb=1 << 24), UNSUPPORTED), (dict(B=16384, mb=1 << 18), UNSUPPORTED),
])
def test_page_tables_refuse(lib, change, code):
    assert tables(lib, **change) == code
    assert lib.msa_last_error()


def at(x):
    return ctypes.c_void_p(x)


@pytest.mark.parametrize("change", [
    # [4] lengths, [10] free pages, [16] rows, a table of 4 x 8: an output that overlaps an input ...
    dict(prev=at(0x10000), seq=at(0x10000 + 12)), dict(new=at(0x10000 + 12), cu=at(0x10000)),
    dict(free=at(0x10000), slots=at(0x10000 + 36)), dict(free=at(0x10000 + 60), pos=at(0x10000)),
    dict(used=at(0x10000 + 16), cu=at(0x10000)), dict(prev=at(0x10000 + 124), table=at(0x10000)),
    dict(free=at(0x10000), table=at(0x10000 + 36)), dict(used=at(0x10000 + 4), table=at(0x10000)),
    dict(shared=at(0x10000), nshared=8, slots=at(0x10000 + 28)),
    # ... or another output
    dict(slots=OUT[3]), dict(seq=OUT[1]), dict(out=OUT[5]), dict(cu=at(0x10000), pos=at(0x10000 + 16)),
    dict(table=at(0x10000), seq=at(0x10000 + 124)), dict(slots=at(0x10000 + 60), pos=at(0x10000)),
])
def test_page_tables_refuse_overlapping_outputs(lib, change):
    assert tables(lib, **change) == ARG
    assert b"overlap" in lib.msa_last_error()


def append(lib, **kw):
    a = dict(k=FAKE, ks=1024, v=FAKE, vs=1024, x=FAKE, xs=1024, slots=FAKE, T=4, Hkv=8, D=128, Di=128,
             pages=16, kc=OUT[0], vc=OUT[1], xc=OUT[2])
    a.update(kw)
    return lib.msa_append_kv(*a.values(), None)


@pytest.mark.parametrize("change,code", [
    (dict(k=None), ARG), (dict(v=None), ARG), (dict(k=None, v=None, x=None), ARG), (dict(slots=None), ARG),
    (dict(kc=None), ARG), (dict(vc=None), ARG), (dict(xc=None), ARG), (dict(T=-1), ARG),
    (dict(pages=0), ARG), (dict(ks=1028), ARG), (dict(vs=-8), ARG), (dict(xs=4), ARG),
    (dict(k=ctypes.c_void_p(0x1008)), ARG), (dict(xc=ctypes.c_void_p(0x1002)), ARG),
    (dict(Hkv=3), UNSUPPORTED), (dict(Hkv=32), UNSUPPORTED), (dict(D=64), UNSUPPORTED),
    (dict(Di=96), UNSUPPORTED), (dict(pages=1 << 24), UNSUPPORTED),
])
def test_append_refuses(lib, change, code):
    assert append(lib, **change) == code
    assert lib.msa_last_error()


def decode(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, table=FAKE, seq=FAKE, shared=FAKE, B=4, N=1, Hq=64, Hkv=8, D=128, mb=16,
             pages=64, o=FAKE, lse=None, ws=ctypes.c_void_p(0x10000), nbytes=1 << 30)
    a.update(kw)
    return lib.msa_shared_prefix_decode(*a.values(), None)


@pytest.mark.parametrize("change,code", [
    (dict(q=None), ARG), (dict(k=None), ARG), (dict(v=None), ARG), (dict(table=None), ARG),
    (dict(seq=None), ARG), (dict(shared=None), ARG), (dict(o=None), ARG), (dict(B=-1), ARG),
    (dict(N=0), ARG), (dict(mb=0), ARG), (dict(pages=0), ARG), (dict(q=ctypes.c_void_p(0x1008)), ARG),
    (dict(N=17), UNSUPPORTED), (dict(D=64), UNSUPPORTED), (dict(Hkv=3, Hq=24), UNSUPPORTED),
    (dict(Hq=60), UNSUPPORTED), (dict(Hq=256), UNSUPPORTED), (dict(Hq=0), UNSUPPORTED),
    (dict(pages=1 << 24), UNSUPPORTED), (dict(mb=1 << 24), UNSUPPORTED),
    (dict(B=1 << 16, mb=1 << 13), UNSUPPORTED), (dict(B=1 << 30), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(nbytes=1024), WORKSPACE),
    (dict(ws=ctypes.c_void_p(0x10010)), WORKSPACE),
])
def test_decode_refuses(lib, change, code):
    assert decode(lib, **change) == code
    assert lib.msa_last_error()


def test_empty_batches(lib):
    # no-ops, except where an output would have a value (the pages used, cu_tokens[0])
    assert tables(lib, B=0, T=0) == ARG
    assert append(lib, T=0) == 0
    assert decode(lib, B=0) == 0


def test_decode_workspace_size(lib):
    size = lib.msa_shared_prefix_decode_workspace_size
    # at least one fp32 partial of every row
    assert size(64, 1, 64, 8) >= 64 * 64 * 128 * 4
    assert size(256, 4, 64, 8) > size(256, 1, 64, 8) > size(1, 1, 64, 8) > 0
    for bad in ((0, 1, 64, 8), (4, 0, 64, 8), (4, 17, 64, 8), (4, 1, 60, 8), (4, 1, 0, 8), (4, 1, 96, 3)):
        assert size(*bad) == 0


@pytest.mark.parametrize("sizes,megabytes", [
    ((64, 1, 64, 8), 26), ((256, 1, 64, 8), 59), ((4096, 1, 64, 8), 920), ((512, 4, 128, 8), 930),
    ((256, 16, 256, 16), 2400),
])
def test_decode_workspace_is_as_large_as_documented(lib, sizes, megabytes):
    # the documented figures are for 152 SMs; without a device the library counts 148
    got = lib.msa_shared_prefix_decode_workspace_size(*sizes) / 1e6
    assert 0.95 * megabytes <= got <= 1.05 * megabytes


def test_binding_refuses_cpu_tensors_and_shapes(lib):
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        msa.build_page_tables(i, i, torch.zeros((2, 4), dtype=torch.int32), i, i[:1], T=2, num_pages=4)
    b = torch.zeros((2, 8, 128), dtype=torch.bfloat16)
    c = torch.zeros((1, 128, 8, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        msa.append_kv(b, b, None, i, c, c, None)
    with pytest.raises(ValueError, match="CUDA"):
        msa.shared_prefix_decode(b, c, c, torch.zeros((2, 1), dtype=torch.int32), i, i[:1])


@pytest.mark.parametrize("sizes", [dict(T=2 ** 32 + 2), dict(T=2 ** 31), dict(T=2, num_pages=2 ** 64 + 4)])
def test_binding_refuses_sizes_past_int32(lib, sizes):
    # the C arguments would wrap around: 2^32 + 2 rows would be a call for 2
    i = torch.zeros(2, dtype=torch.int32)
    a = dict(num_pages=4)
    a.update(sizes)
    with pytest.raises(ValueError, match="int32"):
        msa.build_page_tables(i, i, torch.zeros((2, 4), dtype=torch.int32), i, i[:1], **a)


def test_sizes_of_tensors_past_int32():
    from block_sparse_attention_msa_gb300 import _sizes
    _sizes("name", 0, 5, 2 ** 31 - 1)
    with pytest.raises(ValueError, match="name.*int32"):
        _sizes("name", 3, 2 ** 31, 7)
