"""Chunk attention refuses outputs and workspaces that overlap an input or one another, on the host. No check
follows these, so the calls that pass them are made only where there is no device to launch on."""
import ctypes

import pytest
import torch

import block_sparse_attention_msa_gb300 as msa

at = ctypes.c_void_p
ARG = -1
B, T, HQ, HKV, MB, PAGES = 4, 100, 64, 8, 16, 64
Q, K, V, TABLE, SEQ, CU, O, LSE, WS = (n << 32 for n in range(1, 10))     # addresses, far apart
ROW, CACHE = HQ * 256, PAGES * 128 * HKV * 256


@pytest.fixture(scope="module")
def lib():
    from block_sparse_attention_msa_gb300 import build
    build.build()
    return msa.load()


def call(lib, stride=8192, T=T, **kw):
    a = dict(q=Q, k=K, v=V, table=TABLE, seq=SEQ, cu=CU, o=O, lse=LSE, ws=WS)
    a.update(kw)
    need = lib.msa_chunk_attention_workspace_size(B, T, HQ, HKV, MB)
    return lib.msa_chunk_attention(at(a["q"]), stride, at(a["k"]), at(a["v"]), at(a["table"]), at(a["seq"]),
                                   at(a["cu"]), B, T, HQ, HKV, 128, MB, PAGES, at(a["o"]),
                                   None if a["lse"] is None else at(a["lse"]), at(a["ws"]), need, None)


@pytest.mark.parametrize("change", [
    dict(o=Q), dict(o=Q + T * ROW - 16), dict(o=Q - T * ROW + 16), dict(o=K), dict(o=K + CACHE - 16),
    dict(o=V - T * ROW + 16), dict(o=TABLE), dict(o=SEQ - 256), dict(o=CU - 1024), dict(o=LSE - 16),
    dict(lse=Q + 4), dict(lse=Q + T * ROW - 4), dict(lse=K + CACHE - 4), dict(lse=V), dict(lse=TABLE + B * MB * 4 - 4),
    dict(lse=SEQ + B * 4 - 4), dict(lse=CU + B * 4), dict(lse=CU - T * HQ * 4 + 4), dict(lse=O + 256),
    dict(lse=O + T * ROW - 4), dict(ws=Q), dict(ws=K + CACHE - 256), dict(ws=O), dict(ws=O + T * ROW - 256),
    dict(lse=WS), dict(o=WS + 256), dict(ws=SEQ), dict(ws=CU),
    # q's rows apart: the second row, and what reaches from before it
    dict(o=Q + (1 << 20), stride=1 << 19), dict(lse=Q + (1 << 20), stride=1 << 19),
    dict(lse=Q + (1 << 20) - 256, stride=1 << 19), dict(lse=Q + 99 * (1 << 20) + ROW - 4, stride=1 << 19),
])
def test_overlaps_are_refused(lib, change):
    assert call(lib, **change) == ARG
    assert b"overlaps" in lib.msa_last_error()


@pytest.mark.skipif(torch.cuda.is_available(), reason="the calls would be launched")
@pytest.mark.parametrize("change", [
    dict(), dict(lse=None), dict(o=Q + T * ROW), dict(o=Q - T * ROW), dict(o=K + CACHE), dict(lse=O + T * ROW),
    dict(lse=O - T * HQ * 4), dict(lse=CU + (B + 1) * 4), dict(k=V), dict(table=SEQ),
    dict(lse=Q + ROW, stride=1 << 19), dict(lse=Q + 98 * (1 << 20) + ROW, stride=1 << 19),
    dict(lse=Q + (1 << 20) - T * HQ * 4, stride=1 << 19), dict(o=Q + ROW, stride=1 << 23),
    dict(lse=Q + 99 * (1 << 20) + ROW, stride=1 << 19),
])
def test_neighbours_and_the_gaps_between_rows_are_not(lib, change):
    assert call(lib, **change) != 0                 # no device to launch on
    assert b"overlaps" not in lib.msa_last_error()
