"""GPU tests of ``chunk_attention`` with token ranges that overlap: the call ends soon with bit 1 of the device
error word, writes nothing outside the rows of its outputs, and leaves the next call right."""
import pytest
import torch

import block_sparse_attention_msa_gb300 as msa
from test_gpu_chunk_attention import BAD_LEN, D, DEV, PAGE, check, i32, make, reference, run

pytestmark = pytest.mark.gpu
ROOM = 1 << 20      # elements around an output


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


def with_room(shape, dtype):
    """An output between stretches of 7."""
    n = 1
    for s in shape:
        n *= s
    flat = torch.full((n + 2 * ROOM,), 7.0, dtype=dtype, device=DEV)
    return flat, flat[ROOM:ROOM + n].view(shape)


@pytest.mark.parametrize("B,T,mb,ranges", [
    # 41 requests claim all rows, of which each alone takes an eighth of what a call's counts hold: equal runs
    (16384, 131072, 1500, 82),
    (16384, 131072, 1500, 16384),
    # a million pairs of tiles and more: a list
    (2000, 40000, 20, 2000),
    (600, 40000, 2, 600),
    # some more than the rows there are
    (5, 5000, 3, 5), (5, 80, 3, 5),
])
def test_requests_that_claim_the_same_rows(B, T, mb, ranges):
    Hq, Hkv = 64, 4
    cu = torch.zeros(B + 1, dtype=torch.int32)
    cu[1:ranges:2] = T           # 0, T, 0, T, ...: every second request has them all
    q = torch.zeros((T, Hq, D), dtype=torch.bfloat16, device=DEV)
    kc = torch.zeros((2, PAGE, Hkv, D), dtype=torch.bfloat16, device=DEV)
    table = torch.ones((B, mb), dtype=torch.int32, device=DEV)
    seq = torch.full((B,), mb * PAGE, dtype=torch.int32, device=DEV)
    room_o, o = with_room((T, Hq, D), torch.bfloat16)
    room_l, lse = with_room((T, Hq), torch.float32)
    msa.chunk_attention(q, kc, kc, table, seq, cu.to(DEV), out=(o, lse))
    assert msa.device_error() == BAD_LEN
    for x in (room_o, room_l):
        assert (x[:ROOM] == 7).all() and (x[-ROOM:] == 7).all()


@pytest.mark.parametrize("cu", [[0, 24, 10, 30], [5, 3, 3, 30], [-4, 2, 2, 2], [0, 8, 30, 50000], [0, 30, 0, 30],
                                [0, 40000, 0, 40000], [40000, 0, 40000, 0]])
def test_ranges_out_of_order_in_a_call_that_lists_its_work(cu):
    w = make([8, 2, 20], [50, 9, 300], 16, 2, seed=12)
    w["q"] = torch.cat([w["q"], torch.zeros((40000 - 30, 16, D), dtype=torch.bfloat16)])
    room_o, o = with_room((40000, 16, D), torch.bfloat16)
    room_l, lse = with_room((40000, 16), torch.float32)
    run(dict(w, cu=i32(cu)), out=(o, lse))
    assert msa.device_error() == BAD_LEN
    for x in (room_o, room_l):
        assert (x[:ROOM] == 7).all() and (x[-ROOM:] == 7).all()
    ref = reference(dict(w, q=w["q"][:30]))
    o, lse = run(w)
    check((o[:30], lse[:30]), ref)
