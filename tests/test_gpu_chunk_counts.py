"""GPU tests of ``chunk_attention`` whose answers count every step of 64 keys (``_chunk_counts``), for both ways in
which a call cuts its keys: equal runs, and the list of a plan kernel on calls of thousands of live rows."""
import pytest
import torch

import _chunk_counts as counts
import block_sparse_attention_msa_gb300 as msa
from test_gpu_chunk_attention import DEV, check, make, reference, run

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


def lists(w, Hq, Hkv):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return counts.lists_its_work(w["seq"].numel(), w["q"].shape[0], Hq, Hkv, w["table"].shape[1], sms)


def mixed(n, seed, choices, top):
    g = torch.Generator().manual_seed(seed)
    new = [choices[i] for i in torch.randint(0, len(choices), (n,), generator=g).tolist()]
    return new, torch.randint(0, top, (n,), generator=g).tolist()


EQUAL = [
    # new tokens, tokens held before, Hq, Hkv, one score for all
    ([1], [60000], 8, 1, False), ([1], [99999], 4, 4, False), ([1, 1], [40000, 33], 16, 4, False),
    ([2000], [3000], 16, 4, False), ([1100, 900, 1, 1], [0, 6000, 9000, 1], 32, 2, False),
    ([3, 17, 1], [70000, 9000, 50000], 16, 2, False), ([1], [1000000], 8, 1, True), ([3, 1], [300000, 700000], 16, 2, True),
    (*mixed(64, 1, [1], 12000), 64, 8, False), (*mixed(61, 2, [1, 1, 1, 9, 90], 9000), 32, 4, False),
    (*mixed(2000, 3, [0, 1, 1, 2], 300), 8, 4, False), (*mixed(300, 4, [1, 7, 8, 9], 700), 16, 1, False),
]
LISTED = [
    ([5000], [3000], 64, 8, False),                                  # a chunk
    ([2500, 1, 700, 40, 0, 17, 300], [0, 7000, 100, 0, 5, 900, 20000], 32, 4, False),
    (*mixed(1300, 5, [17, 23, 40], 500), 16, 2, False),              # more requests, and live items, than the plan's threads
    (*mixed(1500, 6, [0, 1, 16, 33, 70], 200), 64, 8, False),
    ([10000], [0], 8, 8, False), ([9300, 900], [10, 3000], 8, 8, False),   # G 1
    ([2600, 100], [700, 0], 32, 2, False),                           # G 16
    (*mixed(300, 7, [17, 9, 24, 33], 900), 16, 1, False),            # one group: halves
    ([16384], [0], 64, 8, False),                                    # thousands of tickets
    ([2048], [60032], 64, 8, False),                                 # tiles in over a hundred pieces
    ([3000], [997000], 32, 4, True),
]


@pytest.mark.parametrize("new,held,Hq,Hkv,flat", EQUAL)
def test_equal_runs_count_every_step(new, held, Hq, Hkv, flat):
    w = counts.make(new, held, Hq, Hkv, seed=len(new), pad=len(new) % 3, flat=flat, device=DEV)
    assert not lists(w, Hq, Hkv)
    counts.check(run(w), new, held, Hq, Hkv, flat)


@pytest.mark.parametrize("new,held,Hq,Hkv,flat", LISTED)
def test_listed_units_count_every_step(new, held, Hq, Hkv, flat):
    w = counts.make(new, held, Hq, Hkv, seed=len(new), pad=len(new) % 3, flat=flat, device=DEV)
    assert lists(w, Hq, Hkv)
    for _ in range(2):      # another call, another order of tickets
        counts.check(run(w), new, held, Hq, Hkv, flat)


@pytest.mark.parametrize("B,Hq,Hkv", [(64, 64, 8), (3000, 16, 2), (16384, 4, 1)])
def test_decode_rows_in_a_step_of_large_capacity(B, Hq, Hkv):
    # captured for many more rows than it holds: the list of a few short units
    new, held = mixed(B, 8, [1], 5000 if B < 100 else 150)
    pad = B * (128 * Hkv // Hq) + 300
    w = counts.make(new, held, Hq, Hkv, seed=B, pad=pad, device=DEV)
    assert lists(w, Hq, Hkv)
    counts.check(run(w), new, held, Hq, Hkv)


@pytest.mark.parametrize("new,held,Hq,Hkv", [
    ([3000, 1, 50], [500, 4000, 0], 64, 8),
    ([700] * 12, [0] * 12, 16, 4),
    (*mixed(400, 9, [17, 40, 5], 300), 32, 2),
    (*mixed(500, 10, [17, 40, 5], 300), 8, 1),
])
def test_listed_units_against_64_bits(new, held, Hq, Hkv):
    w = make(new, held, Hq, Hkv, seed=len(new))
    assert lists(w, Hq, Hkv)
    check(run(w), reference(w, DEV))


def test_a_captured_call_that_lists_its_work_replays_with_other_lengths():
    Hq, Hkv, T, B = 32, 4, 6000, 5
    cases = [([5000, 1, 900, 0, 33], [100, 9000, 0, 7, 64]), ([1, 1, 1, 1, 1], [30000, 5, 64, 0, 900]),
             ([16, 2000, 17, 3000, 900], [0, 0, 500, 2000, 1]), ([0, 0, 0, 0, 6000], [3, 0, 0, 0, 10])]
    pages = mb = 300
    ws = [counts.make(n, h, Hq, Hkv, seed=i, pad=T - sum(n), device=DEV, pages=pages, mb=mb) for i, (n, h) in enumerate(cases)]
    d = {k: x.clone() for k, x in ws[0].items()}
    assert lists(d, Hq, Hkv)
    call = lambda: msa.chunk_attention(d["q"], d["kc"], d["vc"], d["table"], d["seq"], d["cu"])
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call()
    for i in (1, 2, 3, 0, 1):
        for k, x in ws[i].items():
            d[k].copy_(x)
        for _ in range(2):
            g.replay()
        counts.check(out, *cases[i], Hq, Hkv)
