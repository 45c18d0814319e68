"""GPU tests of the serving-batch operators against plain 64-bit implementations written here:
``build_page_tables`` (integers: equal), ``append_kv`` (copies: equal), ``shared_prefix_decode``,
and a run of the three together with the sparse path on the same caches.

Attention tolerance, per output element, from the roundings the kernel makes. With w the exact
softmax weights, A = sum_n w_n |v_n| and ref the exact output:
  * P = 2^(s - m) is rounded to bf16 for its product: at most 2^-8 of each term, 2^-8 A in all
    (m a reference near the row's maximum);
  * o is rounded to bf16 once: 2^-8 of the value;
  * a score is an fp32 sum of 128 exact products of bf16 numbers, at most 2^-23 of sum |q_d k_d| per
    addition (truncating adds counted), then scaled to log2 units: ds = 2^-23 * 128 * max_n
    sum_d |q_d k_nd| + 2^-21 * max |s|, which moves weights by at most 2 ds A;
  * 2^x, the fp32 sums of P V and l and the joins: 2^-21 + n * 2^-24 per key count n, of A.
LSE: ds + 2^-21 + n * 2^-24 absolute, + 2^-23 of the value.
"""
import numpy as np
import pytest
import torch

import _long_runs as lr
import block_sparse_attention_msa_gb300 as msa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
PAGE = 128
D = 128
BAD_PAGE, BAD_LEN, NO_PAGE = 1, 2, 8


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_sparse_attention_msa_gb300 import build
    build.build()
    msa.load()
    assert msa.device_error() == 0  # nothing left over from earlier tests
    yield
    assert msa.device_error() == 0


@pytest.fixture(autouse=True)
def no_error_left():
    yield
    assert msa.device_error() == 0  # a wait that ran out shows in its own test


def i32(x):
    return torch.from_numpy(np.array(x, dtype=np.int32))


# ------------------------------------------------------------------------------ page tables

def ref_tables(prev, new, table, free, used, T, shared=None, num_pages=1 << 30):
    """The documented rules, one token at a time."""
    table = table.copy()
    B, mb = table.shape
    seq, cu, slots, pos = [], [0], [-1] * T, [-1] * T
    for b in range(B):
        p = min(max(int(prev[b]), 0), mb * PAGE)
        n = min(max(int(new[b]), 0), mb * PAGE - p)
        if shared is not None and p >= len(shared) * PAGE:
            table[b, :len(shared)] = shared
        length = p
        stopped = False
        for i in range(n):
            at = p + i
            if at % PAGE == 0:
                if used < len(free):
                    page = int(free[used])
                    used += 1
                    table[b, at // PAGE] = page if 0 <= page < num_pages else -1
                else:
                    table[b, at // PAGE] = -1
                    stopped = True
            if not stopped:
                length = at + 1
            t = cu[-1] + i
            if t < T:
                pos[t] = at
                page = -1 if stopped else int(table[b, at // PAGE])
                slots[t] = page * PAGE + at % PAGE if 0 <= page < num_pages else -1
        seq.append(length)
        cu.append(cu[-1] + n)
    return table, seq, cu, slots, pos, used


def check_tables(prev, new, mb, free, used, T, shared=None, num_pages=1 << 20, expect=0, seed=0):
    rng = np.random.default_rng(seed)
    B = len(prev)
    table = rng.integers(0, min(num_pages, 1 << 20), (B, mb)).astype(np.int32)
    table_d = i32(table).to(DEV)
    shared_d = None if shared is None else i32(shared).to(DEV)
    free_d = i32(free).to(DEV)
    ins = (i32(prev).to(DEV), i32(new).to(DEV), free_d, i32([used]).to(DEV))
    copies = [x.clone() for x in ins]
    got = msa.build_page_tables(ins[0], ins[1], table_d, free_d, ins[3], T=T, num_pages=num_pages,
                                shared_pages=shared_d)
    assert msa.device_error() == expect
    want = ref_tables(prev, new, table, free, min(max(used, 0), len(free)), T, shared, num_pages)
    assert np.array_equal(table_d.cpu().numpy(), want[0])
    for name, g, w in zip(("seq_lens", "cu_tokens", "slot_map", "positions"), got, want[1:5]):
        assert np.array_equal(g.cpu().numpy(), np.asarray(w, dtype=np.int32)), name
    assert int(got[4]) == want[5]
    for a, b in zip(ins, copies):
        assert torch.equal(a, b)  # inputs are left alone
    return got


@pytest.mark.parametrize("prev,new,pad", [
    ([0], [1], 0),                                   # the first token of a request
    ([0], [0], 3),                                   # nothing to do, padding rows only
    ([127], [1], 0), ([128], [1], 0), ([127], [2], 5),   # around a page border
    ([0, 5, 128, 255, 300], [0, 1, 1, 1, 0], 2),     # idle rows in a decode step
    ([700, 0, 1, 129], [300, 513, 0, 128], 0),       # chunks
    ([0] * 7, [0, 0, 1000, 0, 0, 1, 0], 9),          # empty requests around a long one
])
def test_page_tables_small(prev, new, pad):
    total = sum(new)
    check_tables(prev, new, 12, np.arange(100, 140)[::-1], 3, total + pad)


@pytest.mark.parametrize("B,hi,mb", [(61, 900, 40), (255, 3, 9), (256, 5, 9), (257, 300, 16), (1500, 2, 10)])
def test_page_tables_ragged(B, hi, mb):
    rng = np.random.default_rng(B)
    prev = rng.integers(0, (mb - 8) * PAGE, B)
    new = rng.integers(0, hi + 1, B)
    free = rng.permutation(1 << 16)[:B * 9 + 5]
    check_tables(prev, new, mb, free, 2, int(new.sum()) + 11, seed=B)


@pytest.mark.parametrize("B,hi,mb,shared", [
    (6143, 3, 5, 0), (6144, 2, 5, 0),    # the scans around 48 KB of shared memory
    (16384, 2, 4, 2), (16384, 130, 4, 0),    # the largest batch
])
def test_page_tables_large_batches(B, hi, mb, shared):
    rng = np.random.default_rng(B + hi)
    prev = rng.integers(0, (mb - 2) * PAGE + 1, B)
    prev[::3] = (mb - 2) * PAGE    # at a page border: holds the shared pages, opens one
    new = rng.integers(0, hi + 1, B)
    free = rng.permutation(1 << 16)[:2 * B + 5]
    check_tables(prev, new, mb, free, 3, int(new.sum()) + 77, seed=B,
                 shared=rng.integers(0, 1 << 16, shared) if shared else None)


def test_page_tables_shared_prefix():
    shared = np.array([9, 3, 77, 5])
    prev = [512, 512, 600, 511, 0, 512]   # requests 3 and 4 do not hold the whole prefix
    check_tables(prev, [1, 0, 200, 1, 130, 129], 16, np.arange(50, 90), 0, 470, shared=shared)


def test_page_tables_free_list_runs_out():
    # 6 fresh pages needed, 4 left: request 1 is cut after its first fresh page, request 2 gets none
    check_tables([128, 128, 128], [256, 256, 256], 8, np.arange(20, 30), 7, 768, expect=NO_PAGE)
    check_tables([130, 100], [1, 1], 8, np.zeros(0, dtype=np.int32), 0, 2)  # none needed


def test_page_tables_bad_values():
    # lengths out of range are clamped, rows past T dropped, a bad index into the list clamped
    check_tables([-5, 10, 4 * PAGE + 9], [3, -1, 7], 4, np.arange(9), 0, 30, expect=BAD_LEN)
    check_tables([0], [4 * PAGE + 50], 4, np.arange(9), 0, 4 * PAGE, expect=BAD_LEN)
    check_tables([0, 5], [100, 100], 4, np.arange(9), 1, 150, expect=BAD_LEN)
    check_tables([0], [3], 4, np.arange(9), -4, 3, expect=BAD_LEN)
    # a page of the free list outside the cache
    check_tables([0, 0], [200, 100], 4, np.array([5, 64, 7, -1]), 0, 300, num_pages=64,
                 expect=BAD_PAGE)


def test_page_tables_captured_and_replayed_with_other_lengths():
    B, mb, T = 5, 8, 64
    prev = torch.zeros(B, dtype=torch.int32, device=DEV)
    new = torch.ones(B, dtype=torch.int32, device=DEV)
    table = torch.zeros((B, mb), dtype=torch.int32, device=DEV)
    free = torch.arange(100, dtype=torch.int32, device=DEV)
    used = torch.zeros(1, dtype=torch.int32, device=DEV)
    msa.build_page_tables(prev, new, table, free, used, T=T, num_pages=100)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = msa.build_page_tables(prev, new, table, free, used, T=T, num_pages=100)
    for seed in range(3):
        rng = np.random.default_rng(seed)
        pv, nw = rng.integers(0, 700, B), rng.integers(0, 14, B)
        prev.copy_(i32(pv))
        new.copy_(i32(nw))
        used.fill_(seed)
        table.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        want = ref_tables(pv, nw, np.full((B, mb), 7, dtype=np.int32), np.arange(100), seed, T)
        assert np.array_equal(table.cpu().numpy(), want[0])
        for g, w in zip(out, want[1:5]):
            assert np.array_equal(g.cpu().numpy(), np.asarray(w, dtype=np.int32))
        assert int(out[4]) == want[5]


def test_page_tables_into_given_outputs_step_after_step():
    # a decode loop's two sets of buffers, each step's lengths and pages used the next one's inputs
    B, mb, T = 5, 6, 9
    zeros = lambda n: torch.zeros(n, dtype=torch.int32, device=DEV)
    sets = [[zeros(B), zeros(B + 1), zeros(T), zeros(T), zeros(1)] for _ in range(2)]
    table, new = torch.full((B, mb), -1, dtype=torch.int32, device=DEV), zeros(B)
    free = torch.arange(60, dtype=torch.int32, device=DEV).flip(0)
    prev, used, want_table = [126, 0, 250, 255, 128], 0, np.full((B, mb), -1, dtype=np.int32)
    table[:, :2] = want = torch.arange(50, 60, dtype=torch.int32).view(B, 2).to(DEV)
    want_table[:, :2] = want.cpu().numpy()
    sets[1][0].copy_(i32(prev))
    for step in range(6):
        old, out = sets[(step + 1) % 2], sets[step % 2]
        tokens = [1, 2, 0, 1, 3] if step % 2 else [1, 1, 1, 1, 1]
        new.copy_(i32(tokens))
        got = msa.build_page_tables(old[0], new, table, free, old[4], T=T, num_pages=60, out=out)
        assert all(g.data_ptr() == o.data_ptr() for g, o in zip(got, out, strict=True))
        want_table, prev, cu, slots, pos, used = ref_tables(prev, tokens, want_table, free.cpu().numpy(), used, T)
        for g, w in zip((*out, table), (prev, cu, slots, pos, [used], want_table), strict=True):
            assert np.array_equal(g.cpu().numpy(), np.asarray(w, dtype=np.int32))


def test_page_tables_refuse_outputs_that_do_not_fit():
    zeros = lambda n, dtype=torch.int32: torch.zeros(n, dtype=dtype, device=DEV)
    B, T = 3, 7
    args = (zeros(B), zeros(B), zeros((B, 4)), zeros(9), zeros(1))
    good = [zeros(B), zeros(B + 1), zeros(T), zeros(T), zeros(1)]
    msa.build_page_tables(*args, T=T, num_pages=9, out=good)
    for at, x, error in ((0, zeros(B + 1), ValueError), (2, zeros(T - 1), ValueError),
                         (3, zeros(T, torch.int64), TypeError), (4, zeros(2)[:0], ValueError),
                         (1, zeros(2 * B + 2)[::2], ValueError), (0, args[0], msa.MSAError),
                         (3, good[2], msa.MSAError), (0, good[1][1:], msa.MSAError)):
        with pytest.raises(error):
            msa.build_page_tables(*args, T=T, num_pages=9, out=[x if i == at else o for i, o in enumerate(good)])
    with pytest.raises(ValueError):
        msa.build_page_tables(*args, T=T, num_pages=9, out=good[:4])


def test_page_tables_without_token_rows():
    # no rows are asked for: lengths and tables alone
    check_tables([0, 100], [0, 0], 4, np.arange(9), 0, 0)
    check_tables([0, 100, 128], [200, 29, 0], 4, np.arange(9), 0, 0, expect=BAD_LEN)  # every row is past T


# ------------------------------------------------------------------------------ append

@pytest.mark.parametrize("T,Hkv,Di,strided", [
    (1, 8, 128, False), (3, 1, 64, True), (37, 2, 64, True), (513, 16, 128, False),
    (1000, 4, 128, True), (129, 8, 64, True),
])
def test_append_kv(T, Hkv, Di, strided):
    g = torch.Generator(device=DEV).manual_seed(T)
    P = T // PAGE + 3
    rnd = lambda *s: torch.randn(s, generator=g, device=DEV).to(torch.bfloat16)
    if strided:
        qkv = rnd(T, 3 * Hkv * D + Hkv * Di)
        k = qkv[:, Hkv * D:2 * Hkv * D].unflatten(1, (Hkv, D))
        v = qkv[:, 2 * Hkv * D:3 * Hkv * D].unflatten(1, (Hkv, D))
        x = qkv[:, 3 * Hkv * D:].unflatten(1, (Hkv, Di))
    else:
        k, v, x = rnd(T, Hkv, D), rnd(T, Hkv, D), rnd(T, Hkv, Di)
    k[0, 0, 0], v[0, 0, 1] = float("nan"), float("-inf")  # bits are copied, whatever they say
    slots = torch.randperm(P * PAGE, generator=g, device=DEV)[:T].to(torch.int32)
    slots[T // 3::7] = -1
    caches = [rnd(P, PAGE, Hkv, D), rnd(P, PAGE, Hkv, D), rnd(P, PAGE, Hkv, Di)]
    want = [c.clone() for c in caches]
    live = slots >= 0
    for c, rows in zip(want, (k, v, x)):
        c.view(-1, *c.shape[2:])[slots[live].long()] = rows[live]
    msa.append_kv(k, v, x, slots, *caches)
    for c, w in zip(caches, want):
        assert torch.equal(c.view(torch.int16), w.view(torch.int16))
    # K/V alone, and the key index alone
    again = [torch.zeros_like(c) for c in caches]
    msa.append_kv(k, v, None, slots, again[0], again[1], None)
    msa.append_kv(None, None, x, slots, None, None, again[2])
    cells = slots[live].long()
    for c, w in zip(again, want):
        flat, ref = c.view(-1, *c.shape[2:]), w.view(-1, *w.shape[2:])
        assert torch.equal(flat[cells].view(torch.int16), ref[cells].view(torch.int16))
        flat[cells] = 0
        assert not flat.any()


@pytest.mark.parametrize("n", [1, 37, 127, 128])
def test_append_kv_copies_a_page_within_the_caches(n):
    # the private copies of a partly filled shared page: the rows are cells of the caches
    g = torch.Generator(device=DEV).manual_seed(n)
    caches = [torch.randn((6, PAGE, 4, d), generator=g, device=DEV).to(torch.bfloat16) for d in (D, D, 64)]
    want = [c.clone() for c in caches]
    for c in want:
        for page in (0, 4):
            c[page, :n] = c[2, :n]
    for page in (0, 4):
        slots = torch.arange(n, dtype=torch.int32, device=DEV) + page * PAGE
        msa.append_kv(*(c[2, :n] for c in caches), slots, *caches)
    for c, w in zip(caches, want):
        assert torch.equal(c, w)


def test_append_kv_skips_bad_slots_and_empty_batches():
    k = torch.ones((3, 2, D), dtype=torch.bfloat16, device=DEV)
    caches = [torch.zeros((2, PAGE, 2, D), dtype=torch.bfloat16, device=DEV) for _ in range(3)]
    msa.append_kv(k, k, k, i32([2 * PAGE, -7, 2 * PAGE - 1]).to(DEV), *caches)
    assert msa.device_error() == BAD_PAGE
    for c in caches:
        assert c.view(-1, 2, D)[-1].eq(1).all() and c.view(-1, 2, D)[:-1].eq(0).all()
    none = k[:0]
    msa.append_kv(none, none, none, i32([]).to(DEV), *caches)


# ------------------------------------------------------------------------------ decode

def make_decode(seq, shared, N, Hq, Hkv, seed, scale=1.0):
    """Caches whose unused cells are NaN, one page table per request, shared pages in common."""
    g = torch.Generator().manual_seed(seed)
    B = len(seq)
    whole = shared // PAGE
    blocks = [(n + PAGE - 1) // PAGE for n in seq]
    mb = max(1, max(blocks), whole)
    pages = whole + sum(max(0, n - whole) for n in blocks) + 2
    perm = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.randint(0, pages, (B, mb), generator=g).to(torch.int32)  # unused entries: any page
    kc = torch.full((pages, PAGE, Hkv, D), float("nan"), dtype=torch.bfloat16)
    vc = kc.clone()
    rnd = lambda n: (torch.randn((n, Hkv, D), generator=g) * scale).to(torch.bfloat16)
    pk, pv = rnd(shared), torch.randn((shared, Hkv, D), generator=g).to(torch.bfloat16)
    used = whole
    for b, n in enumerate(seq):
        if n == 0:
            continue
        table[b, :whole] = perm[:whole]
        for j in range(whole, blocks[b]):
            table[b, j] = perm[used]
            used += 1
        own = n - shared
        k = torch.cat([pk, rnd(own)]) if own >= 0 else rnd(n)
        v = torch.cat([pv, rnd(own)]) if own >= 0 else rnd(n)
        for j in range(blocks[b]):
            m = min(PAGE, n - j * PAGE)
            kc[table[b, j], :m] = k[j * PAGE:j * PAGE + m]
            vc[table[b, j], :m] = v[j * PAGE:j * PAGE + m]
    q = (torch.randn((B * N, Hq, D), generator=g) * D ** -0.5).to(torch.bfloat16)
    return dict(q=q, kc=kc, vc=vc, table=table, seq=i32(seq), N=N, shared=shared)


def ref_decode(w, device="cpu"):
    """o, lse, and per element / row the tolerances of the module docstring, in 64 bits."""
    q, N = w["q"].double(), w["N"]
    R, Hq, _ = q.shape
    Hkv = w["kc"].shape[2]
    G = Hq // Hkv
    o = torch.zeros((R, Hq, D), dtype=torch.float64, device=device)
    lse = torch.full((R, Hq), float("-inf"), dtype=torch.float64, device=device)
    to, tl = torch.zeros_like(o), torch.zeros_like(lse)
    for b, n in enumerate(w["seq"].tolist()):
        pages = w["table"][b, :(n + PAGE - 1) // PAGE].long()
        k = w["kc"][pages].flatten(0, 1)[:n].double().permute(1, 2, 0)
        v = w["vc"][pages].flatten(0, 1)[:n].double().transpose(0, 1)
        for i in range(N):
            vis = n - N + i + 1
            if vis <= 0:
                continue
            qi = q[b * N + i].view(Hkv, G, D)
            s = qi @ k[:, :, :vis]
            z = torch.logsumexp(s, -1, keepdim=True)
            p = torch.exp(s - z)
            ref = p @ v[:, :vis]
            A = p @ v[:, :vis].abs()
            dots = (qi.abs() @ k[:, :, :vis].abs()).amax(-1, keepdim=True)
            ds = 2.0 ** -23 * 128 * dots + 2.0 ** -21 * s.abs().amax(-1, keepdim=True)
            acc = 2.0 ** -21 + vis * 2.0 ** -24
            r = b * N + i
            o[r], lse[r] = ref.reshape(Hq, D), z.reshape(Hq)
            to[r] = (2.0 ** -8 * (ref.abs() + A) * (1 + 2.0 ** -7) + (2 * ds + acc) * A).reshape(Hq, D)
            tl[r] = (ds + acc + 2.0 ** -23 * z.abs()).reshape(Hq)
    return o, lse, to, tl


def run_decode(w, shared=None, **kw):
    d = {k: x.to(DEV) for k, x in w.items() if isinstance(x, torch.Tensor)}
    sl = i32([w["shared"] if shared is None else shared]).to(DEV)
    return msa.shared_prefix_decode(d["q"], d["kc"], d["vc"], d["table"], d["seq"], sl, N=w["N"], **kw)


def check_decode(got, ref):
    o, lse, to, tl = ref
    go, gl = got[0].double().cpu(), got[1].double().cpu()
    err = (go - o).abs()
    assert (err <= to).all(), f"o: worst error / tolerance {(err / to.clamp_min(1e-300)).max():.3f}"
    empty = torch.isneginf(lse)
    assert torch.equal(torch.isneginf(gl), empty)
    assert (go[empty] == 0).all()
    err = (gl - lse).abs()[~empty]
    assert (err <= tl[~empty]).all(), f"lse: worst error / tolerance {(err / tl[~empty]).max():.3f}"


CASES = [
    # seq, shared, N, Hq, Hkv
    ([1], 0, 1, 8, 2),                               # one token, one request
    ([1], 1, 1, 1, 1),                               # ... all of it shared: below a step, private
    ([64], 64, 1, 8, 2), ([65], 64, 1, 8, 2),        # exactly the prefix; one key more
    ([2048], 1000, 1, 8, 2),                         # one odd tile, private remainder
    ([300, 301, 427, 1000, 256], 256, 1, 64, 8),     # shared pages, ragged
    ([700, 645, 641, 1500], 640, 3, 32, 4),          # several rows per request, causal
    ([777] * 9, 513, 1, 16, 16),                     # one head per group
    ([129, 200, 190], 129, 16, 16, 1),               # G 16, N 16: two tiles per request
    ([400 + 3 * i for i in range(20)], 384, 1, 64, 4),    # 320 rows per group: a pair and an odd tile
    ([520 + i for i in range(32)], 500, 1, 64, 8),   # 256 rows per group: one pair exactly
    ([1030 + 7 * i for i in range(48)], 1024, 2, 16, 2),  # 768 rows: three pairs
    ([0, 90, 0, 700, 5, 0], 0, 1, 8, 1),             # padding requests
    ([0, 900, 0, 700, 650, 0] * 9, 600, 1, 8, 1),    # ... in the prefix tiles too
    ([2, 500, 16, 1], 0, 8, 8, 2),                   # rows at negative positions
    ([60, 300, 200], 190, 4, 16, 2),                 # a request shorter than shared_len claims
    ([5000, 3, 70, 4100], 0, 1, 64, 8),              # private only, one short among long
    ([9000], 8960, 1, 64, 8),                        # a long prefix cut over every CTA
    ([130 + (i * 37) % 200 for i in range(300)], 128, 1, 8, 2),   # many requests
    ([0, 0, 0], 128, 2, 8, 2),                       # nobody is active
    ([400, 333, 512], 192, 5, 64, 8),                # 40 rows per request: one area, one buffer
    ([400, 333, 512, 300, 311], 256, 16, 8, 1),      # 128 rows per request, wide query areas
    ([210, 340, 199], 128, 16, 16, 1),               # two tiles per request behind a pair
    ([200 + i % 50 for i in range(144)], 192, 1, 16, 1),  # nine pairs in rounds
    ([100 + i % 150 for i in range(150)], 64, 1, 32, 2),  # four pairs and an odd tile with 96 rows
    ([1 + (i * 53) % 90 for i in range(700)], 0, 1, 4, 1),    # more requests than threads, all short
    ([65 + i % 3 for i in range(600)], 64, 1, 1, 1),      # ... with a prefix of one step
    ([64 * k + d for k in (1, 2, 5) for d in (-1, 0, 1)], 0, 2, 16, 4),  # lengths around the steps
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_shared_prefix_decode(case):
    seq, shared, N, Hq, Hkv = CASES[case]
    w = make_decode(seq, shared if min([n for n in seq if n] or [0]) >= shared else 0, N, Hq, Hkv,
                    seed=case)
    check_decode(run_decode(w, shared=shared), ref_decode(w))


@pytest.mark.parametrize("B,N,Hq,Hkv,shared,own", [
    (1, 1, 16, 16, 0, 45000),      # a lane walks more than 32 steps of one request
    (64, 1, 32, 2, 40000, 100),    # ... and of the prefix, four pairs abreast
    (3, 1, 8, 1, 70001, 333),      # ... and of an odd tile
])
def test_long_runs(B, N, Hq, Hkv, shared, own):
    """Sizes for which the 64-bit reference runs on the GPU too."""
    g = torch.Generator(device=DEV).manual_seed(B)
    seq = torch.randint(max(1, own // 2), own + 1, (B,), generator=g, device=DEV) + shared
    seq[0] = shared + own
    mb = (shared + own + PAGE - 1) // PAGE
    whole = shared // PAGE
    pages = whole + B * (mb - whole)
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.empty((B, mb), dtype=torch.int32, device=DEV)
    table[:, :whole] = perm[:whole]
    table[:, whole:] = perm[whole:].view(B, mb - whole)
    kc, vc = (torch.randn((pages, PAGE, Hkv, D), generator=g, device=DEV).to(torch.bfloat16)
              for _ in range(2))
    if shared % PAGE:
        for c in (kc, vc):
            c[table[:, whole].long(), :shared % PAGE] = c[table[0, whole].long(), :shared % PAGE].clone()
    q = (torch.randn((B * N, Hq, D), generator=g, device=DEV) * D ** -0.5).to(torch.bfloat16)
    w = dict(q=q, kc=kc, vc=vc, table=table, seq=seq.to(torch.int32), N=N, shared=shared)
    ref = [x.cpu() for x in ref_decode(w, DEV)]
    check_decode(run_decode(w), ref)


@pytest.mark.parametrize("short", [1, 5, 63, 64, 65, 300, 579, 639, 640])
@pytest.mark.parametrize("B,N,Hq,Hkv", [(4, 1, 64, 8), (5, 3, 32, 2), (24, 1, 64, 4)])
def test_a_short_request_cuts_the_prefix_not_the_answer(short, B, N, Hq, Hkv):
    # one request holds fewer of the same 640 leading keys than the others: the prefix pass covers
    # the whole steps of its first row, down to none
    w = make_decode([641 + 37 * b for b in range(B)], 640, N, Hq, Hkv, seed=40 + B)
    w["seq"][B // 2] = short
    check_decode(run_decode(w), ref_decode(w))


LONG = [(1, 1, 16, 16, 0, 45000, [0]),           # B, N, Hq, Hkv, shared, own, claims of shared_len
        (64, 1, 32, 2, 40000, 100, [40000, 0]),  # pairs abreast, and the same keys as private ones
        (3, 1, 8, 1, 70001, 333, [70001, 35000, 0]),   # an odd tile
        (16, 4, 32, 4, 20011, 300, [20011]),     # several rows per request: two pairs
        (9, 1, 64, 4, 10007, 5000, [10007])]     # a pair and an odd tile, long private parts
LONG = [(*c[:6], claim) for c in LONG for claim in c[6]]


def long_call(w, q, claim):
    dev = w["kc"].device
    return msa.shared_prefix_decode(q, w["kc"], w["vc"], w["table"], i32(w["lens"]).to(dev),
                                    i32([claim]).to(dev), N=w["N"])


@pytest.mark.parametrize("case", LONG, ids=str)
def test_long_runs_count_every_key_once(case):
    w = lr.counting(*case[:6], DEV)
    lr.check_counting(w, *long_call(w, w["q"], case[6]))


@pytest.mark.parametrize("case", LONG, ids=str)
def test_long_runs_read_every_step_where_it_stands(case):
    w = lr.pointing(*case[:6], DEV)
    for turn in range(lr.turns(w)):
        q, pos = lr.point_at(w, turn, DEV)
        lr.check_pointing(w, pos, *long_call(w, q, case[6]))


@pytest.mark.parametrize("shared", [-3, 0, 63, 64, 100, 511, 512, 1 << 30])
def test_shared_len_changes_the_work_not_the_answer(shared):
    # every request holds 512 shared tokens; any claim up to them (or past every row) must agree
    w = make_decode([512, 513, 600, 1000], 512, 1, 32, 4, seed=5)
    if shared > 512:
        w = make_decode([700] * 3, 700, 1, 32, 4, seed=6)
    check_decode(run_decode(w, shared=shared), ref_decode(w))


def test_large_scores_rescale_the_output():
    # scores of +-150 that keep growing along the keys: the running max moves many times
    w = make_decode([1500, 1100, 1283], 1024, 1, 32, 4, seed=7, scale=20.0)
    ramp = torch.linspace(0.1, 3.0, 12)
    for j in range(11):
        for b in range(3):
            if j < w["table"].shape[1] and (j >= 8 or b == 0):
                w["kc"][w["table"][b, j]] = (w["kc"][w["table"][b, j]].float() * ramp[j]).to(torch.bfloat16)
    check_decode(run_decode(w), ref_decode(w))


def test_rounded_weights_and_output_are_the_only_errors_that_show():
    """RMS of the error of o over RMS of o, on random values. A rounding to bf16 is off by d, uniform in
    [-2^-8, 2^-8] relative to the lower end of its binade at worst: RMS(d) <= 2^-8 / sqrt(3). With
    independent V of mean 0, o = sum w_n v_n and the weights' share sum w_n d_n v_n have variances
    sum w_n^2 and sum w_n^2 d_n^2 times V's, so their ratio is at most 2^-8 / sqrt(3) too; the two
    roundings add as variances: 2^-8 * sqrt(2/3) = 3.19e-3, with 10 % for the samples' spread (rows
    share V, so 4 * 128 channels count as independent: 1 / sqrt(2 * 512) = 3 %, three times). fp32
    sums are below 1e-5."""
    w = make_decode([1700, 1600, 1555], 1500, 1, 32, 4, seed=31)
    o = run_decode(w)[0].double().cpu()
    ref = ref_decode(w)[0]
    rms = ((o - ref).square().mean() / ref.square().mean()).sqrt()
    assert rms <= 2.0 ** -8 * (2 / 3) ** 0.5 * 1.1, float(rms)


def test_runs_agree_bit_for_bit_and_inputs_stay():
    w = make_decode([900 + 13 * i for i in range(40)], 800, 1, 64, 4, seed=8)
    d = {k: x.to(DEV) for k, x in w.items() if isinstance(x, torch.Tensor)}
    copies = {k: x.clone() for k, x in d.items()}
    sl = i32([800]).to(DEV)
    args = (d["q"], d["kc"], d["vc"], d["table"], d["seq"], sl)
    o1, l1 = msa.shared_prefix_decode(*args)
    ws = msa.Workspace()
    nbytes = msa.load().msa_shared_prefix_decode_workspace_size(40, 1, 64, 4)
    buf = ws.get("shared_prefix", nbytes + 4096, DEV)
    buf.fill_(0xff)                                  # scratch of any contents: here, NaN patterns
    out = (torch.full_like(o1, 3.0), torch.full_like(l1, 3.0))
    o2, l2 = msa.shared_prefix_decode(*args, workspace=ws, out=out)
    assert o2.data_ptr() == out[0].data_ptr()
    assert torch.equal(o1.view(torch.int16), o2.view(torch.int16)) and torch.equal(l1, l2)
    assert (buf[nbytes:] == 0xff).all()              # nothing written past the stated size
    o3, l3 = msa.shared_prefix_decode(*args, with_lse=False)
    assert l3 is None and torch.equal(o1.view(torch.int16), o3.view(torch.int16))
    for k, x in d.items():
        assert torch.equal(x.view(torch.int16), copies[k].view(torch.int16))


def test_captured_decode_replays_with_other_lengths_and_two_graphs_overlap():
    cases = [([900, 1000, 640, 777], 640), ([1100, 0, 700, 701], 512), ([64, 65, 66, 67], 64)]
    ws = [make_decode(seq, sh, 1, 32, 4, seed=20 + i) for i, (seq, sh) in enumerate(cases)]
    pages = max(w["kc"].shape[0] for w in ws)
    mb = max(w["table"].shape[1] for w in ws)

    def buffers():
        return dict(q=torch.zeros((4, 32, D), dtype=torch.bfloat16, device=DEV),
                    kc=torch.zeros((pages, PAGE, 4, D), dtype=torch.bfloat16, device=DEV),
                    vc=torch.zeros((pages, PAGE, 4, D), dtype=torch.bfloat16, device=DEV),
                    table=torch.zeros((4, mb), dtype=torch.int32, device=DEV),
                    seq=torch.zeros(4, dtype=torch.int32, device=DEV),
                    sl=torch.zeros(1, dtype=torch.int32, device=DEV))

    def fill(d, w):
        for k in ("q", "kc", "vc", "table", "seq"):
            x = w[k]
            d[k][tuple(slice(0, n) for n in x.shape)] = x.to(DEV)
        d["sl"].fill_(w["shared"])

    sets, graphs, outs = [buffers(), buffers()], [], []
    for d in sets:
        fill(d, ws[0])
        call = lambda: msa.shared_prefix_decode(d["q"], d["kc"], d["vc"], d["table"], d["seq"], d["sl"])
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call())
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for a, b in ((0, 1), (1, 2), (2, 0)):
        fill(sets[0], ws[a])
        fill(sets[1], ws[b])
        torch.cuda.synchronize()
        for _ in range(3):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        check_decode(outs[0], ref_decode(ws[a]))
        check_decode(outs[1], ref_decode(ws[b]))


def test_garbage_in_the_queries_of_padding_requests_reaches_no_other_row():
    for seq, shared, N, Hq, Hkv in (([0, 900, 0, 700, 650, 0] * 9, 600, 1, 8, 1), ([0, 500, 513], 448, 3, 32, 2),
                                    ([300, 0, 417, 0], 0, 2, 16, 4)):
        w = make_decode(seq, shared, N, Hq, Hkv, seed=50)
        clean = run_decode(w)
        check_decode(clean, ref_decode(w))
        pad = (w["seq"] == 0).repeat_interleave(N)
        for junk in (float("nan"), float("inf"), -3e38):
            w["q"][pad] = junk
            o, lse = run_decode(w)
            assert torch.equal(o.view(torch.int16), clean[0].view(torch.int16)) and torch.equal(lse, clean[1])


@pytest.mark.parametrize("case", [
    (3000, 1, 16, 2, 192, 70, 192),       # 94 pairs, more requests than threads
    (2960, 1, 4, 1, 64, 130, 64),         # 46 pairs and an odd tile
    (40, 16, 256, 16, 500, 200, 500),     # every size at its largest
    (16384, 1, 1, 1, 130, 9, 130),        # as many requests as the page tables take
    (2000, 3, 8, 8, 64, 90, 64),
], ids=str)
def test_large_batches(case):
    w = lr.counting(*case[:6], DEV)
    lr.check_counting(w, *long_call(w, w["q"], case[6]))
    if case[0] <= 128:  # codes of 7 bits
        w = lr.pointing(*case[:6], DEV)
        for turn in range(lr.turns(w)):
            q, pos = lr.point_at(w, turn, DEV)
            lr.check_pointing(w, pos, *long_call(w, q, case[6]))


def test_append_on_a_side_stream_in_a_captured_step():
    """The append runs on a second stream beside other work and joins before the attention, eager and
    in a graph: the attention waits for both of the streams that it depends on."""
    w = make_decode([400 + 31 * b for b in range(8)], 320, 1, 32, 4, seed=51)
    ref = ref_decode(w)
    d = {k: w[k].to(DEV) for k in ("q", "kc", "vc", "table", "seq")}
    sl = i32([320]).to(DEV)
    last = torch.stack([w["table"][b, (n - 1) // PAGE] * PAGE + (n - 1) % PAGE
                        for b, n in enumerate(w["seq"].tolist())]).to(torch.int32).to(DEV)
    k, v = (c.view(-1, 4, D)[last.long()].clone() for c in (d["kc"], d["vc"]))
    q_in, big = torch.zeros_like(d["q"]), torch.zeros(1 << 28, dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()

    def spoil():
        for c in (d["kc"], d["vc"]):
            c.view(-1, 4, D)[last.long()] = 7.0
        q_in.fill_(3.0)

    def step():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            big.add_(1)  # some 80 us before the append
            msa.append_kv(k, v, None, last, d["kc"], d["vc"], None)
        q_in.copy_(d["q"])
        main.wait_stream(side)
        return msa.shared_prefix_decode(q_in, d["kc"], d["vc"], d["table"], d["seq"], sl)

    spoil()
    check_decode(step(), ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        spoil()
        graph.replay()
        torch.cuda.synchronize()
        check_decode(out, ref)


def test_threads_that_call_at_once_on_streams_of_their_own():
    import concurrent.futures as cf
    cases = [([900 - 50 * i, 777, 640 + i], 600, 1, 32, 4) for i in range(4)]
    ws = [make_decode(*c, seed=60 + i) for i, c in enumerate(cases)]
    refs = [ref_decode(w) for w in ws]
    rng = np.random.default_rng(3)
    lens = [(rng.integers(0, 200, B), rng.integers(0, 3, B)) for B in (5, 7000, 300, 12000)]

    def work(i):
        w, (prev, new) = ws[i], lens[i]
        with torch.cuda.stream(torch.cuda.Stream()):
            d = {k: x.to(DEV) for k, x in w.items() if isinstance(x, torch.Tensor)}
            sl = i32([600]).to(DEV)
            for _ in range(20):
                o, lse = msa.shared_prefix_decode(d["q"], d["kc"], d["vc"], d["table"], d["seq"], sl)
                table = torch.zeros((len(prev), 3), dtype=torch.int32, device=DEV)
                free = torch.arange(len(prev) * 2, dtype=torch.int32, device=DEV)
                got = msa.build_page_tables(i32(prev).to(DEV), i32(new).to(DEV), table, free, i32([0]).to(DEV),
                                            T=int(new.sum()) + 3, num_pages=1 << 16)
            torch.cuda.current_stream().synchronize()
            return (o, lse), [x.cpu() for x in (table, *got)]

    with cf.ThreadPoolExecutor(4) as ex:
        for i, (out, got) in enumerate(ex.map(work, range(4))):
            check_decode(out, refs[i])
            prev, new = lens[i]
            want = ref_tables(prev, new, np.zeros((len(prev), 3), dtype=np.int32), np.arange(len(prev) * 2), 0,
                              int(new.sum()) + 3)
            for g, x in zip(got, (*want[:5], [want[5]]), strict=True):
                assert np.array_equal(g.numpy(), np.asarray(x, dtype=np.int32))


FRESH = """
import sys
sys.path[:0] = [sys.argv[1], sys.argv[1] + "/tests"]
import test_gpu_serving_batch as t, torch, block_sparse_attention_msa_gb300 as msa
w = t.make_decode([300, 400], 256, 1, 16, 2, seed=1)
d = {k: x.cuda() for k, x in w.items() if isinstance(x, torch.Tensor)}
z = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")
sl, prev, new, table, free, used = z(1) + 256, z(7000) + 5, z(7000) + 1, z((7000, 2)), z(9), z(1)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    seq = msa.build_page_tables(prev, new, table, free, used, T=7000, num_pages=9)[0]
    out = msa.shared_prefix_decode(d["q"], d["kc"], d["vc"], d["table"], d["seq"], sl)
g.replay()
torch.cuda.synchronize()
assert (seq == 6).all() and msa.device_error() == 0
t.check_decode(out, t.ref_decode(w))
"""


def test_the_first_call_of_a_process_can_be_a_captured_one():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FRESH, root], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("seq,shared,N,Hq,Hkv", [
    ([300, 421, 515, 260], 256, 4, 32, 4), ([130, 129, 143, 144, 128], 64, 16, 64, 4),
    ([3, 2, 1, 70, 5], 0, 6, 8, 2), ([1030 + i for i in range(40)], 1024, 2, 64, 4),
    ([64, 65, 66, 67, 68], 0, 5, 16, 1),
])
@pytest.mark.parametrize("what", ["v", "k"])
def test_non_finite_later_tokens_reach_no_earlier_row(seq, shared, N, Hq, Hkv, what):
    """Token j of the last N holds NaN or infinity: rows at its position and behind it show it, rows
    before it are what they are without."""
    w = make_decode(seq, shared, N, Hq, Hkv, seed=70 + N)
    clean = ref_decode(w)
    for back, junk in ((0, float("nan")), (N // 2, float("inf")), (N - 2, float("-inf"))):
        bad = dict(w, kc=w["kc"].clone(), vc=w["vc"].clone())
        sees = torch.zeros(len(seq) * N, dtype=torch.bool)
        for b, n in enumerate(seq):
            at = n - 1 - back
            if at < 0 or b % 3 == 2:  # some requests have nothing of the kind
                continue
            bad[what + "c"][w["table"][b, at // PAGE], at % PAGE] = junk
            sees[b * N + N - 1 - back:(b + 1) * N] = True
        o, lse = run_decode(bad)
        check_decode((o[~sees.to(DEV)], lse[~sees.to(DEV)]), [x[~sees] for x in clean])
        seen = o.cpu()[sees]
        if what == "v":
            assert not torch.isfinite(seen).any()
            assert torch.equal(torch.isfinite(lse.cpu()), torch.isfinite(clean[1]))
        elif back == 0:
            assert torch.isnan(seen).all()


def test_out_of_range_page_reads_page_zero():
    w = make_decode([300, 520], 256, 1, 16, 2, seed=9)
    bad = dict(w, table=w["table"].clone())
    bad["table"][1, 3] = w["kc"].shape[0] + 5
    bad["table"][0, 2] = -1
    ref = dict(w, table=w["table"].clone())
    ref["table"][1, 3] = 0
    ref["table"][0, 2] = 0
    for c in ("kc", "vc"):
        ref[c] = torch.nan_to_num(w[c], nan=0.25)
        bad[c] = ref[c]
    got = run_decode(bad)
    assert msa.device_error() == BAD_PAGE
    check_decode(got, ref_decode(ref))


def test_length_past_the_table_is_clamped():
    w = make_decode([256, 384], 128, 1, 16, 2, seed=10)
    bad = dict(w, seq=i32([256, 5000]))
    got = run_decode(bad)
    assert msa.device_error() == BAD_LEN
    check_decode(got, ref_decode(w))


# ------------------------------------------------------------------------------ together

def test_steps_of_a_batch_behind_a_cached_prompt():
    """Prompt once, then admission on its pages, chunks and decode steps: tables, append and the
    shared decode against attention over the tokens kept on the host; the sparse path reads the
    same caches (with every block selected it equals the dense answer)."""
    g = torch.Generator(device=DEV).manual_seed(3)
    Hq, Hkv, Di, B, P, mb = 16, 2, 64, 5, 64, 12
    rnd = lambda *s: torch.randn(s, generator=g, device=DEV).to(torch.bfloat16)
    kc, vc = (torch.full((P, PAGE, Hkv, D), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    xc = torch.zeros((P, PAGE, Hkv, Di), dtype=torch.bfloat16, device=DEV)
    free = torch.randperm(P, generator=g, device=DEV).to(torch.int32)
    used = torch.zeros(1, dtype=torch.int32, device=DEV)
    # the prompt: 384 tokens of one request
    t0 = torch.zeros((1, mb), dtype=torch.int32, device=DEV)
    n = 384
    pk, pv, px = rnd(n, Hkv, D), rnd(n, Hkv, D), rnd(n, Hkv, Di)
    _, _, slots, _, used = msa.build_page_tables(i32([0]).to(DEV), i32([n]).to(DEV), t0, free, used,
                                                 T=n, num_pages=P)
    msa.append_kv(pk, pv, px, slots, kc, vc, xc)
    shared_pages = t0[0, :3].clone()
    # five requests behind it; the last is a padding row
    table = torch.zeros((B, mb), dtype=torch.int32, device=DEV)
    lens = i32([n, n, n, n, 0]).to(DEV)
    hist = [[pk.cpu()] for _ in range(4)], [[pv.cpu()] for _ in range(4)]
    for step, new in enumerate(([200, 1, 130, 64, 0], [1, 1, 1, 1, 0], [1, 1, 1, 1, 0], [3, 3, 3, 3, 0])):
        T = sum(new) + 6
        k, v, x = rnd(T, Hkv, D), rnd(T, Hkv, D), rnd(T, Hkv, Di)
        lens, cu, slots, _, used = msa.build_page_tables(
            lens, i32(new).to(DEV), table, free, used, T=T, num_pages=P,
            shared_pages=shared_pages if step == 0 else None)
        msa.append_kv(k, v, x, slots, kc, vc, xc)
        at = 0
        for b in range(4):
            hist[0][b].append(k[at:at + new[b]].cpu())
            hist[1][b].append(v[at:at + new[b]].cpu())
            at += new[b]
        assert lens.tolist() == [sum(len(c) for c in hist[0][b]) for b in range(4)] + [0]
        N = 1 if step < 3 else 3
        q = (rnd(B * N, Hq, D).float() * D ** -0.5).to(torch.bfloat16)
        got = msa.shared_prefix_decode(q, kc, vc, table, lens, i32([n]).to(DEV), N=N)
        # the same keys as a contiguous one-request-per-page-run cache on the host
        flat = dict(q=q.cpu(), seq=lens.cpu(), N=N,
                    table=torch.arange(B * mb, dtype=torch.int32).view(B, mb),
                    kc=torch.zeros((B * mb, PAGE, Hkv, D), dtype=torch.bfloat16),
                    vc=torch.zeros((B * mb, PAGE, Hkv, D), dtype=torch.bfloat16))
        for c, h in zip(("kc", "vc"), hist):
            for b in range(4):
                rows = torch.cat(h[b])
                flat[c].view(B, mb * PAGE, Hkv, D)[b, :len(rows)] = rows
        ref = ref_decode(flat)
        check_decode(got, ref)
        if N == 1:  # the sparse path over every block of the same caches
            qi = rnd(4, Hkv, Di)
            ids, _ = msa.index_score_topk(qi, xc, table[:4].contiguous(), lens[:4].contiguous(), N=1, topk=mb)
            fpt, kl = msa.build_sparse_page_table(ids, table[:4].contiguous(), lens[:4].contiguous(), N=1,
                                                  num_pages=P)
            o, lse = msa.paged_sparse_decode(q[:4].contiguous(), torch.nan_to_num(kc), torch.nan_to_num(vc),
                                             fpt, kl)
            check = [r[:4] for r in ref]
            assert (lse.double().cpu() - check[1]).abs().max() <= 1e-3
            assert (o.double().cpu() - check[0]).abs().max() <= 2e-2


def test_a_whole_step_captured_with_copies_around_it_equals_the_eager_step():
    """Copies, tables, append, decode and copies in one graph, replayed over several steps: each
    kernel waits for what precedes it, copies included, and leaves what the eager step leaves."""
    Hq, Hkv, Di, B, P, mb, T, n = 32, 4, 64, 6, 96, 12, 64, 640
    g = torch.Generator(device=DEV).manual_seed(4)
    rnd = lambda *s: torch.randn(s, generator=g, device=DEV).to(torch.bfloat16)
    prompt = rnd(P, PAGE, Hkv, D), rnd(P, PAGE, Hkv, D)
    free = torch.randperm(P, generator=g, device=DEV).to(torch.int32)
    zeros = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)

    def state():
        d = dict(lens=zeros(B), used=zeros(1), table=zeros(B, mb), new=zeros(B), sl=zeros(1),
                 kc=prompt[0].clone(), vc=prompt[1].clone(),
                 xc=torch.zeros((P, PAGE, Hkv, Di), dtype=torch.bfloat16, device=DEV))
        d["table"][:, :n // PAGE] = free[:n // PAGE]
        d["lens"].fill_(n)
        d["used"].fill_(n // PAGE)
        d["sl"].fill_(n)
        for k, s in (("k", (T, Hkv, D)), ("v", (T, Hkv, D)), ("x", (T, Hkv, Di)), ("q", (B, Hq, D))):
            d[k] = torch.zeros(s, dtype=torch.bfloat16, device=DEV)
        return d

    given = {k: torch.zeros_like(x) for k, x in state().items() if k in ("new", "k", "v", "x", "q")}

    def step(d):
        for k, x in given.items():
            d[k].copy_(x)
        seq, _, slots, _, used = msa.build_page_tables(d["lens"], d["new"], d["table"], free, d["used"], T=T,
                                                       num_pages=P)
        msa.append_kv(d["k"], d["v"], d["x"], slots, d["kc"], d["vc"], d["xc"])
        o, lse = msa.shared_prefix_decode(d["q"], d["kc"], d["vc"], d["table"], seq, d["sl"])
        d["lens"].copy_(seq)
        d["used"].copy_(used)
        again, _ = msa.shared_prefix_decode(d["q"], d["kc"], d["vc"], d["table"], seq, d["sl"])
        return o, lse, again

    eager, captured = state(), state()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(captured)
    for new in ([1, 2, 3, 4, 5, 0], [10] * 6, [1] * 6, [0, 60, 0, 0, 0, 1]):
        given["new"].copy_(i32(new))
        for k in ("k", "v", "x", "q"):
            given[k].copy_(rnd(*given[k].shape) * (0.1 if k == "q" else 1.0))
        graph.replay()
        want = step(eager)
        torch.cuda.synchronize()
        for a, b in zip((*out, *captured.values()), (*want, *eager.values()), strict=True):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
        assert torch.equal(out[0], out[2])
        assert torch.isfinite(out[1]).all() and captured["lens"].tolist() == eager["lens"].tolist()
