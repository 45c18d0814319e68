"""GPU tests of ``chunk_attention`` against plain 64-bit attention written here, and of a run of steps
with the page tables and the append around it.

Tolerance, per output element, from the roundings the kernel makes (w the exact softmax weights,
A = sum_n w_n |v_n|, ref the exact output):
  * P = 2^(s - m) is rounded to bf16 for its product: at most 2^-8 of each term, 2^-8 A in all;
  * o is rounded to bf16 once: 2^-8 of the value;
  * a score is an fp32 sum of 128 exact products of bf16 numbers, at most 2^-23 of sum |q_d k_d| per
    addition (truncating adds counted), then scaled to log2 units: ds = 2^-23 * 128 * max_n
    sum_d |q_d k_nd| + 2^-21 * max |s|, which moves weights by at most 2 ds A;
  * 2^x, the fp32 sums of P V and l and the joins: 2^-21 + n * 2^-24 per key count n, of A.
LSE: ds + 2^-21 + n * 2^-24 absolute, + 2^-23 of the value.
"""
import concurrent.futures as cf

import numpy as np
import pytest
import torch

import block_sparse_attention_msa_gb300 as msa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
PAGE = 128
D = 128
BAD_PAGE, BAD_LEN = 1, 2
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_sparse_attention_msa_gb300 import build
    build.build()
    msa.load()
    assert msa.device_error() == 0  # nothing left over from earlier tests


@pytest.fixture(autouse=True)
def no_error_left():
    yield
    assert msa.device_error() == 0  # a wait that ran out shows in its own test


def i32(x):
    return torch.from_numpy(np.array(x, dtype=np.int32))


def make(new, held, Hq, Hkv, seed, pad=0, scale=1.0):
    """Requests of `held` tokens before their `new` ones; cells that nothing uses are NaN, and so are
    the queries of padding rows."""
    g = torch.Generator().manual_seed(seed)
    seq = [h + n for h, n in zip(held, new)]
    blocks = [(s + PAGE - 1) // PAGE for s in seq]
    mb, pages = max(1, max(blocks)) + 1, sum(blocks) + 2
    perm = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.randint(0, pages, (len(new), mb), generator=g).to(torch.int32)  # unused entries: any page
    kc = torch.full((pages, PAGE, Hkv, D), NAN, dtype=torch.bfloat16)
    vc = kc.clone()
    used = 0
    for b, s in enumerate(seq):
        table[b, :blocks[b]] = perm[used:used + blocks[b]]
        used += blocks[b]
        for c, f in ((kc, scale), (vc, 1.0)):
            rows = torch.full((blocks[b] * PAGE, Hkv, D), NAN, dtype=torch.bfloat16)
            rows[:s] = (torch.randn((s, Hkv, D), generator=g) * f).to(torch.bfloat16)
            c[table[b, :blocks[b]].long()] = rows.view(-1, PAGE, Hkv, D)
    cu = np.concatenate([[0], np.cumsum(new)])
    T = int(cu[-1]) + pad
    q = torch.full((T, Hq, D), NAN, dtype=torch.bfloat16)
    q[:cu[-1]] = (torch.randn((int(cu[-1]), Hq, D), generator=g) * D ** -0.5).to(torch.bfloat16)
    return dict(q=q, kc=kc, vc=vc, table=table, seq=i32(seq), cu=i32(cu))


def reference(w, device="cpu"):
    """o, lse, and their tolerances (module docstring), in 64 bits, for the rows of requests."""
    w = {k: x.to(device) for k, x in w.items()}
    q = w["q"].double()
    T, Hq, _ = q.shape
    Hkv = w["kc"].shape[2]
    G = Hq // Hkv
    o = torch.zeros((T, Hq, D), dtype=torch.float64, device=device)
    lse = torch.full((T, Hq), float("-inf"), dtype=torch.float64, device=device)
    to, tl = torch.zeros_like(o), torch.zeros_like(lse)
    cu = w["cu"].tolist()
    for b, s_len in enumerate(w["seq"].tolist()):
        n = cu[b + 1] - cu[b]
        pages = w["table"][b, :(s_len + PAGE - 1) // PAGE].long()
        k = w["kc"][pages].flatten(0, 1)[:s_len].double().transpose(0, 1)      # [Hkv, s, D]
        v = w["vc"][pages].flatten(0, 1)[:s_len].double().transpose(0, 1)
        for i0 in range(0, n, 64):
            m = min(64, n - i0)
            r = slice(cu[b] + i0, cu[b] + i0 + m)
            vis = s_len - n + i0 + m
            if vis <= 0:
                continue
            qi = q[r].view(m, Hkv, G, D).permute(1, 0, 2, 3).reshape(Hkv, m * G, D)
            pos = (s_len - n + i0 + torch.arange(m, device=device)).repeat_interleave(G)[:, None]
            seen = torch.arange(vis, device=device)[None] <= pos                 # [m*G, vis]
            s = (qi @ k[:, :vis].transpose(1, 2)).masked_fill(~seen, float("-inf"))
            z = torch.logsumexp(s, -1, keepdim=True)
            p = torch.where(torch.isneginf(z), 0.0, torch.exp(s - z))
            vv = v[:, :vis].nan_to_num(0.0, 0.0, 0.0) if not torch.isfinite(v).all() else v[:, :vis]
            ref, A = p @ vv, p @ vv.abs()
            dots = (qi.abs() @ k[:, :vis].abs().transpose(1, 2)).masked_fill(~seen, 0).amax(-1, keepdim=True)
            top = s.abs().masked_fill(~seen, 0).amax(-1, keepdim=True)
            ds = 2.0 ** -23 * 128 * dots + 2.0 ** -21 * top
            acc = 2.0 ** -21 + (pos + 1).clamp(min=0) * 2.0 ** -24
            back = lambda x: x.view(Hkv, m, G, -1).permute(1, 0, 2, 3).reshape(m, Hq, -1)
            o[r], lse[r] = back(ref), back(z).squeeze(-1)
            to[r] = back(2.0 ** -8 * (ref.abs() + A) * (1 + 2.0 ** -7) + (2 * ds + acc) * A)
            tl[r] = back(ds + acc + 2.0 ** -23 * z.abs()).squeeze(-1)
    return o, lse, to, tl


def run(w, **kw):
    d = {k: x.to(DEV) for k, x in w.items()}
    return msa.chunk_attention(d["q"], d["kc"], d["vc"], d["table"], d["seq"], d["cu"], **kw)


def check(got, ref, rows=None):
    o, lse, to, tl = (x.cpu() for x in ref)
    go, gl = got[0].double().cpu(), got[1].double().cpu()
    rows = slice(0, go.shape[0]) if rows is None else rows
    o, lse, to, tl, go, gl = (x[rows] for x in (o, lse, to, tl, go, gl))
    err = (go - o).abs()
    assert (err <= to).all(), f"o: worst error / tolerance {(err / to.clamp_min(1e-300)).max():.3f}"
    empty = torch.isneginf(lse)
    assert torch.equal(torch.isneginf(gl), empty)
    assert (go[empty] == 0).all()
    err = (gl - lse).abs()[~empty]
    assert (err <= tl[~empty]).all(), f"lse: worst error / tolerance {(err / tl[~empty]).max():.3f}"


CASES = [
    # new tokens, tokens held before, Hq, Hkv
    ([1], [0], 1, 1),                              # one token in all
    ([1], [2047], 8, 2),                           # one decode row
    ([1], [63], 8, 1), ([1], [64], 8, 1), ([1], [127], 8, 1),    # lengths around steps and pages
    ([1, 1, 1, 1], [5, 700, 0, 64], 16, 4),        # decode rows
    ([16], [0], 64, 8), ([17], [0], 64, 8), ([32], [0], 64, 8), ([33], [100], 64, 8),   # around a tile, a pair
    ([48], [0], 32, 4), ([129], [0], 4, 4), ([256], [31], 2, 2), ([257], [0], 1, 1),    # G 8, 1, 1, 1
    ([8, 9, 16, 17], [3, 0, 61, 200], 32, 2),      # G 16
    ([300], [0], 8, 2), ([300], [777], 16, 8),     # a prompt, a chunk behind a prefix; G 4, 2
    ([0, 5, 0, 1, 130, 0, 64, 1], [9, 0, 0, 300, 64, 0, 500, 0], 16, 2),    # mixed, requests without tokens
    ([1] * 40 + [70, 3], [11 * i for i in range(42)], 8, 8),     # decode rows, G 1, with a chunk
    ([2, 1, 3], [700, 1500, 90], 4, 1),            # one group: the lanes halve the keys
    ([150], [2900], 16, 1), ([1] * 9, [37 * i for i in range(9)], 1, 1),
    ([1 + i % 5 for i in range(300)], [(i * 29) % 250 for i in range(300)], 4, 2),    # many requests
    ([1] * 1500, [i % 70 for i in range(1500)], 2, 2),       # more than the plan's threads
    ([700, 1, 2], [1300, 4000, 64], 64, 8),        # long enough to be cut
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_64_bits(case):
    new, held, Hq, Hkv = CASES[case]
    w = make(new, held, Hq, Hkv, seed=case, pad=case % 4)
    check(run(w), reference(w), slice(0, sum(new)))


@pytest.mark.parametrize("new,held,Hq,Hkv", [
    ([1, 1], [40000, 33], 16, 4),     # a long cache cut over every CTA, more than 32 steps a run
    ([1], [50001], 1, 1),             # ... in halves
    ([2000], [3000], 16, 4),          # many pairs, the last of them cut
    ([1100, 900, 1, 1], [0, 6000, 9000, 1], 32, 2),
])
def test_long(new, held, Hq, Hkv):
    w = make(new, held, Hq, Hkv, seed=len(new))
    check(run(w), reference(w, DEV))


@pytest.mark.parametrize("new", [1, 2, 5, 9, 16, 23])
@pytest.mark.parametrize("pad", [0, 1 << 14])
def test_a_tile_in_any_number_of_pieces(new, pad):
    """Tiles of 8 to 128 rows (and a pair) whose keys are cut into few, several and many pieces, by calls
    that cut equal runs and by calls that list their work (many
    padding rows)."""
    Hq, Hkv = 16, 2
    for held in (64, 190, 330, 500, 640, 1000, 1500, 2600):
        w = make([new], [held], Hq, Hkv, seed=held + new)
        ref = reference(w, DEV)
        if pad:
            w["q"] = torch.cat([w["q"], torch.zeros((pad, Hq, D), dtype=torch.bfloat16)])
        o, lse = run(w)
        check((o[:new], lse[:new]), ref)


@pytest.mark.parametrize("Hq,Hkv", [(32, 4), (16, 1)])
@pytest.mark.parametrize("pad", [0, 1 << 17])
def test_units_of_all_kinds_in_turn_from_caches_beyond_l2(Hq, Hkv, pad):
    """Decode rows, short chunks and long ones alternate, so that slots of K and V change between lanes
    that share steps and lanes that do not, while loads take long (some 300 MB of cache). With many
    padding rows the call is one that lists its work, else one that cuts it into equal runs."""
    g = np.random.default_rng(Hq)
    B = 48
    new = [int(x) for x in g.choice([1, 1, 1, 3, 17, 40, 75], B)]
    held = [int(x) for x in g.integers(0, 26000 // Hkv, B)]
    w = make(new, held, Hq, Hkv, seed=90 + Hq, pad=0)
    ref = reference(w, DEV)
    if pad:
        w["q"] = torch.cat([w["q"], torch.zeros((pad, Hq, D), dtype=torch.bfloat16)])
    for _ in range(3):
        o, lse = run(w)
        check((o[:sum(new)], lse[:sum(new)]), ref)


def test_large_scores_rescale_the_output():
    # scores that grow along the keys: the softmax's reference has to move many times
    w = make([40, 1], [600, 900], 16, 2, seed=3, scale=30.0)
    for b, n in enumerate(w["seq"].tolist()):
        for j in range((n + PAGE - 1) // PAGE):
            f = torch.linspace(0.02 + 0.15 * j, 0.17 + 0.15 * j, PAGE)[:, None, None]
            w["kc"][w["table"][b, j]] = (w["kc"][w["table"][b, j]].float() * f).to(torch.bfloat16)
    check(run(w), reference(w))


@pytest.mark.parametrize("scores", ["-inf", "lowest"])
def test_rows_whose_scores_are_extreme(scores):
    # -inf scores leave no weight; scores at fp32's end keep finite weights
    w = make([5, 1], [100, 70], 8, 2, seed=4)
    if scores == "-inf":
        w["q"][2] = 1.0
        cells = w["table"][0, :1].long()
        w["kc"][cells, :, 1] = torch.where(torch.isnan(w["kc"][cells, :, 1]), NAN, float("-inf")).to(torch.bfloat16)
        o, lse = run(w)
        heads = slice(4, 8)  # of group 1
        assert (o[2, heads] == 0).all() and torch.isneginf(lse[2, heads]).all()
        assert torch.isfinite(o[2, :4].float()).all()
        check((o[5:6], lse[5:6]), [x[5:6] for x in reference(w)])
    else:
        w["kc"] = torch.where(torch.isnan(w["kc"]), w["kc"], torch.tensor(-1e30, dtype=torch.bfloat16))
        w["q"] = torch.ones_like(w["q"])
        o, lse = run(w)    # equal scores: the mean of V
        for t, (b, vis) in enumerate([(0, 101 + i) for i in range(5)] + [(1, 71)]):
            pages = w["table"][b, :1].long()
            mean = w["vc"][pages].flatten(0, 1)[:vis].double().mean(0).repeat_interleave(4, 0)
            assert (o[t].double().cpu() - mean).abs().max() <= 2.0 ** -8 * 2
        assert (lse < -1e31).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("new,held,Hq,Hkv", [
    ([40, 1, 17], [60, 500, 0], 64, 8), ([300], [33], 4, 4), ([130, 20], [1000, 128], 16, 1),
    ([6, 6], [0, 61], 8, 8),
])
@pytest.mark.parametrize("what", ["v", "k"])
def test_non_finite_later_tokens_reach_no_earlier_row(new, held, Hq, Hkv, what):
    """A new token holds NaN or infinity: rows at its position and behind it show it, rows before it are
    what they are without."""
    w = make(new, held, Hq, Hkv, seed=70 + Hkv)
    clean = reference(w)
    cu = w["cu"].tolist()
    for at, junk in ((0.99, NAN), (0.5, float("inf")), (0.2, float("-inf"))):
        bad = dict(w, kc=w["kc"].clone(), vc=w["vc"].clone())
        sees = torch.zeros(sum(new), dtype=torch.bool)
        for b, n in enumerate(new):
            i = int(at * n)
            pos = held[b] + i
            bad[what + "c"][w["table"][b, pos // PAGE], pos % PAGE] = junk
            sees[cu[b] + i:cu[b + 1]] = True
        o, lse = run(bad)
        if (~sees).any():
            check((o[~sees.to(DEV)], lse[~sees.to(DEV)]), [x[~sees] for x in clean])
        seen = o.cpu()[sees]
        if what == "v":
            assert not torch.isfinite(seen).any()
            assert torch.equal(torch.isfinite(lse.cpu()), torch.isfinite(clean[1]))
        elif junk != junk:
            assert torch.isnan(seen).all()


def test_padding_rows_and_outputs_of_other_callers_are_left_alone():
    w = make([3, 40, 1], [200, 0, 77], 32, 4, seed=8, pad=21)
    d = {k: x.to(DEV) for k, x in w.items()}
    copies = {k: x.clone() for k, x in d.items()}
    args = (d["q"], d["kc"], d["vc"], d["table"], d["seq"], d["cu"])
    T = d["q"].shape[0]
    live = slice(0, 44)
    ws = msa.Workspace()
    nbytes = msa.load().msa_chunk_attention_workspace_size(3, T, 32, 4, w["table"].shape[1])
    buf = ws.get("chunk", nbytes + 4096, DEV)
    buf.fill_(0xff)                                   # scratch of any contents: here, NaN patterns
    out = (torch.full((T, 32, D), 3.0, dtype=torch.bfloat16, device=DEV), torch.full((T, 32), 5.0, device=DEV))
    o, lse = msa.chunk_attention(*args, workspace=ws, out=out)
    assert o is out[0] and lse is out[1]
    check((o, lse), reference(w), live)
    assert (o[44:] == 3).all() and (lse[44:] == 5).all()
    assert (buf[nbytes:] == 0xff).all()               # nothing written past the stated size
    for _ in range(3):                                # runs agree bit for bit
        o2, none = msa.chunk_attention(*args, with_lse=False)
        assert none is None and torch.equal(o2[live].view(torch.int16), o[live].view(torch.int16))
    for k, x in d.items():
        assert torch.equal(x.view(torch.int16), copies[k].view(torch.int16))


def test_queries_of_a_fused_projection():
    w = make([70, 1, 9], [100, 333, 0], 16, 4, seed=9)
    d = {k: x.to(DEV) for k, x in w.items()}
    T = d["q"].shape[0]
    qkv = torch.full((T, (16 + 2 * 4) * D), NAN, dtype=torch.bfloat16, device=DEV)
    q = qkv[:, :16 * D].unflatten(1, (16, D))
    q.copy_(d["q"])
    check(msa.chunk_attention(q, d["kc"], d["vc"], d["table"], d["seq"], d["cu"]), reference(w))


def test_rows_at_negative_positions_and_lengths_out_of_range():
    w = make([20, 3], [40, 100], 16, 2, seed=10)
    w["seq"][0] = 8                                   # 20 new tokens of a request of 8: 12 rows see nothing
    o, lse = run(w)
    assert msa.device_error() == BAD_LEN
    check((o, lse), reference(w))
    w = make([20, 3], [40, 100], 16, 2, seed=10)
    w["seq"][1] = w["table"].shape[1] * PAGE + 1000   # past the table: clamped to it
    w["kc"], w["vc"] = w["kc"].nan_to_num(0.25), w["vc"].nan_to_num(0.5)
    got = run(w)
    assert msa.device_error() == BAD_LEN
    w["seq"][1] = w["table"].shape[1] * PAGE
    check(got, reference(w))


@pytest.mark.parametrize("cu", [[0, 24, 10, 30], [5, 3, 3, 30], [-4, 2, 2, 2], [0, 8, 30, 41], [0, 30, 0, 30]])
def test_token_ranges_out_of_order_end_with_an_error(cu):
    # what the rows hold then is not defined; nothing outside the outputs is written, and the next call is right
    w = make([8, 2, 20], [50, 9, 300], 16, 2, seed=12)
    bad = dict(w, cu=i32(cu))
    run(bad)
    assert msa.device_error() == BAD_LEN
    check(run(w), reference(w))


def test_out_of_range_page_reads_page_zero():
    w = make([4, 1], [300, 140], 16, 2, seed=11)
    w["kc"], w["vc"] = w["kc"].nan_to_num(0.0), w["vc"].nan_to_num(0.0)
    w["table"][0, 1], w["table"][1, 0] = w["kc"].shape[0], -3
    got = run(w)
    assert msa.device_error() == BAD_PAGE
    w["table"][0, 1] = w["table"][1, 0] = 0
    check(got, reference(w))


def test_empty_calls():
    w = make([2], [5], 8, 2, seed=13)
    d = {k: x.to(DEV) for k, x in w.items()}
    o, lse = msa.chunk_attention(d["q"][:0], d["kc"], d["vc"], d["table"], d["seq"], i32([0, 0]).to(DEV))
    assert o.shape == (0, 8, D) and lse.shape == (0, 8)
    out = (torch.ones_like(d["q"]), torch.ones((2, 8), device=DEV))
    msa.chunk_attention(d["q"], d["kc"], d["vc"], d["table"], d["seq"], i32([0, 0]).to(DEV), out=out)
    assert (out[0] == 1).all() and (out[1] == 1).all()


def test_captured_call_replays_with_other_lengths_and_two_graphs_overlap():
    T, B, Hq, Hkv = 150, 4, 32, 4
    cases = [([100, 1, 1, 30], [0, 900, 33, 600]), ([1, 1, 1, 1], [700, 20, 1, 64]), ([0, 140, 10, 0], [5, 300, 0, 9])]
    ws = [make(n, h, Hq, Hkv, seed=20 + i, pad=T - sum(n)) for i, (n, h) in enumerate(cases)]
    refs = [reference(w) for w in ws]
    pages, mb = max(w["kc"].shape[0] for w in ws), max(w["table"].shape[1] for w in ws)

    def buffers():
        z = lambda *s, dtype=torch.int32: torch.zeros(s, dtype=dtype, device=DEV)
        bf = torch.bfloat16
        return dict(q=z(T, Hq, D, dtype=bf), kc=z(pages, PAGE, Hkv, D, dtype=bf), vc=z(pages, PAGE, Hkv, D, dtype=bf),
                    table=z(B, mb), seq=z(B), cu=z(B + 1))

    def fill(d, w):
        for k, x in w.items():
            d[k][tuple(slice(0, n) for n in x.shape)] = x.to(DEV)

    sets, graphs, outs = [buffers(), buffers()], [], []
    for d in sets:
        fill(d, ws[0])
        call = lambda: msa.chunk_attention(d["q"], d["kc"], d["vc"], d["table"], d["seq"], d["cu"])
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
        check(outs[0], refs[a], slice(0, sum(cases[a][0])))
        check(outs[1], refs[b], slice(0, sum(cases[b][0])))


def test_threads_that_call_at_once_on_streams_of_their_own():
    cases = [([90 + i, 1, 1], [300, 777, 40 + i]) for i in range(4)]
    ws = [make(*c, 32, 4, seed=60 + i) for i, c in enumerate(cases)]
    refs = [reference(w) for w in ws]

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            d = {k: x.to(DEV) for k, x in ws[i].items()}
            for _ in range(20):
                got = msa.chunk_attention(d["q"], d["kc"], d["vc"], d["table"], d["seq"], d["cu"])
            torch.cuda.current_stream().synchronize()
            return got

    with cf.ThreadPoolExecutor(4) as ex:
        for i, got in enumerate(ex.map(work, range(4))):
            check(got, refs[i])


def test_equals_the_shared_prefix_decode_and_the_sparse_prefill_that_selects_everything():
    # two other entry points of the library that compute the same where their ranges meet
    w = make([3] * 5, [200, 61, 500, 7, 129], 16, 4, seed=14)
    ref = reference(w)
    d = {k: x.to(DEV) for k, x in w.items()}
    check(msa.shared_prefix_decode(d["q"], d["kc"], d["vc"], d["table"], d["seq"],
                                   torch.zeros(1, dtype=torch.int32, device=DEV), N=3), ref)
    check(run(w), ref)
    w = make([500], [0], 16, 4, seed=15)
    d = {k: x.to(DEV) for k, x in w.items()}
    ids = torch.where(torch.arange(4)[None] <= torch.arange(500)[:, None] // PAGE, torch.arange(4)[None], -1)
    ids = ids[:, None].expand(-1, 4, -1).to(torch.int32).contiguous().to(DEV)
    o, lse = msa.sparse_prefill_paged(d["q"], d["kc"].nan_to_num(0.0), d["vc"].nan_to_num(0.0),
                                      d["table"][0, :4].contiguous(), ids, 500)
    o2, lse2 = run(w)
    # both are bf16 roundings of the same numbers, with weights rounded to bf16 before: 2 * (2^-8 + 2^-8) A
    assert (o.float() - o2.float()).abs().max() <= 4 * 2.0 ** -8 * 4.5
    assert (lse - lse2).abs().max() <= 1e-4


def test_steps_of_a_scheduler():
    """Page tables, append and attention over several steps: prompts in chunks, then decode rows, and
    requests that pause, against attention over everything appended so far."""
    g = torch.Generator().manual_seed(5)
    B, Hq, Hkv, mb, T = 4, 16, 2, 8, 200
    P = B * mb
    bf = torch.bfloat16
    kc = torch.full((P, PAGE, Hkv, D), NAN, dtype=bf, device=DEV)
    vc = torch.full_like(kc, NAN)
    table = torch.full((B, mb), -1, dtype=torch.int32, device=DEV)
    free = torch.randperm(P, generator=g).to(torch.int32).to(DEV)
    used = torch.zeros(1, dtype=torch.int32, device=DEV)
    prev = torch.zeros(B, dtype=torch.int32, device=DEV)
    for new in ([100, 0, 60, 1], [90, 70, 0, 1], [1, 64, 1, 1], [1, 1, 1, 0], [0, 1, 130, 1]):
        n = sum(new)
        q = (torch.randn((T, Hq, D), generator=g) * D ** -0.5).to(bf).to(DEV)
        k, v = (torch.randn((T, Hkv, D), generator=g).to(bf).to(DEV) for _ in range(2))
        seq, cu, slots, _, used = msa.build_page_tables(prev, i32(new).to(DEV), table, free, used, T=T, num_pages=P)
        msa.append_kv(k, v, None, slots, kc, vc, None)
        got = msa.chunk_attention(q, kc, vc, table, seq, cu)
        w = dict(q=q, kc=kc, vc=vc, table=table.clamp(min=0), seq=seq, cu=cu)
        check(got, reference({a: x.cpu() for a, x in w.items()}), slice(0, n))
        prev = seq


FRESH = """
import sys
sys.path[:0] = [sys.argv[1], sys.argv[1] + "/tests"]
import test_gpu_chunk_attention as t, torch, block_sparse_attention_msa_gb300 as msa
for new, held in (([5, 1, 40], [300, 77, 0]), ([900], [100])):
    w = t.make(new, held, 64, 8, seed=1)
    d = {k: x.cuda() for k, x in w.items()}
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = msa.chunk_attention(d["q"], d["kc"], d["vc"], d["table"], d["seq"], d["cu"])
    g.replay()
    torch.cuda.synchronize()
    assert msa.device_error() == 0
    t.check(out, t.reference(w))
"""


def test_the_first_call_of_a_process_can_be_a_captured_one():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FRESH, root], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_refusals():
    w = make([3, 1], [10, 5], 8, 2, seed=1)
    d = {k: x.to(DEV) for k, x in w.items()}
    names = ("q", "kc", "vc", "table", "seq", "cu")

    def call(out=None, **kw):
        a = dict(d, **kw)
        return msa.chunk_attention(*(a[n] for n in names), out=out)

    call()
    for bad, err in ((dict(q=d["q"].float()), TypeError), (dict(q=d["q"].cpu()), ValueError),
                     (dict(q=d["q"][:, :, :64]), ValueError), (dict(q=d["q"].flatten(1)), ValueError),
                     (dict(q=d["q"][:, ::2]), ValueError), (dict(kc=d["kc"].float()), TypeError),
                     (dict(vc=d["vc"][:1]), ValueError), (dict(table=d["table"][:1]), ValueError),
                     (dict(table=d["table"].long()), TypeError), (dict(seq=d["seq"][:1]), ValueError),
                     (dict(cu=d["cu"][:2]), ValueError), (dict(cu=d["cu"].cpu()), ValueError),
                     (dict(kc=d["kc"][:, :64].contiguous(), vc=d["vc"][:, :64].contiguous()), ValueError),
                     (dict(q=d["q"][:, :3].contiguous()), msa.MSAError),   # three heads on two groups
                     (dict(out=(torch.empty_like(d["q"]), torch.empty((4, 7), device=DEV))), ValueError),
                     (dict(out=(torch.empty_like(d["q"][:3]), None)), ValueError)):
        with pytest.raises(err):
            call(**bad)
    odd = torch.zeros(4 * 8 * D + 4, dtype=torch.bfloat16, device=DEV)[4:].view(4, 8, D)  # 8-byte aligned
    with pytest.raises(msa.MSAError, match="aligned"):
        call(q=odd)
