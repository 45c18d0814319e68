"""GPU tests of the quantised cache: ``append_kv_fp8`` and ``gather_kv_fp8`` (bytes and values: equal
to plain 64-bit implementations written here), ``paged_sparse_decode_fp8`` against 64-bit attention on the
values that the caches hold, and a run of them with the page tables, the scorer and dense attention.

Attention tolerance, per output element, from the roundings the kernel makes (w the exact softmax
weights, A = sum_n w_n |v_n|, ref the exact output):
  * the weights times their values' powers of two, relative to the largest, are rounded to fp16: 2^-11 of
    each term, and 2^-25 below 2^-14: n * 2^-25 * 448 * max_n w_n 2^b_n, at most n * 2^-24 * max_n w_n |v_n|_max;
  * q is rounded to fp16 after a power of two that leaves its largest magnitude at 2^14 or more: 2^-39 of
    that per channel, so a score is off by at most 2^-39 |q|_max sum_d |k_d|;
  * a score is an fp32 sum of 128 products, at most 2^-23 of sum |q_d k_d| per addition (truncating adds
    counted), then scaled to log2 units: ds = 2^-23 * 128 * max_n sum_d |q_d k_nd| + 2^-21 * max |s| with
    the line above;
  * 2^x, the fp32 sums and the merge of partials: 2^-20 + n * 2^-24 per key count n, of A;
  * o is rounded to bf16 once: 2^-8 of the value.
LSE: ds + 2^-20 + n * 2^-24 absolute, + 2^-22 of the value.
"""
import numpy as np
import pytest
import torch

import block_sparse_attention_msa_gb300 as msa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
PAGE = 128
D = 128
BAD_PAGE = 1
F8 = torch.float8_e4m3fn
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
    assert msa.device_error() == 0


def i32(x):
    return torch.from_numpy(np.array(x, dtype=np.int32))


# The 256 e4m3 numbers, from the format: sign, 4 bits of exponent (bias 7), 3 of fraction.
CODES = np.arange(256)
E, F = CODES >> 3 & 15, CODES & 7
VALUES = np.where(E > 0, (1 + F / 8) * 2.0 ** (E - 7), F / 8 * 2.0 ** -6) * np.where(CODES >= 128, -1, 1)
VALUES[(CODES & 127) == 127] = np.nan
POSITIVE = VALUES[:127]    # 0 .. 448, ascending


def ref_quantise(x):
    """Rows [..., D] (float64, bf16 values) -> (e4m3 codes, e + 127): the documented rule, by search."""
    finite = np.isfinite(x)
    a = np.where(finite, np.abs(x), 0).max(-1)
    e = np.full(a.shape, -127)
    for p in range(-127, 119):
        e = np.where(a > 448.0 * 2.0 ** p, p + 1, e)
    y = np.minimum(np.where(finite, np.abs(x), 0) * 2.0 ** -e.astype(np.float64)[..., None], 448.0)
    hi = np.searchsorted(POSITIVE, y)                 # POSITIVE[hi - 1] < y <= POSITIVE[hi]
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = y - POSITIVE[lo], POSITIVE[hi] - y
    code = np.where((dhi < dlo) | ((dhi == dlo) & (hi % 2 == 0)), hi, lo)
    code = np.where(finite, code | (np.signbit(x) << 7), 127)
    return code.astype(np.uint8), (e + 127).astype(np.uint8)


def ref_values(code, scale):
    return VALUES[code] * 2.0 ** (scale.astype(np.float64) - 127)[..., None]


def f64(t):
    return t.double().cpu().numpy()


def u8(t):
    return t.view(torch.uint8).cpu().numpy()


def caches(P, Hkv, fill=0x55):
    c = [torch.full((P, Hkv, PAGE, D), fill, dtype=torch.uint8, device=DEV).view(F8) for _ in range(2)]
    return c + [torch.full((P, Hkv, PAGE), fill, dtype=torch.uint8, device=DEV) for _ in range(2)]


def check_stored(c, slots, k, v):
    """The caches hold the quantised rows at their slots, and what they held before everywhere else."""
    live = slots >= 0
    page, off = slots[live] // PAGE, slots[live] % PAGE
    for rows, cache, scale in ((k, c[0], c[2]), (v, c[1], c[3])):
        code, e = ref_quantise(f64(rows)[live])
        got, ge = u8(cache), scale.cpu().numpy()
        assert np.array_equal(ge[page, :, off], e)
        g = got[page, :, off]
        nan = (code & 127) == 127
        assert np.array_equal((g & 127) == 127, nan) and np.array_equal(g[~nan], code[~nan])
        got, ge = got.copy(), ge.copy()
        got[page, :, off], ge[page, :, off] = 0x55, 0x55
        assert (got == 0x55).all() and (ge == 0x55).all()


@pytest.mark.parametrize("T,Hkv,strided", [(1, 8, False), (3, 1, True), (37, 2, True), (513, 16, False),
                                           (1000, 4, True), (129, 8, True)])
def test_append_and_gather(T, Hkv, strided):
    g = torch.Generator(device=DEV).manual_seed(T)
    P = T // PAGE + 3
    rnd = lambda *s: (torch.randn(s, generator=g, device=DEV) *
                      torch.exp(4 * torch.randn(s[:-1] + (1,), generator=g, device=DEV))).to(torch.bfloat16)
    if strided:
        qkv = rnd(T, 4 * Hkv, D)
        k, v = qkv[:, Hkv:2 * Hkv], qkv[:, 3 * Hkv:]
    else:
        k, v = rnd(T, Hkv, D), rnd(T, Hkv, D)
    slots = torch.randperm(P * PAGE, generator=g, device=DEV)[:T].to(torch.int32)
    slots[T // 3::7] = -1
    c = caches(P, Hkv)
    msa.append_kv_fp8(k, v, slots, *c)
    s = slots.cpu().numpy()
    check_stored(c, s, k, v)
    # read back: the values, exactly; rows with a negative slot left alone; the order free
    order = torch.randperm(T, generator=g, device=DEV)
    out = [torch.full((T, Hkv, D), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    got = msa.gather_kv_fp8(*c, slots[order].contiguous(), out=out)
    assert got[0] is out[0] and got[1] is out[1]
    live = (slots >= 0)[order].cpu().numpy()
    for rows, back in ((k, got[0]), (v, got[1])):
        want = ref_values(*ref_quantise(f64(rows[order])))
        assert np.array_equal(f64(back)[live], want[live])
        assert (f64(back)[~live] == 7).all()
    # what was read back is held exactly when written again. (The bytes may differ: a largest magnitude of
    # 225 * 2^e, just above 448 * 2^(e - 1), is stored as 224 * 2^e, which then takes the power e - 1.)
    again = caches(P, Hkv)
    msa.append_kv_fp8(got[0], got[1], slots[order].contiguous(), *again)
    back = msa.gather_kv_fp8(*again, slots[order].contiguous())
    for a, b in zip(got, back):
        assert torch.equal(a[live], b[live])


@pytest.mark.parametrize("shift", [0, 8, 16, 24])
def test_rows_at_every_16_byte_offset(shift):
    # rows and outputs that are aligned to 16 bytes, not to 32
    g = torch.Generator(device=DEV).manual_seed(shift)
    T, Hkv = 300, 4
    flat = torch.randn(2 * T * (Hkv * D + 8) + 64, generator=g, device=DEV).to(torch.bfloat16)
    rows = flat[shift:shift + 2 * T * (Hkv * D + 8)].view(2, T, Hkv * D + 8)
    k, v = (rows[i, :, :Hkv * D].unflatten(1, (Hkv, D)) for i in range(2))    # strides of 16-byte multiples
    slots = torch.randperm(4 * PAGE, generator=g, device=DEV)[:T].to(torch.int32)
    c = caches(4, Hkv)
    msa.append_kv_fp8(k, v, slots, *c)
    check_stored(c, slots.cpu().numpy(), k, v)
    space = torch.zeros(2 * T * Hkv * D + 64, dtype=torch.bfloat16, device=DEV)
    out = [space[shift + i * T * Hkv * D:shift + (i + 1) * T * Hkv * D].view(T, Hkv, D) for i in range(2)]
    msa.gather_kv_fp8(*c, slots, out=out)
    for x, back in ((k, out[0]), (v, out[1])):
        assert np.array_equal(f64(back), ref_values(*ref_quantise(f64(x))))
    assert not space[:shift].any() and not space[shift + 2 * T * Hkv * D:].any()


def test_append_at_the_borders_of_the_format():
    """Every bf16 magnitude as a row's largest, ties, zeros, subnormals, NaN and infinities."""
    bits = torch.arange(0x7f80, dtype=torch.int32)                    # the finite magnitudes
    top = bits.to(torch.int16).view(torch.bfloat16)
    rows = torch.zeros((len(bits), 1, D), dtype=torch.bfloat16)
    rows[:, 0, 0] = -top
    # multiples of 1/32 of the largest: ties of e4m3 among them; then far below it
    rows[:, 0, 1:65] = (top[:, None].double() * torch.arange(64) / 64).to(torch.bfloat16)
    rows[:, 0, 65:97] = (top[:, None].double() * 2.0 ** -torch.arange(32)).to(torch.bfloat16)
    rows[:, 0, 97:] = -(top[:, None].double() * 1.0625 * 2.0 ** -torch.arange(31)).to(torch.bfloat16)
    rows[::3, 0, 5] = NAN
    rows[::5, 0, 9] = float("inf")
    rows[1::5, 0, 120] = float("-inf")
    rows = rows.nan_to_num(NAN, float("inf"), float("-inf"))
    odd = torch.zeros((4, 1, D), dtype=torch.bfloat16)                # nothing finite but zeros; nothing at all
    odd[0], odd[1], odd[2, 0, 0] = NAN, float("inf"), -0.0
    rows = torch.cat([rows, odd]).to(DEV)
    T = rows.shape[0]
    P = T // PAGE + 1
    slots = torch.arange(T, dtype=torch.int32, device=DEV)
    c = caches(P, 1)
    msa.append_kv_fp8(rows, rows, slots, *c)
    check_stored(c, slots.cpu().numpy(), rows, rows)
    k, v = msa.gather_kv_fp8(*c, slots)
    # exact in bf16, but for what lies below its range: rounded once
    want = torch.from_numpy(ref_values(*ref_quantise(f64(rows)))).to(torch.bfloat16)
    for back in (k, v):
        assert torch.equal(back.cpu().nan_to_num(9e9), want.nan_to_num(9e9))


def test_every_code_and_every_scale_is_read_back():
    P, Hkv = 2, 16
    code = torch.arange(P * Hkv * PAGE * D, dtype=torch.int64)
    kc = ((code * 37 + code // 256) % 256).to(torch.uint8).view(P, Hkv, PAGE, D).to(DEV)
    ks = (torch.arange(P * Hkv * PAGE) % 247).to(torch.uint8).view(P, Hkv, PAGE).to(DEV)
    slots = torch.arange(P * PAGE, dtype=torch.int32, device=DEV).flip(0).repeat(2)    # a slot for two rows
    k, v = msa.gather_kv_fp8(kc.view(F8), kc.flip(0).contiguous().view(F8), ks, ks, slots)
    for back, src in ((k, kc), (v, kc.flip(0))):
        want = ref_values(src.cpu().numpy(), ks.cpu().numpy()).transpose(0, 2, 1, 3).reshape(-1, Hkv, D)
        want = torch.from_numpy(want[slots.cpu().numpy()]).to(torch.bfloat16)
        assert torch.equal(back.cpu().nan_to_num(9e9), want.nan_to_num(9e9))


def test_append_and_gather_skip_bad_slots_and_empty_batches():
    k = torch.ones((3, 2, D), dtype=torch.bfloat16, device=DEV)
    c = caches(2, 2)
    slots = i32([2 * PAGE, -7, 2 * PAGE - 1])
    msa.append_kv_fp8(k, k, slots.to(DEV), *c)
    assert msa.device_error() == BAD_PAGE
    check_stored(c, np.array([-1, -1, 2 * PAGE - 1]), k, k)
    out = [torch.full((3, 2, D), 5.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    msa.gather_kv_fp8(*c, slots.to(DEV), out=out)
    assert msa.device_error() == BAD_PAGE
    for o in out:
        assert (o[:2] == 5).all() and (o[2] == 1).all()
    msa.append_kv_fp8(k[:0], k[:0], i32([]).to(DEV), *c)
    none = msa.gather_kv_fp8(*c, i32([]).to(DEV))
    assert none[0].shape == (0, 2, D)


# ------------------------------------------------------------------------------ decode

def make(lens, topk, Hq, Hkv, seed, spread=1.0, pages=40):
    """R rows x Hkv flattened rows of the given visible lengths on random pages; what no length covers
    is NaN with scales of any value. `spread`: of the rows' magnitudes, in powers of e."""
    g = torch.Generator().manual_seed(seed)
    R = len(lens) // Hkv
    rows = lambda: (torch.randn((pages, Hkv, PAGE, D), generator=g) *
                    torch.exp(spread * torch.randn((pages, Hkv, PAGE, 1), generator=g))).to(torch.bfloat16)
    fpt = torch.full((R * Hkv, topk), -1, dtype=torch.int64)
    seen = np.zeros((pages, Hkv, PAGE), dtype=bool)
    for f, n in enumerate(lens):
        m = (n + PAGE - 1) // PAGE
        page = torch.randperm(pages, generator=g)[:m]
        fpt[f, :m] = page * PAGE * Hkv + f % Hkv
        for i, p in enumerate(page.tolist()):
            seen[p, f % Hkv, :min(PAGE, n - i * PAGE)] = True
    w = dict(q=(torch.randn((R, Hq, D), generator=g) * D ** -0.5).to(torch.bfloat16), fpt=fpt.to(torch.int32),
             lens=i32(lens))
    for x in "kv":
        code, e = ref_quantise(f64(rows()))
        code[~seen], e[~seen] = 0x7f, np.random.default_rng(seed).integers(0, 256, (~seen).sum())
        w[x + "c"], w[x + "s"] = torch.from_numpy(code), torch.from_numpy(e)
    return w


def reference(w):
    q, fpt = w["q"].double(), w["fpt"].long()
    R, Hq, _ = q.shape
    Hkv = w["kc"].shape[1]
    G = Hq // Hkv
    o = torch.zeros((R, Hq, D), dtype=torch.float64)
    lse = torch.full((R, Hq), float("-inf"), dtype=torch.float64)
    to, tl = torch.zeros_like(o), torch.zeros_like(lse)
    topk = fpt.shape[1]
    for f, n in enumerate(w["lens"].tolist()):
        n = min(max(n, 0), topk * PAGE)
        if n == 0:
            continue
        r, h = f // Hkv, slice(f % Hkv * G, (f % Hkv + 1) * G)
        vp = fpt[f, :(n + PAGE - 1) // PAGE]
        page, g = vp // (PAGE * Hkv), vp % (PAGE * Hkv)
        k, v = (torch.from_numpy(ref_values(w[x + "c"][page, g].numpy(), w[x + "s"][page, g].numpy())).flatten(0, 1)[:n]
                for x in "kv")
        qi = q[r, h]
        s = qi @ k.T
        z = torch.logsumexp(s, -1, keepdim=True)
        p = torch.exp(s - z)
        ref, A = p @ v, p @ v.abs()
        ds = 2.0 ** -23 * 128 * (qi.abs() @ k.abs().T).amax(-1, keepdim=True) + 2.0 ** -21 * s.abs().amax(-1, keepdim=True) \
            + 2.0 ** -39 * qi.abs().amax(-1, keepdim=True) * k.abs().sum(-1).max()
        acc = 2.0 ** -20 + n * 2.0 ** -24
        small = n * 2.0 ** -24 * (p * v.abs().amax(-1)).amax(-1, keepdim=True)
        o[r, h], lse[r, h] = ref, z.squeeze(-1)
        to[r, h] = 2.0 ** -8 * ref.abs() * (1 + 2.0 ** -9) + (2.0 ** -11 * (1 + 2.0 ** -7) + 2 * ds + acc) * A + small
        tl[r, h] = (ds + acc + 2.0 ** -22 * z.abs()).squeeze(-1)
    return o, lse, to, tl


def run(w, **kw):
    d = {k: x.to(DEV) for k, x in w.items()}
    return msa.paged_sparse_decode_fp8(d["q"], d["kc"].view(F8), d["vc"].view(F8), d["ks"], d["vs"], d["fpt"],
                                       d["lens"], **kw)


def check(got, ref):
    o, lse, to, tl = ref
    go, gl = got[0].double().cpu(), got[1].double().cpu()
    err = (go - o).abs()
    assert (err <= to).all(), f"o: worst error / tolerance {(err / to.clamp_min(1e-300)).max():.3f}"
    empty = torch.isneginf(lse)
    assert torch.equal(torch.isneginf(gl), empty)
    assert (go[empty] == 0).all()
    err = (gl - lse).abs()[~empty]
    assert (err <= tl[~empty]).all(), f"lse: worst error / tolerance {(err / tl[~empty]).max():.3f}"


def _lens(n, seed, topk, lo=1):
    return np.random.default_rng(seed).integers(lo, topk * PAGE + 1, n).tolist()


CASES = [
    # lengths, topk, Hq, Hkv
    ([1], 2, 1, 1), ([31], 2, 8, 1), ([32], 2, 8, 1), ([33], 2, 16, 1),      # around a step
    ([127, 128], 2, 8, 2), ([129, 256], 2, 32, 2), ([300, 511, 512, 5], 4, 8, 4),   # around a page
    ([0, 700, 0, 12], 16, 32, 4),                       # empty rows
    (_lens(16, 0, 16), 16, 64, 8),                      # few rows: a cluster each
    (_lens(48, 1, 32), 32, 16, 16),                     # one head per group
    (_lens(64, 2, 16), 16, 64, 8), (_lens(80, 3, 5), 5, 16, 1), (_lens(96, 4, 7), 7, 8, 2),
    (_lens(160, 5, 3, 0), 3, 256, 16), (_lens(600, 6, 2), 2, 4, 1), ([64 * PAGE] * 40 + [1] * 8, 64, 32, 8),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_decode_against_64_bits(case):
    lens, topk, Hq, Hkv = CASES[case]
    w = make(lens, topk, Hq, Hkv, seed=case, pages=max(40, topk))
    check(run(w), reference(w))


@pytest.mark.parametrize("R", [1, 40])
def test_decode_of_rows_whose_magnitudes_differ_by_orders(R):
    # values whose powers of two differ by 2^40 and more, keys with large scores, small and large queries
    w = make(_lens(R * 4, 9, 6, 200), 6, 32, 4, seed=30, spread=5.0)
    w["ks"] = torch.where(w["ks"] > 130, 130, w["ks"]).to(torch.uint8)
    w["q"][:, ::3] *= 2.0 ** -60
    w["q"][:, 1::3] *= 2.0 ** 4
    check(run(w), reference(w))
    w["vs"] = (w["vs"].int() - 100).clamp(0, 246).to(torch.uint8)       # ... and values near fp32's end
    check(run(w), reference(w))


@pytest.mark.parametrize("R", [1, 60])
def test_what_is_not_finite_shows_in_the_rows_that_see_it(R):
    w = make([300] * (2 * R), 4, 16, 2, seed=31)
    clean = run(w)
    page = int(w["fpt"][0, 1]) // (PAGE * 2)
    only = (w["fpt"] // (PAGE * 2) == page).any(1)
    bad = dict(w, vc=w["vc"].clone())
    bad["vc"][page, 0, 3, 50] = 0x7f
    o, lse = run(bad)
    sees = only.view(R, 2)[:, 0].repeat_interleave(8).view(R, 8).to(DEV)
    assert torch.isnan(o[:, :8, 50])[sees].all()
    o[:, :8, 50] = torch.where(sees, clean[0][:, :8, 50], o[:, :8, 50])
    assert torch.equal(o, clean[0]) and torch.equal(lse, clean[1])
    bad = dict(w, kc=w["kc"].clone())
    bad["kc"][page, 0, 3, 50] = 0xff
    o, lse = run(bad)
    assert torch.isnan(o[:, :8][sees]).all() and torch.isnan(lse[:, :8][sees]).all()
    assert torch.equal(o[:, 8:], clean[0][:, 8:]) and torch.equal(lse[:, 8:], clean[1][:, 8:])


def test_decode_bad_pages_and_lengths():
    w = make([300, 300] * 40, 4, 16, 2, seed=32)
    w["kc"][0], w["vc"][0], w["ks"][0], w["vs"][0] = 0x38, 0x31, 127, 127
    w["fpt"][0, 1], w["fpt"][3, 0] = 40 * PAGE * 2, -5
    got = run(w)
    assert msa.device_error() == BAD_PAGE
    w["fpt"][0, 1] = w["fpt"][3, 0] = 0
    check(got, reference(w))
    w["lens"][5], w["lens"][6] = -3, 300
    got = run(w)
    check(got, reference(w))


def test_decode_runs_agree_bit_for_bit_and_inputs_stay():
    for lens in (_lens(16, 0, 16), _lens(160, 1, 16)):      # a cluster per row; partials and a merge
        w = make(lens, 16, 64, 8, seed=33)
        d = {k: x.to(DEV) for k, x in w.items()}
        copies = {k: x.clone() for k, x in d.items()}
        args = (d["q"], d["kc"].view(F8), d["vc"].view(F8), d["ks"], d["vs"], d["fpt"], d["lens"])
        o1, l1 = msa.paged_sparse_decode_fp8(*args)
        ws = msa.Workspace()
        R = w["q"].shape[0]
        nbytes = msa.load().msa_paged_sparse_decode_workspace_size(R, 64, 8, 16)
        buf = ws.get("decode_fp8", nbytes + 4096, DEV)
        buf.fill_(0xff)
        out = (torch.full_like(o1, 3.0), torch.full_like(l1, 3.0))
        o2, l2 = msa.paged_sparse_decode_fp8(*args, workspace=ws, out=out)
        assert o2 is out[0] and torch.equal(o1.view(torch.int16), o2.view(torch.int16)) and torch.equal(l1, l2)
        assert (buf[nbytes:] == 0xff).all()
        o3, l3 = msa.paged_sparse_decode_fp8(*args, with_lse=False)
        assert l3 is None and torch.equal(o1.view(torch.int16), o3.view(torch.int16))
        for k, x in d.items():
            assert torch.equal(x.view(torch.uint8), copies[k].view(torch.uint8))


def test_captured_decodes_replay_with_other_tables_and_overlap():
    cases = [_lens(160, s, 8, 0) for s in (1, 2, 3)]
    ws = [make(lens, 8, 32, 4, seed=40 + i) for i, lens in enumerate(cases)]
    refs = [reference(w) for w in ws]
    sets, graphs, outs = [], [], []
    for _ in range(2):
        d = {k: x.to(DEV) for k, x in ws[0].items()}
        call = lambda: msa.paged_sparse_decode_fp8(d["q"], d["kc"].view(F8), d["vc"].view(F8), d["ks"], d["vs"],
                                                   d["fpt"], d["lens"])
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call())
        sets.append(d)
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for a, b in ((0, 1), (1, 2), (2, 0)):
        for d, w in ((sets[0], ws[a]), (sets[1], ws[b])):
            for k, x in w.items():
                d[k].copy_(x)
        torch.cuda.synchronize()
        for _ in range(3):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        check(outs[0], refs[a])
        check(outs[1], refs[b])


def test_a_request_on_the_quantised_cache():
    """A prompt in two chunks, then decode steps, on e4m3 caches: page tables, quantised append, the prefix
    read back into bf16 pages for dense attention of the second chunk, and sparse decode with the
    scorer's selections, in the same tables as the bf16 cache's."""
    g = torch.Generator().manual_seed(50)
    B, Hq, Hkv, Di, mb, topk = 2, 16, 2, 64, 10, 4
    P = B * mb
    bf = torch.bfloat16
    rnd = lambda *s: torch.randn(s, generator=g).to(bf).to(DEV)
    c = caches(P, Hkv, fill=0x7f)
    idx = torch.zeros((P, PAGE, Hkv, Di), dtype=bf, device=DEV)
    table = torch.full((B, mb), -1, dtype=torch.int32, device=DEV)
    free = torch.randperm(P, generator=g).to(torch.int32).to(DEV)
    used, prev = (torch.zeros(n, dtype=torch.int32, device=DEV) for n in (1, B))
    held = [[] for _ in range(B)]           # the quantised values of every token, from the rule
    for new in ([300, 210], [170, 333], [1, 1], [1, 1]):
        T = sum(new)
        q, k, v = (rnd(T, Hq, D).float() * D ** -0.5).to(bf), rnd(T, Hkv, D), rnd(T, Hkv, D)
        seq, cu, slots, _, used = msa.build_page_tables(prev, i32(new).to(DEV), table, free, used, T=T, num_pages=P)
        msa.append_kv_fp8(k, v, slots, *c)
        msa.append_kv(None, None, rnd(T, Hkv, Di), slots, None, None, idx)
        at = cu.tolist()
        for b in range(B):
            rows = slice(at[b], at[b + 1])
            held[b].append([torch.from_numpy(ref_values(*ref_quantise(f64(x[rows])))) for x in (k, v)])
        full = [[torch.cat([h[i] for h in held[b]]) for i in range(2)] for b in range(B)]
        if T > 2:
            # every request's tokens in order, as bf16 pages with a table of their own
            blocks = (seq + PAGE - 1) // PAGE
            most = int(blocks.max())
            pos = torch.arange(most * PAGE, device=DEV)
            slot = (table[:, :most].repeat_interleave(PAGE, 1) * PAGE + pos % PAGE).to(torch.int32)
            slot = torch.where(pos < seq[:, None], slot, -1).to(torch.int32).view(-1)
            kb, vb = msa.gather_kv_fp8(*c, slot)
            o, lse = msa.chunk_attention(q, kb.view(-1, PAGE, Hkv, D), vb.view(-1, PAGE, Hkv, D),
                                         torch.arange(B * most, dtype=torch.int32, device=DEV).view(B, most), seq, cu)
        else:
            ids, _ = msa.index_score_topk(rnd(B, Hkv, Di), idx, table.clamp(min=0), seq, N=1, topk=topk)
            fpt, lens = msa.build_sparse_page_table(ids, table.clamp(min=0), seq, N=1, num_pages=P)
            o, lse = msa.paged_sparse_decode_fp8(q, *c, fpt, lens)
        for b in range(B):
            n, end = new[b], int(seq[b])
            fk, fv = full[b]
            for i in range(0, n, 7 if n > 1 else 1):
                r, vis = at[b] + i, end - n + i + 1
                for h in range(Hq):
                    grp = h // (Hq // Hkv)
                    s = fk[:vis, grp] @ q[r, h].double().cpu()
                    if n == 1:
                        block = torch.arange(vis) // PAGE
                        s[~torch.isin(block, ids[b, grp].cpu().long())] = float("-inf")
                    p = torch.softmax(s, 0)
                    A = (p @ fv[:vis, grp].abs())
                    # weights and output rounded to bf16 at the coarsest, as derived above
                    tol = 2.0 ** -8 * (1 + 2.0 ** -6) * (A + (p @ fv[:vis, grp]).abs()) + 1e-4 * A
                    assert ((o[r, h].double().cpu() - p @ fv[:vis, grp]).abs() <= tol).all()
                    assert abs(float(lse[r, h]) - float(torch.logsumexp(s, 0))) <= 1e-4
        prev = seq


def test_refusals():
    c = caches(2, 2)
    k = torch.zeros((3, 2, D), dtype=torch.bfloat16, device=DEV)
    slots = i32([0, 1, 2]).to(DEV)

    def append(**kw):
        a = dict(k=k, v=k, slots=slots, kc=c[0], vc=c[1], ks=c[2], vs=c[3])
        a.update(kw)
        msa.append_kv_fp8(*a.values())

    append()
    for bad, err in ((dict(k=k.float()), TypeError), (dict(k=None), TypeError), (dict(v=k[:2]), ValueError),
                     (dict(k=k.cpu()), ValueError), (dict(slots=slots.long()), TypeError), (dict(kc=c[0].float()), TypeError),
                     (dict(kc=c[0][:1]), ValueError), (dict(vc=c[1][:, :1]), ValueError), (dict(ks=c[2][:, :, :64]), ValueError),
                     (dict(vs=c[3].to(torch.int8)), TypeError), (dict(kc=c[0].transpose(1, 2)), ValueError),
                     (dict(k=torch.zeros((3, 2, 2 * D), dtype=torch.bfloat16, device=DEV)[:, :, ::2]), ValueError),
                     (dict(k=torch.zeros((3, 2 * D + 4), dtype=torch.bfloat16, device=DEV)[:, :2 * D].unflatten(1, (2, D))),
                      msa.MSAError)):
        with pytest.raises(err):
            append(**bad)
    out = [torch.zeros_like(k) for _ in range(2)]
    for bad, err in ((dict(out=(out[0], out[1][:2])), ValueError), (dict(out=(out[0].float(), out[1])), TypeError),
                     (dict(out=(out[0].cpu(), out[1])), ValueError)):
        with pytest.raises(err):
            msa.gather_kv_fp8(*c, slots, **bad)
    q = torch.zeros((1, 8, D), dtype=torch.bfloat16, device=DEV)
    fpt, lens = torch.zeros((2, 4), dtype=torch.int32, device=DEV), torch.ones(2, dtype=torch.int32, device=DEV)

    def decode(out=None, **kw):
        a = dict(q=q, kc=c[0], vc=c[1], ks=c[2], vs=c[3], fpt=fpt, lens=lens)
        a.update(kw)
        return msa.paged_sparse_decode_fp8(*a.values(), out=out)

    decode()
    for bad, err in ((dict(q=q.float()), TypeError), (dict(q=q[:, :, :64].contiguous()), ValueError),
                     (dict(fpt=fpt[:1]), ValueError), (dict(lens=lens[:1]), ValueError), (dict(lens=lens.long()), TypeError),
                     (dict(q=q[:, :5].contiguous()), msa.MSAError), (dict(ks=c[2][:1]), ValueError),
                     (dict(out=(q[:, :4].contiguous(), None)), ValueError),
                     (dict(fpt=torch.zeros((2, 65), dtype=torch.int32, device=DEV)), msa.MSAError)):
        with pytest.raises(err):
            decode(**bad)
