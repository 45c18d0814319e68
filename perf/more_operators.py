"""Measured cases of the quantised cache and of dense attention for ragged batches: K and V
quantised to 8 bits as they are written, read back, sparse decode attention on the quantised
cache, and causal attention of every request's new tokens over the paged cache.

``run`` computes an operator either in its plain form (elementary torch operations, fp32) or
through the package's entry points (``own = True``); ``exact`` computes the same outputs in 64
bits straight from the definitions. Conventions are those of the package: 128-token pages, bf16
caches [num_pages, 128, Hkv, D], a page table [B, max_blocks] int32, slots page * 128 + offset,
virtual pages page * 128 * Hkv + group. The quantised caches are [num_pages, Hkv, 128, D] e4m3
with one power-of-two scale per token and head, [num_pages, Hkv, 128] uint8 (exponent + 127).
"""
from __future__ import annotations

import math

import torch

own = False

PAGE = 128
D = 128


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step: the new tokens of eight requests, quantised as they are written (and
        # read back as the values that the cache holds)
        dict(name="append_decode_8", op="append", T=8, pad=0, Hkv=8, pages=480),
        # a 32768-token prefill chunk written to the quantised cache
        dict(name="append_chunk_32768", op="append", T=32768, pad=0, Hkv=8, pages=300),
        # a ragged set of rows padded to a captured size (rows behind the last token: slot -1)
        dict(name="gather_ragged_1777", op="gather", T=1777, pad=271, Hkv=4, pages=96),
        # a 60032-token prefix read back for a prefill chunk behind it
        dict(name="gather_prefix_60032", op="gather", T=60032, pad=0, Hkv=8, pages=520),
        # the small layer (Hq 8, Hkv 2, k 4): latency only
        dict(name="sparse_tiny_1x2048", op="sparse", B=1, N=1, Hq=8, Hkv=2, topk=4, lo=2048, hi=2048),
        # a decode batch of 64 requests of 8K to 128K tokens
        dict(name="sparse_64_on_8k_128k", op="sparse", B=64, N=1, Hq=64, Hkv=8, topk=16, lo=8192,
             hi=131072),
        # few rows at a context of a million tokens
        dict(name="sparse_4_on_1m", op="sparse", B=4, N=1, Hq=64, Hkv=8, topk=32, lo=1048576,
             hi=1048576),
        # one new token of one request of the small layer: latency only
        dict(name="chunk_tiny_1x2048", op="chunk", B=1, chunks=0, new=1, ctx=2047, Hq=8, Hkv=2, pad=0),
        # a decode step of 64 requests, each with its own cache
        dict(name="chunk_decode_64", op="chunk", B=64, chunks=0, new=1, ctx=16384, Hq=64, Hkv=8, pad=0),
        # a scheduler step that mixes 56 decode rows with five prompt chunks, token rows padded to
        # the step's capacity
        dict(name="chunk_mixed_61", op="chunk", B=61, chunks=5, new=1073, ctx=20000, Hq=64, Hkv=8,
             pad=131),
        # a chunk of new tokens behind a long cached prefix
        dict(name="chunk_2048_on_60032", op="chunk", B=1, chunks=1, new=2048, ctx=60032, Hq=64, Hkv=8,
             pad=0),
        # a whole prompt
        dict(name="chunk_prompt_16384", op="chunk", B=1, chunks=1, new=16384, ctx=0, Hq=64, Hkv=8,
             pad=0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    """One more case of the listed ranges, none dearer than the largest listed one of its kind."""
    op = rng.choice(["append", "gather", "sparse", "sparse", "chunk", "chunk", "chunk"])
    if op in ("append", "gather"):
        Hkv = rng.choice([1, 2, 4, 8, 16])
        T = _log_int(rng, 1, (32768 if op == "append" else 60032) * 8 // max(Hkv, 8))
        return dict(op=op, T=T, pad=rng.choice([0, 0, rng.randint(1, 300)]), Hkv=Hkv,
                    pages=T // PAGE + rng.randint(2, 60))
    if op == "sparse":
        while True:
            Hkv, G = rng.choice([1, 2, 4, 8, 8, 16]), rng.choice([1, 2, 4, 8, 8, 16])
            B, N = _log_int(rng, 1, 64), rng.choice([1, 1, 1, 2, rng.randint(2, 16)])
            hi = _log_int(rng, 16, 131072)
            c = dict(op=op, B=B, N=N, Hq=Hkv * G, Hkv=Hkv, topk=rng.choice([4, 16, 32, rng.randint(2, 64)]),
                     lo=max(N, hi // rng.randint(1, 16)), hi=max(N, hi))
            if B * N * Hkv * c["topk"] <= 64 * 8 * 16 and B * c["hi"] * Hkv <= 64 * 70000 * 8:
                return c
    while True:
        Hkv, G = rng.choice([1, 2, 4, 8, 8, 16]), rng.choice([1, 2, 4, 8, 8, 16])
        B = _log_int(rng, 1, 64)
        c = dict(op=op, B=B, chunks=rng.choice([0, B, rng.randint(0, B)]), new=_log_int(rng, 1, 16384),
                 ctx=rng.choice([0, _log_int(rng, 1, 60032), _log_int(rng, 1, 60032)]), Hq=Hkv * G,
                 Hkv=Hkv, pad=rng.choice([0, 0, rng.randint(1, 300)]))
        tokens = c["chunks"] * c["new"] + B - c["chunks"]
        keys = B * c["ctx"] + tokens
        if tokens * Hkv * G * (c["ctx"] + c["new"]) <= 16384 * 64 * 16384 and tokens <= 16384 and \
                keys * Hkv <= 64 * 16384 * 8:
            return c


# ------------------------------------------------------------------------------ inputs

def _rows(shape, gen, dev):
    """Rows of a projection: normal values, the magnitude of a row (one token, one head) its own."""
    x = torch.randn(shape, generator=gen, device=dev)
    return (x * torch.exp(0.7 * torch.randn(shape[:-1] + (1,), generator=gen, device=dev))).to(torch.bfloat16)


def _quantised(shape, gen, dev):
    """A quantised cache of random rows: ([P, Hkv, 128, D] e4m3, [P, Hkv, 128] uint8)."""
    cache = torch.empty(shape, dtype=torch.float8_e4m3fn, device=dev)
    scale = torch.empty(shape[:3], dtype=torch.uint8, device=dev)
    step = max(1, (1 << 28) // (shape[1] * PAGE * D))
    for p in range(0, shape[0], step):
        cache[p:p + step], scale[p:p + step] = _quantise(_rows((min(step, shape[0] - p),) + shape[1:], gen, dev))
    return cache, scale


def _slots(case, gen, dev):
    """T token rows on pages in random order, rows behind them -1."""
    T, P = case["T"], case["pages"]
    slots = torch.full((T + case["pad"],), -1, dtype=torch.int32, device=dev)
    order = torch.randperm(P, generator=gen, device=dev)
    pos = torch.arange(T, device=dev) + 37 % (P * PAGE - T)
    slots[:T] = (order[pos // PAGE] * PAGE + pos % PAGE).to(torch.int32)
    return slots


def _chunk_lens(case, seed):
    """(new tokens, tokens held with them) of every request, on the host."""
    gen = torch.Generator().manual_seed(int(seed))
    B, ctx = case["B"], case["ctx"]
    new = torch.ones(B, dtype=torch.int64)
    where = torch.randperm(B, generator=gen)[:case["chunks"]]
    if case["chunks"] == 1:
        new[where] = case["new"]
    else:
        new[where] = torch.randint(max(1, case["new"] // 2), case["new"] + 1, (case["chunks"],), generator=gen)
    held = torch.full((B,), ctx, dtype=torch.int64)
    if B > 1 and ctx:
        held = torch.randint(max(1, ctx // 4), ctx + 1, (B,), generator=gen)
    return new, held + new


def _pieces(new, seq, Hq):
    """The plain form's plan: lists of (requests, first new token, tokens, keys) whose padded scores
    fit 4 GB; requests of like sizes share one."""
    out, cur = [], None
    for b in sorted(range(len(new)), key=lambda b: (new[b], seq[b])):
        n, s = new[b], seq[b]
        rows = max(1, (1 << 30) // (Hq * s))
        if cur and cur[2] == n and (len(cur[0]) + 1) * n * Hq * s <= 1 << 30 and 4 * cur[3] >= s:
            cur[0].append(b)
            cur[3] = s
            continue
        cur = None
        for i in range(0, n, rows):
            out.append([[b], i, min(rows, n - i), s])
        if rows >= n:
            cur = out[-1]
    return out


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed) + 1)
    op, Hkv = case["op"], case["Hkv"]
    bf16 = torch.bfloat16
    st = {"case": dict(case)}
    if op in ("append", "gather"):
        T, P, rows = case["T"], case["pages"], case["T"] + case["pad"]
        st["slots"] = _slots(case, gen, dev)
        if op == "append":
            # k and v as the projection leaves them: slices of one [rows, (G + 2) * Hkv * D] matrix
            qkv = _rows((rows, 4 * Hkv, D), gen, dev)
            st["k"], st["v"] = qkv[:, 2 * Hkv:3 * Hkv], qkv[:, 3 * Hkv:]
            st["kc"], st["vc"] = (torch.zeros((P, Hkv, PAGE, D), dtype=torch.float8_e4m3fn, device=dev)
                                  for _ in range(2))
            st["ks"], st["vs"] = (torch.zeros((P, Hkv, PAGE), dtype=torch.uint8, device=dev) for _ in range(2))
        else:
            st["kc"], st["ks"] = _quantised((P, Hkv, PAGE, D), gen, dev)
            st["vc"], st["vs"] = _quantised((P, Hkv, PAGE, D), gen, dev)
        st["out"] = tuple(torch.zeros((rows, Hkv, D), dtype=bf16, device=dev) for _ in range(2))
        return st
    B, Hq = case["B"], case["Hq"]
    if op == "sparse":
        N, topk = case["N"], case["topk"]
        seq = torch.randint(case["lo"], case["hi"] + 1, (B,), generator=gen, device=dev)
        blocks = (seq + PAGE - 1) // PAGE
        mb = int(blocks.max())
        P = int(blocks.sum()) + 3
        st["kc"], st["ks"] = _quantised((P, Hkv, PAGE, D), gen, dev)
        st["vc"], st["vs"] = _quantised((P, Hkv, PAGE, D), gen, dev)
        perm = torch.randperm(P, generator=gen, device=dev)
        cols = torch.arange(mb, device=dev)
        table = torch.zeros((B, mb), dtype=torch.int64, device=dev)
        table[cols[None] < blocks[:, None]] = perm[:P - 3]
        # the selections of stage 1: the sink block, the local block, random others, ascending
        pos = (seq[:, None] - N + torch.arange(N, device=dev)).reshape(-1)
        local = pos // PAGE
        pick = torch.rand((B * N, Hkv, mb), generator=gen, device=dev)
        pick[..., 0] = 2.0
        pick.scatter_(2, local[:, None, None].expand(-1, Hkv, 1), 3.0)
        pick.masked_fill_(cols > local[:, None, None], -1.0)
        val, ids = pick.topk(min(topk, mb), dim=2)
        ids = torch.where(val >= 0, ids, mb).sort(dim=2).values
        held = (ids < mb).sum(2)
        pages = table.repeat_interleave(N, 0)[:, None].expand(-1, Hkv, -1).gather(2, ids.clamp(max=mb - 1))
        fpt = torch.full((B * N, Hkv, topk), -1, dtype=torch.int64, device=dev)
        groups = torch.arange(Hkv, device=dev)[None, :, None]
        fpt[..., :ids.shape[2]] = torch.where(ids < mb, pages * PAGE * Hkv + groups, -1)
        lens = (held - 1) * PAGE + (pos % PAGE + 1)[:, None]
        st["fpt"] = fpt.view(-1, topk).to(torch.int32)
        st["lens"] = lens.reshape(-1).to(torch.int32)
        st["q"] = (torch.randn((B * N, Hq, D), generator=gen, device=dev) * D ** -0.5).to(bf16)
        return st
    new, seq = _chunk_lens(case, seed)
    blocks = (seq + PAGE - 1) // PAGE
    P = int(blocks.sum()) + 3
    mb = int(blocks.max())
    perm = torch.randperm(P, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros((B, mb), dtype=torch.int32, device=dev)
    table[torch.arange(mb, device=dev)[None] < blocks.to(dev)[:, None]] = perm[:P - 3]
    cu = torch.zeros(B + 1, dtype=torch.int64)
    cu[1:] = new.cumsum(0)
    T = case["chunks"] * case["new"] + B - case["chunks"] + case["pad"]         # the step's capacity
    for name in ("kc", "vc"):
        st[name] = torch.randn((P, PAGE, Hkv, D), generator=gen, device=dev, dtype=bf16)
    q = (torch.randn((T, Hq, D), generator=gen, device=dev) * D ** -0.5).to(bf16)
    pieces = [(torch.tensor(p[0], device=dev), *p[1:]) for p in _pieces(new.tolist(), seq.tolist(), Hq)]
    st.update(q=q, table=table, seq=seq.to(dev, torch.int32), cu=cu.to(dev, torch.int32), pieces=pieces,
              out=(torch.zeros((T, Hq, D), dtype=bf16, device=dev),
                   torch.zeros((T, Hq), dtype=torch.float32, device=dev)))
    return st


# ------------------------------------------------------------------------------ passes

def _quantise(x):
    """Rows [..., D] as (e4m3 values, exponent + 127 of the smallest power of two that brings the
    row's largest magnitude to at most 448)."""
    xf = x.float()
    frac, exp = torch.frexp(xf.abs().amax(-1))                   # a = frac * 2^exp, frac in [0.5, 1)
    e = (exp - 9 + (frac > 0.875).int()).clamp(-127, 119)        # 448 = 0.875 * 2^9
    y = torch.ldexp(xf, -e[..., None]).clamp(-448, 448)
    return y.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _dequantise(x, scale):
    """fp32 values of quantised rows."""
    return torch.ldexp(x.float(), scale.int()[..., None] - 127)


def _append_plain(st):
    live = st["slots"] >= 0
    # padding rows write the first live row once more, so that no row needs a host decision
    src = torch.where(live, torch.arange(live.numel(), device=live.device), 0)
    dst = st["slots"].long()[src]
    page, off = dst // PAGE, dst % PAGE
    st["kc"][page, :, off], st["ks"][page, :, off] = _quantise(st["k"][src])
    st["vc"][page, :, off], st["vs"][page, :, off] = _quantise(st["v"][src])
    return _gather_plain(st)


def _gather_plain(st):
    live = (st["slots"] >= 0)[:, None, None]
    dst = st["slots"].long().clamp(min=0)
    page, off = dst // PAGE, dst % PAGE
    k = _dequantise(st["kc"][page, :, off], st["ks"][page, :, off])
    v = _dequantise(st["vc"][page, :, off], st["vs"][page, :, off])
    st["out"][0].copy_(torch.where(live, k.to(torch.bfloat16), st["out"][0]))
    st["out"][1].copy_(torch.where(live, v.to(torch.bfloat16), st["out"][1]))
    return st["out"]


def _softmax_v(s, v):
    """Output and log-sum-exp of masked scores s [..., G, n] on values v [..., n, D]."""
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), 0.0, m)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / l, (m + torch.log(l)).squeeze(-1)


def _sparse_plain(st):
    Hkv, topk = st["case"]["Hkv"], st["case"]["topk"]
    R, Hq, _ = st["q"].shape
    vp = st["fpt"].long().view(R * Hkv, topk).clamp(min=0)
    page, g = vp // (PAGE * Hkv), vp % (PAGE * Hkv)
    k = _dequantise(st["kc"][page, g], st["ks"][page, g]).view(R * Hkv, topk * PAGE, D)
    v = _dequantise(st["vc"][page, g], st["vs"][page, g]).view(R * Hkv, topk * PAGE, D)
    s = torch.matmul(st["q"].float().view(R * Hkv, Hq // Hkv, D), k.transpose(1, 2))
    seen = torch.arange(topk * PAGE, device=s.device) < st["lens"][:, None]
    o, lse = _softmax_v(s.masked_fill_(~seen[:, None, :], float("-inf")), v)
    return o.view(R, Hq, D).to(torch.bfloat16), lse.view(R, Hq)


def _chunk_plain(st):
    table, cu, seq = st["table"], st["cu"].long(), st["seq"].long()
    Hkv = st["case"]["Hkv"]
    o_out, lse_out = st["out"]
    T, Hq, _ = st["q"].shape
    G = Hq // Hkv
    kc, vc = st["kc"].view(-1, Hkv, D), st["vc"].view(-1, Hkv, D)
    for reqs, first, count, most in st["pieces"]:
        i = first + torch.arange(count, device=table.device)
        row = cu[reqs][:, None] + i                                              # [b, n]
        pos = (seq - cu.diff())[reqs][:, None] + i                               # [b, n]
        key = torch.arange(most, device=table.device)
        at = torch.minimum(key, seq[reqs][:, None] - 1)
        cell = table[reqs].gather(1, at // PAGE).long() * PAGE + at % PAGE       # [b, keys]
        q = st["q"][row].float().view(-1, count, Hkv, G, D).transpose(1, 2).reshape(-1, Hkv, count * G, D)
        s = torch.matmul(q, kc[cell].float().permute(0, 2, 3, 1)).view(-1, Hkv, count, G, most)
        s.masked_fill_((key > pos[..., None])[:, None, :, None, :], float("-inf"))
        o, lse = _softmax_v(s.view(-1, Hkv, count * G, most), vc[cell].float().transpose(1, 2))
        o_out[row] = o.view(-1, Hkv, count, G, D).transpose(1, 2).reshape(-1, count, Hq, D).to(torch.bfloat16)
        lse_out[row] = lse.view(-1, Hkv, count, G).transpose(1, 2).reshape(-1, count, Hq)
    return o_out, lse_out


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"append": _append_plain, "gather": _gather_plain, "sparse": _sparse_plain,
                "chunk": _chunk_plain}[op](state)
    import block_sparse_attention_msa_gb300 as msa
    if op == "chunk":
        return msa.chunk_attention(state["q"], state["kc"], state["vc"], state["table"], state["seq"],
                                   state["cu"], out=state["out"])
    if op == "sparse":
        return msa.paged_sparse_decode_fp8(state["q"], state["kc"], state["vc"], state["ks"], state["vs"],
                                           state["fpt"], state["lens"])
    if op == "append":
        msa.append_kv_fp8(state["k"], state["v"], state["slots"], state["kc"], state["vc"], state["ks"],
                          state["vs"])
    return msa.gather_kv_fp8(state["kc"], state["vc"], state["ks"], state["vs"], state["slots"],
                             out=state["out"])


# ------------------------------------------------------------------------------ work

def work(case):
    """Bytes and operations one pass cannot do without (expected sizes where lengths are drawn)."""
    op, Hkv = case["op"], case["Hkv"]
    if op == "append":   # rows in, quantised rows out and in again, values out
        return {"bytes": case["T"] * Hkv * 2 * (2 * D + 2 * (D + 1) + 2 * D) + 4 * (case["T"] + case["pad"]),
                "flops": 0}
    if op == "gather":
        return {"bytes": case["T"] * Hkv * 2 * (D + 1 + 2 * D) + 4 * (case["T"] + case["pad"]), "flops": 0}
    if op == "sparse":
        rows, mean = case["B"] * case["N"], (case["lo"] + case["hi"]) / 2
        keys = rows * Hkv * min(case["topk"] * PAGE - PAGE / 2, mean)
        return {"bytes": keys * 2 * (D + 1) + rows * case["Hq"] * (4 * D + 4) + rows * Hkv * (case["topk"] + 1) * 4,
                "flops": 4 * D * keys * case["Hq"] / Hkv}
    B, chunks, ctx, Hq = case["B"], case["chunks"], case["ctx"], case["Hq"]
    new = case["new"] if chunks == 1 else (max(1, case["new"] // 2) + case["new"]) / 2
    held = ctx if B == 1 or not ctx else (max(1, ctx // 4) + ctx) / 2
    tokens = chunks * new + B - chunks
    pairs = chunks * new * (held + (new + 1) / 2) + (B - chunks) * (held + 1)
    keys = B * held + tokens
    return {"bytes": keys * Hkv * D * 4 + tokens * Hq * (D * 4 + 4) + keys / PAGE * 4 + B * 8,
            "flops": 4 * D * pairs * Hq}


# ------------------------------------------------------------------------------ exact

def _e4m3_of(row):
    """Rows in 64 bits as the values that their quantised form stands for: with e the smallest
    integer for which every |x| <= 448 * 2^e (within [-127, 119]), the nearest multiple of the
    spacing of e4m3 numbers around x / 2^e, ties to even, at most 448, times 2^e."""
    a = row.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(a > 0, a, 1.0) / 448.0))
    e = torch.where(a > 448.0 * torch.exp2(e), e + 1, e)
    e = torch.where(a <= 448.0 * torch.exp2(e - 1), e - 1, e)
    e = torch.where(a > 0, e, -127.0).clamp(-127, 119)
    x = row * torch.exp2(-e)
    exp = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -20))).clamp(min=-6)
    exp = torch.where(x.abs() >= torch.exp2(exp + 1), exp + 1, exp)
    exp = torch.where((x.abs() < torch.exp2(exp)) & (exp > -6), exp - 1, exp)
    step = torch.exp2(exp - 3)
    return (torch.round(x / step) * step).clamp(-448, 448) * torch.exp2(e)


def _code_values(dev):
    """The 256 values of e4m3 by their bit patterns: sign, 4 bits of exponent (bias 7), 3 of fraction."""
    c = torch.arange(256, device=dev)
    exp, frac = ((c >> 3) & 15).double(), (c & 7).double()
    mag = torch.where(exp > 0, (1 + frac / 8) * torch.exp2(exp - 7), frac / 8 * 2.0 ** -6)
    mag[(c & 127) == 127] = float("nan")
    return torch.where(c >= 128, -mag, mag)


def exact(case, seed):
    st = prepare(case, seed)
    op, Hkv = case["op"], case["Hkv"]
    dev = st["kc"].device
    if op in ("append", "gather"):
        T = case["T"]
        outs = []
        for x in ("k", "v"):
            out = torch.zeros((T + case["pad"], Hkv, D), dtype=torch.float64, device=dev)
            if op == "append":
                out[:T] = _e4m3_of(st[x][:T].double())
            else:
                slot = st["slots"][:T].long()
                codes = st[x + "c"].view(torch.uint8)[slot // PAGE, :, slot % PAGE].long()
                power = st[x + "s"][slot // PAGE, :, slot % PAGE].double() - 127
                out[:T] = _code_values(dev)[codes] * torch.exp2(power)[..., None]
            outs.append(out)
        return tuple(outs)
    Hq = case["Hq"]
    G = Hq // Hkv
    q = st["q"].double()
    if op == "sparse":
        R = q.shape[0]
        value = _code_values(dev)
        o = torch.empty((R, Hq, D), dtype=torch.float64, device=dev)
        lse = torch.empty((R, Hq), dtype=torch.float64, device=dev)
        lens = st["lens"].view(R, Hkv).tolist()
        for r in range(R):
            for g in range(Hkv):
                n = lens[r][g]
                page = st["fpt"][r * Hkv + g, :(n + PAGE - 1) // PAGE].long() // (PAGE * Hkv)
                kv = []
                for x in ("k", "v"):
                    power = torch.exp2(st[x + "s"][page, g].double() - 127)
                    kv.append((value[st[x + "c"].view(torch.uint8)[page, g].long()] * power[..., None]).flatten(0, 1)[:n])
                s = q[r, g * G:(g + 1) * G] @ kv[0].T
                z = torch.logsumexp(s, -1)
                o[r, g * G:(g + 1) * G] = torch.exp(s - z[:, None]) @ kv[1]
                lse[r, g * G:(g + 1) * G] = z
        return o, lse
    new, seq = _chunk_lens(case, seed)
    T = q.shape[0]
    o = torch.zeros((T, Hq, D), dtype=torch.float64, device=dev)
    lse = torch.zeros((T, Hq), dtype=torch.float64, device=dev)
    row = 0
    for b in range(case["B"]):
        n, length = int(new[b]), int(seq[b])
        pages = st["table"][b, :(length + PAGE - 1) // PAGE].long()
        step = max(1, min(n, (1 << 27) // (G * length)))
        for g in range(Hkv):
            k = st["kc"][pages, :, g].flatten(0, 1)[:length].double()
            v = st["vc"][pages, :, g].flatten(0, 1)[:length].double()
            for i in range(0, n, step):
                m = min(step, n - i)
                end = length - n + i + m                                          # keys the last row sees
                rows = q[row + i:row + i + m, g * G:(g + 1) * G]
                s = torch.einsum("mhd,nd->mhn", rows, k[:end])
                limit = end - m + torch.arange(m, device=dev)
                s.masked_fill_((torch.arange(end, device=dev) > limit[:, None])[:, None], float("-inf"))
                z = torch.logsumexp(s, -1, keepdim=True)
                o[row + i:row + i + m, g * G:(g + 1) * G] = torch.einsum("mhn,nd->mhd", torch.exp(s - z), v[:end])
                lse[row + i:row + i + m, g * G:(g + 1) * G] = z.squeeze(-1)
        row += n
    return o, lse
