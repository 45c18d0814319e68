"""Measured cases of the serving-batch operators: page tables and slot maps built on the GPU,
the append of new tokens to the paged caches, and decode attention for a batch whose requests
share a prefix.

``run`` computes an operator either in its plain form (elementary torch operations, fp32) or
through the package's entry points (``own = True``); ``exact`` computes the same outputs in 64
bits straight from the definitions. Layouts, names and conventions are those of the package:
128-token pages, caches [num_pages, 128, Hkv, D] bf16, a page table [B, max_blocks] int32, and
query rows b*N + i at the last N positions of request b.
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
        # one decode step of eight long requests (8 x 60032 tokens): every request gets one token,
        # some cross into a new page
        dict(name="tables_decode_8", op="tables", B=8, ctx=60032, new_max=1, shared_pages=0,
             max_blocks=512),
        # a scheduler step that mixes prompt chunks of many lengths (about 32768 tokens), token rows
        # padded to the step's capacity as a captured step does
        dict(name="tables_chunks_32k", op="tables", B=61, ctx=20000, new_max=1073, shared_pages=0,
             max_blocks=1024),
        # admission of a large batch behind one cached 32768-token prompt
        dict(name="tables_admit_512_shared", op="tables", B=512, ctx=0, new_max=513,
             shared_pages=256, max_blocks=1024),
        # one decode step: the new tokens of eight requests
        dict(name="append_decode_8", op="append", T=8, pad=0, Hkv=8, Di=128, pages=480),
        # a ragged step padded to a captured size (rows behind the last token carry slot -1)
        dict(name="append_ragged_1777", op="append", T=1777, pad=271, Hkv=4, Di=64, pages=96),
        # a 32768-token prefill chunk
        dict(name="append_chunk_32768", op="append", T=32768, pad=0, Hkv=8, Di=128, pages=300),
        # one request of the small layer (Hq 8, Hkv 2) behind a short prefix: latency only
        dict(name="decode_tiny_1x2048", op="decode", B=1, N=1, Hq=8, Hkv=2, shared=1000,
             suffix=1048, ragged=False),
        # agentic traffic: a 60K prefix cache and eight concurrent requests
        dict(name="decode_8_on_60k", op="decode", B=8, N=1, Hq=64, Hkv=8, shared=60032,
             suffix=512, ragged=True),
        # speculative verify: four rows per request, odd lengths
        dict(name="verify_16x4_on_20011", op="decode", B=16, N=4, Hq=64, Hkv=8, shared=20011,
             suffix=777, ragged=True),
        # many requests with long private parts behind a short system prompt
        dict(name="decode_64_private_8k", op="decode", B=64, N=1, Hq=64, Hkv=8, shared=2000,
             suffix=8192, ragged=True),
        # 64 requests on one 64K document
        dict(name="decode_64_on_64k", op="decode", B=64, N=1, Hq=64, Hkv=8, shared=65536,
             suffix=2048, ragged=True),
        # a full serving batch on a 32K prompt
        dict(name="decode_256_on_32k", op="decode", B=256, N=1, Hq=64, Hkv=8, shared=32768,
             suffix=1024, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    """One more case of the listed ranges; a decode draw stays within the largest listed cost."""
    op = rng.choice(["tables", "append", "decode", "decode"])
    if op == "tables":
        shared = rng.choice([0, 0, _log_int(rng, 1, 256)])
        B = _log_int(rng, 1, 512)
        new_max = min(_log_int(rng, 1, 1073), max(1, 2 * 131328 // B))
        ctx = 0 if shared else _log_int(rng, 1, 60032)
        return dict(op=op, B=B, ctx=ctx, new_max=new_max, shared_pages=shared, max_blocks=1024)
    if op == "append":
        Hkv = rng.choice([1, 2, 4, 8, 16])
        T = _log_int(rng, 1, 32768 * 8 // max(Hkv, 8))
        return dict(op=op, T=T, pad=rng.choice([0, 0, rng.randint(1, 300)]), Hkv=Hkv,
                    Di=rng.choice([64, 128]), pages=T // PAGE + rng.randint(2, 60))
    while True:
        Hkv = rng.choice([1, 2, 4, 8, 8, 16])
        G = rng.choice([1, 2, 4, 8, 8, 16])
        c = dict(op=op, B=_log_int(rng, 1, 256), N=rng.choice([1, 1, 1, 2, 4, rng.randint(2, 16)]),
                 Hq=Hkv * G, Hkv=Hkv, shared=_log_int(rng, 1, 65536),
                 suffix=_log_int(rng, 1, 8192), ragged=rng.random() < 0.8)
        c["suffix"] = max(c["suffix"], c["N"])
        pairs = c["B"] * c["N"] * c["Hq"] * (c["shared"] + c["suffix"])
        tokens = (c["shared"] + c["B"] * c["suffix"]) * Hkv
        if pairs <= 256 * 64 * 33000 and tokens <= (2000 + 64 * 8192) * 8:
            return c


# ------------------------------------------------------------------------------ inputs

def _suffix_lens(case, gen):
    """Private tokens of each request: uniform in [N, suffix], or all equal."""
    B, N, hi = case["B"], case["N"], case["suffix"]
    if not case["ragged"]:
        return torch.full((B,), hi, dtype=torch.int64)
    return torch.randint(N, hi + 1, (B,), generator=gen)


def _tables_lens(case, gen):
    B = case["B"]
    new = torch.randint(1, case["new_max"] + 1, (B,), generator=gen)
    if case["shared_pages"]:
        prev = torch.full((B,), case["shared_pages"] * PAGE, dtype=torch.int64)
    else:
        prev = torch.randint(max(1, case["ctx"] // 2), case["ctx"] + 1, (B,), generator=gen)
    return prev, new


def _host_gen(seed):
    return torch.Generator().manual_seed(int(seed))


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed) + 1)
    hgen = _host_gen(seed)
    st = {"case": dict(case)}
    if case["op"] == "tables":
        prev, new = _tables_lens(case, hgen)
        B, mb, S = case["B"], case["max_blocks"], case["shared_pages"]
        held = (prev + PAGE - 1) // PAGE
        need = (prev + new + PAGE - 1) // PAGE - held
        own_held = 0 if S else int(held.sum())
        pages = S + own_held + int(need.sum()) + 64
        perm = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
        table = torch.full((B, mb), -1, dtype=torch.int32, device=dev)
        if not S:
            cols = torch.arange(mb, device=dev)
            mask = cols[None, :] < held.to(dev)[:, None]
            table[mask] = perm[S:S + own_held]
        st.update(table=table, prev=prev.to(dev, torch.int32), new=new.to(dev, torch.int32),
                  free=perm[S + own_held:].contiguous(),
                  used=torch.tensor([5], dtype=torch.int32, device=dev), T=B * case["new_max"],
                  num_pages=pages, shared=perm[:S].contiguous() if S else None)
        return st
    if case["op"] == "append":
        T, Hkv, Di, P = case["T"], case["Hkv"], case["Di"], case["pages"]
        rows = T + case["pad"]
        # k and v as the projection leaves them: slices of one [rows, (G + 2) * Hkv * D] matrix
        qkv = torch.randn((rows, 4 * Hkv * D), generator=gen, device=dev).to(torch.bfloat16)
        st["k"] = qkv[:, 2 * Hkv * D:3 * Hkv * D].unflatten(1, (Hkv, D))
        st["v"] = qkv[:, 3 * Hkv * D:].unflatten(1, (Hkv, D))
        st["k_idx"] = torch.randn((rows, Hkv, Di), generator=gen, device=dev).to(torch.bfloat16)
        slots = torch.full((rows,), -1, dtype=torch.int32, device=dev)
        order = torch.randperm(P, generator=gen, device=dev)
        t = torch.arange(T, device=dev)
        start = 37 % (P * PAGE - T) if P * PAGE > T else 0
        pos = t + start
        slots[:T] = (order[pos // PAGE] * PAGE + pos % PAGE).to(torch.int32)
        st["slots"] = slots
        st["kc"] = torch.zeros((P, PAGE, Hkv, D), dtype=torch.bfloat16, device=dev)
        st["vc"] = torch.zeros((P, PAGE, Hkv, D), dtype=torch.bfloat16, device=dev)
        st["ic"] = torch.zeros((P, PAGE, Hkv, Di), dtype=torch.bfloat16, device=dev)
        return st
    B, N, Hq, Hkv, shared = (case[x] for x in ("B", "N", "Hq", "Hkv", "shared"))
    suffix = _suffix_lens(case, hgen)
    seq = shared + suffix
    whole = shared // PAGE                       # pages every request shares
    blocks = (seq + PAGE - 1) // PAGE
    private = blocks - whole                     # a partly filled shared page is a private copy
    pages = whole + int(private.sum()) + 3
    perm = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    mb = int(blocks.max())
    table = torch.zeros((B, mb), dtype=torch.int32, device=dev)
    table[:, :whole] = perm[:whole]
    cols = torch.arange(mb, device=dev)[None, :]
    table[(cols >= whole) & (cols < blocks.to(dev)[:, None])] = perm[whole:pages - 3]
    kc = torch.randn((pages, PAGE, Hkv, D), generator=gen, device=dev, dtype=torch.bfloat16)
    vc = torch.randn((pages, PAGE, Hkv, D), generator=gen, device=dev, dtype=torch.bfloat16)
    if shared % PAGE:                            # the copies of the partly filled page agree
        tail = table[:, whole].long()
        kc[tail, :shared % PAGE] = kc[tail[0], :shared % PAGE].clone()
        vc[tail, :shared % PAGE] = vc[tail[0], :shared % PAGE].clone()
    q = torch.randn((B * N, Hq, D), generator=gen, device=dev) * D ** -0.5
    st.update(q=q.to(torch.bfloat16), kc=kc, vc=vc, table=table, seq=seq.to(dev, torch.int32),
              shared_len=torch.tensor([shared], dtype=torch.int32, device=dev),
              shared=shared, max_suffix=int(suffix.max()))
    return st


# ------------------------------------------------------------------------------ passes

def _tables_plain(st):
    table, free, used, T = st["table"], st["free"], st["used"], st["T"]
    prev, new = st["prev"].long(), st["new"].long()
    B, mb = table.shape
    seq = prev + new
    held = (prev + PAGE - 1) // PAGE
    upto = (seq + PAGE - 1) // PAGE
    need = upto - held
    first = used.long() + need.cumsum(0) - need
    cols = torch.arange(mb, device=table.device)[None, :]
    if st["shared"] is not None:
        table[:, :st["shared"].numel()] = st["shared"]
    fresh = (cols >= held[:, None]) & (cols < upto[:, None])
    take = (first[:, None] + cols - held[:, None]).clamp(0, free.numel() - 1)
    table.copy_(torch.where(fresh, free[take], table))
    cu = torch.zeros(B + 1, dtype=torch.int64, device=table.device)
    cu[1:] = new.cumsum(0)
    t = torch.arange(T, device=table.device)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=B - 1)
    live = t < cu[-1]
    pos = torch.where(live, prev[b] + t - cu[b], 0)
    slot = table[b, pos // PAGE].long() * PAGE + pos % PAGE
    i32 = torch.int32
    return (table, seq.to(i32), cu.to(i32), torch.where(live, slot, -1).to(i32),
            torch.where(live, pos, -1).to(i32), (used.long() + need.sum()).to(i32))


def _append_plain(st):
    live = st["slots"] >= 0
    # padding rows write the first live row once more, so that no row needs a host decision
    first = torch.argmax(live.to(torch.int32))
    src = torch.where(live, torch.arange(live.numel(), device=live.device), first)
    dst = st["slots"].long()[src]
    for cache, rows in ((st["kc"], st["k"]), (st["vc"], st["v"]), (st["ic"], st["k_idx"])):
        cache.view(-1, *cache.shape[2:])[dst] = rows[src]
    return st["kc"], st["vc"], st["ic"]


def _decode_plain(st):
    """Two parts joined by their log-sum-exps: the shared keys once for all rows, then every
    request's own keys (padded to the longest)."""
    c = st["case"]
    N, Hkv, S = c["N"], c["Hkv"], st["shared"]
    q, table, seq = st["q"], st["table"], st["seq"].long()
    R, Hq, _ = q.shape
    B, G = R // N, Hq // Hkv
    dev = q.device
    kc = st["kc"].view(-1, Hkv, D)
    vc = st["vc"].view(-1, Hkv, D)
    qf = q.float().view(R, Hkv, G, D)
    qpos = (seq[:, None] - N + torch.arange(N, device=dev)[None, :])           # [B, N]
    # shared part: [Hkv, R*G, S]
    t = torch.arange(S, device=dev)
    rows = table[0, t // PAGE].long() * PAGE + t % PAGE
    qs = qf.permute(1, 0, 2, 3).reshape(Hkv, R * G, D)
    s1 = torch.matmul(qs, kc[rows].float().permute(1, 2, 0))
    m1 = s1.amax(-1, keepdim=True)
    s1 = torch.exp(s1 - m1)
    l1 = s1.sum(-1, keepdim=True)
    o1 = torch.matmul(s1, vc[rows].float().transpose(0, 1))
    del s1
    back = lambda x: x.view(Hkv, B, N, G, -1).permute(1, 2, 0, 3, 4)           # [B, N, Hkv, G, .]
    m1, l1, o1 = back(m1), back(l1), back(o1)
    # private part: [B, Hkv, N*G, M], a few requests at a time
    M = st["max_suffix"]
    step = max(1, (1 << 19) // (M * Hkv // 4 + 1))
    parts = []
    for b0 in range(0, B, step):
        b1 = min(B, b0 + step)
        pos = S + torch.arange(M, device=dev)[None, :].expand(b1 - b0, M)
        held = pos < seq[b0:b1, None]
        cell = torch.where(held, pos, S)
        rows = table[b0:b1].gather(1, cell // PAGE).long() * PAGE + cell % PAGE
        qp = qf.view(B, N, Hkv, G, D)[b0:b1].permute(0, 2, 1, 3, 4).reshape(b1 - b0, Hkv, N * G, D)
        s2 = torch.matmul(qp, kc[rows].float().permute(0, 2, 3, 1)).view(b1 - b0, Hkv, N, G, M)
        seen = pos[:, None, :] <= qpos[b0:b1, :, None]                           # [b, N, M]
        s2 = torch.where(seen[:, None, :, None, :], s2, float("-inf"))
        m2 = s2.amax(-1, keepdim=True)
        p2 = torch.exp(s2 - m2)
        l2 = p2.sum(-1, keepdim=True)
        o2 = torch.matmul(p2.view(b1 - b0, Hkv, N * G, M), vc[rows].float().transpose(1, 2))
        o2 = o2.view(b1 - b0, Hkv, N, G, D)
        parts.append([x.permute(0, 2, 1, 3, 4) for x in (m2, l2, o2)])
    m2, l2, o2 = (torch.cat(x) for x in zip(*parts))
    m = torch.maximum(m1, m2)
    w1, w2 = torch.exp(m1 - m), torch.exp(m2 - m)
    l = l1 * w1 + l2 * w2
    o = (o1 * w1 + o2 * w2) / l
    return o.reshape(R, Hq, D).to(torch.bfloat16), (m + torch.log(l)).reshape(R, Hq)


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"tables": _tables_plain, "append": _append_plain, "decode": _decode_plain}[op](state)
    import block_sparse_attention_msa_gb300 as msa
    if op == "tables":
        seq, cu, slots, pos, used = msa.build_page_tables(
            state["prev"], state["new"], state["table"], state["free"], state["used"],
            T=state["T"], num_pages=state["num_pages"], shared_pages=state["shared"])
        return state["table"], seq, cu, slots, pos, used
    if op == "append":
        msa.append_kv(state["k"], state["v"], state["k_idx"], state["slots"], state["kc"],
                      state["vc"], state["ic"])
        return state["kc"], state["vc"], state["ic"]
    return msa.shared_prefix_decode(state["q"], state["kc"], state["vc"], state["table"],
                                    state["seq"], state["shared_len"], N=state["case"]["N"])


# ------------------------------------------------------------------------------ work

def work(case):
    """Bytes and operations one pass cannot do without (expected sizes where lengths are drawn)."""
    if case["op"] == "tables":
        B, T = case["B"], case["B"] * case["new_max"]
        live = case["B"] * (case["new_max"] + 1) / 2
        fresh = live / PAGE + (B * 0.5 if not case["shared_pages"] else 0)
        ints = 2 * B + 1 + fresh * 2 + case["shared_pages"] * (B + 1) + B + (B + 1) + 2 * T + 1
        if not case["shared_pages"]:
            ints += B                            # the partly filled page of each request
        return {"bytes": 4 * ints, "flops": 0}
    if case["op"] == "append":
        row = case["Hkv"] * (2 * D + case["Di"]) * 2
        return {"bytes": case["T"] * row * 2 + 4 * (case["T"] + case["pad"]), "flops": 0}
    B, N, Hq, Hkv = (case[x] for x in ("B", "N", "Hq", "Hkv"))
    mean = case["suffix"] if not case["ragged"] else (N + case["suffix"]) / 2
    keys = case["shared"] + B * mean
    rows = B * N * Hq
    return {"bytes": keys * Hkv * D * 4 + rows * (D * 4 + 4) + B * 4 + keys / PAGE * 4 + 4,
            "flops": 4 * D * rows * (case["shared"] + mean - (N - 1) / 2)}


# ------------------------------------------------------------------------------ exact

def exact(case, seed):
    st = prepare(case, seed)
    dev = st["table"].device if "table" in st else st["slots"].device
    if case["op"] == "tables":
        table = st["table"].cpu().numpy().copy()
        prev, new = st["prev"].cpu().numpy(), st["new"].cpu().numpy()
        free, used = st["free"].cpu().numpy(), int(st["used"])
        T = st["T"]
        slots, pos = [-1] * T, [-1] * T
        cu = [0]
        for b in range(case["B"]):
            if st["shared"] is not None:
                table[b, :case["shared_pages"]] = st["shared"].cpu().numpy()
            for i in range(int(new[b])):
                p = int(prev[b]) + i
                if p % PAGE == 0:                # the token opens a page
                    table[b, p // PAGE] = free[used]
                    used += 1
                slots[cu[-1] + i] = int(table[b, p // PAGE]) * PAGE + p % PAGE
                pos[cu[-1] + i] = p
            cu.append(cu[-1] + int(new[b]))
        as_i32 = lambda x: torch.as_tensor(x, dtype=torch.int32).to(dev)
        return (as_i32(table), as_i32(prev + new), as_i32(cu), as_i32(slots), as_i32(pos),
                as_i32([used]))
    if case["op"] == "append":
        caches = []
        live = torch.nonzero(st["slots"] >= 0).flatten()
        for cache, rows in ((st["kc"], st["k"]), (st["vc"], st["v"]), (st["ic"], st["k_idx"])):
            flat = cache.double().view(-1, *cache.shape[2:])
            flat.index_copy_(0, st["slots"][live].long(), rows[live].double())
            caches.append(flat.view(cache.shape))
        return tuple(caches)
    N, Hq, Hkv = case["N"], case["Hq"], case["Hkv"]
    G = Hq // Hkv
    q, table, seq = st["q"], st["table"], st["seq"].tolist()
    R = q.shape[0]
    if R * Hq * (case["shared"] + case["suffix"]) > 256 * 64 * 40000:
        return None
    o = torch.empty((R, Hq, D), dtype=torch.float64, device=dev)
    lse = torch.empty((R, Hq), dtype=torch.float64, device=dev)
    for b, n in enumerate(seq):
        pages = table[b, :(n + PAGE - 1) // PAGE].long()
        k = st["kc"][pages].flatten(0, 1)[:n].double().permute(1, 2, 0)          # [Hkv, D, n]
        v = st["vc"][pages].flatten(0, 1)[:n].double().transpose(0, 1)           # [Hkv, n, D]
        qb = q[b * N:(b + 1) * N].double().view(N, Hkv, G, D)
        for i in range(N):
            vis = n - N + i + 1
            s = qb[i] @ k[:, :, :vis]                                            # [Hkv, G, vis]
            z = torch.logsumexp(s, -1, keepdim=True)
            o[b * N + i] = (torch.exp(s - z) @ v[:, :vis]).reshape(Hq, D)
            lse[b * N + i] = z.reshape(Hq)
    return o, lse
