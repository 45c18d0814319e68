"""Inputs for long shared-prefix decodes whose answers show every 64-key step, and what they must be.

On random values the softmax averages over so many keys that a step more or less stays within any
honest tolerance. Two kinds of input show it:

``counting``: q = 0, so every visible key has weight 1/n, and V marks the key's step in two of the
128 channels: step % 64 and 64 + step // 64. o is then count / n per channel, with at most 64 steps
(256 K keys) sharing a channel, and lse = log n. All of P, l and O are whole numbers below 2^24, hence
exact, and 2^0 = 1. Left are, for o, its rounding to bf16 (2^-8) and 1/l and the product (2^-23): a
step missing from a channel of at most 64 changes it by 2^-6. For lse, log2f is off by one unit of
the last place at most, 2^-19 for values below 32, its product with ln 2 by 2^-24 and the constant
by 2^-25 of 12: together 1.4e-6 + 1.1e-6, tolerance 4e-6. One key of 71000 is 1.4e-5.

``pointing``: K holds the code of its position, +-1 in 17 bits, five times, in private keys that of
their request too, 7 bits, five times. A row's q is 4 times the code of one position, so its own
score is 4 * 85 (4 * 120 for a private one) and every other at least 40 lower: the weights of all others
together are below 17 * 2 * e^-40 < 1e-15. o is that key's V, the same codes as +-1 (0 for the request
of a shared key). P is rounded to bf16 (2^-8; its reference may be below the maximum, so P need not be
1) and o once more (2^-8), the sums are off by 2^-21: (2^-7)(1 + 2^-6). lse is the score: the dot product
is exact, the scaling to log2 units and back are fp32 products and a log2f, below 2^-20 of it. A step
that is missing loses the row's key, one that counts twice adds log 2 to lse. Each group has its own
signs, which both K and q carry."""
import torch

PAGE, STEP, D, BITS, REQ_BITS, REPEAT = 128, 64, 128, 17, 7, 5
A = 4.0


def bits(x, n):
    """+-1 code of whole numbers."""
    return ((x[..., None] >> torch.arange(n, device=x.device)) & 1).float() * 2 - 1


def layout(B, shared, lens, seed, device):
    """Page tables of requests of lens[b] keys behind `shared` common ones: (table, pages)."""
    g = torch.Generator().manual_seed(seed)
    whole = shared // PAGE
    mb = (max(lens) + PAGE - 1) // PAGE
    pages = whole + B * (mb - whole)
    perm = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.empty((B, mb), dtype=torch.int32)
    table[:, :whole] = perm[:whole]
    table[:, whole:] = perm[whole:].view(B, mb - whole)
    return table.to(device), pages


def fill(table, pages, shared, Hkv, rows):
    """A cache [pages, 128, Hkv, D] whose cell of request b's key n holds rows(b, n) [len(n), Hkv, D]."""
    B, mb = table.shape
    cache = torch.zeros((pages, PAGE, Hkv, D), dtype=torch.bfloat16, device=table.device)
    for b in range(B):
        first = 0 if b == 0 else shared // PAGE
        n = torch.arange(first * PAGE, mb * PAGE, device=table.device)
        cache[table[b, first:].long()] = rows(b, n).to(torch.bfloat16).view(mb - first, PAGE, Hkv, D)
    return cache


def signs(Hkv, device):
    g = torch.Generator().manual_seed(5)
    return (torch.randint(0, 2, (Hkv, D), generator=g).float() * 2 - 1).to(device)


def key_codes(b, n, shared):
    """[..., D]: the codes of position n and, for private keys, of request b."""
    out = torch.zeros((*n.shape, D), device=n.device)
    out[..., :BITS * REPEAT] = bits(n, BITS).repeat_interleave(REPEAT, -1)
    req = bits(b, REQ_BITS).repeat_interleave(REPEAT, -1) * (n >= shared)[..., None]
    out[..., BITS * REPEAT:(BITS + REQ_BITS) * REPEAT] = req
    return out


def value_codes(b, n, shared, g):
    b, n, g = torch.broadcast_tensors(b, n, g)
    out = torch.zeros((*n.shape, D), device=n.device)
    out[..., :BITS] = bits(n, BITS)
    out[..., BITS:BITS + REQ_BITS] = bits(b, REQ_BITS) * (n >= shared)[..., None]
    out[..., BITS + REQ_BITS:BITS + REQ_BITS + 4] = bits(g, 4)
    return out


def lengths(B, shared, own, N):
    """own down to own // 2 private keys, the first request the longest."""
    return [shared + own - (b * 37) % (own // 2 + 1) for b in range(B)]


def visible(lens, N, device):
    """Keys that row b*N + i sees: [B, N]."""
    return torch.tensor(lens, device=device)[:, None] - N + 1 + torch.arange(N, device=device)


# ------------------------------------------------------------------------------ counting

def private_weight(b):
    return 1 + b % 7


def counting(B, N, Hq, Hkv, shared, own, device):
    lens = lengths(B, shared, own, N)
    table, pages = layout(B, shared, lens, 1, device)

    def values(b, n):
        step = n // STEP
        v = torch.zeros((len(n), D), device=n.device)
        w = 1.0 + (private_weight(b) - 1) * (n >= shared).float()
        v.scatter_(1, (step % 64)[:, None], w[:, None])
        v.scatter_(1, (64 + step // 64)[:, None], w[:, None])
        return v[:, None, :].expand(-1, Hkv, -1)

    g = torch.Generator(device=device).manual_seed(2)
    kc = torch.randn((pages, PAGE, Hkv, D), generator=g, device=device).to(torch.bfloat16)
    return dict(q=torch.zeros((B * N, Hq, D), dtype=torch.bfloat16, device=device), kc=kc,
                vc=fill(table, pages, shared, Hkv, values), table=table, lens=lens, N=N, shared=shared)


def check_counting(w, o, lse):
    B, N = len(w["lens"]), w["N"]
    dev = o.device
    vis = visible(w["lens"], N, dev)                                   # [B, N]
    steps = torch.arange((max(w["lens"]) + STEP - 1) // STEP, device=dev)
    here = (vis[..., None] - steps * STEP).clamp(0, STEP)             # visible keys of a step
    own = (vis[..., None] - (steps * STEP).clamp(min=w["shared"])).clamp(min=0)
    own = torch.minimum(own, (steps * STEP + STEP - w["shared"]).clamp(0, STEP))   # ... private ones
    extra = torch.tensor([private_weight(b) - 1 for b in range(B)], device=dev)[:, None, None]
    count = (here + own * extra).double()
    want = torch.zeros((B, N, D), dtype=torch.float64, device=dev)
    want.index_add_(2, steps % 64, count)
    want.index_add_(2, 64 + steps // 64, count)
    want = (want / vis[..., None]).view(B * N, 1, D)
    err = (o.double() - want).abs()
    assert (err <= want * (2.0 ** -8 + 2.0 ** -15)).all(), "a step counts too often or not at all"
    err = (lse.double() - vis.double().log().view(B * N, 1)).abs()
    assert (err <= 4e-6).all(), f"lse is {float(err.max()):.2g} off the log of the number of keys"


# ------------------------------------------------------------------------------ pointing

def pointing(B, N, Hq, Hkv, shared, own, device):
    lens = lengths(B, shared, own, N)
    table, pages = layout(B, shared, lens, 3, device)
    sg = signs(Hkv, device)
    groups = torch.arange(Hkv, device=device)
    req = lambda b, n: torch.full_like(n, b)
    kc = fill(table, pages, shared, Hkv, lambda b, n: key_codes(req(b, n), n, shared)[:, None, :] * sg)
    vc = fill(table, pages, shared, Hkv,
              lambda b, n: value_codes(req(b, n)[:, None], n[:, None], shared, groups))
    return dict(kc=kc, vc=vc, table=table, lens=lens, N=N, shared=shared, Hq=Hq, Hkv=Hkv, sg=sg)


def borders(w, device):
    """First and last key of every step, and the last key of all."""
    s = torch.arange((max(w["lens"]) + STEP - 1) // STEP, device=device) * STEP
    return torch.cat([s, s + STEP - 1])


def point_at(w, turn, device):
    """Queries of a call: (q, the position that each row points at [R, Hkv, G]). The turns together
    point at every border from each request and group; a row that does not see its border points at
    the last key that it sees."""
    B, N, Hq, Hkv = len(w["lens"]), w["N"], w["Hq"], w["Hkv"]
    G = Hq // Hkv
    at = borders(w, device)
    rows = torch.arange(N * G, device=device).view(1, N, 1, G).expand(B, N, Hkv, G)
    pos = at[(turn * N * G + rows) % len(at)]
    pos = torch.minimum(pos, visible(w["lens"], N, device)[:, :, None, None] - 1)
    b = torch.arange(B, device=device)[:, None, None, None].expand_as(pos)
    q = A * key_codes(b, pos, w["shared"]) * w["sg"][:, None, :]
    return q.reshape(B * N, Hq, D).to(torch.bfloat16), pos


def turns(w):
    G = w["Hq"] // w["Hkv"]
    return (len(borders(w, "cpu")) + w["N"] * G - 1) // (w["N"] * G)


def check_pointing(w, pos, o, lse):
    B, N, Hkv, G = pos.shape
    b = torch.arange(B, device=pos.device)[:, None, None, None].expand_as(pos)
    g = torch.arange(Hkv, device=pos.device)[:, None].expand_as(pos)
    want = value_codes(b, pos, w["shared"], g).view(B * N, Hkv * G, D)
    err = (o.float() - want).abs()
    assert (err <= 2.0 ** -7 * (1 + 2.0 ** -6) * want.abs() + 2.0 ** -20).all(), "a row got another key's values"
    score = A * (BITS * REPEAT + REQ_BITS * REPEAT * (pos >= w["shared"])).view(B * N, Hkv * G)
    err = (lse.float() - score).abs()
    assert (err <= 2.0 ** -20 * score).all(), f"lse is {float(err.max()):.2g} off the one key's score"
