"""Inputs for dense attention whose answer counts the steps: every 64 keys leave a mark of their own.

The keys of step s of a request have scores -j ln 2 with a small whole j(s) (or 0, `flat`), so that softmax weights
are powers of two, which every format holds exactly; their values are 1 in one channel c(s) (moved by the request and the
group) and 0 elsewhere. So o holds for each channel the weighted number of the row's keys in the channel's steps over
that of all its keys, and lse the logarithm of the latter. A step that is left out, taken twice, taken in another's
place or read with another's keys changes a channel by far more than the roundings:

  * the weights are 2^-j to 2^-18 (a score is a sum of three bf16 numbers, 2^-24 off at most, and 2^x is good to
    2^-21), and exact once they are rounded to bf16 for their product with V; products and sums of V are exact, fp32
    sums of the weights off by 2^-24 per addition of 64 keys, and 40 within and between parts: (n / 64 + 40) 2^-24;
    with flat scores they are whole numbers, and exact;
  * o is rounded to bf16 once, 2^-8 of the value at most;
  * lse: the logarithm's argument to the same sums, and 2^-22 of the value.
"""
import math

import numpy as np
import torch

PAGE, D, STEP = 128, 128, 64
POWERS = 4
KEY_CHANNELS = 3


_TABLE = torch.randint(0, POWERS, (4099,), generator=torch.Generator().manual_seed(0))


def power_of(steps, flat):
    """j of each step, at random: a slot's stale keys have another one three times of four."""
    return torch.zeros_like(steps) if flat else _TABLE.to(steps.device)[steps % len(_TABLE)]


def channel_of(steps, b, g):
    return (steps + 11 * b + 37 * g) % D


def scores(flat):
    """The bf16 parts whose sum is -j ln 2."""
    out = torch.zeros((POWERS, KEY_CHANNELS), dtype=torch.bfloat16)
    if not flat:
        for j in range(POWERS):
            rest = -j * math.log(2)
            for i in range(KEY_CHANNELS):
                out[j, i] = rest
                rest -= float(out[j, i])
    return out


def make(new, held, Hq, Hkv, seed, pad=0, flat=False, device="cpu", pages=None, mb=None, shuffle=True):
    """Requests of `held` tokens before their `new` ones, on pages in random order; what nothing uses is NaN."""
    seq = [h + n for h, n in zip(held, new)]
    blocks = [(s + PAGE - 1) // PAGE for s in seq]
    P = max(sum(blocks) + 2, pages or 0)
    mb = max(max(blocks) + 1, mb or 0)
    g = torch.Generator().manual_seed(seed)
    perm = torch.randperm(P, generator=g) if shuffle else torch.arange(P)
    table = torch.randint(0, P, (len(new), mb), generator=g).to(torch.int32)
    kc = torch.full((P, PAGE, Hkv, D), float("nan"), dtype=torch.bfloat16, device=device)
    vc = torch.full_like(kc, float("nan"))
    parts = scores(flat).to(device)
    used = 0
    for b, s in enumerate(seq):
        if s == 0:
            continue
        mine = perm[used:used + blocks[b]]
        used += blocks[b]
        table[b, :blocks[b]] = mine.to(torch.int32)
        pos = torch.arange(s, device=device)
        cell = mine.to(device)[pos // PAGE] * PAGE + pos % PAGE
        step = pos // STEP
        k = torch.zeros((s, Hkv, D), dtype=torch.bfloat16, device=device)
        k[:, :, :KEY_CHANNELS] = parts[power_of(step, flat)][:, None]
        kc.view(-1, Hkv, D)[cell] = k
        v = torch.zeros((s, Hkv, D), dtype=torch.bfloat16, device=device)
        c = channel_of(step[:, None], b, torch.arange(Hkv, device=device)[None])
        v.scatter_(2, c[..., None], 1.0)
        vc.view(-1, Hkv, D)[cell] = v
        del k, v
    cu = np.concatenate([[0], np.cumsum(new)])
    q = torch.full((int(cu[-1]) + pad, Hq, D), float("nan"), dtype=torch.bfloat16, device=device)
    q[:int(cu[-1])] = 0
    q[:int(cu[-1]), :, :KEY_CHANNELS] = 1
    i32 = lambda x: torch.from_numpy(np.array(x, dtype=np.int32)).to(device)
    return dict(q=q, kc=kc, vc=vc, table=table.to(device), seq=i32(seq), cu=i32(cu))


def weights(n, b, g, first, last, flat, device="cpu"):
    """Weighted keys by channel, [last - first, D] in 64 bits, of rows that see first + 1 .. last keys of a request of n
    tokens."""
    steps = torch.arange((n + STEP - 1) // STEP, device=device)
    w = torch.exp2(-power_of(steps, flat).double())
    one = torch.zeros((len(steps), D), dtype=torch.float64, device=device)
    one[steps, channel_of(steps, b, g)] = w
    before = torch.cat([torch.zeros((1, D), dtype=torch.float64, device=device), (STEP * one).cumsum(0)])
    seen = torch.arange(first + 1, last + 1, device=device)
    at = (seen - 1) // STEP
    return before[at] + (seen - at * STEP)[:, None] * one[at]


def tolerances(total, seen, flat):
    """Relative of o, absolute of lse, for rows that see `seen` keys of weight `total`."""
    sums = 2.0 ** -18 + (0.0 if flat else 1.0) * (seen.double() / STEP + 40) * 2.0 ** -24
    return 2.0 ** -8 + sums, sums + 2.0 ** -22 * torch.log(total).abs()


def expected(new, held, Hkv, b, flat, device):
    """o [n, Hkv, D], lse [n], and their tolerances, of request b's new tokens."""
    n, s = new[b], held[b] + new[b]
    per = [weights(s, b, g, s - n, s, flat, device) for g in range(Hkv)]
    total = per[0].sum(-1)
    seen = torch.arange(s - n + 1, s + 1, device=device)
    rel, tl = tolerances(total, seen, flat)
    o = torch.stack([x / total[:, None] for x in per], 1)
    return o, torch.log(total), rel, tl


def check(got, new, held, Hq, Hkv, flat=False):
    """Every row of every request, on the outputs' device."""
    o, lse = got
    row = 0
    for b, n in enumerate(new):
        if n == 0:
            continue
        want, z, rel, tl = expected(new, held, Hkv, b, flat, o.device)
        G = Hq // Hkv
        for i in range(0, n, 1024):
            r = slice(row + i, row + min(n, i + 1024))
            w, t = want[i:i + 1024], rel[i:i + 1024]
            err = (o[r].double().view(-1, Hkv, G, D) - w[:, :, None]).abs()
            bad = ~(err <= w[:, :, None] * t[:, None, None, None])
            assert not bad.any(), (f"request {b}: {int(bad.sum())} elements off, the first at (row, group, head, "
                                   f"channel) {(bad.nonzero()[0] + torch.tensor([i, 0, 0, 0], device=o.device)).tolist()}")
            bad = ~((lse[r].double() - z[i:i + 1024, None]).abs() <= tl[i:i + 1024, None])
            assert not bad.any(), f"request {b}: lse of {int(bad.sum())} rows and heads off"
        row += n


def lists_its_work(B, T, Hq, Hkv, mb, sms):
    """Which way a call cuts its keys (the rule of chunk_attention.cu's layout): True for a list made by the plan
    kernel, False for equal runs."""
    tpt = 128 // (Hq // Hkv)
    pairs = Hkv * (T // (2 * tpt))
    items = pairs + Hkv * min(B, T)
    equal = (T <= B * tpt or pairs <= 2 * sms) and items * ((2 * mb + 1) * 7 + 7) <= 2 ** 31 - 1
    return not equal
