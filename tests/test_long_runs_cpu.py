"""The long-run inputs of the shared-prefix decode see the mistakes that they are made for: an exact
answer passes their checks, one with a step left out, taken twice or read from a wrong place does not.
The mistakes are made here, in a plain 64-bit answer."""
import pytest
import torch

import _long_runs as lr

CASES = [(1, 1, 2, 2, 0, 45000), (2, 1, 4, 2, 40000, 100), (1, 1, 8, 1, 70001, 333), (2, 4, 4, 2, 20011, 300)]


def answer(w, q, cells=None, v_cells=None, drop=(), twice=()):
    """o, lse of the rows in 64 bits. cells(b, n), v_cells(b, n): where key n of request b is read
    (default: through the table); drop, twice: keys that are left out or counted twice."""
    N, table = w["N"], w["table"].long()
    R, Hq, D = q.shape
    kc, vc = (w[c].flatten(0, 1) for c in ("kc", "vc"))
    Hkv = kc.shape[1]
    G = Hq // Hkv
    plain = lambda b, n: table[b, n // lr.PAGE] * lr.PAGE + n % lr.PAGE
    o, lse = torch.zeros((R, Hq, D), dtype=torch.float64), torch.zeros((R, Hq), dtype=torch.float64)
    for b, length in enumerate(w["lens"]):
        n = torch.arange(length)
        at = (cells or plain)(b, n)
        k = kc[at].double()
        v = vc[(v_cells or cells or plain)(b, n)].double()
        mass = torch.ones(length, dtype=torch.float64)
        mass[list(drop)] = 0
        mass[list(twice)] = 2
        for i in range(N):
            vis = length - N + i + 1
            for g in range(Hkv):
                s = q[b * N + i, g * G:(g + 1) * G].double() @ k[:vis, g].T
                m = s.amax(1, keepdim=True)
                p = torch.exp(s - m) * mass[:vis]
                l = p.sum(1, keepdim=True)
                o[b * N + i, g * G:(g + 1) * G] = p @ v[:vis, g] / l
                lse[b * N + i, g * G:(g + 1) * G] = (m + l.log())[:, 0]
    return o.to(torch.bfloat16), lse.float()


def wrong_page(w, page, other):
    """Cells when block `page` of request 0 is read from block `other`."""
    table = w["table"].long().clone()
    table[0, page] = table[0, other]
    return lambda b, n: table[b, n // lr.PAGE] * lr.PAGE + n % lr.PAGE


def mistakes(case, w):
    n = min(w["lens"])
    last = n // lr.PAGE - 1
    step = lambda i: range(i * lr.STEP, (i + 1) * lr.STEP)
    return {
        "a step left out": dict(drop=step(33)), "the first step left out": dict(drop=step(0)),
        "the last whole step left out": dict(drop=step((n - w["N"]) // lr.STEP - 1)),
        "a step twice": dict(twice=step(32)),
        "a wrong page": dict(cells=wrong_page(w, 16, 17)), "a page of steps 32 pages later": dict(
            cells=wrong_page(w, 16, 48)),
        "the first page for a late one": dict(cells=wrong_page(w, last, 0)),
        "values of a wrong page": dict(v_cells=wrong_page(w, 31, 30)),
    }


def seen(check, *args):
    try:
        check(*args)
    except AssertionError:
        return True
    return False


@pytest.mark.parametrize("case", CASES)
def test_counting(case):
    w = lr.counting(*case, "cpu")
    lr.check_counting(w, *answer(w, w["q"]))
    for name, how in [*mistakes(case, w).items(), ("one key left out", dict(drop=[4321])),
                      ("the first key twice", dict(twice=[0]))]:
        assert seen(lr.check_counting, w, *answer(w, w["q"], **how)), name


@pytest.mark.parametrize("case", CASES)
def test_pointing(case):
    w = lr.pointing(*case, "cpu")
    at = lr.borders(w, "cpu").tolist()
    rows = w["N"] * w["Hq"] // w["Hkv"]
    for turn in (0, lr.turns(w) // 2, lr.turns(w) - 1):
        q, pos = lr.point_at(w, turn, "cpu")
        lr.check_pointing(w, pos, *answer(w, q))
    wrong = {**mistakes(case, w), "keys of a wrong page": dict(cells=wrong_page(w, 16, 17),
                                                             v_cells=wrong_page(w, 16, 16))}
    for name, how in wrong.items():
        # some turn points at a key that the mistake touches
        touched = {"a step left out": 33, "the first step left out": 0, "a step twice": 32,
                   "the last whole step left out": (min(w["lens"]) - w["N"]) // lr.STEP - 1,
                   "values of a wrong page": 62, "the first page for a late one":
                       2 * (min(w["lens"]) // lr.PAGE - 1)}.get(name, 32)
        q, pos = lr.point_at(w, at.index(touched * lr.STEP) // rows, "cpu")
        assert seen(lr.check_pointing, w, pos, *answer(w, q, **how)), name


def test_the_turns_point_at_every_border():
    w = lr.pointing(2, 4, 4, 2, 2011, 300, "cpu")
    seen = [set() for _ in range(2)]
    for t in range(lr.turns(w)):
        pos = lr.point_at(w, t, "cpu")[1]
        for b in range(2):
            seen[b] |= set(pos[b, :, 0].flatten().tolist())
    for b, n in enumerate(w["lens"]):
        # rows that do not see a border of the last step point at their own last key
        assert {x for x in lr.borders(w, "cpu").tolist() if x <= n - w["N"]} <= seen[b]
        assert max(seen[b]) <= n - 1
