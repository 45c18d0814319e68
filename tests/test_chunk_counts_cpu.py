"""The inputs that count steps (``_chunk_counts``), without a GPU: what they say is what attention in 64 bits gives,
and a single step left out or taken twice is always beyond the tolerances."""
import pytest
import torch

import _chunk_counts as counts


@pytest.mark.parametrize("flat", [False, True])
def test_the_expected_outputs_are_those_of_attention(flat):
    new, held, Hq, Hkv = [3, 70, 1], [0, 100, 513], 4, 2
    w = counts.make(new, held, Hq, Hkv, seed=1, flat=flat)
    row = 0
    for b, n in enumerate(new):
        s = held[b] + n
        pages = w["table"][b, :(s + 127) // 128].long()
        k, v = (w[x][pages].flatten(0, 1)[:s].double() for x in ("kc", "vc"))
        o, lse, _, _ = counts.expected(new, held, Hkv, b, flat, "cpu")
        for i in range(n):
            vis = held[b] + i + 1
            for h in range(Hq):
                g = h // (Hq // Hkv)
                sc = k[:vis, g] @ w["q"][row + i, h].double()
                p = torch.softmax(sc, 0)
                assert ((p @ v[:vis, g]) - o[i, g]).abs().max() <= 2.0 ** -20
                assert (torch.logsumexp(sc, 0) - lse[i]).abs() <= 2.0 ** -20
        row += n


@pytest.mark.parametrize("n,flat", [(65, False), (1000, False), (16384, False), (62080, False), (1000, True),
                                    (300000, True), (1000003, True)])
def test_a_step_lost_or_taken_twice_is_beyond_the_tolerances(n, flat):
    right = counts.weights(n, 1, 1, n - 1, n, flat)[0]
    rel, tl = (x[0] for x in counts.tolerances(right.sum()[None], torch.tensor([n]), flat))
    o, z = right / right.sum(), torch.log(right.sum())
    steps = torch.arange(n // 64)         # the whole ones
    share = 64 * torch.exp2(-counts.power_of(steps, flat).double())
    channel = counts.channel_of(steps, 1, 1)
    for sign in (-1, 1):
        total = right.sum() + sign * share
        assert ((torch.log(total) - z).abs() > 2 * tl).all()
        got = (right[channel] + sign * share) / total
        # beyond, even after a rounding of the wrong value towards the right one
        if n > 200:                       # else one channel holds nearly all weight
            assert ((got - o[channel]).abs() > (rel + 2.0 ** -8) * torch.maximum(o[channel], got)).all()


def test_neighbouring_steps_have_other_weights():
    s = torch.arange(5000)
    j = counts.power_of(s, False)
    for d in range(1, 12):       # slots of a ring apart: a stale or a wrong slot's keys
        assert (j[d:] != j[:-d]).double().mean() > 0.6


def test_the_rule_that_tells_lists_from_equal_runs_is_the_library_s():
    """By the workspace: equal runs have two pieces per SM and no list."""
    import block_sparse_attention_msa_gb300 as msa
    from block_sparse_attention_msa_gb300 import build
    build.build()
    size = msa.load().msa_chunk_attention_workspace_size
    sms = torch.cuda.get_device_properties(0).multi_processor_count if torch.cuda.is_available() else 148
    up = lambda x: (x + 255) // 256 * 256
    seen = set()
    for B in (1, 7, 300, 16384):
        for T in (1, 40, 1000, 5000, 40000):
            for Hq, Hkv in ((64, 8), (8, 8), (32, 2), (16, 1)):
                for mb in (1, 500, 40000):
                    rows = min(128, (T * (Hq // Hkv) + 7) // 8 * 8)
                    equal = 256 + up(2 * sms * 32) + up(2 * sms * 2 * rows * 8) + up(2 * sms * 2 * rows * 512) \
                        + (sms * 128 * 128 * 4 if Hkv == 1 else 0)
                    lists = counts.lists_its_work(B, T, Hq, Hkv, mb, sms)
                    assert (size(B, T, Hq, Hkv, mb) != equal) == lists, (B, T, Hq, Hkv, mb)
                    seen.add(lists)
    assert seen == {True, False}
