"""verify_drafts: u times the total is rounded once to fp64, whatever the total is."""
from fractions import Fraction

import pytest

import paged_kv_prep_gb300 as pkv

torch = pytest.importorskip("torch")


def row(n1, n2, run, low, extra):
    """n1 weights of 1, `run` of `low` * 2^-40 and one of `extra` * 2^-40, n2 of 1: the weights, and their sums in
    multiples of 2^-40."""
    small = torch.tensor([low, extra], dtype=torch.float64) * 2.0 ** -40
    w = torch.ones(n1 + run + 1 + n2, dtype=torch.float32)
    w[n1:n1 + run], w[n1 + run] = small[0], small[1]
    assert torch.equal(w[n1:n1 + run].double().unique(), small[:1]) and float(w[n1 + run]) == float(small[1])
    return w, n1 << 40, run * low + extra, n2 << 40


def token_of(aim, n1, first, low, run):
    """The first token whose running sum exceeds the aim, which lies in the run."""
    assert first <= aim < first + run * low
    return n1 + (aim - first) // low


def cases():
    """Totals just above 2^60, whose fp64 neighbours are 2^8 apart, with an aim in a run of weights of 2^5 where rounding
    the total first would give another token: (weights, u, the token)."""
    found = []
    gen = torch.Generator().manual_seed(3)
    total_ones = 1 << 20
    while len(found) < 6:
        n1 = int(torch.randint(total_ones // 2, total_ones, (1,), generator=gen))
        run, low = 1 << 19, 32
        extra = int(torch.randint(1, 1 << 20, (1,), generator=gen))
        n2 = total_ones - n1
        u = Fraction(n1, total_ones)
        total = (total_ones << 40) + run * low + extra
        once = int(float(u * total))                         # float() of a fraction rounds once, to nearest even
        twice = int(float(u) * float(total))
        a, b = (token_of(x, n1, n1 << 40, low, run) for x in (once, twice))
        if a != b:
            w, *_ = row(n1, n2, run, low, extra)
            found.append((w, float(u), a))
    return found


def test_the_cases_tell_the_two_apart():
    for w, u, token in cases():
        total = int((w.double() * 2.0 ** 40).long().sum())
        assert float(torch.tensor(u, dtype=torch.float32)) == u and total > 1 << 60
        below = torch.cumsum((w.double() * 2.0 ** 40).long(), 0)
        aim = int(float(Fraction(u) * total))
        assert int(torch.searchsorted(below, torch.tensor(aim), right=True)) == token


@pytest.mark.gpu
def test_u_times_the_total_is_rounded_once():
    from paged_kv_prep_gb300 import build as pbuild
    pbuild.build()
    for w, u, token in cases():
        got, accepted = pkv.verify_drafts(w[None].cuda(), torch.zeros(0, dtype=torch.int32, device="cuda"),
                                          torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                                          torch.tensor([u], device="cuda"), 0)
        assert got.tolist() == [[token]] and accepted.tolist() == [0]
