"""kv4_store, every group by itself: codes are held to the scale that was stored, whichever of two it is at a
rounding border, and what is not stored stays as it was."""
import pytest

import paged_kv_prep_gb300 as pkv
from tests import kv4_reference as ref
from tests.test_kv4_store_gpu import SHAPES, TYPES, Step, near_border

torch = pytest.importorskip("torch")


def check_codes(got, before, s, k, units):
    """got, before: [k codes, v codes, k scales, v scales] after and before a store of the finite lines k and s.v at
    s.slots.  A quotient in the kernel is off by at most 2^-22 of itself (two roundings of 2^-24), so that a scale or a
    code may only differ where its quotient in 64 bits is that near to the middle between two.  How many scales differ."""
    on = s.slots >= 0
    block, off = s.slots[on] // s.bs, s.slots[on] % s.bs
    kept = torch.ones(s.blocks, s.bs, dtype=torch.bool)
    kept[block, off] = False
    for a, b in zip(got, before):
        assert torch.equal(a.transpose(1, 2)[kept], b.transpose(1, 2)[kept])
    moved = 0
    for which, x, unit in ((0, k, units[0]), (1, s.v.double(), units[1])):
        x = x[on].unflatten(-1, (-1, 16))                    # [tokens, heads, groups, 16]
        scale, codes = got[which + 2][block, :, off], ref.unpack(got[which][block, :, off]).unflatten(-1, (-1, 16))
        quotient = x.abs().amax(-1) / (6.0 * unit)
        other = scale != ref.scale_code(quotient)
        assert near_border(quotient, ref.e4m3(torch.arange(127, dtype=torch.uint8)))[other].all()
        moved += int(other.sum())
        by = (ref.e4m3(scale) * unit)[..., None]
        y = torch.where(by > 0, x / torch.where(by > 0, by, 1.0), 0.0)
        want = ref.unpack(ref.pack(ref.element_code(y).flatten(-2))).view_as(y)
        assert near_border(y.abs(), ref.E2M1)[codes != want].all()
    return moved


def stored(s, units):
    """The plain implementation's caches after and before the store, and the keys."""
    before, after = s.cache4(), s.cache4()
    keys = s.rotated(s.k).double()
    ref.store(keys, s.v.double(), after[:2], after[2:], s.slots, *units)
    return after, before, keys


def at_a_border(s):
    """The first stored token's first group gets a maximum half way between two scales: (1 + 1.125) / 2 = 17 / 16, times 6."""
    t = int((s.slots >= 0).nonzero()[0])
    s.positions[:, t] = 0                                    # cosines of 1
    s.k[t, 0, :16] = torch.linspace(-6.0, 6.0, 16).to(s.k.dtype)
    s.k[t, 0, 3] = 6 * 17 / 16
    return t


def test_the_plain_store_passes_and_planted_mistakes_do_not():
    units = (1.0, 1.0)
    for dtype in TYPES:
        s = Step(11, 2, 1, 128, 128, dtype, seed=5)
        t = at_a_border(s)
        assert int(s.slots[1]) == -1 and t == 0
        got, before, keys = stored(s, units)
        assert check_codes(got, before, s, keys, units) == 0
        block, off = int(s.slots[t]) // s.bs, int(s.slots[t]) % s.bs

        def planted(which, index, value):
            bad = [x.clone() for x in got]
            bad[which][index] = value
            return bad
        # the other scale at the border, with its own codes, passes
        other = planted(2, (block, 0, off, 0), int(got[2][block, 0, off, 0]) + 1)
        by = ref.e4m3(other[2][block, 0, off, :1])
        other[0][block, 0, off, :8] = ref.pack(ref.element_code(keys[t, 0, :16] / by))
        assert check_codes(other, before, s, keys, units) == 1
        # beside it one wrong code of any other line does not, nor a scale that is nowhere near a border
        last = int(s.slots[-1])
        for bad in (planted(0, (last // s.bs, 1, last % s.bs, 9), int(got[0][last // s.bs, 1, last % s.bs, 9]) ^ 0x10),
                    planted(1, (last // s.bs, 0, last % s.bs, 0), int(got[1][last // s.bs, 0, last % s.bs, 0]) ^ 0x8),
                    planted(3, (last // s.bs, 0, last % s.bs, 2), int(got[3][last // s.bs, 0, last % s.bs, 2]) ^ 0x1)):
            bad[2][block, 0, off, 0] = other[2][block, 0, off, 0]
            bad[0][block, 0, off, :8] = other[0][block, 0, off, :8]
            with pytest.raises(AssertionError):
                check_codes(bad, before, s, keys, units)
        # a token that is not stored leaves every line as it was
        spare = next(x for x in range(s.blocks * s.bs) if x not in s.slots.tolist())
        for which in range(4):
            bad = planted(which, (spare // s.bs, 1, spare % s.bs, 1), int(before[which][spare // s.bs, 1, spare % s.bs, 1]) ^ 1)
            with pytest.raises(AssertionError):
                check_codes(bad, before, s, keys, units)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,group,d,rot", SHAPES)
@pytest.mark.parametrize("units", [(1.0, 1.0), (0.37, 2.5), (2.0 ** -9, 3.0)])
def test_every_group(heads, group, d, rot, dtype, units):
    from paged_kv_prep_gb300 import build as pbuild
    pbuild.build()
    s = Step(1500 // heads, heads, group, d, rot, dtype, 3, heads % 2 == 1, bs=48 if heads == 3 else 16, seed=heads + rot)
    at_a_border(s)
    dev = [x.cuda() for x in s.cache4()]
    kw = dict(positions=s.positions.cuda(), table=s.table.cuda(), axes=s.axes, interleaved=s.interleaved)
    pkv.kv4_store(s.k.cuda(), s.v.cuda(), *dev, s.slots.cuda(), k_unit=units[0], v_unit=units[1], **kw)
    check_codes([x.cpu() for x in dev], s.cache4(), s, s.rotated(s.k).double(), [float(torch.tensor(u)) for u in units])
