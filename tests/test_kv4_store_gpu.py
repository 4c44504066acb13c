"""rope_store, kv4_store and kv4_load on the GPU against plain implementations.

The rotation is defined operation by operation in fp32, so rotated lines are equal to
the bit after their rounding.  Codes and scales are held to the 64-bit quotient's rounding;
the kernel rounds the quotient to fp32 first, which moves it by at most 2^-24 of itself,
so a code may only differ where the quotient is that near to the middle between two."""
import pytest

import paged_kv_prep_gb300 as pkv
from tests import kv4_reference as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

TYPES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_prep_gb300 import build as pbuild
    pbuild.build()
    yield
    torch.cuda.empty_cache()


def make_table(gen, rows, rot):
    ang = torch.arange(rows, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))
    return torch.cat([ang.cos(), ang.sin()], 1).float()


class Step:
    """A step's fused projection rows (q, k and v are views), its positions and slots."""

    def __init__(self, tokens, heads, group, d, rot, dtype, axes=1, interleaved=False, bs=16, seed=1, rows=500, skip=True):
        gen = torch.Generator().manual_seed(seed)
        self.gen, self.heads, self.d, self.bs, self.interleaved = gen, heads, d, bs, interleaved
        hq = heads * group
        x = torch.randn(tokens, (hq + 2 * heads) * d + 16, generator=gen) * torch.exp2(torch.randint(-6, 7, (tokens, 1), generator=gen).float())
        self.rows = x.to(dtype)
        self.parts = (hq, heads, heads)
        self.q, self.k, self.v = self.split(self.rows)
        self.table = make_table(gen, rows, rot)
        self.positions = torch.randint(0, rows, (axes, tokens), generator=gen, dtype=torch.int32)
        self.axes = None if axes == 1 else [min(i * axes // (rot // 2), axes - 1) if seed % 2 else (i * 7) % axes for i in range(rot // 2)]
        self.blocks = tokens // bs + 3
        self.slots = torch.randperm(self.blocks * bs, generator=gen)[:tokens]
        if skip and tokens > 2:
            self.slots[1] = -1

    def split(self, rows):
        out, at = [], 0
        for h in self.parts:
            out.append(rows[:, at:at + h * self.d].unflatten(1, (h, self.d)))
            at += h * self.d
        return out

    def rope(self):
        return dict(positions=self.positions.cuda(), table=self.table.cuda(), axes=self.axes, interleaved=self.interleaved)

    def rotated(self, x):
        return ref.rotate32(x, self.positions, self.table, self.axes, self.interleaved)

    def cache4(self):
        gen = torch.Generator().manual_seed(99)
        return [torch.randint(0, 256, (self.blocks, self.heads, self.bs, n), generator=gen, dtype=torch.uint8)
                for n in (self.d // 2, self.d // 2, self.d // 16, self.d // 16)]


def bits(x):
    return x.cpu().contiguous().view(torch.int16)


SHAPES = [(8, 4, 128, 128), (2, 1, 128, 64), (1, 8, 64, 64), (3, 5, 64, 16), (5, 2, 256, 256), (1, 1, 256, 96), (1, 33, 128, 32)]


@pytest.mark.parametrize("axes,interleaved", [(1, False), (1, True), (3, False), (3, True), (8, False)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,group,d,rot", SHAPES)
@pytest.mark.parametrize("tokens", [1, 37])
def test_rope_store(tokens, heads, group, d, rot, dtype, axes, interleaved):
    s = Step(tokens, heads, group, d, rot, dtype, axes, interleaved, seed=heads + rot)
    q, k, v = s.split(s.rows.cuda())
    kc = torch.full((s.blocks * s.bs, heads, d), 7.0, dtype=dtype, device="cuda")
    vc = kc.clone()
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = pkv.rope_store(k, v, kc, vc, s.slots.cuda(), q=q, d_error=word.data_ptr(), **s.rope())
    assert word.item() == 0 and out.is_contiguous()
    assert torch.equal(bits(out), bits(s.rotated(s.q).to(dtype)))
    want_k, want_v = torch.full_like(kc, 7.0).cpu(), torch.full_like(kc, 7.0).cpu()
    on = s.slots >= 0
    want_k[s.slots[on]], want_v[s.slots[on]] = s.rotated(s.k).to(dtype)[on], s.v[on]
    assert torch.equal(bits(kc), bits(want_k)) and torch.equal(bits(vc), bits(want_v))
    # the same for the queries in their own place, without keys' rows being touched
    rows = s.rows.cuda()
    q, k, v = s.split(rows)
    assert pkv.rope_store(k, v, kc, vc, s.slots.cuda(), q=q, q_out=q, **s.rope()) is q
    assert torch.equal(bits(q), bits(out)) and torch.equal(rows[:, q.shape[1] * d:].cpu(), s.rows[:, q.shape[1] * d:])


def near_border(value, grid):
    """Whether `value` is within 2^-22 of itself of the middle between two neighbours of `grid`."""
    mid = (grid[1:] + grid[:-1]) / 2
    return ((value[..., None] - mid).abs() <= 2.0 ** -22 * mid).any(-1)


def check_stored(got, want, s, k, units):
    """got, want: [k codes, v codes, k scales, v scales]; differences only at borders."""
    for which, x, unit in ((0, k, units[0]), (1, s.v.double(), units[1])):
        block, off = s.slots.clamp(min=0) // s.bs, s.slots.clamp(min=0) % s.bs
        a, b = got[which + 2].cpu(), want[which + 2]
        if not torch.equal(a, b):
            y = x.unflatten(-1, (-1, 16)).abs().amax(-1) / (6.0 * unit)
            near = near_border(y, ref.e4m3(torch.arange(127, dtype=torch.uint8)))
            d = torch.zeros_like(b, dtype=torch.bool)
            d[block, :, off] = near
            assert d[a != b].all()
            continue
        a, b = got[which].cpu(), want[which]
        if not torch.equal(ref.unpack(a), ref.unpack(b)):
            by = (ref.e4m3(want[which + 2]) * unit)[block, :, off].repeat_interleave(16, -1)
            near = near_border((x / by).abs(), ref.E2M1)
            d = torch.zeros(*b.shape[:3], s.d, dtype=torch.bool)
            d[block, :, off] = near
            assert d[ref.unpack(a) != ref.unpack(b)].all()


@pytest.mark.parametrize("axes,interleaved", [(0, False), (1, False), (1, True), (3, False)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,group,d,rot", SHAPES)
@pytest.mark.parametrize("units", [(1.0, 1.0), (0.37, 2.5)])
def test_kv4_store(heads, group, d, rot, dtype, axes, interleaved, units):
    s = Step(41, heads, group, d, rot, dtype, max(axes, 1), interleaved, bs=48 if heads == 3 else 16, seed=heads + rot)
    q, k, v = s.split(s.rows.cuda())
    dev = [x.cuda() for x in s.cache4()]
    want = s.cache4()
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(q=q, **s.rope()) if axes else {}
    out = pkv.kv4_store(k, v, *dev, s.slots.cuda(), k_unit=units[0], v_unit=units[1], d_error=word.data_ptr(), **kw)
    assert word.item() == 0
    if axes:
        assert torch.equal(bits(out), bits(s.rotated(s.q).to(dtype)))
    else:
        assert out is None
    u32 = [float(torch.tensor(u)) for u in units]                     # units are fp32 in the kernel
    keys = (s.rotated(s.k) if axes else s.k).double()
    ref.store(keys, s.v.double(), want[:2], want[2:], s.slots, *u32)
    check_stored(dev, want, s, keys, u32)
    # read back: exact products, the unit's in fp32, one rounding
    pick = torch.cat([s.slots, torch.tensor([-1, 0, s.blocks * s.bs - 1])])
    dev[3].copy_(torch.where(dev[3] % 128 == 127, 0, dev[3]))          # what was there before may hold NaN scales
    got = pkv.kv4_load(*dev, pick.cuda(), dtype=dtype, k_unit=units[0], v_unit=units[1])
    for y, codes, scales, unit in ((got[0], dev[0], dev[2], u32[0]), (got[1], dev[1], dev[3], u32[1])):
        full = (ref.values(codes.cpu(), scales.cpu(), 1.0).float() * unit).to(dtype).transpose(1, 2).reshape(-1, heads, d)
        line = torch.where((pick >= 0)[:, None, None], full[pick.clamp(min=0)], torch.zeros((), dtype=dtype))
        assert torch.equal(y.cpu().isnan(), line.isnan())
        assert torch.equal(y.cpu().nan_to_num(), line.nan_to_num())


def test_values_half_way_between_two_codes():
    """Multiples of the codes' middles, as 16-bit values often are: to the even code, for every scale."""
    mids = (ref.E2M1[1:] + ref.E2M1[:-1]) / 2
    group = torch.cat([mids, -mids, torch.tensor([6.0, -6.0]).double()])
    mantissa = torch.tensor([1, 1.125, 1.25, 1.375, 1.5, 1.625, 1.75, 1.875]).double()
    x = torch.stack([group * m * 2.0 ** e for e in range(-5, 6) for m in mantissa])      # [88, 16]
    x = x.to(torch.bfloat16)
    k = x.unflatten(0, (-1, 8)).flatten(1).unflatten(1, (1, 128)).contiguous()           # [11, 1, 128]
    caches = [torch.zeros(1, 1, 16, n, dtype=torch.uint8) for n in (64, 64, 8, 8)]
    dev = [c.cuda() for c in caches]
    slots = torch.arange(11)
    pkv.kv4_store(k.cuda(), -k.cuda(), *dev, slots.cuda())
    ref.store(k.double(), -k.double(), caches[:2], caches[2:], slots, 1.0, 1.0)
    for a, b in zip(dev, caches):
        assert torch.equal(a.cpu(), b)


def test_nan_and_infinity():
    s = Step(5, 2, 1, 128, 128, torch.bfloat16, skip=False)
    k, v = s.k.clone(), s.v.clone()
    k[0, 1, 20] = float("nan")
    v[1, 0, 100] = float("nan")
    k[2, 0, 5], v[2, 1, 6] = float("inf"), -float("inf")
    v[3, 1, 3], v[3, 1, 4] = float("nan"), float("inf")
    dev, want = [x.cuda() for x in s.cache4()], s.cache4()
    pkv.kv4_store(k.cuda(), v.cuda(), *dev, s.slots.cuda())
    ref.store(k.double(), v.double(), want[:2], want[2:], s.slots, 1.0, 1.0)
    for a, b in zip(dev[2:], want[2:]):
        assert torch.equal(a.cpu(), b)
    for a, b in zip(dev[:2], want[:2]):
        assert torch.equal(ref.unpack(a.cpu()), ref.unpack(b))
    lk, lv = (x.cpu() for x in pkv.kv4_load(*dev, s.slots.cuda()))
    assert lk[0, 1, 16:32].isnan().all() and not lk[0, 1, 32:].isnan().any() and not lk[0, 0].isnan().any()
    assert lk[1, 0, :16].isnan().all() and not lk[1, 0, 16:].isnan().any() and not lv.isnan().any()
    assert lk[2, 0, 5] == 6 * 448 and lv[2, 1, 6] == -6 * 448 and lk[3, 1, :16].isnan().all()


def test_tiny_and_zero_lines():
    k = torch.zeros(3, 1, 64, dtype=torch.bfloat16)
    k[1] = 2.0 ** -40                                             # below the smallest scale: zeros
    k[2, 0, :16] = torch.linspace(-1, 1, 16).bfloat16() * 2.0 ** -7
    caches = [torch.full((1, 1, 16, n), 255, dtype=torch.uint8) for n in (32, 32, 4, 4)]
    dev = [c.cuda() for c in caches]
    pkv.kv4_store(k.cuda(), k.cuda(), *dev, torch.arange(3).cuda())
    ref.store(k.double(), k.double(), caches[:2], caches[2:], torch.arange(3), 1.0, 1.0)
    for a, b in zip(dev, caches):
        assert torch.equal(a.cpu(), b)


@pytest.mark.parametrize("four", [False, True])
def test_bad_slots_and_positions(four):
    s = Step(6, 2, 2, 64, 64, torch.float16, axes=3, skip=False)
    s.positions[2, 1], s.positions[0, 4] = 500, -1
    s.slots[2], s.slots[3] = s.blocks * s.bs, 2 ** 40
    q, k, v = s.split(s.rows.cuda())
    out = torch.full((6, 4, 64), 9.0, dtype=torch.float16, device="cuda")
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    on = torch.tensor([0, 5])
    kw = dict(q=q, q_out=out, d_error=word.data_ptr(), **s.rope())
    if four:
        dev, want = [x.cuda() for x in s.cache4()], s.cache4()
        pkv.kv4_store(k, v, *dev, s.slots.cuda(), **kw)
        some = torch.full_like(s.slots, -1)
        some[on] = s.slots[on]
        s.positions.clamp_(0, 499)
        ref.store(s.rotated(s.k).double(), s.v.double(), want[:2], want[2:], some, 1.0, 1.0)
        s.slots = some
        check_stored(dev, want, s, s.rotated(s.k).double(), (1.0, 1.0))
    else:
        kc, vc = (torch.zeros(s.blocks * s.bs, 2, 64, dtype=torch.float16, device="cuda") for _ in range(2))
        pkv.rope_store(k, v, kc, vc, s.slots.cuda(), **kw)
        s.positions.clamp_(0, 499)
        want = torch.zeros_like(kc).cpu()
        want[s.slots[on]] = s.rotated(s.k).half()[on]
        assert torch.equal(bits(kc), bits(want)) and int((vc != 0).any(-1).any(-1).sum()) == 2
    assert word.item() == pkv.DEVERR_SLOT | pkv.DEVERR_POSITION
    good = torch.tensor([0, 2, 3, 5])
    assert torch.equal(bits(out)[good], bits(s.rotated(s.q).half())[good]) and (out[[1, 4]] == 9.0).all()


def test_load_past_the_cache_is_reported():
    s = Step(3, 2, 1, 64, 64, torch.bfloat16, skip=False)
    dev = [x.cuda() for x in s.cache4()]
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, v = pkv.kv4_load(*dev, torch.tensor([s.blocks * s.bs, -5, 2 ** 40]).cuda(), d_error=word.data_ptr())
    assert word.item() == pkv.DEVERR_SLOT and (k == 0).all() and (v == 0).all()


def test_streams_capture_and_empty_steps():
    s = Step(50, 4, 2, 128, 128, torch.bfloat16, axes=3)
    q, k, v = s.split(s.rows.cuda())
    slots, rope = s.slots.cuda(), s.rope()
    first = [x.cuda() for x in s.cache4()]
    want = pkv.kv4_store(k, v, *first, slots, q=q, **rope)
    lines = [torch.zeros(s.blocks * s.bs, 4, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    assert torch.equal(pkv.rope_store(k, v, *lines, slots, q=q, **rope), want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        again = [x.cuda() for x in s.cache4()]
        torch.cuda.synchronize()
        out = pkv.kv4_store(k, v, *again, slots, q=q, stream=stream, **rope)
        got = pkv.kv4_load(*again, slots, stream=stream)
        side.synchronize()
        assert torch.equal(out, want) and all(torch.equal(a, b) for a, b in zip(first, again))
        assert torch.equal(got[0], pkv.kv4_load(*first, slots)[0])
    # captured, and replayed with other values in the same places
    again, more = [x.cuda() for x in s.cache4()], [torch.zeros_like(x) for x in lines]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = pkv.kv4_store(k, v, *again, slots, q=q, **rope)
        pkv.rope_store(k, v, *more, slots, q=q, q_out=out, **rope)
        got = pkv.kv4_load(*again, slots)
    rows = q._base if q._base is not None else q
    rows.copy_(torch.flip(s.rows, [1]).cuda())
    graph.replay()
    torch.cuda.synchronize()
    fresh = [x.cuda() for x in s.cache4()]
    assert torch.equal(out, pkv.kv4_store(k, v, *fresh, slots, q=q, **rope))
    assert all(torch.equal(a, b) for a, b in zip(fresh, again)) and torch.equal(got[1], pkv.kv4_load(*fresh, slots)[1])
    assert torch.equal(more[0][slots[2:]], s.rotated(s.split(torch.flip(s.rows, [1]))[1]).bfloat16().cuda()[2:])
    # no tokens
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    assert pkv.kv4_store(k[:0], v[:0], *again, none, q=q[:0], **{**rope, "positions": rope["positions"][:, :0]}).shape[0] == 0
    assert pkv.kv4_load(*again, none)[0].shape == (0, 4, 128)


def test_many_heads_and_long_caches():
    """1024 KV heads; lines whose bytes start past 2^32."""
    s = Step(3, 1024, 1, 256, 256, torch.bfloat16, skip=False)
    q, k, v = s.split(s.rows.cuda())
    dev, want = [x.cuda() for x in s.cache4()], s.cache4()
    out = pkv.kv4_store(k, v, *dev, s.slots.cuda(), q=q, **s.rope())
    assert torch.equal(bits(out), bits(s.rotated(s.q).bfloat16()))
    ref.store(s.rotated(s.k).double(), s.v.double(), want[:2], want[2:], s.slots, 1.0, 1.0)
    check_stored(dev, want, s, s.rotated(s.k).double(), (1.0, 1.0))
    s = Step(9, 8, 1, 128, 128, torch.bfloat16, skip=False)
    q, k, v = s.split(s.rows.cuda())
    blocks = 600000                                               # 4.9 GB of codes
    dev = [torch.zeros(blocks, 8, 16, n, dtype=torch.uint8, device="cuda") for n in (64, 64, 8, 8)]
    small = [torch.zeros(s.blocks, 8, 16, n, dtype=torch.uint8, device="cuda") for n in (64, 64, 8, 8)]
    shift = (blocks - s.blocks) * 16
    pkv.kv4_store(k, v, *dev, s.slots.cuda() + shift, **s.rope())
    pkv.kv4_store(k, v, *small, s.slots.cuda(), **s.rope())
    assert all(torch.equal(a[-s.blocks:], b) and not a[:1000].any() for a, b in zip(dev, small))
    for a, b in zip(pkv.kv4_load(*dev, s.slots.cuda() + shift), pkv.kv4_load(*small, s.slots.cuda())):
        assert torch.equal(a, b)
    lines = [torch.zeros(2400000, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pkv.rope_store(k, v, *lines, s.slots.cuda() + 2390000, **s.rope())
    assert torch.equal(bits(lines[0][2390000 + s.slots.cuda()]), bits(s.rotated(s.k).bfloat16()))


@pytest.mark.parametrize("tokens", [5000])
def test_many_tokens(tokens):
    s = Step(tokens, 2, 3, 64, 32, torch.float16, axes=3, interleaved=True)
    q, k, v = s.split(s.rows.cuda())
    dev, want = [x.cuda() for x in s.cache4()], s.cache4()
    out = pkv.kv4_store(k, v, *dev, s.slots.cuda(), q=q, **s.rope())
    assert torch.equal(bits(out), bits(s.rotated(s.q).half()))
    ref.store(s.rotated(s.k).double(), s.v.double(), want[:2], want[2:], s.slots, 1.0, 1.0)
    check_stored(dev, want, s, s.rotated(s.k).double(), (1.0, 1.0))


def test_more_rows_than_slots():
    """A padded step: rows past the slots are not touched, and what is allocated is for the slots' tokens."""
    s = Step(20, 2, 2, 64, 64, torch.bfloat16, skip=False)
    q, k, v = s.split(s.rows.cuda())
    dev, want = [x.cuda() for x in s.cache4()], s.cache4()
    slots = s.slots[:13].contiguous()
    out = pkv.kv4_store(k, v, *dev, slots.cuda(), q=q, **s.rope())
    assert out.shape == (13, 4, 64) and torch.equal(bits(out), bits(s.rotated(s.q).bfloat16()[:13]))
    keys = s.rotated(s.k).double()
    ref.store(keys, s.v.double(), want[:2], want[2:], slots, 1.0, 1.0)
    for a, b in zip(dev[2:], want[2:]):
        assert torch.equal(a.cpu(), b)
    given = torch.full_like(q, 7.0).contiguous()
    pkv.kv4_store(k, v, *dev, slots.cuda(), q=q, q_out=given, **s.rope())
    assert torch.equal(given[:13], out) and (given[13:] == 7.0).all()
