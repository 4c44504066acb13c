"""kv8_attention on the GPU against its plain implementation in 64 bits.

Tolerances, with A = sum p |v| of an output element, X = a row's largest sum
|q k| softmax_scale and the half steps 2^-11 (f16), 2^-8 (bf16), 2^-24 (fp32):
a logit is a sum of exact products in fp32, off by at most 2^-19 X (room for
sixteen half-step roundings along it twice over), and the logarithm of the value
scale (up to 26 here) rides on it, which costs two more half steps of values up
to 64, 2^-17; a weight times its value
scale is rounded to f16 once, 2^-11 of itself, or 2^-25 of the row's largest
when it is far smaller; sums in fp32 add 2^-17; the output is rounded once."""
import math

import pytest

import paged_kv_prep_gb300 as pkv
import pkv_workloads as workloads
from tests import kv8_reference as ref
from tests.gpu_helpers import build_states

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_prep_gb300 import build as pbuild
    pbuild.build()
    yield
    torch.cuda.empty_cache()


class Case:
    def __init__(self, reqs, bs, heads, group, d, dtype=torch.bfloat16, seed=1, spread=2, pad=0, width=0, magnitude=1.0):
        """reqs: (scheduled tokens, cached tokens) of each request."""
        gen = torch.Generator().manual_seed(seed)
        self.gen, self.reqs, self.bs, self.heads, self.group, self.d, self.dtype = gen, reqs, bs, heads, group, d, dtype
        self.lens = [x for _, x in reqs]
        self.starts = [0]
        for c, _ in reqs:
            self.starts.append(self.starts[-1] + c)
        need = [max(0, -(-x // bs)) for x in self.lens]
        self.blocks = sum(need) + 2
        perm = torch.randperm(self.blocks, generator=gen).tolist()
        self.tables = torch.full((len(reqs), max(max(need), 1) + width), -1, dtype=torch.int32)
        for i, n in enumerate(need):
            for j in range(n):
                self.tables[i, j] = perm.pop()
        slots = self.blocks * bs
        # every byte a NaN code first: whatever is not a cached token must not be read into a sum
        self.caches = [torch.full((slots, heads, d), 127, dtype=torch.uint8) for _ in range(2)]
        self.scales = [torch.exp2(torch.randint(-spread, spread + 1, (self.blocks, heads), generator=gen).float() - 6)
                       for _ in range(2)]
        for i, x in enumerate(self.lens):
            for s in range(max(x, 0)):
                b = int(self.tables[i, s // bs])
                for c in self.caches:
                    c[b * bs + s % bs] = ref.encode(torch.randn(heads, d, generator=gen).double() * 64)
        T, hq = self.starts[-1], heads * group
        rows = (torch.randn(T, hq * d + pad, generator=gen) * magnitude).to(dtype)
        self.q = rows[:, :hq * d].view(T, hq, d) if not pad else rows[:, :hq * d].unflatten(1, (hq, d))

    def args(self):
        kc, vc = [c.view(c.shape[0], -1).cuda() for c in self.caches]
        ks, vs = [s.cuda() for s in self.scales]
        rows = self.q.as_strided((self.q.shape[0], self.q.stride(0)), (self.q.stride(0), 1)) if self.q.shape[0] > 1 else None
        if rows is not None and self.q.stride(0) != self.q.shape[1] * self.d:
            q = rows.cuda()[:, :self.q.shape[1] * self.d].unflatten(1, self.q.shape[1:])
        else:
            q = self.q.contiguous().cuda()
        return (q, kc, vc, ks, vs, self.tables.cuda(), torch.tensor(self.starts, dtype=torch.int32).cuda(),
                torch.tensor(self.lens, dtype=torch.int32).cuda())

    def reference(self, scale, window, weights=None):
        return ref.attention(self.q, *self.caches, *self.scales, self.tables, self.starts, self.lens, scale, window, weights)


def compare(case, out, lse, want, vmax=448.0):
    w_out, w_lse, size, reach = want
    out, lse = out.cpu().double(), lse.cpu().double()
    assert torch.equal(torch.isinf(lse), torch.isinf(w_lse)) and torch.equal(lse.isnan(), w_lse.isnan())
    fine = torch.isfinite(w_lse)
    logit = 2.0 ** -19 * reach + 2.0 ** -22 * w_lse.abs().clamp(max=1e30) + 2.0 ** -17
    assert (((lse - w_lse).abs() <= logit)[fine]).all(), float((lse - w_lse)[fine].abs().max())
    assert torch.equal(out.isnan(), w_out.isnan())
    largest = float(max(s.max() for s in case.scales[1:])) * vmax
    most = max(list(case.lens) + [1])
    tol = (2.0 ** -11 + 2.0 ** -17 + 2 * logit[..., None]) * size + most * 2.0 ** -25 * largest
    tol = tol + HALF[case.dtype] * (w_out.abs() + tol) + 2.0 ** -25
    bad = (out - w_out).abs() > tol
    bad &= ~w_out.isnan()
    assert not bad.any(), (int(bad.sum()), float(((out - w_out).abs() / tol)[bad].max()))


def check(case, window=0, scale=None, weights=True):
    scale = case.d ** -0.5 if scale is None else scale
    a = case.args()
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = torch.rand(case.blocks * case.bs, generator=case.gen)
    got = before.cuda()
    out, lse = pkv.kv8_attention(*a, softmax_scale=scale, window=window, weights=got if weights else None,
                                 d_error=word.data_ptr())
    assert word.item() == 0
    sums = torch.zeros(case.blocks * case.bs, dtype=torch.float64)
    want = case.reference(scale, window, sums)
    compare(case, out, lse, want)
    if weights:
        reach = float(want[3].max()) if want[3].numel() else 0.0
        top = float(want[1][torch.isfinite(want[1])].abs().max()) if torch.isfinite(want[1]).any() else 0.0
        rel = 4 * (2.0 ** -19 * reach + 2.0 ** -22 * top) + 2.0 ** -15
        total = before.double() + sums
        assert ((got.cpu().double() - total).abs() <= rel * sums + 2.0 ** -22 * total).all()
        assert torch.equal(got.cpu()[sums == 0], before[sums == 0])
    return out, lse


DECODES = [(1, x) for x in (1, 15, 16, 17, 200, 33, 640, 1000)]
MIXED = [(1, 1), (1, 77), (2, 2), (3, 50), (5, 5), (17, 100), (40, 90), (1, 300)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("heads,group,d", [(8, 4, 128), (2, 8, 128), (1, 1, 128), (3, 5, 64), (2, 7, 256), (1, 12, 64),
                                           (5, 1, 64)])
@pytest.mark.parametrize("reqs", [DECODES, MIXED], ids=["decodes", "mixed"])
def test_matches_plain(reqs, heads, group, d, dtype):
    check(Case(reqs, 16, heads, group, d, dtype, seed=heads * 100 + group))


@pytest.mark.parametrize("bs", [1, 7, 24, 32, 48, 100])
def test_block_sizes(bs):
    check(Case(MIXED, bs, 2, 4, 128, seed=bs, width=2))


@pytest.mark.parametrize("window", [1, 2, 16, 30, 64, 4096, 2 ** 31 - 1])
def test_windows(window):
    check(Case(MIXED + [(1, 1), (30, 33)], 16, 2, 4, 128, seed=window % 97), window=window)


@pytest.mark.parametrize("group", [4, 16])
def test_rows_that_see_nothing(group):
    """More scheduled tokens than cached ones, no cached tokens, no scheduled tokens, freed blocks."""
    case = Case([(1, 0), (0, 40), (9, 4), (1, 64), (3, 70)], 16, 2, group, 128, seed=2)
    case.tables[3, :] = -1
    case.tables[4, 1:3] = -1
    out, lse = check(case)
    assert (lse[0] == -math.inf).all() and (out[0] == 0).all()
    assert (lse[1:6] == -math.inf).all() and torch.isfinite(lse[6:10]).all()
    assert (lse[10] == -math.inf).all()


def test_one_long_request_is_split():
    check(Case([(1, 6000)], 32, 1, 4, 64, seed=3))
    check(Case([(2, 3001), (1, 9)], 16, 2, 8, 64, seed=4), window=2500)


@pytest.mark.parametrize("spread", [10, 20])
def test_scales_that_differ_between_blocks(spread):
    """Value scales up to 2^40 apart: the f16 operand carries the scale, so no row loses its own."""
    case = Case([(1, 100), (1, 33), (6, 60)], 16, 2, 4, 128, seed=5, spread=spread)
    case.scales[0] = torch.exp2(torch.randint(-8, -5, case.scales[0].shape, generator=case.gen).float())
    check(case)


def test_extreme_queries_and_logits():
    """Queries far from 1, rows with tiny and large elements, a scale that saturates the softmax."""
    case = Case([(1, 90), (1, 17), (4, 40)], 16, 2, 4, 128, seed=6)
    case.q = case.q.clone()
    case.q[0] *= 2.0 ** 40
    case.q[1] *= 2.0 ** -60
    case.q[2, :, ::2] *= 2.0 ** -12
    case.q[3] = 0
    for i in range(2):
        case.scales[i] = torch.exp2(torch.randint(-8, -5, case.scales[i].shape, generator=case.gen).float())
    check(case, scale=2.0 ** -38)
    check(case, scale=0.0)
    check(Case([(1, 300), (3, 20)], 16, 2, 4, 128, seed=7, magnitude=8.0), scale=1.0)


def test_nan_and_infinity_stay_in_their_rows():
    """A NaN key or value reaches the rows that see it and no other; so does an infinite query."""
    case = Case([(8, 40), (1, 20), (1, 20), (2, 30)], 16, 2, 4, 128, seed=8)
    b = case.tables
    case.caches[1][int(b[0, 2]) * 16 + 5, 0, 3] = 127       # position 37: queries 5..7 of request 0, head 0, dim 3
    case.caches[0][int(b[0, 2]) * 16 + 6, 1, 9] = 255       # position 38: queries 6, 7, head 1
    case.caches[1][int(b[1, 0]) * 16 + 2, 1, 100] = 127
    case.q = case.q.clone()
    case.q[9, 0, 0] = math.nan
    case.q[11, 3] = math.nan
    scale = case.d ** -0.5
    out, lse = pkv.kv8_attention(*case.args(), softmax_scale=scale)
    want = case.reference(scale, 0)
    assert want[0].isnan().any() and not want[0][:5].isnan().any()
    w_out, w_lse, size, reach = want
    assert torch.equal(out.cpu().isnan(), w_out.isnan()) and torch.equal(lse.cpu().isnan(), w_lse.isnan())
    ok = ~w_out.isnan()
    assert (out.cpu().double() - w_out)[ok].abs().max() < 0.05 * w_out[ok].abs().max()


def test_bad_tables_are_reported_and_not_read():
    case = Case([(1, 100), (1, 60), (1, 30), (2, 20)], 16, 2, 4, 128, seed=9)
    case.tables[0, 2] = case.blocks
    case.tables[1, 0] = 2 ** 31 - 1
    a = list(case.args())
    lens = a[7].clone()
    lens[2] = case.tables.shape[1] * 16 + 40                # longer than the table: the rest is not seen
    a[7] = lens
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = pkv.kv8_attention(*a, d_error=word.data_ptr())
    assert word.item() == pkv.DEVERR_BLOCK
    case.lens[2] = int(lens[2])
    want = case.reference(case.d ** -0.5, 0)
    compare(case, out, lse, want)


def test_bad_locations_skip_the_request():
    case = Case([(1, 30), (1, 40), (2, 20), (1, 10)], 16, 2, 4, 128, seed=10)
    a = list(case.args())
    a[6] = torch.tensor([0, 1, 2, 1, 900], dtype=torch.int32).cuda()
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(a[0], 7.0)
    out, lse = pkv.kv8_attention(*a, out=out, d_error=word.data_ptr())
    assert word.item() == pkv.DEVERR_COUNT
    want = case.reference(case.d ** -0.5, 0)
    compare_rows = [0, 1]
    assert (out.cpu().double() - want[0])[compare_rows].abs().max() < 0.05 * want[0].abs().max()
    assert (out[2:] == 7.0).all()


def test_strided_rows_and_given_buffers():
    """q as a view of fused projection rows, out as a view of wider rows, a workspace kept by the caller."""
    case = Case(MIXED, 16, 2, 4, 128, seed=11, pad=2 * 2 * 128)
    a = case.args()
    assert a[0].stride(0) == (8 + 4) * 128
    wide = torch.full((a[0].shape[0], 8 * 128 + 64), 5.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, :8 * 128].unflatten(1, (8, 128))
    lse = torch.empty(a[0].shape[0], 8, device="cuda")
    ws = torch.full((pkv.kv8_attention_workspace(a[0].shape[0], 8, 128),), 255, dtype=torch.uint8, device="cuda")
    want = case.reference(case.d ** -0.5, 0)
    for _ in range(2):
        pkv.kv8_attention(*a, out=out, lse=lse, workspace=ws)
        compare(case, out, lse, want)
        assert (wide[:, 8 * 128:] == 5.0).all()
    assert pkv.kv8_attention(*a, workspace=ws[:1024], check=False) == pkv.ERR_INVALID_ARG


def test_repeats_are_bit_identical_and_streams_and_capture():
    case = Case(MIXED + [(1, 2000), (64, 400)], 16, 2, 4, 128, seed=12)
    a = case.args()
    first = pkv.kv8_attention(*a)
    for _ in range(3):
        again = pkv.kv8_attention(*a)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    other = pkv.kv8_attention(*a, stream=side)
    side.synchronize()
    assert torch.equal(first[0], other[0])
    w = torch.zeros(case.blocks * case.bs, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out, lse = pkv.kv8_attention(*a, weights=w)
    w.zero_()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first[0], out)
    once = w.clone()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.allclose(w, 2 * once, rtol=2 ** -23, atol=0)


def test_prepared_batch_runs_the_whole_step():
    """prepare_batch -> kv8_store -> kv8_attention -> kv8_evict, as a step uses them."""
    wl = workloads.random_small(seed=5, num_requests=12, max_ctx=120, max_chunk=30, decode_frac=0.5)
    st, _, rows_map = build_states(wl)
    rows, ns = workloads.schedule_arrays(wl, rows_map)
    batch = st.prepare_batch(rows, ns)
    T, heads, group, d = batch.total_tokens, 2, 4, 128
    blocks, bs = wl.groups[0].num_blocks, wl.groups[0].block_size
    n = batch.seq_lens.numel()
    extra = n * 2
    gen = torch.Generator().manual_seed(13)
    codes = torch.randint(0, 120, ((blocks + extra) * bs, heads, d), generator=gen, dtype=torch.uint8)
    scale = torch.full((blocks + extra, heads), 2.0 ** -6)
    kc, vc, ks, vs = codes.clone(), codes.clone(), scale.clone(), scale.clone()
    dev = [kc.view(-1, heads * d).cuda(), vc.view(-1, heads * d).cuda(), ks.cuda(), vs.cuda()]
    k, v = [torch.randn(T, heads, d, generator=gen).bfloat16() for _ in range(2)]
    q = torch.randn(T, heads * group, d, generator=gen).bfloat16()
    weights = torch.zeros((blocks + extra) * bs, device="cuda")
    slots = batch.slot_mapping[0]
    pkv.kv8_store(k.cuda(), v.cuda(), *dev, slots)
    out, lse = pkv.kv8_attention(q.cuda(), *dev, batch.block_tables[0], batch.query_start_loc, batch.seq_lens, weights=weights)
    fresh = (torch.arange(extra, dtype=torch.int32).view(n, 2) + blocks).cuda()
    new, kept = pkv.kv8_evict(*dev, weights, batch.block_tables[0], batch.seq_lens, fresh, 2 * bs - 3, keep_first=1, keep_last=4)

    ref.store(k, v, kc, vc, ks, vs, slots.cpu(), blocks + extra)
    case = Case([(1, 1)], bs, heads, group, d)
    case.scales, case.lens, case.dtype = [ks, vs], batch.seq_lens.tolist(), torch.bfloat16
    want = ref.attention(q, kc, vc, ks, vs, batch.block_tables[0].cpu(), batch.query_start_loc.tolist(), case.lens, d ** -0.5, 0)
    compare(case, out, lse, want)
    w = weights.cpu().clone()
    w.view(-1, bs)[blocks:] = 0
    want_new, want_kept = ref.evict(kc, vc, ks, vs, w, batch.block_tables[0].cpu(), case.lens, fresh.cpu(), 2 * bs - 3, 1, 4)
    assert new.tolist() == want_new and torch.equal(kept.cpu(), want_kept)
    assert ref.same_codes(dev[0].cpu().view(kc.shape), kc) and ref.same_codes(dev[1].cpu().view(vc.shape), vc)
    st.close()


def test_cache_past_32_bits():
    """Blocks whose bytes start past 2^32."""
    heads, group, d, bs = 8, 4, 128, 16
    blocks = 300000
    small = Case([(1, 60), (3, 20)], bs, heads, group, d, seed=14)
    q, kc, vc, ks, vs, tab, qsl, lens = small.args()
    shift = blocks - small.blocks
    big = [torch.full((blocks * bs, heads * d), 127, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scale = [torch.ones(blocks, heads, device="cuda") for _ in range(2)]
    for b, c in zip(big, (kc, vc)):
        b[shift * bs:] = c
    for b, c in zip(scale, (ks, vs)):
        b[shift:] = c
    want = pkv.kv8_attention(q, kc, vc, ks, vs, tab, qsl, lens)
    w = torch.zeros(blocks * bs, device="cuda")
    got = pkv.kv8_attention(q, *big, *scale, torch.where(tab >= 0, tab + shift, tab), qsl, lens, weights=w)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    assert float(w.sum()) == pytest.approx(4 * heads * group, rel=1e-4)


def test_thousands_of_requests():
    """More requests than a CTA has threads: the plan's chunks hold several."""
    gen = torch.Generator().manual_seed(2)
    lens = torch.randint(0, 8, (3000,), generator=gen).tolist()
    reqs = [(int(torch.randint(0, x + 1, (1,), generator=gen)) if x else 0, x) for x in lens]
    check(Case(reqs, 16, 1, 3, 64, seed=15))
    check(Case([(1, max(x, 1)) for x in lens] + [(40, 50)], 16, 1, 2, 64, seed=16))


def test_many_short_requests_are_not_cut():
    """Short tables and many tiles: a warp takes a whole row tile."""
    gen = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 250, (60,), generator=gen).tolist()
    check(Case([(1, x) for x in lens], 16, 8, 4, 64, seed=17))
    check(Case([(1 + x % 3, x) for x in lens] + [(30, 100)], 16, 8, 4, 64, seed=18), window=100)
    check(Case([(1, x) for x in lens[:20]], 24, 16, 1, 64, seed=19))


def test_no_tokens():
    case = Case([(1, 5)], 16, 1, 1, 64)
    q, kc, vc, ks, vs, tab, qsl, lens = case.args()
    out, lse = pkv.kv8_attention(q[:0], kc, vc, ks, vs, tab[:0], qsl[:1], lens[:0])
    assert out.shape == (0, 1, 64) and lse.shape == (0, 1)


CHUNKS = [(1, 20), (9, 9), (33, 33), (64, 64), (65, 200), (130, 131), (200, 1500), (257, 700)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("heads,group,d", [(2, 4, 128), (1, 8, 128), (3, 1, 128), (2, 5, 64), (1, 33, 64)])
def test_chunks_match_plain(heads, group, d, dtype):
    """Prompt chunks: row tiles of one and two halves, odd lengths, ranges cut inside a tile."""
    check(Case(CHUNKS, 16, heads, group, d, dtype, seed=heads * 10 + group))


@pytest.mark.parametrize("heads,d,window", [(8, 64, 0), (8, 64, 333), (5, 128, 0), (9, 256, 150)])
def test_many_chunks_share_out_their_weights(heads, d, window):
    """More token tiles than clusters: each works through several, of one request and of the next."""
    reqs = [(3 + 7 * i % 61, 64 + 41 * i % 900) for i in range(60)]
    check(Case(reqs, 16, heads, 2, d, seed=heads + d), window=window)


@pytest.mark.parametrize("window", [1, 17, 100, 128, 1000])
@pytest.mark.parametrize("bs", [16, 48])
def test_chunks_with_windows(window, bs):
    case = Case(CHUNKS, bs, 1, 4, 128, seed=window + bs)
    for i, (c, x) in enumerate(CHUNKS):                     # blocks before the window are freed
        case.tables[i, :max(0, x - c - window + 1) // bs] = -1
    check(case, window=window)


def test_chunks_that_see_little():
    """Chunks longer than their cache, freed blocks in the middle, far-apart value scales, a negative scale."""
    case = Case([(60, 30), (50, 50), (40, 300), (90, 200)], 16, 2, 4, 128, seed=3)
    case.tables[1, 0] = -1
    case.tables[2, 3:12] = -1
    out, lse = check(case)
    assert (lse[:30] == -math.inf).all() and (out[:30] == 0).all() and (lse[60:76] == -math.inf).all()
    check(Case([(40, 100), (100, 300)], 16, 2, 4, 128, seed=4, spread=18))
    check(Case([(40, 100), (100, 300)], 16, 2, 4, 64, seed=5), scale=-0.2)


def test_chunks_nan_stays_in_its_rows():
    case = Case([(120, 200), (40, 40), (64, 500)], 16, 2, 4, 128, seed=8)
    b = case.tables
    case.caches[1][int(b[0, 9]) * 16 + 5, 0, 3] = 127        # position 149: queries 69.. of request 0, head 0
    case.caches[1][int(b[0, 9]) * 16 + 7, 0, 101] = 255
    case.caches[0][int(b[1, 1]) * 16 + 6, 1, 9] = 255        # position 22: queries 22.. of request 1, head 1
    case.q = case.q.clone()
    case.q[170, 0, 0] = math.nan
    scale = case.d ** -0.5
    w = torch.zeros(case.blocks * case.bs, device="cuda")
    out, lse = pkv.kv8_attention(*case.args(), softmax_scale=scale)
    w_out, w_lse, size, reach = case.reference(scale, 0)
    assert w_out.isnan().any() and not w_out[:60].isnan().any()
    assert torch.equal(out.cpu().isnan(), w_out.isnan()) and torch.equal(lse.cpu().isnan(), w_lse.isnan())
    ok = ~w_out.isnan()
    assert (out.cpu().double() - w_out)[ok].abs().max() < 0.05 * w_out[ok].abs().max()
    # a NaN value changes no weight: request 0 keeps its sums
    pkv.kv8_attention(*case.args(), softmax_scale=scale, weights=w)
    slots = (b[0, :12].long()[:, None] * 16 + torch.arange(16)).view(-1)
    assert torch.isfinite(w.cpu()[slots]).all()


def test_chunks_repeat_bit_identically():
    case = Case([(1, 900), (100, 3000), (300, 333)], 16, 2, 4, 128, seed=12)
    a = case.args()
    first = pkv.kv8_attention(*a)
    for _ in range(5):
        again = pkv.kv8_attention(*a)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("reqs", [[(1, 5), (1, 3)], [(2, 4), (1, 3)]], ids=["decodes", "mixed"])
@pytest.mark.parametrize("heads,d", [(912, 256), (913, 256), (1024, 256), (1024, 64)])
def test_more_heads_than_warps(heads, d, reqs):
    """Up to the 1024 KV heads that a cache may have: with head_dim 256 more than the SMs hold warps."""
    case = Case(reqs, 16, heads, 1, d, seed=heads)
    a = case.args()
    out, lse = torch.full_like(a[0], 7.0), torch.full(a[0].shape[:2], 7.0, device="cuda")
    pkv.kv8_attention(*a, out=out, lse=lse)
    compare(case, out, lse, case.reference(d ** -0.5, 0))
    check(case)


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_what_a_call_makes_is_not_in_use_by_the_current_stream(raw):
    """Work queued on the current stream still writes to tensors of the sizes that a call on another stream
    makes, freed before it: the call's outputs and workspace are not theirs, and the call does not wait for
    that work."""
    case = Case([(1, 300), (1, 40), (40, 90)], 16, 2, 4, 128, seed=20)
    a = case.args()
    T, hq, d = a[0].shape
    w = torch.zeros(case.blocks * case.bs, device="cuda")
    want = case.reference(d ** -0.5, 0)
    side = torch.cuda.Stream()
    stream = side.cuda_stream if raw else side
    sizes = [T * hq * d * 2, T * hq * 4, pkv.kv8_attention_workspace(T, hq, d, True)]
    torch.empty(1, dtype=torch.uint8, device="cuda").fill_(255)
    torch.cuda._sleep(1000)
    torch.cuda.synchronize()
    pkv.kv8_attention(*a, weights=w, stream=stream)          # kernels are loaded and that stream's pool filled: both may wait
    torch.cuda.synchronize()
    done = torch.cuda.Event()
    theirs = [torch.empty(x, dtype=torch.uint8, device="cuda") for x in sizes]
    at = {(x.data_ptr(), x.data_ptr() + x.numel()) for x in theirs}
    torch.cuda._sleep(400_000_000)
    for x in theirs:
        x.fill_(255)
    done.record()
    del theirs, x
    out, lse = pkv.kv8_attention(*a, weights=w, stream=stream)
    side.synchronize()
    assert not done.query()                                  # the current stream's work is still to come
    for y in (out, lse):
        lo, hi = y.data_ptr(), y.data_ptr() + y.numel() * y.itemsize
        assert all(hi <= p or lo >= q for p, q in at)
    torch.cuda.synchronize()
    compare(case, out, lse, want)


def test_outputs_freed_early_are_not_handed_out_while_in_use():
    """Outputs of a call on another stream that the current stream still reads when they are freed: the next
    call on that stream gets other memory."""
    case = Case([(1, 300), (40, 90)], 16, 2, 4, 128, seed=21)
    a = case.args()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out, lse = pkv.kv8_attention(*a, stream=side)
    side.synchronize()
    want, at = out.clone(), out.data_ptr()
    late = out + 0
    torch.cuda._sleep(1000)
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)
    late = out + 0                                           # queued behind the sleep
    del out, lse
    again, _ = pkv.kv8_attention(*a, softmax_scale=0.5, stream=side)
    assert again.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(late, want)


def own_tolerance(case, want, scale, window=0):
    """As in compare, but with what a row itself carries in the place of the cache's largest value scale: a
    weight times its value scale is rounded to f16 by 2^-11 of itself, or by 2^-25 of the row's reference
    where it is 2^-14 of that or less; the reference is below twice the largest of the row, and a weight that
    has moved with it was rounded twice.  A code is at most 448."""
    w_out, w_lse, size, reach = want
    most, count = ref.carried(case.q, *case.caches, *case.scales, case.tables, case.starts, case.lens, scale, window)
    logit = 2.0 ** -19 * reach + 2.0 ** -22 * w_lse.abs().clamp(max=1e30) + 2.0 ** -17
    tol = (2.0 ** -11 + 2.0 ** -17 + 2 * logit[..., None]) * size
    tol = tol + (count[:, None] * 2.0 ** -23 * 448.0 * most)[..., None]
    return tol + HALF[case.dtype] * (w_out.abs() + tol) + 2.0 ** -25


@pytest.mark.parametrize("spread", [10, 20])
@pytest.mark.parametrize("reqs", [[(1, 100), (1, 33), (1, 250)], [(1, 100), (6, 60)], [(40, 100), (100, 300)]],
                         ids=["decodes", "short", "chunks"])
def test_rows_keep_what_is_small_in_the_cache(reqs, spread):
    """Value scales up to 2^40 apart between requests, 2^20 within one: each row is held to what it carries
    itself, so that a row of small values lost as a whole would show."""
    case = Case(reqs, 16, 2, 4, 128, seed=22 + spread, dtype=torch.float16)
    for i in range(2):
        case.scales[i] = torch.exp2(torch.randint(-8, -5, case.scales[i].shape, generator=case.gen).float())
    step = torch.linspace(-spread, spread, len(reqs)).round()
    for i in range(len(reqs)):
        used = case.tables[i][case.tables[i] >= 0].long()
        case.scales[1][used] = torch.exp2(step[i] + torch.randint(-spread // 2, spread // 2 + 1, (len(used), case.heads),
                                                                   generator=case.gen).float() - 6).clamp(max=2.0)
    scale = case.d ** -0.5
    out, lse = pkv.kv8_attention(*case.args(), softmax_scale=scale)
    want = case.reference(scale, 0)
    tol = own_tolerance(case, want, scale)
    lost = (want[0].abs() > tol).double().mean((1, 2))       # the share of a row whose loss would show
    assert (lost > 0.5).double().mean() > 0.9, lost
    compare(case, out, lse, want)
    bad = (out.cpu().double() - want[0]).abs() > tol
    assert not bad.any(), (int(bad.sum()), float(((out.cpu().double() - want[0]).abs() / tol).max()))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("high,low", [(22, 7), (30, 7), (24, 0), (9, 7)])
def test_weights_before_a_moved_reference_keep_their_bits(high, low, d):
    """Chunks whose second unit of 128 keys raises the rows' reference in its second half: the weights of its
    first half, already rounded, follow the reference.  The key that raises it has the value zero in some
    dimensions, where the output is what those weights carry."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    one = Case([(16, 272)], 16, 1, 4, d, torch.float16, seed=23)
    gen = one.gen
    order = one.tables[0, :17].long()
    slots = (order[:, None] * 16 + torch.arange(16)).view(-1)
    one.scales = [torch.ones_like(s) for s in one.scales]
    value = torch.zeros(272, dtype=torch.float64)            # a key's first element; a query's is 0.95 ln 2
    value[128:192], value[200] = low, high
    keys = torch.zeros(272, 1, d, dtype=torch.float64)
    keys[:, 0, 0] = value
    values = torch.randint(64, 127, (272, 1, d), generator=gen, dtype=torch.uint8)   # 2 to 448
    values[200, 0, :d // 2] = 0
    one.caches[0][slots], one.caches[1][slots] = ref.encode(keys), values
    one.q = torch.zeros_like(one.q)
    one.q[:, :, 0] = 0.95 * math.log(2)
    want = one.reference(1.0, 0)
    tol = own_tolerance(one, want, 1.0)
    # as many requests on the same blocks as give every CTA whole requests
    n = 2 * sms
    q, kc, vc, ks, vs, tab, _, lens = one.args()
    starts = torch.arange(0, 16 * n + 1, 16, dtype=torch.int32, device="cuda")
    out, lse = pkv.kv8_attention(q.repeat(n, 1, 1), kc, vc, ks, vs, tab.repeat(n, 1), starts, lens.repeat(n), softmax_scale=1.0)
    out, lse = out.cpu().double().view(n, 16, 4, d), lse.cpu().double().view(n, 16, 4)
    assert ((lse - want[1]).abs() <= 2.0 ** -19 * want[3] + 2.0 ** -22 * want[1].abs() + 2.0 ** -17).all()
    bad = (out - want[0]).abs() > tol
    assert not bad.any(), (int(bad.sum()), float(((out - want[0]).abs() / tol).max()))


@pytest.mark.parametrize("bad", [math.nan, math.inf, 0.0, -1.0])
def test_scales_before_the_window_do_not_count(bad):
    """A block that no query of the call sees, still in the table, whose scales hold anything: a freed block that
    another request has been given and not yet written."""
    case = Case([(1, 100), (1, 300), (3, 120), (40, 200)], 16, 2, 4, 128, seed=24)
    window = 20
    seen = torch.zeros(case.blocks, dtype=torch.bool)
    for i, (c, x) in enumerate(case.reqs):
        seen[case.tables[i, max(0, x - c - window + 1) // 16:-(-x // 16)].long()] = True
    for s in case.scales:
        s[~seen] = bad
    a = case.args()
    w = torch.zeros(case.blocks * case.bs, device="cuda")
    out, lse = pkv.kv8_attention(*a, window=window, weights=w)
    for s in case.scales:                                    # what they hold must not matter
        s[~seen] = 1.0
    want = case.reference(case.d ** -0.5, window)
    compare(case, out, lse, want)
    assert torch.isfinite(w).all() and not seen.all()


@pytest.mark.parametrize("d", [64, 128])
def test_a_nan_in_a_long_context_is_found_where_it_is(d):
    """NaN values far apart in a context of more units than a CTA numbers apart: every row takes those it sees,
    and looking for them is little beside the call."""
    L, T, group, bs = 140000, 4864, 8, 16
    gen = torch.Generator(device="cuda").manual_seed(25)
    blocks = L // bs
    kc = torch.randint(0, 100, (L, d), generator=gen, device="cuda", dtype=torch.uint8)
    vc = torch.randint(0, 100, (L, d), generator=gen, device="cuda", dtype=torch.uint8)
    sc = torch.full((blocks, 1), 2.0 ** -6, device="cuda")
    table = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)[None]
    q = torch.randn(T, group, d, generator=gen, device="cuda").bfloat16()
    qsl, lens = torch.tensor([0, T], dtype=torch.int32, device="cuda"), torch.tensor([L], dtype=torch.int32, device="cuda")
    word = torch.zeros(1, dtype=torch.int32, device="cuda")

    def timed():
        best = math.inf
        for _ in range(4):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            out, lse = pkv.kv8_attention(q, kc, vc, sc, sc, table, qsl, lens, d_error=word.data_ptr())
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return out, lse, best

    plain, plain_lse, plain_ms = timed()
    want = torch.zeros(T, d, dtype=torch.bool)
    pos = torch.arange(L - T, L)
    for at, dim in ((3, 5), (70001, 33), (136000, 63), (136001, 62), (139990, 1)):
        vc[int(table[0, at // bs]) * bs + at % bs, dim] = 127 if at % 2 else 255
        want[:, dim] |= pos >= at
    out, lse, ms = timed()
    assert word.item() == 0 and torch.equal(lse, plain_lse)
    assert torch.equal(out.isnan().cpu(), want[:, None].expand(T, group, d))
    same = ~want.cuda()[:, None].expand(T, group, d)
    assert torch.equal(out[same], plain[same])
    assert ms < 4 * plain_ms, (ms, plain_ms)


@pytest.mark.parametrize("reqs", [[(1, 90), (1, 70), (1, 200), (1, 64)], [(1, 90), (30, 70), (80, 200), (3, 64)]],
                         ids=["decodes", "mixed"])
def test_blocks_shared_by_requests(reqs):
    """Requests with a common prefix on the same blocks: each block adds up what every request gave it."""
    case = Case(reqs, 16, 2, 4, 128, seed=26)
    for i in range(1, len(reqs)):
        case.tables[i, :3] = case.tables[0, :3]
    check(case)
    case.tables[1, 3] = case.tables[0, 3]                    # one that the first request fills further
    check(case, window=50)
