"""kv4_attention on the GPU against its plain implementation in 64 bits.

Tolerances, with A = sum p |v| of an output element, X = a row's largest sum
|q k| softmax_scale, n = the tokens a row sees, V = the cache's largest |value| and the half
steps 2^-11 (f16), 2^-8 (bf16), 2^-24 (fp32): a logit is a sum of exact products in
fp32, off by at most 2^-19 X (room for sixteen half-step roundings along it twice over); it
is scaled and moved by the reference with roundings of values of its own size (2^-22 |lse|) and of the
difference (up to 32 where a weight matters: 2^-19), and the exponential is off by two units
(2^-22): 2^-18 in all.  A weight is rounded to f16, 2^-11 of itself, or 2^-25 where it is below
2^-14; the row's largest is above 2^8, and one that moved with its reference is rounded twice, so n
tokens are off by n 2^-32 V together.  Sums in fp32 add 2^-17 of A; the output is rounded once."""
import math

import pytest

import paged_kv_prep_gb300 as pkv
import pkv_workloads as workloads
from tests import kv4_reference as ref
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
    def __init__(self, reqs, bs, heads, group, d, dtype=torch.bfloat16, seed=1, lo=40, hi=56, pad=0, width=0, magnitude=1.0,
                 units=(1.0, 1.0)):
        """reqs: (scheduled tokens, cached tokens) of each request; lo, hi: the e4m3 codes of the scales."""
        gen = torch.Generator().manual_seed(seed)
        self.gen, self.bs, self.heads, self.group, self.d, self.dtype, self.units = gen, bs, heads, group, d, dtype, units
        self.lens = [x for _, x in reqs]
        self.starts = [0]
        for c, _ in reqs:
            self.starts.append(self.starts[-1] + c)
        need = [max(0, -(-x // bs)) for x in self.lens]
        self.blocks = sum(need) + 2
        perm = torch.randperm(self.blocks, generator=gen)
        self.tables = torch.full((len(reqs), max(max(need), 1) + width), -1, dtype=torch.int32)
        at = 0
        for i, n in enumerate(need):
            self.tables[i, :n] = perm[at:at + n]
            at += n
        # every scale a NaN first: whatever is not a cached token must not be read into a sum
        self.caches = [torch.randint(0, 256, (self.blocks, heads, bs, d // 2), generator=gen, dtype=torch.uint8) for _ in range(2)]
        self.scales = [torch.full((self.blocks, heads, bs, d // 16), 127, dtype=torch.uint8) for _ in range(2)]
        for i, x in enumerate(self.lens):
            if x > 0:
                s = torch.arange(x)
                b = self.tables[i].long()[s // bs]
                for c in self.scales:
                    c[b, :, s % bs] = torch.randint(lo, hi + 1, (x, heads, d // 16), generator=gen, dtype=torch.uint8)
        T, hq = self.starts[-1], heads * group
        self.rows = (torch.randn(T, hq * d + pad, generator=gen) * magnitude).to(dtype)
        self.q = self.rows[:, :hq * d].unflatten(1, (hq, d))

    def args(self):
        q = self.rows.cuda()[:, :self.q.shape[1] * self.d].unflatten(1, self.q.shape[1:])
        return (q, *[x.cuda() for x in self.caches + self.scales], self.tables.cuda(),
                torch.tensor(self.starts, dtype=torch.int32).cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda())

    def kw(self):
        return dict(k_unit=self.units[0], v_unit=self.units[1])

    def reference(self, scale, window):
        units = [float(torch.tensor(u)) for u in self.units]
        return ref.attention(self.q, self.caches, self.scales, units, self.tables, self.starts, self.lens, scale, window)

    def largest(self):
        s = ref.e4m3(self.scales[1])
        return float(s[~s.isnan()].max()) * 6 * self.units[1] if (~s.isnan()).any() else 0.0


def compare(case, out, lse, want):
    w_out, w_lse, size, reach, count = want
    out, lse = out.cpu().double(), lse.cpu().double()
    assert torch.equal(torch.isinf(lse), torch.isinf(w_lse)) and torch.equal(lse.isnan(), w_lse.isnan())
    fine = torch.isfinite(w_lse)
    logit = 2.0 ** -19 * reach + 2.0 ** -22 * w_lse.abs().nan_to_num().clamp(max=1e30) + 2.0 ** -18
    assert (((lse - w_lse).abs() <= logit)[fine]).all(), float((lse - w_lse)[fine].abs().max())
    assert torch.equal(out.isnan(), w_out.isnan())
    tol = (2.0 ** -11 + 2.0 ** -17 + 2 * logit[..., None]) * size + count[:, None, None] * 2.0 ** -32 * case.largest()
    tol = tol + HALF[case.dtype] * (w_out.abs() + tol) + 2.0 ** -25
    bad = (out - w_out).abs() > tol
    bad &= ~w_out.isnan()
    assert not bad.any(), (int(bad.sum()), float(((out - w_out).abs() / tol)[bad].max()))


def check(case, window=0, scale=None):
    scale = case.d ** -0.5 if scale is None else scale
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = pkv.kv4_attention(*case.args(), softmax_scale=scale, window=window, d_error=word.data_ptr(), **case.kw())
    assert word.item() == 0
    compare(case, out, lse, case.reference(scale, window))
    return out, lse


DECODES = [(1, x) for x in (1, 15, 16, 17, 200, 33, 640, 1000)]
MIXED = [(1, 1), (1, 77), (2, 2), (3, 50), (5, 5), (17, 100), (40, 90), (1, 300)]
CHUNKS = [(1, 20), (9, 9), (33, 33), (64, 64), (65, 200), (130, 131), (200, 1500), (257, 700)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("heads,group,d", [(8, 4, 128), (2, 8, 128), (1, 1, 128), (3, 5, 64), (2, 7, 256), (1, 12, 64),
                                           (5, 1, 64), (2, 3, 256), (1, 40, 128)])
@pytest.mark.parametrize("reqs", [DECODES, MIXED], ids=["decodes", "mixed"])
def test_matches_plain(reqs, heads, group, d, dtype):
    check(Case(reqs, 16, heads, group, d, dtype, seed=heads * 100 + group))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("heads,group,d", [(2, 4, 128), (1, 8, 128), (3, 1, 128), (2, 5, 64), (1, 33, 64), (1, 4, 256)])
def test_chunks_match_plain(heads, group, d, dtype):
    check(Case(CHUNKS, 16, heads, group, d, dtype, seed=heads * 100 + group))


@pytest.mark.parametrize("bs", [16, 32, 48, 64, 112, 1024])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_block_sizes(bs, d):
    check(Case(MIXED + [(1, 333), (90, 300)], bs, 2, 4, d, seed=bs, width=2))


@pytest.mark.parametrize("window", [1, 2, 16, 17, 30, 64, 100, 128, 1000, 4096, 2 ** 31 - 1])
@pytest.mark.parametrize("d", [64, 128])
def test_windows(window, d):
    check(Case(MIXED + CHUNKS[4:] + [(1, 1), (30, 33)], 16, 2, 4, d, seed=window % 97), window=window)


@pytest.mark.parametrize("units", [(1.0, 1.0), (2.0 ** -20, 2.0 ** 30), (0.3, 7.0)])
@pytest.mark.parametrize("reqs", [DECODES, MIXED + [(64, 300)]], ids=["decodes", "mixed"])
def test_units(reqs, units):
    scale = 128 ** -0.5 / units[0]
    check(Case(reqs, 16, 2, 4, 128, seed=3, units=units), scale=scale)


@pytest.mark.parametrize("scale", [0.0, -0.1, 1.0, 1e-30])
@pytest.mark.parametrize("reqs", [DECODES, MIXED + [(64, 300)]], ids=["decodes", "mixed"])
def test_softmax_scales(reqs, scale):
    check(Case(reqs, 16, 2, 4, 128, seed=4), scale=scale)


@pytest.mark.parametrize("reqs", [[(1, 100), (1, 33), (1, 250)], [(1, 100), (6, 60)], [(40, 100), (100, 300)]],
                         ids=["decodes", "short", "chunks"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_rows_keep_what_is_small_in_the_cache(reqs, dtype):
    """Value scales over all of e4m3, 2^-9 to 448, and sharp logits: the tolerance's last term is what a weight
    far below the row's largest may lose."""
    case = Case(reqs, 16, 2, 4, 128, dtype, seed=5, magnitude=4.0)
    some = case.scales[1] != 127
    case.scales[1][some] = torch.randint(1, 127, (int(some.sum()),), generator=case.gen, dtype=torch.uint8)
    check(case)


def test_extreme_queries_and_logits():
    case = Case(MIXED + [(64, 300)], 16, 2, 4, 128, seed=6)
    case.rows[0] = 0.0
    case.rows[2] *= 2.0 ** 60
    case.rows[4] *= 2.0 ** -80
    case.rows[6, ::3] *= 2.0 ** 30
    case.rows[30] *= 2.0 ** 40
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = pkv.kv4_attention(*case.args(), d_error=word.data_ptr())
    assert word.item() == 0
    want = case.reference(128 ** -0.5, 0)
    # a row whose logits are off by more than a weight is held to its lse
    soft = 2.0 ** -19 * want[3] < 2.0 ** -4
    w = [x.clone() for x in want]
    hard = ~soft
    got = out.cpu().double()
    got[hard], w[0][hard] = 0.0, 0.0
    compare(case, got, lse, w)
    assert out.isfinite().all()


@pytest.mark.parametrize("reqs", [[(1, 90), (1, 200)], [(5, 90), (12, 100)], [(70, 90), (100, 500), (1, 64)]], ids=["decodes", "short", "chunks"])
def test_nan_keys_stay_with_the_rows_that_see_them(reqs):
    case = Case(reqs, 16, 2, 4, 128, seed=7)
    for i, s, h, g in ((0, 88, 1, 3), (0, 3, 0, 0), (1, 97, 0, 7), (1, 60, 1, 1)):
        case.scales[0][int(case.tables[i, s // 16]), h, s % 16, g] = 127
    check(case)
    check(case, window=16)


def test_scales_before_the_window_do_not_count():
    """Blocks given away before the window hold anything, NaN value scales among it."""
    for reqs in ([(1, 300), (1, 77)], [(4, 300), (3, 90)], [(100, 300), (70, 200)]):
        case = Case(reqs, 16, 2, 4, 128, seed=8)
        window = 40
        for i, (c, x) in enumerate(reqs):
            for s in range(max(0, x - c - window + 1)):
                b = int(case.tables[i, s // 16])
                for f in case.scales:
                    f[b, :, s % 16] = 255
        check(case, window=window)


@pytest.mark.parametrize("group", [4, 16])
def test_rows_that_see_nothing(group):
    case = Case([(1, 60), (3, 50), (1, 0), (70, 200), (2, 1)], 16, 2, group, 128, seed=9)
    case.lens[4] = 1                                         # more queries than cached tokens: the first sees nothing
    case.tables[0] = -1
    case.tables[1, :2] = -1
    case.tables[3, 2:9] = -1
    out, lse = check(case)
    assert (out[0] == 0).all() and (lse[0] == -math.inf).all()
    check(case, window=3)


def test_bad_tables_are_reported_and_not_read():
    case = Case([(1, 100), (1, 60), (1, 30), (2, 20), (80, 300)], 16, 2, 4, 128, seed=10)
    case.tables[0, 2] = case.blocks
    case.tables[1, 0] = 2 ** 31 - 1
    case.tables[4, 5] = -7
    a = list(case.args())
    a[7] = a[7].clone()
    a[7][2] = case.tables.shape[1] * 16 + 40                # longer than the table: the rest is not seen
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = pkv.kv4_attention(*a, d_error=word.data_ptr())
    assert word.item() == pkv.DEVERR_BLOCK
    case.lens[2] = int(a[7][2])
    compare(case, out, lse, case.reference(case.d ** -0.5, 0))
    case.tables[4, 3] = case.blocks + 1
    a[5] = case.tables.cuda()
    word.zero_()
    out, lse = pkv.kv4_attention(*a, d_error=word.data_ptr())
    assert word.item() == pkv.DEVERR_BLOCK
    compare(case, out, lse, case.reference(case.d ** -0.5, 0))


def test_bad_locations_skip_the_request():
    case = Case([(1, 30), (1, 40), (2, 20), (1, 10)], 16, 2, 4, 128, seed=11)
    a = list(case.args())
    a[6] = torch.tensor([0, 1, 2, 1, 900], dtype=torch.int32).cuda()
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full(a[0].shape, 7.0, dtype=a[0].dtype, device="cuda")
    lse = torch.full(a[0].shape[:2], 7.0, device="cuda")
    pkv.kv4_attention(*a, out=out, lse=lse, d_error=word.data_ptr())
    assert word.item() == pkv.DEVERR_COUNT
    want = case.reference(case.d ** -0.5, 0)
    assert (out.cpu().double() - want[0])[:2].abs().max() < 2.0 ** -6 * want[2][:2].max()
    assert (out[2:] == 7.0).all() and (lse[2:] == 7.0).all()


def test_rows_behind_the_last_request_stay():
    case = Case(MIXED, 16, 2, 4, 128, seed=12)
    a = list(case.args())
    T = case.starts[-1]
    a[0] = torch.cat([a[0], a[0][:5]])
    out = torch.full(a[0].shape, 7.0, dtype=a[0].dtype, device="cuda")
    lse = torch.full(a[0].shape[:2], 7.0, device="cuda")
    pkv.kv4_attention(*a, out=out, lse=lse)
    compare(case, out[:T], lse[:T], case.reference(case.d ** -0.5, 0))
    assert (out[T:] == 7.0).all() and (lse[T:] == 7.0).all()


def test_strided_rows_and_given_buffers():
    """q as a view of fused projection rows, out as a view of wider rows, a workspace kept by the caller."""
    case = Case(MIXED + [(64, 90)], 16, 2, 4, 128, seed=13, pad=2 * 2 * 128)
    a = case.args()
    assert a[0].stride(0) == (8 + 4) * 128
    wide = torch.full((a[0].shape[0], 8 * 128 + 64), 5.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, :8 * 128].unflatten(1, (8, 128))
    lse = torch.empty(a[0].shape[0], 8, device="cuda")
    ws = torch.full((pkv.kv4_attention_workspace(128),), 255, dtype=torch.uint8, device="cuda")
    want = case.reference(case.d ** -0.5, 0)
    for _ in range(2):
        pkv.kv4_attention(*a, out=out, lse=lse, workspace=ws)
        compare(case, out, lse, want)
        assert (wide[:, 8 * 128:] == 5.0).all()
    assert pkv.kv4_attention(*a, workspace=ws[:1024], check=False) == pkv.ERR_INVALID_ARG


def test_repeats_are_bit_identical_and_streams_and_capture():
    case = Case(MIXED + [(1, 2000), (64, 400)], 16, 2, 4, 128, seed=14)
    a = case.args()
    first = pkv.kv4_attention(*a)
    for _ in range(3):
        again = pkv.kv4_attention(*a)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        other = pkv.kv4_attention(*a, stream=stream)
        side.synchronize()
        assert torch.equal(first[0], other[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out, lse = pkv.kv4_attention(*a)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first[0], out) and torch.equal(first[1], lse)


def test_two_calls_at_once():
    """On two streams, each with its own workspace."""
    cases = [Case(MIXED + [(1, 3000)], 16, 2, 4, 128, seed=15), Case(CHUNKS, 16, 2, 4, 128, seed=16)]
    args = [c.args() for c in cases]
    want = [pkv.kv4_attention(*a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        got = [pkv.kv4_attention(*a, stream=s) for a, s in zip(args, streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


def test_one_long_request_is_split():
    check(Case([(1, 20000)], 16, 1, 4, 128, seed=17))
    check(Case([(5, 6000)], 32, 2, 3, 64, seed=18))


def test_many_requests():
    """More requests than a CTA has threads, short tables (a warp takes a whole row tile), requests without tokens."""
    gen = torch.Generator().manual_seed(2)
    lens = torch.randint(0, 8, (3000,), generator=gen).tolist()
    check(Case([(int(torch.randint(0, x + 1, (1,), generator=gen)) if x else 0, x) for x in lens], 16, 1, 3, 64, seed=19))
    lens = torch.randint(1, 250, (60,), generator=gen).tolist()
    check(Case([(1, x) for x in lens], 16, 8, 4, 64, seed=20))
    check(Case([(1 + x % 3, x + 2) for x in lens] + [(30, 100)], 16, 8, 4, 128, seed=21), window=100)


@pytest.mark.parametrize("group,run", [(1, 3), (4, 4), (7, 2), (16, 1), (12, 2)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_long_chains_of_pieces(d, group, run):
    """Few requests, long contexts: every row in many pieces, the last tile of few rows, one request next to nothing."""
    check(Case([(run, 7000), (1, 3), (run, 2001)], 16, 2, group, d, seed=27))


@pytest.mark.parametrize("d,heads", [(64, 2), (128, 2), (128, 1)])
@pytest.mark.parametrize("reqs", [[(300, 700), (1, 90), (0, 5), (1, 1), (5, 260), (1, 2000)], [(70, 70)], [(9, 500)]])
def test_small_batches_with_chunks(reqs, d, heads):
    """Between narrow tables and wide ones the kernels change; a window ends a request's units early."""
    for width in (None, 20000):
        case = Case(reqs, 16, heads, 4, d, seed=28)
        if width:
            case.tables = torch.cat([case.tables, torch.full((len(reqs), width - case.tables.shape[1]), -1, dtype=torch.int32)], 1)
        check(case)
        check(case, window=100)


@pytest.mark.parametrize("d,bs,window", [(64, 16, 0), (128, 32, 9)])
def test_many_chunks(d, bs, window):
    """More requests than a CTA has threads, of more rows than the decode kernel takes; single and no tokens between them."""
    gen = torch.Generator().manual_seed(3)
    runs = torch.randint(9, 80, (1500,), generator=gen).tolist()
    check(Case([(0 if x % 7 == 0 else 1 if x % 11 == 0 else x, x + x % 5) for x in runs], bs, 2, 4, d, seed=24), window=window)


def test_two_graphs_share_a_workspace():
    """Replayed in turn on one stream: a call leaves nothing in the workspace that the next one reads."""
    cases = [Case(MIXED + [(1, 3000)], 16, 2, 4, 128, seed=25), Case(CHUNKS, 16, 2, 4, 128, seed=26)]
    args = [c.args() for c in cases]
    work = torch.empty(pkv.kv4_attention_workspace(128), dtype=torch.uint8, device="cuda")
    work.fill_(0xff)
    want = [pkv.kv4_attention(*a) for a in args]
    got = [[torch.zeros_like(x) for x in w] for w in want]
    graphs, stream = [], torch.cuda.Stream()
    torch.cuda.synchronize()
    for a, (out, lse) in zip(args, got):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            pkv.kv4_attention(*a, out=out, lse=lse, workspace=work)
        graphs.append(graph)
    for which in (0, 1, 1, 0, 1):
        for x in got[which]:
            x.zero_()
        graphs[which].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, w) for x, w in zip(got[which], want[which]))


@pytest.mark.parametrize("reqs", [[(1, 5), (1, 3)], [(2, 4), (1, 3)]], ids=["decodes", "mixed"])
@pytest.mark.parametrize("heads,d", [(1024, 256), (1024, 64), (1023, 128)])
def test_more_heads_than_warps(heads, d, reqs):
    check(Case(reqs, 16, heads, 1, d, seed=22))


def test_no_tokens():
    case = Case([(1, 5)], 16, 1, 1, 64)
    q, kc, vc, ks, vs, tab, qsl, lens = case.args()
    out, lse = pkv.kv4_attention(q[:0], kc, vc, ks, vs, tab[:0], qsl[:1], lens[:0])
    assert out.shape == (0, 1, 64) and lse.shape == (0, 1)


def test_cache_past_32_bits():
    """Blocks whose bytes start past 2^32."""
    heads, group, d, bs = 8, 4, 128, 16
    blocks = 600000
    small = Case([(1, 60), (3, 20), (50, 70)], bs, heads, group, d, seed=23)
    q, kc, vc, ks, vs, tab, qsl, lens = small.args()
    shift = blocks - small.blocks
    big = [torch.full((blocks, heads, bs, d // n), 127, dtype=torch.uint8, device="cuda") for n in (2, 2, 16, 16)]
    for b, c in zip(big, (kc, vc, ks, vs)):
        b[shift:] = c
    want = pkv.kv4_attention(q, kc, vc, ks, vs, tab, qsl, lens)
    got = pkv.kv4_attention(q, *big, torch.where(tab >= 0, tab + shift, tab), qsl, lens)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_what_a_call_makes_is_not_in_use_by_the_current_stream(raw):
    """Work queued on the current stream still writes to tensors of the sizes that a call on another stream
    makes, freed before it: the call's outputs and workspace are not theirs, and the call does not wait for
    that work."""
    case = Case([(1, 300), (1, 40), (40, 90)], 16, 2, 4, 128, seed=24)
    a = case.args()
    T, hq, d = a[0].shape
    want = case.reference(d ** -0.5, 0)
    side = torch.cuda.Stream()
    stream = side.cuda_stream if raw else side
    sizes = [T * hq * d * 2, T * hq * 4, pkv.kv4_attention_workspace(d)]
    torch.empty(1, dtype=torch.uint8, device="cuda").fill_(255)
    torch.cuda._sleep(1000)
    torch.cuda.synchronize()
    pkv.kv4_attention(*a, stream=stream)                     # kernels are loaded and that stream's pool filled: both may wait
    torch.cuda.synchronize()
    done = torch.cuda.Event()
    theirs = [torch.empty(x, dtype=torch.uint8, device="cuda") for x in sizes]
    at = {(x.data_ptr(), x.data_ptr() + x.numel()) for x in theirs}
    torch.cuda._sleep(400_000_000)
    for x in theirs:
        x.fill_(255)
    done.record()
    del theirs, x
    out, lse = pkv.kv4_attention(*a, stream=stream)
    side.synchronize()
    assert not done.query()                                  # the current stream's work is still to come
    for y in (out, lse):
        lo, hi = y.data_ptr(), y.data_ptr() + y.numel() * y.itemsize
        assert all(hi <= p or lo >= q for p, q in at)
    torch.cuda.synchronize()
    compare(case, out, lse, want)


def test_a_step_with_drafts():
    """prepare_batch -> kv4_store with the rotation -> kv4_attention -> verify_drafts -> the state, as a step of a
    few requests with drafted tokens uses them."""
    heads, group, d, bs, vocab, most = 2, 4, 128, 16, 500, 3
    st = pkv.State(8, 256, [(bs, 16, 64)])
    gen = torch.Generator().manual_seed(25)
    history, drafts = [40, 17, 90], [3, 0, 2]
    rows, tokens = [], []
    for i, (n, k) in enumerate(zip(history, drafts)):
        ids = torch.randint(0, vocab, (n + 1 + k,), generator=gen).tolist()
        tokens.append(ids)
        rows.append(st.add_request(ids, n, [list(range(8 * i, 8 * i + 8))]))
    batch = st.prepare_batch(rows, [1 + k for k in drafts])
    T = batch.total_tokens
    cache = [torch.zeros(64, heads, bs, n, dtype=torch.uint8) for n in (d // 2, d // 2, d // 16, d // 16)]
    for c in cache[:2]:
        c.copy_(torch.randint(0, 256, c.shape, generator=gen, dtype=torch.uint8))
    for c in cache[2:]:
        c.copy_(torch.randint(40, 57, c.shape, generator=gen, dtype=torch.uint8))
    dev = [c.cuda() for c in cache]
    q = torch.randn(T, heads * group, d, generator=gen).bfloat16()
    k, v = (torch.randn(T, heads, d, generator=gen).bfloat16() for _ in range(2))
    pair = torch.arange(d // 2, dtype=torch.float64)
    ang = torch.arange(256, dtype=torch.float64)[:, None] * 10000.0 ** (-pair / (d // 2))
    table = torch.cat([ang.cos(), ang.sin()], 1).float()
    slots = batch.slot_mapping[0]
    turned = pkv.kv4_store(k.cuda(), v.cuda(), *dev, slots, batch.positions, table.cuda(), q=q.cuda(), d_error=st.error_word)
    out, lse = pkv.kv4_attention(turned, *dev, batch.block_tables[0], batch.query_start_loc, batch.seq_lens, d_error=st.error_word)

    pos = batch.positions.cpu()[None]
    keys = ref.rotate32(k, pos, table, None, False)
    ref.store(keys.double(), v.double(), cache[:2], cache[2:], slots.cpu(), 1.0, 1.0)
    assert all(torch.equal(a.cpu(), b) for a, b in zip(dev[2:], cache[2:]))
    assert all(torch.equal(ref.unpack(a.cpu()), ref.unpack(b)) for a, b in zip(dev[:2], cache[:2]))
    case = Case([(1, 1)], bs, heads, group, d)
    case.q, case.caches, case.scales, case.dtype = ref.rotate32(q, pos, table, None, False).bfloat16(), cache[:2], cache[2:], torch.bfloat16
    assert torch.equal(turned.cpu(), case.q)
    case.tables, case.starts, case.lens = batch.block_tables[0].cpu(), batch.query_start_loc.tolist(), batch.seq_lens.tolist()
    compare(case, out, lse, case.reference(d ** -0.5, 0))

    # a head on the output gives the target's probabilities; the drafts are the batch's own input ids
    head = torch.randn(heads * group * d, vocab, generator=gen) * 0.02
    probs = torch.softmax(out.float().flatten(1) @ head.cuda(), -1)
    ids = batch.input_ids
    u = torch.rand(T, generator=gen).cuda()
    for t in (0, 2):                                         # some drafts are sure to stand
        probs[t, ids[t + 1].long()] = 1.0
    got, accepted = pkv.verify_drafts(probs, ids[1:], batch.query_start_loc, u, most, d_error=st.error_word)
    want = ref.verify(probs.cpu(), ids[1:].cpu(), case.starts, u.cpu(), most)
    assert torch.equal(got.cpu(), want[0]) and torch.equal(accepted.cpu(), want[1])
    assert st.get_error() == 0
    order = batch.index_mapping.tolist()
    for i, row in enumerate(order):
        j = rows.index(row)
        stand = int(accepted[i])
        assert got[i, :stand].tolist() == tokens[j][history[j] + 1:history[j] + 1 + stand]
        st.update_request(row, num_computed=history[j] + 1 + stand)
    st.close()
