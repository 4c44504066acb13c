"""verify_drafts on the GPU against its plain implementation: whole numbers, equal."""
import pytest

import paged_kv_prep_gb300 as pkv
from tests import kv4_reference as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_prep_gb300 import build as pbuild
    pbuild.build()
    yield
    torch.cuda.empty_cache()


def make(counts, vocab, dtype=torch.float32, seed=1, near=0.5, sharp=2.0, pad=0):
    """Target and draft rows (a stride of vocab + pad), drafts drawn from the draft's rows, uniforms."""
    gen = torch.Generator().manual_seed(seed)
    rows = sum(counts)
    logits = sharp * torch.randn(rows, vocab, generator=gen)
    wide = [torch.full((rows, vocab + pad), 3.0, dtype=dtype) for _ in range(2)]
    target, draft = (w[:, :vocab] for w in wide)
    target.copy_(torch.softmax(logits, -1))
    draft.copy_(torch.softmax(logits + near * torch.randn(rows, vocab, generator=gen), -1))
    ids = torch.multinomial(draft.float(), 1, generator=gen)[:, 0].int() if rows else torch.zeros(0, dtype=torch.int32)
    starts = [0]
    for c in counts:
        starts.append(starts[-1] + c)
    return target, draft, ids, starts, torch.rand(rows, generator=gen)


def on_gpu(x):
    return x.cuda() if x.is_contiguous() or x.numel() == 0 else x._base.cuda()[:, :x.shape[1]]


def check(target, ids, starts, u, most, draft=None, errors=0, word=True):
    w = torch.zeros(1, dtype=torch.int32, device="cuda")
    tokens, accepted = pkv.verify_drafts(on_gpu(target), ids.cuda(), torch.tensor(starts, dtype=torch.int32).cuda(), u.cuda(), most,
                                         draft_probs=None if draft is None else on_gpu(draft),
                                         d_error=w.data_ptr() if word else None)
    want = ref.verify(target.float(), ids, starts, u, most, None if draft is None else draft.float())
    assert torch.equal(accepted.cpu(), want[1]) and torch.equal(tokens.cpu(), want[0])
    assert w.item() == errors
    return tokens.cpu(), accepted.cpu()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("vocab", [1, 3, 129, 1000, 4096, 20011, 65537, 131072])
@pytest.mark.parametrize("with_draft", [True, False])
def test_matches_plain(vocab, dtype, with_draft):
    counts = [1, 2, 5, 4, 1, 3, 5]
    target, draft, ids, starts, u = make(counts, vocab, dtype, seed=vocab % 97)
    check(target, ids, starts, u, 4, draft if with_draft else None)


@pytest.mark.parametrize("pad", [1, 2, 3, 8, 61])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_apart(dtype, pad):
    """Rows at every alignment; the draft's at another one than the target's."""
    counts = [3, 4, 2, 1, 5] * 3
    target, draft, ids, starts, u = make(counts, 5003, dtype, seed=pad, pad=pad)
    check(target, ids, starts, u, 4, draft)
    tight = draft.contiguous()
    check(target, ids, starts, u, 4, tight)


def test_views_off_a_16_byte_boundary():
    target, draft, ids, starts, u = make([3, 2, 4], 1000, torch.float32, seed=4, pad=9)
    for shift in (1, 2, 3):
        t = target._base.cuda()[:, shift:shift + 900]
        q = draft._base.cuda()[:, 9:909]
        got = pkv.verify_drafts(t, ids.clamp(max=899).cuda(), torch.tensor(starts, dtype=torch.int32).cuda(), u.cuda(), 3, draft_probs=q)
        want = ref.verify(t.cpu(), ids.clamp(max=899), starts, u, 3, q.cpu())
        assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[1].cpu(), want[1])


def test_batches_of_all_sizes():
    for n, seed in ((1, 1), (2, 2), (300, 3), (2500, 4)):
        gen = torch.Generator().manual_seed(seed)
        counts = torch.randint(1, 8, (n,), generator=gen).tolist()
        target, draft, ids, starts, u = make(counts, 203, seed=seed)
        _, accepted = check(target, ids, starts, u, 7, draft)
        assert n < 300 or n / 4 < int(accepted.sum()) < sum(counts) - n - n / 4        # some fall, some stand


def test_more_drafts_than_a_warp_has_lanes():
    counts = [40, 100, 1, 33, 34]
    target, draft, ids, starts, u = make(counts, 64, seed=5, near=0.05)
    tokens, accepted = check(target, ids, starts, u, 99, draft)
    u = u * 0
    tokens, accepted = check(target, ids, starts, u, 99, draft)                 # every draft stands
    assert accepted.tolist() == [c - 1 for c in counts]


def test_uniforms_at_the_ends():
    target, draft, ids, starts, u = make([4, 4, 4, 4], 1000, seed=6)
    last = 1.0 - 2.0 ** -24
    for value in (0.0, last, 2.0 ** -30):
        check(target, ids, starts, torch.full_like(u, value), 3, draft)
        check(target, ids, starts, torch.full_like(u, value), 3)
    # the aim falls on a token's very border: the next one's turn
    p = torch.tensor([[0.25, 0.25, 0.0, 0.5]])
    for value, want in ((0.0, 0), (0.25, 1), (0.5, 3), (0.75, 3), (0.24999999, 0), (0.49999997, 1)):
        tokens, _ = check(p, torch.zeros(1, dtype=torch.int32), [0, 1], torch.tensor([value]), 0)
        assert tokens.tolist() == [[want]]


def test_what_is_subtracted_leaves_nothing():
    """Rejected with p == q everywhere (u = 1 is no uniform, but ends nothing): p itself is drawn from; a row of
    zeros gives -1."""
    p = torch.softmax(torch.randn(4, 300, generator=torch.Generator().manual_seed(7)), -1)
    ids = torch.tensor([5, 6, 7, 8], dtype=torch.int32)
    u = torch.tensor([1.0, 0.3, 0.9, 0.6])
    tokens, accepted = check(p, ids, [0, 4], u, 3, p.clone())
    assert accepted.tolist() == [0] and int(tokens[0, 0]) >= 0 and tokens[0, 1:].tolist() == [-1] * 3
    p[1] = 0.0
    tokens, accepted = check(p, ids, [0, 1, 2, 4], u, 3)
    assert int(tokens[1, 0]) == -1
    one = torch.zeros(2, 300)
    one[0, 5] = one[1, 9] = 1.0
    u = torch.tensor([0.99, 0.5])
    tokens, accepted = check(one, torch.tensor([5, 0], dtype=torch.int32), [0, 2], u, 1)      # certain on both sides
    assert tokens.tolist() == [[5, 9]] and accepted.tolist() == [1]
    tokens, accepted = check(one, torch.tensor([4, 0], dtype=torch.int32), [0, 2], u, 1)
    assert tokens.tolist() == [[5, -1]] and accepted.tolist() == [0]


def test_values_that_are_no_probabilities():
    target, draft, ids, starts, u = make([3, 3, 3, 3], 777, seed=8)
    target[1, 100:200] = float("nan")
    target[4, 5], target[7, 6] = float("inf"), -1.0
    draft[4, 50:90] = float("nan")
    draft[8, :] = float("inf")
    check(target, ids, starts, u, 2, draft)
    check(target * 5, ids, starts, u, 2, draft * 3)                             # weights above 1 count as 1
    ids[0], ids[3], ids[6] = -1, 777, 2 ** 31 - 1                                # drafts outside the vocabulary
    _, accepted = check(target, ids, starts, u, 2, draft)
    assert accepted[:3].tolist() == [0, 0, 0]
    check(target, ids, starts, u, 2)


def test_tiny_probabilities():
    """Below 2^-41 a weight counts as 0; halves of 2^-40 go to the even multiple."""
    p = torch.full((3, 64), 2.0 ** -41)
    p[0, 10] = 2.0 ** -40
    p[1, 11], p[1, 12] = 3 * 2.0 ** -41, 5 * 2.0 ** -41
    u = torch.tensor([0.0, 0.5, 0.5])
    tokens, _ = check(p, torch.zeros(3, dtype=torch.int32), [0, 1, 2, 3], u, 0)
    assert tokens.tolist() == [[10], [12], [-1]]


def test_bad_locations_skip_the_request():
    target, draft, ids, starts, u = make([3, 3, 3, 3], 100, seed=9)
    check(target, ids, [0, 3, 3, 6, 9, 12], u, 2, draft)                        # one without rows: no error
    check(target, ids, [0, 3, 2, 9, 9, 13], u, 2, draft, errors=pkv.DEVERR_COUNT)
    check(target, ids, [-1, 3, 6], u, 2, draft, errors=pkv.DEVERR_COUNT)
    check(target, ids, [0, 3, 6], u, 1, draft, errors=pkv.DEVERR_COUNT)         # more rows than max_drafts + 1
    check(target, ids, [0, 4], u, 2, draft, word=False, errors=0)


def test_streams_capture_and_given_outputs():
    counts = [1, 4, 3, 5, 2]
    target, draft, ids, starts, u = make(counts, 50021, seed=10)
    a = (target.cuda(), ids.cuda(), torch.tensor(starts, dtype=torch.int32).cuda(), u.cuda(), 4)
    want = pkv.verify_drafts(*a, draft_probs=draft.cuda())
    for _ in range(3):
        again = pkv.verify_drafts(*a, draft_probs=draft.cuda())
        assert torch.equal(want[0], again[0]) and torch.equal(want[1], again[1])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    q = draft.cuda()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        got = pkv.verify_drafts(*a, draft_probs=q, stream=stream)
        side.synchronize()
        assert torch.equal(want[0], got[0])
    tokens, accepted = torch.full((5, 5), 77, dtype=torch.int32, device="cuda"), torch.zeros(5, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.verify_drafts(*a, draft_probs=q, tokens=tokens, accepted=accepted)
    a[3].copy_(1 - a[3])
    graph.replay()
    torch.cuda.synchronize()
    want = ref.verify(target, ids, starts, a[3].cpu(), 4, draft)
    assert torch.equal(tokens.cpu(), want[0]) and torch.equal(accepted.cpu(), want[1])


def test_a_single_row_needs_no_draft_and_no_requests_no_rows():
    target, _, _, _, u = make([1], 500, seed=11)
    check(target, torch.zeros(0, dtype=torch.int32), [0, 1], u, 0)
    check(target, torch.zeros(0, dtype=torch.int32), [0, 1], u, 3)
    none = pkv.verify_drafts(target.cuda(), torch.zeros(0, dtype=torch.int32).cuda(), torch.zeros(1, dtype=torch.int32).cuda(), u.cuda(), 3)
    assert none[0].shape == (0, 4) and none[1].shape == (0,)
    empty = pkv.verify_drafts(target[:0].cuda(), torch.zeros(0, dtype=torch.int32).cuda(), torch.zeros(3, dtype=torch.int32).cuda(), u[:0].cuda(), 1)
    assert empty[0].tolist() == [[-1, -1], [-1, -1]] and empty[1].tolist() == [0, 0]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_largest_vocabulary_of_weights_that_are_no_probabilities(dtype):
    """2^22 tokens of weight 1 (and a stretch of smaller ones): a total of almost 2^62."""
    vocab = 1 << 22
    p = torch.ones(3, vocab, dtype=dtype)
    p[1, 1000:2000000] = 0.25
    p[2] = torch.rand(vocab, generator=torch.Generator().manual_seed(12)).to(dtype)
    check(p, torch.zeros(3, dtype=torch.int32), [0, 1, 2, 3], torch.tensor([0.999, 0.4, 0.6]), 0)
