"""kv8_attention: a NaN value in a piece of a request that weighs nothing beside the others, and the ends of
the integers that count positions."""
import math

import pytest

import paged_kv_prep_gb300 as pkv
from tests.test_kv8_attention_gpu import Case, compare

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_prep_gb300 import build as pbuild
    pbuild.build()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("reqs", [[(1, 3100), (1, 900)], [(4, 3100), (3, 900)], [(300, 3000), (1, 900)]],
                         ids=["decodes", "drafts", "chunk"])
def test_a_nan_in_a_piece_whose_weights_vanish(reqs, d):
    """The first third of each context has logits of 0, the rest of 2 d: 0 times NaN is NaN."""
    case = Case(reqs, 16, 2, 4, d, seed=31)
    case.q.fill_(2.0)
    case.scales[0].fill_(1.0)
    for i, (_, x) in enumerate(reqs):
        s = torch.arange(x)
        slot = case.tables[i].long()[s // 16] * 16 + s % 16
        case.caches[0][slot] = torch.where(s < x // 3, 0, 0x38).to(torch.uint8)[:, None, None]      # 0 and 1
        if i == 0:
            case.caches[1][slot[10], 1, 5] = 127
    out, lse = pkv.kv8_attention(*case.args(), softmax_scale=1.0)
    compare(case, out, lse, case.reference(1.0, 0))
    nan = out[:case.starts[1]].isnan()
    # the queries of the chunk stand behind the NaN's token
    assert nan[:, 4:, 5].all() and not nan[:, :4].any() and int(nan.sum()) == 4 * nan.shape[0]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("reqs", [[(6, 2), (1, 40), (9, 3)], [(70, 5), (1, 40)]], ids=["drafts", "chunk"])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 5])
def test_windows_of_all_positions_before_the_first(reqs, d, window):
    """More queries than cached tokens: the first ones stand before position 0."""
    a = Case(reqs, 16, 2, 4, d, seed=32).args()
    out, lse = pkv.kv8_attention(*a, window=window)
    plain = pkv.kv8_attention(*a)
    assert torch.equal(out, plain[0]) and torch.equal(lse, plain[1])


@pytest.mark.parametrize("reqs", [(1, 4), (40, 8)], ids=["decode", "chunk"])
def test_lengths_up_to_the_largest_integer(reqs):
    """Tables that name one block of 2^24 tokens for all of 2^31 positions, of which those of the last are not seen.  Logits
    of 0 and values of 1: the output is 1, the log-sum the logarithm of the visible tokens' number (half a step of fp32 there
    is 2^-20; the sum's, logarithm's and product's roundings are less than four)."""
    T, group = reqs
    bs, most = 1 << 24, 2 ** 31 - (1 << 24)
    codes = [torch.full((bs, 64), c, dtype=torch.uint8, device="cuda") for c in (0, 0x38)]
    scales = [torch.ones(1, 1, device="cuda") for _ in range(2)]
    table = torch.zeros(1, 128, dtype=torch.int32, device="cuda")
    q = torch.ones(T, group, 64, dtype=torch.bfloat16, device="cuda")
    starts = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    for length, window in ((2 ** 31 - 1, 0), (most, 0), (most + 60, 100), (2 ** 31 - 1, 1000), (most, 100), (-7, 0), (-7, 5)):
        word.zero_()
        out, lse = pkv.kv8_attention(q, *codes, *scales, table, starts, torch.tensor([length], dtype=torch.int32, device="cuda"),
                                     window=window, d_error=word.data_ptr())
        assert word.item() == (pkv.DEVERR_BLOCK if length > most else 0)
        for j in range(T):
            pos = length - T + j
            seen = min(pos + 1, most) - (max(0, pos - window + 1) if window else 0)
            if seen > 0:
                assert (out[j] == 1.0).all() and ((lse[j] - math.log(seen)).abs() < 2.0 ** -18).all(), (length, window, j)
            else:
                assert (out[j] == 0.0).all() and (lse[j] == -math.inf).all(), (length, window, j)
