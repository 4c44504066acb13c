"""kv4_attention where a request's pieces are far apart in size; against the plain implementation in 64 bits, with
the tolerances of test_kv4_attention_gpu."""
import pytest

from tests.test_kv4_attention_gpu import Case, check

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_prep_gb300 import build as pbuild
    pbuild.build()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("reqs", [[(1, 3100), (1, 900)], [(4, 3100), (3, 900)], [(70, 5000), (1, 900)], [(1, 1500)] * 150],
                         ids=["decodes", "drafts", "chunk", "many"])
def test_a_nan_in_a_piece_whose_weights_vanish(reqs, d):
    """The first third of each context has logits of 0 and the rest of 2 d (256 and more binary orders above): a piece
    of the first third alone weighs nothing beside the others, but its NaN key reaches the rows that see it."""
    case = Case(reqs, 16, 2, 4, d, seed=31)
    case.rows.fill_(2.0)
    case.caches[0].fill_(0x22)                               # ones
    for i, (_, x) in enumerate(reqs):
        s = torch.arange(x)
        block = case.tables[i].long()[s // 16]
        case.scales[0][block, :, s % 16] = torch.where(s < x // 3, 0, 0x38).to(torch.uint8)[:, None, None]
        if i != 1:                                           # one request has no NaN
            case.scales[0][int(case.tables[i, 0]), 1, 10, 2] = 127
    out, lse = check(case, scale=1.0)
    assert out[0, 4:].isnan().all() and out[0, :4].isfinite().all() and out[case.starts[1]:case.starts[2]].isfinite().all()
