"""kv4_attention with queries whose elements are many binary orders apart.

A row of queries is scaled so that its largest magnitude M lies in [2^14, 2^15) and rounded to f16, whose smallest step
is 2^-24: an element keeps all its bits down to 2^-28 M (fp16's 11 bits) or 2^-31 M (bf16's 8), and a smaller one is
off by half a step, 2^-25, at most, which is 2^-39 M.  Where the keys are zero in M's dimension these elements are the
whole logit: it is off by softmax_scale * sum |k| * 2^-39 M more than the tolerances of test_kv4_attention_gpu say."""
import pytest

import paged_kv_prep_gb300 as pkv
from tests import kv4_reference as ref
from tests.test_kv4_attention_gpu import Case, compare

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_prep_gb300 import build as pbuild
    pbuild.build()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype,apart", [(torch.bfloat16, 24), (torch.bfloat16, 34), (torch.bfloat16, 37), (torch.float16, 22), (torch.float16, 29)])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("reqs", [[(1, 100), (1, 33), (1, 250)], [(1, 100), (6, 60)], [(40, 100), (100, 300)]],
                         ids=["decodes", "short", "chunks"])
def test_an_outlier_that_meets_zeros(reqs, d, dtype, apart):
    """One dimension 2^apart times the others, which fp16 holds as subnormals in the widest case; logits of the others'
    size."""
    case = Case(reqs, 16, 2, 4, d, dtype, seed=41)
    top = 14 if dtype is torch.float16 else 20
    case.rows.copy_(case.rows.float() * 2.0 ** (top - apart))
    case.q[:, :, 5] = 2.0 ** top * (1 + case.q[:, :, 5].float().sign() / 2)
    case.caches[0][..., 2] &= 0x0f                           # dimension 5: the upper half of byte 2
    scale = 2.0 ** (apart - top) * d ** -0.5
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = pkv.kv4_attention(*case.args(), softmax_scale=scale, d_error=word.data_ptr())
    assert word.item() == 0
    w_out, w_lse, size, reach, count = case.reference(scale, 0)
    most = torch.where(case.scales[0] == 127, 0, case.scales[0])
    k = ref.values(case.caches[0], most, 1.0).abs().sum(-1).amax()                      # the largest sum |k|
    lost = float(scale * k) * 2.0 ** -39 * case.q.double().abs().amax(-1)
    compare(case, out, lse, (w_out, w_lse, size, reach + lost * 2.0 ** 19, count))      # the tolerance counts 2^-19 of it


@pytest.mark.parametrize("reqs", [[(1, 100), (1, 250)], [(100, 300)]], ids=["decodes", "chunks"])
def test_tiny_queries_lose_nothing(reqs):
    """bf16 rows far below 2^-100, subnormals among them: multiples of 2^-133, which times 2^114 f16 holds."""
    case = Case(reqs, 16, 2, 4, 128, seed=42)
    case.rows.copy_((case.rows.double() * 2.0 ** -122).to(torch.bfloat16))
    assert ((case.rows.double().abs() < 2.0 ** -126) & (case.rows != 0)).any()
    scale = 2.0 ** 120
    out, lse = pkv.kv4_attention(*case.args(), softmax_scale=scale)
    compare(case, out, lse, case.reference(scale, 0))
