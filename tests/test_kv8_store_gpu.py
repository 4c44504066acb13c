"""kv8_store on the GPU against its plain implementation: scales and codes are
equal, untouched lines and scales included."""
import math

import pytest

import paged_kv_prep_gb300 as pkv
import pkv_workloads as workloads
from tests import kv8_reference as ref
from tests.gpu_helpers import build_states

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_prep_gb300 import build as pbuild
    pbuild.build()
    yield
    torch.cuda.empty_cache()


def filled(blocks, bs, heads, d, gen, spread=2):
    """A cache with arbitrary finite codes and power-of-two scales."""
    codes = torch.randint(0, 256, (blocks * bs, heads * d), generator=gen, dtype=torch.uint8)
    codes = torch.where(codes & 127 == 127, 5, codes).to(torch.uint8)
    scale = torch.exp2(torch.randint(-spread, spread + 1, (blocks, heads), generator=gen).float())
    return codes, scale


def check(k, v, slots, blocks, bs, heads, d, gen, err=0, spread=2):
    kc, ks = filled(blocks, bs, heads, d, gen, spread)
    vc, vs = filled(blocks, bs, heads, d, gen, spread)
    dev = [x.cuda() for x in (kc, vc, ks, vs)]
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.kv8_store(k.cuda() if not k.is_cuda else k, v.cuda() if not v.is_cuda else v, *dev, slots.cuda(),
                  d_error=word.data_ptr())
    assert word.item() == err
    shape = (blocks * bs, heads, d)
    ref.store(k.cpu().view(-1, heads, d), v.cpu().view(-1, heads, d), kc.view(shape), vc.view(shape), ks, vs,
              slots, blocks)
    assert torch.equal(dev[2].cpu(), ks) and torch.equal(dev[3].cpu(), vs)
    assert ref.same_codes(dev[0].cpu(), kc) and ref.same_codes(dev[1].cpu(), vc)


def runs_of(gen, bs, blocks, lengths):
    """slot_mapping of requests whose new tokens start anywhere in a block."""
    perm = torch.randperm(blocks, generator=gen).tolist()
    slots = []
    for n in lengths:
        at = int(torch.randint(0, bs, (1,), generator=gen))
        block = perm.pop()
        for _ in range(n):
            if at == bs:
                at, block = 0, perm.pop()
            slots.append(block * bs + at)
            at += 1
    return torch.tensor(slots, dtype=torch.int64)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("heads,d", [(1, 64), (8, 128), (2, 256), (5, 64), (3, 128)])
@pytest.mark.parametrize("bs,lengths", [(16, [1]), (16, [1] * 40), (32, [100, 1, 33, 64, 2]), (7, [50, 3]),
                                        (1, [20]), (100, [150, 1, 99]), (33, [31, 32, 33])])
def test_store_matches_plain(dtype, heads, d, bs, lengths):
    gen = torch.Generator().manual_seed(bs * 100 + len(lengths) + heads)
    blocks = sum(-(-n // bs) + 1 for n in lengths) + 3
    slots = runs_of(gen, bs, blocks, lengths)
    T = len(slots)
    mag = torch.exp2(torch.randint(-6, 7, (T, 1), generator=gen).float())
    k, v = [(torch.randn(T, heads * d, generator=gen) * mag).to(dtype) for _ in range(2)]
    check(k, v, slots, blocks, bs, heads, d, gen)


def test_strides_skips_and_bad_slots():
    """K and V as views of wider rows; -1 splits a run; a slot past the cache is reported and not stored."""
    gen = torch.Generator().manual_seed(5)
    heads, d, bs, blocks = 4, 128, 16, 12
    slots = runs_of(gen, bs, blocks - 2, [40, 9])
    slots[5] = slots[20] = -1
    slots[30] = blocks * bs + 3
    slots[31] = 1 << 40
    rows = torch.randn(len(slots), 3 * heads * d + 8, generator=gen).to(torch.bfloat16).cuda()
    k, v = rows[:, 8:8 + heads * d], rows[:, 8 + heads * d:8 + 2 * heads * d]
    kk = k.cpu().contiguous()
    vv = v.cpu().contiguous()
    # the -1 and bad slots split their block's run: later pieces of the same block must not be part of the
    # call, so they go too
    seen, previous = set(), None
    for t, s in enumerate(slots.tolist()):
        b = s // bs if 0 <= s < blocks * bs else None
        if b is not None and b != previous and b in seen:
            slots[t] = -1
            b = None
        if b is not None:
            seen.add(b)
        previous = b
    kc, ks = filled(blocks, bs, heads, d, gen)
    vc, vs = filled(blocks, bs, heads, d, gen)
    dev = [x.cuda() for x in (kc, vc, ks, vs)]
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.kv8_store(k, v, *dev, slots.cuda(), d_error=word.data_ptr())
    assert word.item() == pkv.DEVERR_SLOT
    ref.store(kk.view(-1, heads, d), vv.view(-1, heads, d), kc.view(-1, heads, d), vc.view(-1, heads, d), ks, vs,
              slots, blocks)
    assert torch.equal(dev[2].cpu(), ks) and ref.same_codes(dev[0].cpu(), kc) and ref.same_codes(dev[1].cpu(), vc)


def test_special_values():
    """Zeros, infinities, NaN, the largest bf16, values below the smallest scale."""
    gen = torch.Generator().manual_seed(6)
    heads, d, bs, blocks = 2, 64, 16, 8
    k = torch.randn(48, heads * d, generator=gen)
    k[0:16] = 0
    k[16, 3], k[17, 70], k[18, 5] = math.inf, -math.inf, math.nan
    k[32:48] *= 1e-30
    v = torch.randn(48, heads * d, generator=gen)
    v[5] = 3.3e38
    v[20:32] = math.nan
    slots = torch.cat([torch.arange(32, 48), torch.arange(64, 80), torch.arange(0, 16)])
    check(k.bfloat16(), v.bfloat16(), slots, blocks, bs, heads, d, gen)


def test_token_by_token_equals_plain_and_keeps_its_mantissas():
    """A block filled by sixteen single-token steps with growing values: every step equals the plain
    implementation, and codes that stay normal lose nothing by the rescaling."""
    gen = torch.Generator().manual_seed(7)
    heads, d, bs = 8, 128, 16
    kc = torch.zeros(2 * bs, heads * d, dtype=torch.uint8)
    vc, ks, vs = kc.clone(), torch.full((2, heads), 1.0), torch.full((2, heads), 1.0)
    dev = [x.cuda() for x in (kc, vc, ks, vs)]
    x = (torch.rand(bs, heads * d, generator=gen) + 0.5).bfloat16() * torch.exp2(torch.arange(bs).float() * 0.25)[:, None]
    x = x.bfloat16()
    for t in range(bs):
        slot = torch.tensor([bs + t])
        pkv.kv8_store(x[t:t + 1].cuda(), x[t:t + 1].cuda(), *dev, slot.cuda())
        ref.store(x[t:t + 1].view(1, heads, d), x[t:t + 1].view(1, heads, d), kc.view(-1, heads, d),
                  vc.view(-1, heads, d), ks, vs, slot, 2)
        assert torch.equal(dev[0].cpu(), kc) and torch.equal(dev[2].cpu(), ks)
    values = ref.decode(dev[0].cpu()[bs:]).view(bs, heads, d) * ks[1].double()[None, :, None]
    # one rounding to three mantissa bits: at most half a step, 2^-4 of the value
    assert ((values - x.double().view(bs, heads, d)).abs() <= 2.0 ** -4 * x.double().view(bs, heads, d).abs()).all()


def test_prepared_batch_other_stream_and_capture():
    """slot_mapping from prepare_batch; the store on a stream of its own and as a captured graph."""
    wl = workloads.random_small(seed=3, num_requests=20, max_ctx=200, max_chunk=40, decode_frac=0.5)
    st, _, rows_map = build_states(wl)
    rows, ns = workloads.schedule_arrays(wl, rows_map)
    batch = st.prepare_batch(rows, ns)
    T, heads, d = batch.total_tokens, 2, 128
    blocks, bs = wl.groups[0].num_blocks, wl.groups[0].block_size
    gen = torch.Generator().manual_seed(8)
    k, v = [torch.randn(T, heads, d, generator=gen).half() for _ in range(2)]
    kc, ks = filled(blocks, bs, heads, d, gen)
    want = [kc.clone(), kc.clone(), ks.clone(), ks.clone()]
    slots = batch.slot_mapping[0]
    ref.store(k, v, want[0].view(-1, heads, d), want[1].view(-1, heads, d), want[2], want[3], slots.cpu(), blocks)
    kd, vd = k.cuda(), v.cuda()
    for how in ("stream", "graph"):
        dev = [kc.cuda(), kc.cuda(), ks.cuda(), ks.cuda()]
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        if how == "stream":
            pkv.kv8_store(kd, vd, *dev, slots, stream=side)
        else:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                pkv.kv8_store(kd, vd, *dev, slots)
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a.cpu(), b) for a, b in zip(dev[2:], want[2:]))
        assert all(ref.same_codes(a.cpu(), b) for a, b in zip(dev[:2], want[:2]))
    st.close()


def test_no_tokens():
    kc = torch.zeros(32, 128, dtype=torch.uint8, device="cuda")
    sc = torch.ones(2, 1, device="cuda")
    k = torch.zeros(0, 1, 128, dtype=torch.float16, device="cuda")
    assert pkv.kv8_store(k, k, kc, kc, sc, sc, torch.zeros(0, dtype=torch.int64, device="cuda")) == pkv.OK


def test_slots_past_32_bits():
    """A cache of more than 2^32 bytes: the last blocks are addressed in 64 bits."""
    heads, d, bs, blocks = 8, 128, 16, 300000
    kc = torch.zeros(blocks * bs, heads * d, dtype=torch.uint8, device="cuda")
    ks = torch.ones(blocks, heads, device="cuda")
    k = torch.randn(20, heads, d, device="cuda").bfloat16()
    slots = torch.arange(blocks * bs - 32, blocks * bs - 12, device="cuda")
    vc, vs = torch.zeros_like(kc), torch.ones_like(ks)
    pkv.kv8_store(k, k, kc, vc, ks, vs, slots)
    small = torch.zeros(2 * bs, heads, d, dtype=torch.uint8)
    ss = torch.ones(2, heads)
    ref.store(k.cpu(), k.cpu(), small, small.clone(), ss, ss.clone(), torch.arange(0, 20), 2)
    assert torch.equal(kc[-32:].cpu().view(small.shape), small) and torch.equal(vc[-32:], kc[-32:])
    assert torch.equal(ks[-2:].cpu(), ss) and int(kc[:-32].max()) == 0


def test_more_tokens_than_a_round():
    """So many tokens that a CTA takes several segments of the line one after the other."""
    gen = torch.Generator().manual_seed(9)
    heads, d, bs = 2, 256, 32
    lengths = [9001, 700, 1, 33, 11003]
    blocks = sum(-(-n // bs) + 1 for n in lengths) + 3
    slots = runs_of(gen, bs, blocks, lengths)
    T = len(slots)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert -(-12 * sms // -(-T // 32)) < 2 * heads * d // 256
    mag = torch.exp2(torch.randint(-6, 7, (T, 1), generator=gen).float())
    k, v = [(torch.randn(T, heads * d, generator=gen) * mag).bfloat16() for _ in range(2)]
    check(k, v, slots, blocks, bs, heads, d, gen)
