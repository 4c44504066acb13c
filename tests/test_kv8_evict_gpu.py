"""kv8_evict on the GPU against its plain implementation: kept positions,
lengths, weights, scales and codes are equal."""
import math

import pytest

import paged_kv_prep_gb300 as pkv
from tests import kv8_reference as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_prep_gb300 import build as pbuild
    pbuild.build()
    yield
    torch.cuda.empty_cache()


def make(lens, bs, heads, d, budget, seed, shape="heavy", spread=3):
    gen = torch.Generator().manual_seed(seed)
    need = [-(-x // bs) for x in lens]
    more = [-(-min(x, budget) // bs) for x in lens]
    blocks = sum(need) + sum(more) + 2
    perm = torch.randperm(blocks, generator=gen).tolist()
    W, W2 = max(max(need), 1) + 1, -(-budget // bs)
    table, fresh = torch.full((len(lens), W), -1, dtype=torch.int32), torch.full((len(lens), W2), -1, dtype=torch.int32)
    for i in range(len(lens)):
        for j in range(need[i]):
            table[i, j] = perm.pop()
        for j in range(more[i]):
            fresh[i, j] = perm.pop()
    caches = []
    for _ in range(2):
        c = torch.randint(0, 256, (blocks * bs, heads * d), generator=gen, dtype=torch.uint8)
        caches.append(torch.where(c & 127 == 127, 9, c).to(torch.uint8))
    scales = [torch.exp2(torch.randint(-spread, spread + 1, (blocks, heads), generator=gen).float()) for _ in range(2)]
    w = torch.exp(3 * torch.randn(blocks * bs, generator=gen))
    if shape == "ties":
        w = torch.randint(0, 4, (blocks * bs,), generator=gen).float() * 0.5 - 0.5
        w[w == 0] *= torch.where(torch.rand(int((w == 0).sum()), generator=gen) < 0.5, -1.0, 1.0)
    elif shape == "special":
        pick = torch.randint(0, 6, (blocks * bs,), generator=gen)
        w = torch.where(pick == 0, math.nan, torch.where(pick == 1, math.inf, torch.where(pick == 2, -math.inf, w)))
        w = torch.where(pick == 3, 1e-42, w)
    elif shape == "equal":
        w = torch.ones(blocks * bs)
    return [*caches, *scales, w], table, fresh


def check(lens, bs, heads, d, budget, first, last, seed=1, shape="heavy"):
    state, table, fresh = make(lens, bs, heads, d, budget, seed, shape)
    dev = [x.cuda() for x in state]
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    new, kept = pkv.kv8_evict(*dev, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), fresh.cuda(), budget,
                              keep_first=first, keep_last=last, d_error=word.data_ptr())
    assert word.item() == 0
    kc, vc, ks, vs, w = state
    want_new, want_kept = ref.evict(kc.view(-1, heads, d), vc.view(-1, heads, d), ks, vs, w, table, lens, fresh,
                                    budget, first, last)
    assert new.tolist() == want_new
    assert torch.equal(kept.cpu(), want_kept)
    assert torch.equal(dev[2].cpu(), ks) and torch.equal(dev[3].cpu(), vs)
    assert torch.equal(torch.nan_to_num(dev[4].cpu(), nan=-7.0), torch.nan_to_num(w, nan=-7.0))
    assert ref.same_codes(dev[0].cpu(), kc) and ref.same_codes(dev[1].cpu(), vc)


@pytest.mark.parametrize("shape", ["heavy", "ties", "special", "equal"])
@pytest.mark.parametrize("lens,bs,budget,first,last", [
    ([200, 64, 65, 1, 0, 130], 16, 64, 4, 16), ([300, 77], 7, 50, 0, 0), ([2500, 1025], 32, 999, 1, 100),
    ([100], 16, 20, 5, 15), ([40, 9], 1, 8, 0, 8), ([500], 100, 130, 130, 0), ([33, 34], 48, 33, 1, 1)])
def test_evict_matches_plain(lens, bs, budget, first, last, shape):
    check(lens, bs, 2, 64, budget, first, last, seed=budget, shape=shape)


@pytest.mark.parametrize("heads,d", [(1, 64), (8, 128), (3, 256), (5, 128)])
def test_layouts(heads, d):
    check([150, 90], 16, heads, d, 61, 2, 9, seed=heads)


def test_long_request():
    check([70001, 3000], 32, 1, 64, 4097, 4, 64, seed=3)


def test_bad_tables_leave_a_request_alone():
    """A missing or foreign block, a table that is too short: the request is refused with -1 and
    nothing of it is written; the others go through."""
    lens, bs, heads, d, budget = [100, 100, 100, 100, 100], 16, 2, 64, 40
    state, table, fresh = make(lens, bs, heads, d, budget, 4)
    blocks = state[2].shape[0]
    table[0, 3] = -1
    table[1, 2] = blocks
    fresh[2, 1] = -1
    sent = list(lens)
    sent[3] = table.shape[1] * bs + 1
    dev = [x.cuda() for x in state]
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    new, kept = pkv.kv8_evict(*dev, table.cuda(), torch.tensor(sent, dtype=torch.int32).cuda(), fresh.cuda(), budget,
                              keep_first=2, keep_last=3, d_error=word.data_ptr())
    assert new.tolist() == [-1, -1, -1, -1, 40]
    assert int(kept[:4].max()) == -1
    assert word.item() == pkv.DEVERR_BLOCK | pkv.DEVERR_POSITION
    kc, vc, ks, vs, w = state
    _, want = ref.evict(kc.view(-1, heads, d), vc.view(-1, heads, d), ks, vs, w, table[4:], lens[4:], fresh[4:], budget, 2, 3)
    assert torch.equal(kept[4:].cpu(), want)
    assert ref.same_codes(dev[0].cpu(), kc) and ref.same_codes(dev[1].cpu(), vc) and torch.equal(dev[2].cpu(), ks)


def test_shared_source_blocks_stay():
    """Two requests that share their first blocks: the old blocks keep every byte."""
    lens, bs, heads, d, budget = [96, 96], 16, 2, 64, 40
    state, table, fresh = make(lens, bs, heads, d, budget, 5)
    table[1, :3] = table[0, :3]
    dev = [x.cuda() for x in state]
    new, kept = pkv.kv8_evict(*dev, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), fresh.cuda(), budget,
                              keep_last=8)
    kc, vc, ks, vs, w = [x.clone() for x in state]
    _, want = ref.evict(kc.view(-1, heads, d), vc.view(-1, heads, d), ks, vs, w, table, lens, fresh, budget, 0, 8)
    assert torch.equal(kept.cpu(), want) and ref.same_codes(dev[0].cpu(), kc)
    used = table[table >= 0].long().unique()
    for now, before in ((dev[0], state[0]), (dev[1], state[1])):
        assert torch.equal(now.cpu().view(-1, bs, heads * d)[used], before.view(-1, bs, heads * d)[used])


def test_other_stream_and_capture():
    lens, bs, heads, d, budget = [200, 300], 16, 2, 128, 64
    state, table, fresh = make(lens, bs, heads, d, budget, 6)
    want = [x.clone() for x in state]
    _, want_kept = ref.evict(want[0].view(-1, heads, d), want[1].view(-1, heads, d), *want[2:], table, lens, fresh, budget, 1, 4)
    tab, fr, ln = table.cuda(), fresh.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    for how in ("stream", "graph"):
        dev = [x.cuda() for x in state]
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        if how == "stream":
            _, kept = pkv.kv8_evict(*dev, tab, ln, fr, budget, keep_first=1, keep_last=4, stream=side)
        else:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                _, kept = pkv.kv8_evict(*dev, tab, ln, fr, budget, keep_first=1, keep_last=4)
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(kept.cpu(), want_kept)
        assert ref.same_codes(dev[0].cpu(), want[0]) and torch.equal(dev[4].cpu(), want[4])


def test_no_requests():
    state, table, fresh = make([16], 16, 1, 64, 8, 7)
    dev = [x.cuda() for x in state]
    new, kept = pkv.kv8_evict(*dev, table[:0].cuda(), torch.zeros(0, dtype=torch.int32).cuda(), fresh[:0].cuda(), 8)
    assert new.numel() == 0 and kept.shape == (0, 8)


def narrow(lens, bs, heads, d, budget, wide, seed):
    """New tables that hold `budget` tokens, as rows of a larger tensor, for calls with the larger budget `wide`."""
    state, table, fresh = make(lens, bs, heads, d, budget, seed)
    whole = torch.full((len(lens) * fresh.shape[1] + wide // bs + 1,), 2 ** 31 - 1, dtype=torch.int32)
    whole[:fresh.numel()] = fresh.view(-1)
    return state, table, fresh, whole.cuda()[:fresh.numel()].view(fresh.shape)


def test_new_tables_narrower_than_the_budget():
    """What fits the new table goes through; a request that does not is refused with its reason."""
    lens, bs, heads, d, wide = [20, 100, 32, 0, 33], 16, 2, 64, 4096
    state, table, fresh, given = narrow(lens, bs, heads, d, 32, wide, 8)
    dev = [x.cuda() for x in state]
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    new, kept = pkv.kv8_evict(*dev, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), given, wide,
                              keep_first=2, keep_last=3, d_error=word.data_ptr())
    assert new.tolist() == [20, -1, 32, 0, -1] and word.item() == pkv.DEVERR_POSITION
    kc, vc, ks, vs, w = state
    fits = [0, 2, 3]
    _, want = ref.evict(kc.view(-1, heads, d), vc.view(-1, heads, d), ks, vs, w, table[fits], [lens[i] for i in fits],
                        fresh[fits], wide, 2, 3)
    assert torch.equal(kept.cpu()[fits], want) and int(kept[[1, 4]].max()) == -1
    assert ref.same_codes(dev[0].cpu(), kc) and ref.same_codes(dev[1].cpu(), vc)
    assert torch.equal(dev[2].cpu(), ks) and torch.equal(dev[3].cpu(), vs) and torch.equal(dev[4].cpu(), w)


@pytest.mark.parametrize("lens,fits,wide", [([20, 32], 32, 4096), ([20, 5], 32, 1 << 20), ([9, 12], 64, 64)])
def test_the_copy_starts_no_block_past_a_table(lens, fits, wide):
    """The launches of a call, captured and looked at but not run: a CTA per block of the new tables, and no
    more of them than either table is wide."""
    import ctypes as C
    cuda = C.CDLL("libcuda.so.1")

    class Node(C.Structure):                                 # a kernel node's parameters
        _fields_ = [("func", C.c_void_p), ("grid", C.c_uint * 3), ("block", C.c_uint * 3), ("shared", C.c_uint),
                    ("params", C.c_void_p), ("extra", C.c_void_p), ("kern", C.c_void_p), ("ctx", C.c_void_p)]

    state, table, fresh, given = narrow(lens, 16, 2, 64, fits, wide, 9)
    dev, tab, ln = [x.cuda() for x in state], table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    new, kept = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(2, wide, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    handle, graph = C.c_void_p(side.cuda_stream), C.c_void_p()
    assert cuda.cuStreamBeginCapture_v2(handle, 2) == 0
    pkv.kv8_evict(*dev, tab, ln, given, wide, new_seq_lens=new, kept=kept, stream=side)
    assert cuda.cuStreamEndCapture(handle, C.byref(graph)) == 0
    count = C.c_size_t(8)
    nodes = (C.c_void_p * 8)()
    assert cuda.cuGraphGetNodes(graph, nodes, C.byref(count)) == 0
    grids = []
    for k in range(count.value):
        node = Node()
        assert cuda.cuGraphKernelNodeGetParams_v2(C.c_void_p(nodes[k]), C.byref(node)) == 0
        grids.append(tuple(node.grid))
    cuda.cuGraphDestroy(graph)
    copies = [g for g in grids if g[1] == len(lens)]
    assert len(copies) == 1 and copies[0][0] <= min(fresh.shape[1], table.shape[1], -(-wide // 16)), grids


@pytest.mark.parametrize("shape", ["heavy", "ties"])
def test_more_candidates_than_are_held(shape):
    """A request whose keys do not fit a cluster's shared memory, beside one whose keys do."""
    check([140001, 20000], 32, 1, 64, 2001, 4, 64, seed=10, shape=shape)
