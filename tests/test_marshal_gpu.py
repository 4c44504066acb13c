"""The binding's C++ calls and its Python ones make the same calls, and refuse the same."""
import sys

import pytest
import torch

import paged_kv_prep_gb300 as pkv
from paged_kv_prep_gb300 import _lib
from paged_kv_prep_gb300 import build as pbuild

NAMES = ["rope_store", "kv4_store", "kv4_load", "kv4_attention", "verify_drafts"]


@pytest.fixture(scope="module", autouse=True)
def built():
    pbuild.build()


def step(device):
    """A step's operands by name, and each function's arguments in its own order."""
    gen = torch.Generator().manual_seed(1)
    rand = lambda *shape: torch.randn(*shape, generator=gen).bfloat16().to(device)
    heads, group, d, bs, blocks, T = 2, 4, 128, 16, 12, 7
    rows = rand(T, (heads * group + 2 * heads) * d)
    q, k, v = (x.unflatten(1, (-1, d)) for x in rows.split([heads * group * d, heads * d, heads * d], 1))
    lines = [rand(blocks * bs, heads, d) for _ in range(2)]
    cache = [torch.zeros(blocks, heads, bs, d // n, dtype=torch.uint8).to(device) for n in (2, 2, 16, 16)]
    ints = lambda *x: torch.tensor(x, dtype=torch.int32).to(device)
    slots = torch.arange(3, 3 + T).to(device)
    positions, table = torch.stack([ints(*range(T)), ints(*range(5, 5 + T))]), torch.randn(64, d, generator=gen).to(device)
    axes = [i % 2 for i in range(d // 2)]
    probs = torch.rand(T, 501, generator=gen).to(device)
    turn = dict(positions=positions, table=table, axes=axes, interleaved=False, q=q, q_out=None)
    last = dict(d_error=None, stream=None, check=True)
    four = dict(zip(("k_cache", "v_cache", "k_scale", "v_scale"), cache))
    units = dict(k_unit=0.5, v_unit=2.0)
    return {
        "rope_store": dict(k=k, v=v, k_cache=lines[0], v_cache=lines[1], slot_mapping=slots, **turn, **last),
        "kv4_store": dict(k=k, v=v, **four, slot_mapping=slots, **turn, **units, **last),
        "kv4_load": dict(**four, slots=slots, dtype=torch.float16, k=None, v=None, **units, **last),
        "kv4_attention": dict(q=q, **four, block_tables=ints(*range(8)).view(2, 4), query_start_loc=ints(0, 1, 7),
                              seq_lens=ints(9, 10), softmax_scale=None, window=0, **units, out=None, lse=None,
                              workspace=None, **last),
        "verify_drafts": dict(target_probs=probs, draft_ids=ints(*range(T - 1)), query_start_loc=ints(0, 3, 7),
                              uniforms=torch.rand(T, generator=gen).to(device), max_drafts=3,
                              draft_probs=probs.flip(1).contiguous(), tokens=None, accepted=None, **last),
    }


def short(name, kw):
    return getattr(_lib._short(), name)(*kw.values())


def tensors(x):
    return [t for t in (x if isinstance(x, tuple) else (x,)) if t is not None]


@pytest.mark.parametrize("name", NAMES)
def test_what_is_not_on_the_gpu_is_left_to_the_checks(name):
    kw = step("cpu")[name]
    assert short(name, kw) is NotImplemented
    assert getattr(_lib._short(), name)() is NotImplemented
    assert getattr(_lib._short(), name)(*[None] * len(kw)) is NotImplemented
    assert getattr(_lib._short(), name)(*[object()] * (len(kw) - 2), None, True) is NotImplemented
    with pytest.raises(ValueError, match="CUDA"):
        getattr(pkv, name)(**kw)


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_both_ways_give_the_same(name):
    ways = []
    for stream in (None, "current"):
        all_ = step("cuda")
        kw = dict(all_[name])
        if name in ("kv4_load", "kv4_attention"):            # something to read
            pkv.kv4_store(**{**all_["kv4_store"], **{x: kw[x] for x in ("k_cache", "v_cache", "k_scale", "v_scale")}})
        if stream:
            kw["stream"] = torch.cuda.current_stream()
            assert short(name, kw) is NotImplemented
        else:
            assert short(name, kw) is not NotImplemented
        made = getattr(pkv, name)(**kw)
        torch.cuda.synchronize()
        ways.append([t.cpu() for t in tensors(made)] + [t.cpu() for x, t in kw.items() if "cache" in x or "scale" in x and torch.is_tensor(t)])
    assert len(ways[0]) == len(ways[1]) and len(ways[0]) > 0
    for a, b in zip(*ways):
        assert a.dtype == b.dtype and a.shape == b.shape and torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_given_outputs_and_error_words(name):
    kw = step("cuda")[name]
    want = tensors(getattr(pkv, name)(**kw))
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = {"rope_store": ["q_out"], "kv4_store": ["q_out"], "kv4_load": ["k", "v"], "kv4_attention": ["out", "lse"],
            "verify_drafts": ["tokens", "accepted"]}[name]
    given = {x: torch.empty_like(t) for x, t in zip(outs, want)}
    if name == "kv4_attention":
        given["workspace"] = torch.empty(pkv.kv4_attention_workspace(128), dtype=torch.uint8, device="cuda")
    got = tensors(getattr(pkv, name)(**{**kw, **given, "d_error": word.data_ptr()}))
    for x, t, w in zip(outs, got, want):
        assert t.data_ptr() == given[x].data_ptr() and torch.equal(t, w)
    assert word.item() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("name,change", [
    ("rope_store", dict(slot_mapping=torch.zeros(8, dtype=torch.int64))), ("rope_store", dict(table=torch.zeros(64, 128, dtype=torch.float64))),
    ("rope_store", dict(axes=[0] * 63)), ("rope_store", dict(axes=[256] + [0] * 63)), ("rope_store", dict(q_out=torch.zeros(3))),
    ("kv4_store", dict(positions=None)), ("kv4_store", dict(k=torch.zeros(7, 2, 128))), ("kv4_store", dict(k_unit="x")),
    ("kv4_load", dict(dtype=torch.float32)), ("kv4_load", dict(slots=torch.zeros(3, dtype=torch.int32))),
    ("kv4_attention", dict(block_tables=torch.zeros(1, 4, dtype=torch.int32))), ("kv4_attention", dict(window=2 ** 31)),
    ("kv4_attention", dict(lse=torch.zeros(7, 7))), ("kv4_attention", dict(seq_lens=torch.zeros(2, dtype=torch.int64))),
    ("verify_drafts", dict(draft_ids=torch.zeros(5, dtype=torch.int32))), ("verify_drafts", dict(max_drafts=-1)),
    ("verify_drafts", dict(draft_probs=torch.zeros(7, 500))), ("verify_drafts", dict(tokens=torch.zeros(2, 3, dtype=torch.int32)))])
def test_refusals_are_the_checks(name, change):
    kw = {**step("cuda")[name], **{x: t.cuda() if torch.is_tensor(t) else t for x, t in change.items()}}
    assert short(name, kw) is NotImplemented
    with pytest.raises((ValueError, TypeError)):
        getattr(pkv, name)(**kw)


@pytest.mark.gpu
def test_the_librarys_refusals_are_raised_or_returned():
    kw = step("cuda")["kv4_attention"]
    kw["workspace"] = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(pkv.PkvError):
        pkv.kv4_attention(**kw)
    assert pkv.kv4_attention(**{**kw, "check": False}) == pkv.ERR_INVALID_ARG
    kw = step("cuda")["kv4_store"]
    with pytest.raises(pkv.PkvError):
        pkv.kv4_store(**{**kw, "k_unit": 0.0})
    with pytest.raises(pkv.PkvError):
        pkv.kv4_store(**{**kw, "axes": [7] * 64})            # no such axis


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_nothing_is_kept(name):
    kw = step("cuda")[name]
    getattr(pkv, name)(**kw)
    torch.cuda.synchronize()
    memory, held = torch.cuda.memory_allocated(), {x: sys.getrefcount(t) for x, t in kw.items() if torch.is_tensor(t)}
    for _ in range(50):
        getattr(pkv, name)(**kw)
        getattr(pkv, name)(**{**kw, "check": 1})             # the other way
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() == memory
    assert held == {x: sys.getrefcount(t) for x, t in kw.items() if torch.is_tensor(t)}
