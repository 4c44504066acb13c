"""The operators on the 8-bit paged cache refuse bad arguments before any CUDA
call, and their plain test implementation agrees with torch's e4m3 type."""
import ctypes as C

import pytest
import torch

import paged_kv_prep_gb300 as pkv
from paged_kv_prep_gb300 import _lib
from paged_kv_prep_gb300 import build as pbuild
from paged_kv_prep_gb300._lib import Kv8CacheArgs
from tests import kv8_reference as ref

P = 4096


@pytest.fixture(scope="module", autouse=True)
def L():
    pbuild.build()
    return pkv.lib()


def cache(**kw):
    a = dict(k_cache=P, v_cache=P, k_scale=P, v_scale=P, num_blocks=10, block_size=16, num_heads=2, head_dim=128)
    a.update(kw)
    return Kv8CacheArgs(**a)


BAD_CACHE = [(dict(head_dim=96), pkv.ERR_INVALID_ARG), (dict(num_heads=0), pkv.ERR_INVALID_ARG),
             (dict(num_heads=1025), pkv.ERR_INVALID_ARG), (dict(block_size=0), pkv.ERR_INVALID_ARG),
             (dict(num_blocks=-1), pkv.ERR_INVALID_ARG), (dict(num_blocks=1 << 31), pkv.ERR_INVALID_ARG),
             (dict(k_cache=None), pkv.ERR_INVALID_ARG), (dict(v_scale=None), pkv.ERR_INVALID_ARG),
             (dict(v_cache=P + 8), pkv.ERR_ALIGN), (dict(k_scale=P + 2), pkv.ERR_ALIGN)]


def store(L, c=None, k=P, v=P, ks=512, vs=512, dtype=0, slots=P, T=4):
    return L.pkv_kv8_store(C.byref(c or cache()), k, v, ks, vs, dtype, slots, T, None, None)


def attention(L, c=None, q=P, qs=2048, dtype=0, hq=8, tables=P, W=4, qsl=P, lens=P, n=2, T=4, window=0,
              out=P, os=2048, lse=P, weights=None, ws=P, wsb=1 << 40):
    return L.pkv_kv8_attention(C.byref(c or cache()), q, qs, dtype, hq, tables, W, qsl, lens, n, T, 1.0, window,
                               out, os, lse, weights, ws, wsb, None, None)


def evict(L, c=None, weights=P, tables=P, W=4, lens=P, n=2, fresh=P, W2=4, budget=64, first=4, last=8,
          new=P, kept=P):
    return L.pkv_kv8_evict(C.byref(c or cache()), weights, tables, W, lens, n, fresh, W2, budget, first, last,
                           new, kept, None, None)


@pytest.mark.parametrize("kw,code", BAD_CACHE)
@pytest.mark.parametrize("call", [store, attention, evict])
def test_bad_cache(L, call, kw, code):
    assert call(L, cache(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), pkv.ERR_INVALID_ARG), (dict(slots=None), pkv.ERR_INVALID_ARG), (dict(dtype=2), pkv.ERR_INVALID_ARG),
    (dict(T=-1), pkv.ERR_INVALID_ARG), (dict(T=1 << 26), pkv.ERR_INVALID_ARG), (dict(ks=496), pkv.ERR_INVALID_ARG),
    (dict(vs=520), pkv.ERR_ALIGN), (dict(k=P + 2), pkv.ERR_ALIGN), (dict(ks=-512), pkv.ERR_INVALID_ARG),
    (dict(T=0), pkv.OK), (dict(T=0, k=None, slots=None), pkv.OK)])
def test_store_refusals(L, kw, code):
    assert store(L, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), pkv.ERR_INVALID_ARG), (dict(out=None), pkv.ERR_INVALID_ARG), (dict(qsl=None), pkv.ERR_INVALID_ARG),
    (dict(lens=None), pkv.ERR_INVALID_ARG), (dict(tables=None), pkv.ERR_INVALID_ARG), (dict(ws=None), pkv.ERR_INVALID_ARG),
    (dict(hq=7), pkv.ERR_INVALID_ARG), (dict(hq=0), pkv.ERR_INVALID_ARG), (dict(dtype=-1), pkv.ERR_INVALID_ARG),
    (dict(n=-1), pkv.ERR_INVALID_ARG), (dict(n=16385), pkv.ERR_INVALID_ARG), (dict(T=-1), pkv.ERR_INVALID_ARG),
    (dict(window=-1), pkv.ERR_INVALID_ARG), (dict(W=-1), pkv.ERR_INVALID_ARG), (dict(qs=1024), pkv.ERR_INVALID_ARG),
    (dict(os=1024), pkv.ERR_INVALID_ARG), (dict(q=P + 8), pkv.ERR_ALIGN), (dict(out=P + 8), pkv.ERR_ALIGN),
    (dict(qs=2056), pkv.ERR_ALIGN), (dict(ws=P + 8), pkv.ERR_ALIGN), (dict(weights=P, lse=None), pkv.ERR_INVALID_ARG),
    (dict(n=0), pkv.OK), (dict(T=0), pkv.OK)])
def test_attention_refusals(L, kw, code):
    assert attention(L, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(weights=None), pkv.ERR_INVALID_ARG), (dict(tables=None), pkv.ERR_INVALID_ARG), (dict(fresh=None), pkv.ERR_INVALID_ARG),
    (dict(lens=None), pkv.ERR_INVALID_ARG), (dict(new=None), pkv.ERR_INVALID_ARG), (dict(kept=None), pkv.ERR_INVALID_ARG),
    (dict(W=0), pkv.ERR_INVALID_ARG), (dict(W2=0), pkv.ERR_INVALID_ARG), (dict(budget=0), pkv.ERR_INVALID_ARG),
    (dict(first=-1), pkv.ERR_INVALID_ARG), (dict(last=-1), pkv.ERR_INVALID_ARG), (dict(first=60), pkv.ERR_INVALID_ARG),
    (dict(first=2 ** 31 - 1, last=2 ** 31 - 1), pkv.ERR_INVALID_ARG), (dict(n=16385), pkv.ERR_INVALID_ARG),
    (dict(n=0), pkv.OK)])
def test_evict_refusals(L, kw, code):
    assert evict(L, **kw) == code


def test_binding_refusals():
    """The binding checks shapes and types before it calls the library."""
    bs, blocks, heads, d = 16, 4, 2, 128
    kc = torch.zeros(bs * blocks, heads * d, dtype=torch.uint8)
    sc = torch.ones(blocks, heads)
    k = torch.zeros(3, heads, d, dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int64)
    tab, qsl, lens = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    w = torch.zeros(bs * blocks)
    q = torch.zeros(3, 8, d, dtype=torch.bfloat16)
    bad = [
        lambda: pkv.kv8_store(k.float(), k.float(), kc, kc, sc, sc, slots, stream=0),
        lambda: pkv.kv8_store(k, k.half(), kc, kc, sc, sc, slots, stream=0),
        lambda: pkv.kv8_store(k, k, kc, kc, sc, sc, slots.int(), stream=0),
        lambda: pkv.kv8_store(k[:2], k[:2], kc, kc, sc, sc, slots, stream=0),
        lambda: pkv.kv8_store(k[:, :1], k[:, :1], kc, kc, sc, sc, slots, stream=0),
        lambda: pkv.kv8_store(k.transpose(0, 1), k.transpose(0, 1), kc, kc, sc, sc, slots[:2], stream=0),
        lambda: pkv.kv8_store(k, k, kc[:61], kc[:61], sc, sc, slots, stream=0),
        lambda: pkv.kv8_store(k, k, kc.float(), kc, sc, sc, slots, stream=0),
        lambda: pkv.kv8_store(k, k, kc, kc, sc.double(), sc, slots, stream=0),
        lambda: pkv.kv8_attention(q.float(), kc, kc, sc, sc, tab, qsl, lens, stream=0),
        lambda: pkv.kv8_attention(q[:, :, :64], kc, kc, sc, sc, tab, qsl, lens, stream=0),
        lambda: pkv.kv8_attention(q, kc, kc, sc, sc, tab.long(), qsl, lens, stream=0),
        lambda: pkv.kv8_attention(q, kc, kc, sc, sc, tab, qsl[:1], lens, stream=0),
        lambda: pkv.kv8_attention(q, kc, kc, sc, sc, tab, qsl, lens, weights=w[:5], stream=0),
        lambda: pkv.kv8_attention(q, kc, kc, sc, sc, tab, qsl, lens, out=q[:2], stream=0),
        lambda: pkv.kv8_attention(q, kc, kc, sc, sc, tab, qsl, lens, lse=torch.zeros(3, 7), stream=0),
        lambda: pkv.kv8_evict(kc, kc, sc, sc, w.double(), tab, lens, tab, 8, stream=0),
        lambda: pkv.kv8_evict(kc, kc, sc, sc, w, tab, lens, tab.long(), 8, stream=0),
        lambda: pkv.kv8_evict(kc, kc, sc, sc, w, tab, lens, tab, 8, kept=torch.zeros(1, 7, dtype=torch.int32), stream=0),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()


def test_reference_rounding_is_e4m3():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(20000, generator=g) * torch.exp2(torch.randint(-14, 9, (20000,), generator=g).float())
    x = torch.cat([x, torch.tensor([0.0, -0.0, 448.0, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -9, 17.0, 19.0])])
    want = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(ref.encode(x.double()), want)
    assert ref.decode(ref.encode(torch.tensor([float("nan")]).double())).isnan().all()
    assert ref.block_scale(448.0) == 1.0 and ref.block_scale(448.5) == 2.0 and ref.block_scale(0.0) == 2.0 ** -64


def calls():
    """The three calls on operands that fit together but for their place."""
    bs, blocks, heads, d = 16, 4, 2, 128
    kc = torch.zeros(bs * blocks, heads * d, dtype=torch.uint8)
    sc = torch.ones(blocks, heads)
    k = torch.zeros(3, heads, d, dtype=torch.bfloat16)
    tab = torch.zeros(1, 4, dtype=torch.int32)
    qsl, lens = torch.zeros(2, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    q, w = torch.zeros(3, 8, d, dtype=torch.bfloat16), torch.zeros(bs * blocks)
    return [lambda **kw: pkv.kv8_store(k, k, kc, kc, sc, sc, torch.zeros(3, dtype=torch.int64), **kw),
            lambda **kw: pkv.kv8_attention(q, kc, kc, sc, sc, tab, qsl, lens, weights=w, **kw),
            lambda **kw: pkv.kv8_evict(kc, kc, sc, sc, w, tab, lens, tab, 8, **kw)]


@pytest.mark.parametrize("which", range(3))
@pytest.mark.parametrize("stream", [None, 0])
def test_operands_are_on_a_cuda_device(which, stream, monkeypatch):
    """Host operands never reach the library."""
    reached = []
    monkeypatch.setattr(_lib, "lib", lambda: reached.append(1))
    with pytest.raises(ValueError):
        calls()[which](stream=stream)
    assert not reached


def test_operands_and_stream_are_on_one_device():
    class On:
        def __init__(self, device):
            self.device_index = device

        def get_device(self):
            return self.device_index

    assert _lib._kv8_device(None, On(1), On(1), None, On(1)) == 1
    assert _lib._kv8_device(On(1), On(1)) == 1 and _lib._kv8_device(77, On(1)) == 1
    for bad in ((None, On(0), On(1)), (None, On(0), On(-1)), (None, On(-1), On(-1)), (On(0), On(1), On(1))):
        with pytest.raises(ValueError):
            _lib._kv8_device(*bad)


class FakeDevices:
    """Two devices of which `now` is the current one; a library that notes under which it was called."""

    def __init__(self, monkeypatch):
        self.now, self.seen = 0, []
        fake = self

        class Switch:
            def __init__(self, device):
                self.to = device

            def __enter__(self):
                self.back, fake.now = fake.now, self.to

            def __exit__(self, *a):
                fake.now = self.back

        class Library:
            def __getattr__(self, name):
                def call(*a):
                    fake.seen.append((name, fake.now))
                    if name == "pkv_kv8_attention_workspace":
                        a[-1]._obj.value = 1000 * (1 + fake.now)
                    return pkv.OK
                return call

        monkeypatch.setattr(_lib, "_KV8", _lib._kv8_types()[:6] + (lambda: fake.now,))
        monkeypatch.setattr(torch.cuda, "current_device", lambda: fake.now)
        monkeypatch.setattr(torch.cuda, "device", Switch)
        monkeypatch.setattr(_lib, "lib", Library)
        monkeypatch.setattr(_lib, "_KV8_WORKSPACE", {})


@pytest.mark.parametrize("which", range(3))
def test_the_operands_device_is_current_in_the_call(which, monkeypatch):
    fake = FakeDevices(monkeypatch)
    monkeypatch.setattr(_lib, "_kv8_device", lambda *a: 1)
    monkeypatch.setattr(_lib, "_kv8_stream", lambda stream, device: 10 + device)
    calls()[which]()
    assert fake.seen and all(device == 1 for _, device in fake.seen) and fake.now == 0


def test_workspace_sizes_go_by_the_device(monkeypatch):
    fake = FakeDevices(monkeypatch)
    for device, tokens, want in ((0, 4, 1000), (1, 4, 2000), (0, 9, 1000), (1, 9, 2000)):
        fake.now = device
        assert _lib._kv8_workspace(device, tokens, 8, 128, False) == want
    assert len(fake.seen) == 2
    assert _lib._kv8_workspace(0, 4, 8, 128, True) == 2000 and len(fake.seen) == 3    # asked each time


@pytest.mark.parametrize("args", [(-1, 8, 128), (4, 0, 128), (4, 8, 96)])
def test_workspace_refusals(args):
    """The library's own, also where there is no device."""
    with pytest.raises(pkv.PkvError) as e:
        pkv.kv8_attention_workspace(*args)
    assert e.value.code == pkv.ERR_INVALID_ARG


def test_a_workspace_with_gaps_is_refused(monkeypatch):
    """Its bytes are written one behind the other: what lies between the elements of a view is not its."""
    fake = FakeDevices(monkeypatch)
    monkeypatch.setattr(_lib, "_kv8_device", lambda *a: 0)
    calls()[1](workspace=torch.zeros(4096, dtype=torch.uint8), stream=0, lse=torch.zeros(3, 8), out=torch.zeros(3, 8, 128).bfloat16())
    assert [name for name, _ in fake.seen] == ["pkv_kv8_attention"]
    with pytest.raises(ValueError):
        calls()[1](workspace=torch.zeros(8192, dtype=torch.uint8)[::2], stream=0, lse=torch.zeros(3, 8),
                   out=torch.zeros(3, 8, 128).bfloat16())
    assert len(fake.seen) == 1


@pytest.mark.parametrize("which,kw", [(1, dict(window=2 ** 32 + 5)), (1, dict(window=-2 ** 32 + 5)), (2, dict(keep_first=2 ** 32 + 1)),
                                      (2, dict(keep_last=2 ** 33)), (1, dict(window=2 ** 31))])
def test_sizes_past_32_bits_are_refused(which, kw, monkeypatch):
    """Not taken by their low 32 bits."""
    fake = FakeDevices(monkeypatch)
    monkeypatch.setattr(_lib, "_kv8_device", lambda *a: 0)
    monkeypatch.setattr(_lib, "_kv8_stream", lambda stream, device: 0)
    calls()[which]()
    reached = len(fake.seen)
    assert reached > 0
    with pytest.raises(ValueError):
        calls()[which](**kw)
    assert len(fake.seen) == reached
