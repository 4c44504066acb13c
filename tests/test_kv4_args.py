"""The appending rotation, the operators on the 4-bit paged cache and the
verification of drafts refuse bad arguments before any CUDA call, and the plain
test implementations agree with torch's e4m3 type."""
import ctypes as C

import pytest
import torch

import paged_kv_prep_gb300 as pkv
from paged_kv_prep_gb300 import _lib
from paged_kv_prep_gb300 import build as pbuild
from paged_kv_prep_gb300._lib import Kv4CacheArgs, RopeArgs
from tests import kv4_reference as ref

P = 4096
INVALID, ALIGN, OK = pkv.ERR_INVALID_ARG, pkv.ERR_ALIGN, pkv.OK


@pytest.fixture(scope="module", autouse=True)
def L():
    pbuild.build()
    return pkv.lib()


def cache(**kw):
    a = dict(k_cache=P, v_cache=P, k_scale=P, v_scale=P, num_blocks=10, block_size=16, num_heads=2, head_dim=128,
             k_unit=1.0, v_unit=1.0)
    a.update(kw)
    return Kv4CacheArgs(**a)


def rope(**kw):
    a = dict(table=P, positions=P, pair_axes=None, axis_stride=0, max_position=100, rot_dim=64, num_axes=1, interleaved=0)
    a.update(kw)
    return RopeArgs(**a)


def store(L, c=None, r=None, k=P, v=P, ks=512, vs=512, dtype=0, q=P, qs=2048, hq=8, qo=P, qos=2048, slots=P, T=4):
    return L.pkv_kv4_store(C.byref(c or cache()), C.byref(r or rope()), k, v, ks, vs, dtype, q, qs, hq, qo, qos, slots, T,
                           None, None)


def rope_store(L, r=None, k=P, v=P, ks=512, vs=512, heads=2, d=128, dtype=0, q=P, qs=2048, hq=8, qo=P, qos=2048, kc=P,
               vc=P, num_slots=64, slots=P, T=4):
    return L.pkv_rope_store(C.byref(r or rope()), k, v, ks, vs, heads, d, dtype, q, qs, hq, qo, qos, kc, vc, num_slots,
                            slots, T, None, None)


def load(L, c=None, slots=P, count=4, dtype=0, k=P, v=P):
    return L.pkv_kv4_load(C.byref(c or cache()), slots, count, dtype, k, v, None, None)


def attention(L, c=None, q=P, qs=2048, dtype=0, hq=8, tables=P, W=4, qsl=P, lens=P, n=2, T=4, window=0, out=P, os=2048,
              lse=P, ws=P, wsb=1 << 40):
    return L.pkv_kv4_attention(C.byref(c or cache()), q, qs, dtype, hq, tables, W, qsl, lens, n, T, 1.0, window, out, os,
                               lse, ws, wsb, None, None)


def verify(L, p=P, ps=1000, q=P, qs=1000, dtype=2, vocab=1000, rows=6, ids=P, qsl=P, n=2, u=P, most=3, tokens=P, acc=P):
    return L.pkv_verify_drafts(p, ps, q, qs, dtype, vocab, rows, ids, qsl, n, u, most, tokens, acc, None, None)


BAD_CACHE = [(dict(head_dim=96), INVALID), (dict(num_heads=0), INVALID), (dict(num_heads=1025), INVALID),
             (dict(block_size=0), INVALID), (dict(block_size=24), INVALID), (dict(num_blocks=-1), INVALID),
             (dict(num_blocks=1 << 31), INVALID), (dict(num_blocks=1 << 28, block_size=16), INVALID),
             (dict(k_cache=None), INVALID), (dict(v_scale=None), INVALID), (dict(v_cache=P + 8), ALIGN),
             (dict(k_scale=P + 4), ALIGN), (dict(k_unit=0.0), INVALID), (dict(v_unit=-1.0), INVALID),
             (dict(k_unit=float("nan")), INVALID), (dict(v_unit=float("inf")), INVALID), (dict(k_unit=1e30), INVALID)]


@pytest.mark.parametrize("kw,code", BAD_CACHE)
@pytest.mark.parametrize("call", [store, load, attention])
def test_bad_cache(L, call, kw, code):
    assert call(L, cache(**kw)) == code


BAD_ROPE = [(dict(table=None), INVALID), (dict(positions=None), INVALID), (dict(rot_dim=0), INVALID),
            (dict(rot_dim=24), INVALID), (dict(rot_dim=144), INVALID), (dict(rot_dim=-16), INVALID),
            (dict(num_axes=0), INVALID), (dict(num_axes=9, axis_stride=4), INVALID), (dict(max_position=0), INVALID),
            (dict(num_axes=3, axis_stride=3), INVALID), (dict(pair_axes=bytes([0] * 31 + [1])), INVALID),
            (dict(num_axes=3, axis_stride=4, pair_axes=bytes([0] * 16 + [3] + [1] * 15)), INVALID),
            (dict(table=P + 8), ALIGN), (dict(positions=P + 2), ALIGN)]


@pytest.mark.parametrize("kw,code", BAD_ROPE)
@pytest.mark.parametrize("call", [store, rope_store])
def test_bad_rotation(L, call, kw, code):
    assert call(L, r=rope(**kw)) == code


@pytest.mark.parametrize("call", [store, rope_store])
@pytest.mark.parametrize("kw,code", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(slots=None), INVALID), (dict(dtype=2), INVALID),
    (dict(T=-1), INVALID), (dict(T=1 << 26), INVALID), (dict(ks=496), INVALID), (dict(vs=520), ALIGN),
    (dict(k=P + 2), ALIGN), (dict(ks=-512), INVALID), (dict(q=None), INVALID), (dict(qo=None), INVALID),
    (dict(hq=-1), INVALID), (dict(qs=2032), INVALID), (dict(qos=2056), ALIGN), (dict(qo=P + 8), ALIGN),
    (dict(slots=P + 4), ALIGN), (dict(T=0), OK), (dict(T=0, k=None, q=None, slots=None), OK)])
def test_append_refusals(L, call, kw, code):
    assert call(L, **kw) == code


def test_store_without_rotation_takes_no_queries(L):
    c = cache()
    assert L.pkv_kv4_store(C.byref(c), None, P, P, 512, 512, 0, P, 2048, 8, P, 2048, P, 4, None, None) == INVALID
    assert L.pkv_kv4_store(C.byref(c), None, P, P, 512, 512, 0, None, 0, 0, None, 0, P, 0, None, None) == OK
    assert L.pkv_rope_store(None, P, P, 512, 512, 2, 128, 0, None, 0, 0, None, 0, P, P, 64, P, 4, None, None) == INVALID


@pytest.mark.parametrize("kw,code", [(dict(kc=None), INVALID), (dict(vc=P + 8), ALIGN), (dict(num_slots=-1), INVALID),
                                     (dict(num_slots=1 << 32), INVALID), (dict(heads=0), INVALID), (dict(d=96), INVALID),
                                     (dict(heads=1025, ks=1 << 20, vs=1 << 20), INVALID)])
def test_rope_store_refusals(L, kw, code):
    assert rope_store(L, **kw) == code


@pytest.mark.parametrize("kw,code", [(dict(slots=None), INVALID), (dict(count=-1), INVALID), (dict(dtype=2), INVALID),
                                     (dict(k=P + 8), ALIGN), (dict(slots=P + 4), ALIGN), (dict(count=0), OK),
                                     (dict(k=None, v=None), OK)])
def test_load_refusals(L, kw, code):
    assert load(L, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(qsl=None), INVALID), (dict(lens=None), INVALID),
    (dict(tables=None), INVALID), (dict(ws=None), INVALID), (dict(hq=7), INVALID), (dict(hq=0), INVALID),
    (dict(dtype=-1), INVALID), (dict(n=-1), INVALID), (dict(n=16385), INVALID), (dict(T=-1), INVALID),
    (dict(window=-1), INVALID), (dict(W=-1), INVALID), (dict(qs=1024), INVALID), (dict(os=1024), INVALID),
    (dict(q=P + 8), ALIGN), (dict(out=P + 8), ALIGN), (dict(qs=2056), ALIGN), (dict(ws=P + 8), ALIGN), (dict(n=0), OK),
    (dict(T=0), OK)])
def test_attention_refusals(L, kw, code):
    assert attention(L, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(p=None), INVALID), (dict(ids=None), INVALID), (dict(qsl=None), INVALID), (dict(u=None), INVALID),
    (dict(tokens=None), INVALID), (dict(acc=None), INVALID), (dict(dtype=3), INVALID), (dict(vocab=0), INVALID),
    (dict(vocab=(1 << 22) + 1, ps=1 << 23, qs=1 << 23), INVALID),
    (dict(rows=-1), INVALID), (dict(n=-1), INVALID), (dict(n=16385), INVALID), (dict(most=-1), INVALID),
    (dict(ps=999), INVALID), (dict(qs=999), INVALID), (dict(ps=-1), INVALID), (dict(p=P + 2), ALIGN), (dict(q=P + 2), ALIGN),
    (dict(ids=P + 2), ALIGN), (dict(u=P + 1), ALIGN), (dict(n=0), OK), (dict(n=0, qsl=None), OK)])
def test_verify_refusals(L, kw, code):
    assert verify(L, **kw) == code


def operands():
    bs, blocks, heads, d = 16, 4, 2, 128
    o = {"codes": torch.zeros(blocks, heads, bs, d // 2, dtype=torch.uint8),
         "scales": torch.zeros(blocks, heads, bs, d // 16, dtype=torch.uint8),
         "lines": torch.zeros(bs * blocks, heads, d, dtype=torch.bfloat16),
         "k": torch.zeros(3, heads, d, dtype=torch.bfloat16), "q": torch.zeros(3, 8, d, dtype=torch.bfloat16),
         "slots": torch.zeros(3, dtype=torch.int64), "pos": torch.zeros(3, dtype=torch.int32),
         "table": torch.zeros(50, 64), "tab": torch.zeros(1, 4, dtype=torch.int32),
         "qsl": torch.zeros(2, dtype=torch.int32), "lens": torch.ones(1, dtype=torch.int32),
         "p": torch.zeros(3, 100), "ids": torch.zeros(3, dtype=torch.int32), "u": torch.zeros(3)}
    return o


def calls():
    """The calls on operands that fit together but for their place."""
    o = operands()
    c = (o["codes"], o["codes"], o["scales"], o["scales"])

    def call(f, a, kw, more):
        return f(*a, **{**kw, **more})
    return [lambda **m: call(pkv.rope_store, (o["k"], o["k"], o["lines"], o["lines"], o["slots"], o["pos"], o["table"]), dict(q=o["q"]), m),
            lambda **m: call(pkv.kv4_store, (o["k"], o["k"], *c, o["slots"], o["pos"], o["table"]), dict(q=o["q"]), m),
            lambda **m: call(pkv.kv4_load, (*c, o["slots"]), {}, m),
            lambda **m: call(pkv.kv4_attention, (o["q"], *c, o["tab"], o["qsl"], o["lens"]), {}, m),
            lambda **m: call(pkv.verify_drafts, (o["p"], o["ids"], o["qsl"], o["u"], 2), {}, m)]


@pytest.mark.parametrize("which", range(5))
@pytest.mark.parametrize("stream", [None, 0])
def test_operands_are_on_a_cuda_device(which, stream, monkeypatch):
    """Host operands never reach the library."""
    reached = []
    monkeypatch.setattr(_lib, "lib", lambda: reached.append(1))
    with pytest.raises(ValueError, match="CUDA device"):
        calls()[which](stream=stream)
    assert not reached


def fake_devices(monkeypatch):
    """Two devices of which 0 is current; a library that notes under which it was called."""
    state = {"now": 0, "seen": []}

    class Switch:
        def __init__(self, device):
            self.to = device

        def __enter__(self):
            self.back, state["now"] = state["now"], self.to

        def __exit__(self, *a):
            state["now"] = self.back

    class Library:
        def __getattr__(self, name):
            def call(*a):
                state["seen"].append((name, state["now"]))
                return pkv.OK
            return call
    monkeypatch.setattr(_lib, "_KV8", _lib._kv8_types()[:6] + (lambda: state["now"],))
    monkeypatch.setattr(torch.cuda, "device", Switch)
    monkeypatch.setattr(_lib, "lib", Library)
    monkeypatch.setattr(_lib, "_KV4_WORKSPACE", {})
    monkeypatch.setattr(_lib, "_kv8_stream", lambda stream, device: 10 + device)
    return state


@pytest.mark.parametrize("which", range(5))
def test_the_operands_device_is_current_in_the_call(which, monkeypatch):
    state = fake_devices(monkeypatch)
    monkeypatch.setattr(_lib, "_kv8_device", lambda *a: 1)
    calls()[which]()
    assert state["seen"] and all(d == 1 for _, d in state["seen"]) and state["now"] == 0


def test_binding_refusals(monkeypatch):
    """The binding checks shapes and types before it calls the library."""
    state = fake_devices(monkeypatch)
    monkeypatch.setattr(_lib, "_kv8_device", lambda *a: 0)
    o = operands()
    k, q, lines, slots, pos, table = (o[n] for n in ("k", "q", "lines", "slots", "pos", "table"))
    c = (o["codes"], o["codes"], o["scales"], o["scales"])
    rs = lambda k=k, v=None, kc=lines, vc=None, slots=slots, pos=pos, table=table, **kw: pkv.rope_store(  # noqa: E731
        k, k if v is None else v, kc, kc if vc is None else vc, slots, pos, table, **kw)
    st = lambda k=k, c=c, slots=slots, **kw: pkv.kv4_store(k, k, *c, slots, **kw)     # noqa: E731
    at = lambda q=q, c=c, tab=o["tab"], qsl=o["qsl"], lens=o["lens"], **kw: pkv.kv4_attention(q, *c, tab, qsl, lens, **kw)  # noqa: E731
    vd = lambda p=o["p"], ids=o["ids"], qsl=o["qsl"], u=o["u"], most=2, **kw: pkv.verify_drafts(p, ids, qsl, u, most, **kw)  # noqa: E731
    bad = [
        lambda: rs(k=k.float()), lambda: rs(v=k.half()), lambda: rs(kc=lines.half()), lambda: rs(kc=lines[:, :1]),
        lambda: rs(kc=lines[::2]), lambda: rs(slots=slots.int()), lambda: rs(pos=pos.long()), lambda: rs(pos=pos[:2]),
        lambda: rs(table=table.double()), lambda: rs(table=table[:, ::2]), lambda: rs(table=table[0]),
        lambda: rs(axes=[0] * 31), lambda: rs(axes=[300] + [0] * 31), lambda: rs(axes=[-1] + [0] * 31),
        lambda: rs(q=q.half()), lambda: rs(q=q[:2]), lambda: rs(q=q[:, :, :64]), lambda: rs(q=q, q_out=q[:, :4]),
        lambda: rs(q_out=q), lambda: rs(pos=torch.zeros(3, 3, dtype=torch.int32).T.contiguous().T),
        lambda: rs(k=k[:2]), lambda: rs(k=k.transpose(1, 2).contiguous().transpose(1, 2)),
        lambda: st(c=(o["codes"], o["codes"][:3], o["scales"], o["scales"])), lambda: st(c=(o["codes"],) * 4),
        lambda: st(c=(o["codes"], o["codes"], o["scales"].float(), o["scales"])),
        lambda: st(c=tuple(x[:, :, ::2] for x in c)), lambda: st(q=q), lambda: st(axes=[0] * 32), lambda: st(positions=pos),
        lambda: st(table=table), lambda: st(k=k[:, :1]), lambda: st(k=k.float()),
        lambda: pkv.kv4_load(*c, slots.int()), lambda: pkv.kv4_load(*c, slots, dtype=torch.float32),
        lambda: pkv.kv4_load(*c, slots, k=k.half(), dtype=torch.bfloat16), lambda: pkv.kv4_load(*c, slots, v=k[:2]),
        lambda: at(q=q.float()), lambda: at(q=q[:, :, :64]), lambda: at(tab=o["tab"].long()), lambda: at(qsl=o["qsl"][:1]),
        lambda: at(out=q[:2]), lambda: at(lse=torch.zeros(3, 7)), lambda: at(window=1 << 31), lambda: at(window=(1 << 32) + 5),
        lambda: at(workspace=torch.zeros(8192, dtype=torch.uint8)[::2]),
        lambda: vd(p=o["p"].double()), lambda: vd(p=o["p"][0]), lambda: vd(p=o["p"][:, ::2]), lambda: vd(ids=o["ids"].long()),
        lambda: vd(ids=o["ids"][:1]), lambda: vd(u=o["u"][:2]), lambda: vd(u=o["u"].double()), lambda: vd(most=-1),
        lambda: vd(most=1 << 31), lambda: vd(draft_probs=o["p"].half()), lambda: vd(draft_probs=o["p"][:2]),
        lambda: vd(tokens=torch.zeros(1, 2, dtype=torch.int32)), lambda: vd(accepted=torch.zeros(2, dtype=torch.int32)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(f"call {i} was not refused")
    assert not state["seen"]
    for call in calls():
        call()
    assert len(state["seen"]) == 6                      # the attention asks for its workspace's size too


def test_an_error_is_raised_or_returned(monkeypatch):
    fake_devices(monkeypatch)
    monkeypatch.setattr(_lib, "_kv8_device", lambda *a: 0)

    class Library:
        def __getattr__(self, name):
            return lambda *a: pkv.OK if name.endswith("workspace") else pkv.ERR_ALIGN
    monkeypatch.setattr(_lib, "lib", Library)
    for call in calls():
        with pytest.raises(pkv.PkvError):
            call()
        assert call(check=False) == pkv.ERR_ALIGN


def test_workspace_refusals():
    with pytest.raises(pkv.PkvError) as e:
        pkv.kv4_attention_workspace(96)
    assert e.value.code == pkv.ERR_INVALID_ARG


def test_reference_rounding():
    g = torch.Generator().manual_seed(3)
    x = (torch.randn(20000, generator=g) * torch.exp2(torch.randint(-14, 9, (20000,), generator=g).float())).abs()
    x = torch.cat([x, torch.tensor([0.0, 448.0, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -9, 17.0, 19.0, 1e9])])
    assert torch.equal(ref.scale_code(x.double()), x.clamp(max=448).to(torch.float8_e4m3fn).view(torch.uint8))
    at = torch.tensor([0.0, 0.25, 0.26, 0.75, 1.25, 1.3, 1.75, 2.5, 3.5, 5.0, 5.1, 6.0, 9.0]).double()
    assert ref.element_code(at).tolist() == [0, 0, 1, 2, 2, 3, 4, 4, 6, 6, 7, 7, 7]
    assert ref.element_code(-at).tolist()[1:] == [8, 9, 10, 10, 11, 12, 12, 14, 14, 15, 15, 15]
    codes = torch.randint(0, 256, (5, 8), generator=g, dtype=torch.uint8)
    back = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    assert torch.equal(ref.pack(back), codes)
    y = torch.randn(50, 32, generator=g).double()
    c, s, nan = ref.quantise(y, 0.5)
    got = ref.values(ref.pack(c), s, 0.5)
    step = y.unflatten(-1, (-1, 16)).abs().amax(-1) / 6
    # half a step of the coarse end of the grid (1), and what a scale rounded down by 2^-4 cuts off (6 / 16)
    assert ((got - y).unflatten(-1, (-1, 16)).abs().amax(-1) <= step * 1.0625 + 1e-12).all() and not nan.any()


def test_reference_rotation_keeps_lengths():
    g = torch.Generator().manual_seed(5)
    ang = torch.rand(20, 16, generator=g) * 6.28
    table = torch.cat([ang.cos(), ang.sin()], 1)
    x = torch.randn(7, 3, 64, generator=g)
    pos = torch.randint(0, 20, (3, 7), generator=g)
    for inter in (False, True):
        y = ref.rotate32(x, pos, table, [i % 3 for i in range(16)], inter)
        assert torch.allclose(y.norm(dim=-1), x.norm(dim=-1), rtol=1e-5) and torch.equal(y[..., 32:], x[..., 32:])
