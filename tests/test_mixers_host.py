"""Refusals of the packed mixers (linear attention with a decay per head, causal attention) that
need no GPU: the C entries return their codes before any launch, the binding raises before any
library call; and the numbering of packed blocks."""
import ctypes

import pytest
import torch

import mixers_ref as ref
import state_space_model_05_b200 as ssd
from state_space_model_05_b200 import binding
from state_space_model_05_b200.build import build

FAKE = 0x10000                                     # aligned, never dereferenced: the calls fail first
OK, NULL, SHAPE, DTYPE, ALIGN, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4, 5, 8
f32, bf = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    build()
    return binding.lib()


def linattn(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, qs=256, ks=256, vs=512, ld=FAKE, init=0, cu=FAKE, nseq=3, total=100, hq=2, hv=4,
             dk=128, dv=128, scale=1.0, dtype=1, out=FAKE, final=FAKE, ws=FAKE, nbytes=1 << 40)
    a.update(kw)
    return lib.ssd_linattn_prefill(*a.values(), None)


def linattn_step(lib, **kw):
    a = dict(state=FAKE, q=FAKE, k=FAKE, v=FAKE, ld=FAKE, batch=3, hq=2, hv=4, dk=128, dv=128, scale=1.0, dtype=1,
             out=FAKE)
    a.update(kw)
    return lib.ssd_linattn_decode_step(*a.values(), None)


def attn(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, qs=512, ks=256, vs=256, cu=FAKE, nseq=3, total=100, hq=4, hkv=2, dim=128, scale=1.0,
             dtype=1, out=FAKE)
    a.update(kw)
    return lib.ssd_attn_prefill(*a.values(), None)


def attn_step(lib, **kw):
    a = dict(kc=FAKE, vc=FAKE, lens=FAKE, q=FAKE, k=FAKE, v=FAKE, batch=3, capacity=100, hq=4, hkv=2, dim=128, scale=1.0,
             dtype=1, out=FAKE, ws=FAKE, nbytes=1 << 40)
    a.update(kw)
    return lib.ssd_attn_decode_step(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), DTYPE), (dict(total=-1), SHAPE), (dict(nseq=0), SHAPE), (dict(nseq=(1 << 20) + 1), SHAPE),
    (dict(total=(1 << 31) - 1023), SHAPE),
    (dict(hq=0), SHAPE), (dict(hv=0), SHAPE), (dict(hv=5), SHAPE), (dict(hv=65536), SHAPE), (dict(dk=12), SHAPE),
    (dict(dv=0), SHAPE), (dict(dk=136, qs=272, ks=272), UNSUPPORTED), (dict(dv=256, vs=1024), UNSUPPORTED),
    (dict(qs=248), SHAPE), (dict(ks=260), SHAPE), (dict(vs=504), SHAPE), (dict(vs=1 << 40), SHAPE), (dict(q=0), NULL),
    (dict(k=0), NULL), (dict(v=0), NULL), (dict(ld=0), NULL), (dict(cu=0), NULL), (dict(out=0), NULL),
    (dict(final=0), NULL), (dict(q=FAKE + 8), ALIGN), (dict(init=FAKE + 4), ALIGN), (dict(cu=FAKE + 2), ALIGN),
    (dict(final=FAKE + 8), ALIGN), (dict(ws=FAKE + 8), ALIGN), (dict(ws=0), WORKSPACE), (dict(nbytes=64), WORKSPACE)])
def test_linattn_prefill_refusals(lib, kw, code):
    assert linattn(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), DTYPE), (dict(batch=-1), SHAPE), (dict(hv=3), SHAPE), (dict(dk=4), SHAPE), (dict(dv=136), UNSUPPORTED),
    (dict(batch=1 << 30), SHAPE), (dict(state=0), NULL), (dict(ld=0), NULL), (dict(out=0), NULL), (dict(k=FAKE + 2), ALIGN),
    (dict(state=FAKE + 8), ALIGN), (dict(batch=0, state=0), OK)])
def test_linattn_step_refusals(lib, kw, code):
    assert linattn_step(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), DTYPE), (dict(total=-1), SHAPE), (dict(nseq=0), SHAPE), (dict(hkv=0), SHAPE), (dict(hq=5), SHAPE),
    (dict(total=(1 << 31) - 1023), SHAPE),
    (dict(dim=20), SHAPE), (dict(dim=136, qs=544, ks=272, vs=272), UNSUPPORTED), (dict(qs=504), SHAPE),
    (dict(ks=255), SHAPE), (dict(vs=8), SHAPE), (dict(q=0), NULL), (dict(cu=0), NULL), (dict(out=0), NULL),
    (dict(v=FAKE + 8), ALIGN), (dict(cu=FAKE + 1), ALIGN), (dict(total=0, q=0), OK)])
def test_attn_prefill_refusals(lib, kw, code):
    assert attn(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), DTYPE), (dict(batch=-1), SHAPE), (dict(capacity=0), SHAPE), (dict(hq=3), SHAPE), (dict(dim=4), SHAPE),
    (dict(dim=192), UNSUPPORTED), (dict(kc=0), NULL), (dict(lens=0), NULL), (dict(out=0), NULL), (dict(vc=FAKE + 8), ALIGN),
    (dict(lens=FAKE + 2), ALIGN), (dict(ws=0), WORKSPACE), (dict(nbytes=1), WORKSPACE), (dict(batch=0, q=0), OK)])
def test_attn_step_refusals(lib, kw, code):
    assert attn_step(lib, **kw) == code


def test_workspace_sizes(lib):
    """Zero for sizes that the call refuses, and never less for more tokens, sequences or rows."""
    lw, aw = lib.ssd_linattn_prefill_workspace_bytes, lib.ssd_attn_decode_workspace_bytes
    assert lw(3, 100, 2, 5, 128, 128, 1) == 0 and lw(0, 100, 2, 4, 128, 128, 1) == 0 and lw(3, 100, 2, 4, 128, 128, 9) == 0
    assert aw(3, 0, 4, 2, 128, 1) == 0 and aw(3, 100, 3, 2, 128, 1) == 0
    for dtype in (0, 1):
        assert 0 < lw(1, 100, 2, 4, 128, 128, dtype) < 1 << 30
        assert 0 < aw(1, 1, 4, 2, 128, dtype) <= aw(64, 1, 4, 2, 128, dtype) <= aw(64, 4096, 4, 2, 128, dtype) < 1 << 30


# ---------------------------------------------------------------- the binding
@pytest.fixture
def no_library(monkeypatch, tmp_path):
    monkeypatch.setattr(binding, "LIB_PATH", str(tmp_path / "missing.so"))
    monkeypatch.setattr(binding, "_lib", None)


def z(*shape, dtype=f32):
    return torch.empty(shape, dtype=dtype, device="meta")


def accepted(fn):
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        fn()


def test_binding_linattn_shapes(no_library):
    n, hq, hv, dk, dv = 20, 2, 4, 64, 128
    q, v, ld, cu = z(n, hq, dk, dtype=bf), z(n, hv, dv, dtype=bf), z(hv), torch.zeros(4, dtype=torch.int32)
    st = z(3, hv, dk, dv)
    call = lambda **kw: ssd.ssd_linattn_prefill(kw.get("q", q), kw.get("k", q), kw.get("v", v), kw.get("ld", ld),  # noqa: E731
                                                kw.get("cu", cu), init_states=kw.get("init"), out=kw.get("out"),
                                                final_states=kw.get("final"))
    accepted(lambda: call())
    accepted(lambda: call(init=st, final=st, out=v))
    for kw in (dict(k=z(n, hq, dk + 8, dtype=bf)), dict(v=z(n + 1, hv, dv, dtype=bf)), dict(ld=z(hv + 1)),
               dict(init=z(4, hv, dk, dv)), dict(final=z(3, hv, dv, dk)), dict(out=z(n, hv, dk, dtype=bf)),
               dict(q=z(n, hq * dk, dtype=bf)), dict(cu=cu.reshape(2, 2)), dict(cu=cu[:1])):
        with pytest.raises(ValueError, match="shape|offsets"):
            call(**kw)


def test_binding_steps_shapes(no_library):
    b, hq, hv, dk, dv = 3, 2, 4, 64, 128
    st, q, v, ld = z(b, hv, dk, dv), z(b, hq, dk), z(b, hv, dv), z(hv)
    call = lambda **kw: ssd.ssd_linattn_decode_step(kw.get("st", st), q, kw.get("k", q), v, kw.get("ld", ld))  # noqa: E731
    accepted(lambda: call())
    for kw in (dict(st=z(b, hv, dv, dk)), dict(k=z(b, hq, dk + 8)), dict(ld=z(b, hv))):
        with pytest.raises(ValueError, match="shape"):
            call(**kw)
    cache, new, lens = z(b, 50, 2, 64), z(b, 2, 64), z(b, dtype=torch.int32)
    q = z(b, 8, 64)
    call = lambda **kw: ssd.ssd_attn_decode_step(kw.get("kc", cache), kw.get("vc", cache), kw.get("lens", lens), q,  # noqa: E731
                                                 kw.get("k", new), new, out=kw.get("out"))
    accepted(lambda: call())
    for kw in (dict(vc=z(b, 51, 2, 64)), dict(kc=z(b, 50, 64)), dict(lens=z(b + 1, dtype=torch.int32)),
               dict(k=z(b, 2, 72)), dict(out=z(b, 2, 64))):
        with pytest.raises(ValueError, match="shape"):
            call(**kw)


def test_binding_attn_shapes(no_library):
    q, k, cu = z(20, 8, 64, dtype=bf), z(20, 2, 64, dtype=bf), torch.zeros(4, dtype=torch.int32)
    call = lambda **kw: ssd.ssd_attn_prefill(q, kw.get("k", k), kw.get("v", k), kw.get("cu", cu), out=kw.get("out"))  # noqa: E731
    accepted(lambda: call())
    for kw in (dict(k=z(19, 2, 64, dtype=bf)), dict(v=z(20, 2, 128, dtype=bf)), dict(out=k), dict(cu=cu[:1])):
        with pytest.raises(ValueError, match="shape|offsets"):
            call(**kw)


def test_token_strides():
    fused = torch.empty(10, 400)
    assert binding._packed(fused[:, 16:272].unflatten(1, (4, 64))) == 400
    assert binding._packed(torch.empty(1, 4, 64)) == 256 and binding._packed(torch.empty(0, 4, 64)) == 256
    assert binding._packed(fused[:1, 16:272].unflatten(1, (4, 64))) == 256        # one token: nothing lies apart
    for t in (torch.empty(10, 64, 4).transpose(1, 2), torch.empty(10, 8, 64)[:, ::2]):
        with pytest.raises(ValueError, match="contiguous"):
            binding._packed(t)


# ---------------------------------------------------------------- the numbering of packed blocks
@pytest.mark.parametrize("block", [32, 64, 128])
@pytest.mark.parametrize("lens", [[1], [0], [128], [0, 0, 0], [5, 0, 130, 1, 256, 0], [(7 * i) % 5 for i in range(300)],
                                  [(97 * i) % 400 for i in range(50)]])
def test_packed_blocks_cover_every_token_once(lens, block):
    """Block j of sequence s is number cu[s] // Q + s + j: the numbers are distinct, below
    total // Q + nseq, and the last s with cu[s] // Q + s <= i finds the sequence of number i."""
    cu = ref.offsets(lens)
    base = [cu[s] // block + s for s in range(len(lens))]
    numbers = {base[s] + j: (s, j) for s, n in enumerate(lens) for j in range(max(1, -(-n // block)))}
    assert len(numbers) == sum(max(1, -(-n // block)) for n in lens)
    assert max(numbers) < cu[-1] // block + len(lens)
    for i, (s, j) in numbers.items():
        found = max(x for x in range(len(lens)) if base[x] <= i)
        assert (found, i - base[found]) == (s, j)


def test_reference_forms_agree():
    """The blockwise reference of linear attention against its own token-by-token steps."""
    g = torch.Generator().manual_seed(0)
    n, hq, hv, dk, dv = 300, 1, 2, 8, 16
    q, k, v = (torch.randn(n, h, d, generator=g) for h, d in ((hq, dk), (hq, dk), (hv, dv)))
    ld = torch.tensor([-0.01, float("-inf")])
    init = torch.randn(1, hv, dk, dv, generator=g)
    out, final, _, _ = ref.linattn(q, k, v, ld, [n], 0.5, init)
    state = init.double()
    for t in range(n):
        o, state, _, _ = ref.linattn_step(state, q[t:t + 1], k[t:t + 1], v[t:t + 1], ld, 0.5)
        torch.testing.assert_close(o[0], out[t], rtol=1e-10, atol=1e-10)
    torch.testing.assert_close(state, final, rtol=1e-10, atol=1e-10)


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("capacity", [(1 << 31) - 1, (1 << 31) - 64, (1 << 31) - 65])
def test_workspace_of_the_largest_caches(lib, capacity, dtype):
    """A cache of any capacity needs no more pieces than CTAs fit the GPU at once."""
    aw = lib.ssd_attn_decode_workspace_bytes
    assert aw(1, capacity, 4, 2, 128, dtype) == aw(1, 1 << 20, 4, 2, 128, dtype)
    assert attn_step(lib, capacity=capacity, nbytes=aw(3, capacity, 4, 2, 128, dtype) - 1, dtype=dtype) == WORKSPACE
