"""Where the binding allocates for a call on a stream of its own (``stream=``).

A tensor from the current stream's memory may be handed out again as soon as it is dropped, in that
stream's order only.  A call on another stream runs in its own order: its workspace, dropped when the
call returns, would be the next call's while the first still writes it.  Everything that a call allocates
therefore comes from the memory of the stream that it runs on; what it returns is also marked as used by
the current stream.  The first part needs no GPU: the library, the streams and the argument checks are
stand-ins, and every allocation is watched.
"""
import contextlib

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import mixers_ref as ref
import state_space_model_05_b200 as ssd
from state_space_model_05_b200 import binding

f32, bf, u8 = torch.float32, torch.bfloat16, torch.uint8


class FakeLibrary:
    """Accepts every call; asks for 4096 bytes of workspace."""

    def __getattr__(self, name):
        return lambda *a: 4096 if name.endswith("_bytes") else 0


class Allocations(TorchDispatchMode):
    def __init__(self, now):
        super().__init__()
        self.now, self.seen = now, []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if "empty" in func.__name__:
            self.seen.append((out.dtype, tuple(out.shape), self.now[-1]))
        return out


@pytest.fixture
def streams(monkeypatch):
    """Stand-ins: (the stack of current streams, (tensor, stream) pairs of record_stream calls)."""
    now, used = ["current"], []

    @contextlib.contextmanager
    def enter(stream):
        now.append(stream)
        yield
        now.pop()

    monkeypatch.setattr(binding, "_lib", FakeLibrary())
    monkeypatch.setattr(binding, "_check_args", lambda *a: None)
    monkeypatch.setattr(binding, "_check_mixer", lambda *a: None)
    monkeypatch.setattr(binding, "_stream", lambda s=None: 0)
    monkeypatch.setattr(torch.cuda, "stream", enter)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: now[-1])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: used.append((t, s)))
    binding._workspace_bytes.cache_clear()
    yield now, used
    binding._workspace_bytes.cache_clear()


def calls(device="cpu", dtype=bf, tokens=40):
    """name -> a call of every entry point that allocates, as a function of its keyword arguments."""
    t = lambda *s, dtype=dtype: torch.ones(s, dtype=dtype, device=device)  # noqa: E731
    cu = torch.tensor([0, tokens // 4, tokens], dtype=torch.int32, device=device)
    x, dt, A, B = t(tokens, 4, 64), t(tokens, 4, dtype=f32), -t(4, dtype=f32), t(tokens, 1, 128)
    q, k, ld = t(tokens, 8, 64), t(tokens, 2, 64), -t(8, dtype=f32)
    lens = torch.full((2,), 7, dtype=torch.int32, device=device)
    step = lambda y: y[None]  # noqa: E731
    return {
        "prefill": lambda **kw: ssd.ssd_prefill(step(x), step(dt), A, step(B), step(B), A, 128, **kw),
        "prefill_dtraw": lambda **kw: ssd.ssd_prefill(step(x), step(dt), A, step(B), step(B), A, 128, dt_softplus=True, **kw),
        "prefill_varlen": lambda **kw: ssd.ssd_prefill_varlen(x, dt, A, B, B, A, cu, 128, **kw),
        "decode_step": lambda **kw: ssd.ssd_decode_step(t(2, 4, 64, 128, dtype=f32), x[:2], dt[:2], A, B[:2], B[:2], A, **kw),
        "decode_steps": lambda **kw: ssd.ssd_decode_steps(t(2, 4, 64, 128, dtype=f32), step(x[:2]), step(dt[:2]), A,
                                                          step(B[:2]), step(B[:2]), A, **kw),
        "gdn_decode_step": lambda **kw: ssd.ssd_gdn_decode_step(t(2, 8, 64, 64, dtype=f32), k[:2], k[:2], q[:2],
                                                                t(2, 8, dtype=f32), t(2, 8, dtype=f32), **kw),
        "linattn_prefill": lambda **kw: ssd.ssd_linattn_prefill(k, k, q, ld, cu, **kw),
        "linattn_decode_step": lambda **kw: ssd.ssd_linattn_decode_step(t(2, 8, 64, 64, dtype=f32), k[:2], k[:2], q[:2], ld, **kw),
        "attn_prefill": lambda **kw: ssd.ssd_attn_prefill(q, k, k, cu, **kw),
        "attn_decode_step": lambda **kw: ssd.ssd_attn_decode_step(t(2, 64, 2, 64), t(2, 64, 2, 64), lens, q[:2], k[:2], k[:2], **kw),
    }


@pytest.mark.parametrize("name", calls())
def test_a_call_on_a_stream_allocates_there(streams, name):
    now, used = streams
    call = calls()[name]
    for stream, where in (("side", "side"), (None, "current")):
        used.clear()
        with Allocations(now) as made:
            result = call(stream=stream)
        assert made.seen and all(at == where for _, _, at in made.seen), made.seen
        results = result if isinstance(result, tuple) else (result,)
        if stream is None:
            assert not used
        else:                                      # what comes back may be used and dropped on the current stream
            assert all(any(u is r and s == "current" for u, s in used) for r in results)
            assert all(u.dtype != u8 for u, _ in used)


@pytest.mark.parametrize("name", calls())
def test_shapes_and_types_do_not_depend_on_the_stream(streams, name):
    now, _ = streams
    seen = []
    for stream in ("side", None):
        with Allocations(now) as made:
            calls()[name](stream=stream)
        seen.append([(dtype, shape) for dtype, shape, _ in made.seen])
    assert seen[0] == seen[1]


# ---------------------------------------------------------------- on the GPU
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("name", ["prefill", "prefill_varlen", "linattn_prefill", "attn_decode_step"])
def test_calls_on_two_streams_one_after_the_other(name, dtype):
    """Two calls in a row on streams of their own, without a workspace: each gives, bit for bit, what it
    gives alone."""
    from state_space_model_05_b200.build import build
    build()
    lens, hq, hv, dim = [1500, 0, 2600], 2, 8, 64
    n = sum(lens)
    cu, at = ref.cu(lens), torch.tensor([2999, 40, 2000, 1], dtype=torch.int32, device="cuda")
    r = lambda *s, seed, dtype=dtype: ref.randn(*s, seed=seed, dtype=dtype)  # noqa: E731

    def problem(i):
        if name == "linattn_prefill":
            q, k, v, s0 = r(n, hq, dim, seed=i), r(n, hq, dim, seed=i + 1), r(n, hv, dim, seed=i + 2), ref.randn(3, hv, dim, dim, seed=i + 3)
            ld = torch.full((hv,), -1e-3, device="cuda")
            return lambda **kw: ssd.ssd_linattn_prefill(q, k, v, ld, cu, scale=0.1, init_states=s0, **kw)
        if name == "attn_decode_step":
            kc, vc = r(4, 3000, hq, dim, seed=i), r(4, 3000, hq, dim, seed=i + 1)
            q, k, v = r(4, hv, dim, seed=i + 2), r(4, hq, dim, seed=i + 3), r(4, hq, dim, seed=i + 4)
            return lambda **kw: (ssd.ssd_attn_decode_step(kc, vc, at, q, k, v, **kw),)
        x, b, c = r(n, hv, 64, seed=i), r(n, 1, 128, seed=i + 1), r(n, 1, 128, seed=i + 2)
        dt, A = 0.1 + 0.1 * torch.rand(n, hv, generator=torch.Generator().manual_seed(i)).cuda(), -torch.ones(hv, device="cuda")
        if name == "prefill_varlen":
            return lambda **kw: ssd.ssd_prefill_varlen(x, dt, A, b, c, -A, cu, 128, **kw)
        return lambda **kw: ssd.ssd_prefill(x[None], dt[None], A, b[None], c[None], -A, 128, **kw)

    two = [problem(10 * i + 1) for i in range(2)]
    want = []
    for call in two:
        want.append([z.clone() for z in call()])
        torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in two]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [call(stream=s) for call, s in zip(two, sides)]
        for s in sides:
            torch.cuda.current_stream().wait_stream(s)
        assert all(torch.equal(x, y) for g, w in zip(got, want) for x, y in zip(g, w))
        del got                                    # dropped on the current stream, which has read it
        for s in sides:
            s.wait_stream(torch.cuda.current_stream())
    assert ssd.ssd_device_status() == 0
