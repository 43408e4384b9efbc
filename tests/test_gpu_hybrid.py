"""The mixers together, as a hybrid model runs them: a stack of a state-space, a linear-attention and
an attention layer takes packed prompts, keeps its states and caches, and goes on one token at a time,
step by step and as captured graphs that share a workspace.  Every call's outputs are checked against
fp64 on the inputs that the stack gave it, which follow from the layers before it."""
import pytest
import torch

import mixers_ref as ref
import state_space_model_05_b200 as ssd

pytestmark = pytest.mark.gpu

bf, f32 = torch.bfloat16, torch.float32
WIDTH, CAPACITY = 128, 320
HQ, HKV, DIM = 8, 2, 64                            # attention
LQ, LV, DK, DV = 2, 4, 64, 64                      # linear attention
SH, SP, SN = 4, 64, 128                            # state space


@pytest.fixture(autouse=True, scope="module")
def _built():
    from state_space_model_05_b200.build import build
    build()


class Stack:
    """Two layers of each kind; `seen` keeps what the new calls were given and gave."""

    def __init__(self, dtype, batch):
        w = lambda rows, cols, seed: (ref.randn(rows, cols, seed=seed) * rows ** -0.5).to(dtype)  # noqa: E731
        self.dtype, self.layers, self.seen = dtype, [], None
        for i, kind in enumerate(["ssd", "lin", "attn"] * 2):
            cols = {"ssd": SH * SP + 2 * SN, "lin": 2 * LQ * DK + LV * DV, "attn": (HQ + 2 * HKV) * DIM}[kind]
            back = {"ssd": SH * SP, "lin": LV * DV, "attn": HQ * DIM}[kind]
            layer = dict(kind=kind, win=w(WIDTH, cols, 10 * i), wout=w(back, WIDTH, 10 * i + 1))
            if kind == "ssd":
                layer.update(A=-torch.rand(SH, device="cuda") - 0.1, D=torch.ones(SH, device="cuda"),
                             state=torch.zeros(batch, SH, SP, SN, device="cuda"))
            elif kind == "lin":
                layer.update(ld=-0.02 * torch.arange(LV, device="cuda"), state=torch.zeros(batch, LV, DK, DV, device="cuda"))
            else:
                layer.update(kc=torch.full((batch, CAPACITY, HKV, DIM), float("nan"), dtype=dtype, device="cuda"),
                             vc=torch.full((batch, CAPACITY, HKV, DIM), float("nan"), dtype=dtype, device="cuda"))
            self.layers.append(layer)
        code = 0 if dtype == f32 else 1
        self.workspace = torch.empty(ssd.binding.lib().ssd_attn_decode_workspace_bytes(batch, CAPACITY, HQ, HKV, DIM, code),
                                     dtype=torch.uint8, device="cuda")

    def tensors(self):
        return [L[n] for L in self.layers for n in ("state", "kc", "vc") if n in L]

    def split(self, layer, x):
        norm = torch.nn.functional.rms_norm(x.float(), (WIDTH,)).to(self.dtype)
        p, t = norm @ layer["win"], x.shape[0]
        if layer["kind"] == "ssd":
            x, b, c = p.split([SH * SP, SN, SN], 1)
            return x.reshape(t, SH, SP), b.reshape(t, 1, SN), c.reshape(t, 1, SN)
        sizes, heads = (([LQ * DK, LQ * DK, LV * DV], (LQ, LQ, LV)) if layer["kind"] == "lin" else
                        ([HQ * DIM, HKV * DIM, HKV * DIM], (HQ, HKV, HKV)))
        return [y.unflatten(1, (h, -1)) for y, h in zip(p.split(sizes, 1), heads)]   # slices, not copies

    def dt(self, t):
        return torch.full((t, SH), 0.1, device="cuda")

    def note(self, *what):
        if self.seen is not None:
            self.seen.append(what)

    def prefill(self, x, lens):
        offsets, cu = ref.offsets(lens), ref.cu(lens)
        for L in self.layers:
            q, k, v = self.split(L, x)
            if L["kind"] == "ssd":
                q, k, v = (z.contiguous() for z in (q, k, v))
                y, L["state"] = ssd.ssd_prefill_varlen(q, self.dt(len(x)), L["A"], k, v, L["D"], cu, 128)
            elif L["kind"] == "lin":
                y, L["state"] = ssd.ssd_linattn_prefill(q, k, v, L["ld"], cu, scale=DK ** -0.5)
                self.note("lin", q, k, v, L["ld"], y, L["state"].clone())
            else:
                y = ssd.ssd_attn_prefill(q, k, v, cu)
                for b, n in enumerate(lens):
                    L["kc"][b, :n], L["vc"][b, :n] = (z[offsets[b]:offsets[b + 1]] for z in (k, v))
                self.note("attn", q, k, v, y)
            x = x + y.flatten(1).to(self.dtype) @ L["wout"]
        return x

    def step(self, x, lens):
        """lens: cached tokens per row, int32 on the device; advanced."""
        for L in self.layers:
            q, k, v = (z.contiguous() for z in self.split(L, x))
            if L["kind"] == "ssd":
                y = ssd.ssd_decode_step(L["state"], q, self.dt(len(x)), L["A"], k, v, L["D"])
            elif L["kind"] == "lin":
                before = L["state"].clone()
                y = ssd.ssd_linattn_decode_step(L["state"], q, k, v, L["ld"], scale=DK ** -0.5)
                self.note("lin", before, q, k, v, L["ld"], y, L["state"].clone())
            else:
                y = ssd.ssd_attn_decode_step(L["kc"], L["vc"], lens, q, k, v, workspace=self.workspace)
                self.note("attn", L["kc"].clone(), L["vc"].clone(), lens.tolist() if self.seen is not None else None, q, k, v, y)
            x = x + y.flatten(1).to(self.dtype) @ L["wout"]
        lens += 1
        return x


@pytest.mark.parametrize("dtype", [bf, f32])
def test_prompts_then_tokens(dtype):
    lens = [150, 1, 0, 290, 64]
    stack = Stack(dtype, len(lens))
    stack.seen = []
    x = stack.prefill(ref.randn(sum(lens), WIDTH, seed=1, dtype=dtype), lens)
    assert torch.isfinite(x).all()
    for kind, q, k, v, *rest in stack.seen:
        if kind == "lin":
            wo, wf, to, tf = ref.linattn(q, k, v, rest[0], lens, DK ** -0.5)
            ref.assert_within(rest[1], wo, to, "linear attention")
            ref.assert_within(rest[2], wf, tf, "linear attention: states")
        else:
            wo, to = ref.attn(q, k, v, lens, DIM ** -0.5)
            ref.assert_within(rest[0], wo, to, "attention")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for i in range(3):
        stack.seen = []
        x = stack.step(ref.randn(len(lens), WIDTH, seed=2 + i, dtype=dtype), n)
        assert torch.isfinite(x).all()
        for kind, *a in stack.seen:
            if kind == "lin":
                before, q, k, v, ld, y, after = a
                wo, ws, to, ts = ref.linattn_step(before, q, k, v, ld, DK ** -0.5)
                ref.assert_within(y, wo, to, f"token {i}: linear attention")
                ref.assert_within(after, ws, ts, f"token {i}: linear attention: states")
            else:
                kc, vc, at, q, k, v, y = a
                wo, to = ref.attn_step(kc, vc, at, q, k, v, DIM ** -0.5)
                ref.assert_within(y, wo, to, f"token {i}: attention")
    assert n.tolist() == [m + 3 for m in lens] and ssd.ssd_device_status() == 0


@pytest.mark.parametrize("dtype", [bf, f32])
def test_captured_steps_share_a_workspace(dtype):
    """Two stacks' steps captured as two graphs over one workspace, replayed in turn, equal eager steps."""
    lens, tokens = [150, 1, 0, 290, 64], 4
    prompts = [ref.randn(sum(lens), WIDTH, seed=20 + i, dtype=dtype) for i in range(2)]
    steps = [[ref.randn(len(lens), WIDTH, seed=30 + 10 * i + t, dtype=dtype) for t in range(tokens)] for i in range(2)]
    stacks = [Stack(dtype, len(lens)) for _ in range(2)]
    stacks[1].workspace = stacks[0].workspace
    want, kept, graphs = [], [], []
    for stack, prompt, xs in zip(stacks, prompts, steps):
        stack.prefill(prompt, lens)
        kept.append([z.clone() for z in stack.tensors()])
        n = torch.tensor(lens, dtype=torch.int32, device="cuda")
        want.append([stack.step(x, n) for x in xs])
        want[-1].append([z.clone() for z in stack.tensors()])
    for stack in stacks:
        x, n = torch.zeros(len(lens), WIDTH, dtype=dtype, device="cuda"), torch.tensor(lens, dtype=torch.int32, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = stack.step(x, n)
        graphs.append((graph, x, n, y))
    for stack, was in zip(stacks, kept):
        for z, old in zip(stack.tensors(), was):
            z.copy_(old)
    for t in range(tokens):
        for i, (graph, x, _, y) in enumerate(graphs):
            x.copy_(steps[i][t])
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want[i][t]), f"stack {i}, token {t}"
    for stack, w in zip(stacks, want):
        for z, old in zip(stack.tensors(), w[-1]):
            assert torch.equal(z.nan_to_num(7.0), old.nan_to_num(7.0))
    assert ssd.ssd_device_status() == 0


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("op", ["linattn_prefill", "linattn_step", "attn_prefill", "attn_step"])
@pytest.mark.parametrize("eager", [True, False])
def test_inputs_of_three_streams(dtype, op, eager):
    """Queries written by a kernel of the call's own stream just before it, keys by a copy of a second
    stream and values and lengths by kernels of a third: the call waits for all of them, eager and as a
    node of a graph with several nodes before it; a replay sees new inputs."""
    lens, n, dim, hq, hkv = [300, 0, 77, 1], 378, 64, 4, 2
    rows = n if op.endswith("prefill") else len(lens)
    src = [ref.randn(rows, h, dim, seed=60 + i, dtype=dtype) for i, h in enumerate((hq, hkv, hkv) if "attn_" in op and "lin" not in op else (hkv, hkv, hq))]
    q, k, v = (torch.zeros_like(z) for z in src)
    cu, given = ref.cu(lens), torch.tensor([9, 0, 63, 64], dtype=torch.int32, device="cuda")
    ld, at = -0.1 * torch.ones(hq, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    state = ref.randn(4, hq, dim, dim, seed=70)
    kc, vc = (ref.randn(4, 80, hkv, dim, seed=71 + i, dtype=dtype) for i in range(2))
    out = torch.empty(rows, hq, dim, dtype=dtype, device="cuda")
    fin = torch.empty(4, hq, dim, dim, device="cuda")
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    big = torch.ones(1 << 26, device="cuda")               # keeps each stream busy before it writes
    streams = [torch.cuda.Stream() for _ in range(2)]

    def run():
        main = torch.cuda.current_stream()
        for s in streams:
            s.wait_stream(main)
        with torch.cuda.stream(streams[0]):
            big[:1 << 24].mul_(1.0)
            k.copy_(src[1])
        with torch.cuda.stream(streams[1]):
            big[1 << 24:1 << 25].mul_(1.0)
            torch.mul(src[2], 1, out=v)
            torch.mul(given, 1, out=at)
        big[1 << 25:].mul_(1.0)
        torch.mul(src[0], 1, out=q)
        for s in streams:
            main.wait_stream(s)
        if op == "linattn_prefill":
            ssd.ssd_linattn_prefill(q, k, v, ld, cu, init_states=state, out=out, final_states=fin, workspace=ws)
        elif op == "linattn_step":
            ssd.ssd_linattn_decode_step(state, q, k, v, ld, out=out)
        elif op == "attn_prefill":
            ssd.ssd_attn_prefill(q, k, v, cu, out=out)
        else:
            ssd.ssd_attn_decode_step(kc, vc, at, q, k, v, out=out, workspace=ws)

    def want():
        if op == "linattn_prefill":
            w = ref.linattn(*src, ld, lens, 1.0, state)
            return w[0], w[2]
        if op == "linattn_step":
            w = ref.linattn_step(state, *src, ld, 1.0)
            return w[0], w[2]
        if op == "attn_prefill":
            return ref.attn(*src, lens, dim ** -0.5)
        return ref.attn_step(kc, vc, given.tolist(), *src, dim ** -0.5)

    if not eager:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
    for i in range(3):
        for z in (q, k, v, out):
            z.zero_()
        at.fill_(5)
        src[0].mul_(-1)
        src[2].mul_(-0.5)
        expected, tol = want()
        torch.cuda.synchronize()
        run() if eager else graph.replay()
        torch.cuda.synchronize()
        ref.assert_within(out, expected, tol, f"{op}, run {i}")
    assert ssd.ssd_device_status() == 0


@pytest.mark.parametrize("dtype", [bf, f32])
def test_calls_at_once_on_several_streams(dtype):
    """Calls of three kinds on streams of their own, again and again: bit for bit what each gives alone."""
    lens = [700, 0, 33, 1500, 129]
    n, dim = sum(lens), 64
    q, k, v = (ref.randn(n, h, dim, seed=80 + i, dtype=dtype) for i, h in enumerate((8, 4, 4)))
    cu, ld, s0 = ref.cu(lens), -0.01 * torch.ones(8, device="cuda"), ref.randn(5, 8, dim, dim, seed=84)
    kc, vc = (ref.randn(5, 900, 4, dim, seed=85 + i, dtype=dtype) for i in range(2))
    at = torch.tensor([899, 0, 400, 64, 3], dtype=torch.int32, device="cuda")
    wide = ref.randn(n, 8, dim, seed=87, dtype=dtype)
    calls = [lambda: ssd.ssd_linattn_prefill(k, v, wide, ld, cu, init_states=s0),
             lambda: (ssd.ssd_attn_prefill(q, k, v, cu),),
             lambda: (ssd.ssd_attn_decode_step(kc, vc, at, q[:5], k[:5], v[:5]),),
             lambda: ssd.ssd_linattn_prefill(k, wide[:, :4].contiguous(), wide, ld, cu)]
    want = []
    for call in calls:
        want.append(call())
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[] for _ in calls]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(8):
        for i, (call, s) in enumerate(zip(calls, streams)):
            with torch.cuda.stream(s):
                got[i].append(call())
    torch.cuda.synchronize()
    for i, w in enumerate(want):
        for g in got[i]:
            assert all(torch.equal(x, y) for x, y in zip(g, w)), i
    assert ssd.ssd_device_status() == 0


@pytest.mark.parametrize("dtype", [bf, f32])
def test_most_sequences_and_most_heads(dtype):
    """2^20 sequences of one token, and 65535 heads: a lone token's attention is its own value, and its
    linear attention's state k v^T."""
    for n, heads, offsets in ((1 << 20, 1, None), (2, 65535, [0, 1, 2])):
        cu = torch.arange(n + 1, dtype=torch.int32, device="cuda") if offsets is None else ref.cu([1, 1])
        q, k, v = (ref.randn(n, heads, 8, seed=90 + i, dtype=dtype) for i in range(3))
        assert torch.equal(ssd.ssd_attn_prefill(q, k, v, cu), v)
        out, fin = ssd.ssd_linattn_prefill(q, k, v, torch.zeros(heads, device="cuda"), cu)
        kv = k.double()[..., :, None] * v.double()[..., None, :]
        # one rounding of a product, or its value as a sum of three bf16 numbers
        assert ((fin.double() - kv).abs() <= 2.0 ** -23 * kv.abs()).all()
        want = (q.double() * k.double()).sum(-1, keepdim=True) * v.double()
        size = (q.double() * k.double()).abs().sum(-1, keepdim=True) * v.double().abs()
        half = ref.HALF[dtype]                             # of the score and of the output, and fp32 sums
        assert ((out.double() - want).abs() <= half * want.abs() + ((half if dtype == bf else 0.0) + 12 * ref.F32) * size * (1 + half)).all()
    assert ssd.ssd_device_status() == 0
