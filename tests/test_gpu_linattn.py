"""GPU parity of linear attention with a decay per head (packed prefill and single-token step)
against the fp64 recurrence; tolerances from the kernels' roundings (mixers_ref)."""
import pytest
import torch

import mixers_ref as ref
import state_space_model_05_b200 as ssd

pytestmark = pytest.mark.gpu

bf, f32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True, scope="module")
def _built():
    from state_space_model_05_b200.build import build
    build()


def problem(lens, hq, hv, dk, dv, dtype, seed=0, init=False):
    n = sum(lens)
    q, k = ref.randn(n, hq, dk, seed=seed, dtype=dtype), ref.randn(n, hq, dk, seed=seed + 1, dtype=dtype)
    v = ref.randn(n, hv, dv, seed=seed + 2, dtype=dtype)
    ld = -torch.exp(-6 * torch.rand(hv, generator=torch.Generator().manual_seed(seed + 3))).cuda()
    s0 = ref.randn(len(lens), hv, dk, dv, seed=seed + 4) if init else None
    return q, k, v, ld, s0


def check(lens, q, k, v, ld, s0, scale, what, **kw):
    out, fin = ssd.ssd_linattn_prefill(q, k, v, ld, ref.cu(lens), scale=scale, init_states=s0, **kw)
    torch.cuda.synchronize()
    assert ssd.ssd_device_status() == 0
    wo, wf, to, tf = ref.linattn(q, k, v, ld, lens, scale, s0)
    ref.assert_within(out[:sum(lens)], wo, to, f"{what}: out")
    ref.assert_within(fin, wf, tf, f"{what}: final states")
    return out, fin


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("hq,hv,dk,dv", [(1, 1, 8, 8), (2, 4, 64, 64), (2, 2, 128, 128), (1, 3, 72, 40), (2, 4, 128, 64),
                                         (1, 2, 64, 128), (3, 3, 16, 120)])
def test_shapes(dtype, hq, hv, dk, dv):
    lens = [0, 1, 130, 17, 0, 256, 63]
    q, k, v, ld, s0 = problem(lens, hq, hv, dk, dv, dtype, seed=dk + dv, init=True)
    check(lens, q, k, v, ld, s0, dk ** -0.5, f"{hq}/{hv} heads, {dk} x {dv}")


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("n", [1, 2, 7, 8, 31, 32, 33, 63, 64, 65, 127, 128, 129, 192, 255, 256, 257, 640, 1000])
def test_lengths(dtype, n):
    q, k, v, ld, s0 = problem([n], 1, 2, 64 if n % 2 else 128, 128 if n % 3 else 64, dtype, seed=n)
    check([n], q, k, v, ld, s0, 0.125, f"{n} tokens")


@pytest.mark.parametrize("dtype", [bf, f32])
def test_long_prompt_with_neighbours(dtype):
    """Long enough that the tensor-core path splits it, between short sequences."""
    lens = [3, 5003, 129]
    q, k, v, ld, s0 = problem(lens, 1, 2, 128, 128, dtype, seed=5, init=True)
    check(lens, q, k, v, ld, s0, 0.1, "long prompt")


@pytest.mark.parametrize("dtype", [bf, f32])
def test_one_long_prompt_without_state(dtype):
    q, k, v, ld, s0 = problem([2999], 2, 2, 64, 128, dtype, seed=6)
    check([2999], q, k, v, ld, s0, 0.1, "one long prompt")


@pytest.mark.parametrize("dtype", [bf, f32])
def test_decays(dtype):
    """No decay, almost none, decays that underflow within a block, one that forgets everything, growth."""
    lens = [300, 41]
    q, k, v, _, s0 = problem(lens, 1, 6, 64, 64, dtype, seed=7, init=True)
    ld = torch.tensor([0.0, -1e-7, -3.0, -200.0, float("-inf"), 0.01], device="cuda")
    check(lens, q, k, v, ld, s0, 0.125, "decays")


@pytest.mark.parametrize("dtype", [bf, f32])
def test_many_short_sequences(dtype):
    lens = [(7 * i) % 5 for i in range(300)]
    q, k, v, ld, s0 = problem(lens, 1, 2, 64, 64, dtype, seed=8, init=True)
    check(lens, q, k, v, ld, s0, 1.0, "short sequences")


@pytest.mark.parametrize("dtype", [bf, f32])
def test_slices_of_a_fused_projection_and_rows_behind(dtype):
    """Strided q, k, v; rows past the last sequence are neither read into results nor written."""
    lens, hq, hv, dk, dv = [70, 200], 2, 4, 64, 64
    n, pad = sum(lens), 9
    width = (2 * hq * dk + hv * dv) + 8
    fused = ref.randn(n + pad, width, seed=9, dtype=dtype)
    fused[n:] = float("nan")
    q = fused[:, :hq * dk].unflatten(1, (hq, dk))
    k = fused[:, hq * dk:2 * hq * dk].unflatten(1, (hq, dk))
    v = fused[:, 2 * hq * dk:2 * hq * dk + hv * dv].unflatten(1, (hv, dv))
    ld = -torch.rand(hv, generator=torch.Generator().manual_seed(1)).cuda() * 0.1
    out = torch.full((n + pad, hv, dv), 7.0, dtype=dtype, device="cuda")
    ssd.ssd_linattn_prefill(q, k, v, ld, ref.cu(lens), scale=0.2, out=out)
    assert ssd.ssd_device_status() == 0
    assert bool((out[n:] == 7.0).all())
    wo, _, to, _ = ref.linattn(q[:n], k[:n], v[:n], ld, lens, 0.2)
    ref.assert_within(out[:n], wo, to, "strided")


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_sequence_stays_its_own(dtype, bad):
    lens = [40, 100, 200]
    q, k, v, ld, s0 = problem(lens, 1, 2, 64, 64, dtype, seed=10, init=True)
    for x in (q, k, v):
        x[40:140] = bad
    out, fin = ssd.ssd_linattn_prefill(q, k, v, ld, ref.cu(lens), init_states=s0)
    assert ssd.ssd_device_status() == 0
    for i, rows in ((0, slice(0, 40)), (2, slice(140, 340))):
        wo, wf, to, tf = ref.linattn(q[rows], k[rows], v[rows], ld, [lens[i]], 1.0, s0[i:i + 1])
        ref.assert_within(out[rows], wo, to, f"sequence {i}")
        ref.assert_within(fin[i:i + 1], wf, tf, f"state {i}")
    assert not torch.isfinite(out[40:140]).any()


@pytest.mark.parametrize("dtype", [bf, f32])
def test_later_tokens_do_not_reach_back(dtype):
    """Tokens from t on hold NaN and infinities: the outputs before t are what they were."""
    q, k, v, ld, s0 = problem([300], 1, 2, 64, 64, dtype, seed=11)
    want, _ = ssd.ssd_linattn_prefill(q, k, v, ld, ref.cu([300]))
    for t in (1, 77, 129, 290):
        k2, v2 = k.clone(), v.clone()
        k2[t:], v2[t:] = float("nan"), float("inf")
        got, _ = ssd.ssd_linattn_prefill(q, k2, v2, ld, ref.cu([300]))
        assert torch.isfinite(got[:t]).all(), t
        wo, _, to, _ = ref.linattn(q[:t], k[:t], v[:t], ld, [t], 1.0)
        ref.assert_within(got[:t], wo, to, f"before token {t}")
        assert not torch.isfinite(got[t:]).any()


def test_state_buffer_may_be_reused():
    lens = [150, 0, 30]
    q, k, v, ld, s0 = problem(lens, 1, 2, 64, 128, bf, seed=12, init=True)
    out, fin = ssd.ssd_linattn_prefill(q, k, v, ld, ref.cu(lens), init_states=s0)
    buf = s0.clone()
    out2, fin2 = ssd.ssd_linattn_prefill(q, k, v, ld, ref.cu(lens), init_states=buf, final_states=buf)
    assert fin2 is buf and torch.equal(out, out2) and torch.equal(fin, fin2)


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("hv,dk,dv", [(8, 128, 128), (6, 40, 72), (40, 128, 64)])
def test_state_buffer_may_be_reused_by_long_prompts(dtype, hv, dk, dv):
    """Sequences whose parts run side by side, each of which starts from the initial state that the
    last one replaces; decays near 1, so that it counts to the end."""
    lens = [2500, 1, 0, 3001, 130]
    q, k, v, ld, s0 = problem(lens, 2, hv, dk, dv, dtype, seed=15, init=True)
    ld, s0 = ld * 1e-4, s0 * 30
    out, fin = check(lens, q, k, v, ld, s0, 0.1, "separate states")
    for _ in range(3):
        buf = s0.clone()
        out2, fin2 = ssd.ssd_linattn_prefill(q, k, v, ld, ref.cu(lens), scale=0.1, init_states=buf, final_states=buf)
        assert fin2 is buf and torch.equal(out, out2) and torch.equal(fin, fin2)


def test_no_tokens_copies_the_states():
    z = lambda *s: torch.zeros(s, device="cuda", dtype=bf)
    s0 = ref.randn(2, 2, 64, 64, seed=13)
    out, fin = ssd.ssd_linattn_prefill(z(0, 1, 64), z(0, 1, 64), z(0, 2, 64), torch.zeros(2, device="cuda"),
                                       ref.cu([0, 0]), init_states=s0)
    assert out.shape == (0, 2, 64) and torch.equal(fin, s0)
    _, fin = ssd.ssd_linattn_prefill(z(0, 1, 64), z(0, 1, 64), z(0, 2, 64), torch.zeros(2, device="cuda"),
                                     ref.cu([0, 0]))
    assert not fin.any()


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("offsets", [[0, 50, 40, 100], [0, 50, 101], [-4, 50, 100], [5, 50, 100]])
def test_bad_offsets_are_reported(dtype, offsets):
    q, k, v, ld, _ = problem([100], 1, 2, 64, 64, dtype, seed=14)
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    ssd.ssd_linattn_prefill(q, k, v, ld, cu)
    assert ssd.ssd_device_status() == 2                      # SSD_ERR_SHAPE
    assert ssd.ssd_device_status() == 0


@pytest.mark.parametrize("dtype", [bf, f32])
def test_graph_and_side_stream_match(dtype):
    lens = [900, 3, 260]
    q, k, v, ld, s0 = problem(lens, 2, 4, 128, 64, dtype, seed=15, init=True)
    cu = ref.cu(lens)
    out, fin = ssd.ssd_linattn_prefill(q, k, v, ld, cu, init_states=s0)
    torch.cuda.synchronize()
    ws = torch.empty(ssd.binding.lib().ssd_linattn_prefill_workspace_bytes(3, sum(lens), 2, 4, 128, 64,
                                                                          0 if dtype == f32 else 1), dtype=torch.uint8,
                     device="cuda")
    o2, f2 = torch.empty_like(out), torch.empty_like(fin)
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        ssd.ssd_linattn_prefill(q, k, v, ld, cu, init_states=s0, out=o2, final_states=f2, workspace=ws)
    for _ in range(2):
        o2.zero_(), f2.zero_()
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, o2) and torch.equal(fin, f2)
    with torch.cuda.stream(stream):
        o3, f3 = ssd.ssd_linattn_prefill(q, k, v, ld, cu, init_states=s0)
    torch.cuda.synchronize()
    assert torch.equal(out, o3) and torch.equal(fin, f3)


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("batch,hq,hv,dk,dv", [(1, 16, 32, 128, 128), (3, 2, 4, 64, 128), (5, 1, 3, 72, 40),
                                               (64, 4, 4, 128, 64), (2, 1, 1, 8, 8), (70, 3, 9, 64, 64)])
def test_decode_steps(dtype, batch, hq, hv, dk, dv):
    state = ref.randn(batch, hv, dk, dv, seed=dk)
    ld = -torch.exp(-6 * torch.rand(hv, generator=torch.Generator().manual_seed(hv))).cuda()
    for t in range(3):
        q, k = (ref.randn(batch, hq, dk, seed=10 * t + i, dtype=dtype) for i in (1, 2))
        v = ref.randn(batch, hv, dv, seed=10 * t + 3, dtype=dtype)
        wo, ws, to, ts = ref.linattn_step(state, q, k, v, ld, 0.3)
        out = ssd.ssd_linattn_decode_step(state, q, k, v, ld, scale=0.3)
        ref.assert_within(out, wo, to, f"step {t}: out")
        ref.assert_within(state, ws, ts, f"step {t}: state")
    assert ssd.ssd_device_status() == 0


def test_decode_limits():
    """No memory at all, none lost, and an empty batch."""
    state = ref.randn(1, 2, 64, 64, seed=3)
    old = state.clone()
    q, k, v = ref.randn(1, 1, 64, seed=4), ref.randn(1, 1, 64, seed=5), ref.randn(1, 2, 64, seed=6)
    ssd.ssd_linattn_decode_step(state, q, k, v, torch.tensor([float("-inf"), 0.0], device="cuda"))
    kv = k[0, 0][:, None] * v[0, :, None, :]
    assert torch.equal(state[0, 0], kv[0])
    torch.testing.assert_close(state[0, 1], old[0, 1] + kv[1], rtol=2 ** -22, atol=2 ** -22)
    e = lambda *s: torch.empty(s, device="cuda")
    assert ssd.ssd_linattn_decode_step(e(0, 2, 64, 64), e(0, 1, 64), e(0, 1, 64), e(0, 2, 64), e(2)).shape == (0, 2, 64)


@pytest.mark.parametrize("dtype", [bf, f32])
def test_prefill_then_steps_is_prefill(dtype):
    """The state after T tokens and k steps is the state after T + k tokens."""
    q, k, v, ld, s0 = problem([205], 2, 4, 64, 128, dtype, seed=16, init=True)
    out, state = ssd.ssd_linattn_prefill(q[:200], k[:200], v[:200], ld, ref.cu([200]), scale=0.1, init_states=s0)
    outs = [ssd.ssd_linattn_decode_step(state, q[t:t + 1], k[t:t + 1], v[t:t + 1], ld, scale=0.1) for t in range(200, 205)]
    wo, wf, to, tf = ref.linattn(q, k, v, ld, [205], 0.1, s0)
    ref.assert_within(torch.cat([out, *outs]), wo, to, "outputs")
    ref.assert_within(state, wf, tf, "state")


@pytest.mark.parametrize("dtype", [bf, f32])
def test_offsets_whose_difference_overflows_touch_nothing(dtype):
    """A next offset near the lowest 32-bit value: reported, and neither the workspace's surroundings
    nor the states of that sequence are written."""
    q, k, v, ld, _ = problem([100], 1, 2, 64, 64, dtype, seed=18)
    cu = torch.tensor([0, 100, -(1 << 31) + 50, 100], dtype=torch.int32, device="cuda")
    need = ssd.binding.lib().ssd_linattn_prefill_workspace_bytes(3, 100, 1, 2, 64, 64, 0 if dtype == f32 else 1)
    room = torch.full((need + (64 << 20),), 77, dtype=torch.uint8, device="cuda")
    fin = torch.full((3, 2, 64, 64), 7.0, device="cuda")
    ssd.ssd_linattn_prefill(q, k, v, ld, cu, final_states=fin, workspace=room[32 << 20:(32 << 20) + need])
    assert ssd.ssd_device_status() == 2                      # SSD_ERR_SHAPE
    assert bool((room[:32 << 20] == 77).all()) and bool((room[(32 << 20) + need:] == 77).all())
    assert bool((fin[1:] == 7.0).all())


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("hq,hv,dk,dv", [(1, 2, 64, 64), (2, 2, 128, 128), (1, 3, 72, 40), (1, 2, 64, 128), (1, 1, 128, 64)])
def test_values_that_are_not_finite_reach_their_own_columns(dtype, hq, hv, dk, dv):
    """Infinite and NaN values of a few tokens, two of them in one block and one in a block's last row:
    their columns are not finite from those tokens on, with the value's sign in its own block (all
    queries and keys are positive); all else is what it is without them."""
    lens = [300, 70, 128]
    q, k, v, ld, s0 = problem(lens, hq, hv, dk, dv, dtype, seed=21, init=True)
    q, k = q.abs(), k.abs()
    bad = [(0, 100, 5, float("inf")), (0, 103, 5, float("inf")), (0, 110, dv - 1, float("-inf")), (0, 127, 9, float("nan")),
           (370, 497, 16, float("-inf")), (300, 369, 3, float("nan"))]
    v2 = v.clone()
    for _, t, col, x in bad:
        v[t, 0, col], v2[t, 0, col] = x, 0.0
    out, fin = ssd.ssd_linattn_prefill(q, k, v, ld, ref.cu(lens), scale=0.1, init_states=s0)
    assert ssd.ssd_device_status() == 0
    wo, wf, to, tf = ref.linattn(q, k, v2, ld, lens, 0.1, s0)
    clean = torch.ones(out.shape, dtype=torch.bool)
    clean_state = torch.ones(fin.shape, dtype=torch.bool)
    for start, t, col, x in bad:
        i = ref.offsets(lens).index(start)
        end = start + lens[i]
        clean[t:end, 0, col], clean_state[i, 0, :, col] = False, False
        block = min(end, start + ((t - start) // 64 + 1) * 64)         # (64: the shorter of the two paths' blocks)
        got = out[t:block, 0, col]
        assert bool(torch.isnan(got).all() if x != x else (got == x).all()), (t, col)
        assert not torch.isfinite(out[t:end, 0, col]).any() and not torch.isfinite(fin[i, 0, :, col]).any()
    ref.assert_within(out.cpu()[clean], wo[clean], to[clean], "outputs")
    ref.assert_within(fin.cpu()[clean_state], wf[clean_state], tf[clean_state], "states")


@pytest.mark.parametrize("what", ["one", "inf", "nan", "inf on positive keys"])
def test_values_that_are_not_finite_cost_little(what):
    """A block of 128 tokens takes a few microseconds; one whose values are not finite may take a
    hundred more (128 tokens of 128 products and 128 columns in each of 128 rows: some 64,000
    instructions a warp), not the milliseconds of forming every output anew.  Where all of a block's
    state is infinite, its 16 groups of columns are formed anew one after the other, 128 tokens each:
    some 0.4 ms."""
    n = 2048
    q, k, v, ld, _ = problem([n], 2, 4, 128, 128, bf, seed=22)
    if what == "one":
        v[5::128, :, 7] = float("inf")
    else:
        v[:] = float(what.split()[0])
        k = k.abs() if "positive" in what else k
    cu, best = ref.cu([n]), 1e9
    for _ in range(4):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        out, _ = ssd.ssd_linattn_prefill(q, k, v, ld, cu)
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    assert ssd.ssd_device_status() == 0
    assert not torch.isfinite(out[5:, :, 7]).any()
    limit = 12.8 if "positive" in what else 3.2              # 16 blocks of 0.4 ms or 0.1 ms, and as much again
    assert best < limit, f"{best:.3f} ms"
    print(what, f"{1e3 * best:.0f} us")


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("lens,hq,hv,dk,dv", [([300, 70, 128], 1, 2, 64, 64), ([200, 129], 2, 2, 128, 128), ([257], 1, 3, 72, 40),
                                              ([40, 5003, 3], 1, 2, 64, 128), ([1500], 1, 1, 128, 64)])
@pytest.mark.parametrize("start", [True, False])
def test_states_with_infinities_are_those_of_the_recurrence(dtype, lens, hq, hv, dk, dv, start):
    """Infinite values, infinite keys, both, infinities that meet their opposite or a zero, and products
    that overflow: every element of the final states is the infinity, the NaN or the number that the
    recurrence gives.  (Decays whose powers stay within fp32 over the longest sequence.)"""
    q, k, v, _, s0 = problem(lens, hq, hv, dk, dv, dtype, seed=23, init=start)
    ld = -torch.linspace(0.001, 0.01, hv).cuda()
    inf, nan = float("inf"), float("nan")
    at = ref.offsets(lens)[lens.index(max(lens))]          # the longest sequence's first token
    n = max(lens)
    k[at + 10, 0, 7] = 0.0
    k2, v2 = k.clone(), v.clone()
    for t, col, x in ((10, 3, inf), (100, 4, -inf), (130, 4, -inf), (50, 5, inf), (190, 5, -inf), (n - 1, 6, inf), (77, 8, nan)):
        v[at + t, 0, col], v2[at + t, 0, col] = x, 0.0
    for t, row, x in ((20, 11, inf), (128, 12, -inf), (60, 13, inf), (61, 13, -inf), (n - 2, 14, -inf)):
        k[at + t, 0, row], k2[at + t, 0, row] = x, 0.0
    k[at + 150, 0, 20] = k2[at + 150, 0, 20] = v[at + 151, hv - 1, 21] = v2[at + 151, hv - 1, 21] = 3e38
    k[at + 151, 0, 20] = k2[at + 151, 0, 20] = -3e38       # with both at token 151, the product passes fp32
    _, fin = ssd.ssd_linattn_prefill(q, k, v, ld, ref.cu(lens), init_states=s0)
    assert ssd.ssd_device_status() == 0
    _, _, _, tol = ref.linattn(q, k2, v2, ld, lens, 1.0, s0)
    head = torch.arange(hv) // (hv // hq)
    for i, n in enumerate(lens):
        g = torch.exp(ld.cpu().double())[:, None, None]
        S = torch.zeros(hv, dk, dv, dtype=torch.float64) if s0 is None else s0[i].cpu().double()
        size = S.abs()                                     # the same recurrence on the finite products' sizes
        most = size.clone()                                # and the largest it ever was
        a = ref.offsets(lens)[i]
        for kt, vt in zip(k[a:a + n].cpu().double(), v[a:a + n].cpu().double()):
            kv = kt[head][:, :, None] * vt[:, None, :]
            S, size = g * S + kv, g * size + kv.abs().nan_to_num(0.0, 0.0)
            most = torch.maximum(most, size)
        got, want = fin[i].cpu(), S.float()
        # sums whose finite terms' sizes reach past fp32 (2^128) on the way are infinite, NaN or finite by
        # the order in which they are formed: row 20 and column 21 of some heads
        sure = most < 2.0 ** 127
        assert sure[:, [r for r in range(dk) if r != 20]][..., [c for c in range(dv) if c != 21]].all()
        if a == at:
            assert torch.isinf(want[sure]).any() and torch.isnan(want[sure]).any()
        wrong = sure & ((torch.isnan(got) != torch.isnan(want)) | (torch.isinf(want) & (got != want) & ~torch.isnan(got)))
        assert not wrong.any(), (i, wrong.nonzero()[:10].tolist(), got[wrong][:10].tolist(), want[wrong][:10].tolist())
        fine = sure & torch.isfinite(want)
        ref.assert_within(got[fine], S[fine], tol[i][fine] + 2 * ref.F32 * S[fine].abs(), f"sequence {i}")
