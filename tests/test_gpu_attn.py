"""GPU parity of causal softmax attention (packed prompts, and one token against a cache) against
fp64; tolerances from the kernels' roundings (mixers_ref)."""
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


def problem(n, hq, hkv, dim, dtype, seed=0):
    return (ref.randn(n, hq, dim, seed=seed, dtype=dtype), ref.randn(n, hkv, dim, seed=seed + 1, dtype=dtype),
            ref.randn(n, hkv, dim, seed=seed + 2, dtype=dtype))


def check(lens, q, k, v, scale, what):
    out = ssd.ssd_attn_prefill(q, k, v, ref.cu(lens), scale=scale)
    torch.cuda.synchronize()
    assert ssd.ssd_device_status() == 0
    wo, to = ref.attn(q, k, v, lens, scale)
    ref.assert_within(out, wo, to, what)
    return out


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("hq,hkv,dim", [(1, 1, 8), (4, 1, 64), (4, 4, 128), (6, 2, 72), (8, 1, 128), (5, 1, 64), (14, 2, 40),
                                        (3, 3, 120), (32, 1, 64)])
def test_shapes(dtype, hq, hkv, dim):
    lens = [0, 1, 130, 17, 0, 256, 63]
    check(lens, *problem(sum(lens), hq, hkv, dim, dtype, seed=dim), dim ** -0.5, f"{hq}/{hkv} heads of {dim}")


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 191, 255, 256, 257, 513, 700])
def test_lengths(dtype, n):
    hq, dim = (4, 64) if n % 2 else (2, 128)
    check([n], *problem(n, hq, 1, dim, dtype, seed=n), 0.2, f"{n} tokens")


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("hq,hkv,dim", [(2, 2, 128), (4, 1, 64)])
def test_long_prompt_with_neighbours(dtype, hq, hkv, dim):
    lens = [5, 1900, 131]
    check(lens, *problem(sum(lens), hq, hkv, dim, dtype, seed=3), dim ** -0.5, "long prompt")


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("hq,hkv,dim", [(8, 8, 128), (12, 4, 64), (16, 8, 40)])
def test_many_short_sequences(dtype, hq, hkv, dim):
    """More blocks of work than run at a time, several times over, with empty sequences between them
    and now and then a sequence of several blocks."""
    lens = [(37 * i) % 130 if i % 31 else 400 for i in range(230)]
    check(lens, *problem(sum(lens), hq, hkv, dim, dtype, seed=31), dim ** -0.5, f"{hq}/{hkv} heads of {dim}")


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_scales(dtype, scale):
    """Uniform weights, a negative scale, and one whose softmax is nearly one key."""
    check([300], *problem(300, 4, 2, 64, dtype, seed=4), scale, f"scale {scale}")


@pytest.mark.parametrize("dtype", [bf, f32])
def test_growing_scores(dtype):
    """Each key scores higher than all before it, by much: the running maximum moves on every tile."""
    n = 700
    q, k, v = problem(n, 2, 1, 64, dtype, seed=5)
    q[:] = 1.0
    k[:] = (torch.arange(n, device="cuda") / 8)[:, None, None].to(dtype)
    check([n], q, k, v, 1.0, "growing scores")
    check([n], q, -k, v, 1.0, "falling scores")


@pytest.mark.parametrize("dtype", [bf, f32])
def test_slices_of_a_fused_projection_and_rows_behind(dtype):
    lens, hq, hkv, dim = [70, 200], 4, 2, 64
    n, pad = sum(lens), 9
    fused = ref.randn(n + pad, (hq + 2 * hkv) * dim + 8, seed=9, dtype=dtype)
    fused[n:] = float("nan")
    q = fused[:, :hq * dim].unflatten(1, (hq, dim))
    k = fused[:, hq * dim:(hq + hkv) * dim].unflatten(1, (hkv, dim))
    v = fused[:, (hq + hkv) * dim:(hq + 2 * hkv) * dim].unflatten(1, (hkv, dim))
    out = torch.full((n + pad, hq, dim), 7.0, dtype=dtype, device="cuda")
    ssd.ssd_attn_prefill(q, k, v, ref.cu(lens), out=out)
    assert ssd.ssd_device_status() == 0
    assert bool((out[n:] == 7.0).all())
    wo, to = ref.attn(q[:n], k[:n], v[:n], lens, dim ** -0.5)
    ref.assert_within(out[:n], wo, to, "strided")


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_sequence_stays_its_own(dtype, bad):
    lens = [40, 100, 200]
    q, k, v = problem(340, 4, 2, 64, dtype, seed=10)
    for x in (q, k, v):
        x[40:140] = bad
    out = ssd.ssd_attn_prefill(q, k, v, ref.cu(lens))
    assert ssd.ssd_device_status() == 0
    for i, rows in ((0, slice(0, 40)), (2, slice(140, 340))):
        wo, to = ref.attn(q[rows], k[rows], v[rows], [lens[i]], 0.125)
        ref.assert_within(out[rows], wo, to, f"sequence {i}")
    assert not torch.isfinite(out[40:140]).any()


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("group", [1, 4, 6])
def test_later_tokens_do_not_reach_back(dtype, group):
    """Tokens from t on hold NaN keys and infinite values: the outputs before t are what they were."""
    q, k, v = problem(300, group, 1, 64, dtype, seed=11)
    for t in (1, 77, 129, 290):
        k2, v2 = k.clone(), v.clone()
        k2[t:], v2[t:] = float("nan"), float("inf")
        got = ssd.ssd_attn_prefill(q, k2, v2, ref.cu([300]))
        assert torch.isfinite(got[:t]).all(), t
        wo, to = ref.attn(q[:t], k[:t], v[:t], [t], 0.125)
        ref.assert_within(got[:t], wo, to, f"before token {t}")
        assert not torch.isfinite(got[t:]).any()


@pytest.mark.parametrize("dtype", [bf, f32])
def test_an_infinite_value_reaches_its_own_column(dtype):
    q, k, v = problem(300, 2, 1, 64, dtype, seed=12)
    v[100, 0, 5] = float("inf")
    v[250, 0, 9] = float("-inf")
    out = ssd.ssd_attn_prefill(q, k, v, ref.cu([300]))
    assert (out[100:, :, 5] == float("inf")).all() and (out[250:, :, 9] == float("-inf")).all()
    rest = torch.ones(64, dtype=torch.bool)
    rest[[5, 9]] = False
    v2 = v.clone()
    v2[:, 0, [5, 9]] = 0
    wo, to = ref.attn(q, k, v2, [300], 0.125)
    ref.assert_within(out[..., rest], wo[..., rest], to[..., rest], "other columns")
    assert torch.isfinite(out[:100]).all()


@pytest.mark.parametrize("dtype", [bf, f32])
def test_scores_of_minus_infinity(dtype):
    """Keys whose score is -inf weigh nothing, also where a row's first keys all are."""
    q, k, v = problem(300, 2, 1, 64, dtype, seed=13)
    q[..., 0] = 1.0
    k[1:200, 0, 0] = float("-inf")
    out = ssd.ssd_attn_prefill(q, k, v, ref.cu([300]))
    keep = torch.ones(300, 300, dtype=torch.bool).tril()
    keep[:, 1:200] = False
    for h in range(2):
        wo, to = ref.attend(q[:, h], k[:, 0], v[:, 0], 0.125, keep)
        ref.assert_within(out[:, h], wo, to, f"head {h}")
    k[0, 0, 0] = float("-inf")
    out = ssd.ssd_attn_prefill(q, k, v, ref.cu([300]))
    assert torch.isnan(out[:200]).all()                      # no key weighs anything
    keep[:, 0] = False
    for h in range(2):
        wo, to = ref.attend(q[200:, h], k[:, 0], v[:, 0], 0.125, keep[200:])
        ref.assert_within(out[200:, h], wo, to, f"head {h}, first tiles -inf")


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("offsets", [[0, 50, 40, 100], [0, 50, 101], [-4, 50, 100], [5, 50, 100]])
def test_bad_offsets_are_reported(dtype, offsets):
    q, k, v = problem(100, 2, 1, 64, dtype, seed=14)
    ssd.ssd_attn_prefill(q, k, v, torch.tensor(offsets, dtype=torch.int32, device="cuda"))
    assert ssd.ssd_device_status() == 2                      # SSD_ERR_SHAPE
    assert ssd.ssd_device_status() == 0


@pytest.mark.parametrize("dtype", [bf, f32])
def test_graph_and_side_stream_match(dtype):
    lens = [900, 3, 260]
    q, k, v = problem(sum(lens), 8, 2, 128, dtype, seed=15)
    cu = ref.cu(lens)
    out = ssd.ssd_attn_prefill(q, k, v, cu)
    torch.cuda.synchronize()
    o2 = torch.empty_like(out)
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        ssd.ssd_attn_prefill(q, k, v, cu, out=o2)
    for _ in range(2):
        o2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, o2)
    with torch.cuda.stream(stream):
        o3 = ssd.ssd_attn_prefill(q, k, v, cu)
    torch.cuda.synchronize()
    assert torch.equal(out, o3)


# ---------------------------------------------------------------- one token against a cache
def cached(lens, capacity, hq, hkv, dim, dtype, seed=0):
    b = len(lens)
    kc, vc = (ref.randn(b, capacity, hkv, dim, seed=seed + i, dtype=dtype) for i in (0, 1))
    for i, n in enumerate(lens):                             # rows past a length are never read
        kc[i, max(n, 0):], vc[i, max(n, 0):] = float("nan"), float("nan")
    q = ref.randn(b, hq, dim, seed=seed + 2, dtype=dtype)
    k, v = (ref.randn(b, hkv, dim, seed=seed + i, dtype=dtype) for i in (3, 4))
    return kc, vc, q, k, v


def check_step(lens, capacity, hq, hkv, dim, dtype, seed=0, scale=None, what=""):
    kc, vc, q, k, v = cached(lens, capacity, hq, hkv, dim, dtype, seed)
    k0, v0 = kc.clone(), vc.clone()
    out = torch.full_like(q, 7.0)
    ssd.ssd_attn_decode_step(kc, vc, torch.tensor(lens, dtype=torch.int32, device="cuda"), q, k, v, scale=scale, out=out)
    torch.cuda.synchronize()
    assert ssd.ssd_device_status() == 0
    wo, to = ref.attn_step(k0, v0, lens, q, k, v, dim ** -0.5 if scale is None else scale)
    live = [i for i, n in enumerate(lens) if n >= 0]
    ref.assert_within(out[live], wo[live], to[live], what or f"{lens}")
    for i, n in enumerate(lens):
        if n >= 0:
            k0[i, n], v0[i, n] = k[i], v[i]
        else:
            assert bool((out[i] == 7.0).all())
    bits = lambda x: x.view(torch.int16 if dtype == bf else torch.int32)  # noqa: E731  (NaN rows included)
    assert torch.equal(bits(kc), bits(k0)) and torch.equal(bits(vc), bits(v0))


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("hq,hkv,dim", [(1, 1, 8), (4, 1, 64), (4, 4, 128), (6, 2, 72), (8, 1, 128), (5, 1, 64), (17, 1, 40),
                                        (40, 2, 128), (32, 8, 128)])
def test_decode_shapes(dtype, hq, hkv, dim):
    check_step([0, 1, 63, 64, 65, 200], 300, hq, hkv, dim, dtype, seed=dim)


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("lens,capacity", [([0], 1), ([15], 16), ([16], 17), ([4999], 5000), ([127, 128, 129], 130),
                                           ([2000, 0, 3, 1999], 2001), ([-1, 40, -1, 0], 64), ([-1], 8)])
def test_decode_lengths(dtype, lens, capacity):
    check_step(lens, capacity, 4, 2, 64, dtype, seed=2)


@pytest.mark.parametrize("dtype", [bf, f32])
def test_decode_many_rows(dtype):
    check_step([(37 * i) % 90 - 1 for i in range(300)], 100, 2, 1, 64, dtype, seed=3)


@pytest.mark.parametrize("dtype", [bf, f32])
def test_decode_one_long_row_among_short(dtype):
    check_step([3, 9000, 1, 70], 9001, 8, 2, 128, dtype, seed=4)


@pytest.mark.parametrize("dtype", [bf, f32])
@pytest.mark.parametrize("scale", [0.0, -0.5, 6.0])
def test_decode_scales(dtype, scale):
    check_step([500, 40], 512, 4, 2, 64, dtype, seed=5, scale=scale)


@pytest.mark.parametrize("dtype", [bf, f32])
def test_decode_full_row_is_reported_and_left(dtype):
    kc, vc, q, k, v = cached([10, 10, 10], 20, 4, 2, 64, dtype, seed=6)
    k0 = kc.clone()
    out = torch.full_like(q, 7.0)
    lens = torch.tensor([10, 20, 10], dtype=torch.int32, device="cuda")
    ssd.ssd_attn_decode_step(kc, vc, lens, q, k, v, out=out)
    assert ssd.ssd_device_status() == 2                      # SSD_ERR_SHAPE
    assert bool((out[1] == 7.0).all()) and torch.equal(kc[1].nan_to_num(), k0[1].nan_to_num())
    for i in (0, 2):
        assert torch.equal(kc[i, 10], k[i])
        wo, to = ref.attn_step(k0[i:i + 1], vc[i:i + 1], [10], q[i:i + 1], k[i:i + 1], v[i:i + 1], 0.125)
        ref.assert_within(out[i:i + 1], wo, to, f"row {i}")


@pytest.mark.parametrize("dtype", [bf, f32])
def test_decode_graph_advances_with_the_lengths(dtype):
    """A captured step, its lengths advanced on the device between replays, equals eager steps."""
    lens = [100, 0, 333]
    kc, vc, q, k, v = cached(lens, 400, 8, 2, 64, dtype, seed=7)
    ke, ve, n = kc.clone(), vc.clone(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    ng, out = n.clone(), torch.empty_like(q)
    ws = torch.empty(ssd.binding.lib().ssd_attn_decode_workspace_bytes(3, 400, 8, 2, 64, 0 if dtype == f32 else 1),
                     dtype=torch.uint8, device="cuda")
    want = []
    for _ in range(4):
        want.append(ssd.ssd_attn_decode_step(ke, ve, n, q, k, v).clone())
        n += 1
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        ssd.ssd_attn_decode_step(kc, vc, ng, q, k, v, out=out, workspace=ws)
        ng += 1
    for i in range(4):
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i]), i
    assert torch.equal(kc.nan_to_num(), ke.nan_to_num()) and torch.equal(vc.nan_to_num(), ve.nan_to_num())


@pytest.mark.parametrize("dtype", [bf, f32])
def test_prefill_then_steps_is_prefill(dtype):
    q, k, v = problem(205, 4, 2, 64, dtype, seed=16)
    kc, vc = (torch.empty(1, 256, 2, 64, dtype=dtype, device="cuda") for _ in range(2))
    kc[0, :200], vc[0, :200] = k[:200], v[:200]
    outs = [ssd.ssd_attn_prefill(q[:200], k[:200], v[:200], ref.cu([200]))]
    for t in range(200, 205):
        n = torch.tensor([t], dtype=torch.int32, device="cuda")
        outs.append(ssd.ssd_attn_decode_step(kc, vc, n, q[t:t + 1], k[t:t + 1], v[t:t + 1]))
    wo, to = ref.attn(q, k, v, [205], 0.125)
    ref.assert_within(torch.cat(outs), wo, to, "outputs")


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(43, 1), (64, 1), (65, 1), (128, 1), (129, 1), (258, 2)])
def test_many_query_heads_on_a_key_head(hq, hkv, dim):
    """bf16: tiles of three tokens, of two, of one with rows to spare and of one that fills the tile; and
    groups past 128, which run on the CUDA cores."""
    lens = [3, 0, 130, 1, 20]
    check(lens, *problem(sum(lens), hq, hkv, dim, bf, seed=hq), dim ** -0.5, f"{hq}/{hkv} heads of {dim}")
