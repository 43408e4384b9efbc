"""The token mixers of a hybrid stack, each as one pass that can be measured.

Four operators on queries, keys and values laid out [tokens][heads][dim]:

* ``linattn_prefill``: linear attention with a decay per head over packed prompts (chunked form);
* ``linattn_decode``: the same recurrence for one token per sequence, the state updated in place;
* ``attn_prefill``: causal softmax attention over packed prompts, query heads grouped on key/value heads;
* ``attn_decode``: one token per sequence: its key and value join the cache, then attention over the cache.

``run`` computes an operator in its plain form (elementary torch operations in 32 bits, rounded once
at the end) or, with ``own``, through the package's entry points.
"""
from __future__ import annotations

import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _linattn(name, op, **kw):
    return {"name": name, "op": op, "dtype": "bf16", "seqs": 1, "tokens": 1, "cuts": 0, "heads_qk": 16,
            "heads_v": 32, "dk": 128, "dv": 128, "init": False, **kw}


def _attn(name, op, **kw):
    return {"name": name, "op": op, "dtype": "bf16", "seqs": 1, "tokens": 1, "cuts": 0, "heads_q": 32,
            "heads_kv": 8, "dim": 128, **kw}


def listed():
    return [
        # a handful of short requests that continue from cached states, an empty and a one-token
        # sequence among them: the latency of one call
        _linattn("linattn_prefill_short", "linattn_prefill", seqs=5, tokens=131, cuts=3, init=True),
        # one long prompt on its own, where few (sequence, head) pairs have to fill the GPU
        _linattn("linattn_prefill_prompt", "linattn_prefill", tokens=8192, heads_qk=32),
        # a serving batch of prompts of very different lengths, value heads grouped on key heads
        _linattn("linattn_prefill_packed", "linattn_prefill", seqs=31, tokens=16384, cuts=1, dv=64, init=True),
        # the same operator in 32 bits, at odd lengths
        _linattn("linattn_prefill_f32", "linattn_prefill", dtype="f32", seqs=3, tokens=1501, cuts=2, heads_qk=8,
                 heads_v=8, dk=64, dv=64),
        # one user's token: 2 MB of state
        _linattn("linattn_decode_one", "linattn_decode"),
        # a full batch's token: 134 MB of state, more than the L2 holds
        _linattn("linattn_decode_batch", "linattn_decode", seqs=64),
        # a few short requests, an empty one among them: the latency of one call
        _attn("attn_prefill_short", "attn_prefill", seqs=4, tokens=203, cuts=3),
        # one long prompt: the largest case
        _attn("attn_prefill_long", "attn_prefill", tokens=16384, heads_q=16, heads_kv=4),
        # a serving batch of prompts of very different lengths, half-size heads
        _attn("attn_prefill_packed", "attn_prefill", seqs=31, tokens=16384, cuts=1, dim=64),
        # the same operator in 32 bits, at odd lengths
        _attn("attn_prefill_f32", "attn_prefill", dtype="f32", seqs=2, tokens=1031, cuts=2, heads_q=8, heads_kv=2,
              dim=64),
        # one user's token against a long cache, where the cache's length has to fill the GPU
        _attn("attn_decode_long", "attn_decode", tokens=64999, capacity=65536),
        # a batch's token against caches of very different lengths
        _attn("attn_decode_batch", "attn_decode", seqs=32, tokens=60001, cuts=4, capacity=4096),
    ]


def draw(rng):
    """A case of the listed ones' ranges; no larger than the largest of them, the square of scores
    that the plain form holds for its longest sequence included."""
    def spread(lo, hi):
        return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))

    def square(c):
        return c.get("heads_v", c.get("heads_q")) * max(_lengths(c)) ** 2 if c["op"].endswith("prefill") else 0

    most, widest = [work(c) for c in listed()], max(square(c) for c in listed())
    while True:
        op = rng.choice(["linattn_prefill", "linattn_decode", "attn_prefill", "attn_decode"])
        f32 = rng.random() < 0.25
        case = {"op": op, "dtype": "f32" if f32 else "bf16", "cuts": rng.randrange(1 << 30)}
        shared, group = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 1, 2, 3, 4, 8])
        dim = lambda: rng.choice([64, 128, 128, 8 * rng.randrange(2, 17)])  # noqa: E731
        if op.startswith("linattn"):
            case |= {"heads_qk": shared, "heads_v": shared * group, "dk": dim(), "dv": dim(), "init": rng.random() < 0.5}
        else:
            case |= {"heads_q": shared * group, "heads_kv": shared, "dim": dim()}
        if op.endswith("prefill"):
            case["tokens"] = spread(1, 2000 if f32 else 16384)
            case["seqs"] = spread(1, 40)
        else:
            case["seqs"] = spread(1, 64)
            case["tokens"] = 1
        if op == "attn_decode":
            case["capacity"] = spread(16, 65536 if case["seqs"] < 4 else 4096)
            case["tokens"] = spread(1, case["seqs"] * (case["capacity"] - 1))
        w = work(case)
        if (w["bytes"] <= max(m["bytes"] for m in most) and w["flops"] <= max(m["flops"] for m in most)
                and square(case) <= widest):
            return case


def _lengths(case):
    """The sequences' lengths: ``tokens`` split at seeded places, so that some are short, some
    long and some may be empty; a decode cache's length stays below its capacity."""
    n, total = case["seqs"], case["tokens"]
    if n == 1:
        return [total]
    rng = random.Random(case["cuts"])
    weights = [rng.expovariate(1.0) for _ in range(n)]
    ends, lens = 0.0, []
    for w in weights:
        a = round(total * ends / sum(weights))
        ends += w
        lens.append(round(total * ends / sum(weights)) - a)
    if case["op"] != "attn_decode":
        if n > 3 and lens[1] > 0:                   # an empty sequence and one of a single token
            lens[0] += lens[1]
            lens[1] = 0
        if n > 4 and lens[3] > 1:
            lens[2] += lens[3] - 1
            lens[3] = 1
        return lens
    most, spare = case["capacity"] - 1, 0
    for i, length in enumerate(lens):               # what a cache cannot hold goes to the others
        spare += max(0, length - most)
        lens[i] = min(length, most)
    for i, length in enumerate(lens):
        take = min(spare, most - length)
        lens[i] += take
        spare -= take
    return lens


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dtype = _DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)

    lens = _lengths(case)
    n, total = case["seqs"], sum(lens)
    s = {"op": case["op"], "lens": lens}
    if case["op"].startswith("linattn"):
        hq, hv, dk, dv = case["heads_qk"], case["heads_v"], case["dk"], case["dv"]
        rows = total if case["op"] == "linattn_prefill" else n
        s |= {"q": normal(rows, hq, dk), "k": normal(rows, hq, dk), "v": normal(rows, hv, dv), "scale": dk ** -0.5}
        # decays of e^-1 to e^-1/512 a token, spread over the heads
        s["log_decay"] = -torch.exp(-math.log(512.0) * torch.rand((hv,), generator=g, device="cuda"))
        if case["op"] == "linattn_decode":
            s["state"] = torch.randn((n, hv, dk, dv), generator=g, device="cuda")
        else:
            s["init"] = torch.randn((n, hv, dk, dv), generator=g, device="cuda") if case["init"] else None
    else:
        hq, hkv, d = case["heads_q"], case["heads_kv"], case["dim"]
        rows = total if case["op"] == "attn_prefill" else n
        s |= {"q": normal(rows, hq, d), "k": normal(rows, hkv, d), "v": normal(rows, hkv, d), "scale": d ** -0.5}
        if case["op"] == "attn_decode":
            s |= {"k_cache": normal(n, case["capacity"], hkv, d), "v_cache": normal(n, case["capacity"], hkv, d),
                  "cache_lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    if case["op"].endswith("prefill"):
        s["cu_seqlens"] = torch.tensor([sum(lens[:i]) for i in range(n + 1)], dtype=torch.int32, device="cuda")
    return s


def prepare(case, seed):
    return _inputs(case, seed)


def run(state):
    return _OWN[state["op"]](state) if own else _PLAIN[state["op"]](state)


# ---------------------------------------------------------------- the plain forms
def _plain_linattn_prefill(s):
    q, k, v, ld = s["q"].float() * s["scale"], s["k"].float(), s["v"].float(), s["log_decay"]
    group = v.shape[1] // q.shape[1]
    outs, finals, at = [], [], 0
    for i, n in enumerate(s["lens"]):
        qs = q[at:at + n].transpose(0, 1).repeat_interleave(group, 0)                 # [hv][n][dk]
        ks = k[at:at + n].transpose(0, 1).repeat_interleave(group, 0)
        vs = v[at:at + n].transpose(0, 1)                                             # [hv][n][dv]
        at += n
        t = torch.arange(n, device=q.device, dtype=torch.float32)
        gap = t[:, None] - t[None, :]
        weights = (ld[:, None, None] * gap.clamp_min(0)).exp_().mul_(gap >= 0)
        out = weights.mul_(qs @ ks.transpose(1, 2)) @ vs
        final = (ks * torch.exp(ld[:, None] * (n - 1 - t))[:, :, None]).transpose(1, 2) @ vs
        if s["init"] is not None:
            out += (qs * torch.exp(ld[:, None] * (t + 1))[:, :, None]) @ s["init"][i]
            final += torch.exp(ld * n)[:, None, None] * s["init"][i]
        outs.append(out.transpose(0, 1))
        finals.append(final)
    return {"out": torch.cat(outs).to(s["v"].dtype), "final_states": torch.stack(finals)}


def _plain_linattn_decode(s):
    q, k, v = s["q"].float() * s["scale"], s["k"].float(), s["v"].float()
    group = v.shape[1] // q.shape[1]
    q, k = q.repeat_interleave(group, 1), k.repeat_interleave(group, 1)
    s["state"].mul_(torch.exp(s["log_decay"])[:, None, None]).add_(k[..., :, None] * v[..., None, :])
    out = (q[..., None, :] @ s["state"])[..., 0, :]
    return {"out": out.to(s["v"].dtype), "state": s["state"]}


def _plain_attn_prefill(s):
    q, k, v = s["q"].float() * s["scale"], s["k"].float(), s["v"].float()
    hkv, group = k.shape[1], q.shape[1] // k.shape[1]
    outs, at = [], 0
    for n in s["lens"]:
        qs = q[at:at + n].transpose(0, 1).unflatten(0, (hkv, group))                  # [hkv][group][n][d]
        ks, vs = k[at:at + n].transpose(0, 1), v[at:at + n].transpose(0, 1)
        at += n
        t = torch.arange(n, device=q.device)
        p = qs @ ks[:, None].transpose(2, 3)
        p.masked_fill_(t[None, :] > t[:, None], -math.inf)
        if n:
            p.sub_(p.amax(-1, keepdim=True)).exp_()
        out = (p @ vs[:, None]) / p.sum(-1, keepdim=True)
        outs.append(out.flatten(0, 1).transpose(0, 1))
    return torch.cat(outs).to(s["q"].dtype)


def _plain_attn_decode(s):
    rows = torch.arange(s["q"].shape[0], device=s["q"].device)
    lens = s["cache_lens"].long()
    s["k_cache"][rows, lens] = s["k"]
    s["v_cache"][rows, lens] = s["v"]
    hkv = s["k"].shape[1]
    q = (s["q"].float() * s["scale"]).unflatten(1, (hkv, -1))                         # [b][hkv][group][d]
    k, v = s["k_cache"].float().transpose(1, 2), s["v_cache"].float().transpose(1, 2)  # [b][hkv][capacity][d]
    p = q @ k.transpose(2, 3)
    behind = torch.arange(k.shape[2], device=q.device) > lens[:, None]
    p.masked_fill_(behind[:, None, None, :], -math.inf)
    p.sub_(p.amax(-1, keepdim=True)).exp_()
    out = (p @ v) / p.sum(-1, keepdim=True)
    return {"out": out.flatten(1, 2).to(s["q"].dtype), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


_PLAIN = {"linattn_prefill": _plain_linattn_prefill, "linattn_decode": _plain_linattn_decode,
          "attn_prefill": _plain_attn_prefill, "attn_decode": _plain_attn_decode}


# ---------------------------------------------------------------- the package's entry points
def _own_linattn_prefill(s):
    import state_space_model_05_b200 as ssd
    out, final = ssd.ssd_linattn_prefill(s["q"], s["k"], s["v"], s["log_decay"], s["cu_seqlens"], scale=s["scale"],
                                         init_states=s["init"])
    return {"out": out, "final_states": final}


def _own_linattn_decode(s):
    import state_space_model_05_b200 as ssd
    out = ssd.ssd_linattn_decode_step(s["state"], s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"])
    return {"out": out, "state": s["state"]}


def _own_attn_prefill(s):
    import state_space_model_05_b200 as ssd
    return ssd.ssd_attn_prefill(s["q"], s["k"], s["v"], s["cu_seqlens"], scale=s["scale"])


def _own_attn_decode(s):
    import state_space_model_05_b200 as ssd
    out = ssd.ssd_attn_decode_step(s["k_cache"], s["v_cache"], s["cache_lens"], s["q"], s["k"], s["v"],
                                   scale=s["scale"])
    return {"out": out, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


_OWN = {"linattn_prefill": _own_linattn_prefill, "linattn_decode": _own_linattn_decode,
        "attn_prefill": _own_attn_prefill, "attn_decode": _own_attn_decode}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    n, lens = case["seqs"], _lengths(case)
    if case["op"].startswith("linattn"):
        hq, hv, dk, dv = case["heads_qk"], case["heads_v"], case["dk"], case["dv"]
        rows = sum(lens) if case["op"] == "linattn_prefill" else n
        states = n * hv * dk * dv * 4 * (2 if case["op"] == "linattn_decode" or case["init"] else 1)
        # the recurrence: k v^T into the state and q^T S out of it
        return {"bytes": rows * (2 * hq * dk + 2 * hv * dv) * size + states + hv * 4, "flops": rows * hv * 4 * dk * dv}
    hq, hkv, d = case["heads_q"], case["heads_kv"], case["dim"]
    if case["op"] == "attn_prefill":
        return {"bytes": sum(lens) * (2 * hq + 2 * hkv) * d * size,
                "flops": sum(m * (m + 1) // 2 for m in lens) * hq * 4 * d}
    # the cached rows are read, the new ones read and written
    return {"bytes": (sum(lens) * 2 * hkv + n * (2 * hq + 4 * hkv)) * d * size,
            "flops": sum(m + 1 for m in lens) * hq * 4 * d}


# ---------------------------------------------------------------- 64 bits, from the definitions
def exact(case, seed):
    s = _inputs(case, seed)
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    if case["op"].startswith("linattn"):
        # the recurrence itself, token by token, all sequences side by side
        decay, group = torch.exp(s["log_decay"].double())[:, None, None], v.shape[1] // q.shape[1]
        head = torch.arange(v.shape[1], device=q.device) // group
        one = case["op"] == "linattn_decode"
        lens = [1] * case["seqs"] if one else s["lens"]
        start = s["state"] if one else s["init"]
        S = (torch.zeros((len(lens), v.shape[1], q.shape[2], v.shape[2]), dtype=torch.float64, device=q.device)
             if start is None else start.double())
        out = torch.empty_like(v)
        n = torch.tensor(lens, device=q.device)
        first = n.cumsum(0) - n
        order = sorted(range(len(lens)), key=lambda i: -lens[i])
        order_t = torch.tensor(order, device=q.device)
        S, first = S[order_t], first[order_t]
        live = len(lens)
        for t in range(max(lens)):
            while lens[order[live - 1]] <= t:
                live -= 1
            r = first[:live] + t
            S[:live] = decay * S[:live] + k[r][:, head, :, None] * v[r][:, :, None, :]
            out[r] = torch.einsum("bhk,bhkd->bhd", q[r][:, head], S[:live]) * s["scale"]
        back = torch.empty_like(S)
        back[order_t] = S
        return {"out": out, "state" if one else "final_states": back}
    group = q.shape[1] // k.shape[1]
    if case["op"] == "attn_prefill":
        out, at = torch.empty_like(q), 0
        for n in s["lens"]:
            rows = slice(at, at + n)
            at += n
            for h in range(q.shape[1]):
                a = torch.softmax(torch.full((n, n), -math.inf, dtype=torch.float64, device=q.device).triu_(1)
                                  + s["scale"] * (q[rows, h] @ k[rows, h // group].T), -1)
                out[rows, h] = a @ v[rows, h // group]
        return out
    out = torch.empty_like(q)
    for b, n in enumerate(s["lens"]):
        s["k_cache"][b, n], s["v_cache"][b, n] = s["k"][b], s["v"][b]
        for h in range(q.shape[1]):
            a = torch.softmax(s["scale"] * (s["k_cache"][b, :n + 1, h // group].double() @ q[b, h]), 0)
            out[b, h] = a @ s["v_cache"][b, :n + 1, h // group].double()
    return {"out": out, "k_cache": None, "v_cache": None}
