"""Plain fp64 forms of the packed mixers (linear attention with a decay per head, causal softmax
attention) and the error that the kernels' own roundings allow, element by element.

A rounding to bf16 is off by at most 2^-8 of the value, one to fp32 by at most 2^-24.  The kernels
round, besides the output itself:

* softmax attention, bf16: the probabilities p (their sum is taken before), so the output may move by
  2^-8 sum p |v| / sum p;
* linear attention, bf16: the masked, decayed scores P of a 128-token block and the carried state's
  operand image, so by 2^-8 (sum |P| |v| + g^(t+1) sum |q| |S|), S being the state at the block's start;
* everything else in fp32: a score of `dim` products by (dim + 2) 2^-24 sum |q| |k|, a sum of n terms
  by n 2^-24 of the terms' absolute sum, an exponential by 2^-20 of itself (its argument's rounding
  included).
"""
from __future__ import annotations

import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
F32 = 2.0 ** -24
BLOCK = 128                                        # tokens per block of the tensor-core path


def offsets(lens):
    return [int(x) for x in np.concatenate([[0], np.cumsum(lens)])]


def cu(lens, device="cuda"):
    return torch.tensor(offsets(lens), dtype=torch.int32, device=device)


def linattn(q, k, v, log_decay, lens, scale, init=None):
    """out, final states, and the tolerance of each, in fp64 on the CPU."""
    dtype = q.dtype
    half = HALF[dtype]
    q, k, v, ld = (x.detach().cpu().double() for x in (q, k, v, log_decay))
    hv, dk, dv = v.shape[1], q.shape[2], v.shape[2]
    head = torch.arange(hv) // (hv // q.shape[1])
    out, tol = torch.zeros_like(v), torch.zeros_like(v)
    finals, ftol = [], []
    # g^n, 1 at n = 0 also where log_decay is -inf
    power = lambda n: torch.where(n == 0, torch.ones((), dtype=torch.float64),  # noqa: E731
                                  torch.exp(ld.reshape(hv, *[1] * n.dim()) * n.clamp_min(1)))
    for i, n in enumerate(lens):
        at = offsets(lens)[i]
        S = torch.zeros(hv, dk, dv, dtype=torch.float64) if init is None else init[i].detach().cpu().double().clone()
        A = S.abs()                                                    # the same recurrence on absolute values
        for b in range(0, n, BLOCK):
            m = min(BLOCK, n - b)
            rows = slice(at + b, at + b + m)
            qb, kb, vb = q[rows][:, head].transpose(0, 1), k[rows][:, head].transpose(0, 1), v[rows].transpose(0, 1)
            t = torch.arange(m)
            gap = t[:, None] - t[None, :]
            w = torch.where(gap >= 0, power(gap.clamp_min(0)), torch.zeros((), dtype=torch.float64))
            P = w * (qb @ kb.transpose(1, 2))
            g = power(t + 1)[:, :, None]
            o = P @ vb + g * (qb @ S)
            moved = P.abs() @ vb.abs() + g * (qb.abs() @ S.abs())
            sums = (w * (qb.abs() @ kb.abs().transpose(1, 2))) @ vb.abs() + g * (qb.abs() @ A)
            inner = half if dtype == torch.bfloat16 else 0.0
            out[rows] = scale * o.transpose(0, 1)
            tol[rows] = abs(scale) * (half * o.abs() + inner * (1 + half) * moved
                                      + ((dk + m + 16) * F32 + 2.0 ** -20) * sums).transpose(0, 1)
            to_end = power(m - 1 - t)[:, None, :]
            whole = power(torch.tensor(m))[:, None, None]
            S = whole * S + (kb.transpose(1, 2) * to_end) @ vb
            A = whole * A + (kb.abs().transpose(1, 2) * to_end) @ vb.abs()
        finals.append(S)
        ftol.append(((min(n, 512) + 16) * F32 + 2.0 ** -19) * A)
    return out, torch.stack(finals), tol + 1e-30, torch.stack(ftol) + 1e-30


def linattn_step(state, q, k, v, log_decay, scale):
    """out, new state and the tolerance of each for one token."""
    half = HALF[q.dtype]
    S, q, k, v, ld = (x.detach().cpu().double() for x in (state, q, k, v, log_decay))
    hv, dk = v.shape[1], q.shape[2]
    head = torch.arange(hv) // (hv // q.shape[1])
    q, k = q[:, head], k[:, head]
    kv = k[..., :, None] * v[..., None, :]
    old = torch.exp(ld)[:, None, None] * S
    new = old + kv
    out = scale * torch.einsum("bhk,bhkd->bhd", q, new)
    size = abs(scale) * torch.einsum("bhk,bhkd->bhd", q.abs(), old.abs() + kv.abs())
    return out, new, half * out.abs() + (dk + 16) * F32 * size + 1e-30, 2.0 ** -21 * (old.abs() + kv.abs()) + 1e-30


def attend(q, k, v, scale, visible):
    """Softmax attention of rows q [n][d] over keys k, v [m][d] with a visible [n][m] mask: output and
    its tolerance.  Keys that a row does not see play no part, whatever they hold."""
    half = HALF[q.dtype]
    q, k, v = (x.detach().cpu().double() for x in (q, k, v))
    out, tol = torch.zeros(q.shape[0], v.shape[1], dtype=torch.float64), torch.zeros(q.shape[0], v.shape[1], dtype=torch.float64)
    s = scale * (q @ k.T)
    size = abs(scale) * (q.abs() @ k.abs().T)
    s = torch.where(visible, s, torch.full((), -torch.inf, dtype=torch.float64))
    p = torch.softmax(s, 1)
    p = torch.where(visible, p, torch.zeros((), dtype=torch.float64))
    seen = visible.any(0)                                # a key that no row sees may hold anything
    p, k, v = p[:, seen], k[seen], v[seen]
    out = p @ v
    absv = p @ v.abs()
    n = int(seen.sum())
    off = (q.shape[1] + 4) * F32 * torch.where(visible, size, torch.zeros((), dtype=torch.float64)).amax(1, keepdim=True)
    inner = half if half > F32 else 0.0
    tol = half * out.abs() + (inner * (1 + half) + 2 * off + (n + 16) * F32 + 2.0 ** -19) * absv + 1e-30
    return out, tol


def attn(q, k, v, lens, scale):
    """Causal attention over packed sequences: output and its tolerance."""
    group = q.shape[1] // k.shape[1]
    out, tol = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    for i, n in enumerate(lens):
        rows = slice(offsets(lens)[i], offsets(lens)[i] + n)
        if n == 0:
            continue
        for h in range(q.shape[1]):
            out[rows, h], tol[rows, h] = attend(q[rows, h], k[rows, h // group], v[rows, h // group], scale,
                                                torch.ones(n, n, dtype=torch.bool).tril())
    return out, tol


def attn_step(k_cache, v_cache, lens, q, k, v, scale):
    """One token per sequence against its cache (the caches as they were before the step)."""
    group = q.shape[1] // k.shape[1]
    out, tol = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    for b, n in enumerate(lens):
        if n < 0:
            continue
        for h in range(q.shape[1]):
            kk = torch.cat([k_cache[b, :n, h // group], k[b, h // group][None]])
            vv = torch.cat([v_cache[b, :n, h // group], v[b, h // group][None]])
            o, t = attend(q[b, h][None], kk, vv, scale, torch.ones(1, n + 1, dtype=torch.bool))
            out[b, h], tol[b, h] = o[0], t[0]
    return out, tol


def assert_within(got, want, tol, what):
    d = (got.detach().cpu().double() - want).abs()
    worst = float((d / tol).max()) if d.numel() else 0.0
    assert not torch.isnan(d).any(), f"{what}: NaN"
    assert worst <= 1.0, f"{what}: {worst:.3f} of the tolerance, max error {float(d.max()):.3e}"
    return worst


def randn(*shape, seed, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).cuda()
