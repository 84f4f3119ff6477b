"""Plain 64-bit forms of the calls on new tokens (norm + rotation, paged append, chunk attention)
and the error bounds the GPU tests hold the kernels to.  numpy only, on the host; sequences and
heads are looped over, and nothing is shared with the kernels."""
from __future__ import annotations

import numpy as np
import torch

PAGE, D = 64, 128
U32 = 2.0 ** -24  # half a step of fp32
BF16 = 2.0 ** -8  # half a step of bf16


def batch(qlens, ctx):
    """(cu_seqlens, ctx_lens) as int32 arrays."""
    return (np.concatenate([[0], np.cumsum(qlens)]).astype(np.int32), np.asarray(ctx, np.int32))


def positions(qlens, ctx):
    return np.concatenate([np.arange(c, c + n) for n, c in zip(qlens, ctx)] + [np.zeros(0)]).astype(np.int64)


def pages_for(qlens, ctx, rng, spare=2, extra_cols=0):
    """(page_table, n_phys): each sequence's pages at shuffled slots, -1 behind them."""
    n = [(c + q + PAGE - 1) // PAGE for q, c in zip(qlens, ctx)]
    n_phys = sum(n) + spare
    perm = rng.permutation(n_phys).astype(np.int32)
    table = np.full((len(n), max(max(n), 1) + extra_cols), -1, np.int32)
    at = 0
    for b, k in enumerate(n):
        table[b, :k] = perm[at:at + k]
        at += k
    return table, n_phys


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def norm_rope(x, pos, weight=None, eps=1e-6, rot=0, base=10000.0, interleaved=False):
    """x [T, H, 128] f64 -> (y, bound): the exact result and how far an fp32 evaluation may be off
    before its final rounding.  Each of the two factors of a term passes a handful of fp32 roundings
    (the norm's 16-term sums and three adds, its square root and products; the table's and the
    rotation's own): 32 half steps cover them, relative to the terms, not to their difference."""
    y = x.copy()
    if weight is not None:
        y = y / np.sqrt((y ** 2).mean(-1, keepdims=True) + eps) * weight
    b = np.abs(y)
    if rot:
        a = pos[:, None] * base ** (-np.arange(0, rot, 2) / rot)
        c, s = np.cos(a)[:, None], np.sin(a)[:, None]
        i = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
        j = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
        u, v = y[..., i].copy(), y[..., j].copy()
        y[..., i], y[..., j] = u * c - v * s, u * s + v * c
        b[..., i] = b[..., j] = np.abs(u) + np.abs(v)
    return y, 32 * U32 * b


def assert_bf16(got: torch.Tensor, ref, bound, what=""):
    """A value within `bound` of ref, then rounded to bf16 (half a step of the value it rounds)."""
    g = f64(got)
    tol = bound + BF16 * (np.abs(ref) + bound) + 2.0 ** -134
    bad = ~(np.abs(g - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(g - ref) / tol):.3g} of the bound"


def e4m3_values() -> np.ndarray:
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = np.nan if (c & 127) == 127 else (-x if c >= 128 else x)
    return v


VALUES = e4m3_values()


def assert_e4m3(codes, ref, bound, what=""):
    """A value within `bound` of ref (clamped to the format's range), rounded to E4M3: half a step
    is 2^-4 of a normal value and 2^-10 below 2^-6."""
    g, r = VALUES[codes], np.clip(ref, -448, 448)
    tol = bound + np.maximum(2.0 ** -4 * (np.abs(r) + bound), 2.0 ** -10)
    bad = ~(np.abs(g - r) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off"


def attn(Q, K_pages, V_pages, table, qlens, ctx, k_scale, v_scale, sm_scale, window=0):
    """Q [T, Hq, 128] f64, pages uint8 -> (O, lse, bound_O, bound_lse) in 64 bits.

    Bounds before the output's rounding.  Scores: products of the tensor cores summed in fp32, off
    by at most 2^-20 of sum |q k|; that and the exponential (2^-21) move each weight by e relative,
    and the softmax by 2 e.  Weights enter P V rounded to f16 (half a step 2^-11; below 2^-14 an
    absolute 2^-25 of a row whose largest weight is at least 1; with few rows the largest is at least
    2^-4, and the errors of its small weights, of either sign, stay inside the first term), summed in
    fp32."""
    T, Hq, _ = Q.shape
    Hkv = K_pages.shape[1]
    G = Hq // Hkv
    O, lse = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    bO, bl = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    at = 0
    for b, (n, c) in enumerate(zip(qlens, ctx)):
        L = c + n
        pg = table[b, :(L + PAGE - 1) // PAGE]
        for h in range(Hkv if n else 0):
            lo = max(0, c - window + 1) // PAGE * PAGE if window else 0
            p2 = pg[lo // PAGE:]
            k = VALUES[K_pages[p2, h]].reshape(-1, D)[:L - lo] * k_scale
            v = VALUES[V_pages[p2, h]].reshape(-1, D)[:L - lo] * v_scale
            i = np.arange(c, L)[:, None]
            j = np.arange(lo, L)
            seen = j <= i
            if window:
                seen = seen & (j > i - window)
            # what no token of the chunk sees may hold anything
            any_seen = seen.any(0)
            k, v = np.where(any_seen[:, None], k, 0.0), np.where(any_seen[:, None], v, 0.0)
            for g in range(G):
                q = Q[at:at + n, h * G + g]
                s = np.where(seen, q @ k.T * sm_scale, -np.inf)
                mag = np.where(seen, np.abs(q) @ np.abs(k).T * sm_scale, 0).max(-1)
                m = s.max(-1, keepdims=True)
                p = np.exp(s - m)
                l = p.sum(-1, keepdims=True)
                w = p / l
                O[at:at + n, h * G + g] = w @ v
                lse[at:at + n, h * G + g] = (m + np.log(l))[:, 0]
                e = 2.0 ** -20 * mag + 2.0 ** -21
                A = w @ np.abs(v)
                nk = seen.sum(-1)[:, None]
                bO[at:at + n, h * G + g] = ((2.0 ** -11 + 2 * e[:, None] + 2.0 ** -18) * A
                                            + nk * 2.0 ** -25 * np.abs(v).max())
                bl[at:at + n, h * G + g] = e + 2.0 ** -20 + 2.0 ** -22 * np.abs(lse[at:at + n, h * G + g])
        at += n
    return O, lse, bO, bl
