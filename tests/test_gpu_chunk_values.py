"""pw_chunk_attn where the values are what can go wrong: NaN marks of short tiles, equal bits of repeated
calls on ragged batches, queries with one large element, small weights that count by their number alone,
large scores (tokens_ref.py holds the plain 64-bit forms)."""
import numpy as np
import pytest
import torch

from dynamic_sparse_attention_pw_b200 import api

import parity
import tokens_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
S = 2.0 ** -6  # cache scale


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).to(DEV)


def _codes(rng, shape):
    x = torch.from_numpy(np.clip(rng.standard_normal(shape) * 64.0, -448, 448))
    return x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def _dev(x):
    return torch.from_numpy(x).to(DEV)


@pytest.mark.parametrize("B,q,ctx,Hq,Hkv,max_q", [
    (500, 16, 0, 8, 1, 16),     # one half of a large tile, one block
    (500, 16, 120, 8, 1, 16),   # two blocks
    (300, 30, 0, 8, 1, 30),     # both halves
    (700, 4, 0, 8, 1, 4),       # the small tiles
])
def test_nan_marks_of_many_short_tiles(B, q, ctx, Hq, Hkv, max_q):
    """Every CTA works on many short tiles whose first block holds NaN values that some rows see: those
    rows are NaN and no other, in every one of several calls."""
    rng = np.random.default_rng(1)
    qlens, ctxs = [q] * B, [ctx] * B
    cu, cl = ref.batch(qlens, ctxs)
    table, n_phys = ref.pages_for(qlens, ctxs, rng)
    Kp, Vp = _codes(rng, (n_phys, Hkv, 64, 128)), _codes(rng, (n_phys, Hkv, 64, 128))
    first = rng.integers(1, q, B)  # first token of each sequence that sees a NaN
    first[::5] = q                 # none does
    for b in range(B):
        if first[b] < q:
            p = ctx + first[b]
            Vp[table[b, p // 64], :, p % 64, rng.integers(0, 128)] = 0x7F
    # rows far apart, so that the queries of a tile arrive at different times
    Q = torch.from_numpy(rng.standard_normal((cu[-1], 16 * Hq, 128), np.float32)).to(torch.bfloat16).to(DEV)[:, ::16]
    sees = torch.from_numpy((np.arange(q)[None] >= first[:, None]).reshape(-1)).to(DEV)
    args = (Q, _dev(Kp), _dev(Vp), _i32(table), _i32(cu), _i32(cl))
    clean = _dev(np.where((Vp & 0x7F) == 0x7F, 0, Vp).astype(np.uint8))
    kw = dict(max_q_len=max_q, k_scale=S, v_scale=S, workspace=api.chunk_workspace(B, int(cu[-1]), Hq, Hkv, max_q_len=max_q, device=DEV))
    want = api.pw_chunk_attn(args[0], args[1], clean, *args[3:], **kw)
    for i in range(10):
        got = api.pw_chunk_attn(*args, **kw)
        torch.cuda.synchronize()
        assert bool(got[sees].isnan().any(-1).all()), i
        assert torch.equal(got[~sees], want[~sees]), i


@pytest.mark.parametrize("qlens,ctx,Hq,Hkv,window", [
    ([1] * 9, [40 * 5 ** (i % 6) for i in range(9)], 16, 2, 0),       # tiles of 16 rows
    ([5, 1, 4, 0, 5], [3000, 9000, 64, 10, 700], 8, 2, 0),             # 24
    ([7, 8, 1], [5000, 100, 20000], 8, 2, 0),                          # 32
    ([200, 1, 0, 333, 70], [4000, 9000, 5, 0, 1500], 8, 2, 0),         # large ones
    ([200, 1, 0, 333, 70], [4000, 9000, 5, 0, 1500], 8, 2, 600),
])
def test_ragged_batches_give_the_same_bits_again(qlens, ctx, Hq, Hkv, window):
    rng = np.random.default_rng(2)
    cu, cl = ref.batch(qlens, ctx)
    table, n_phys = ref.pages_for(qlens, ctx, rng)
    Q = torch.from_numpy(rng.standard_normal((cu[-1], Hq, 128))).to(torch.bfloat16).to(DEV)
    args = (Q, _dev(_codes(rng, (n_phys, Hkv, 64, 128))), _dev(_codes(rng, (n_phys, Hkv, 64, 128))), _i32(table), _i32(cu), _i32(cl))
    runs = []
    for _ in range(8):
        lse = torch.empty(Q.shape[:2], device=DEV)
        runs.append((api.pw_chunk_attn(*args, max_q_len=max(qlens), k_scale=S, v_scale=S, window=window, lse=lse), lse))
    torch.cuda.synchronize()
    for O, lse in runs[1:]:
        assert torch.equal(O, runs[0][0]) and torch.equal(lse, runs[0][1])


@pytest.mark.parametrize("qlens,ctx", [([1], [700]), ([5, 2], [300, 64]), ([8], [300]), ([150, 40], [200, 0])])
@pytest.mark.parametrize("octaves", [10, 12, 13, 14, 18])
def test_queries_with_one_large_element(qlens, ctx, octaves):
    """One element of every query lies octaves above the others, in a dimension in which the keys are next to
    nothing: the scores are what the small elements make of them.  Elements within 2^13 of the largest enter
    exactly, smaller ones are off by at most 2^-21 of the largest."""
    rng = np.random.default_rng(octaves)
    Hq, Hkv, big = 8, 2, 37
    cu, cl = ref.batch(qlens, ctx)
    table, n_phys = ref.pages_for(qlens, ctx, rng)
    Kp, Vp = _codes(rng, (n_phys, Hkv, 64, 128)), _codes(rng, (n_phys, Hkv, 64, 128))
    Kp[..., big] = rng.integers(0, 2, Kp.shape[:-1])  # zero, or the smallest code
    q = rng.uniform(1.0, 2.0, (cu[-1], Hq, 128)) * rng.choice([-1.0, 1.0], (cu[-1], Hq, 128))
    q[..., big] = 2.0 ** octaves
    Q = torch.from_numpy(q).to(torch.bfloat16).to(DEV)
    lse = torch.empty(Q.shape[:2], device=DEV)
    O = api.pw_chunk_attn(Q, _dev(Kp), _dev(Vp), _i32(table), _i32(cu), _i32(cl), max_q_len=max(qlens), k_scale=S, v_scale=S, lse=lse)
    torch.cuda.synchronize()
    x = ref.f64(Q)
    want, wl, bO, bl = ref.attn(x, Kp, Vp, table, qlens, ctx, S, S, 128 ** -0.5)
    # what the small elements' error moves a score by, at most: each times the largest key in its dimension
    k_most, v_most = np.nanmax(np.abs(ref.VALUES[Kp]), (0, 1, 2)) * S, np.nanmax(np.abs(ref.VALUES[Vp])) * S
    top = np.abs(x).max(-1, keepdims=True)
    e = (np.where(np.abs(x) < top * 2.0 ** -13, top * 2.0 ** -21, 0.0) * k_most).sum(-1) * 128 ** -0.5
    # a score's error moves the log-sum-exp by as much at most, and the weights by twice that
    ref.assert_bf16(O, want, bO + 2 * e[..., None] * v_most, "O")
    assert (np.abs(ref.f64(lse) - wl) <= bl + e).all(), f"lse off by {np.abs(ref.f64(lse) - wl).max():.3g}"


@pytest.mark.parametrize("q,B", [(1, 592), (2, 300), (32, 148)])
def test_one_key_above_many(q, B):
    """64k or 128k keys behind one that outweighs each of them by 2^17 to 2^24 and whose value is zero: the others'
    small weights, which only their number makes count, are the output."""
    rng = np.random.default_rng(3)
    n, Hq = 131072, 8
    if q > 16:
        n = 65536
    pages = n // 64
    Kp, Vp = _codes(rng, (pages, 1, 64, 128)), _codes(rng, (pages, 1, 64, 128))
    Vp[:] = 0x38 + Vp % 4  # 1 to 1.375, so that nothing cancels
    Kp[..., 0] = 0
    Kp[0, 0, 0] = 0
    Kp[0, 0, 0, 0] = 0x78  # 256
    Vp[0, 0, 0] = 0
    gap = np.linspace(17, 24, Hq)  # octaves
    x = np.where(np.arange(128) == 0, (gap * np.log(2) / 256)[:, None], 0.5 / (64 * 127 ** 0.5))[None] * np.ones((q, 1, 1))
    Q = torch.from_numpy(x).to(torch.bfloat16)
    table = np.broadcast_to(np.arange(pages, dtype=np.int32), (B, pages))  # all sequences read the same pages
    cu, cl = ref.batch([q] * B, [n - q] * B)
    O = api.pw_chunk_attn(Q.repeat(B, 1, 1).to(DEV), _dev(Kp), _dev(Vp), _i32(table), _i32(cu), _i32(cl), max_q_len=q, sm_scale=1.0)
    torch.cuda.synchronize()
    want, _, bO, _ = ref.attn(ref.f64(Q), Kp, Vp, table[:1], [q], [n - q], 1.0, 1.0, 1.0)
    # A weight below f16's normal range is off by at most half of its smallest step, 2^-25, and a row's largest
    # weight is at least 1/4 when it rounds: 2^-23 of it a key, of which 2^-25 is in the bound already.
    bO = bO + n * 3 * 2.0 ** -25 * 1.375
    for i in range(0, B, 37):
        ref.assert_bf16(O[i * q:(i + 1) * q], want, bO, f"sequence {i}")


@pytest.mark.parametrize("qlens,ctx", [([1], [900]), ([5], [900]), ([200], [900])])
def test_scores_up_to_the_stated_limit(qlens, ctx):
    """Scores of up to 2^23 (base 2): a row is little but its largest key, and finite.  The scores themselves are
    off by at most 2^-20 of sum |q k|, and so is the log-sum-exp."""
    rng = np.random.default_rng(4)
    cu, cl = ref.batch(qlens, ctx)
    table, n_phys = ref.pages_for(qlens, ctx, rng)
    Kp, Vp = _codes(rng, (n_phys, 2, 64, 128)), _codes(rng, (n_phys, 2, 64, 128))
    Q = torch.from_numpy(rng.standard_normal((cu[-1], 8, 128)) * 1500).to(torch.bfloat16).to(DEV)
    lse = torch.empty(Q.shape[:2], device=DEV)
    O = api.pw_chunk_attn(Q, _dev(Kp), _dev(Vp), _i32(table), _i32(cu), _i32(cl), max_q_len=max(qlens), sm_scale=1.0, v_scale=S, lse=lse)
    torch.cuda.synchronize()
    want, wl, _, bl = ref.attn(ref.f64(Q), Kp, Vp, table, qlens, ctx, 1.0, S, 1.0)
    assert 2.0 ** 22 < np.abs(wl).max() * 1.4427 < 2.0 ** 24
    assert (np.abs(ref.f64(lse) - wl) <= bl).all()
    top = np.abs(ref.VALUES[Vp]).max() * S
    assert bool((O.abs() <= top * (1 + 2.0 ** -8) * (1 + 2.0 ** -10)).all())  # an average of values; weights and output are rounded


@pytest.mark.parametrize("qlens,ctx,Hq,Hkv", [
    ([1] * 24, [90 * i for i in range(24)], 64, 8),        # tiles of 16 rows
    ([5] * 6, [100, 2000, 700, 0, 5000, 64], 32, 8),       # 24
    ([4] * 6, [100, 2000, 700, 0, 5000, 64], 64, 8),       # 32
    ([300, 40, 1], [2000, 0, 900], 32, 8),                 # large ones
])
def test_outputs_within_the_bar_of_the_sparse_attention(qlens, ctx, Hq, Hkv):
    """Max-abs 2e-2 and rel-L2 1e-3 of the 64-bit result rounded to bf16: the bar that pw_attn is held to."""
    rng = np.random.default_rng(5)
    cu, cl = ref.batch(qlens, ctx)
    table, n_phys = ref.pages_for(qlens, ctx, rng)
    Kp, Vp = _codes(rng, (n_phys, Hkv, 64, 128)), _codes(rng, (n_phys, Hkv, 64, 128))
    Q = torch.from_numpy(rng.standard_normal((cu[-1], Hq, 128)) * np.linspace(0.5, 3.0, Hq)[:, None]).to(torch.bfloat16).to(DEV)
    O = api.pw_chunk_attn(Q, _dev(Kp), _dev(Vp), _i32(table), _i32(cu), _i32(cl), max_q_len=max(qlens), k_scale=S, v_scale=S)
    torch.cuda.synchronize()
    want = ref.attn(ref.f64(Q), Kp, Vp, table, qlens, ctx, S, S, 128 ** -0.5)[0]
    got = O.view(torch.int16).cpu().numpy().view(np.uint16)
    parity.compare_rows(got.reshape(-1, 128), want.reshape(-1, 128), "pw_chunk_attn")
