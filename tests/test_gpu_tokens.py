"""pw_qk_norm_rope, pw_append, pw_chunk_attn and extend on the GPU against plain 64-bit forms
(tokens_ref.py), at the sizes, strides and masks where they can go wrong."""
import numpy as np
import pytest
import torch

from dynamic_sparse_attention_pw_b200 import _lib, api

import tokens_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).to(DEV)


def _bf16(rng, *shape, scale=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * scale).to(torch.bfloat16).to(DEV)


def _codes(rng, shape, scale=64.0):
    x = torch.from_numpy(np.clip(rng.standard_normal(shape) * scale, -448, 448))
    return x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def _ok(status):
    torch.cuda.synchronize()
    assert int(status.item()) == 0


# ---------------------------------------------------------------------------------------
# pw_qk_norm_rope
# ---------------------------------------------------------------------------------------

NORM_CASES = [
    # qlens, ctx, Hq, Hk, rot, interleaved, weight per head, norm
    ([1], [0], 1, 1, 128, False, False, True),
    ([1], [8191], 32, 8, 128, False, False, True),
    ([5, 0, 1, 130], [0, 3, 70000, 17], 6, 2, 128, True, True, True),
    ([33, 64], [10, 0], 64, 8, 64, False, False, True),
    ([7], [100], 3, 5, 16, True, True, True),
    ([40], [1], 5, 1, 48, False, True, False),
    ([9, 2], [2, 2], 8, 2, 0, False, False, True),
    ([1] * 70, list(range(0, 7000, 100)), 8, 2, 128, False, False, True),
    ([0, 1] * 600 + [0], [3] * 1201, 2, 1, 96, True, False, False),
]


@pytest.mark.parametrize("qlens,ctx,Hq,Hk,rot,inter,per_head,norm", NORM_CASES)
def test_norm_rope(qlens, ctx, Hq, Hk, rot, inter, per_head, norm):
    rng = np.random.default_rng(len(qlens) + Hq)
    cu, cl = ref.batch(qlens, ctx)
    T = int(cu[-1])
    packed = _bf16(rng, T, Hq + 2 * Hk, 128, scale=2.0)  # rows of a packed projection
    Q, K = packed[:, :Hq], packed[:, Hq:Hq + Hk]
    wq = _bf16(rng, *((Hq, 128) if per_head else (128,))) if norm else None
    wk = _bf16(rng, *((Hk, 128) if per_head else (128,))) if norm else None
    table = api.rope_table(70200, rot, device=DEV) if rot else None
    status = api.new_status(DEV)
    Qo, Ko = api.pw_qk_norm_rope(Q, K, _i32(cu), _i32(cl), q_weight=wq, k_weight=wk, eps=1e-5, rope=table,
                                 interleaved=inter, status=status)
    _ok(status)
    pos = ref.positions(qlens, ctx)
    for x, w, y in ((Q, wq, Qo), (K, wk, Ko)):
        want, bound = ref.norm_rope(ref.f64(x), pos, None if w is None else ref.f64(w), 1e-5, rot, interleaved=inter)
        ref.assert_bf16(y, want, bound, "norm + rotation")


def test_norm_rope_in_place_and_one_side_only():
    rng = np.random.default_rng(3)
    packed = _bf16(rng, 50, 12, 128)
    keep = packed.clone()
    table, cu = api.rope_table(64, device=DEV), _i32([0, 50])
    w = _bf16(rng, 128)
    want, _ = api.pw_qk_norm_rope(packed[:, :8], None, cu, q_weight=w, rope=table)
    Q = packed[:, :8]
    got, none = api.pw_qk_norm_rope(Q, None, cu, q_weight=w, rope=table, Q_out=Q)
    assert none is None and got is Q
    torch.cuda.synchronize()
    assert torch.equal(packed[:, :8], want) and torch.equal(packed[:, 8:], keep[:, 8:])
    _, k = api.pw_qk_norm_rope(None, keep[:, 8:10], cu, rope=table)
    ref_k, bound = ref.norm_rope(ref.f64(keep[:, 8:10]), np.arange(50), rot=128)
    ref.assert_bf16(k, ref_k, bound)


def test_norm_rope_heads_outermost_and_padded_rows_stay():
    rng = np.random.default_rng(4)
    x = _bf16(rng, 4, 20, 128)  # [H, T, 128]
    out = torch.full((4, 20, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    status = api.new_status(DEV)
    table = api.rope_table(40, device=DEV)
    api.pw_qk_norm_rope(x.transpose(0, 1), None, _i32([0, 6, 13]), _i32([1, 20]), rope=table,
                        Q_out=out.transpose(0, 1), status=status)
    _ok(status)
    want, bound = ref.norm_rope(ref.f64(x.transpose(0, 1))[:13], ref.positions([6, 7], [1, 20]), rot=128)
    ref.assert_bf16(out.transpose(0, 1)[:13], want, bound)
    assert bool((out[:, 13:] == 7.0).all())


def test_norm_rope_special_values_stay_in_their_row():
    x = torch.zeros(3, 2, 128, dtype=torch.bfloat16, device=DEV)
    x[0, 0, 5], x[0, 1, 7], x[2, 0] = float("nan"), float("inf"), 1.0
    w = torch.ones(128, dtype=torch.bfloat16, device=DEV)
    y, _ = api.pw_qk_norm_rope(x, None, _i32([0, 3]), q_weight=w, rope=api.rope_table(8, device=DEV))
    torch.cuda.synchronize()
    assert bool(y[0, 0].isnan().all()) and bool(y[0, 1].isnan().any())
    assert bool((y[1] == 0).all()) and bool((y[2, 1] == 0).all()) and bool(y[2, 0].isfinite().all())


def test_norm_rope_position_outside_the_table_is_reported():
    rng = np.random.default_rng(5)
    x = _bf16(rng, 4, 2, 128)
    status = api.new_status(DEV)
    y, _ = api.pw_qk_norm_rope(x, None, _i32([0, 4]), _i32([6]), rope=api.rope_table(8, device=DEV), status=status)
    torch.cuda.synchronize()
    with pytest.raises(_lib.PwError):
        api.check_status(status)
    want, bound = ref.norm_rope(ref.f64(x[:2]), np.array([6, 7]), rot=128)
    ref.assert_bf16(y[:2], want, bound)
    assert torch.equal(y[2:], x[2:])  # not rotated


# ---------------------------------------------------------------------------------------
# pw_append
# ---------------------------------------------------------------------------------------

APPEND_CASES = [
    # qlens, ctx, Hkv, rot, interleaved, norm, k_scale, v_scale
    ([1], [0], 1, 128, False, True, 1.0, 1.0),
    ([1], [63], 8, 128, False, True, 2.0 ** -6, 2.0 ** -6),
    ([1], [64], 8, 64, True, False, 2.0 ** -6, 0.031),
    ([5, 0, 1, 130], [62, 3, 1000, 17], 2, 128, True, True, 0.013, 0.02),
    ([200, 64], [0, 128], 3, 0, False, False, 1.0, 1.0),
    ([1] * 70, list(range(0, 700, 10)), 8, 128, False, True, 2.0 ** -6, 2.0 ** -6),
    ([77], [51], 16, 32, False, True, 2.0 ** -9, 2.0 ** -12),
]


@pytest.mark.parametrize("qlens,ctx,Hkv,rot,inter,norm,ks,vs", APPEND_CASES)
def test_append(qlens, ctx, Hkv, rot, inter, norm, ks, vs):
    rng = np.random.default_rng(len(qlens) + Hkv)
    cu, cl = ref.batch(qlens, ctx)
    T = int(cu[-1])
    packed = _bf16(rng, T + 3, 2 * Hkv + 4, 128)  # three padded rows behind the last sequence
    K, V = packed[:, 4:4 + Hkv], packed[:, 4 + Hkv:]
    w = _bf16(rng, 128) if norm else None
    table, n_phys = ref.pages_for(qlens, ctx, rng, extra_cols=2)
    old = rng.integers(0, 256, (2, n_phys, Hkv, 64, 128)).astype(np.uint8)  # NaN codes among them
    Kp, Vp = torch.from_numpy(old[0]).to(DEV), torch.from_numpy(old[1]).to(DEV)
    status = api.new_status(DEV)
    api.pw_append(K, V, Kp, Vp, _i32(table), _i32(cu), _i32(cl), k_scale=ks, v_scale=vs, k_weight=w, eps=1e-6,
                  rope=api.rope_table(1200, rot, device=DEV) if rot else None, interleaved=inter, status=status)
    _ok(status)
    pos = ref.positions(qlens, ctx)
    seq = np.repeat(np.arange(len(qlens)), qlens)
    phys, slot = table[seq, pos // 64], pos % 64
    k, bound = ref.norm_rope(ref.f64(K[:T]), pos, None if w is None else ref.f64(w), 1e-6, rot, interleaved=inter)
    gk, gv = Kp.cpu().numpy(), Vp.cpu().numpy()
    # the product by the scale's reciprocal adds a few half steps of fp32
    ref.assert_e4m3(gk[phys, :, slot], k / ks, (bound + 4 * ref.U32 * np.abs(k)) / ks, "K")
    v = ref.f64(V[:T])
    ref.assert_e4m3(gv[phys, :, slot], v / vs, 4 * ref.U32 * np.abs(v) / vs, "V")
    if vs in (1.0, 2.0 ** -6):  # exact scales: exact codes
        want = (V[:T].float() / vs).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).cpu().numpy()
        assert np.array_equal(gv[phys, :, slot], want)
    # nothing else was written
    old[0][phys, :, slot], old[1][phys, :, slot] = gk[phys, :, slot], gv[phys, :, slot]
    assert np.array_equal(gk, old[0]) and np.array_equal(gv, old[1])


def test_append_saturates_and_keeps_nan():
    V = torch.zeros(1, 1, 128, dtype=torch.bfloat16, device=DEV)
    V[0, 0, :6] = torch.tensor([1e30, -1e30, float("inf"), -float("inf"), float("nan"), 460.0], device=DEV)
    pages = torch.zeros(2, 1, 1, 64, 128, dtype=torch.uint8, device=DEV)
    api.pw_append(V, V, pages[0], pages[1], _i32([[0]]), _i32([0, 1]), _i32([7]))
    torch.cuda.synchronize()
    for got in ref.VALUES[pages[:, 0, 0, 7].cpu().numpy()]:
        assert got[:4].tolist() == [448, -448, 448, -448] and np.isnan(got[4]) and got[5] == 448 and (got[6:] == 0).all()


@pytest.mark.parametrize("where", ["column", "slot", "negative", "rope"])
def test_append_bad_pages_are_reported_and_skipped(where):
    rng = np.random.default_rng(6)
    K = _bf16(rng, 3, 2, 128)
    pages = torch.zeros(2, 3, 2, 64, 128, dtype=torch.uint8, device=DEV)
    table, ctx = {"column": ([[0, 1]], 126), "slot": ([[0, 1, 3]], 126), "negative": ([[0, 1, -1]], 126),
                  "rope": ([[0, 1, 2]], 126)}[where]
    status = api.new_status(DEV)
    api.pw_append(K, K, pages[0], pages[1], _i32(table), _i32([0, 3]), _i32([ctx]),
                  rope=api.rope_table(128 if where == "rope" else 200, device=DEV), status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == _lib.PW_ERR_INVALID_ARG
    assert bool((pages[1, 1, :, 62:] != 0).any()) and bool((pages[:, [0, 2]] == 0).all())


# ---------------------------------------------------------------------------------------
# pw_chunk_attn
# ---------------------------------------------------------------------------------------

def _attn_inputs(rng, qlens, ctx, Hq, Hkv, pad=0, q_scale=1.0, sharp=True):
    cu, cl = ref.batch(qlens, ctx)
    T = int(cu[-1])
    table, n_phys = ref.pages_for(qlens, ctx, rng, extra_cols=1)
    scale = np.linspace(0.5, 3.0, Hq)[:, None] if sharp else 1.0
    Q = torch.from_numpy(rng.standard_normal((T + pad, Hq, 128)) * scale * q_scale).to(torch.bfloat16).to(DEV)
    Kp, Vp = _codes(rng, (n_phys, Hkv, 64, 128)), _codes(rng, (n_phys, Hkv, 64, 128))
    # slots that hold no key yet, and pages of nobody: any code, NaN among them
    for b, (n, c) in enumerate(zip(qlens, ctx)):
        L = n + c
        if L % 64:
            for P in (Kp, Vp):
                P[table[b, L // 64], :, L % 64:] = rng.integers(0, 256, (Hkv, 64 - L % 64, 128))
                P[table[b, L // 64], :, L % 64:, ::5] = 0x7F
    nobody = np.setdiff1d(np.arange(n_phys), table.ravel())
    Kp[nobody], Vp[nobody] = 0x7F, 0xFF
    return cu, cl, table, Q, Kp, Vp


def _check_attn(qlens, ctx, Hq, Hkv, window=0, max_q_len=None, seed=0, ks=2.0 ** -6, vs=2.0 ** -6, sm=128 ** -0.5,
                pad=0, q_scale=1.0):
    rng = np.random.default_rng(seed)
    cu, cl, table, Q, Kp, Vp = _attn_inputs(rng, qlens, ctx, Hq, Hkv, pad, q_scale)
    T = int(cu[-1])
    O = torch.full((T + pad, Hq, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T + pad, Hq), 7.0, device=DEV)
    status = api.new_status(DEV)
    api.pw_chunk_attn(Q, torch.from_numpy(Kp).to(DEV), torch.from_numpy(Vp).to(DEV), _i32(table), _i32(cu), _i32(cl),
                      max_q_len=max_q_len or max(max(qlens), 1), k_scale=ks, v_scale=vs, sm_scale=sm, window=window,
                      O=O, lse=lse, status=status)
    _ok(status)
    want, wl, bO, bl = ref.attn(ref.f64(Q)[:T], Kp, Vp, table, qlens, ctx, ks, vs, sm, window)
    ref.assert_bf16(O[:T], want, bO, "O")
    err = np.abs(ref.f64(lse)[:T] - wl)
    assert (err <= bl).all(), f"lse: worst {(err / bl).max():.3g} of the bound"
    assert bool((O[T:] == 7.0).all()) and bool((lse[T:] == 7.0).all())


ATTN_CASES = [
    # qlens, ctx, Hq, Hkv, window, max_q_len
    ([1], [0], 1, 1, 0, None),
    ([1], [0], 8, 1, 0, None),
    ([1], [62], 32, 8, 0, None),
    ([1], [63], 64, 8, 0, None),
    ([1], [64], 8, 8, 0, None),
    ([1], [127], 8, 2, 0, None),
    ([1], [128], 8, 2, 0, None),
    ([1], [5000], 8, 1, 0, None),
    ([1, 1, 1], [0, 1000, 4095], 32, 8, 0, None),
    ([1] * 40, [37 * i for i in range(40)], 16, 2, 0, None),
    ([1, 0, 1, 0], [300, 20, 128, 0], 12, 4, 0, None),
    ([5, 2, 8], [700, 0, 131], 8, 2, 0, None),
    ([3], [2000], 64, 2, 0, None),         # 32 heads a group
    ([6, 1, 5, 0], [900, 0, 127, 3], 8, 2, 0, None),  # 24 rows a tile
    ([3, 2], [4000, 64], 14, 2, 200, None),           # 21
    ([1], [700], 17, 1, 0, None),
    ([1, 1], [2500, 1], 50, 2, 0, None),              # 25
    ([2], [500], 33, 1, 0, None),          # an odd number of heads a group
    ([1], [500], 130, 1, 0, None),
    ([16], [0], 8, 1, 0, None),
    ([64], [64], 8, 2, 0, None),
    ([129], [0], 8, 2, 0, None),
    ([100, 1, 0, 300], [0, 777, 5, 1000], 8, 2, 0, None),
    ([257], [3000], 4, 2, 0, None),
    ([40], [1500], 40, 8, 0, None),        # 5 heads a group
    ([700], [0], 1, 1, 0, None),
    ([1], [5000], 8, 2, 1, None),          # windows: only itself, across pages, wider than the context
    ([1], [5000], 8, 2, 100, None),
    ([1, 1], [5000, 3], 8, 2, 4096, None),
    ([300], [900], 8, 2, 64, None),
    ([300, 6], [900, 0], 8, 2, 1, None),
    ([200], [1000], 8, 2, 777, None),
    ([5], [3000], 8, 2, 130, None),
    # a wrong hint changes nothing
    ([70, 1], [100, 900], 8, 2, 0, 1),
    ([1, 2], [100, 900], 8, 2, 0, 4096),
]


@pytest.mark.parametrize("qlens,ctx,Hq,Hkv,window,max_q_len", ATTN_CASES)
def test_chunk_attn(qlens, ctx, Hq, Hkv, window, max_q_len):
    _check_attn(qlens, ctx, Hq, Hkv, window, max_q_len, seed=len(qlens) + Hq + window, pad=2)


@pytest.mark.parametrize("qlens,ctx,max_q", [
    ([1] * 300, [(7 * i) % 190 for i in range(300)], 1),                            # more sequences than are counted at once
    ([1, 0, 0] * 100 + [0] * 40, [(11 * i) % 260 for i in range(340)], 1),
    ([(3 * i) % 41 for i in range(150)], [(13 * i) % 150 for i in range(150)], 40),  # the same with large tiles
    ([0] * 140 + [200], [5] * 141, 200),
])
def test_chunk_attn_many_sequences(qlens, ctx, max_q):
    _check_attn(qlens, ctx, 16 if max_q > 1 else 8, 2, 0, max_q, seed=17, pad=1)


@pytest.mark.parametrize("max_q", [1, 300])
def test_chunk_attn_no_tokens_at_all(max_q):
    rng = np.random.default_rng(18)
    Q, pages = _bf16(rng, 4, 8, 128), torch.zeros(2, 2, 64, 128, dtype=torch.uint8, device=DEV)
    O, lse = torch.full((4, 8, 128), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((4, 8), 7.0, device=DEV)
    status = api.new_status(DEV)
    api.pw_chunk_attn(Q, pages, pages, _i32([[0], [1]]), _i32([0, 0, 0]), _i32([3, 0]), max_q_len=max_q, O=O, lse=lse, status=status)
    _ok(status)
    assert bool((O == 7.0).all()) and bool((lse == 7.0).all())
    none = api.pw_chunk_attn(Q[:0], pages, pages, _i32([[0]]), _i32([0, 0]), max_q_len=max_q, status=status)
    _ok(status)
    assert none.shape == (0, 8, 128)


@pytest.mark.parametrize("qlens,max_q", [([1, 1, 1], 1), ([7], 7), ([180], 180)])
def test_chunk_attn_special_queries_stay_in_their_row(qlens, max_q):
    rng = np.random.default_rng(19)
    ctx = [300] * len(qlens)
    cu, cl, table, Q, Kp, Vp = _attn_inputs(rng, qlens, ctx, 8, 2)
    T = int(cu[-1])
    clean = ref.f64(Q)
    Q[T // 2, 3, 77], Q[T - 1, 4, 0], Q[0, 5, 127] = float("nan"), float("inf"), -float("inf")
    status = api.new_status(DEV)
    lse = torch.empty(T, 8, device=DEV)
    O = api.pw_chunk_attn(Q, torch.from_numpy(Kp).to(DEV), torch.from_numpy(Vp).to(DEV), _i32(table), _i32(cu), _i32(cl), max_q_len=max_q,
                          k_scale=2.0 ** -6, v_scale=2.0 ** -6, lse=lse, status=status)
    _ok(status)
    bad = np.zeros((T, 8), bool)
    bad[T // 2, 3] = bad[T - 1, 4] = bad[0, 5] = True
    assert bool(O[torch.from_numpy(bad).to(DEV)].isnan().all()) and bool(lse[torch.from_numpy(bad).to(DEV)].isnan().all())
    want, wl, bO, bl = ref.attn(clean, Kp, Vp, table, qlens, ctx, 2.0 ** -6, 2.0 ** -6, 128 ** -0.5)
    good = torch.from_numpy(~bad).to(DEV)
    ref.assert_bf16(O[good], want[~bad], bO[~bad])
    assert (np.abs(ref.f64(lse[good]) - wl[~bad]) <= bl[~bad]).all()


@pytest.mark.parametrize("cu,ctx", [([0, 3, 2], [1, 1]), ([0, 9, 4], [1, 1]), ([-1, 2, 4], [1, 1]), ([0, 2, 4], [-5, 1])])
@pytest.mark.parametrize("max_q", [1, 200])
def test_chunk_attn_bad_offsets_are_reported(cu, ctx, max_q):
    """Falling offsets, offsets outside the rows, a negative context: recorded, and nothing outside the
    buffers is touched (the guard rows stay)."""
    rng = np.random.default_rng(25)
    Q, pages = _bf16(rng, 4, 8, 128), torch.zeros(4, 2, 64, 128, dtype=torch.uint8, device=DEV)
    guard = torch.full((6, 8, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    status = api.new_status(DEV)
    api.pw_chunk_attn(Q, pages, pages, _i32([[0, 1], [2, 3]]), _i32(cu), _i32(ctx), max_q_len=max_q, O=guard[1:5], status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == _lib.PW_ERR_INVALID_ARG
    assert bool((guard[0] == 7.0).all()) and bool((guard[5] == 7.0).all())


@pytest.mark.parametrize("qlens", [[1], [200]])
@pytest.mark.parametrize("q_scale,sm", [(1e-20, 128 ** -0.5), (1e-3, 128 ** -0.5), (30.0, 128 ** -0.5), (1.0, 1e-6), (1e4, 1e-5)])
def test_chunk_attn_score_ranges(qlens, q_scale, sm):
    _check_attn(qlens, [900], 8, 2, seed=7, q_scale=q_scale, sm=sm)


@pytest.mark.parametrize("qlens,ctx", [([1], [1000]), ([150], [500])])
def test_chunk_attn_scores_that_rise_and_fall(qlens, ctx):
    """Keys whose scores rise by large steps along the context (the running maximum moves at every
    tile), then fall: late keys add nothing."""
    rng = np.random.default_rng(11)
    cu, cl, table, Q, Kp, Vp = _attn_inputs(rng, qlens, ctx, 8, 2, sharp=False)
    L = qlens[0] + ctx[0]
    Q = torch.ones_like(Q)
    ramp = np.concatenate([np.linspace(-200, 200, 2 * L // 3), np.linspace(200, -200, L - 2 * L // 3)])
    rows = torch.from_numpy(ramp / 4).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    for p in range(L):
        Kp[table[0, p // 64], :, p % 64, :] = rows[p]
    status = api.new_status(DEV)
    lse = torch.empty(Q.shape[:2], device=DEV)
    O = api.pw_chunk_attn(Q, torch.from_numpy(Kp).to(DEV), torch.from_numpy(Vp).to(DEV), _i32(table), _i32(cu), _i32(cl),
                          max_q_len=qlens[0], v_scale=2.0 ** -6, lse=lse, status=status)
    _ok(status)
    want, wl, bO, bl = ref.attn(ref.f64(Q), Kp, Vp, table, qlens, ctx, 1.0, 2.0 ** -6, 128 ** -0.5)
    ref.assert_bf16(O, want, bO)
    assert (np.abs(ref.f64(lse) - wl) <= bl).all()


def test_chunk_attn_strided_queries_and_zero_queries():
    rng = np.random.default_rng(12)
    cu, cl, table, Q, Kp, Vp = _attn_inputs(rng, [3, 40], [100, 30], 8, 2)
    packed = torch.full((43, 12, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    packed[:, 2:10] = Q
    packed[5, 2:10] = 0  # a row of zeros weighs all its keys alike
    K, V = torch.from_numpy(Kp).to(DEV), torch.from_numpy(Vp).to(DEV)
    status = api.new_status(DEV)
    O = api.pw_chunk_attn(packed[:, 2:10], K, V, _i32(table), _i32(cu), _i32(cl), max_q_len=40, k_scale=2.0 ** -6,
                          v_scale=2.0 ** -6, status=status)
    _ok(status)
    want, _, bO, _ = ref.attn(ref.f64(packed[:, 2:10]), Kp, Vp, table, [3, 40], [100, 30], 2.0 ** -6, 2.0 ** -6, 128 ** -0.5)
    ref.assert_bf16(O, want, bO)


@pytest.mark.parametrize("q", [1, 100])
def test_chunk_attn_bad_pages_are_reported(q):
    rng = np.random.default_rng(13)
    for col, entry in ((1, -1), (0, 99)):
        cu, cl, table, Q, Kp, Vp = _attn_inputs(rng, [q], [200], 8, 2)
        table[0, col] = entry
        status = api.new_status(DEV)
        api.pw_chunk_attn(Q, torch.from_numpy(Kp).to(DEV), torch.from_numpy(Vp).to(DEV), _i32(table), _i32(cu), _i32(cl),
                          max_q_len=q, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == _lib.PW_ERR_INVALID_ARG
    # a context that the table's row cannot hold
    cu, cl, table, Q, Kp, Vp = _attn_inputs(rng, [q], [200], 8, 2)
    status = api.new_status(DEV)
    api.pw_chunk_attn(Q, torch.from_numpy(Kp).to(DEV), torch.from_numpy(Vp).to(DEV), _i32(table[:, :2]), _i32(cu), _i32(cl),
                      max_q_len=q, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == _lib.PW_ERR_INVALID_ARG


@pytest.mark.parametrize("q", [1, 130])
def test_chunk_attn_pages_outside_the_window_are_not_touched(q):
    """A sliding window lets a user free the pages behind it: their table entries may be -1."""
    rng = np.random.default_rng(14)
    cu, cl, table, Q, Kp, Vp = _attn_inputs(rng, [q], [1000], 8, 2)
    first = max(0, 1000 - 150 + 1)
    freed = table[0, :first // 64].copy()
    Kp[freed], Vp[freed] = 0x7F, 0x7F
    table[0, :first // 64] = -1
    status = api.new_status(DEV)
    O = api.pw_chunk_attn(Q, torch.from_numpy(Kp).to(DEV), torch.from_numpy(Vp).to(DEV), _i32(table), _i32(cu), _i32(cl),
                          max_q_len=q, k_scale=2.0 ** -6, v_scale=2.0 ** -6, window=150, status=status)
    _ok(status)
    table[0, :first // 64] = freed  # the plain form drops those pages itself
    want, _, bO, _ = ref.attn(ref.f64(Q), Kp, Vp, table, [q], [1000], 2.0 ** -6, 2.0 ** -6, 128 ** -0.5, 150)
    ref.assert_bf16(O, want, bO)


@pytest.mark.parametrize("q,ctx,window,max_q", [(5, 120, 0, 5), (8, 1000, 0, 8), (6, 300, 100, 6), (60, 0, 0, 60), (200, 500, 0, 200),
                                                (150, 400, 90, 150), (70, 100, 0, 1)])
@pytest.mark.parametrize("which", ["keys", "values"])
def test_chunk_attn_nan_reaches_the_rows_that_see_it_alone(q, ctx, window, max_q, which):
    """A NaN in the cache makes the tokens that attend to it NaN, and no other token of the chunk."""
    rng = np.random.default_rng(16)
    cu, cl, table, Q, Kp, Vp = _attn_inputs(rng, [q], [ctx], 8, 2)
    clean = [Kp.copy(), Vp.copy()]
    bad = [ctx + q // 2, ctx + q - 1] + ([max(0, ctx - window + 2)] if window else [])
    for p in bad:
        (Kp if which == "keys" else Vp)[table[0, p // 64], 1, p % 64, 7] = 0xFF
    status = api.new_status(DEV)
    kw = dict(max_q_len=max_q, k_scale=2.0 ** -6, v_scale=2.0 ** -6, window=window, status=status)
    run = lambda K, V: api.pw_chunk_attn(Q, torch.from_numpy(K).to(DEV), torch.from_numpy(V).to(DEV), _i32(table),  # noqa: E731
                                         _i32(cu), _i32(cl), **kw)
    got = run(Kp, Vp)
    _ok(status)
    want, _, bO, _ = ref.attn(ref.f64(Q), *clean, table, [q], [ctx], 2.0 ** -6, 2.0 ** -6, 128 ** -0.5, window)
    pos = ctx + np.arange(q)
    sees = np.zeros(q, bool)
    for p in bad:
        sees |= (p <= pos) & ((window == 0) | (p > pos - window))
    assert sees.any() and not sees.all()
    assert bool(got[torch.from_numpy(sees).to(DEV), 4:, 7].isnan().all())  # kv head 1: query heads 4..7
    ref.assert_bf16(got[:, :4], want[:, :4], bO[:, :4], "the other kv head")
    ref.assert_bf16(got[torch.from_numpy(~sees).to(DEV)], want[~sees], bO[~sees], "rows that do not see it")


def test_chunk_attn_same_bits_every_time_and_any_batch_order():
    rng = np.random.default_rng(15)
    for q in (1, 90):
        cu, cl, table, Q, Kp, Vp = _attn_inputs(rng, [q], [9000], 16, 2)
        K, V = torch.from_numpy(Kp).to(DEV), torch.from_numpy(Vp).to(DEV)
        runs = [api.pw_chunk_attn(Q, K, V, _i32(table), _i32(cu), _i32(cl), max_q_len=q, k_scale=2.0 ** -6) for _ in range(3)]
        torch.cuda.synchronize()
        assert all(torch.equal(runs[0], r) for r in runs[1:])


@pytest.mark.parametrize("change", [
    dict(Q=lambda a: a["Q"].half()), dict(Q=lambda a: a["Q"][..., :64]), dict(Q=lambda a: a["Q"].transpose(1, 2)),
    dict(K_pages=lambda a: a["K_pages"][:1]), dict(K_pages=lambda a: a["K_pages"].cpu()), dict(V_pages=lambda a: a["V_pages"].view(torch.int8)),
    dict(page_table=lambda a: a["page_table"].long()), dict(page_table=lambda a: a["page_table"][:1]),
    dict(cu_seqlens=lambda a: a["cu_seqlens"].long()), dict(ctx_lens=lambda a: a["ctx_lens"][:1]),
    dict(lse=lambda a: torch.empty(4, 7, device=DEV)), dict(O=lambda a: a["Q"][:, :4].clone()), dict(O=lambda a: a["Q"].float()),
    dict(workspace=lambda a: torch.empty(1 << 20, dtype=torch.uint8)), dict(status=lambda a: torch.zeros(1, device=DEV)),
])
def test_chunk_attn_refuses_tensors_that_do_not_fit(change):
    rng = np.random.default_rng(27)
    a = dict(Q=_bf16(rng, 4, 8, 128), K_pages=torch.zeros(2, 2, 64, 128, dtype=torch.uint8, device=DEV),
             V_pages=torch.zeros(2, 2, 64, 128, dtype=torch.uint8, device=DEV), page_table=_i32([[0], [1]]),
             cu_seqlens=_i32([0, 1, 4]), ctx_lens=_i32([0, 5]), max_q_len=3)
    api.pw_chunk_attn(**a)
    with pytest.raises(AssertionError):
        api.pw_chunk_attn(**{**a, **{k: f(a) for k, f in change.items()}})
    torch.cuda.synchronize()


def test_calls_refuse_sizes_on_the_host():
    rng = np.random.default_rng(28)
    Q, pages, cu = _bf16(rng, 2, 7, 128), torch.zeros(2, 2, 64, 128, dtype=torch.uint8, device=DEV), _i32([0, 2])
    with pytest.raises(_lib.PwError):  # 7 query heads over 2
        api.pw_chunk_attn(Q, pages, pages, _i32([[0]]), cu, max_q_len=2)
    with pytest.raises(_lib.PwError):
        api.pw_chunk_attn(Q[:, :6], pages, pages, _i32([[0]]), cu, max_q_len=2, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    with pytest.raises(_lib.PwError):
        api.pw_qk_norm_rope(Q, None, cu, rope=torch.zeros(8, 24, device=DEV))
    with pytest.raises(_lib.PwError):
        api.pw_append(Q[:, :2], Q[:, :2], pages, pages, _i32([[0]]), cu, k_scale=0.0)
    with pytest.raises(AssertionError):
        api.pw_append(Q[:, :3], Q[:, :2], pages, pages, _i32([[0]]), cu)
    with pytest.raises(AssertionError):
        api.pw_qk_norm_rope(Q, None, cu, q_weight=_bf16(rng, 6, 128))
    with pytest.raises(AssertionError):
        api.pw_qk_norm_rope(Q, None, cu, Q_out=_bf16(rng, 2, 6, 128))
    torch.cuda.synchronize()
    assert bool((pages == 0).all())


# ---------------------------------------------------------------------------------------
# Together, as they are used
# ---------------------------------------------------------------------------------------

class Model:
    """The state of one attention layer: projections come from outside, the cache is kept here."""

    def __init__(self, rng, B, Hq, Hkv, max_len):
        self.Hq, self.Hkv, self.B = Hq, Hkv, B
        cols = (max_len + 63) // 64
        self.table = rng.permutation(B * cols).astype(np.int32).reshape(B, cols)
        self.K = torch.full((B * cols, Hkv, 64, 128), 0x7F, dtype=torch.uint8, device=DEV)
        self.V = self.K.clone()
        self.wq, self.wk = _bf16(rng, 128, scale=0.3) + 1, _bf16(rng, 128, scale=0.3) + 1
        self.rope = api.rope_table(max_len, device=DEV)
        self.dev_table = _i32(self.table)

    def step(self, qkv, cu, ctx, **kw):
        Hq, Hkv = self.Hq, self.Hkv
        return api.extend(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], self.K, self.V, self.dev_table, cu, ctx,
                          q_weight=self.wq, k_weight=self.wk, rope=self.rope, k_scale=2.0 ** -6, v_scale=2.0 ** -6, **kw)

    def expected(self, qkv, qlens, ctx):
        """Plain form of one step on the cache as it stands after it (its codes are taken as given)."""
        Hq = self.Hq
        q, _ = ref.norm_rope(ref.f64(qkv[:, :Hq]), ref.positions(qlens, ctx), ref.f64(self.wq), rot=128)
        q = torch.from_numpy(q).to(torch.bfloat16)
        O, _, b, _ = ref.attn(ref.f64(q), self.K.cpu().numpy(), self.V.cpu().numpy(), self.table, qlens, ctx, 2.0 ** -6,
                              2.0 ** -6, 128 ** -0.5)
        # a query element next to a rounding border may round the other way: half a step of bf16 in q
        # moves a score by at most 2^-8 sum |q k|, the softmax by twice that; in practice a few do
        return O, b


def _close(got, want, what):
    err = np.linalg.norm(ref.f64(got) - want) / np.linalg.norm(want)
    # bf16's own rounding is uniform within half a step: 2^-8 / sqrt(3) of the norm at most; the rest
    # of the bound (2^-11 of the weights, a few queries rounded the other way) stays below that again
    assert err <= 2.0 ** -8, f"{what}: {err:.2e}"


def test_prompt_chunk_and_decode_steps_share_one_cache():
    rng = np.random.default_rng(20)
    m = Model(rng, 3, 8, 2, 400)
    ctx = [0, 0, 0]
    status = api.new_status(DEV)
    for qlens in ([130, 1, 64], [1, 200, 0], [1, 1, 1], [1, 1, 1], [5, 4, 66]):
        cu, cl = ref.batch(qlens, ctx)
        qkv = _bf16(rng, int(cu[-1]), 12, 128)
        O = m.step(qkv, _i32(cu), _i32(cl), max_q_len=max(qlens), status=status)
        _ok(status)
        want, _ = m.expected(qkv, qlens, ctx)
        _close(O, want, f"step {qlens}")
        ctx = [c + n for c, n in zip(ctx, qlens)]


def test_appended_pages_are_what_the_sparse_prefill_reads():
    """pw_append's pages under pw_group + pw_attn with every causal page selected equal the dense call."""
    rng = np.random.default_rng(21)
    qlens = [200, 77]
    m = Model(rng, 2, 8, 2, 256)
    cu, _ = ref.batch(qlens, [0, 0])
    qkv = _bf16(rng, 277, 12, 128)
    status = api.new_status(DEV)
    dense = m.step(qkv, _i32(cu), None, max_q_len=200, status=status)
    Qn, _ = api.pw_qk_norm_rope(qkv[:, :8], None, _i32(cu), q_weight=m.wq, rope=m.rope)
    own = ref.positions(qlens, [0, 0]) // 64
    sel = np.where(np.arange(4) <= own[:, None], np.arange(4), -1).astype(np.int32)
    sel = np.repeat(sel[:, None], 2, 1)
    sm = 128 ** -0.5
    # keys behind a sequence's end are part of its last page: give them finite codes
    m.K[m.K == 0x7F], m.V[m.V == 0x7F] = 0, 0
    sparse, _ = api.prefill(Qn, m.K, m.V, m.dev_table, _i32(sel), _i32(cu), cu, 16, 8, k_scale=2.0 ** -6,
                            v_scale=2.0 ** -6, sm_scale=sm, status=status)
    _ok(status)
    _close(dense, ref.f64(sparse), "dense against sparse")


def test_captured_steps_replay_with_growing_contexts():
    rng = np.random.default_rng(22)
    B = 3
    m, twin = Model(rng, B, 8, 2, 300), None
    cu = _i32(np.arange(B + 1))
    ctx = _i32([0, 62, 200])
    qkv = _bf16(rng, B, 12, 128)
    ws = api.chunk_workspace(B, B, 8, 2, max_q_len=1, device=DEV)
    status = api.new_status(DEV)
    m.K.zero_(), m.V.zero_()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        m.step(qkv, cu, ctx, max_q_len=1, workspace=ws, status=status)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        O = m.step(qkv, cu, ctx, max_q_len=1, workspace=ws, status=status)
    for step in range(4):
        qkv.copy_(_bf16(rng, B, 12, 128))
        g.replay()
        _ok(status)
        c = ctx.cpu().tolist()
        want, _ = m.expected(qkv, [1] * B, c)
        _close(O, want, f"replay {step}")
        ctx += 1


def test_two_captured_graphs_with_a_workspace_each():
    """Two graphs, replayed at the same time on two streams."""
    rng = np.random.default_rng(26)
    jobs = []
    for q, c in ((1, 3000), (150, 700)):
        cu, cl, table, Q, Kp, Vp = _attn_inputs(rng, [q], [c], 8, 2)
        args = (Q, torch.from_numpy(Kp).to(DEV), torch.from_numpy(Vp).to(DEV), _i32(table), _i32(cu), _i32(cl))
        kw = dict(max_q_len=q, k_scale=2.0 ** -6, workspace=api.chunk_workspace(1, q, 8, 2, max_q_len=q, device=DEV))
        want = api.pw_chunk_attn(*args, **kw)
        torch.cuda.synchronize()
        g, out = torch.cuda.CUDAGraph(), torch.empty_like(want)
        with torch.cuda.graph(g):
            api.pw_chunk_attn(*args, O=out, **kw)
        jobs.append((g, out, want, torch.cuda.Stream(), args, kw))  # a graph keeps none of its tensors alive
    for _ in range(5):
        for g, out, _, s, _, _ in jobs:
            with torch.cuda.stream(s):
                out.zero_()
                g.replay()
        torch.cuda.synchronize()
        for _, out, want, _, _, _ in jobs:
            assert torch.equal(out, want)


def test_two_streams_with_a_workspace_each():
    rng = np.random.default_rng(23)
    jobs = []
    for q, c in ((1, 6000), (120, 2000)):
        cu, cl, table, Q, Kp, Vp = _attn_inputs(rng, [q], [c], 8, 2)
        args = (Q, torch.from_numpy(Kp).to(DEV), torch.from_numpy(Vp).to(DEV), _i32(table), _i32(cu), _i32(cl))
        kw = dict(max_q_len=q, k_scale=2.0 ** -6, v_scale=2.0 ** -6)
        jobs.append((args, kw, api.pw_chunk_attn(*args, **kw), torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [[api.pw_chunk_attn(*a, **kw, stream=s) for a, kw, _, s in jobs] for _ in range(5)]
    torch.cuda.synchronize()
    for run in outs:
        for (_, _, want, _), got in zip(jobs, run):
            assert torch.equal(want, got)


def test_cache_offsets_past_32_bits():
    """Physical pages whose byte offset passes 2^31 and 2^32."""
    n_phys, Hkv = 70000, 8  # 4.6 GB each
    K = torch.zeros(n_phys, Hkv, 64, 128, dtype=torch.uint8, device=DEV)
    V = torch.zeros(n_phys, Hkv, 64, 128, dtype=torch.uint8, device=DEV)
    rng = np.random.default_rng(24)
    for qlens, ctx in (([1, 1], [150, 100]), ([140, 20], [0, 100])):
        cu, cl = ref.batch(qlens, ctx)
        table = np.array([[69999, 33000, 1], [40000, 66000, 2]], np.int32)
        T = int(cu[-1])
        codes = _codes(rng, (2, 8, Hkv, 64, 128))
        ids = np.unique(table)
        small = np.searchsorted(ids, table)
        K[ids.tolist()], V[ids.tolist()] = torch.from_numpy(codes[0, :6]).to(DEV), torch.from_numpy(codes[1, :6]).to(DEV)
        Q = _bf16(rng, T, 16, 128)
        k_new, v_new = _bf16(rng, T, Hkv, 128), _bf16(rng, T, Hkv, 128)
        status = api.new_status(DEV)
        api.pw_append(k_new, v_new, K, V, _i32(table), _i32(cu), _i32(cl), k_scale=2.0 ** -6, v_scale=2.0 ** -6, status=status)
        O = api.pw_chunk_attn(Q, K, V, _i32(table), _i32(cu), _i32(cl), max_q_len=max(qlens), k_scale=2.0 ** -6,
                              v_scale=2.0 ** -6, status=status)
        _ok(status)
        kc, vc = K[ids.tolist()].cpu().numpy(), V[ids.tolist()].cpu().numpy()
        pos, seq = ref.positions(qlens, ctx), np.repeat(np.arange(2), qlens)
        ref.assert_e4m3(kc[small[seq, pos // 64], :, pos % 64], ref.f64(k_new) * 64, 0.0)
        want, _, bO, _ = ref.attn(ref.f64(Q), kc, vc, small, qlens, ctx, 2.0 ** -6, 2.0 ** -6, 128 ** -0.5)
        ref.assert_bf16(O, want, bO)
