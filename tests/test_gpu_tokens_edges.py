"""pw_append and extend on the GPU: codes under scales that are no power of two, extend's outputs
(tokens_ref.py holds the plain 64-bit forms)."""
import numpy as np
import pytest
import torch

from dynamic_sparse_attention_pw_b200 import api

import tokens_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).to(DEV)


def _bf16(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape)).to(torch.bfloat16).to(DEV)


@pytest.mark.parametrize("scale", [2.0 ** -6, 0.013, 3 / 64, 0.75, 1.1, 1e-30, 1e30])
def test_append_codes_are_of_the_product_with_the_reciprocal(scale):
    """Rows that are neither normalised nor rotated: the codes are exactly those of x * fl32(1 / scale), and
    within half a step of the quotient."""
    rng = np.random.default_rng(30)
    T, H = 130, 3
    spread = 2.0 ** rng.integers(-12, 12, (T, H, 128)) * scale
    K = torch.from_numpy(rng.standard_normal((T, H, 128)) * spread).to(torch.bfloat16).to(DEV)
    V = torch.from_numpy(rng.integers(-448, 449, (T, H, 128)) / 16 * scale).to(torch.bfloat16).to(DEV)  # quotients on and next to borders
    cu, cl = ref.batch([T], [50])
    table, n_phys = ref.pages_for([T], [50], rng)
    pages = torch.zeros(2, n_phys, H, 64, 128, dtype=torch.uint8, device=DEV)
    status = api.new_status(DEV)
    api.pw_append(K, V, pages[0], pages[1], _i32(table), _i32(cu), _i32(cl), k_scale=scale, v_scale=scale, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    s32 = np.float32(scale)
    inv = torch.from_numpy(np.array(np.float32(1) / s32))
    pos = 50 + np.arange(T)
    got = pages.cpu().numpy()[:, table[0, pos // 64], :, pos % 64].swapaxes(0, 1)
    for x, codes in ((K, got[0]), (V, got[1])):
        want = (x.cpu().float() * inv).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        assert np.array_equal(codes, want)
        quotient = ref.f64(x) / np.float64(s32)
        ref.assert_e4m3(codes, quotient, 2 * ref.U32 * np.abs(quotient))  # the reciprocal's rounding and the product's


@pytest.mark.parametrize("qlens,ctx", [([1, 1, 1], [0, 62, 300]), ([70, 5], [100, 0])])
def test_extend_into_the_callers_outputs(qlens, ctx):
    """O and lse of the caller are what the single calls give, and rows behind the last sequence stay."""
    rng = np.random.default_rng(31)
    Hq, Hkv, pad = 8, 2, 3
    cu, cl = ref.batch(qlens, ctx)
    T = int(cu[-1])
    table, n_phys = ref.pages_for(qlens, ctx, rng)
    codes = torch.from_numpy(rng.standard_normal((2, n_phys, Hkv, 64, 128)) * 64).to(torch.float8_e4m3fn).view(torch.uint8).to(DEV)
    qkv = _bf16(rng, T + pad, Hq + 2 * Hkv, 128)
    Q, K, V = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    wq, wk, rope = _bf16(rng, 128), _bf16(rng, 128), api.rope_table(400, device=DEV)
    status = api.new_status(DEV)
    dev = (_i32(table), _i32(cu), _i32(cl))
    scales = dict(k_scale=2.0 ** -6, v_scale=2.0 ** -6)

    one = codes.clone()
    O = torch.full((T + pad, Hq, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T + pad, Hq), 7.0, device=DEV)
    got = api.extend(Q, K, V, one[0], one[1], *dev, max_q_len=max(qlens), q_weight=wq, k_weight=wk, rope=rope, status=status, O=O,
                     lse=lse, **scales)
    two = codes.clone()
    Qn, _ = api.pw_qk_norm_rope(Q, None, *dev[1:], q_weight=wq, rope=rope)
    api.pw_append(K, V, two[0], two[1], *dev, k_weight=wk, rope=rope, status=status, **scales)
    lse2 = torch.empty_like(lse)
    want = api.pw_chunk_attn(Qn, two[0], two[1], *dev, max_q_len=max(qlens), lse=lse2, status=status, **scales)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and got is O
    assert torch.equal(one, two) and torch.equal(O[:T], want[:T]) and torch.equal(lse[:T], lse2[:T])
    assert bool((O[T:] == 7.0).all()) and bool((lse[T:] == 7.0).all())
