"""pw_append on the GPU: codes under scales that are no power of two
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
