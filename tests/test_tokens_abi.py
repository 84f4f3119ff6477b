"""pw_qk_norm_rope, pw_append and pw_chunk_attn: refusals on the host (nothing here reaches a GPU),
and pins of the plain 64-bit forms the GPU tests compare with."""
import ctypes as C

import numpy as np
import pytest
import torch

from dynamic_sparse_attention_pw_b200 import _lib, api, build

import tokens_ref as ref

OK, INVALID, UNSUPPORTED, CAPACITY = (_lib.PW_OK, _lib.PW_ERR_INVALID_ARG, _lib.PW_ERR_UNSUPPORTED,
                                      _lib.PW_ERR_CAPACITY)


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.load()


NORM = dict(Q=256, qt=1024, qh=128, Hq=8, K=256, kt=256, kh=128, Hk=2, qw=256, qws=0, kw=256, kws=128, eps=1e-6,
            rope=256, max_pos=64, rot=128, inter=0, cu=256, ctx=256, B=1, T=4, Qo=256, qot=1024, qoh=128,
            Ko=256, kot=256, koh=128, status=256, stream=None)
APPEND = dict(K=256, kt=256, kh=128, V=256, vt=256, vh=128, Hkv=2, kw=256, kws=0, eps=1e-6, rope=256, max_pos=64,
              rot=64, inter=1, cu=256, ctx=None, B=1, T=4, table=256, max_pages=2, n_phys=2, ks=1.0, vs=1.0,
              Kp=256, Vp=256, status=None, stream=None)
ATTN = dict(Q=256, qt=1024, qh=128, Hq=8, Kp=256, Vp=256, Hkv=2, table=256, max_pages=2, n_phys=2, cu=256, ctx=256,
            B=1, T=4, max_q=4, window=0, ks=1.0, vs=1.0, sm=0.1, O=256, lse=None, ws=256, wsb=1 << 30, status=None,
            stream=None)


def _call(fn, base, **change):
    assert set(change) <= set(base)
    return fn(*{**base, **change}.values())


@pytest.mark.parametrize("change,code", [
    (dict(Q=None), INVALID), (dict(Q=264), INVALID), (dict(qt=1028), INVALID), (dict(qh=4), INVALID),
    (dict(Qo=None), INVALID), (dict(K=None), INVALID), (dict(Ko=None), INVALID), (dict(Hq=0, Hk=0), INVALID),
    (dict(Hq=-1), INVALID), (dict(qot=0), INVALID), (dict(qoh=0), INVALID), (dict(qot=896), INVALID),
    (dict(koh=64), INVALID), (dict(kws=64), INVALID), (dict(qw=264), INVALID), (dict(rot=24), UNSUPPORTED),
    (dict(rot=144), UNSUPPORTED), (dict(rot=-16), INVALID), (dict(max_pos=0), INVALID), (dict(rope=264), INVALID),
    (dict(cu=None), INVALID), (dict(B=0), INVALID), (dict(T=-1), INVALID), (dict(T=1 << 31), UNSUPPORTED),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(T=0), OK), (dict(T=0, Q=None, K=None, Qo=None, Ko=None), OK),
])
def test_norm_rope_refusals(L, change, code):
    assert _call(L.pw_qk_norm_rope, NORM, **change) == code


@pytest.mark.parametrize("change,code", [
    (dict(K=None), INVALID), (dict(V=None), INVALID), (dict(V=260), INVALID), (dict(vt=4), INVALID),
    (dict(Hkv=0), INVALID), (dict(kws=1), INVALID), (dict(rot=8), UNSUPPORTED), (dict(cu=None), INVALID),
    (dict(B=0), INVALID), (dict(T=-1), INVALID), (dict(table=None), INVALID), (dict(max_pages=-1), INVALID),
    (dict(n_phys=-1), INVALID), (dict(ks=0.0), INVALID), (dict(vs=-1.0), INVALID), (dict(ks=float("nan")), INVALID),
    (dict(vs=float("inf")), INVALID), (dict(ks=1e-40), INVALID), (dict(Kp=None), INVALID), (dict(Vp=264), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(T=0), OK),
])
def test_append_refusals(L, change, code):
    assert _call(L.pw_append, APPEND, **change) == code


@pytest.mark.parametrize("change,code", [
    (dict(Q=None), INVALID), (dict(Q=264), INVALID), (dict(qt=4), INVALID), (dict(Hq=7), UNSUPPORTED),
    (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(Kp=None), INVALID), (dict(Vp=264), INVALID),
    (dict(table=None), INVALID), (dict(max_pages=0), INVALID), (dict(n_phys=0), INVALID), (dict(cu=None), INVALID),
    (dict(max_pages=1 << 25), UNSUPPORTED), (dict(n_phys=1 << 25), UNSUPPORTED), (dict(B=0), INVALID),
    (dict(T=-1), INVALID), (dict(T=1 << 31), UNSUPPORTED), (dict(max_q=0), INVALID), (dict(window=-1), INVALID),
    (dict(ks=0.0), INVALID), (dict(vs=float("nan")), INVALID), (dict(sm=-0.1), INVALID), (dict(sm=float("inf")), INVALID),
    (dict(sm=1e-30, ks=1e-30), INVALID), (dict(O=None), INVALID), (dict(O=264), INVALID), (dict(ws=None), CAPACITY),
    (dict(wsb=0), CAPACITY), (dict(ws=264), INVALID), (dict(T=0), OK),
])
def test_chunk_attn_refusals(L, change, code):
    assert _call(L.pw_chunk_attn, ATTN, **change) == code


def test_chunk_workspace_size(L):
    n = C.c_size_t()
    assert L.pw_chunk_workspace_size(3, 100, 32, 8, 50, C.byref(n)) == OK and n.value >= 256
    m = C.c_size_t()
    assert L.pw_chunk_workspace_size(3, 1 << 20, 32, 8, 1 << 16, C.byref(m)) == OK
    assert m.value < 1 << 28  # it grows with neither the tokens nor the contexts
    for bad in ((0, 1, 8, 2, 1), (1, -1, 8, 2, 1), (1, 1, 0, 2, 1), (1, 1, 8, 0, 1), (1, 1, 8, 2, 0)):
        assert L.pw_chunk_workspace_size(*bad, C.byref(n)) == INVALID
    assert L.pw_chunk_workspace_size(1, 1, 7, 2, 1, C.byref(n)) == UNSUPPORTED
    assert L.pw_chunk_workspace_size(1, 1, 8, 2, 1, None) == INVALID


def test_binding_refuses_host_tensors(L):
    cu = torch.tensor([0, 1], dtype=torch.int32)
    x = torch.zeros(1, 2, 128, dtype=torch.bfloat16)
    pages = torch.zeros(1, 2, 64, 128, dtype=torch.uint8)
    table = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(AssertionError):
        api.pw_qk_norm_rope(x, x, cu)
    with pytest.raises(AssertionError):
        api.pw_append(x, x, pages, pages, table, cu)
    with pytest.raises(AssertionError):
        api.pw_chunk_attn(x, pages, pages, table, cu)


def test_rope_table_is_rounded_once():
    t = api.rope_table(70000, 64, device="cpu")
    pos = np.array([0, 1, 63, 4097, 69999])
    a = pos[:, None] * 10000.0 ** (-np.arange(0, 64, 2) / 64)
    want = np.concatenate([np.cos(a), np.sin(a)], 1)
    # half a step of fp32, and the angle's own 64-bit rounding at these positions
    assert np.all(np.abs(t[pos].double().numpy() - want) <= 2.0 ** -24 * np.abs(want) + 1e-10)
    assert t.dtype == torch.float32 and t.shape == (70000, 64)


# ---- the plain forms themselves ----------------------------------------------------------

def test_plain_rotation_by_complex_numbers_and_relative_positions():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 2, 128))
    pos = np.array([0, 5, 1000])
    for inter in (False, True):
        y, _ = ref.norm_rope(x, pos, rot=128, interleaved=inter)
        z = x[..., 0::2] + 1j * x[..., 1::2] if inter else x[..., :64] + 1j * x[..., 64:]
        z = z * np.exp(1j * pos[:, None, None] * 10000.0 ** (-np.arange(0, 128, 2) / 128))
        got = y[..., 0::2] + 1j * y[..., 1::2] if inter else y[..., :64] + 1j * y[..., 64:]
        assert np.allclose(got, z, atol=1e-12) and np.array_equal(y[0], x[0])
        # a score depends on the distance alone
        q, k = rng.standard_normal((2, 1, 1, 128))
        at = lambda v, p: ref.norm_rope(v, np.array([p]), rot=128, interleaved=inter)[0].ravel()  # noqa: E731
        assert abs(at(q, 17) @ at(k, 10) - at(q, 507) @ at(k, 500)) < 1e-10


def test_plain_e4m3_values_are_the_formats():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, ref.VALUES, equal_nan=True)


def test_plain_attention_against_one_dense_softmax():
    rng = np.random.default_rng(1)
    qlens, ctx = [3, 0, 2], [5, 7, 62]
    table, n_phys = ref.pages_for(qlens, ctx, rng)
    codes = rng.integers(0, 127, (2, n_phys, 2, 64, 128)).astype(np.uint8)
    Q = rng.standard_normal((5, 4, 128))
    O, lse, _, _ = ref.attn(Q, codes[0], codes[1], table, qlens, ctx, 0.01, 0.02, 0.3, window=4)
    t, hq = 4, 3  # last token: sequence 2, position 63
    k = ref.VALUES[codes[0][table[2, 0], 1]] * 0.01
    v = ref.VALUES[codes[1][table[2, 0], 1]] * 0.02
    s = (k @ Q[t, hq] * 0.3)[60:64]
    w = np.exp(s) / np.exp(s).sum()
    assert np.allclose(O[t, hq], w @ v[60:64]) and np.isclose(lse[t, hq], np.log(np.exp(s).sum()))
