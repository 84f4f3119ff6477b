"""api.py's calls on new tokens: what needs no GPU."""
import pytest

from dynamic_sparse_attention_pw_b200 import _lib, api, build


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def test_chunk_workspace_refuses_what_the_call_refuses():
    """A longest chunk of 0 is no hint left out: pw_chunk_attn refuses it, and so does its workspace."""
    with pytest.raises(_lib.PwError):
        api.chunk_workspace(1, 4, 8, 2, max_q_len=0, device="cpu")
    few = api.chunk_workspace(4, 4, 8, 2, max_q_len=1, device="cpu").numel()
    many = api.chunk_workspace(4, 400, 8, 2, max_q_len=100, device="cpu").numel()
    assert api.chunk_workspace(4, 400, 8, 2, device="cpu").numel() == many > few
    assert api.chunk_workspace(1, 0, 8, 2, device="cpu").numel() == few
