"""What the 4-bit cache's calls refuse and what they take, as far as the host decides it (CPU)."""
import pytest

import llama_decoder_forward_fwd_b200 as L
from llama_decoder_forward_fwd_b200 import build as B


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


def _attend(lib, **kw):
    """A call that no size lets through: its workspace is one byte."""
    a = dict(q=1 << 40, pool=2 << 40, n_pages=4, page_size=16, table=3 << 40, max_blocks=4, lens=4 << 40, q_start=5 << 40, B=2,
             N=2, max_new=1, H=4, Hk=2, d=128, out=6 << 40, workspace=7 << 40, workspace_bytes=1, stream=None)
    assert set(kw) <= set(a)
    rc = lib.llm_op_attention_kv4(*(a | kw).values())
    assert rc != L.LLM_OK
    return rc, lib.llm_last_error().decode()


# 64k new tokens of 64 heads, one prompt as long as its table, 16 of 32k, 16 of 128k
@pytest.mark.parametrize("kw", [dict(N=65536, H=64, Hk=8, max_blocks=1024, page_size=128, max_new=65536),
                                dict(B=1, N=131072, H=32, Hk=8, max_blocks=2048, page_size=64, max_new=131072),
                                dict(B=16, N=524288, H=32, Hk=8, max_blocks=512, page_size=64, max_new=32768),
                                dict(B=16, N=2097152, H=32, Hk=8, max_blocks=2048, page_size=64, max_new=131072)])
def test_large_steps_are_taken(lib, kw):
    rc, why = _attend(lib, **kw)
    assert rc == L.LLM_ERR_BAD_ARG and "workspace" in why, why
    ws = lib.llm_op_attention_kv4_workspace(kw.get("B", 2), kw["N"], kw["max_new"], kw["H"], kw["Hk"], 128, kw["max_blocks"],
                                            kw["page_size"])
    assert ws > 0


@pytest.mark.parametrize("kw", [dict(N=1 << 30, H=4, Hk=1), dict(N=1 << 22, H=64, Hk=8, max_blocks=1 << 14, page_size=128),
                                dict(B=1 << 20, N=1, H=32, Hk=8, max_blocks=1 << 19),
                                dict(B=1, N=1 << 24, H=8, Hk=1, max_blocks=1 << 16, page_size=128)])
def test_steps_that_are_too_large_are_refused(lib, kw):
    rc, why = _attend(lib, **kw)
    assert rc == L.LLM_ERR_UNSUPPORTED and "one call" in why, why


def test_the_workspace_of_expanded_prompts_is_bounded(lib):
    """By the tables' width while that stays within 1 GiB, by 64 MiB beyond; with what else a call needs, some 50 MiB."""
    def size(B, tokens, Hk=8):
        return lib.llm_op_attention_kv4_workspace(B, 4096, 2048, 4 * Hk, Hk, 128, -(-tokens // 64), 64)
    last = 0
    for tokens in (2048, 8192, 16384, 65536):
        assert last < size(2, tokens) < (2 * tokens // 128 * 8 << 16) + (50 << 20)
        last = size(2, tokens)
    for B, tokens in ((3, 131072), (16, 32768), (2, 1 << 24), (64, 1 << 20)):
        assert (64 << 20) < size(B, tokens) < (64 + 50 << 20)
