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


# ---------------------------------------------------------------- operands that overlap
# Refusals only: with the overlap taken away these addresses would be read.
MB = 1 << 20
PAGES = dict(lens=1 * MB, n_new=2 * MB, B=4, page_size=16, free_pages=3 * MB, n_free=9, used_in=4 * MB, table=5 * MB,
             max_blocks=8, q_start=6 * MB, positions=7 * MB, slots=8 * MB, N=10, new_lens=9 * MB, used_out=10 * MB, stream=None)


@pytest.mark.parametrize("kw", [dict(q_start=PAGES["new_lens"] - 16), dict(used_out=PAGES["q_start"] + 16),
                                dict(positions=PAGES["slots"] + 76), dict(table=PAGES["positions"] - 124),
                                dict(new_lens=PAGES["table"])])
def test_plan_refuses_outputs_that_overlap(lib, kw):
    assert lib.llm_op_kv_pages(*(PAGES | kw).values()) == L.LLM_ERR_BAD_ARG
    assert "overlaps" in lib.llm_last_error().decode()


APPEND = dict(q=16 * MB, k=32 * MB, v=48 * MB, q_ld=6 * 128, k_ld=6 * 128, v_ld=6 * 128, dtype=L.LLM_BF16, q_norm=1 * MB,
              k_norm=2 * MB, norm_dtype=L.LLM_F32, eps=1e-5, rope_cos=3 * MB, rope_sin=4 * MB, n_pos=10, positions=5 * MB,
              slots=6 * MB, N=3, H=4, Hk=1, d=128, q_out=64 * MB, pool=80 * MB, n_pages=2, page_size=16, k_out=96 * MB,
              v_out=112 * MB, stream=None)


@pytest.mark.parametrize("kw", [
    dict(q_out=APPEND["q"]),                                   # rows of other strides
    dict(q_out=APPEND["q"], q_ld=4 * 128, dtype=L.LLM_F32),    # and of another type
    dict(q_out=APPEND["q"] + 16, q_ld=4 * 128),
    dict(q_out=APPEND["k"]), dict(k_out=APPEND["v"]), dict(k_out=APPEND["k"] + 2 * 6 * 128 * 2 + 240),
    dict(q_out=APPEND["q_norm"]), dict(v_out=APPEND["rope_sin"] + 2544), dict(pool=APPEND["slots"] - 5104),
    dict(k_out=APPEND["v_out"] + 752), dict(q_out=APPEND["pool"] + 5104), dict(pool=APPEND["v"] - 16),
    dict(q_out=APPEND["positions"])])
def test_append_refuses_operands_that_overlap(lib, kw):
    assert lib.llm_op_qk_norm_rope_kv4(*(APPEND | kw).values()) == L.LLM_ERR_BAD_ARG
    assert "overlaps" in lib.llm_last_error().decode()


ATTEND = dict(q=16 * MB, pool=32 * MB, n_pages=4, page_size=16, table=1 * MB, max_blocks=4, lens=2 * MB, q_start=3 * MB, B=2,
              N=2, max_new=1, H=4, Hk=2, d=128, out=48 * MB, workspace=64 * MB, workspace_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("kw", [dict(out=ATTEND["q"]), dict(out=ATTEND["q"] - 2032), dict(out=ATTEND["pool"] + 16),
                                dict(out=ATTEND["lens"]), dict(workspace=ATTEND["q"] + 2032), dict(out=ATTEND["workspace"] + 4096),
                                dict(workspace=ATTEND["table"]), dict(workspace=ATTEND["q_start"])])
def test_attention_refuses_operands_that_overlap(lib, kw):
    assert lib.llm_op_attention_kv4(*(ATTEND | kw).values()) == L.LLM_ERR_BAD_ARG
    assert "overlaps" in lib.llm_last_error().decode()


# ---------------------------------------------------------------- what the binding sees before any call
def test_binding_refuses_operands_of_another_rank(lib):
    import torch
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    f, bf = torch.zeros, lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    i64 = lambda *s: torch.zeros(*s, dtype=torch.int64)
    pages = dict(lens=i(2), n_new=i(2), page_size=16, free_pages=i(4), used_in=i(1), table=i(2, 3), q_start=i(3), positions=i(5),
                 slots=i64(5), new_lens=i(2), used_out=i(1))
    append = dict(q=bf(5, 4, 128), k=bf(5, 2, 128), v=bf(5, 2, 128), positions=i(5), slots=i64(5), rope_cos=f(9, 64),
                  rope_sin=f(9, 64), q_out=bf(5, 4, 128), pool=u8(3, 5120), page_size=16)
    attend = dict(q=bf(5, 4, 128), pool=u8(3, 5120), page_size=16, Hk=2, table=i(2, 3), lens=i(2), q_start=i(3), max_new=5,
                  out=bf(5, 512), workspace=u8(64))
    for call, good, names in ((L.llm_op_kv_pages, pages, ("lens", "free_pages", "table", "positions", "n_new", "used_out")),
                              (L.llm_op_qk_norm_rope_kv4, append, ("q", "k", "v", "rope_cos", "rope_sin", "positions", "q_out")),
                              (L.llm_op_attention_kv4, attend, ("q", "pool", "table", "lens", "q_start", "out"))):
        for name in names:
            for x in (good[name].flatten() if good[name].dim() > 1 else good[name][None], good[name].sum()):
                with pytest.raises(L.LlmError) as e:
                    call(**(good | {name: x}))
                assert e.value.code == L.LLM_ERR_BAD_ARG, name
