"""The model's own 4-bit cache (LLM_FLAG_KV4): its pages after refused calls and from step to step, and
prompts of a model with room for many long sequences (GPU)."""
import pytest
import torch

import seeded_inputs as S

pytestmark = pytest.mark.gpu
DEV = "cuda"

BASE = S.ModelShape(dim=512, n_layers=1, n_heads=4, n_kv_heads=1, head_dim=128, ffn_hidden=256, vocab=512,
                    max_seq_len=256, norm_eps=1e-5, rope_theta=500000.0, dtype="bf16", tie_embeddings=False)


def _model(shape, batch, tokens):
    import llama_decoder_forward_fwd_b200 as L
    glob, layers = S.make_weights(shape, 7)
    return L.Model(shape, glob, layers, max_batch=batch, max_tokens=tokens, flags=L.LLM_FLAG_KV4)


def _prefill(L, m, tokens):
    B = tokens.shape[0]
    nxt, lg = torch.empty(B, dtype=torch.int32, device=DEV), torch.empty(B, m.shape.vocab, device=DEV)
    L.llm_prefill(m.h, tokens.to(DEV), nxt, lg)
    L.llm_synchronize(m.h)
    return lg


def test_refused_calls_take_no_pages(lib):
    """Prompts that are more than one attention call takes over page tables this wide: each is refused, and however many
    there were, what follows is as in a model that never had one."""
    import llama_decoder_forward_fwd_b200 as L
    shape = BASE.replace(dim=1024, n_heads=16, n_kv_heads=2, head_dim=64, max_seq_len=1 << 25)
    T = 40000
    m = _model(shape, 1, T)
    x, nxt = torch.zeros(1, T, dtype=torch.int32, device=DEV), torch.empty(1, dtype=torch.int32, device=DEV)
    for _ in range((1 << 25) // T + 2):
        with pytest.raises(L.LlmError) as e:
            L.llm_prefill(m.h, x, nxt)
        assert e.value.code == L.LLM_ERR_UNSUPPORTED
    assert L.llm_kv_cache_get_lens(m.h, 1) == [0]
    chunks = [S.make_tokens(11, 1, n, shape.vocab) for n in (120, 90, 1)]
    got = [_prefill(L, m, t) for t in chunks]
    m.free()
    m = _model(shape.replace(max_seq_len=512), 1, 256)
    for a, t in zip(got, chunks):
        assert torch.equal(a, _prefill(L, m, t))
    m.free()


def test_pages_follow_the_lengths(lib):
    """Steps of some of the sequences, of all and of some again, to the last position; then the cache is used anew."""
    import llama_decoder_forward_fwd_b200 as L
    m = _model(BASE.replace(max_seq_len=200), 3, 3 * 200)
    one = [_model(BASE.replace(max_seq_len=200), 1, 200) for _ in range(3)]
    for _ in range(2):
        at = [0, 0, 0]
        tokens = S.make_tokens(12, 3, 200, BASE.vocab)
        for B, T in ((1, 70), (3, 20), (2, 64), (3, 1), (3, 45)):
            x = torch.stack([tokens[b, at[b]:at[b] + T] for b in range(B)])
            lg = _prefill(L, m, x)
            for b in range(B):
                alone = _prefill(L, one[b], x[b:b + 1])
                # another batch size may take other kernels: both are within the bf16 models' 2e-2 of the oracle
                assert (lg[b] - alone[0]).norm() <= 4e-2 * alone[0].norm(), (B, T, b)
                at[b] += T
        for x in (m, *one):
            L.llm_kv_cache_reset(x.h)
    for x in (m, *one):
        x.free()


def test_room_for_many_long_sequences_keeps_the_prompt_kernel(lib):
    """A prompt gives the same bits in a model of 16 sequences of 36k positions as in one made for it alone."""
    import llama_decoder_forward_fwd_b200 as L
    shape = BASE.replace(dim=2048, n_heads=32, n_kv_heads=8, head_dim=64, vocab=256)
    T = 600
    tokens = S.make_tokens(13, 1, T, shape.vocab)
    got = []
    for seq, batch in ((640, 1), (36864, 16)):
        m = _model(shape.replace(max_seq_len=seq), batch, T)
        got.append(_prefill(L, m, tokens))
        m.free()
    assert torch.equal(*got)
