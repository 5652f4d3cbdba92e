"""Attention over the 4-bit cache in large calls (GPU): schedules of more than 2^31 units, page tables much wider than the
sequences, workspaces with room for some of the prompts."""
import math

import numpy as np
import pytest
import torch

from kv4_case import MANY, Case, marked

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _held(pool, Hk, d, P, which, g):
    """Values of KV head g of a pool whose pages lie in order, float64 [tokens, d]."""
    rec = pool.view(pool.shape[0], Hk, -1)[:, g]
    a, b = P * d // 2, P * d // 8
    c = rec[:, which * a:(which + 1) * a].reshape(-1, d // 2)
    sz = rec[:, 2 * a + which * b:2 * a + (which + 1) * b].reshape(-1, d // 8).view(torch.bfloat16).double()
    c = torch.stack((c & 15, c >> 4), -1).reshape(-1, d // 32, 32).double()
    return (c * sz[:, 0::2, None] + sz[:, 1::2, None]).to(torch.bfloat16).double().reshape(-1, d)


def test_more_units_than_32_bits_count(lib):
    """131k new tokens over their own keys, announced as one: 8 of their 4 x 131k rows at a time pass over all keys."""
    import llama_decoder_forward_fwd_b200 as L
    N, H, Hk, d, P = 132096, 32, 8, 64, 128
    assert (N * H // Hk // 8) * Hk * (N // 32) > 2**31
    g = torch.Generator(device=DEV).manual_seed(3)
    n_pages = N // P
    pool = torch.randint(0, 256, (n_pages, L.llm_kv4_page_bytes(Hk, d, P)), dtype=torch.uint8, device=DEV, generator=g)
    rec = pool.view(n_pages, Hk, -1)
    pairs = P * d // 8 * 2
    sz = (torch.rand(n_pages, Hk, pairs // 4, 2, device=DEV, generator=g) * torch.tensor([0.2, -2.0], device=DEV)).to(torch.bfloat16)
    rec[:, :, -pairs:] = sz.view(torch.uint8).reshape(n_pages, Hk, pairs)
    q = torch.randn(N, H, d, device=DEV, generator=g).to(torch.bfloat16)
    i32 = dict(dtype=torch.int32, device=DEV)
    table, lens = torch.arange(n_pages, **i32)[None].contiguous(), torch.tensor([N], **i32)
    q_start, out = torch.tensor([0, N], **i32), torch.zeros(N, H * d, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(L.llm_op_attention_kv4_workspace(1, N, 1, H, Hk, d, n_pages, P), dtype=torch.uint8, device=DEV)
    L.llm_op_attention_kv4(q, pool, P, Hk, table, lens, q_start, 1, out, ws)
    L.llm_op_synchronize()
    rows = torch.tensor([0, 1, 31, 32, 4095, 40000, 65535, 65536, 100001, 128000, N - 2, N - 1], device=DEV)
    mask = torch.arange(N, device=DEV)[None] > rows[:, None]
    for h in (0, 7, 17, H - 1):
        k, v = (_held(pool, Hk, d, P, w, h // 4) for w in (0, 1))
        w = torch.softmax((q[rows, h].double() @ k.T / math.sqrt(d)).masked_fill(mask, -math.inf), -1)
        want = w @ v
        bound = 2.0**-8 * want.abs() + (2.0**-8 + 2.0**-11) * (w @ v.abs())
        got = out[rows, h * d:(h + 1) * d].double()
        assert ((got - want).abs() <= bound).all(), h


@pytest.mark.parametrize("d,P", [(128, 128), (64, 64)])
def test_wide_page_tables_do_not_change_the_kernel(lib, d, P):
    """Prompts whose tables reach 270k tokens are expanded like those of tables that fit them: the same bits."""
    import llama_decoder_forward_fwd_b200 as L
    lens, new = [600, 450, 40], [500, 450, 1]
    outs = []
    for blocks in (5 * 128 // P, 270000 // P):
        case = Case(lens, new, 8, 4, d, P, 9, blocks=blocks)
        outs.append(case.run(L, MANY))
        case.check(outs[-1])
    assert np.array_equal(outs[0], outs[1])


@pytest.mark.parametrize("d,P,lens,new", [(128, 16, [300, 140, 700, 40, 90], [150, 140, 300, 1, 20]),
                                          (64, 64, [700, 130, 260], [500, 130, 3])])
def test_a_workspace_with_room_for_some_of_the_prompts(lib, d, P, lens, new):
    """From none of the expanded tiles to all of them: what has no room is expanded row block by row block."""
    import llama_decoder_forward_fwd_b200 as L
    mark = marked(2, d, lens)

    def make(b, which, r):
        x = mark(b, which, r)
        if which and b % 2:
            x[-7, 1] = np.nan  # of a sequence that turns from the prompts' kernels to the other
        return x
    case = Case(lens, new, 8, 2, d, P, 10, make=make, q_scale=0.1, pad=1)
    shape = (len(lens), case.N + 1)
    full = L.llm_op_attention_kv4_workspace(*shape, MANY, 8, 2, d, case.blocks, P)
    least = L.llm_op_attention_kv4_workspace(*shape, 200, 8, 2, d, case.blocks, P)
    assert least < full
    most = min(shape[0], shape[1] * 4 // 65) * -(-case.blocks * P // 128) * 2  # tiles that tables so wide may ask for
    sizes = {least, least + 1, full - 1, full, full + 100000}
    sizes |= {full - (most - n) * (512 * d + 8) for n in (1, 2, 4, 6, 7, 10, 12, 15, 18, 22, 24, 30)}
    for room in sorted(x for x in sizes if x >= least):
        case.check(case.run(L, MANY, room=room))
    with pytest.raises(L.LlmError) as e:
        case.run(L, MANY, room=least - 1)
    assert e.value.code == L.LLM_ERR_BAD_ARG


# B, new tokens of most, prompts among them, H, Hk, d, promised new tokens, pages a table is wide
@pytest.mark.parametrize("B,n,prompts,H,Hk,d,mx,blocks", [
    (1300, 1, [], 8, 2, 128, None, 4), (700, 3, [], 8, 1, 64, None, 4), (1300, 1, [0, 5, 700, 1299], 8, 2, 128, None, 4),
    (1300, 1, [0, 5, 700, 1023, 1024, 1299], 8, 2, 64, MANY, 4),
    (8, 3, [], 32, 8, 128, None, 1 << 23), (40, 1, [], 32, 8, 64, None, 1 << 21), (600, 1, [], 32, 8, 128, None, 1 << 17),
    (600, 8, [], 32, 8, 64, None, 1 << 16)])
def test_many_sequences_and_tables_that_want_64_bit_counts(lib, B, n, prompts, H, Hk, d, mx, blocks):
    """More sequences than a warp, a CTA and two of them look at in one go; and the schedule in 64 bits, which the tables'
    width alone asks for."""
    import llama_decoder_forward_fwd_b200 as L
    r = np.random.RandomState(B)
    P = 128 if blocks > 4 else 32
    lens = [int(x) for x in r.randint(1, 60, B)]
    new = [min(l, int(r.randint(0, n + 1)) if n > 1 else n) for l in lens]
    for b in prompts:
        lens[b], new[b] = 90 + b % 30, 60 + b % 30
    if blocks > 4:
        assert (sum(new) * H // Hk // 8 + B) * Hk * blocks * P // 32 >= 2**31
    case = Case(lens, new, H, Hk, d, P, 11, make=marked(Hk, d, lens), q_scale=0.1, blocks=blocks, pad=1)
    case.check(case.run(L, mx))


@pytest.mark.parametrize("mx", [None, 60, MANY])
def test_sequences_that_share_pages(lib, mx):
    """Three sequences whose tables begin with the same pages."""
    import llama_decoder_forward_fwd_b200 as L
    lens, new = [200, 200, 200], [2, 40, 1]
    case = Case(lens, new, 8, 2, 128, 32, 12, pad=1)
    case.table[1:, :5] = case.table[0, :5]
    for b in (1, 2):
        for which in (0, 1):
            case.kv[b][which][:160] = case.kv[0][which][:160]
    case.check(case.run(L, mx))
