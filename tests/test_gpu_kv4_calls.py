"""How the 4-bit cache's calls are made (GPU): the first ones of a process inside a capture, with the bounds-checking
build, and without memory of their own."""
import os
import subprocess
import sys

import pytest
import torch

from kv4_case import MANY, Case

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.parametrize("how,variant", [("capture", None), ("checked", "checked")])
def test_in_a_process_of_their_own(lib, how, variant):
    env = dict(os.environ)
    if variant:
        env["LLM_LIB_VARIANT"] = variant
    r = subprocess.run([sys.executable, os.path.join(HERE, "kv4_child.py"), how], env=env, capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0 and f"CHILD OK {how}" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]


def test_no_call_takes_memory(lib):
    """After one call of each form has loaded its kernels, others of the same and other sizes leave the device's free
    memory as it was."""
    import llama_decoder_forward_fwd_b200 as L
    forms = [([300, 77], [1, 2], None), ([300, 177], [150, 1], None), ([300, 177], [150, 1], MANY)]
    more = [([3000, 40], [1, 1], None), ([900, 20], [400, 20], None), ([900, 20], [400, 20], MANY)]
    ops = [Case(lens, new, 8, 2, 128, 32, 3).operands(L, mx) for lens, new, mx in forms + more]
    for a in ops[:3]:
        L.llm_op_attention_kv4(*a)
    L.llm_op_synchronize()
    free = torch.cuda.mem_get_info()[0]
    for _ in range(3):
        for a in ops:
            L.llm_op_attention_kv4(*a)
        L.llm_op_synchronize()
    assert torch.cuda.mem_get_info()[0] == free


@pytest.mark.parametrize("N,H,Hk,d", [(1, 8, 2, 128), (300, 5, 1, 64), (70, 4, 4, 128)])
def test_append_in_place_and_between_rows(lib, N, H, Hk, d):
    """q_out, k_out and v_out may be q, k and v themselves, and may lie between the rows of strided ones."""
    import llama_decoder_forward_fwd_b200 as L
    bf, dev, P = torch.bfloat16, "cuda", 16
    g = torch.Generator(device=dev).manual_seed(N)
    rand = lambda *s: torch.randn(*s, device=dev, generator=g).to(bf)
    q, k, v, w = rand(N, H, d), rand(N, Hk, d), rand(N, Hk, d), rand(d)
    ang = torch.rand(N + 9, d // 2, device=dev, generator=g)
    n_pages = -(-N // P)
    tables = torch.cos(ang), torch.sin(ang)
    pos, slots = torch.randperm(N, device=dev, generator=g).int(), torch.randperm(n_pages * P, device=dev, generator=g)[:N]

    def run(q, k, v, q_out, k_out, v_out):
        pool = torch.zeros(n_pages, L.llm_kv4_page_bytes(Hk, d, P), dtype=torch.uint8, device=dev)
        torch.cuda.synchronize()
        L.llm_op_qk_norm_rope_kv4(q, k, v, pos, slots, *tables, q_out, pool, P, q_norm=w, k_norm=w, k_out=k_out, v_out=v_out)
        L.llm_op_synchronize()
        return q_out, k_out, v_out, pool
    want = run(q, k, v, torch.empty_like(q), torch.empty_like(k), torch.empty_like(v))
    x, y, z = q.clone(), k.clone(), v.clone()
    for a, b in zip(run(x, y, z, x, y, z), want):
        assert torch.equal(a, b)
    # two token rows far apart, with the outputs in the gap; and one wide row that holds all of a token
    if N > 1:
        n = (2 * H + 4 * Hk) * d
        room = torch.empty(2, 2 * n, dtype=bf, device=dev)
        part = lambda at, heads: room[:, at:at + heads * d].unflatten(1, (heads, d))
        ins = part(0, H), part(H * d, Hk), part((H + Hk) * d, Hk)
        for a, b in zip(ins, (q, k, v)):
            a.copy_(b[:2])
        gap, at = room[0, (H + 2 * Hk) * d:], 0
        outs = []
        for heads in (H, Hk, Hk):
            outs.append(gap[at:at + 2 * heads * d].view(2, heads, d))
            at += 2 * heads * d
        pos, slots = pos[:2].clone(), slots[:2].clone()
        got = run(*ins, *outs)
        want = run(q[:2].contiguous(), k[:2].contiguous(), v[:2].contiguous(), *(torch.empty_like(t) for t in outs))
        for a, b in zip(got, want):
            assert torch.equal(a, b)
