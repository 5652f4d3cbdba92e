"""Run by test_gpu_kv4_calls.py in a process of its own (not a test module): the 4-bit cache's calls where nothing of
the library has run before.

capture  the process's first calls into the library are made while a graph is captured
checked  small cases of each call with the bounds-checking build (LLM_LIB_VARIANT=checked)
"""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
sys.path.insert(0, os.path.join(ROOT, "tests"))

import numpy as np  # noqa: E402
import torch  # noqa: E402

import kv4_util as K  # noqa: E402
import llama_decoder_forward_fwd_b200 as L  # noqa: E402
from kv4_case import MANY, Case, marked  # noqa: E402

FORMS = [([300, 77, 1], [1, 2, 1], 8, 2, 128, 32, None), ([300, 177, 140], [150, 3, 140], 8, 2, 64, 64, None),
         ([300, 177, 140], [150, 1, 140], 8, 2, 128, 16, MANY)]
i32 = dict(dtype=torch.int32, device="cuda")


def case_of(form):
    lens, new, H, Hk, d, P, mx = form
    return Case(lens, new, H, Hk, d, P, 5, make=marked(Hk, d, lens), q_scale=0.1), mx


def plan_and_append():
    """Operands of a plan and of the append of its tokens, and a check of what the calls leave."""
    lens, new, P, Hk, H, d = [15, 0], [2, 17], 16, 2, 4, 128
    table, free, N = [[5, -1, -1], [-1, -1, -1]], [8, 3, 0, 1], 20
    want = K.plan(lens, new, P, free, 0, table, 3, N)
    p = dict(lens=torch.tensor(lens, **i32), n_new=torch.tensor(new, **i32), free_pages=torch.tensor(free, **i32),
             used_in=None, table=torch.tensor(table, **i32), q_start=torch.zeros(3, **i32), positions=torch.zeros(N, **i32),
             slots=torch.zeros(N, dtype=torch.int64, device="cuda"), new_lens=torch.zeros(2, **i32), used_out=torch.zeros(1, **i32))
    r = np.random.RandomState(1)
    qkv = r.randn(N, H + 2 * Hk, d).astype(np.float32)
    cos, sin = K.rope_tables(64, d)
    g, dc, ds = (torch.from_numpy(x).cuda() for x in (qkv, cos, sin))
    pool = torch.zeros(9, L.llm_kv4_page_bytes(Hk, d, P), dtype=torch.uint8, device="cuda")
    q_out = torch.zeros(N, H, d, dtype=torch.bfloat16, device="cuda")

    def calls(stream):
        L.llm_op_kv_pages(page_size=P, stream=stream, **p)
        L.llm_op_qk_norm_rope_kv4(g[:, :H], g[:, H:H + Hk], g[:, H + Hk:], p["positions"], p["slots"], dc, ds, q_out, pool, P,
                                  stream=stream)

    def check():
        for k in ("table", "q_start", "positions", "slots", "new_lens"):
            assert np.array_equal(p[k].cpu().numpy(), want[k]), k
        host = K.Pool(9, Hk, d, P)
        for i in range(sum(new)):
            at = [want["positions"][i]]
            key = K.norm_rope(qkv[i:i + 1, H:H + Hk], None, 0, cos[at], sin[at]).astype(np.float32)[0]
            for which, x in ((0, key), (1, qkv[i, H + Hk:])):
                host.store(int(want["slots"][i]), which, *K.quantise(x))
        assert np.array_equal(pool.cpu().numpy(), host.raw)
    return calls, check


def main(how):
    if how == "checked":
        calls, check = plan_and_append()
        calls(None)
        L.llm_op_synchronize()
        check()
        for form in FORMS:
            case, mx = case_of(form)
            case.check(case.run(L, mx))
    else:
        # operands need no call that launches: workspace sizes come from the host
        calls, check = plan_and_append()
        cases = [case_of(f) for f in FORMS]
        ops = [c.operands(L, mx) for c, mx in cases]
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            calls(side)
            for a in ops:
                L.llm_op_attention_kv4(*a, stream=side)
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        check()
        for (c, _), a in zip(cases, ops):
            c.check(a[8].float().cpu().numpy().reshape(c.N, c.H, c.d))
    print("CHILD OK", how)


if __name__ == "__main__":
    main(sys.argv[1])
