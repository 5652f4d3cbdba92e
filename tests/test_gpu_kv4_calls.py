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
