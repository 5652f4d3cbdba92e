"""The append's norms over the whole range of their inputs (GPU)."""
import numpy as np
import pytest
import torch

import kv4_util as K

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128])
def test_norms_of_large_and_small_rows(lib, dtype, d):
    """Rows whose squares pass the range of 32-bit floats, or nearly, beside ordinary ones."""
    import llama_decoder_forward_fwd_b200 as L
    H, Hk, P = 5, 1, 16
    gains = [1.0, 1e18, 3e18, 1e19, 1e25, 1e30, 1e37, 1e-3, 1e-18, 1e-30, 0.0]
    N = len(gains)
    r = np.random.RandomState(d)
    rows = lambda heads: torch.from_numpy((r.randn(N, heads, d) * np.array(gains)[:, None, None]).astype(np.float32)).to(dtype)
    q, k, v = rows(H), rows(Hk), rows(Hk)
    q[0, 1] *= 1e20  # one head among ordinary ones
    w = (1 + 0.2 * r.randn(d)).astype(np.float32)
    cos, sin = K.rope_tables(N, d)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    q_out = torch.zeros(N, H, d, dtype=torch.bfloat16, device="cuda")
    k_out = torch.zeros(N, Hk, d, dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros(1, L.llm_kv4_page_bytes(Hk, d, P), dtype=torch.uint8, device="cuda")
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    L.llm_op_qk_norm_rope_kv4(q.cuda(), k.cuda(), v.cuda(), pos, pos.long(), dev(cos), dev(sin), q_out, pool, P, q_norm=dev(w),
                              k_norm=dev(w), eps=1e-5, k_out=k_out)
    L.llm_op_synchronize()
    want = K.norm_rope(q.double().numpy(), w, 1e-5, cos, sin)
    # bf16 rounds by 2^-8 of a value; a sum of d squares, its root and the rotation in 32 bits, with parts that
    # cancel, by under (d + 16) 2^-24 of a pair's length
    length = np.repeat(np.sqrt(want[..., 0::2] ** 2 + want[..., 1::2] ** 2), 2, -1)
    bound = 2.0**-8 * np.abs(want) + (d + 16) * 2.0**-24 * length + 1e-40
    got = q_out.float().cpu().numpy()
    assert (np.abs(got - want) <= bound).all(), np.argwhere(np.abs(got - want) > bound)[:5]
    key = K.norm_rope(k.double().numpy(), w, 1e-5, cos, sin).astype(np.float32)
    assert np.array_equal(k_out.float().cpu().numpy(), K.values(*K.quantise(key)))
