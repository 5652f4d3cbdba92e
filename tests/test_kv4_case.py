"""What the bound of tests/kv4_case.py can see (CPU)."""
import numpy as np
import pytest

from kv4_case import Case, marked
import kv4_util as K


@pytest.mark.parametrize("lens,new,H,Hk,d,P", [([6001], [1], 8, 1, 128, 64), ([700], [150], 4, 2, 64, 32)])
def test_a_missing_or_doubled_key_fails_the_bound(lens, new, H, Hk, d, P):
    """With values that mark their keys, one key left out of a row is more than the roundings allow."""
    case = Case(lens, new, H, Hk, d, P, 1, make=marked(Hk, d, lens), q_scale=0.1)
    want, bound = case.want(0)
    for key in (0, 15, 16, 333, lens[0] - new[0], lens[0] - new[0] - 1):
        less, _ = case.want(0, drop=[key])
        # where a key is left out, one is counted twice by as much with the other sign
        assert (np.abs(less - want) > bound).any(-1).all(), key


def test_random_values_show_a_lost_part():
    case = Case([6001], [1], 8, 1, 128, 64, 2)
    want, bound = case.want(0)
    less, _ = case.want(0, drop=np.arange(1024, 1088))
    assert (np.abs(less - want) > bound).any(-1).all()


def test_the_definition_agrees_with_the_row_by_row_one():
    case = Case([90, 33], [7, 33], 4, 2, 64, 16, 3)
    for b in range(2):
        q = case.q[case.q_start[b]:case.q_start[b + 1]].double().numpy()
        want, _ = case.want(b)
        assert np.abs(want - K.attention(q, *case.kv[b], case.new[b])).max() < 1e-12
    pool = K.Pool(case.n_pages, 2, 64, 16)
    pool.raw = case.pool
    for which in (0, 1):
        assert np.array_equal(pool.keys(case.table[0], 90, which), case.kv[0][which])
