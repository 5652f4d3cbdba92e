"""Attention over the 4-bit cache where it can go wrong: against the definition in 64 bits, each element within what the
roundings allow, in every variant of the kernels (GPU)."""
import numpy as np
import pytest

from kv4_case import MANY, Case, marked

pytestmark = pytest.mark.gpu

# lens, new, H, Hk, d, P, promised new tokens
FORMS = {
    "8 rows": ([300, 77, 1], [1, 2, 1], 8, 2, 128, 32, None),
    "8 rows d64": ([300, 77, 16], [1, 2, 1], 8, 2, 64, 16, None),
    "16 rows": ([300, 77, 40], [4, 1, 2], 8, 2, 128, 16, None),
    "32 rows": ([300, 177, 40], [8, 1, 5], 8, 2, 128, 64, None),
    "32 rows d64": ([300, 177, 40], [8, 0, 5], 8, 2, 64, 128, None),
    "prompts": ([300, 177, 140], [150, 1, 140], 8, 2, 128, 16, None),
    "prompts d64": ([300, 177, 140], [150, 3, 140], 8, 2, 64, 64, None),
    "expanded": ([300, 177, 140], [150, 1, 140], 8, 2, 128, 16, MANY),
    "expanded d64": ([300, 177, 140], [150, 3, 140], 8, 2, 64, 64, MANY),
}
LONG = {
    "long 8 rows": ([6001, 5], [1, 1], 8, 1, 128, 64, None),
    "long 32 rows": ([5000, 3], [2, 1], 16, 1, 128, 128, None),
    "long 16 rows d64": ([3000, 2500], [2, 4], 4, 1, 64, 16, None),
    "long prompts": ([2600, 40, 300], [70, 1, 129], 4, 2, 128, 64, None),
    "long expanded": ([2600, 40, 300], [300, 1, 129], 4, 2, 128, 64, MANY),
    "long expanded d64": ([1900, 700], [260, 700], 5, 1, 64, 32, MANY),
    "many short": ([37] * 40, [1] * 40, 4, 2, 128, 16, None),
}


@pytest.mark.parametrize("form", list(FORMS) + list(LONG))
def test_each_key_is_summed_once(lib, form):
    """Values that mark their keys: a lost, doubled or wrongly weighted unit, tile or part of a CTA is out of bounds."""
    import llama_decoder_forward_fwd_b200 as L
    lens, new, H, Hk, d, P, mx = (FORMS | LONG)[form]
    case = Case(lens, new, H, Hk, d, P, 5, make=marked(Hk, d, lens), q_scale=0.1, pad=2)
    case.check(case.run(L, mx))


@pytest.mark.parametrize("form", list(FORMS) + list(LONG))
def test_each_element_is_within_the_roundings(lib, form):
    import llama_decoder_forward_fwd_b200 as L
    lens, new, H, Hk, d, P, mx = (FORMS | LONG)[form]
    case = Case(lens, new, H, Hk, d, P, 6, pad=1)
    case.check(case.run(L, mx))


@pytest.mark.parametrize("form", FORMS)
def test_queries_that_are_not_finite_give_nan(lib, form):
    """A NaN or an infinity in a query makes its row NaN, as the definition does, and no other row."""
    import llama_decoder_forward_fwd_b200 as L
    lens, new, H, Hk, d, P, mx = FORMS[form]

    def edit(q):
        q[0, 1, 5] = np.nan
        q[2, 4, :] = np.nan
        q[-1, 0, d - 1] = np.inf
        q[-1, H - 1, 0] = -np.inf
        if len(q) > 40:
            q[40, 2, 7] = np.nan
            q[33, :, 9] = np.inf
    case = Case(lens, new, H, Hk, d, P, 7, edit_q=edit)
    got = case.run(L, mx)
    assert np.isnan(got[0, 1]).all() and np.isnan(got[2, 4]).all()
    case.check(got)


@pytest.mark.parametrize("odd_score", ["inf", "nan"])
@pytest.mark.parametrize("form", FORMS)
def test_one_score_that_is_not_finite_gives_nan(lib, form, odd_score):
    """An infinite query whose scores are -inf but at one place in eight, where they are infinite or (0 * inf) NaN."""
    import llama_decoder_forward_fwd_b200 as L
    lens, new, H, Hk, d, P, mx = FORMS[form]
    places = [at for at in range(8) if lens[0] - new[0] > at]

    for at in places[::3] + [places[-1]]:
        def make(b, which, r):
            if which:
                return None
            x = -np.ones((lens[b], Hk, d), np.float32)
            x[at::8] = 1.0 if odd_score == "inf" else 0.0
            return x

        def edit(q):
            q[:, :, 3] = np.where(np.arange(H)[None] % 3 == 1, np.inf, q[:, :, 3])
        case = Case(lens, new, H, Hk, d, P, 9, make=make, edit_q=edit)
        got = case.run(L, mx)
        assert np.isnan(got[0, 1]).all(), at
        case.check(got, rows=lambda b: np.arange(max(0, at + 1 - (lens[b] - new[b])), new[b]))


@pytest.mark.parametrize("top", [2.0**124, 1e30])
@pytest.mark.parametrize("form", FORMS)
def test_large_finite_values_behind_the_mask_leave_no_trace(lib, form, top):
    """The last new tokens' values are huge: constant groups of 2^124, and groups whose scale passes 2^67. Rows before
    them do not see them."""
    import llama_decoder_forward_fwd_b200 as L
    lens, new, H, Hk, d, P, mx = FORMS[form]
    first = [l - max(1, min(40, n // 2)) if n > 1 else l for l, n in zip(lens, new)]  # the first huge key

    def make(b, which, r):
        if which == 0:
            return None
        x = r.randn(lens[b], Hk, d).astype(np.float32)
        x[first[b]:] = top if top > 1e31 else top * np.arange(1, d + 1, dtype=np.float32)
        return x
    case = Case(lens, new, H, Hk, d, P, 8, make=make)
    case.check(case.run(L, mx), rows=lambda b: np.arange(max(0, new[b] - (lens[b] - first[b]))))
