"""Counts next to 2^31: the kernels count blocks past the last row or key in 32 bits, so these are refused
before any launch (the pointers are never followed)."""
import pytest

from test_serving_ops_cpu import ARG, SHAPE, _prefix, _prompt, _verify

TOP = 2**31 - 1


@pytest.mark.parametrize("n", [TOP, TOP - 63, TOP - 127, TOP - 1022])
def test_counts_that_kernels_cannot_pass_in_32_bits(n):
    one = dict(H=1, Hk=1, sq=128, sk=128, sv=128, so=128, hd=128)
    for dtype in (0, 1):
        assert _prompt(**one, dtype=dtype, n_kv=n) == SHAPE
        assert _prompt(**one, dtype=dtype, n_q=n, n_kv=n) == SHAPE
        few = dict(H=1, Hk=1, sq=128, so=128, dtype=dtype, n_rows=1, n_groups=1)
        assert _prefix(**few, n_prefix=n, n_tail=0) == SHAPE
        assert _prefix(**few, n_prefix=n - 9, n_tail=9) == SHAPE
        assert _prefix(**few, n_prefix=TOP, n_tail=TOP) == SHAPE
    assert _verify(V=1, sp=1, sq=1, n=1, k=n - 1) == ARG
    assert _verify(V=1, sp=1, sq=1, n=TOP, k=TOP) == ARG


def test_counts_below_pass_the_host_checks():
    """Nothing to do is answered before the sizes of an empty call matter; one below the bound is not refused."""
    assert _prompt(n_kv=TOP - 1023, n_q=0) == 0
    assert _prefix(n_prefix=TOP - 1023, n_tail=0, n_groups=0) == 0
    assert _verify(n=0, k=TOP - 1023) == 0
