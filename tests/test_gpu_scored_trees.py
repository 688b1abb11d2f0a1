"""Distances in trees whose rows fill more than one block of a work item (tolerances: test_gpu_scored.py)."""
import numpy as np
import pytest

from tests.test_gpu_cache import Batch, tree
from tests.test_gpu_scored import KINDS, alibi, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sc():
    from speculative_decoding_verification_35_gb300 import speccache
    return speccache


@pytest.mark.parametrize("kind,cache", KINDS)
@pytest.mark.parametrize("window", [0, 3, 40])
@pytest.mark.parametrize("group", [9, 16, 43, 128])
def test_trees_of_several_blocks(sc, kind, cache, window, group):
    """256 rows are a block: 28 tokens of 9 heads, 16 of 16, 4 of 43 and 2 of 128."""
    rng = np.random.default_rng(group)
    chunks = [32, 1, 29, 17, 30]
    par = [tree(rng, n) for n in chunks]
    hkv = 1 if group == 128 else 2
    b = Batch(sc, chunks, [200, 3, 120, 0, 96], hkv * group, hkv, 64, 16, kind, cache, parents=par, seed=group)
    check(b, slopes=alibi(hkv * group) * 4, window=window)
    check(b, cap=8.0, slopes=alibi(hkv * group), window=window)
