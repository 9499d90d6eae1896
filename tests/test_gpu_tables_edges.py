"""pa_build_tables where a step's places, blocks or sequences run out."""
import os
import sys

import numpy as np
import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_gpu_tables import compare, make, oracle_of, run  # noqa: E402
from tree_harness import random_parents  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tree", [False, True])
def test_idle_sequences_behind_the_last_token_place(pa, cuda_device, tree):
    """Sequences whose tokens pass the arrays' end get nothing; idle ones behind them keep their contexts."""
    rng = np.random.default_rng(8)
    for S in (2, 20, 700):
        h = make(rng, S, 40, 0, 9, 16, tree, spare_blocks=4)
        h["new_lens"][0], h["new_lens"][-1] = 8, 0
        N = 4 if S == 2 else int(h["new_lens"].sum()) // 2
        if tree:
            h["parents"] = np.array([x for n in h["new_lens"] for x in random_parents(rng, int(n))], dtype=np.int32)
        want = oracle_of(h, N)
        assert want["context_lens"][-1] == h["context_lens"][-1] > 0 and 0 in want["context_lens"]
        compare(run(pa, cuda_device, h, N, 1), want, 1, f"S={S}")
        assert pa.pa_get_error() == pa.PA_DEVERR_QUERY
