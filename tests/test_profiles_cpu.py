"""The committed profiles of the scoring kernels and the sources they are tied to: no GPU."""
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("name", ["launch_pdl_cluster", "make_rows_map", "misa_kv_cache_t", "attend"])
def test_what_only_cache_and_attention_use_stays_out_of_the_scorers_headers(name):
    """bench.py reports a scoring kernel's DRAM traffic while the hash of its sources, these headers
    among them, is the profile's: a line there for other kernels takes the figure away."""
    for header in ("common.cuh", "internal.h"):
        with open(os.path.join(ROOT, "long_context_sparse_misa_b200", "csrc", header)) as f:
            assert name not in f.read(), header
