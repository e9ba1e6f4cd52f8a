"""The bounds of an attention call, without a GPU: a bound beyond what the page
table holds plans the same launch as one that just covers it."""
import os

import pytest
import torch

from test_serving_host import ATT, ATT_OK

lg = pytest.importorskip("epilogue_scaled_gemm_amd")
from epilogue_scaled_gemm_amd import serving  # noqa: E402


@pytest.fixture()
def handle():
    if torch.cuda.is_available():
        pytest.skip("fake-pointer error paths run on the CPU only")
    if not os.path.exists(lg.LIB_PATH):
        pytest.skip("library not built")
    h = lg.Handle()
    yield h
    h.close()


def outcome(h, max_context):
    d = dict(ATT_OK, tokens=4, pages=64, table_stride=512, max_pages=512, max_nodes=2,
             max_context=max_context)
    rc = lg.library().lin_gemm_tree_attention(
        h._h, serving._ATTENTION.pack(*[d.get(n, 0) for n in ATT]), None)
    return rc, lg.library().lin_gemm_last_error(h._h)


def test_a_bound_beyond_the_table(handle):
    # Without a device a call that is split over workgroups fails where it
    # grows the workspace, one that is not where it launches.
    covered = outcome(handle, 512 * 16)
    assert covered != outcome(handle, 1)
    for bound in (512 * 16 + 1, 1 << 40, 2 ** 63 - 3, 2 ** 63 - 2, 2 ** 63 - 1):
        assert outcome(handle, bound) == covered, bound
