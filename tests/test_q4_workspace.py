"""What the 4-bit cache leaves as it was for the bf16 entry points, without a GPU: the size of a
workspace, and the kernels that the recorded DRAM counters belong to."""
import pytest

import bench
from block_sparse_long_resa_b200 import build as B
from block_sparse_long_resa_b200 import resa as R


@pytest.mark.parametrize("batch,pages", [(1, 16400), (4, 4100)])
def test_a_chunk_workspace_is_the_rectifications(batch, pages):
    """32 rows of 28 / 4 heads: the rectification keeps a partial row group for each SM that divides
    among the (sequence, kv head)s; the 4-bit chunk attention may add one for each of these."""
    B.build()
    cfg = R.make_config(28, 4, 128, 16)
    most = (148 + 4 * batch) * 256 * (128 + 2) * 4 + 1024
    assert R.resa_workspace_size(cfg, batch, pages, 32) - R.resa_workspace_size(cfg, batch, pages, 0) <= most


def test_dram_records_are_of_these_kernels():
    """A record of a kernel whose sources changed is reported as no traffic at all: measure it again."""
    for name in ("decode_step_dram_traffic.json", "sparse_decode_dram_traffic.json"):
        traffic, source = bench.kernel_dram_traffic(name)
        assert traffic, source
