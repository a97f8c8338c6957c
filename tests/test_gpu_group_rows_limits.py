"""gemm_group_rows where its shared memory reaches what a kernel may have."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,sizes", [(500, range(364, 373)), (3000, range(302, 311))])
def test_counters_at_the_default_limit_of_shared_memory(rows, sizes):
    """33 counters a group (and 2048 sums beyond 2048 rows) reach 48 KiB between these numbers
    of groups.  A process of its own: another call with more groups raises the limit."""
    child = f"""
import numpy as np, torch
import dense_gemm_08_gb300 as lib
from test_gpu_group_rows import expected
for groups in {list(sizes)}:
    ids = np.random.default_rng(groups).integers(-1, groups, {rows}).astype(np.int32)
    got = lib.group_rows(torch.from_numpy(ids).cuda(), groups)
    for g, e in zip(got, expected(ids, groups)):
        assert np.array_equal(g.cpu().numpy(), e), groups
"""
    here = os.path.dirname(os.path.abspath(__file__))
    path = os.pathsep.join([here, os.path.dirname(here), os.environ.get("PYTHONPATH", "")])
    r = subprocess.run([sys.executable, "-c", child], env=dict(os.environ, PYTHONPATH=path),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
