"""The number of gate groups that a norm's description means, without a GPU, by the workspace that
the backward pass asks for: a row of sums more for each group."""
import shutil

import pytest

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None, reason="nvcc needed to build")


@pytest.fixture(scope="module")
def z():
    from zero_sharded_mixed_02_gb300 import build
    build.build()
    import zero_sharded_mixed_02_gb300 as z
    z.lib()
    return z


@pytest.mark.parametrize("rows", [1, 4, 1000, (1 << 31) - 1])
@pytest.mark.parametrize("group", [1, 3, 999, 1000, 1001, 1 << 31, (1 << 62) + 1, (1 << 63) - 3, (1 << 63) - 2, (1 << 63) - 1])
def test_groups(z, rows, group):
    """Group sizes up to the type's largest: a group larger than the rows is one group."""
    groups = -(-rows // group)
    size = lambda g: z.zero_norm_workspace(z.norm(1, rows, 64, group_rows=g))  # noqa: E731
    assert size(0) and size(group) == size(0) + (groups - 1) * 2 * 64 * 4


@pytest.mark.gpu
@pytest.mark.parametrize("group", [5, 1 << 32, (1 << 63) - 1])
def test_a_group_larger_than_the_rows(group):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import act_reference as R
    import test_gpu_norm as N
    from zero_sharded_mixed_02_gb300 import build
    build.build()
    import zero_sharded_mixed_02_gb300 as lib
    lib.lib()
    p = N.params(5, 96, R.RMS, R.RMS, group=group)
    N.run_forward((torch, lib), dict(p), R.BF16, R.FP32)
    N.run_backward((torch, lib), dict(p), R.BF16, R.FP32, R.FP32)
