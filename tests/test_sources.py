"""What the kernels' sources must not hold.  No GPU needed."""
import glob
import os

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_copy_is_multicast_over_a_cluster():
    """Every rank of a run on several GPUs loads this library, and a workspace is the caller's: a
    copy that reaches into other CTAs' shared memory is only for memory known to be this GPU's."""
    sources = glob.glob(os.path.join(ROOT, "ternary_weight_dp4a_gb300", "csrc", "**", "*.cu*"), recursive=True)
    assert len(sources) > 10
    for path in sources:
        assert "multicast" not in open(path).read(), path
