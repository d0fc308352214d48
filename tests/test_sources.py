"""What the kernels' sources must not hold.  No GPU needed."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_copy_is_multicast_over_a_cluster():
    """Every rank of a run on several GPUs loads this library, and a workspace is the caller's: a
    copy that reaches into other CTAs' shared memory is only for memory known to be this GPU's."""
    sources = glob.glob(os.path.join(ROOT, "ternary_weight_dp4a_gb300", "csrc", "**", "*.cu*"), recursive=True)
    assert len(sources) > 10
    for path in sources:
        assert "multicast" not in open(path).read(), path


def test_what_earlier_work_writes_is_not_read_as_read_only():
    """The expert layer's kernels start before the work ahead of them in the stream has ended, so
    its outputs are not read-only while they run: no const __restrict__ and no __ldg but for weights."""
    weights = {"gamma", "wsp + b0"}
    seen = 0
    for path in glob.glob(os.path.join(ROOT, "ternary_weight_dp4a_gb300", "csrc", "tq_moe_*.cu*")):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        inputs = re.findall(r"const \w+ \*__restrict__ (\w+)", text)
        inputs += re.findall(r"__ldg\((?:reinterpret_cast<const \w+ \*>\()?([^()]*)\)", text)
        inputs += ["hist"] * len(re.findall(r"int \*__restrict__ hist, int chunks", text))   # read and written
        seen += len(inputs)
        assert set(inputs) <= weights, (path, inputs)
    assert seen == 2
