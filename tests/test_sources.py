"""What the kernels' sources may not hold."""
import glob
import os

from conftest import ROOT


def test_no_load_into_several_ctas():
    """Each CTA loads for itself alone: the library is also what the replicas of a run
    on several GPUs load, and operands may then be another GPU's memory."""
    word = "multi" + "cast"
    found = []
    for pattern in ("csrc/*.cu", "csrc/*.cuh", "csrc/*.h", "csrc/*.cpp"):
        for f in glob.glob(os.path.join(ROOT, "gated_delta_rule_44_gb300", pattern)):
            with open(f) as fh:
                if word in fh.read().lower():
                    found.append(os.path.basename(f))
    assert not found
