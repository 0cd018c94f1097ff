"""What the kernels for long contexts and few rows may have in flight, and wait
for: read from their sources, or worked through on the CPU (a missing wait is
nothing to try on a GPU)."""
import glob
import os
import re

import mla_attention_nvfp4_gb300 as mla

CSRC = os.path.join(os.path.dirname(mla.__file__), "csrc")


def code_of(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_no_copy_or_commit_reaches_another_ctas_shared_memory():
    # the library is every rank's, whatever memory a cache lies in; and a commit that arrives in another CTA may find it ended
    names = [os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*.c*")) + glob.glob(os.path.join(CSRC, "*.h"))]
    assert "fp8_weights.cu" in names
    for name in names:
        assert "multi" + "cast" not in code_of(name), name
