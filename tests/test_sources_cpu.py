"""What the kernel sources may not contain."""
import glob
import os
import re

from transformer_scaled_dot_mha_gb300 import build


def test_no_load_is_multicast_to_a_cluster():
    """Every tile is copied by the CTA that reads it: ranks of one node share nothing but the
    barrier of the bench. (Commits of MMAs may arrive in both CTAs of a pair.)"""
    files = [f for kind in ("*.cu", "*.cuh", "*.h") for f in glob.glob(os.path.join(build.CSRC, kind))]
    assert files
    for f in files:
        with open(f) as src:
            text = re.sub(r'"\s*"', "", src.read())  # adjacent string literals are one
        for op in re.findall(r"cp\.async\.bulk[\w.:]*", text):
            assert "multicast" not in op, (f, op)
