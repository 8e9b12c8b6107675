"""Barrier arrivals in the sources' inline PTX name the scope that their waiters need."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "dense_fp32_matrix_strict_gb300", "csrc")


def arrivals():
    """(file, instruction) of every mbarrier arrival or wait in the sources."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        with open(path) as f:
            for word in re.findall(r"mbarrier\.(?:arrive|try_wait|test_wait)[\w.:]*", f.read()):
                yield os.path.basename(path), word


def test_arrivals_on_another_ctas_barrier_have_cluster_scope():
    # An arrival of CTA scope orders nothing for a thread of another CTA.
    remote = [(f, w) for f, w in arrivals() if "shared::cluster" in w]
    assert len(remote) >= 2
    for f, w in remote:
        assert ".cluster." in w and ".cta." not in w.replace("shared::cta", ""), (f, w)
