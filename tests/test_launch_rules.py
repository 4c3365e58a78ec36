"""Rules of the sources that no run can show to hold."""

import glob
import os
import re


def test_kernels_that_leave_bulk_writes_in_flight_let_no_launch_in_early(repo_root):
    """A kernel may end before its last bulk writes are done (bulk_wait_group_read_all) only where it has not let the
    next launch start early."""
    seen = 0
    for path in glob.glob(os.path.join(repo_root, "blockwise_exact_attention_gb300", "csrc", "*.cu")):
        with open(path) as f:
            source = f.read()
        if "bulk_wait_group_read_all()" not in source:
            continue
        for line in re.findall(r"^.*\bgrid_launch_dependents\(\).*$", source, re.M):
            assert line.strip() == "if (p.pdl_next) grid_launch_dependents();", (path, line)
            seen += 1
        for at in re.finditer(r"bulk_wait_group_read_all\(\)", source):
            assert "if (p.pdl_next) bulk_wait_group_all();" in source[at.start() - 120:at.start()], path
    assert seen == 2                                        # the forward and the backward
