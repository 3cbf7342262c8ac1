"""Draft rows that do not count are not read (a sequence's first one may lie in front of the caller's memory): the order in the
kernel's text, since what a kernel reads and drops shows in no result."""
import re

from test_cluster_starts import kernels


def test_a_draft_row_is_read_after_it_is_known_to_count():
    body = kernels("qmm_verify.cu")["verify_stats"]
    given_up = re.search(r"if \(draft\) \{[^}]*return;", body)
    assert given_up and given_up.end() < body.index("load4<")
