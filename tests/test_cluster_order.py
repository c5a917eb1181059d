"""Order between the CTAs of a cluster, by the kernels' sources.

A CTA that zeroes value rows by ordinary stores tells the CTA that issues the product over both CTAs' memory.  An
mbarrier arrival without a scope orders within its CTA only, so that signal has to be a release at cluster scope,
and the wait for it an acquire at that scope; a run on a device shows nothing as long as the hardware is kind.
"""
import pathlib
import re

import pytest

CSRC = pathlib.Path(__file__).resolve().parents[1] / "sparse_attention_paged_dsa_gb300" / "csrc"


@pytest.mark.parametrize("name, bar", [("mla_tree_kernel.cu", "vz_ready"), ("mla_tree_pair_kernel.cu", "vz_ready"),
                                       ("mla_prefill_kernel.cu", "tail_ready")])
def test_zeroed_rows_are_signalled_at_cluster_scope(name, bar):
    text = re.sub(r"//.*", "", (CSRC / name).read_text())
    uses = [m.start() for m in re.finditer(r"ctl\.%s\[" % bar, text)]
    calls = {re.findall(r"\b(mbar_\w+|wait\w*)\((?:cluster_addr\()?&?$", text[:at])[-1] for at in uses
             if re.search(r"\b(mbar_\w+|wait\w*)\((?:cluster_addr\()?&?$", text[:at])}
    assert calls - {"mbar_init"} == {"mbar_arrive_cluster", "mbar_wait_cluster"}
    assert len(uses) >= 3
