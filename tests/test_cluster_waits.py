"""What a CTA reads of its peers' stores it reads behind a wait that acquires at
cluster scope (a wait of CTA scope does not order them; no run shows that
reliably, so this looks at the source)."""
import os
import re

import pytest

from helpers import ROOT

CSRC = os.path.join(ROOT, "grouped_gemm_top_gb300", "csrc")


@pytest.mark.parametrize("name", sorted(n for n in os.listdir(CSRC) if n.endswith(".cu")))
def test_waits_for_peers(name):
    with open(os.path.join(CSRC, name)) as f:
        src = f.read()
    # barriers that another CTA's st.async counts its bytes on: the last operand
    remote = set()
    for at in re.finditer(r"st\.async\.", src):
        operands = src[at.start():src.index(";", src.index('"memory"', at.start()))]
        remote |= set(re.findall(r"mapa\((\w+)\(", operands))
    for bar in remote - {"smem_u32"}:
        waits = re.findall(r"(mbar_wait\w*)\(" + bar + r"\(", src)
        assert waits and set(waits) == {"mbar_wait_cluster"}, (name, bar, waits)
    if name == "distill.cu":
        assert "xbar" in remote
