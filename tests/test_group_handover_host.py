"""Host check of csrc/gemm_group.cuh: what a thread writes into shared memory
for the tensor cores is handed over inside the CTA whose thread issues the MMA.
An arrival on the other CTA's barrier releases within its own CTA only, so it
may free an accumulator but never announce such writes."""
import os

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tiled_dense_gemm_tma_b200", "csrc")


def test_cleared_rows_are_announced_within_the_leader():
    with open(os.path.join(CSRC, "gemm_group.cuh")) as f:
        text = f.read()
    plain = [line.strip() for line in text.splitlines() if "mbar_arrive_cluster(" in line]
    assert len(plain) == 1 and "tempty" in plain[0]
    # the rows behind a group: cleared by the leader alone, fenced, then an arrival on its own barrier
    part = text[text.index("fix-up (WG, leader only)"):]
    order = [part.index(s) for s in ("rank == 0", "clear_cluster(", "fence_proxy_async_cluster();", "mbar_arrive_two(&full[s]);")]
    assert order == sorted(order)
    assert "mapa" not in text[text.index("void mbar_arrive_two"):][:200]
