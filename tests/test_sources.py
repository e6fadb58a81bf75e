"""What the CUDA sources may not name. The library is loaded on every GPU of a replica run, where a TMA load that
multicasts across a cluster is not used; and a CTA that another one's loads or commits still reach could leave first."""

import os

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp4_moe_expert_gb300", "csrc")


def test_no_cta_reaches_into_another():
    for name in sorted(os.listdir(CSRC)):
        src = open(os.path.join(CSRC, name)).read()
        for word in ("multicast", "ClusterDimension", "__cluster_dims__", "mapa.shared::cluster", "%%cluster_"):
            assert word not in src, f"{name} names {word}"
