"""The committed profiles of the quantiser, the block-scaled product, its training form and the orthogonalised
update were taken from the current kernel sources."""
from __future__ import annotations

import hashlib
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "vocabulary_cross_entropy_row_amd", "csrc")
SHARED = ("ce_device.h", "blocks_internal.h", "linear_mfma.h")
PRODUCT = ("blocks_mfma.h", "blocks_plan.h", "linear_plan.h", "linear_blocks.hip")
SOURCES = {"quantize": SHARED + ("quantize_blocks.hip",), "product": SHARED + PRODUCT,
           "train": SHARED + PRODUCT + ("quantize_blocks.hip", "rms_norm.hip"),
           "ortho": SHARED + ("ortho_plan.h", "orthogonalise.hip")}


def source_hash(operator: str) -> str:
    h = hashlib.sha256()
    for f in SOURCES[operator]:
        with open(os.path.join(CSRC, f), "rb") as fh:
            h.update(f.encode() + b"\0" + fh.read())
    return h.hexdigest()[:16]


@pytest.mark.parametrize("operator", sorted(SOURCES))
def test_profile_is_of_these_sources(operator):
    with open(os.path.join(ROOT, "profiles", "blocks", operator + ".txt")) as f:
        recorded = re.search(r"^kernel_source_sha256_16: (\S+)$", f.read(), re.M)
    assert recorded and recorded.group(1) == source_hash(operator), "taken from other kernel sources: collect it again"
