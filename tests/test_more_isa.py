"""The gated product's and the adapters' tile kernels issue the same matrix
instructions from inline asm as the plain product's; their listings keep the wait
states that the compiler cannot see there."""
import os

import pytest

from test_isa import CSRC, _asm, _bodies
from test_llm_isa import matrix_hazards


@pytest.mark.parametrize("source", ["tq_gated.hip", "tq_adapters.hip"])
def test_products_from_asm_wait(source, tmp_path):
    listing = _asm(os.path.join(CSRC, source), str(tmp_path))
    names = [n for n, body in _bodies(listing) if "k_epi_ring" in n and any(b.startswith("v_mfma_i32") for b in body)]
    assert len(names) == 12                  # three types, four tiles and rings
    # the adapters' products in float are the compiler's own, with its waits; to
    # the instructions from asm they count as any other reader or writer
    hits = matrix_hazards(listing.replace("v_mfma_f32", "v_float_product"), "k_epi_ring")
    assert not hits, "\n".join("%s\n    %s\n    %s" % h for h in hits[:10])
