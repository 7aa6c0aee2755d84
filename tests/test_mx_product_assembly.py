"""The built kernels of MXFP4 products with an epilogue and of experts' products keep the wait states of the matrix instruction, as
tests/test_mx_assembly.py checks them for the plain product, and write their sums to LDS only behind them."""
import os
import re

import pytest

from tests.test_mx_assembly import OBJDUMP, hazards, listing_of

fp4 = pytest.importorskip("block_scaled_fp4_w4a16_amd")


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump of ROCm")
def test_matrix_instructions_keep_their_wait_states(tmp_path):
    texts = [t for t in listing_of(fp4.LIB_PATH, tmp_path) if "product_kernelINS_4Tile" in t]
    # three tiles with an epilogue; four of rows in groups and two of groups' depths; three output types each
    counts = sorted(len(re.findall(r"<_ZN2mx14product_kernelINS_4Tile\S+>:", t)) for t in texts)
    assert counts == [9, 18]
    for text in texts:
        count, bad = hazards(text)
        assert count > 900 and not bad, bad[:5]
