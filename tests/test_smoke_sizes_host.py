"""The block smoke's product is one that CTA pairs take: its 128 x 128 tiles
would need a second wave of the one-CTA kernel (the rule of dmuon_mxfp4_gemm)."""
import pytest

import __graft_entry__ as entry


@pytest.mark.parametrize("sms", [132, 148, 152, 160])
def test_large_product_takes_cta_pairs(sms):
    rows, cols, n = entry._block_sizes(sms)
    assert rows > 128 and n > 128
    assert -(-rows // 128) * -(-n // 128) > sms
