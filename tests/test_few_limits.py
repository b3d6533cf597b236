"""Sizes past what the few-token kernels count are refused on the host, before
anything is launched (no GPU needed)."""
import pytest

import combine_send_counts_gb300 as ep

P = 4096   # never dereferenced


@pytest.fixture(scope="module")
def lib():
    return ep.load()


@pytest.mark.parametrize("N", [2 ** 31 - 63, 2 ** 31 - 10, 2 ** 31 - 1, 2 ** 31, 2 ** 39])
@pytest.mark.parametrize("K,group", [(32, 32), (64, 64), (128, 128)])
def test_matvec_rows_past_32_bits(lib, N, K, group):
    # a block's last row block counts up to 63 rows past N
    assert lib.ep_w4_matvec(P, 1, P, P, None, N, K, group, P, 0, None) == ep.EP_ERR_UNSUPPORTED


@pytest.mark.parametrize("N,K", [(2 ** 39, 2 ** 28), (2 ** 39 + 1, 2 ** 28), (2 ** 36 + 1, 2 ** 30), (2 ** 40 - 1, 2 ** 20),
                                 (2 ** 32, 4096)])
def test_conversions_of_more_than_a_grid(lib, N, K):
    # the first three's products pass 64 bits: their counts wrapped to 0, 2^25 and below 0
    assert lib.ep_w4_quantize(P, N, K, 128, P, P, None, None) == ep.EP_ERR_UNSUPPORTED
    assert lib.ep_w4_dequantize(P, P, None, N, K, 128, P, 0, None) == ep.EP_ERR_UNSUPPORTED
