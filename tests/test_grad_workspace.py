"""Workspace of the gradient norm for lists of any length (on the host)."""
import pytest

import microscaling_quantized_convolution_mx_amd as mx


@pytest.mark.parametrize("count", [1, 95, 96, 97, 1000, 2 ** 20, 2 ** 31 - 96, 2 ** 31 - 95, 2 ** 31 - 1])
def test_workspace_grows_with_the_list(count):
    """8 KiB for every 96 tensors."""
    assert mx.mx_grad_workspace_bytes(count) == (count + 95) // 96 * 8192
