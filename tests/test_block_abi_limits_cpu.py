"""Arguments of the entry points around the feed-forward products at the edge of what
they take, checked on the host (fake pointers, never dereferenced)."""
import pytest

import mlp_megakernel_amd as mk
from test_block_abi_cpu import DEV, INV, NORM, _without_gpu, call  # noqa: F401 (the fixture: these need no GPU)


@pytest.mark.parametrize("eps,status", [(0.0, DEV), (1e-50, DEV), (3.4e38, DEV), (3.5e38, INV), (1e300, INV)])
def test_eps_is_a_number_of_fp32(eps, status):
    assert call("coalesce_layer_norm", NORM, dict(eps=eps)) == status
