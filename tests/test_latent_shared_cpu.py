"""Workspaces of kda_latent_decode_shared: what the kernels of a call use, and no more."""
import pytest

from kimi_delta_attention_varlen_gb300 import _abi


@pytest.mark.parametrize("dl", [256, 512])
@pytest.mark.parametrize("L,h", [(1, 64), (1, 128), (2, 32), (4, 128), (64, 1)])
def test_entries_of_64_rows_need_what_the_plain_call_needs(dl, L, h):
    """They are the plain kernel's in any batch, which keeps no sums a query row."""
    lib = _abi.lib()
    for batch, groups in ((1, 1), (512, 7), (4096, 512)):
        assert lib.kda_latent_decode_shared_workspace_size(batch, groups, L, h, dl, 64) == lib.kda_latent_decode_workspace_size(batch, L, h, dl, 64)


@pytest.mark.parametrize("dl", [256, 512])
@pytest.mark.parametrize("L,h", [(1, 1), (1, 63), (3, 21), (63, 1)])
def test_entries_of_fewer_rows_keep_a_sum_a_query_row(dl, L, h):
    lib = _abi.lib()
    few, many = (lib.kda_latent_decode_shared_workspace_size(b, 4, L, h, dl, 64) for b in (256, 512))
    assert many - few >= 256 * L * h * (4 * dl + 16)
    assert few >= lib.kda_latent_decode_workspace_size(256, L, h, dl, 64) + 256 * L * h * (4 * dl + 16)
