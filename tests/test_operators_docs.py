"""The package's documentation names every operator around the allreduce."""
import pytest

NAMES = ["sar_layer_norm", "sar_layer_norm_backward", "sar_layer_norm_backward_workspace_bytes", "sar_expert_rows",
         "sar_expert_sort", "sar_expert_dispatch", "sar_expert_combine", "sar_expert_combine_backward"]


@pytest.mark.parametrize("name", NAMES)
def test_the_package_lists(name):
    import allreduce_reduction_rank_gb300 as sar
    assert callable(getattr(sar, name))
    assert f":func:`{name}`" in sar.__doc__
