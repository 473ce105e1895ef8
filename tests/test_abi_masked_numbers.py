"""Numbers beyond 32 bits at the bindings of the windowed and the tree attention (no GPU)."""
import pytest

import fp8_paged_kv_kvq_gb300 as kvq

SIZE = dict(num_requests=3, rows_per_request=2, num_q_heads=8, num_kv_heads=8, head_dim=128, block_size=16)


@pytest.mark.parametrize("window,sinks", [(2 ** 31, 0), (2 ** 32, 0), (2 ** 32 + 5, 2 ** 32 + 5), (2 ** 63 + 2 ** 31, 2 ** 31)])
def test_large_windows_and_sinks_mean_all_tokens(window, sinks):
    size = kvq.paged_decode_window_workspace_size
    assert size(**SIZE, max_context_len=100, window=window, num_sinks=sinks) == \
        size(**SIZE, max_context_len=100, window=100) > 0


@pytest.mark.parametrize("most", [2 ** 30 + 1, 2 ** 31, 2 ** 32 + 100, 2 ** 40])
def test_contexts_too_long_are_refused(most):
    assert kvq.paged_decode_window_workspace_size(**SIZE, max_context_len=most, window=9) == 0
    assert kvq.paged_decode_tree_workspace_size(**SIZE, max_context_len=most) == 0


def test_negative_numbers_stay_negative():
    for bad in (dict(window=-2 ** 32 + 5), dict(window=9, num_sinks=-2 ** 32 + 5)):
        assert kvq.paged_decode_window_workspace_size(**SIZE, max_context_len=100, **bad) == 0
    assert kvq.paged_decode_tree_workspace_size(**SIZE, max_context_len=-2 ** 32 + 100) == 0
