"""PA_OPT_WRITE_OVERLAP is off unless asked for and takes 0 or 1 (no GPU)."""
from __future__ import annotations


def test_values(pa_lib):
    from paged_kv_cache_42_gb300 import binding
    assert binding.OPTIONS["write_overlap"] == 9
    for v in (2, -1):
        assert pa_lib.pa_set_option(9, v) == -1  # PA_ERR_INVALID_ARG
    assert pa_lib.pa_set_option(9, 1) == 0
    assert pa_lib.pa_set_option(9, 0) == 0
