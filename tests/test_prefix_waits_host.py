"""The limit of the prefix attention's waits and its test hook, host side (no GPU)."""
import pytest

import persistent_monokernel_decode_gb300 as kie


@pytest.fixture(scope="module", autouse=True)
def built():
    kie.build()
    yield


def test_what_is_refused():
    L = kie.lib()
    assert L.kie_paged_set_timeout_ns(0) == kie.KIE_ERR_INVALID and b"above 0" in L.kie_paged_last_error()
    assert L.kie_paged_debug_stop_loads(3, -1) == kie.KIE_ERR_INVALID and b"half" in L.kie_paged_last_error()
    for ns in (0, -1, 1 << 64):
        with pytest.raises(ValueError):
            kie.paged_set_timeout_ns(ns)


def test_what_is_taken():
    kie.paged_set_timeout_ns(1)
    kie.paged_set_timeout_ns(2_000_000_000)
    assert kie.lib().kie_paged_debug_stop_loads(3, 0) == kie.KIE_OK and kie.lib().kie_paged_debug_stop_loads(-1, -1) == kie.KIE_OK
