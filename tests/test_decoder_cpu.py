"""The decoder example's report of a step that went wrong on the device."""
import pytest

import w4a4_quantized_gemm_gb300 as w4
from w4a4_quantized_gemm_gb300 import decoder


def test_the_status_that_is_read_is_the_one_that_is_raised(monkeypatch):
    """Reading the device status clears it."""
    words = [w4.W4A4_ERR_INDEX]
    monkeypatch.setattr(w4, "w4a4_device_status", lambda: words.pop() if words else 0)
    with pytest.raises(w4.W4A4Error) as e:
        decoder.check_status("decoder step")
    assert e.value.status == w4.W4A4_ERR_INDEX
    decoder.check_status("decoder step")
