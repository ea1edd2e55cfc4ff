"""The decode operators' calls without a GPU: what handles and caches say of themselves."""
import pytest

decode = pytest.importorskip("dense_fp16_gemm_hgemm_amd.decode")


def test_an_inspection_handle_has_no_device():
    with decode.Decode(inspect_only=True) as d:
        assert d.device == decode._device(d.handle) == -1
    assert decode._device(None) == -1
