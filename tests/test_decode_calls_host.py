"""The decode operators' calls without a GPU: what handles and caches say of themselves."""
import pytest
import torch

decode = pytest.importorskip("dense_fp16_gemm_hgemm_amd.decode")
import test_decode_host as host  # noqa: E402


def test_an_inspection_handle_has_no_device():
    with decode.Decode(inspect_only=True) as d:
        assert d.device == decode._device(d.handle) == -1
    assert decode._device(None) == -1


def fused(first, heads, total, hs=64, tokens_apart=None, at=0):
    """Heads first, first + 1, ... of [tokens, total, 64] rows in one buffer."""
    apart = total * 64 if tokens_apart is None else tokens_apart
    return decode._Rows((host.BASE * 9) + 2 * (first * 64 + at), apart, hs)


@pytest.mark.parametrize("k, v, q, status", [
    # 4 query heads, 2 key heads, 2 value heads side by side, in this order and others
    (fused(4, 2, 8), fused(6, 2, 8), fused(0, 4, 8), host.NO_DEVICE),
    (fused(0, 2, 8), fused(2, 2, 8), fused(4, 4, 8), host.NO_DEVICE),
    (fused(6, 2, 8), fused(0, 2, 8), fused(2, 4, 8), host.NO_DEVICE),
    # heads that alternate: 2 queries, a key and a value for each of two groups
    (fused(2, 2, 8, hs=256), fused(3, 2, 8, hs=256), fused(0, 4, 8, hs=64), host.INVALID),
    (fused(4, 2, 8, hs=64), fused(6, 2, 8, hs=64), fused(0, 4, 8, hs=64), host.NO_DEVICE),
    (fused(1, 2, 8, hs=128), fused(8, 2, 16, hs=64), fused(0, 4, 8, hs=128), host.INVALID),  # v of another stride
    (fused(1, 2, 9, hs=128), fused(8, 1, 9, hs=576), fused(0, 4, 9, hs=128), host.NO_DEVICE),  # heads 1 and 3, 8 and the next token's 8, and 0, 2, 4, 6
    # the keys themselves, or some of them
    (fused(0, 2, 8), fused(6, 2, 8), fused(0, 4, 8), host.INVALID),
    (fused(3, 2, 8), fused(6, 2, 8), fused(0, 4, 8), host.INVALID),
    (fused(4, 2, 8), fused(3, 2, 8), fused(0, 4, 8), host.INVALID),
    (fused(4, 2, 8, at=-8), fused(6, 2, 8), fused(0, 4, 8), host.INVALID),
    (fused(4, 2, 8), fused(7, 2, 8), fused(0, 4, 8), host.INVALID),  # v's last head is the next token's first query
])
def test_queries_in_place_hold_no_key_and_no_value(k, v, q, status):
    """Keys and values are read by other workgroups while queries are turned."""
    with decode.Decode(inspect_only=True) as d:
        assert host.append(d.handle, k=k, v=v, q=q, q_out=q) == status


def test_pack_takes_codes_and_zeros_of_four_bits():
    """Numbers outside 0..15 would come back as others."""
    codes, scales = torch.zeros((4, 64), dtype=torch.int32), torch.ones((4, 1)).half()
    codes[1, 2] = 15
    assert decode.w4_unpack(decode.w4_pack(codes, scales, group=64))[1, 2] == 7
    for bad in (16, -1, 300):
        c, z = codes.clone(), torch.full((4, 1), 8)
        c[3, 63] = bad
        z[2, 0] = bad
        with pytest.raises(ValueError, match="codes"):
            decode.w4_pack(c, scales, group=64)
        with pytest.raises(ValueError, match="zeros"):
            decode.w4_pack(codes, scales, z, group=64)
    assert decode.w4_pack(codes[:0], scales[:0], group=64).qweight.shape[0] == 0
