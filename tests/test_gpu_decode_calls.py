"""Calls of the decode operators that leave arguments out, or name another stream."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu
decode = pytest.importorskip("dense_fp16_gemm_hgemm_amd.decode")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
from dense_fp16_gemm_hgemm_amd import decode_step  # noqa: E402
from test_gpu_decode_attend import check, make, put  # noqa: E402

DEV = torch.device("cuda", 0)


@pytest.fixture(scope="module")
def d():
    h = decode.Decode()
    yield h
    h.close()


@pytest.mark.parametrize("new", [[40, 1, 0, 100], [3, 5, 2, 1]])
def test_ragged_calls_without_a_longest_sequence(d, new):
    """cu alone says how many tokens there are: all of them are appended and all rows are computed."""
    past = [10, 0, 33, 64]
    lens = [p + n for p, n in zip(past, new)]
    cache, table, cu, q = make(lens, new, 8, 2, 64, 16, torch.int8, torch.float16, 61)
    other = decode.KvCache(*[x.clone() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)])
    k, v = (torch.randn((cu[-1], 2, 64), device=DEV).half() for _ in range(2))
    dt = table.to(DEV)
    d.kv_append(cache, k, v, dt, put(past), put(cu))
    d.kv_append(other, k, v, dt, put(past), put(cu), max(new))
    for name in ("k", "v", "k_scale", "v_scale"):
        x, y = getattr(cache, name), getattr(other, name)
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), name
    check(d.kv_attend(q, cache, dt, put(lens), put(cu)), cache, q, table, lens, cu)


def test_kv_read_needs_the_number_of_tokens(d):
    """cu lies on the device: without `tokens` only as many as there are sequences were read."""
    cache = decode.KvCache.empty(8, 2, 64, 16)
    table, start, cu = put([[0, 1], [2, 3]]), put([0, 0]), put([0, 20, 25])
    with pytest.raises(ValueError, match="tokens"):
        d.kv_read(cache, table, start, cu)
    k, v = d.kv_read(cache, table, start, cu, tokens=25)
    assert k.shape == v.shape == (25, 2, 64)
    assert d.kv_read(cache, table, start)[0].shape == (2, 2, 64)


def owner(x):
    """The stream that the allocator keeps a tensor's memory for."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= x.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]


def test_results_belong_to_the_stream_that_is_named(d):
    """Each call with stream= and no out: its memory, and its values beside work on both streams."""
    lens = [300, 41]
    cache, table, cu, q = make(lens, [1, 1], 8, 2, 64, 16, torch.int8, torch.float16, 67)
    w = decode.w4_quantize(torch.randn((256, 512), device=DEV).half())
    x, kv = torch.randn((4, 512), device=DEV).half(), torch.randn((2, 2, 64), device=DEV).half()
    table, rope = table.to(DEV), decode.rope_table(table.shape[1] * 16, 64)
    dl, past = put(lens), put([n - 1 for n in lens])

    def calls(**kw):
        yield "w4_linear", d.w4_linear(x, w.qweight, w.scales, n=256, **kw)
        yield "kv_append", d.kv_append(cache, kv, kv, table, past, q=q, rope=rope, **kw)
        yield "kv_read k", d.kv_read(cache, table, past, **kw)[0]
        yield "kv_read v", d.kv_read(cache, table, past, **kw)[1]
        yield "kv_attend", d.kv_attend(q, cache, table, dl, **kw)

    want = dict(calls())
    busy = torch.randn((2048, 2048), device=DEV)
    side = torch.cuda.Stream()
    for handle in (side, side.cuda_stream):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            busy @ busy
        for name, got in calls(stream=handle):
            assert owner(got) == side.cuda_stream, name
            torch.full_like(got, 7.0)  # on the current stream: not the same memory
            side.synchronize()
            assert torch.equal(got, want[name]), name
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    with pytest.raises(TypeError):
        d.w4_linear(x, w.qweight, w.scales, n=256, stream="side")


def test_a_handle_of_another_device_is_refused(d):
    """Its kernels would run there, with a workspace of that device."""
    cache, table, cu, q = make([20], [1], 8, 2, 64, 16, torch.int8, torch.float16, 71)
    w = decode.w4_quantize(torch.randn((32, 64), device=DEV).half(), 64)
    x, kv, table = torch.zeros((1, 64), device=DEV).half(), torch.zeros((1, 2, 64), device=DEV).half(), table.to(DEV)
    with decode.Decode() as other:
        assert other.device == torch.cuda.current_device() == d.device
        other.device += 1  # as a handle that was made there
        for call in (lambda: other.w4_linear(x, w.qweight, w.scales, n=32, group=64),
                     lambda: other.kv_append(cache, kv, kv, table, put([3])),
                     lambda: other.kv_read(cache, table, put([3])),
                     lambda: other.kv_attend(q, cache, table, put([20]))):
            with pytest.raises(ValueError, match="handle is on cuda"):
                call()


def test_a_cache_keeps_its_tensors(d):
    """Another tensor in its place would be shown by the attribute, and not be what the kernels use."""
    cache = decode.KvCache.empty(4, 2, 64, 16)
    for name in ("k", "v", "k_scale", "v_scale", "pages", "page_size", "device"):
        value = getattr(cache, name)
        with pytest.raises(AttributeError):
            setattr(cache, name, value)
    cache.k_scale.fill_(2.0)  # elements may change
    assert float(cache.k_scale[0, 0]) == 2.0


def test_capturing_a_step_leaves_the_caches_as_they_are():
    """The graph's first input may be anything; what is replayed is what counts."""
    config = decode_step.Config(hidden=256, heads=8, kv_heads=2, head_dim=64, inner=352, layers=2, page_size=16, group=32)
    m = decode_step.Model(config, 3, 60, seed=5)
    cu = put([0, 5, 25, 40])
    x = m.forward(torch.randn((40, 256), device=DEV).half(), cu)[cu[1:].long() - 1]
    state = lambda: [t.clone().view(torch.uint8) for layer in m.layers  # noqa: E731
                     for t in (layer.cache.k, layer.cache.v, layer.cache.k_scale, layer.cache.v_scale)] + [m.lens.clone()]
    before = state()
    g, at, out = m.graph(torch.full_like(x, float("inf")))
    for a, b in zip(before, state()):
        assert torch.equal(a, b)
    at.copy_(x)
    g.replay()
    torch.cuda.synchronize()
    assert torch.isfinite(out).all() and m.lens.tolist() == [6, 21, 16]
    m.close()


def test_strides_of_single_elements_do_not_matter(d):
    """One token, one key-value head and one sequence, cut from tensors of odd strides."""
    cache, table, cu, q = make([50], [1], 4, 1, 64, 16, torch.int8, torch.float16, 73)
    kv, rope = torch.randn((1, 1, 64), device=DEV).half(), decode.rope_table(table.shape[1] * 16, 64)
    table, lens, past = table.to(DEV), put([50]), put([49])

    def odd(x, *strides):
        room = torch.zeros(x.numel() + 8, dtype=x.dtype, device=DEV)
        y = room.as_strided(x.shape, strides)
        return y.copy_(x)

    q_out = torch.empty((1, 4, 64), device=DEV).half()
    want = d.kv_append(cache, kv, kv, table, past, q=q, rope=rope)
    got = d.kv_append(cache, odd(kv, 67, 3, 1), odd(kv, 5, 1, 1), odd(table, 3, 1), odd(past, 9), q=odd(q, 1, 64, 1),
                      rope=rope, q_out=odd(q_out, 13, 64, 1))
    assert torch.equal(got, want)
    want = d.kv_attend(q, cache, table, lens)
    assert torch.equal(d.kv_attend(odd(q, 7, 64, 1), cache, odd(table, 0, 1), odd(lens, 11), out=odd(q_out, 3, 64, 1)), want)
    first = odd(table[:, :1], 6, 5)  # a table of one page
    for a, b in zip(d.kv_read(cache, table, put([7])), d.kv_read(cache, first, odd(put([7]), 4))):
        assert torch.equal(a, b)


def test_an_earlier_error_of_the_runtime_is_not_a_calls_own(d):
    """The last error that the runtime keeps may come from anywhere; a launch has a status of its own."""
    with open("/proc/self/maps", encoding="utf-8") as f:
        hip = ctypes.CDLL(next(line.split()[-1] for line in f if "libamdhip64" in line))
    cache, table, cu, q = make([50], [1], 4, 1, 64, 16, torch.int8, torch.float16, 79)
    w = decode.w4_quantize(torch.randn((32, 64), device=DEV).half(), 64)
    x, y, out = torch.zeros((1, 64), device=DEV).half(), torch.ones((1, 32), device=DEV).half(), torch.empty_like(q)
    table, lens = table.to(DEV), put([50])
    want = d.kv_attend(q, cache, table, lens)
    torch.cuda.synchronize()
    try:
        assert hip.hipSetDevice(99) != 0  # a refused call, which the runtime remembers
        d.w4_linear(x, w.qweight, w.scales, n=32, group=64, out=y)
        d.kv_append(cache, x.view(1, 1, 64), x.view(1, 1, 64), table, lens)
        d.kv_attend(q, cache, table, lens, out=out)
    finally:
        hip.hipGetLastError()
    torch.cuda.synchronize()
    assert torch.all(y == 0) and torch.equal(out, want)


def test_more_rows_than_a_launch_can_have_are_unsupported(d):
    w = decode.w4_quantize(torch.randn((1, 8), device=DEV).half(), 32)
    x = torch.zeros((64 * 65535 + 1, 8), device=DEV).half()
    with pytest.raises(decode.DecodeError) as e:
        d.w4_linear(x, w.qweight, w.scales, n=1, group=32)
    assert e.value.status == decode.MI_DECODE_ERR_UNSUPPORTED
    assert torch.all(d.w4_linear(x[1:], w.qweight, w.scales, n=1, group=32) == 0)


def test_steps_past_the_page_table_are_refused():
    """Their tokens would be skipped, and the output computed without them."""
    config = decode_step.Config(hidden=256, heads=8, kv_heads=2, head_dim=64, inner=352, layers=1, page_size=16, group=32)
    m = decode_step.Model(config, 2, 30, seed=7)
    x = m.forward(torch.randn((31, 256), device=DEV).half(), put([0, 30, 31]))[[29, 30]]
    for _ in range(2):
        x = m.forward(x)
    with pytest.raises(ValueError, match="32 tokens"):
        m.forward(x)
    with pytest.raises(ValueError, match="32 tokens"):
        m.forward(torch.randn((33, 256), device=DEV).half(), put([0, 0, 33]))
    assert m.lens.tolist() == [32, 3]
    m.close()
