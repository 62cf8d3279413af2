"""The attention workspace's flag area: zero between calls, and recorded,
not trusted, where it was not zero before one."""
import pytest
import torch

import bit_weight_only_g128_gb300 as w4
from test_gpu_layer import BF16, E4M3, FP16, check_attention, gen, normal, same, scattered

pytestmark = pytest.mark.gpu

FLAGS = 32768


def split_prompt(cache_dtype=FP16, dtype=FP16, D=128):
    """A prompt call whose units are split, its check, and a workspace of zero
    flags with floats of an earlier call behind them."""
    seqs, heads, hk = [(16, 3000), (3, 1400)], 16, 2
    new, lens = [a for a, _ in seqs], [n for _, n in seqs]
    g = gen(31)
    cache, tab = scattered(g, lens, hk, 64, D, cache_dtype)
    starts = [0, 16, 19]
    q = normal(g, 19, heads, D, std=2, dtype=dtype)
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = w4.new_workspace(w4.attn_workspace_size(19, 2, heads, hk, D))
    ws[FLAGS:].view(torch.float32).fill_(1.0)

    def call():
        return w4.attn_prompt(q, cache, tab, st, n, return_lse=True, workspace=ws)

    def check(got, lse):
        check_attention(q, cache, tab, starts, lens, got, lse, D ** -0.5)

    return call, check, ws


@pytest.mark.parametrize("dtype,cache_dtype,D", [(FP16, FP16, 128), (BF16, BF16, 64), (BF16, E4M3, 128)])
def test_what_the_parts_held_before_does_not_matter(dtype, cache_dtype, D):
    call, check, ws = split_prompt(cache_dtype, dtype, D)
    first = None
    for fill in (0x3F800000, -1, 0x7FC00000, 5):
        ws[FLAGS:].view(torch.int32).fill_(fill)
        got, lse = call()
        w4.device_status()
        check(got, lse)
        assert not ws[:FLAGS].any()
        first = first or (got, lse)
        assert same(got, first[0]) and same(lse, first[1])


@pytest.mark.parametrize("parts", [1, -1, 1 << 30, 0x3F800000])
def test_a_count_of_parts_beyond_the_places_is_refused(parts):
    """The last place's count, as no call leaves it: recorded, not followed."""
    call, check, ws = split_prompt()
    want = call()
    w4.device_status()
    places = torch.cuda.get_device_properties(0).multi_processor_count
    ws[:FLAGS].view(torch.int32)[64 + places * 8 - 1] = parts
    got = call()
    with pytest.raises(w4.W4A16Error) as e:
        w4.device_status()
    assert e.value.code == -6 and "0x100" in str(e.value)
    assert not ws[:FLAGS].any()
    assert same(got[0], want[0]) and same(got[1], want[1])
    got, lse = call()
    w4.device_status()
    check(got, lse)


@pytest.mark.parametrize("word,value", [(0, 1), (0, 7), (0, 100000), (0, -5), (2, 3), (3, 1), (3, 1000)])
@pytest.mark.parametrize("split", [True, False])
def test_a_queue_that_was_not_zero_is_recorded(word, value, split):
    """The call has left rows out: it says so, and its buffers and the next
    call with a zero flag area are right."""
    if split:
        call, check, ws = split_prompt()
    else:
        g = gen(32)
        seqs = [(700, 700), (90, 400)]
        lens, starts = [n for _, n in seqs], [0, 700, 790]
        cache, tab = scattered(g, lens, 2, 64, 128, FP16)
        q = normal(g, 790, 8, 128, std=2, dtype=FP16)
        st = torch.tensor(starts, dtype=torch.int32, device="cuda")
        n = torch.tensor(lens, dtype=torch.int32, device="cuda")
        ws = w4.new_workspace(w4.attn_workspace_size(790, 2, 8, 2, 128))

        def call():
            return w4.attn_prompt(q, cache, tab, st, n, return_lse=True, workspace=ws)

        def check(got, lse):
            check_attention(q, cache, tab, starts, lens, got, lse, 128 ** -0.5)

    ws[:FLAGS].view(torch.int32)[word] = value
    call()
    with pytest.raises(w4.W4A16Error) as e:
        w4.device_status()
    assert e.value.code == -6 and "0x100" in str(e.value)
    if word == 0:  # (the blocks that are through were counted right: cleared)
        assert not ws[:FLAGS].any()
    ws[:FLAGS].zero_()
    check(*call())
    w4.device_status()
    assert not ws[:FLAGS].any()


def test_cached_workspaces_are_zero_after_an_error():
    """What a call that gave up may have left in the flag areas of the cached
    workspaces does not reach the next call."""
    call, check, _ = split_prompt()
    seqs, heads, hk, D = [(16, 3000), (3, 1400)], 16, 2, 128
    need = w4.attn_workspace_size(19, 2, heads, hk, D)
    side = torch.cuda.Stream()
    streams = [torch.cuda.current_stream(), side]
    cached = [w4.stream_workspace(need, 0, s.cuda_stream) for s in streams]
    torch.cuda.synchronize()
    for ws in cached:
        ws[:FLAGS].view(torch.int32)[:2000] = 1
    w4.selftest_wait(0)
    with pytest.raises(w4.W4A16Error) as e:
        w4.device_status()
    assert e.value.code == -6
    torch.cuda.synchronize()
    assert [w4.stream_workspace(need, 0, s.cuda_stream) is ws for s, ws in zip(streams, cached)] == [True, True]
    for ws in cached:
        assert not ws[:FLAGS].any()
    w4.device_status()


def test_workspaces_that_the_kernels_cannot_use_are_refused():
    """Host memory, and strided tensors: refused before any launch."""
    g = gen(33)
    cache, tab = scattered(g, [40, 5], 2, 16, 64, FP16)
    q = normal(g, 2, 4, 64, dtype=FP16)
    n = torch.tensor([40, 5], dtype=torch.int32, device="cuda")
    st = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    pw = w4.quantize_pack(normal(g, 1024, 512, std=0.02), 128)
    x = normal(g, 40, 1024, dtype=FP16)
    codes, s = w4.rms_norm(x, normal(g, 1024, dtype=FP16), quant="codes")
    for ws in (torch.zeros(64 << 20, dtype=torch.uint8), w4.new_workspace(128 << 20)[::2]):
        for call in (lambda: w4.attn_decode(q, cache, tab, n, workspace=ws),
                     lambda: w4.attn_prompt(q, cache, tab, st, n, workspace=ws),
                     lambda: w4.gemm(x, pw, path="tensor", parts=4, workspace=ws),
                     lambda: w4.gemm_scaled(codes, s, pw, path="tensor", parts=4, workspace=ws)):
            with pytest.raises(ValueError, match="workspace must be a contiguous CUDA tensor"):
                call()
    w4.device_status()


def test_gemms_on_a_stream_of_their_own():
    """Results and workspace of a stream that has none yet, behind slow work
    on the current one, which their zeros must not wait for."""
    g = gen(34)
    pw = w4.quantize_pack(normal(g, 1024, 512, std=0.02), 128)
    x = normal(g, 40, 1024, dtype=FP16)
    codes, s = w4.rms_norm(x, normal(g, 1024, dtype=FP16), quant="codes")
    calls = [lambda **k: w4.gemm(x, pw, path="tensor", parts=4, **k),
             lambda **k: w4.gemm(x, pw, path="tensor", parts=4, a8=True, **k),
             lambda **k: w4.gemm_scaled(codes, s, pw, path="tensor", parts=4, **k)]
    want = [call() for call in calls]
    big = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for call, y in zip(calls, want):
        own = torch.cuda.Stream()
        for _ in range(10):
            big = big @ big * 1e-3
        got = call(stream=own)
        own.synchronize()
        with torch.cuda.stream(own):
            assert same(got, y)
    w4.device_status()
