"""The Block_FP8 operators on several streams (GPU)."""
import numpy as np
import pytest
import torch

from tests.block_cases import DEV, codes_on_device, draw_codes, draw_scales, groups, on_device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w8():
    import bit_quantized_gemm_token_amd as mod
    return mod


def gemm_inputs(M, N, K):
    print(f"[case] M={M} N={N} K={K}", flush=True)
    g = np.random.default_rng([M, N, K])
    return [codes_on_device(draw_codes(g, M, K)), on_device(draw_scales(g, M, groups(K))),
            codes_on_device(draw_codes(g, N, K)), on_device(draw_scales(g, groups(N), groups(K)))]


def test_split_calls_overlap_without_a_workspace(w8):
    """Calls that split K, interleaved over two streams and none of them given
    a workspace, equal those that run alone, bit for bit; so do the calls after
    them (every arrival counter is left where the next call needs it)."""
    M, N, K = 48, 512, 7168
    assert w8.block_gemm_workspace_size(M, N, K) > 0
    args = gemm_inputs(M, N, K)
    alone = w8.block_gemm(*args, workspace=w8.Workspace(DEV, 64 << 20))
    small = [args[0][:8], args[1][:8], *args[2:]]
    small_alone = w8.gemm_w8a8("Block_FP8", *small, workspace=w8.Workspace(DEV, 64 << 20))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got, got_small = [], []
    for _ in range(20):
        for st in streams:
            got.append(w8.block_gemm(*args, y=torch.empty_like(alone), stream=st))
            got_small.append(w8.gemm_w8a8("Block_FP8", *small, y=torch.empty_like(small_alone),
                                          stream=st))
    torch.cuda.synchronize()
    got += [w8.block_gemm(*args, stream=st) for st in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(y, alone) for y in got)
    assert all(torch.equal(y, small_alone) for y in got_small)


def test_capture_without_a_workspace_after_eager_calls(w8):
    args = gemm_inputs(48, 512, 2048)
    eager = w8.block_gemm(*args)
    y = torch.empty_like(eager)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w8.block_gemm(*args, y=y)
    for _ in range(4):
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager) and torch.equal(w8.block_gemm(*args), eager)


def _later_fill(like):
    """Frees a tensor of this size and type while the current stream has yet to
    write it: the allocator gives its memory to the stream's next tensor."""
    t = torch.empty_like(like)
    torch.cuda._sleep(100_000_000)
    t.fill_(float("nan"))


def test_default_stream_as_a_handle(w8):
    args = gemm_inputs(200, 512, 512)
    want = w8.block_gemm(*args)
    assert torch.equal(w8.block_gemm(*args, stream=0), want)


@pytest.mark.parametrize("given", ["stream", "handle"])
def test_outputs_belong_to_the_stream_they_are_written_on(w8, given):
    """What the current stream still has to do cannot reach them."""
    st = torch.cuda.Stream()
    stream = st if given == "stream" else st.cuda_stream
    args = gemm_inputs(200, 512, 512)
    x = torch.randn(200, 512, device=DEV).bfloat16()
    w = torch.ones(512, dtype=torch.bfloat16, device=DEV)
    off = torch.tensor([0, 200], dtype=torch.int32, device=DEV)
    experts = args[2].view(torch.uint8)[None].view(torch.float8_e4m3fn)
    calls = [lambda **kw: w8.block_gemm(*args, **kw),
             lambda **kw: w8.grouped_gemm(*args[:2], off, experts, args[3][None], **kw),
             lambda **kw: w8.residual_norm(x, x, w, **kw)[1],
             lambda **kw: w8.block_quantize(x, **kw)[1],
             lambda **kw: w8.linear("Block_FP8", x[:8], *args[2:], **kw)]
    for i, call in enumerate(calls):
        want = call()
        torch.cuda.synchronize()
        _later_fill(want)
        got = call(stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got, want), i


def test_capture_on_a_stream_whose_workspace_is_too_small(w8):
    """What eager calls on another stream have sized is enough for it."""
    args, few = gemm_inputs(100, 1024, 8192), gemm_inputs(40, 256, 1024)
    assert w8.block_gemm_workspace_size(100, 1024, 8192) > \
        w8.block_gemm_workspace_size(40, 256, 1024) > 0
    st = torch.cuda.Stream()
    w8.block_gemm(*few, stream=st)
    eager = w8.block_gemm(*args)
    y = torch.empty_like(eager)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        w8.block_gemm(*args, y=y)
    for _ in range(4):
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager) and torch.equal(w8.block_gemm(*args), eager)
