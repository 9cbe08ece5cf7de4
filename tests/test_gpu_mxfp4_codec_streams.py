"""The MXFP4 quantiser captured, replayed on new values, on two streams at once and on one
other than its tensors', bit for bit against calls in a row."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _values(seed, shape, dtype):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, device="cuda", generator=g) * 10).to(dtype)


@pytest.mark.parametrize("shape", [(1, 32), (7, 1, 96), (300, 2880), (2, 129, 256)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_captured(shape, dtype):
    import torch
    from mxfp8_grouped_gemm_x32_b200 import mxfp4
    dtype = getattr(torch, dtype)
    x = _values(1, shape, dtype)
    mxfp4.dequantize(*mxfp4.quantize(x), dtype)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        codes, scales = mxfp4.quantize(x)
        back = mxfp4.dequantize(codes, scales, dtype)
    for seed in (2, 3):
        x.copy_(_values(seed, shape, dtype))
        codes.fill_(77)
        scales.fill_(77)
        graph.replay()
        torch.cuda.synchronize()
        c, s = mxfp4.quantize(x)
        assert torch.equal(codes, c) and torch.equal(scales, s) and torch.equal(back, mxfp4.dequantize(c, s, dtype))


def test_two_streams():
    import torch
    from mxfp8_grouped_gemm_x32_b200 import mxfp4
    xs = [_values(4, (2000, 1024), torch.bfloat16), _values(5, (999, 2880), torch.float32)]
    want = [mxfp4.quantize(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for _ in range(20):
        for n, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[n].append(mxfp4.quantize(xs[n]))
    torch.cuda.synchronize()
    for outs, (c, s) in zip(got, want):
        assert all(torch.equal(a, c) and torch.equal(b, s) for a, b in outs)
