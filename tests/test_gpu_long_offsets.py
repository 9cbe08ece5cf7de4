"""Arrays whose offsets pass 32 bits, batches of many tokens per lane, and sums
over the ranks of a data-parallel job: the same rows in a small call are the
reference, bit for bit."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.empty_cache()


def _randn(g, *shape, dtype):
    """Normal values made in pieces (a whole fp32 copy is not needed)."""
    import torch
    out = torch.empty(*shape, dtype=dtype, device="cuda")
    for part in out.view(-1).split(1 << 28):
        part.copy_(torch.randn(part.numel(), device="cuda", generator=g))
    return out


def _layer(T, E, k):
    from mxfp8_grouped_gemm_x32_b200.layer import GroupedMLP
    return GroupedMLP(T, 32, 64, E, k, backward=False, mxfp8=False)


@pytest.mark.parametrize("E,k", [(256, 8), (250, 9)])
def test_router_past_32_bits(E, k):
    import torch
    from mxfp8_grouped_gemm_x32_b200 import lib
    T, n = 8_700_000, 300                           # T E > 2^31
    g = torch.Generator(device="cuda").manual_seed(E)
    z = _randn(g, T, E, dtype=torch.bfloat16)
    dp, dl = torch.randn(T, k, device="cuda", generator=g), torch.tensor([0.3, 0.1], device="cuda")
    big = _layer(T, E, k)
    idx, prob, losses = big.route_losses(z)
    grad = big.route_backward(z, dp, dl)
    assert torch.equal(big.expert_counts.long(), torch.bincount(idx.flatten().long(), minlength=E))
    assert int(big.routed_tokens) == T
    total = torch.zeros(E, dtype=torch.float64, device="cuda")
    for part in z.split(1 << 20):
        total += torch.softmax(part.float(), 1).double().sum(0)
    assert bool(((big.prob_sums.double() - total).abs() <= 1e-4 * total).all())
    for rows in (slice(0, n), slice(T - n, T), slice((1 << 31) // E - n // 2, (1 << 31) // E + n // 2)):
        small = _layer(n, E, k)
        zs = z[rows].contiguous()
        i, p, _ = small.route_losses(zs)
        assert torch.equal(i, idx[rows]) and torch.equal(p, prob[rows])
        assert torch.equal(small.router_lse, big.router_lse[rows])
        small.expert_counts.copy_(big.expert_counts)
        small.routed_tokens.copy_(big.routed_tokens)
        assert torch.equal(small.route_backward(zs, dp[rows].contiguous(), dl), grad[rows])
    assert lib.moe_get_device_status(0) == 0


@pytest.mark.parametrize("T,E,k", [(1_400_000, 129, 9), (30_000_000, 4, 1), (4_000_000, 40, 4)])
def test_counts_of_many_tokens_per_lane(T, E, k):
    """More than 255 tokens for every group of lanes."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(T)
    z = _randn(g, T, E, dtype=torch.float32)
    z[:, 1] += 6.0                                  # nearly every token keeps it
    layer = _layer(T, E, k)
    idx, _, losses = layer.route_losses(z)
    assert torch.equal(layer.expert_counts.long(), torch.bincount(idx.flatten().long(), minlength=E))
    total = torch.zeros(E, dtype=torch.float64, device="cuda")
    zsum = torch.zeros((), dtype=torch.float64, device="cuda")
    for part in z.split(1 << 20):
        total += torch.softmax(part.double(), 1).sum(0)
        zsum += torch.logsumexp(part.double(), 1).square().sum()
    # fp32 sums of up to some 3000 terms per lane: 3000 2^-24 relative
    assert bool(((layer.prob_sums.double() - total).abs() <= 2e-4 * total).all())
    want = float(E * (layer.expert_counts.double() * total).sum() / (T * k) / T)
    assert abs(float(losses[0]) - want) <= 2e-4 * want
    assert abs(float(losses[1]) - float(zsum) / T) <= 2e-4 * float(zsum) / T


def test_counts_summed_over_ranks():
    """Each half of a batch, with both halves' counts and tokens, gets the rows of
    the whole batch's gradient."""
    import torch
    T, E, k = 1200, 48, 4
    g = torch.Generator(device="cuda").manual_seed(1)
    z, dp = torch.randn(T, E, device="cuda", generator=g), torch.randn(T, k, device="cuda", generator=g)
    mask = torch.rand(T, device="cuda", generator=g) < 0.8
    dl = torch.tensor([0.3, 0.1], device="cuda")
    whole = _layer(T, E, k)
    whole.route_losses(z, mask)
    want = whole.route_backward(z, dp, dl, mask)
    halves = []
    for rows in (slice(0, 500), slice(500, T)):
        layer = _layer(rows.stop - rows.start, E, k)
        args = [t[rows].contiguous() for t in (z, dp, mask)]
        layer.route_losses(args[0], args[2])
        halves.append((layer, args, rows))
    counts = sum(h[0].expert_counts.clone() for h in halves)
    tokens = sum(h[0].routed_tokens.clone() for h in halves)
    assert torch.equal(counts, whole.expert_counts) and torch.equal(tokens, whole.routed_tokens)
    for layer, (zs, dps, ms), rows in halves:
        layer.expert_counts.copy_(counts)
        layer.routed_tokens.copy_(tokens)
        assert torch.equal(layer.route_backward(zs, dps, dl, ms), want[rows])


@pytest.mark.parametrize("groups,rows,K", [(1, 1_100_000, 4096), (3, 500_001, 2880)])
def test_quantiser_past_32_bits(groups, rows, K):
    import torch
    from mxfp8_grouped_gemm_x32_b200 import mxfp4
    g = torch.Generator(device="cuda").manual_seed(K)
    x = _randn(g, groups, rows, K, dtype=torch.bfloat16)      # > 2^32 values
    codes, scales = mxfp4.quantize(x)
    back = mxfp4.dequantize(codes, scales)
    first = rows // 128 * 128 - 256                           # whole scale tiles to the end
    cs, ss = mxfp4.quantize(x[-1, first:].contiguous())
    assert torch.equal(codes[-1, first:], cs)
    assert torch.equal(scales[-ss.numel():], ss)
    assert torch.equal(back[-1, first:], mxfp4.dequantize(cs, ss))
    head = x[0, :256].contiguous()
    ch, sh = mxfp4.quantize(head)
    assert torch.equal(codes[0, :256], ch) and torch.equal(scales[: sh.numel()], sh)


def _mxfp4_weights(g, E, rows, K):
    import torch
    codes = torch.randint(0, 256, (E, rows, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    return codes, torch.randint(117, 123, (E, rows, K // 32), dtype=torch.uint8, device="cuda", generator=g)


def test_rows_past_32_bits():
    """560000 permuted rows of 12288 bytes; the last and the middle tokens alone."""
    import torch
    from mxfp8_grouped_gemm_x32_b200.layer import GroupedMLP
    T, H, I, E, k, n = 70_000, 4096, 64, 8, 8, 5
    g = torch.Generator(device="cuda").manual_seed(7)
    w = _mxfp4_weights(g, E, 2 * I, H) + _mxfp4_weights(g, E, H, I)
    x = torch.randn(T, H, device="cuda", generator=g).bfloat16()
    idx = torch.argsort(torch.rand(T, E, device="cuda", generator=g), 1)[:, :k].int().contiguous()
    prob = torch.rand(T, k, device="cuda", generator=g)

    def run(rows):
        layer = GroupedMLP(rows.stop - rows.start, H, I, E, k, backward=False, mxfp8=False)
        layer.load_weights_mxfp4(*w)
        layer.permute_index(idx[rows].contiguous(), prob[rows].contiguous())
        return layer.forward_mxfp4(x[rows].contiguous())
    out = run(slice(0, T))
    for at in (0, T // 2, T - n):
        assert torch.equal(out[at:at + n], run(slice(at, at + n)))
    assert bool(torch.isfinite(out.float()).all()) and float(out.float().abs().max()) > 0


def test_weights_past_32_bits():
    """74 experts of 59 MB of gate_up codes: the last and a middle one alone."""
    import torch
    from mxfp8_grouped_gemm_x32_b200.layer import GroupedMLP
    H, I, E, T = 4096, 14336, 74, 40
    g = torch.Generator(device="cuda").manual_seed(8)
    w1, s1 = _mxfp4_weights(g, E, 2 * I, H)
    w2, s2 = _mxfp4_weights(g, E, H, I)
    x = torch.randn(T, H, device="cuda", generator=g).bfloat16()
    prob = torch.rand(T, 1, device="cuda", generator=g)
    big = GroupedMLP(T, H, I, E, 1, backward=False, mxfp8=False)
    big.load_weights_mxfp4(w1, s1, w2, s2)
    for e in (E - 1, 36):
        big.permute_index(torch.full((T, 1), e, dtype=torch.int32, device="cuda"), prob)
        out = big.forward_mxfp4(x).clone()
        one = GroupedMLP(T, H, I, 1, 1, backward=False, mxfp8=False)
        one.load_weights_mxfp4(*(t[e:e + 1].contiguous() for t in (w1, s1, w2, s2)))
        one.permute_index(torch.zeros(T, 1, dtype=torch.int32, device="cuda"), prob)
        assert torch.equal(out, one.forward_mxfp4(x)) and float(out.float().abs().max()) > 0
