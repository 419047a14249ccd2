"""The expert operators on tensors of more than 2^31 elements.

Products: the GEMM bound, |y - want| <= 2^-7 |want| + 1e-3 rms, on the last rows and columns."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def randn(shape, seed, std=1.0):
    """BF16 normals, a slice at a time (no FP32 copy of the whole)."""
    gen = torch.Generator(DEV).manual_seed(seed)
    return torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(0.0, std, generator=gen)


def values(q, s):
    """Codes [M,C] with scales [C/128,M] in 64 bits."""
    return q.view(torch.float8_e4m3fn).double() * s.double().t().repeat_interleave(128, 1)


def codes(shape, seed):
    """Finite E4M3 codes of either sign."""
    gen = torch.Generator(DEV).manual_seed(seed)
    q = torch.randint(0, 0x70, shape, dtype=torch.uint8, generator=gen, device=DEV)
    return q.bitwise_or_(torch.randint(0, 2, (shape[0], 1), dtype=torch.uint8, generator=gen, device=DEV) * 128)


def within(y, want):
    rms = want.square().mean().sqrt()
    assert bool(((y.double() - want).abs() <= 2.0 ** -7 * want.abs() + 1e-3 * rms).all())


def index(T, E, k, seed=1):
    gen = torch.Generator(DEV).manual_seed(seed)
    return torch.argsort(torch.rand((T, E), generator=gen, device=DEV), dim=1)[:, :k].to(torch.int32).contiguous()


def test_gather(fp8lib):
    T, E, k, K = 16500, 8, 4, 32768
    rows = fp8lib.expert_rows(index(T, E, k), E)
    x = randn((T, K), 2)
    q, s, qT, sT = fp8lib.expert_gather_quant(x, rows, dual=True)
    assert q.numel() > 2 ** 31
    a, b = fp8lib.quantize_1x128(x)
    for j in range(k):
        r = rows.pos[:, j].long()
        assert torch.equal(q[r], a) and torch.equal(s[:, r], b)
    # the last block of rows that has pairs, by columns
    lo = int(rows.start[-1]) - 128
    src = rows.src[lo:lo + 128].long()
    v = torch.where((src >= 0)[:, None], x[src.clamp(min=0) // k], torch.zeros_like(x[:1]))
    _, _, cT, dT = fp8lib.quantize_1x128(v, dual=True)
    assert torch.equal(qT[:, lo:lo + 128], cT) and torch.equal(sT[lo // 128], dT[0])
    del qT, sT, a, b
    # weights of 1 in the weighted form, rows and columns
    one = fp8lib.expert_gather_quant(x, rows, torch.ones((T, k), device=DEV), dual=True)
    assert torch.equal(one[0], q) and torch.equal(one[1], s)
    assert torch.equal(one[2][:, lo:lo + 128], cT) and torch.equal(one[3][lo // 128], dT[0])
    assert fp8lib.check_status() == 0


def test_combine_and_its_gradient(fp8lib):
    T, E, k, N = 16500, 8, 4, 32768
    rows = fp8lib.expert_rows(index(T, E, k), E)
    y = randn((rows.src.numel(), N), 3)
    assert y.numel() > 2 ** 31
    w = torch.rand((T, k), generator=torch.Generator(DEV).manual_seed(4), device=DEV)
    out = fp8lib.expert_combine(y, rows, w)
    dout = randn((T, N), 5, 1e-3)
    dw = fp8lib.expert_combine_bwd(dout, y, rows, w, dual=False)[4]
    for lo in (0, T - 300):
        v = y[rows.pos[lo:lo + 300].long()].double()
        prod = v * w[lo:lo + 300].double()[:, :, None]
        want = prod.sum(1)
        assert bool(((out[lo:lo + 300].double() - want).abs() <= 2.0 ** -8 * want.abs() + (k + 1) * 2.0 ** -24 * prod.abs().sum(1)).all())
        dots = v * dout[lo:lo + 300].double()[:, None, :]
        assert bool(((dw[lo:lo + 300].double() - dots.sum(2)).abs() <= (N / 32 + 5) * 2.0 ** -24 * dots.abs().sum(2)).all())


@pytest.mark.parametrize("align", [1, 128])
def test_forward_with_a_long_result(fp8lib, align):
    T, E, k, N, K = 33000, 4, 2, 32896, 256
    rows = fp8lib.expert_rows(index(T, E, k), E, align)
    R = rows.src.numel()
    qx, sx, _, _ = fp8lib.expert_gather_quant(randn((T, K), 2), rows)
    qw, sw = codes((E * N, K), 6), torch.rand((E * N // 128, K // 128), device=DEV) * 1e-3
    y = torch.full((R, N), 7.0, dtype=torch.bfloat16, device=DEV)
    assert y.numel() > 2 ** 31
    fp8lib.gemm_experts_fwd(qx, sx, qw, sw, rows, out=y)
    assert fp8lib.check_status() == 0
    e = E - 1
    hi = int(rows.start[e] + rows.count[e])
    x = values(qx[hi - 200:hi], sx[:, hi - 200:hi])
    for n in (0, N - 384):
        a = e * N + n
        w = qw[a:a + 384].view(torch.float8_e4m3fn).double() * sw[a // 128:a // 128 + 3].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
        within(y[hi - 200:hi, n:n + 384], x @ w.t())
    assert bool((y[int(rows.start[-1]):] == 7).all())


@pytest.mark.parametrize("align", [1, 128])
def test_forward_with_long_weights(fp8lib, align):
    T, E, k, N, K = 6, 64, 8, 8192, 4224
    rows = fp8lib.expert_rows(torch.arange(E - T - k + 1, E + 1, device=DEV, dtype=torch.int32).unfold(0, k, 1)[:T].contiguous(), E, align)
    qx, sx, _, _ = fp8lib.expert_gather_quant(randn((T, K), 2), rows)
    qw, sw = codes((E * N, K), 6), torch.rand((E * N // 128, K // 128), device=DEV) * 1e-3
    assert qw.numel() > 2 ** 31
    y = fp8lib.gemm_experts_fwd(qx, sx, qw, sw, rows)
    assert fp8lib.check_status() == 0
    start, count = rows.start.tolist(), rows.count.tolist()
    for e in (E - 1, E - T - 2):
        assert count[e] > 0
        a, b = start[e], start[e] + count[e]
        w = qw[(e + 1) * N - 256:(e + 1) * N].view(torch.float8_e4m3fn).double()
        w = w * sw[((e + 1) * N - 256) // 128:(e + 1) * N // 128].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
        within(y[a:b, -256:], values(qx[a:b], sx[:, a:b]) @ w.t())


def test_gradients_of_long_weights(fp8lib):
    T, E, k, N, K = 500, 64, 2, 8192, 4224
    rows = fp8lib.expert_rows(index(T, E, k), E)
    q, s, qT, sT = fp8lib.expert_gather_quant(randn((T, N), 3, 1e-3), rows, dual=True)
    _, _, qxT, sxT = fp8lib.expert_gather_quant(randn((T, K), 2), rows, dual=True)
    dw = fp8lib.gemm_experts_wgrad(qT, sT, qxT, sxT, rows)
    assert dw.numel() > 2 ** 31 and fp8lib.check_status() == 0
    qwT, sw = codes((K, E * N), 6), torch.rand((E * N // 128, K // 128), device=DEV) * 1e-3
    dx = fp8lib.gemm_experts_dgrad(q, s, qwT, sw, rows)
    assert fp8lib.check_status() == 0
    start, count = rows.start.tolist(), rows.count.tolist()
    for e in (0, E - 1):
        assert count[e] > 0
        a, b = start[e], start[e + 1]
        dyT, xT = values(qT[:, a:b].contiguous(), sT[a // 128:b // 128]), values(qxT[:, a:b].contiguous(), sxT[a // 128:b // 128])
        within(dw[e, -256:], dyT[-256:] @ xT.t())
        w = qwT[-256:, e * N:(e + 1) * N].view(torch.float8_e4m3fn).double()       # [256,N]
        w = w * sw[e * N // 128:(e + 1) * N // 128, -2:].double().t().repeat_interleave(128, 0).repeat_interleave(128, 1)
        within(dx[a:a + count[e], -256:], values(q[a:a + count[e]], s[:, a:a + count[e]]) @ w.t())
