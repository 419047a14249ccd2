"""GPU parity of the expert-layer operators with their 64-bit definitions.

Tolerances.  Integers and 8-bit codes are exact.  Router weights: FP32 scores within 2^-18 relative
(the denominator's additions), a sum of k and a division more, stated as 2^-17.  Products: the GEMM
bound of parity.py.  combine: k + 1 roundings of FP32 on the sum of magnitudes and half a BF16 step.
dweight: FP32 sums of N products, at most N/32 + 5 in a row, on the sum of magnitudes."""
import numpy as np
import pytest
import torch

import expert_reference as ref
from block_scaled_fp8_x1_gb300 import synth

pytestmark = pytest.mark.gpu
DEV = "cuda"


def np64(t):
    return t.detach().double().cpu().numpy()


def ints(t):
    return t.cpu().numpy().astype(np.int64)


def draw_index(T, E, k, seed, missing=0.0):
    r = np.random.default_rng(seed)
    likes = 0.5 * r.standard_normal(E)
    idx = np.argsort(-(likes + r.standard_normal((T, E))), axis=1)[:, :k].astype(np.int32)
    idx[r.random((T, k)) < missing] = -1
    return idx


# ------------------------------------------------------------------ router

ROUTES = [  # T, E, k, kwargs
    (1, 64, 8, dict()), (1, 1, 1, dict()), (5, 2, 2, dict(score="sigmoid")), (33, 8, 2, dict(renormalize=False)),
    (130, 60, 4, dict(scale=2.5)), (257, 96, 6, dict(score="sigmoid", renormalize=False)),
    (64, 256, 8, dict(score="sigmoid", bias=True, n_groups=8, top_groups=4, group_rank=2, scale=2.5)),
    (64, 160, 6, dict(n_groups=8, top_groups=3)), (64, 160, 6, dict(n_groups=8, top_groups=3, group_rank=2)),
    (64, 512, 10, dict(bias=True)), (31, 1024, 32, dict(score="sigmoid", bias=True, n_groups=32, top_groups=32, group_rank=1)),
    (40, 32, 32, dict(score="sigmoid", n_groups=32, top_groups=32)), (17, 384, 8, dict(bias=True, renormalize=False)),
    (40, 24, 3, dict(score="sigmoid", bias=True, n_groups=8, top_groups=1, group_rank=2)),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k,kw", ROUTES)
def test_route(fp8lib, T, E, k, kw, dtype):
    g = torch.Generator(DEV).manual_seed(T + E)
    z = (2.0 * torch.randn((T, E), generator=g, device=DEV)).to(dtype)
    kw = dict(kw)
    bias = 0.1 * torch.randn(E, generator=g, device=DEV) if kw.pop("bias", False) else None
    r = fp8lib.route_topk(z, k, bias=bias, **{"group_rank": 1, **kw})
    w, i = ref.route(np64(z), k, bias=None if bias is None else np64(bias), **{"group_rank": 1, **kw})
    assert np.array_equal(ints(r.index), i)
    assert np.all(np.abs(np64(r.weight) - w) <= 2.0 ** -17 * np.abs(w))
    assert fp8lib.check_status() == 0


def test_route_near_ties(fp8lib):
    """Scores next to each other under FP32's resolution, told apart as the exact values are: biases
    that differ by 2^-30 and less on equal logits, and sums of two that do."""
    r = np.random.default_rng(3)
    T, E, k = 64, 64, 8
    z = np.repeat(np.round(r.standard_normal((T, 1)) * 4) / 4, E, 1).astype(np.float32)
    bias = (0.25 + r.integers(-3, 4, E) * 2.0 ** -26).astype(np.float32)
    for kw in (dict(), dict(n_groups=8, top_groups=3, group_rank=2), dict(n_groups=16, top_groups=8, group_rank=1)):
        for score in ("sigmoid", "softmax"):
            got = fp8lib.route_topk(torch.tensor(z, device=DEV), k, score=score, bias=torch.tensor(bias, device=DEV),
                                    **{"group_rank": 1, **kw})
            _, i = ref.route(z, k, score, bias, **{"group_rank": 1, **kw})
            assert np.array_equal(ints(got.index), i), (score, kw)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("spread", [0.5, 2.0])
def test_route_order_of_scores_that_nearly_agree(fp8lib, spread, score):
    """Biases that bring every score to within their own rounding (2^-27 and less) of one value: the
    order is that of the exact sums wherever these are 2^-38 apart."""
    for seed in range(8):
        r = np.random.default_rng(seed)
        z = (spread * r.uniform(-1, 1, (1, 64))).astype(np.float32)
        s = ref.scores(z.astype(np.float64), score)
        b = (s.mean() - s[0]).astype(np.float32)
        i = ints(fp8lib.route_topk(torch.tensor(z, device=DEV), 8, score=score, bias=torch.tensor(b, device=DEV), group_rank=1).index)[0]
        v = s[0] + b.astype(np.float64)
        assert len(set(i.tolist())) == 8
        assert np.all(v[i[:-1]] >= v[i[1:]] - 2.0 ** -38)
        assert v[i].min() >= np.delete(v, i).max() - 2.0 ** -38


def test_route_without_differences(fp8lib):
    """All logits and biases equal, in every form of the selection: the first experts, in order."""
    for E, k in ((1, 1), (64, 8), (100, 32), (256, 8), (1024, 3)):
        for dtype in (torch.float32, torch.bfloat16):
            z = torch.full((3, E), 0.25, dtype=dtype, device=DEV)
            for bias in (None, torch.zeros(E, device=DEV)):
                for score in ("softmax", "sigmoid"):
                    r = fp8lib.route_topk(z, k, score=score, bias=bias)
                    assert ints(r.index).tolist() == [list(range(k))] * 3
                    assert np.abs(np64(r.weight) - 1.0 / k).max() < 1e-6


@pytest.mark.parametrize("off", [0, 1, 2, 3, 8])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_rows_of_any_alignment(fp8lib, off, dtype):
    wide = torch.randn((20, 300), generator=torch.Generator(DEV).manual_seed(off), device=DEV).to(dtype)
    for E in (64, 96, 256):
        z = wide[:, off:off + E]
        for bias in (None, torch.linspace(-0.1, 0.1, E + 1, device=DEV)[1:]):
            a = fp8lib.route_topk(z, 6, score="sigmoid", bias=bias)
            b = fp8lib.route_topk(z.contiguous(), 6, score="sigmoid", bias=None if bias is None else bias.clone())
            assert torch.equal(a.index, b.index) and torch.equal(a.weight, b.weight)


def test_route_equal_scores_go_to_the_lowest_index(fp8lib):
    z = torch.zeros((3, 100), device=DEV)
    z[1, ::2] = -0.0
    z[2, 50:] = 1.0
    i = ints(fp8lib.route_topk(z, 5).index)
    assert i.tolist() == [[0, 1, 2, 3, 4], [0, 1, 2, 3, 4], [50, 51, 52, 53, 54]]
    b = torch.zeros(100, device=DEV)
    i = ints(fp8lib.route_topk(z, 5, bias=b, score="sigmoid", n_groups=10, top_groups=2).index)
    assert i.tolist() == [[0, 1, 2, 3, 4], [0, 1, 2, 3, 4], [50, 51, 52, 53, 54]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
def test_route_masked_rows(fp8lib, score, bias):
    """Rows of -inf, rows with fewer experts than k, the type's lowest value, large logits."""
    z = torch.full((5, 40), float("-inf"), device=DEV)
    z[1, 7], z[1, 30] = 1.0, 2.0
    z[2] = torch.finfo(torch.float32).min
    z[3] = torch.linspace(-3e4, 3e4, 40, device=DEV)
    z[4, 5:] = torch.linspace(-1, 1, 35, device=DEV)
    b = 0.01 * torch.arange(40, device=DEV, dtype=torch.float32).flip(0).contiguous() if bias else None
    for kw in (dict(), dict(n_groups=4, top_groups=2, group_rank=1), dict(n_groups=4, top_groups=2, group_rank=2),
               dict(renormalize=False)):
        got = fp8lib.route_topk(z, 4, score=score, bias=b, **{"group_rank": 1, **kw})
        w, i = ref.route(np64(z), 4, score, None if b is None else np64(b), **{"group_rank": 1, **kw})
        assert np.array_equal(ints(got.index), i), kw
        assert np.all(np.abs(np64(got.weight) - w) <= 2.0 ** -17 * np.abs(w) + 1e-37), kw
        assert (ints(got.index)[0] == -1).all() and (np64(got.weight)[0] == 0).all()
        d = fp8lib.route_topk_bwd(torch.ones((5, 4), device=DEV), z, got.index, score=score, renormalize=kw.get("renormalize", True))
        assert torch.isfinite(d).all() and (d[0] == 0).all()


def test_route_nan_shows(fp8lib):
    z = torch.randn((4, 64), device=DEV)
    z[1, 20] = float("nan")
    z[2, 5] = float("inf")
    for score in ("softmax", "sigmoid"):
        r = fp8lib.route_topk(z, 4, score=score)
        assert ints(r.index)[1, 0] == 20 and torch.isnan(r.weight[1]).all()
        assert ints(r.index)[2, 0] == 5
        assert torch.isfinite(r.weight[[0, 3]]).all()
        b = torch.zeros(64, device=DEV)
        i = ints(fp8lib.route_topk(z, 4, score=score, bias=b).index)
        assert ((i >= 0) & (i < 64)).all()
        if score == "sigmoid":
            assert i[1, 0] == 20


def test_route_strided_and_permuted_batches_agree(fp8lib):
    wide = torch.randn((70, 96), device=DEV)
    z = wide[:, 10:74]
    a = fp8lib.route_topk(z, 6, score="sigmoid", bias=torch.zeros(64, device=DEV))
    b = fp8lib.route_topk(z.contiguous().flip(0).contiguous(), 6, score="sigmoid", bias=torch.zeros(64, device=DEV))
    assert torch.equal(a.index, b.index.flip(0)) and torch.equal(a.weight, b.weight.flip(0))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (9, 8, 2), (65, 60, 6), (130, 256, 8), (5, 1000, 32)])
def test_route_bwd(fp8lib, T, E, k, renorm, score, dtype):
    g = torch.Generator(DEV).manual_seed(E)
    z = (1.5 * torch.randn((T, E), generator=g, device=DEV)).to(dtype)
    idx = fp8lib.route_topk(z, k, score=score).index
    idx[T // 2, k // 2] = -1
    dw = torch.randn((T, k), generator=g, device=DEV)
    got = np64(fp8lib.route_topk_bwd(dw, z, idx, score=score, renormalize=renorm, scale=1.5))
    want = ref.route_bwd(np64(dw), np64(z), ints(idx), score, renorm, 1.5)
    s = ref.scores(np64(z), score)
    # magnitude of the terms that are added: s_e (|ds_e| + sum s |ds|), |ds| <= 2 max|g| / total
    total = np.array([[sum(s[t, e] for e in row if e >= 0) if renorm else 1.0] for t, row in enumerate(ints(idx))])
    total = np.where(total == 0, 1.0, total)
    size = 4 * 1.5 * np.abs(np64(dw)).max(1, keepdims=True) / total * s
    half = 2.0 ** -8 if dtype is torch.bfloat16 else 0.0
    assert np.all(np.abs(got - want) <= half * np.abs(want) + 2.0 ** -16 * size)


def test_route_bwd_against_differences(fp8lib):
    r = np.random.default_rng(5)
    z = r.standard_normal((3, 16))
    _, idx = ref.route(z, 4)
    dw = r.standard_normal((3, 4))
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            def loss(zz):
                s = ref.scores(zz, score)
                w = np.take_along_axis(s, idx, 1)
                return ((w / (w.sum(1, keepdims=True) + 1e-20) if renorm else w) * 2.5 * dw).sum()
            num = np.zeros_like(z)
            for i in np.ndindex(z.shape):
                h = np.zeros_like(z)
                h[i] = 1e-5
                num[i] = (loss(z + h) - loss(z - h)) / 2e-5
            got = np64(fp8lib.route_topk_bwd(torch.tensor(dw, device=DEV, dtype=torch.float32), torch.tensor(z, device=DEV, dtype=torch.float32),
                                             torch.tensor(idx, device=DEV, dtype=torch.int32), score=score, renormalize=renorm, scale=2.5))
            # differences: h^2 and 1e-16 / h; the kernel: FP32 of terms up to 10
            assert np.abs(got - num).max() < 1e-5


def test_route_bwd_same_expert_twice(fp8lib):
    z = torch.randn((2, 8), device=DEV)
    idx = torch.tensor([[3, 3, 99], [1, -5, 1]], dtype=torch.int32, device=DEV)
    dw = torch.randn((2, 3), device=DEV)
    got = np64(fp8lib.route_topk_bwd(dw, z, idx, score="sigmoid", renormalize=False))
    want = ref.route_bwd(np64(dw), np64(z), ints(idx), "sigmoid", False)
    assert np.abs(got - want).max() < 1e-6


# ------------------------------------------------------------------ expert order

@pytest.mark.parametrize("align", [1, 128])
@pytest.mark.parametrize("T,E,k,missing", [(1, 1, 1, 0), (1, 64, 8, 0), (61, 64, 6, 0), (700, 16, 3, 0.2), (33, 1024, 32, 0.1),
                                           (2049, 8, 1, 0), (1500, 60, 7, 0), (4096, 96, 8, 0.01), (3, 5, 2, 1.0)])
def test_expert_rows(fp8lib, T, E, k, missing, align):
    idx = draw_index(T, max(E, k), k, T + E, missing)
    idx[idx >= E] = E + 3        # outside: no pair
    r = fp8lib.expert_rows(torch.tensor(idx, device=DEV), E, align)
    pos, src, start, count = ref.rows(np.where((idx >= 0) & (idx < E), idx, -1), E, align)
    for got, want in ((r.pos, pos), (r.src, src), (r.start, start), (r.count, count)):
        assert np.array_equal(ints(got), want)
    assert r.align == align


def test_expert_rows_one_expert_has_all(fp8lib):
    idx = torch.full((5000, 2), 6, dtype=torch.int32, device=DEV)
    r = fp8lib.expert_rows(idx, 9)
    assert torch.equal(r.src[:10000], torch.arange(10000, device=DEV, dtype=torch.int32))
    assert ints(r.count).tolist() == [0] * 6 + [10000] + [0] * 2
    assert ints(r.start).tolist() == [0] * 7 + [10112] * 3


# ------------------------------------------------------------------ gather, combine

def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def quant_same(oracle, got, x_bits, dual):
    """Codes and scales of got equal the oracle's quantization of the BF16 rows x_bits."""
    M = x_bits.shape[0]
    pad = -M % 128
    r = oracle.quantize_1x128(np.concatenate([x_bits, np.zeros((pad, x_bits.shape[1]), np.uint16)]) if pad else x_bits)
    q, s, qT, sT = got
    assert np.array_equal(q.cpu().numpy(), r[0][:M])
    assert np.array_equal(s.cpu().numpy().view(np.uint32), np.ascontiguousarray(r[1][:, :M], np.float32).view(np.uint32))
    if dual:
        c = oracle.quantize_1x128(np.ascontiguousarray(x_bits.T))
        assert np.array_equal(qT.cpu().numpy(), c[0])
        assert np.array_equal(sT.cpu().numpy().view(np.uint32), np.asarray(c[1], np.float32).view(np.uint32))


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("T,E,k,K,align,dual,missing", [
    (1, 64, 8, 128, 1, False, 0), (61, 64, 6, 640, 1, False, 0), (7, 4, 3, 256, 1, False, 0.5), (1, 8, 2, 256, 128, True, 0),
    (300, 8, 3, 384, 128, True, 0.1), (300, 8, 3, 384, 128, False, 0), (515, 60, 5, 256, 128, True, 0), (3, 4, 2, 128, 128, True, 1.0)])
def test_gather_quant(fp8lib, oracle, T, E, k, K, align, dual, missing, weighted):
    idx = draw_index(T, max(E, k), k, T, missing)
    rows = fp8lib.expert_rows(torch.tensor(idx, device=DEV), E, align)
    wide = synth.normal_bf16((T, K + 64), 1.0, 7, torch.device(DEV), outlier_channels=2, outlier_scale=30.0)
    x = wide[:, :K]              # strided rows
    w = torch.randn((T, k), device=DEV) if weighted else None
    got = fp8lib.expert_gather_quant(x, rows, w, dual=dual)
    src = ints(rows.src)
    if weighted:
        v = torch.zeros((len(src), K), dtype=torch.bfloat16, device=DEV)
        has = torch.tensor(src >= 0, device=DEV)
        p = torch.tensor(src, device=DEV)[has]
        v[has] = (x[p // k].float() * w.reshape(-1)[p][:, None]).to(torch.bfloat16)
        want = bits(v)
    else:
        want = ref.gather(bits(x), src, k)
    quant_same(oracle, got, want, dual)
    assert fp8lib.check_status() == 0


def test_gather_keeps_nan_and_infinity_of_other_tokens_out(fp8lib, oracle):
    """Padding rows are zeros whatever token 0 (which stands in for them in the copies) holds."""
    idx = torch.tensor([[5], [2], [2]], dtype=torch.int32, device=DEV)
    rows = fp8lib.expert_rows(idx, 8)
    x = synth.normal_bf16((3, 256), 1.0, 7, torch.device(DEV))
    x[0] = float("nan")
    q, s, qT, sT = fp8lib.expert_gather_quant(x, rows, torch.ones((3, 1), device=DEV), dual=True)
    want = ref.gather(bits(x), ints(rows.src), 1)
    lo, hi = 0, 128              # expert 2's rows: tokens 1, 2 and padding
    r = oracle.quantize_1x128(want[lo:hi])
    assert np.array_equal(q.cpu().numpy()[lo:hi], r[0])
    c = oracle.quantize_1x128(np.ascontiguousarray(want[lo:hi].T))
    assert np.array_equal(qT.cpu().numpy()[:, lo:hi], c[0])


def test_gather_of_groups_next_to_zero(fp8lib, oracle):
    """Groups whose scale is below 2^-68 or subnormal, or whose products underflow, beside ordinary ones."""
    T, E, k, K = 260, 3, 2, 256
    idx = draw_index(T, E, k, 5, 0)
    rows = fp8lib.expert_rows(torch.tensor(idx, device=DEV), E)
    x = synth.normal_bf16((T, K), 1.0, 3, torch.device(DEV)).float()
    x[:, :40] *= 2.0 ** -70
    x[:, 128:] *= 2.0 ** -75
    x[7:9] *= 2.0 ** -60
    x[11] = 0
    x = x.to(torch.bfloat16)
    for w in (None, torch.randn((T, k), device=DEV) * 2.0 ** torch.randint(-60, 3, (T, k), device=DEV)):
        src = ints(rows.src)
        v = torch.zeros((len(src), K), dtype=torch.bfloat16, device=DEV)
        has = torch.tensor(src >= 0, device=DEV)
        p = torch.tensor(src, device=DEV)[has]
        v[has] = x[p // k] if w is None else (x[p // k].float() * w.reshape(-1)[p][:, None]).to(torch.bfloat16)
        quant_same(oracle, fp8lib.expert_gather_quant(x, rows, w, dual=True), bits(v), True)


def test_gather_weights_that_are_no_numbers(fp8lib):
    """An infinite or missing weight, an infinite or missing input: the scales tell, other rows stay as they are."""
    T, K = 40, 256
    idx = torch.randint(0, 4, (T, 1), dtype=torch.int32, device=DEV)
    rows = fp8lib.expert_rows(idx, 4, 1)
    x = synth.normal_bf16((T, K), 1.0, 7, torch.device(DEV))
    w = torch.randn((T, 1), device=DEV)
    x[3, 5], x[4, 6], x[5, 200], x[9, 130] = float("inf"), float("nan"), 0, 0
    w[5], w[6], w[7], w[3], w[4] = float("inf"), float("nan"), float("inf"), 0, 0
    x[7] = 1
    q, s, _, _ = fp8lib.expert_gather_quant(x, rows, w)
    y = (x.float() * w).to(torch.bfloat16)
    q1, s1, _, _ = fp8lib.expert_gather_quant(y, rows)
    bad = ~torch.isfinite(s1)
    assert bad.any(0).sum() == 5
    assert torch.equal(torch.isnan(s), torch.isnan(s1)) and torch.equal(s[~torch.isnan(s)], s1[~torch.isnan(s1)])
    same = ~bad.t().repeat_interleave(128, 1)
    assert torch.equal(q[same], q1[same])


def test_gather_by_an_order_at_any_offset(fp8lib, oracle):
    """The arrays of an order need the alignment of their elements alone."""
    T, E, k, K = 150, 5, 3, 256
    rows = fp8lib.expert_rows(torch.tensor(draw_index(T, E, k, 2, 0.1), device=DEV), E)

    def moved(t, by):
        b = torch.empty(t.numel() + by, dtype=t.dtype, device=DEV)
        b[by:] = t.reshape(-1)
        return b[by:].view(t.shape)

    x = synth.normal_bf16((T, K), 1.0, 7, torch.device(DEV))
    w = moved(torch.randn((T, k), device=DEV), 1)
    want = fp8lib.expert_gather_quant(x, rows, w, dual=True)
    for by in (1, 2, 3):
        odd = fp8lib.ExpertRows(*(moved(t, by) for t in rows[:4]), rows.align)
        assert all(torch.equal(a, b) for a, b in zip(fp8lib.expert_gather_quant(x, odd, w, dual=True), want))


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("T,E,k,N,align,res,missing", [
    (1, 64, 8, 128, 1, False, 0), (61, 64, 6, 1000, 1, True, 0), (300, 8, 3, 384, 128, True, 0.2), (5, 4, 2, 8, 1, False, 1.0),
    (513, 16, 16, 264, 128, False, 0)])
def test_combine(fp8lib, T, E, k, N, align, res, missing, weighted):
    idx = draw_index(T, max(E, k), k, T + 1, missing)
    rows = fp8lib.expert_rows(torch.tensor(idx, device=DEV), E, align)
    R = rows.src.numel()
    y = synth.normal_bf16((R, N + 16), 1.0, 3, torch.device(DEV))[:, :N]
    y[rows.src < 0] = float("nan")       # rows of no pair are not read
    w = torch.rand((T, k), device=DEV) if weighted else None
    r = synth.normal_bf16((T, N), 1.0, 4, torch.device(DEV)) if res else None
    out = fp8lib.expert_combine(y, rows, w, residual=r)
    a = (np64(y), ints(rows.pos), None if w is None else np64(w))
    want = ref.combine(*a, None if r is None else np64(r))
    size = ref.combine(np.abs(a[0]), *a[1:], None if r is None else np.abs(np64(r)))
    assert np.all(np.abs(np64(out) - want) <= 2.0 ** -8 * np.abs(want) + (k + 1) * 2.0 ** -24 * size)


def test_combine_into_its_residual(fp8lib):
    idx = torch.tensor(draw_index(50, 8, 2, 1), device=DEV)
    rows = fp8lib.expert_rows(idx, 8, 1)
    y = synth.normal_bf16((100, 256), 1.0, 3, torch.device(DEV))
    r = synth.normal_bf16((50, 256), 1.0, 4, torch.device(DEV))
    want = fp8lib.expert_combine(y, rows, residual=r)
    got = fp8lib.expert_combine(y, rows, residual=r, out=r)
    assert got is r and torch.equal(got, want)


@pytest.mark.parametrize("T,E,k,N,align,dual", [(1, 8, 2, 128, 128, True), (130, 16, 4, 640, 128, True), (61, 64, 6, 256, 1, False)])
def test_combine_bwd(fp8lib, oracle, T, E, k, N, align, dual):
    idx = draw_index(T, E, k, T + 2, 0.1)
    rows = fp8lib.expert_rows(torch.tensor(idx, device=DEV), E, align)
    dev = torch.device(DEV)
    y = synth.normal_bf16((rows.src.numel(), N), 1.0, 3, dev)
    dout = synth.normal_bf16((T, N), 1e-3, 4, dev)
    w = torch.rand((T, k), device=DEV)
    *got, dw = fp8lib.expert_combine_bwd(dout, y, rows, w, dual=dual)
    alone = fp8lib.expert_gather_quant(dout, rows, w, dual=dual)
    for a, b in zip(got, alone):
        assert (a is None and b is None) or torch.equal(a, b)
    pos = ints(rows.pos)
    prod = np.where(pos[:, :, None] >= 0, np64(y)[np.maximum(pos, 0)], 0.0) * np64(dout)[:, None, :]
    assert np.all(np.abs(np64(dw) - prod.sum(2)) <= (N / 32 + 5) * 2.0 ** -24 * np.abs(prod).sum(2))


# ------------------------------------------------------------------ products

def within(y, want):
    """The GEMM bound: |y - want| <= 2^-7 |want| + 1e-3 rms."""
    rms = np.sqrt(np.mean(want * want))
    bad = np.abs(y - want) > 2.0 ** -7 * np.abs(want) + 1e-3 * rms
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} outside the bound"


def weights(fp8lib, E, N, K, seed=5):
    return fp8lib.quantize_128x128(synth.normal_bf16((E * N, K), 0.02, seed, torch.device(DEV)))


FWD = [  # T, E, k, N, K, align, missing
    (1, 8, 2, 128, 128, 1, 0), (1, 64, 8, 256, 1408, 1, 0), (61, 64, 6, 384, 640, 1, 0), (200, 4, 2, 256, 512, 1, 0.1),
    (40, 1024, 3, 128, 256, 1, 0), (500, 3, 1, 128, 384, 1, 0), (1, 8, 2, 128, 128, 128, 0), (300, 8, 3, 384, 384, 128, 0),
    (700, 4, 2, 512, 640, 128, 0.2), (2000, 16, 4, 640, 1408, 128, 0), (130, 300, 2, 128, 256, 128, 0), (257, 2, 1, 1024, 4352, 128, 0)]


@pytest.mark.parametrize("T,E,k,N,K,align,missing", FWD)
def test_product_forward(fp8lib, T, E, k, N, K, align, missing):
    rows = fp8lib.expert_rows(torch.tensor(draw_index(T, E, k, T, missing), device=DEV), E, align)
    x = synth.normal_bf16((T, K), 1.0, 7, torch.device(DEV), outlier_channels=2, outlier_scale=30.0)
    qx, sx, _, _ = fp8lib.expert_gather_quant(x, rows)
    qw, sw, _ = weights(fp8lib, E, N, K)
    R = qx.shape[0]
    out = torch.full((R, N), 7.0, dtype=torch.bfloat16, device=DEV)
    y = fp8lib.gemm_experts_fwd(qx, sx, qw, sw, rows, out=out)
    assert fp8lib.check_status() == 0 and y is out
    start, count = ints(rows.start), ints(rows.count)
    want = ref.product_fwd(ref.values(qx.cpu().numpy(), sx.cpu().numpy()), ref.weight_values(qw.cpu().numpy(), sw.cpu().numpy()), start, count, E)
    got = np64(y)
    if want:
        within(np.concatenate([got[start[e]:start[e] + count[e]] for e in want]), np.concatenate(list(want.values())))
    for e in range(E):      # padding rows have the product of their zeros
        assert (got[start[e] + count[e]:start[e + 1]] == 0).all()
    assert (got[start[E]:] == 7.0).all()     # unused rows are as they were
    again = fp8lib.gemm_experts_fwd(qx, sx, qw, sw, rows, out=torch.full_like(out, 7.0))
    assert torch.equal(again.view(torch.int16), y.view(torch.int16))


@pytest.mark.parametrize("T,E,k,N,K,missing", [(1, 8, 2, 128, 128, 0), (300, 8, 3, 384, 640, 0), (700, 4, 2, 2816, 512, 0.2),
                                               (1111, 32, 4, 640, 3584, 0), (130, 300, 2, 128, 256, 0)])
def test_product_dgrad(fp8lib, T, E, k, N, K, missing):
    rows = fp8lib.expert_rows(torch.tensor(draw_index(T, E, k, T, missing), device=DEV), E)
    qdy, sdy, _, _ = fp8lib.expert_gather_quant(synth.normal_bf16((T, N), 1e-3, 8, torch.device(DEV)), rows)
    qw, sw, qwT = weights(fp8lib, E, N, K)
    out = torch.full((qdy.shape[0], K), 7.0, dtype=torch.bfloat16, device=DEV)
    got = np64(fp8lib.gemm_experts_dgrad(qdy, sdy, qwT, sw, rows, out=out))
    assert fp8lib.check_status() == 0
    start, count = ints(rows.start), ints(rows.count)
    dy, w = ref.values(qdy.cpu().numpy(), sdy.cpu().numpy()), ref.weight_values(qw.cpu().numpy(), sw.cpu().numpy())
    used = [e for e in range(E) if count[e]]
    cut = lambda a, e: a[start[e]:start[e] + count[e]]  # noqa: E731
    within(np.concatenate([cut(got, e) for e in used]), np.concatenate([cut(dy, e) @ w[e * N:(e + 1) * N] for e in used]))
    assert (got[start[E]:] == 7.0).all()


@pytest.mark.parametrize("T,E,k,N,K,missing", [(1, 8, 2, 128, 128, 0), (300, 8, 3, 384, 640, 0), (700, 4, 2, 512, 1408, 0.2),
                                               (1500, 12, 4, 640, 256, 0), (130, 300, 2, 128, 256, 0), (3, 4, 2, 128, 128, 1.0)])
def test_product_wgrad(fp8lib, T, E, k, N, K, missing):
    rows = fp8lib.expert_rows(torch.tensor(draw_index(T, E, k, T, missing), device=DEV), E)
    dev = torch.device(DEV)
    _, _, qdyT, sdyT = fp8lib.expert_gather_quant(synth.normal_bf16((T, N), 1e-3, 8, dev), rows, dual=True)
    _, _, qxT, sxT = fp8lib.expert_gather_quant(synth.normal_bf16((T, K), 1.0, 9, dev), rows, dual=True)
    dw = fp8lib.gemm_experts_wgrad(qdyT, sdyT, qxT, sxT, rows)
    assert fp8lib.check_status() == 0 and dw.shape == (E, N, K)
    start = ints(rows.start)
    dyT, xT = ref.values(qdyT.cpu().numpy(), sdyT.cpu().numpy()), ref.values(qxT.cpu().numpy(), sxT.cpu().numpy())
    want = np.stack([dyT[:, start[e]:start[e + 1]] @ xT[:, start[e]:start[e + 1]].T for e in range(E)])
    got = np64(dw)
    if want.any():
        within(got, want)
    for e in range(E):
        if start[e] == start[e + 1]:
            assert (got[e] == 0).all()


def test_forms_agree_on_exact_sums(fp8lib):
    """Operands whose sums are exact in FP32: both forms of the forward give the same bytes."""
    r = np.random.default_rng(1)
    T, E, k, N, K = 90, 8, 3, 256, 384
    idx = torch.tensor(draw_index(T, E, k, 4), device=DEV)
    x = torch.tensor(r.integers(-3, 4, (T, K)), device=DEV).to(torch.bfloat16)
    x[:, ::128] = 448.0 / 64
    w = torch.tensor(r.integers(-3, 4, (E * N, K)), device=DEV).to(torch.bfloat16)
    w[::128, ::128] = 448.0 / 64
    qw, sw, _ = fp8lib.quantize_128x128(w)
    ys = []
    for align in (1, 128):
        rows = fp8lib.expert_rows(idx, E, align)
        qx, sx, _, _ = fp8lib.expert_gather_quant(x, rows)
        y = fp8lib.gemm_experts_fwd(qx, sx, qw, sw, rows)
        ys.append(fp8lib.expert_combine(y, rows))
    assert torch.equal(ys[0], ys[1])


def test_no_tokens(fp8lib):
    idx = torch.zeros((0, 4), dtype=torch.int32, device=DEV)
    z = torch.zeros((0, 8), device=DEV)
    assert fp8lib.route_topk(z, 4).index.shape == (0, 4)
    assert fp8lib.route_topk_bwd(torch.zeros((0, 4), device=DEV), z, idx).shape == (0, 8)
    for align in (1, 128):
        rows = fp8lib.expert_rows(idx, 8, align)
        assert rows.src.numel() == 0 and ints(rows.count).tolist() == [0] * 8 and ints(rows.start).tolist() == [0] * 9
        x = torch.zeros((0, 256), dtype=torch.bfloat16, device=DEV)
        q, s, _, _ = fp8lib.expert_gather_quant(x, rows)
        qw, sw, qwT = weights(fp8lib, 8, 128, 256)
        assert fp8lib.gemm_experts_fwd(q, s, qw, sw, rows).shape == (0, 128)
        assert fp8lib.expert_combine(x, rows).shape == (0, 256)
    q, s, qT, sT = fp8lib.expert_gather_quant(x, rows, dual=True)
    dw = fp8lib.gemm_experts_wgrad(qT[:128], sT[:, :128].contiguous(), qT, sT, rows)
    assert dw.shape == (8, 128, 256) and (dw == 0).all()
