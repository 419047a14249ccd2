"""Infinities and NaN in rows that have a pair, in both layouts of the gather.

Codes of a group that holds one are unspecified, its scale is no finite number; every other group is as if
they were not there.  The column layout forms its maxima by instructions of its own."""
import pytest
import torch

from block_scaled_fp8_x1_gb300 import synth

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF, NAN = float("inf"), float("nan")


def same_groups(got_q, got_s, want_q, want_s, bad):
    """Codes [M,C], scales [C/128,M], bad [C/128,M]: groups of an infinity or a NaN."""
    assert not torch.isfinite(got_s[bad]).any()
    assert torch.equal(torch.isnan(got_s), torch.isnan(want_s))
    assert torch.equal(got_s[~bad].view(torch.int32), want_s[~bad].view(torch.int32))
    keep = ~bad.t().repeat_interleave(128, 1)
    assert torch.equal(got_q[keep], want_q[keep])


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("T,K", [(200, 256), (70, 640)])
def test_columns_and_rows(fp8lib, T, K, weighted):
    E, k = 4, 2
    gen = torch.Generator(DEV).manual_seed(T)
    idx = torch.stack([torch.randperm(E, generator=gen, device=DEV)[:k] for _ in range(T)]).to(torch.int32)
    rows = fp8lib.expert_rows(idx, E)
    x = synth.normal_bf16((T, K), 1.0, 7, torch.device(DEV))
    # each half of a pair of columns, each sign, and a NaN beside an infinity in one column
    x[3, 5], x[4, 6], x[9, 130], x[11, 131], x[12, 200], x[60, 200], x[33, K - 1] = INF, -NAN, -INF, NAN, INF, NAN, -INF
    w = torch.rand((T, k), generator=gen, device=DEV) + 0.5 if weighted else None
    if weighted:
        w[20, 0], w[21, 1], w[22, 0] = INF, NAN, -INF
        x[22, 7] = 0                     # 0 times an infinity
    src = rows.src.long()
    p = src.clamp(min=0)
    v = x[p // k]
    if weighted:
        v = (v.float() * w.reshape(-1)[p][:, None]).to(torch.bfloat16)
    v = torch.where((src >= 0)[:, None], v, torch.zeros_like(v))
    R = v.shape[0]
    q, s, qT, sT = fp8lib.expert_gather_quant(x, rows, w, dual=True)
    a, b, aT, bT = fp8lib.quantize_1x128(v, dual=True)
    odd = ~torch.isfinite(v)
    same_groups(q, s, a, b, odd.view(R, K // 128, 128).any(2).t())
    same_groups(qT, sT, aT, bT, odd.t().reshape(K, R // 128, 128).any(2).t())
    assert fp8lib.check_status() == 0


def test_a_weight_of_no_number_reaches_the_gradients(fp8lib):
    """The gradient of y and of the weights from a dout that holds an infinity and a NaN: those tokens' alone."""
    T, E, k, N = 90, 4, 2, 256
    gen = torch.Generator(DEV).manual_seed(1)
    idx = torch.stack([torch.randperm(E, generator=gen, device=DEV)[:k] for _ in range(T)]).to(torch.int32)
    rows = fp8lib.expert_rows(idx, E)
    y = synth.normal_bf16((rows.src.numel(), N), 1.0, 3, torch.device(DEV))
    clean = synth.normal_bf16((T, N), 1.0, 4, torch.device(DEV))
    dout = clean.clone()
    dout[5, 17], dout[40, 200] = INF, NAN
    w = torch.rand((T, k), generator=gen, device=DEV)
    got, want = (fp8lib.expert_combine_bwd(d, y, rows, w) for d in (dout, clean))
    odd = torch.zeros(T, dtype=torch.bool, device=DEV)
    odd[[5, 40]] = True
    assert torch.equal(got[4][~odd], want[4][~odd]) and not torch.isfinite(got[4][odd]).any()
    bad = ~torch.isfinite(got[1])
    assert set((rows.src.long()[bad.any(0)] // k).tolist()) == {5, 40}
    assert torch.equal(got[1][~bad], want[1][~bad])
