"""The expert operators together, as a training step and a rollout use them.

E4M3 with a scale per group has a relative error of about 2.6% (RMS of half a step of at most 2^-4); a
product of two such operands 3.7%.  The layer's result has gone through two products and three
quantizations, its gradients through some six more, adding in squares: 7% and 11%.  The test allows
25% of the norm for gradients and 12% for the forward.  Rollout and training quantize the same values
in the same groups; what differs is the order of the FP32 sums inside a product, and now and then a
code of the second product's operand by one step (2^-3 of itself): 1% of the norm."""
import os
import sys

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
DEV = "cuda"


def layer64(h, p, k, index):
    """The layer in 64 bits with the experts given; p of 64-bit tensors."""
    M, H = h.shape
    E = p.router.shape[0]
    z = h / (h.square().mean(1, keepdim=True) + 1e-5).sqrt() * p.gamma
    s = torch.softmax(z @ p.router.t(), 1)
    w = s.gather(1, index)
    w = w / (w.sum(1, keepdim=True) + 1e-20)
    gu_w, dn_w = p.w_gu.view(E, -1, H), p.w_down.view(E, H, -1)
    out = h.clone()
    for j in range(k):
        e = index[:, j]
        g, u = torch.einsum("mh,mnh->mn", z, gu_w[e]).chunk(2, dim=1)
        out = out + w[:, j:j + 1] * torch.einsum("mi,mhi->mh", torch.nn.functional.silu(g) * u, dn_w[e])
    return out


def far(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("M,H,I,E,k", [(200, 256, 128, 8, 2), (77, 384, 256, 12, 3)])
def test_training_step(fp8lib, M, H, I, E, k):
    import expert_block as ex
    p = ex.init(H, I, E, seed=3)
    gen = torch.Generator(DEV).manual_seed(5)
    h = torch.randn((M, H), generator=gen, device=DEV).to(torch.bfloat16)
    dout = (1e-3 * torch.randn((M, H), generator=gen, device=DEV)).to(torch.bfloat16)
    out, dh, grads, index = ex.train_step(h, p, k, dout)
    assert fp8lib.check_status() == 0
    p64 = ex.Experts(*[t.double().requires_grad_() for t in p])
    h64 = h.double().requires_grad_()
    want = layer64(h64, p64, k, index.long())
    want.backward(dout.double())
    assert far(out.double() - h.double(), (want - h64).detach()) < 0.12
    assert far(dh, h64.grad) < 0.25
    for name, got, w in zip(ex.Experts._fields, grads, p64):
        assert far(got, w.grad) < 0.25, name
    # an expert without tokens has no gradient
    idle = sorted(set(range(E)) - set(index.flatten().tolist()))
    for e in idle:
        assert (grads.w_gu.view(E, -1)[e] == 0).all()


def test_gradient_against_differences(fp8lib):
    """The 64-bit layer that the step is compared with: its gradient of the router against differences."""
    import expert_block as ex
    p = ex.Experts(*[t.double() for t in ex.init(128, 128, 4, seed=1)])
    gen = torch.Generator(DEV).manual_seed(2)
    h = torch.randn((6, 128), generator=gen, device=DEV, dtype=torch.float64)
    d = torch.randn((6, 128), generator=gen, device=DEV, dtype=torch.float64)
    index = torch.tensor([[0, 1], [1, 2], [3, 0], [2, 1], [0, 3], [1, 3]], device=DEV)
    r = p.router.clone().requires_grad_()
    (layer64(h, p._replace(router=r), 2, index) * d).sum().backward()
    for i, j in ((0, 3), (2, 100)):
        e = torch.zeros_like(p.router)
        e[i, j] = 1e-5
        num = sum(s * float((layer64(h, p._replace(router=p.router + s * e), 2, index) * d).sum()) for s in (1, -1)) / 2e-5
        assert abs(num - float(r.grad[i, j])) < 1e-6 * max(1.0, abs(num))


@pytest.mark.parametrize("M", [1, 5, 61])
def test_rollout_follows_training(fp8lib, M):
    import expert_block as ex
    p = ex.init(384, 256, 16, seed=4)
    h = torch.randn((200, 384), generator=torch.Generator(DEV).manual_seed(6), device=DEV).to(torch.bfloat16)
    out, _, _, index = ex.train_step(h, p, 4, torch.zeros_like(h))
    got = ex.Rollout(p, 4)(h[:M])
    assert fp8lib.check_status() == 0
    assert far(got.double() - h[:M].double(), out[:M].double() - h[:M].double()) < 0.01


def test_rollout_captured_and_replayed(fp8lib):
    """A captured rollout follows its inputs: other tokens, other experts, the same bytes as eager."""
    import expert_block as ex
    p = ex.init(256, 128, 16, seed=4)
    roll = ex.Rollout(p, 4)
    x = torch.randn((9, 256), device=DEV).to(torch.bfloat16)
    roll(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        roll(x)
        with torch.cuda.graph(g, stream=s):
            y = roll(x)
    for seed in range(3):
        x.copy_(torch.randn((9, 256), generator=torch.Generator(DEV).manual_seed(seed), device=DEV).to(torch.bfloat16))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, roll(x))
    assert fp8lib.check_status() == 0


def test_training_step_captured(fp8lib):
    """Forward and backward in one graph, with experts that change between replays."""
    import expert_block as ex
    p = ex.init(256, 128, 8, seed=4)
    h = torch.randn((150, 256), device=DEV).to(torch.bfloat16)
    d = (1e-3 * torch.randn((150, 256), device=DEV)).to(torch.bfloat16)
    ex.train_step(h, p, 2, d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        ex.train_step(h, p, 2, d)
        with torch.cuda.graph(g, stream=s):
            out, dh, grads, _ = ex.train_step(h, p, 2, d)
    for seed in range(2):
        h.copy_(torch.randn((150, 256), generator=torch.Generator(DEV).manual_seed(seed), device=DEV).to(torch.bfloat16))
        g.replay()
        torch.cuda.synchronize()
        want = ex.train_step(h, p, 2, d)
        assert torch.equal(out, want[0]) and torch.equal(dh, want[1])
        for a, b in zip(grads[2:], want[2][2:]):
            assert torch.equal(a, b)


def test_two_streams_at_once(fp8lib):
    """Rollouts on two streams whose kernels overlap give what they give alone."""
    import expert_block as ex
    rolls = [ex.Rollout(ex.init(256, 128, 16, seed=i), 4) for i in range(2)]
    xs = [torch.randn((40, 256), generator=torch.Generator(DEV).manual_seed(i), device=DEV).to(torch.bfloat16) for i in range(2)]
    want = [r(x) for r, x in zip(rolls, xs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(rolls[i](xs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])
    assert fp8lib.check_status() == 0


def test_padding_tokens(fp8lib):
    """Tokens whose logits are all -inf have no expert: they keep their residual, and the others do not
    change."""
    T, E, k, N, K = 50, 8, 2, 256, 384
    gen = torch.Generator(DEV).manual_seed(3)
    z = torch.randn((T, E), generator=gen, device=DEV)
    pad = torch.arange(T, device=DEV) % 5 == 4
    masked = torch.where(pad[:, None], float("-inf"), z)
    x = torch.randn((T, K), generator=gen, device=DEV).to(torch.bfloat16)
    res = torch.randn((T, N), generator=gen, device=DEV).to(torch.bfloat16)
    qw, sw, _ = fp8lib.quantize_128x128((0.05 * torch.randn((E * N, K), generator=gen, device=DEV)).to(torch.bfloat16))
    outs = []
    for logits in (z, masked):
        for align in (1, 128):
            r = fp8lib.route_topk(logits, k)
            rows = fp8lib.expert_rows(r.index, E, align)
            q, s, _, _ = fp8lib.expert_gather_quant(x, rows)
            outs.append(fp8lib.expert_combine(fp8lib.gemm_experts_fwd(q, s, qw, sw, rows), rows, r.weight, residual=res))
    for plain, part in zip(outs[:2], outs[2:]):
        assert torch.equal(part[pad], res[pad])
        assert torch.equal(part[~pad], plain[~pad])


def test_the_example_runs(fp8lib, capsys):
    import expert_block as ex
    ex.main(["300", "256", "128", "8", "2"])
    said = capsys.readouterr().out
    assert "status 0" in said


def test_index_of_another_width_or_values_is_safe(fp8lib):
    """Indices that a program may hand over by mistake: beyond the experts, negative, repeated."""
    T, E, k, N, K = 300, 6, 4, 128, 256
    r = np.random.default_rng(0)
    idx = r.integers(-3, E + 3, (T, k)).astype(np.int32)
    idx[:, 1] = idx[:, 0]
    x = torch.randn((T, K), device=DEV).to(torch.bfloat16)
    qw, sw, _ = fp8lib.quantize_128x128((0.05 * torch.randn((E * N, K), device=DEV)).to(torch.bfloat16))
    ys = []
    for align in (1, 128):
        rows = fp8lib.expert_rows(torch.tensor(idx, device=DEV), E, align)
        q, s, _, _ = fp8lib.expert_gather_quant(x, rows)
        ys.append(fp8lib.expert_combine(fp8lib.gemm_experts_fwd(q, s, qw, sw, rows), rows))
    assert fp8lib.check_status() == 0
    rms = ys[0].double().square().mean().sqrt()
    assert (ys[0].double() - ys[1].double()).abs().max() < 2.0 ** -6 * ys[0].abs().max() + 1e-3 * rms
    none = torch.tensor(((idx < 0) | (idx >= E)).all(1), device=DEV)
    assert (ys[0][none] == 0).all()


def test_order_captured_with_its_workspace(fp8lib):
    """A large order (two kernels and a workspace) captured twice in one graph and replayed."""
    T, E, k = 3000, 60, 4
    idx = [torch.randint(0, E, (T, k), dtype=torch.int32, device=DEV) for _ in range(2)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        fp8lib.expert_rows(idx[0], E)
        with torch.cuda.graph(g, stream=s):
            rows = [fp8lib.expert_rows(i, E, a) for i, a in zip(idx, (1, 128))]
    for seed in range(2):
        for i in idx:
            i.copy_(torch.randint(-1, E, (T, k), dtype=torch.int32, device=DEV))
        g.replay()
        torch.cuda.synchronize()
        for i, r in zip(idx, rows):
            want = fp8lib.expert_rows(i, E, r.align)
            assert all(torch.equal(a, b) for a, b in zip(r[:4], want[:4]))


def test_copies_of_an_order(fp8lib):
    """An order that was copied, moved or built from tensors gives what the original gives."""
    import copy
    idx = torch.randint(0, 8, (40, 2), dtype=torch.int32, device=DEV)
    rows = fp8lib.expert_rows(idx, 8)
    x = torch.randn((40, 256), device=DEV).to(torch.bfloat16)
    want = fp8lib.expert_gather_quant(x, rows)
    other = fp8lib.expert_rows(idx.flip(0).contiguous(), 8)
    for r in (fp8lib.ExpertRows(*rows), copy.deepcopy(rows), copy.copy(rows), rows._replace(src=rows.src.clone()),
              other._replace(pos=rows.pos, src=rows.src, start=rows.start, count=rows.count)):
        got = fp8lib.expert_gather_quant(x, r)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(ValueError, match="rows.count"):
        fp8lib.expert_gather_quant(x, rows._replace(count=rows.count.cpu()))
    with pytest.raises(RuntimeError, match="SHAPE"):
        fp8lib.expert_gather_quant(x, rows._replace(src=rows.src[:-1]))


@pytest.mark.parametrize("E", [5, 70])
def test_starts_and_counts_that_fit_nothing(fp8lib, E):
    """Starts and counts that no order has (descending, negative, beyond the rows): the products end, and
    write their own result alone."""
    T, k, N, K = 150, 3, 256, 384
    idx = torch.randint(0, E, (T, k), dtype=torch.int32, device=DEV)
    x = torch.randn((T, K), device=DEV).to(torch.bfloat16)
    dy = torch.randn((T, N), device=DEV).to(torch.bfloat16)
    qw, sw, qwT = fp8lib.quantize_128x128((0.05 * torch.randn((E * N, K), device=DEV)).to(torch.bfloat16))
    big = 2 ** 31 - 1

    def fenced(*shape):
        """A result between 64 rows on either side that have to stay."""
        n = int(np.prod(shape))
        b = torch.full((n + 128 * shape[-1],), 7.0, dtype=torch.bfloat16, device=DEV)
        return b, b[64 * shape[-1]:][:n].view(shape)

    for align in (128, 1):
        rows = fp8lib.expert_rows(idx, E, align)
        R = rows.src.numel()
        q, s, qT, sT = fp8lib.expert_gather_quant(x, rows, dual=align > 1)
        if align > 1:
            qd, sd, qdT, sdT = fp8lib.expert_gather_quant(dy, rows, dual=True)
        for pattern in ([0, R], [R, 0], [-5, big], [big, -big], [77, 300]):
            start = torch.tensor((pattern * E)[:E + 1], dtype=torch.int32, device=DEV)
            for count in ([R], [big], [-big, big], [1, R + 1]):
                count = torch.tensor((count * E)[:E], dtype=torch.int32, device=DEV)
                bad = fp8lib.ExpertRows(rows.pos, rows.src, start, count, align)
                runs = [(lambda o: fp8lib.gemm_experts_fwd(q, s, qw, sw, bad, out=o), (R, N))]
                if align > 1:
                    runs += [(lambda o: fp8lib.gemm_experts_dgrad(qd, sd, qwT, sw, bad, out=o), (R, K)),
                             (lambda o: fp8lib.gemm_experts_wgrad(qdT, sdT, qT, sT, bad, out=o), (E, N, K))]
                for f, shape in runs:
                    b, o = fenced(*shape)
                    f(o)
                    status = fp8lib.check_status()
                    assert status in (0, 8) if align == 1 else status == 0
                    edge = 64 * shape[-1]
                    assert (b[:edge] == 7).all() and (b[b.numel() - edge:] == 7).all()
        last = int(rows.start[-1])
        y = [fp8lib.gemm_experts_fwd(q, s, qw, sw, r)[:last] for r in (rows, fp8lib.ExpertRows(*rows))]
        assert torch.equal(*y) and fp8lib.check_status() == 0
