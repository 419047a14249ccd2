"""Host-side argument checks of the expert-layer operators: every refusal answers without a GPU and
launches nothing (the pointers are never dereferenced)."""
import ctypes

import pytest

import expert_reference as ref

FAKE, ODD = 0x10000, 0x10004


@pytest.fixture(scope="module")
def abi():
    from block_scaled_fp8_x1_gb300 import build_library
    from block_scaled_fp8_x1_gb300 import _abi
    build_library()
    return _abi


def status(abi, name):
    return getattr(abi, "FP8RL_OK" if name == "OK" else f"FP8RL_ERR_{name}")


ROUTE = dict(logits=FAKE, ld=64, bf16=0, score=0, bias=None, k=4, n_groups=1, top_groups=1, group_rank=1, renormalize=1,
             scale=1.0, weight=FAKE, index=FAKE)


@pytest.mark.parametrize("kw,T,E,want", [
    ({}, -1, 64, "INVALID_ARG"), ({}, 4, 0, "INVALID_ARG"), (dict(ld=63), 4, 64, "INVALID_ARG"), (dict(k=0), 4, 64, "INVALID_ARG"),
    (dict(score=2), 4, 64, "INVALID_ARG"), (dict(n_groups=0), 4, 64, "INVALID_ARG"), (dict(top_groups=2), 4, 64, "INVALID_ARG"),
    (dict(top_groups=0), 4, 64, "INVALID_ARG"), (dict(group_rank=3), 4, 64, "INVALID_ARG"), (dict(group_rank=0), 4, 64, "INVALID_ARG"),
    (dict(scale=float("nan")), 4, 64, "INVALID_ARG"), (dict(scale=float("inf")), 4, 64, "INVALID_ARG"),
    (dict(ld=1025), 4, 1025, "SHAPE"), (dict(k=33), 4, 64, "SHAPE"), (dict(k=5), 4, 4, "SHAPE"), (dict(n_groups=3), 4, 64, "SHAPE"),
    (dict(n_groups=64, top_groups=4), 4, 64, "SHAPE"), (dict(n_groups=32, top_groups=1), 4, 64, "SHAPE"),
    ({}, 1 << 30, 64, "SHAPE"), (dict(logits=None), 4, 64, "INVALID_ARG"), (dict(weight=None), 4, 64, "INVALID_ARG"),
    (dict(index=None), 4, 64, "INVALID_ARG"), (dict(logits=FAKE + 2), 4, 64, "ALIGN"), (dict(logits=FAKE + 1, bf16=1), 4, 64, "ALIGN"),
    (dict(bias=FAKE + 2), 4, 64, "ALIGN"), (dict(logits=None), 0, 64, "OK"),
])
def test_route_refusals(abi, kw, T, E, want):
    a = abi.RouteArgs(**{**ROUTE, **kw})
    assert abi.lib().fp8rl_route_topk(ctypes.byref(a), T, E, None) == status(abi, want)


BWD = dict(dweight=FAKE, logits=FAKE, ld=64, bf16=0, score=1, index=FAKE, k=4, renormalize=1, scale=1.0, dlogits=FAKE, ldd=64)


@pytest.mark.parametrize("kw,T,E,want", [
    ({}, -1, 64, "INVALID_ARG"), (dict(ldd=60), 4, 64, "INVALID_ARG"), (dict(ld=60), 4, 64, "INVALID_ARG"), (dict(k=0), 4, 64, "INVALID_ARG"),
    (dict(score=-1), 4, 64, "INVALID_ARG"), (dict(scale=float("inf")), 4, 64, "INVALID_ARG"), (dict(k=33), 4, 64, "SHAPE"),
    (dict(ld=2000, ldd=2000), 4, 2000, "SHAPE"), (dict(dweight=None), 4, 64, "INVALID_ARG"), (dict(dlogits=None), 4, 64, "INVALID_ARG"),
    (dict(dlogits=FAKE + 2), 4, 64, "ALIGN"), (dict(dweight=None), 0, 64, "OK"),
])
def test_route_bwd_refusals(abi, kw, T, E, want):
    a = abi.RouteBwdArgs(**{**BWD, **kw})
    assert abi.lib().fp8rl_route_topk_bwd(ctypes.byref(a), T, E, None) == status(abi, want)


def test_capacity(abi):
    f = abi.lib().fp8rl_expert_rows_capacity
    for T, k, E, align in ((1, 1, 1, 1), (1, 8, 64, 1), (1, 8, 64, 128), (100, 3, 7, 128), (0, 4, 8, 128), (5000, 8, 256, 128)):
        assert f(T, k, E, align) == ref.capacity(T, k, E, align)
        assert f(T, k, E, align) % align == 0
    # no index needs more: the worst one leaves one row in the last block of every expert
    for T, k, E in ((3, 1, 2), (129, 2, 3), (300, 4, 8)):
        P, n = T * k, min(E, T * k)
        most = max(sum(-(-c // 128) * 128 for c in [P - (n - 1) * a] + [a] * (n - 1)) for a in (1, 2, P // n) if P - (n - 1) * a >= 0)
        assert f(T, k, E, 128) >= most
    for bad in ((-1, 1, 1, 1), (1, 0, 1, 1), (1, 33, 64, 1), (1, 1, 1025, 1), (1, 1, 0, 1), (1, 1, 1, 64), (1 << 30, 2, 8, 1)):
        assert f(*bad) == 0


def test_sort_workspace(abi):
    f = abi.lib().fp8rl_expert_rows_workspace_bytes
    assert f(1, 8, 64) == 0 and f(0, 8, 64) == 0 and f(256, 8, 64) == 0
    assert f(16384, 8, 256) == 64 * 256 * 4
    assert f(1 << 24, 8, 256) == 128 * 256 * 4     # blocks stop growing


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), "INVALID_ARG"), (dict(k=0), "INVALID_ARG"), (dict(E=0), "INVALID_ARG"), (dict(k=33), "SHAPE"), (dict(E=1025), "SHAPE"),
    (dict(align=64), "SHAPE"), (dict(T=1 << 29), "SHAPE"), (dict(index=None), "INVALID_ARG"), (dict(pos=None), "INVALID_ARG"),
    (dict(src=None), "INVALID_ARG"), (dict(start=None), "INVALID_ARG"), (dict(count=None), "INVALID_ARG"), (dict(src=FAKE + 2), "ALIGN"),
    (dict(start=FAKE + 1), "ALIGN"), (dict(index=FAKE + 2), "ALIGN"), (dict(T=4096), "WORKSPACE"),
    (dict(T=4096, ws=FAKE, ws_bytes=100), "WORKSPACE"), (dict(T=4096, ws=FAKE + 1, ws_bytes=1 << 20), "ALIGN"),
])
def test_expert_rows_refusals(abi, kw, want):
    a = {**dict(index=FAKE, T=4, k=8, E=64, align=128, pos=FAKE, src=FAKE, start=FAKE, count=FAKE, ws=None, ws_bytes=0), **kw}
    assert abi.lib().fp8rl_expert_rows(*[a[n] for n in ("index", "T", "k", "E", "align", "pos", "src", "start", "count", "ws",
                                                        "ws_bytes")], None) == status(abi, want)


def layout(abi, **kw):
    a = {**dict(pos=FAKE, src=FAKE, start=FAKE, count=FAKE, T=4, k=2, E=8, align=128), **kw}
    a.setdefault("R", abi.lib().fp8rl_expert_rows_capacity(a["T"], a["k"], a["E"], a["align"]))
    return abi.ExpertLayout(**a)


LAYOUTS = [(dict(T=-1), "INVALID_ARG"), (dict(k=0), "INVALID_ARG"), (dict(E=0), "INVALID_ARG"), (dict(align=16), "SHAPE"),
           (dict(R=0), "SHAPE"), (dict(R=2048), "SHAPE"), (dict(E=2000), "SHAPE")]


@pytest.mark.parametrize("kw,want", LAYOUTS)
def test_layout_refusals(abi, kw, want):
    L, l = abi.lib(), layout(abi, **kw)
    r = ctypes.byref(l)
    assert L.fp8rl_expert_gather_quant(FAKE, 128, 128, None, r, FAKE, FAKE, None, None, None) == status(abi, want)
    assert L.fp8rl_expert_combine(FAKE, 128, 128, None, None, 0, r, FAKE, 128, None) == status(abi, want)
    assert L.fp8rl_expert_combine_dweight(FAKE, 128, FAKE, 128, 128, r, FAKE, None) == status(abi, want)
    for f in (L.fp8rl_gemm_experts_fwd, L.fp8rl_gemm_experts_dgrad, L.fp8rl_gemm_experts_wgrad):
        assert f(FAKE, FAKE, FAKE, FAKE, FAKE, 128, 128, r, None) == status(abi, want)


@pytest.mark.parametrize("kw,lay,want", [
    (dict(K=0), {}, "INVALID_ARG"), (dict(ldx=64), {}, "INVALID_ARG"), (dict(K=200, ldx=200), {}, "SHAPE"), (dict(x=None), {}, "INVALID_ARG"),
    (dict(q=None), {}, "INVALID_ARG"), (dict(s=None), {}, "INVALID_ARG"), (dict(qT=FAKE), {}, "INVALID_ARG"), (dict(sT=FAKE), {}, "INVALID_ARG"),
    (dict(qT=FAKE, sT=FAKE), dict(align=1), "SHAPE"), (dict(x=ODD), {}, "ALIGN"), (dict(ldx=132), {}, "ALIGN"), (dict(weight=FAKE + 2), {}, "ALIGN"),
    (dict(qT=ODD, sT=FAKE), {}, "ALIGN"), ({}, dict(src=None), "INVALID_ARG"), ({}, dict(src=FAKE + 2), "ALIGN"), ({}, dict(pos=None), "INVALID_ARG"), (dict(x=None), dict(T=0), "OK"),
])
def test_gather_refusals(abi, kw, lay, want):
    a = {**dict(x=FAKE, ldx=128, K=128, weight=None, q=FAKE, s=FAKE, qT=None, sT=None), **kw}
    assert abi.lib().fp8rl_expert_gather_quant(a["x"], a["ldx"], a["K"], a["weight"], ctypes.byref(layout(abi, **lay)), a["q"], a["s"],
                                               a["qT"], a["sT"], None) == status(abi, want)


@pytest.mark.parametrize("kw,lay,want", [
    (dict(N=0), {}, "INVALID_ARG"), (dict(ldy=64), {}, "INVALID_ARG"), (dict(ldo=64), {}, "INVALID_ARG"), (dict(res=FAKE, ldr=64), {}, "INVALID_ARG"),
    (dict(N=100), {}, "SHAPE"), (dict(y=None), {}, "INVALID_ARG"), (dict(out=None), {}, "INVALID_ARG"), (dict(y=ODD), {}, "ALIGN"),
    (dict(ldy=132), {}, "ALIGN"), (dict(ldo=132), {}, "ALIGN"), (dict(res=FAKE, ldr=132), {}, "ALIGN"), (dict(res=ODD, ldr=128), {}, "ALIGN"),
    (dict(weight=FAKE + 1), {}, "ALIGN"), ({}, dict(pos=None), "INVALID_ARG"), (dict(y=None, out=None), dict(T=0), "OK"),
])
def test_combine_refusals(abi, kw, lay, want):
    a = {**dict(y=FAKE, ldy=128, N=128, weight=None, res=None, ldr=0, out=FAKE, ldo=128), **kw}
    r = ctypes.byref(layout(abi, **lay))
    assert abi.lib().fp8rl_expert_combine(a["y"], a["ldy"], a["N"], a["weight"], a["res"], a["ldr"], r, a["out"], a["ldo"],
                                          None) == status(abi, want)
    if not set(kw) & {"res", "weight"}:
        assert abi.lib().fp8rl_expert_combine_dweight(a["y"], a["ldy"], a["out"], a["ldo"], a["N"], r, a["y"], None) == status(abi, want)


@pytest.mark.parametrize("kw,lay,want", [
    (dict(N=0), {}, "INVALID_ARG"), (dict(K=-128), {}, "INVALID_ARG"), (dict(N=200), {}, "SHAPE"), (dict(K=64), {}, "SHAPE"),
    (dict(N=1 << 30), {}, "SHAPE"), (dict(a=None), {}, "INVALID_ARG"), (dict(c=None), {}, "INVALID_ARG"), (dict(sb=None), {}, "INVALID_ARG"),
    (dict(a=ODD), {}, "ALIGN"), (dict(c=ODD), {}, "ALIGN"), ({}, dict(start=None), "INVALID_ARG"), ({}, dict(start=FAKE + 2), "ALIGN"),
])
def test_product_refusals(abi, kw, lay, want):
    g = {**dict(a=FAKE, sa=FAKE, b=FAKE, sb=FAKE, c=FAKE, N=128, K=128), **kw}
    L = abi.lib()
    for f in (L.fp8rl_gemm_experts_fwd, L.fp8rl_gemm_experts_dgrad, L.fp8rl_gemm_experts_wgrad):
        assert f(g["a"], g["sa"], g["b"], g["sb"], g["c"], g["N"], g["K"], ctypes.byref(layout(abi, **lay)), None) == status(abi, want)


def test_products_that_need_aligned_experts(abi):
    L, r = abi.lib(), ctypes.byref(layout(abi, align=1))
    for f in (L.fp8rl_gemm_experts_dgrad, L.fp8rl_gemm_experts_wgrad):
        assert f(FAKE, FAKE, FAKE, FAKE, FAKE, 128, 128, r, None) == abi.FP8RL_ERR_SHAPE
    none = ctypes.byref(layout(abi, T=0))
    assert L.fp8rl_gemm_experts_fwd(None, None, None, None, FAKE, 128, 128, none, None) == abi.FP8RL_OK
    assert L.fp8rl_gemm_experts_fwd(FAKE, FAKE, FAKE, FAKE, FAKE, 128, 128, ctypes.byref(layout(abi, align=1, count=None)), None) == abi.FP8RL_ERR_INVALID_ARG


def test_binding_refusals():
    """The binding's own checks answer before any CUDA call."""
    import torch
    from block_scaled_fp8_x1_gb300 import ops
    z = torch.zeros((4, 8))
    i = torch.zeros((4, 2), dtype=torch.int32)
    b = torch.zeros((4, 128), dtype=torch.bfloat16)
    u = torch.zeros((8, 128), dtype=torch.uint8)
    rows = ops.ExpertRows(i, i[:, 0], i[:, 0], i[:, 0], 128)
    for call in (lambda: ops.route_topk(z, 2), lambda: ops.route_topk_bwd(z, z, i), lambda: ops.expert_rows(i, 8),
                 lambda: ops.expert_gather_quant(b, rows), lambda: ops.expert_combine(b, rows), lambda: ops.expert_combine_bwd(b, b, rows, z),
                 lambda: ops.gemm_experts_fwd(u, z, u, z, rows), lambda: ops.gemm_experts_dgrad(u, z, u, z, rows),
                 lambda: ops.gemm_experts_wgrad(u, z, u, z, rows)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for call in (lambda: ops.route_topk(z.double(), 2), lambda: ops.expert_rows(i.long(), 8), lambda: ops.expert_gather_quant(z, rows),
                 lambda: ops.expert_combine(z, rows), lambda: ops.gemm_experts_fwd(z, z, u, z, rows)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError, match="matrix"):
        ops.route_topk(z[0], 2)
