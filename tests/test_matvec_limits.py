"""How long K may be in fp8rl_matvec_nvfp4: the answer is the same for every token count, and a
refusal comes before anything is launched."""
import pytest
import torch

import block_reference as ref
from block_scaled_fp8_x1_gb300 import _abi, synth

FAKE = 0x10000


@pytest.fixture(scope="module")
def abi():
    from block_scaled_fp8_x1_gb300 import build_library
    build_library()
    return _abi


def answer(abi, M, K, splits, N=128):
    """The call's status without a GPU: FP8RL_ERR_SHAPE, or the missing device's."""
    return abi.lib().fp8rl_matvec_nvfp4(FAKE, M, K, K, FAKE, FAKE, FAKE, N, FAKE, N, splits, None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="calls that are not refused would launch on these pointers")
@pytest.mark.parametrize("splits", range(9))
def test_every_token_count_has_the_same_longest_k(abi, splits):
    longest = 768                      # from here on K has the eight blocks that a cluster of eight needs
    for K in range(1024, 1 << 19, 256):
        one = answer(abi, 1, K, splits)
        for M in range(2, 17):
            assert answer(abi, M, K, splits) == one, (M, K)
        if one != abi.FP8RL_ERR_SHAPE:
            assert longest == K - 256, f"{longest} refused, {K} accepted"
            longest = K
    assert 22016 * max(splits, 1) <= longest < (1 << 19) - 256
    assert answer(abi, 1, 1 << 24, splits) == abi.FP8RL_ERR_SHAPE


def product(fp8lib, x, w, **kw):
    """matvec_nvfp4 within its bound of the 64-bit product: (32 + K / 128) 2^-22 of the terms'
    magnitudes for the sum and one BF16 rounding."""
    y = fp8lib.matvec_nvfp4(x, *w, **kw)
    wd = ref.decode_nvfp4(*w)
    want, mag = x.double() @ wd.t(), x.double().abs() @ wd.abs().t()
    bound = ref.BF16_HALF * want.abs() + (32 + x.shape[1] / 128) * 2.0 ** -22 * mag
    assert bool(((y.double() - want).abs() <= bound).all())
    return y


# 86 blocks of 128 for each CTA and more: two tokens' x fit beside a ring of three units, one
# token's beside a ring of five does not from 166 blocks a CTA on
@pytest.mark.gpu
@pytest.mark.parametrize("M,K,splits", [(1, 22016, 1), (2, 22016, 1), (3, 22016, 1), (5, 22016, 1), (1, 44032, 2), (1, 172032, 0),
                                        (3, 172032, 8), (16, 22016, 1), (1, 45312, 1)])
def test_long_rows(fp8lib, M, K, splits):
    x = synth.normal_bf16((M, K), 1.0, M, "cuda", outlier_channels=2, outlier_scale=30.0)
    w = fp8lib.quantize_nvfp4(synth.normal_bf16((256, K), 0.02, 3, "cuda"))
    y = product(fp8lib, x, w, splits=splits)
    assert torch.equal(y, fp8lib.matvec_nvfp4(x, *w, splits=splits))
    assert fp8lib.check_status() == _abi.FP8RL_OK


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 3, 16])
def test_a_refusal_writes_nothing(fp8lib, M):
    K = 65536
    w = fp8lib.quantize_nvfp4(synth.normal_bf16((128, K), 0.02, 3, "cuda"))
    x = synth.normal_bf16((M, K), 1.0, M, "cuda")
    y = torch.full((M, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(_abi.Fp8rlError) as e:
        fp8lib.matvec_nvfp4(x, *w, out=y, splits=1)
    assert e.value.status == _abi.FP8RL_ERR_SHAPE
    torch.cuda.synchronize()
    assert bool((y == 7.0).all())
