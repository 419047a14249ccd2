"""A request for more CTAs than K has blocks of 128 takes as many as there are blocks."""
import pytest
import torch

from block_scaled_fp8_x1_gb300 import _abi, synth

FAKE = 0x10000


@pytest.mark.skipif(torch.cuda.is_available(), reason="calls that are not refused would launch on these pointers")
@pytest.mark.parametrize("K", [256, 512, 768, 1024])
def test_no_split_is_refused(K):
    from block_scaled_fp8_x1_gb300 import build_library
    build_library()
    for splits in range(9):
        for M in (1, 2, 9, 16):
            st = _abi.lib().fp8rl_matvec_nvfp4(FAKE, M, K, K, FAKE, FAKE, FAKE, 128, FAKE, 128, splits, None)
            assert st in (_abi.FP8RL_ERR_CUDA, _abi.FP8RL_ERR_UNSUPPORTED_DEVICE), (M, splits)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 6, 16])
@pytest.mark.parametrize("K", [256, 768])
def test_more_splits_than_blocks(fp8lib, M, K):
    w = fp8lib.quantize_nvfp4(synth.normal_bf16((384, K), 0.02, 3, "cuda"))
    x = synth.normal_bf16((M, K), 1.0, 4, "cuda")
    want = fp8lib.matvec_nvfp4(x, *w, splits=K // 128)
    for splits in range(K // 128 + 1, 9):
        assert torch.equal(fp8lib.matvec_nvfp4(x, *w, splits=splits), want)
    assert fp8lib.check_status() == _abi.FP8RL_OK
