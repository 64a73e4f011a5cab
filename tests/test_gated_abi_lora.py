"""CPU-only checks of the gated block's torch-level call: a LoRA pair that is not whole is refused, never left out."""
import pytest
import torch

import activation_sparse_gemm_b200 as rl
from activation_sparse_gemm_b200 import build as rl_build

M, D, F, R = 4, 64, 128, 16


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def call(**more):
    rl_build.build()
    return rl.gated_mlp(bf16(M, D), bf16(F, D), bf16(F, D), bf16(D, F), **more)


@pytest.mark.parametrize("pair", [dict(L_A=bf16(D, R)), dict(L_B=bf16(R, F)), dict(L_A=bf16(D, R), L_B=bf16(F)),
                                  dict(L_A=bf16(D, R), L_B=bf16(1, R, F))], ids=lambda p: ",".join(p))
def test_pair_that_is_not_whole(pair):
    with pytest.raises(ValueError, match="L_B"):
        call(mode_down=rl.MODE_SPARSE, **pair)


def test_pair_without_a_mode():
    with pytest.raises(ValueError, match="mode_down"):
        call(L_A=bf16(D, R), L_B=bf16(R, F))


def test_whole_pairs_and_none_reach_the_check_of_the_tensors():
    for more in (dict(), dict(mode_down=rl.MODE_SPARSE), dict(mode_down=rl.MODE_SPARSE, L_A=bf16(D, R), L_B=bf16(R, F)),
                 dict(mode_down=rl.MODE_DENSE_SKIP, L_A=bf16(D, R), L_B=bf16(R, F))):
        with pytest.raises(ValueError, match="CUDA"):
            call(**more)
