"""Which beta1 the 8-bit first moment takes: one that lets it decay (no GPU needed)."""
import ctypes
import os

import pytest
import torch

from block_scaled_fp4_06_amd import nvfp4 as N
from block_scaled_fp4_06_amd import optim
from test_train_checks import FAKE, OK, UNSUPPORTED, table


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(N.LIB_PATH):
        from block_scaled_fp4_06_amd import build
        build.build()
    return N.load()


def stuck(beta1):
    """E4M3 values above the smallest normal one that a step without a gradient leaves."""
    m = torch.arange(9, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    return int(((m * beta1).to(torch.float8_e4m3fn).float() == m).sum())


def test_first_moment_decays_up_to_the_bound():
    assert all(stuck(b) == 0 for b in (0.0, 0.5, 0.8, 0.9, 0.93, 0.944))
    assert stuck(0.945) > 0 and stuck(0.95) > 0 and 0.944 < optim.MAX_BETA1_8 < 0.945


def test_larger_beta1_is_refused_with_8_bits():
    p = [torch.zeros(300)]
    with pytest.raises(ValueError, match="17/18"):
        optim.AdamW(p, betas=(0.95, 0.99), bits=8)
    with pytest.raises(ValueError, match="17/18"):
        optim.AdamW(p, betas=(0.95, 0.99), state=optim.new_state(p, 8))
    optim.AdamW(p, betas=(0.95, 0.99), bits=32)
    optim.AdamW(p, betas=(0.94, 0.99), bits=8)
    for bits, beta1, want in ((8, 0.95, UNSUPPORTED), (8, 0.945, UNSUPPORTED), (8, 17.0 / 18.0, OK),
                              (32, 0.95, OK)):
        rc, at, keep = table(bits=bits, n=0)   # (nothing to launch)
        assert rc == OK
        prm = N.AdamWParams(1e-3, beta1, 0.99, 1e-8, 1, 0, 0, 0, None)
        assert N.nvfp4_adamw_step(at, FAKE, (ctypes.c_void_p * 1)(FAKE), prm, None) == want
