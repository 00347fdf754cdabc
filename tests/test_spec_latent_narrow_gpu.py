"""Attention over 16-bit latents of up to 256 columns: rings that go round many times, windows of
pages, equal ranges and whole units; tolerances as in test_spec_latent_gpu."""

import numpy as np
import pytest
import torch

from test_spec_gpu import tree
from test_spec_latent_gpu import Latents

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("latent,rope", [(256, 64), (256, 32), (136, 8)])
@pytest.mark.parametrize("kv,ql,H,ps,drafts", [
    ([2000, 31], [1, 1], 16, 1, False),           # 16 rows, windows of 8 tiles
    ([1999, 700, 0], [2, 1, 2], 16, 4, True),     # 32
    ([1500, 96], [3, 4], 16, 16, True),           # 48 and 64
    ([800], [20], 8, 8, False),                   # causal, 160 rows
])
def test_narrow_latents(latent, rope, dtype, kv, ql, H, ps, drafts):
    rng = np.random.default_rng(latent + ps)
    s = Latents(kv, ql, H, latent, rope, ps, dtype, None,
                [tree(n, rng) for n in ql] if drafts else None, seed=latent + rope + ps)
    got = s.call()
    s.check(got)
    assert torch.equal(s.call(), got)
    # larger blocks, in fewer and longer ranges
    s.check(s.call(max_kv_len=1 << 20))


def test_a_workgroup_for_each_of_more_units_than_fit():
    """700 requests of 64 rows: more than 512 workgroups, each with tiles of its own."""
    rng = np.random.default_rng(1)
    kv = [int(x) for x in rng.integers(150, 260, 700)]
    s = Latents(kv, [4] * 700, 16, 256, 64, 16, "bf16", None, [tree(4, rng) for _ in kv], seed=2)
    s.check(s.call(), requests=range(0, 700, 23))
