"""Arguments of the speculative decoding calls on the GPU: refused before anything is enqueued."""

import pytest
import torch

from test_spec_gpu import (DEV, Setup, _i32, _sgg, _verify_call, _verify_case, _verify_check,
                           tree)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ws", [torch.zeros(64 << 20, dtype=torch.uint8), "strided", "expanded"],
                         ids=["host", "strided", "expanded"])
def test_workspace_refused(ws):
    if isinstance(ws, str):
        ws = torch.zeros(1 << 24, dtype=torch.uint8, device=DEV)[::2] if ws == "strided" else \
            torch.zeros(1, dtype=torch.uint8, device=DEV).expand(1 << 24)
    s = Setup([3000], [2], 2, 1, 64, trees=[tree(2, None, True)], seed=1)
    with pytest.raises(ValueError, match="workspace"):
        s.call(workspace=ws)
    c = _verify_case([3, 2], 9000, True, 1)
    with pytest.raises(ValueError, match="workspace"):
        _verify_call(c, workspace=ws)


def test_workspace_of_any_type_counts_its_bytes():
    ws = torch.zeros(1 << 20, device=DEV)                   # 4 MiB of floats
    s = Setup([3000], [2], 2, 1, 64, trees=[tree(2, None, True)], seed=1)
    need = s.call()
    assert torch.equal(s.call(workspace=ws), need)
    _verify_check(_verify_case([3, 2], 9000, True, 1), workspace=ws)


def test_mask_of_no_words_is_refused():
    """An empty tensor has no address, and no address stands for a causal call."""
    s = Setup([30], [4], 2, 1, 64, trees=[tree(4, None, True)], seed=1)
    with pytest.raises(ValueError, match="tree_mask"):
        s.call(tree_mask=torch.zeros((4, 0), dtype=torch.int64, device=DEV))


def test_write_takes_one_layer():
    """A cache of several layers is not taken for its first one."""
    k = torch.zeros((2, 3, 4, 1, 64), dtype=torch.bfloat16, device=DEV)
    x = torch.ones((2, 1, 64), dtype=torch.bfloat16, device=DEV)
    args = (_i32([[1, 2]]), _i32([0]), _i32([0, 2]))
    with pytest.raises(ValueError, match="layer"):
        _sgg().spec_kv_write(x, x, k, k.clone(), *args)
    assert not k.any()
    _sgg().spec_kv_write(x, x, k[1:], k.clone()[1:], *args)
    assert k[1, 1, :2].eq(1).all() and k.sum() == 128
