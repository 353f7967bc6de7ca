"""Host-side checks of the activation calls: sizes, and refusals that need no GPU."""
import ctypes

import pytest

from fac_whitening_gb300 import gift as G


def _lib_or_skip():
    try:
        return G.lib()
    except RuntimeError as e:  # not built in this checkout
        pytest.skip(str(e))


def test_checkpoint_sizes():
    _lib_or_skip()
    assert G.gift_act_sizes("e4m3", 10, 256) == (2560, 20)
    assert G.gift_act_sizes("e5m2", 3, 129) == (387, 6)
    assert G.gift_act_sizes("e4m3", 1, 1) == (1, 1)
    assert G.gift_act_sizes("e4m3", 1 << 20, 1 << 16) == (1 << 36, 1 << 29)   # past 32 bits
    for fmt, T, d in (("nvfp4", 4, 128), ("f32", 4, 128), ("e4m3", 0, 128), ("e4m3", 4, 0), ("e4m3", (1 << 30) + 1, 1)):
        with pytest.raises(G.GiftError):
            G.gift_act_sizes(fmt, T, d)


def test_null_context_is_rejected():
    lib = _lib_or_skip()
    e4m3, bf16, n = G.FMT["e4m3"], G.DTYPE["bf16"], None
    for op in ("layernorm_backward", "weight_grad"):
        assert lib.gift_act_workspace_bytes(n, G.OP[op], bf16, 4, 4, 4) == ctypes.c_size_t(-1).value
    assert lib.gift_act_encode(n, n, bf16, 4, 4, e4m3, n, n, n, n) == G.ERR_INVALID_ARG
    assert lib.gift_act_decode(n, n, n, e4m3, 4, 4, n, bf16, n, n) == G.ERR_INVALID_ARG
    assert lib.gift_layernorm_forward(n, n, bf16, 4, 4, n, n, 1e-5, n, n, n, e4m3, n, n, n, n) == G.ERR_INVALID_ARG
    assert lib.gift_layernorm_backward(n, n, bf16, 4, 4, n, 0, n, e4m3, n, n, n, n, n, n, n, 0, n,
                                       n) == G.ERR_INVALID_ARG
    assert lib.gift_weight_grad(n, n, bf16, n, n, e4m3, 4, 4, 4, n, n, n, n, n, 0, n, n) == G.ERR_INVALID_ARG
