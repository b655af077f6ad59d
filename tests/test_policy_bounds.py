"""Sizes that the policy calls refuse, on the CPU."""
import ctypes

import pytest


@pytest.mark.parametrize("T", [2 ** 31 - 1, 2 ** 31 - 1024, 2 ** 31 - 4096])
def test_more_tokens_than_positions_have_bits(T, moe_lib):
    """The loss's sum steps by 1024 past the last token, in 31 bits."""
    lib, p, q = moe_lib.load(), ctypes.c_void_p(256), ctypes.c_void_p(4096)
    c = moe_lib.make_policy_config(T, 1)
    assert lib.moe_policy_loss(ctypes.byref(c), *[p] * 8, q, p, None) == moe_lib.MOE_ERR_UNSUPPORTED
    assert lib.moe_token_logp(ctypes.byref(c), p, p, p, None) == moe_lib.MOE_ERR_UNSUPPORTED
    assert lib.moe_policy_workspace_bytes(ctypes.byref(c)) == 0
    c = moe_lib.make_policy_config(2 ** 31 - 4097, 1)
    assert moe_lib.policy_workspace_bytes(c) >= 4 * (2 ** 31 - 4097)
