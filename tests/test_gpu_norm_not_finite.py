"""What a row that is not finite leaves in the sums over rows: NaN in dgain where s is not finite, nothing in dbias, which
is the sum of dy alone; what is not finite in dy stays in its own row and columns."""
import pytest
import torch

pytestmark = pytest.mark.gpu

T = 300


def backward(moe, d, dtype, s, dy):
    """The gradient with the statistics that the forward pass takes of s."""
    c = moe.make_norm_config(T, d, dtype=dtype)
    gain = torch.linspace(0.5, 1.5, d, device="cuda")
    y, mean, rstd = torch.empty_like(s), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    moe.layer_norm(c, s, gain, None, y, mean=mean, rstd=rstd)
    dx, dgain, dbias = torch.empty_like(s), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    ws = torch.empty(moe.norm_workspace_bytes(c), dtype=torch.uint8, device="cuda")
    moe.layer_norm_backward(c, dy, s, gain, mean, rstd, dx, dgain, dbias, ws)
    moe.get_error()
    return y, dx, dgain, dbias


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f32", 37), ("bf16", 1024), ("f32", 1023), ("bf16", 12288), ("f32", 9001)])
def test_rows_in_the_sums(dtype, d, moe_lib, cuda_device):
    g = torch.Generator(device="cuda").manual_seed(d)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    s = torch.randn(T, d, generator=g, device="cuda").to(dt)
    dy = torch.randn(T, d, generator=g, device="cuda").to(dt)
    y0, dx0, dgain0, dbias0 = backward(moe_lib, d, dtype, s, dy)
    others = torch.ones(T, dtype=torch.bool, device="cuda")
    others[[5, T - 1]] = False
    for value in (float("nan"), float("inf"), float("-inf")):
        bad = s.clone()
        bad[5, d // 2] = bad[T - 1, d - 1] = value
        y, dx, dgain, dbias = backward(moe_lib, d, dtype, bad, dy)
        assert torch.isnan(y[~others]).all() and torch.isnan(dx[~others]).all() and torch.isnan(dgain).all()
        assert torch.equal(dbias, dbias0) and torch.equal(dx[others], dx0[others]) and torch.equal(y[others], y0[others])
        bad = dy.clone()
        bad[5, d // 2] = bad[T - 1, d - 1] = value
        _, dx, dgain, dbias = backward(moe_lib, d, dtype, s, bad)
        spoilt = torch.zeros(d, dtype=torch.bool, device="cuda")
        spoilt[[d // 2, d - 1]] = True
        assert not torch.isfinite(dx[~others]).any() and torch.equal(dx[others], dx0[others])
        assert not torch.isfinite(dgain[spoilt]).any() and not torch.isfinite(dbias[spoilt]).any()
        assert torch.equal(dgain[~spoilt], dgain0[~spoilt]) and torch.equal(dbias[~spoilt], dbias0[~spoilt])


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f32", 37), ("bf16", 1024), ("f32", 1023), ("bf16", 12288), ("f32", 9001)])
def test_sums_beyond_fp32(dtype, d, moe_lib, cuda_device):
    """Finite rows whose squares (row 3) or whose sum (row 4) fp32 does not hold."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    s = torch.randn(8, d, device="cuda").to(dt)
    s[3], s[4] = 1e20, 3e38
    s[3, ::2] = -1e20
    c = moe_lib.make_norm_config(8, d, dtype=dtype)
    bias = torch.linspace(-1, 1, d, device="cuda")
    y, mean, rstd = torch.empty_like(s), torch.empty(8, device="cuda"), torch.empty(8, device="cuda")
    moe_lib.layer_norm(c, s, None, bias, y, mean=mean, rstd=rstd)
    moe_lib.get_error()
    assert float(rstd[3]) == 0 and torch.equal(y[3], bias.to(dt))
    assert torch.isnan(y[4]).all()
    assert torch.isfinite(y[[0, 1, 2, 5, 6, 7]]).all()
