"""Arguments of the mixture-of-experts operators whose shape decides what they mean."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import moe8_reference as R  # noqa: E402

D = torch.float64


@pytest.mark.parametrize("X,N", [(3, 48), (4, 4), (1, 20)])
def test_the_experts_bias(X, N):
    """bias [E, N] alone: another shape of as many values would give channels the values of others."""
    import bit_weight_only_offline_amd as Q
    g = torch.Generator(device="cuda")
    g.manual_seed(X * N)
    w, ws = R.weights(g, (X, N, 160), True)
    x, xs = R.activations(g, 2 * X, 160, True)
    pw, counts = Q.pack_f8(w, ws), torch.full((X,), 2, dtype=torch.int32, device="cuda")
    bias = torch.randint(-9, 10, (X, N), generator=g, device="cuda").to(torch.bfloat16)
    plain = Q.grouped_linear_f8(x, xs, pw, counts, out_dtype=torch.float32)
    ref = plain + bias.float().repeat_interleave(2, 0)
    assert torch.equal(Q.grouped_linear_f8(x, xs, pw, counts, bias=bias, out_dtype=torch.float32), ref)
    # a view of any strides
    turned = bias.t().contiguous().t()
    assert torch.equal(Q.grouped_linear_f8(x, xs, pw, counts, bias=turned, out_dtype=torch.float32), ref)
    for name, bad in {"turned": bias.t().contiguous(), "flat": bias.reshape(-1), "three": bias[None], "halves": bias.reshape(-1, 2)}.items():
        if bad.shape == (X, N):
            continue                                          # as many experts as channels
        with pytest.raises(Q.QLinearError):
            Q.grouped_linear_f8(x, xs, pw, counts, bias=bad)
            print("not refused:", name, flush=True)
