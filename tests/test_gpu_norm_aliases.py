"""The layer norm's results over its inputs, and two results in one place."""
import pytest
import torch

import structured_sparse_state_amd as pk


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("given", ["x", "a view of x", "on a stream"])
def test_h_when_y_goes_over_x(dtype, given):
    """h is x before the call, from which the gradients are taken, also where y
    takes the place of x."""
    gen = torch.Generator().manual_seed(1)
    x, dy = (torch.randn(50, 200, generator=gen).to("cuda:0", dtype) for _ in range(2))
    w, b = torch.randn(200, generator=gen).cuda(), torch.randn(200, generator=gen).cuda()
    want_y, want_h = pk.layer_norm(x, w, b)
    assert want_h is x
    want = pk.layer_norm_bwd(x, dy, w, want_db=True)
    over = x.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kw = {"stream": side} if given == "on a stream" else {}
    y, h = pk.layer_norm(over, w, b, out=over[:] if given == "a view of x" else over, **kw)
    torch.cuda.current_stream().wait_stream(side)
    got = pk.layer_norm_bwd(h, dy, w, want_db=True)
    torch.cuda.synchronize()
    assert torch.equal(y, want_y) and torch.equal(over, want_y) and torch.equal(h, want_h)
    for a, c in zip(got, want):
        assert torch.equal(a, c)
    # a place of the caller's for h, or none that is needed
    over, place = x.clone(), torch.empty_like(x)
    assert pk.layer_norm(over, w, b, out=over, h=place)[1] is place and torch.equal(place, x)
    assert pk.layer_norm(x, w, b, out=torch.empty_like(x))[1] is x


def test_two_results_are_two_tensors():
    x, t = torch.zeros(2, 5, 8), torch.zeros(2, 5, 8)
    for same in (t, t[:]):
        for kw in (dict(), dict(residual=x), dict(residual=x, p=0.5, seed=1)):
            with pytest.raises(ValueError, match="two tensors"):
                pk.layer_norm(x, out=t, h=same, **kw)
        with pytest.raises(ValueError, match="two tensors"):
            pk.layer_norm_bwd(x, x, out=(t, same), p=0.5, seed=1)
