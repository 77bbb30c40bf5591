"""The block operators' binding on the CPU: refusals that a call's tensors meet
before any address reaches the library."""
import pytest
import torch

import structured_sparse_state_amd as pk
from tests.test_layers_binding import GPU, form, moved

Q, V, G, H, S = form(2, 2, 5, 8), form(2, 4, 5, 6), form(2, 4, 5), form(4), form(2, 4, 8, 6)
Q1, V1, G1 = form(2, 2, 8), form(2, 4, 6), form(2, 4)
X, W, R = form(2, 5, 8), form(8), form(2, dtype=torch.int64)
PLANS = {
    "linear": (pk._linear_plan, (Q, Q, V, G, V, S, S)),
    "linear, heads": (pk._linear_plan, (Q, Q, V, H, V, S, S)),
    "linear_bwd": (pk._linear_bwd_plan, (Q, Q, V, G, S, V, S, Q, Q, V, G, S)),
    "linear_bwd, heads": (pk._linear_bwd_plan, (Q, Q, V, H, S, V, S, Q, Q, V, H, S)),
    "linear_step": (pk._linear_step_plan, (Q1, Q1, V1, G1, V1, S, S)),
    "layer_norm": (pk._layer_norm_plan, (X, W, W, X, X, X, R)),
    "layer_norm_bwd": (pk._layer_norm_bwd_plan, (X, W, X, X, X, X, R, True)),
    "dropout": (pk._dropout_plan, (X, X, X, R)),
}


@pytest.mark.parametrize("name", PLANS)
def test_every_tensor_on_the_gpu(name):
    plan, forms = PLANS[name]
    plan(*forms)
    for n, f in enumerate(forms):
        if not isinstance(f, tuple):
            continue
        for other in (moved(f), (*f[:3], GPU + 1)):
            with pytest.raises(ValueError, match="one GPU"):
                plan(*forms[:n], other, *forms[n + 1:])


def test_calls_on_host_tensors():
    """No address of host memory goes to a kernel."""
    q, v, g, s = torch.zeros(2, 2, 5, 8), torch.zeros(2, 4, 5, 6), torch.zeros(2, 4, 5), torch.zeros(2, 4, 8, 6)
    x, w = torch.zeros(2, 5, 8), torch.ones(8)
    for call in (lambda: pk.linear_attention(q, q, v, g), lambda: pk.linear_attention(q, q, v),
                 lambda: pk.linear_attention_bwd(q, q, v, g, v),
                 lambda: pk.linear_attention_step(q[:, :, 0], q[:, :, 0], v[:, :, 0], g[:, :, 0], s),
                 lambda: pk.layer_norm(x, w, w), lambda: pk.layer_norm_bwd(x, x, w), lambda: pk.dropout(x, 0.5, 1)):
        with pytest.raises(ValueError, match="one GPU"):
            call()


def test_strides_of_gates():
    """[Hv] gates go with strides of 0 along sequences and steps, and so do the
    strides of views."""
    rows = lambda plan: [(r.b, r.h, r.l) for r in plan[1]]  # noqa: E731
    assert rows(pk._linear_plan(Q, Q, V, H, V, None, None))[3] == (0, 1, 0)
    assert rows(pk._linear_plan(Q, Q, V, None, V, None, None))[3] == (0, 0, 0)
    token = torch.empty(2, 5, 4).transpose(1, 2)
    f = (token.shape, token.stride(), token.dtype, GPU)
    assert rows(pk._linear_plan(Q, Q, V, f, V, None, None))[3] == (20, 1, 4)
    assert rows(pk._linear_bwd_plan(Q, Q, V, H, None, V, None, Q, Q, V, H, None))[8] == (0, 1, 0)


def test_rows_of_fewer_dimensions():
    for shape in ((8,), (5, 8), (2, 5, 8), (3, 2, 5, 8)):
        f = form(*shape)
        (flag, *sizes), rows = pk._dropout_plan(f, None, f, None)
        assert flag == 0 and tuple(sizes) == (1,) * (4 - len(shape)) + shape
        r = rows[0]
        assert (r.b, r.h, r.l) == (0,) * (4 - len(shape)) + tuple(f[1][:-1])
