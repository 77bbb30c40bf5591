"""The layer operators' binding on the CPU: refusals that a call's tensors meet
before any address reaches the library."""
import pytest
import torch

import structured_sparse_state_amd as pk

GPU, CPU = 0, -1


def form(*shape, dtype=torch.float32, device=GPU):
    """What the plans see of a tensor that lies on a device."""
    t = torch.empty(shape, dtype=dtype)
    return (t.shape, t.stride(), t.dtype, device)


def moved(f):
    return (*f[:3], CPU)


Q, V, G, S = form(2, 2, 5, 8), form(2, 4, 5, 6), form(2, 4, 5), form(2, 4, 8, 6)
Q1, V1, G1 = form(2, 2, 8), form(2, 4, 6), form(2, 4)
X, W, T, P = form(2, 3, 5, 8), form(8), form(9, 2), form(2, 5, dtype=torch.int32)
PLANS = {
    "delta": (pk._delta_plan, (Q, Q, V, G, G, V, S, S)),
    "delta_bwd": (pk._delta_bwd_plan, (Q, Q, V, G, G, S, V, S, Q, Q, V, G, G, S)),
    "step": (pk._step_plan, (Q1, Q1, V1, G1, G1, V1, S, S)),
    "norm": (pk._norm_plan, (X, X, W, W, T, T, P, "rms", "half", X, X)),
    "norm_bwd": (pk._norm_bwd_plan, (X, X, W, W, T, T, P, "rms", "half", X, X, X, X)),
}


@pytest.mark.parametrize("name", PLANS)
def test_every_tensor_on_the_gpu(name):
    plan, forms = PLANS[name]
    plan(*forms)
    for n, f in enumerate(forms):
        if isinstance(f, str):
            continue
        for other in (moved(f), (*f[:3], GPU + 1)):
            with pytest.raises(ValueError, match="one GPU"):
                plan(*forms[:n], other, *forms[n + 1:])


def test_calls_on_host_tensors():
    """No address of host memory goes to a kernel."""
    q, v, g, s = torch.zeros(2, 2, 5, 8), torch.zeros(2, 4, 5, 6), torch.zeros(2, 4, 5), torch.zeros(2, 4, 8, 6)
    x, w = torch.zeros(2, 3, 5, 8), torch.ones(8)
    for call in (lambda: pk.delta_rule(q, q, v, g, g), lambda: pk.delta_rule_bwd(q, q, v, g, g, v),
                 lambda: pk.delta_step(q[:, :, 0], q[:, :, 0], v[:, :, 0], g[:, :, 0], g[:, :, 0], s),
                 lambda: pk.qk_norm_rope(x, x, w, w), lambda: pk.qk_norm_rope_bwd(x, x, x, x, w, w)):
        with pytest.raises(ValueError, match="one GPU"):
            call()


def test_workspaces():
    ws = torch.empty(64, dtype=torch.uint8)
    assert pk._workspace(64, ws, ws.device) is ws
    for bad in (ws[:63], ws[::2], torch.empty(1, dtype=torch.uint8).expand(64), ws.to("meta")):
        with pytest.raises(ValueError):
            pk._workspace(64, bad, ws.device)


def test_alignment_of_tables():
    """Element alignment is asked for where rows are not whole runs, 16 bytes where they are."""
    fake = 1 << 20      # never dereferenced: both calls are refused
    call = lambda cos, R: pk.pdssm_qk_norm_rope_fwd(  # noqa: E731
        fake, fake, None, None, cos, fake, None, fake, fake, 2, 4, 2, 10, 64, R, 10, 1e-6, 1, None, 0)
    assert call(fake + 2, 20) == pk.PDSSM_ERR_ALIGN
    assert call(fake + 4, 32) == pk.PDSSM_ERR_ALIGN


def test_words_and_tables_of_the_norm():
    x, t = torch.zeros(2, 3, 5, 8), torch.zeros(9)
    for kw in (dict(kind="max"), dict(pairs="thirds"), dict(kind=None), dict(cos=t, sin=t),
               dict(cos=t[:8].view(2, 2, 2), sin=t[:8].view(2, 2, 2))):
        with pytest.raises(ValueError):
            pk.qk_norm_rope(x, x, **kw)
        with pytest.raises(ValueError):
            pk.qk_norm_rope_bwd(x, x, x, x, **kw)
    with pytest.raises(ValueError, match="rms, l2"):
        pk.qk_norm_rope(x, x, kind="max")
