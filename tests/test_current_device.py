"""The layer and block operators while another device than the tensors' is the
current one: a launch on a default stream goes to the current device, so the
binding makes the tensors' device current for the call."""
import contextlib

import pytest
import torch

import structured_sparse_state_amd as pk


class Recorder:
    """In the place of torch.cuda.device: notes what is made current."""

    def __init__(self, monkeypatch, current):
        self.made = []
        monkeypatch.setattr(pk, "_current_device", lambda: self.made[-1] if self.made else current)
        monkeypatch.setattr(torch.cuda, "device", self)

    @contextlib.contextmanager
    def __call__(self, device):
        self.made.append(torch.device("cuda", device).index if isinstance(device, int) else device.index)
        yield
        self.made.append(None)


class On:
    is_cuda = True

    def __init__(self, device):
        self.get_device = lambda: device


def test_a_call_runs_on_its_tensors_device(monkeypatch):
    record = Recorder(monkeypatch, current=1)
    seen = []

    def entry(*args):
        seen.append((args, list(record.made)))
        return pk.PDSSM_OK

    pk._run(entry, On(1), 7, "a", "b")
    pk._run(entry, On(0), 7, "c")
    assert seen == [(("a", "b", 7), []), (("c", 7), [0])] and record.made == [0, None]


def test_errors_leave_the_device_as_it_was(monkeypatch):
    Recorder(monkeypatch, current=0)
    with pytest.raises(pk.PdssmError):
        pk._run(lambda *args: pk.PDSSM_ERR_DIM, On(0), 0)


@pytest.mark.gpu
def test_every_operator(monkeypatch):
    """Every entry point with device 1 taken for the current one."""
    gen = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(s, generator=gen).to("cuda:0")  # noqa: E731
    q, v, g, s = r(1, 1, 70, 32) / 6, r(1, 2, 70, 32), -r(1, 2, 70).abs(), r(1, 2, 32, 32)
    beta, w, x = torch.sigmoid(g), r(32), r(9, 32)
    q1, v1, g1, b1 = (t[:, :, 0] for t in (q, v, g, beta))
    after = torch.empty_like(s)
    calls = {
        "delta_rule": lambda: pk.delta_rule(q, q, v, g, beta, s),
        "delta_rule_bwd": lambda: pk.delta_rule_bwd(q, q, v, g, beta, v, s, s),
        "delta_step": lambda: pk.delta_step(q1, q1, v1, g1, b1, s, s_out=after),
        "qk_norm_rope": lambda: pk.qk_norm_rope(q, v, w, w),
        "qk_norm_rope_bwd": lambda: pk.qk_norm_rope_bwd(q, v, q, v, w, w),
        "linear_attention": lambda: pk.linear_attention(q, q, v, g, s),
        "linear_attention_bwd": lambda: pk.linear_attention_bwd(q, q, v, g, v, s, s),
        "linear_attention_step": lambda: pk.linear_attention_step(q1, q1, v1, g1, s, s_out=after),
        "layer_norm": lambda: pk.layer_norm(x, w, w, residual=x, p=0.5, seed=1),
        "layer_norm_bwd": lambda: pk.layer_norm_bwd(x, x, w, p=0.5, seed=1),
        "dropout": lambda: pk.dropout(x, 0.5, 1),
    }
    flat = lambda o: [t for t in (o if isinstance(o, tuple) else (o,)) if t is not None]  # noqa: E731
    for name, call in calls.items():
        print(f"[case] {name}", flush=True)
        want = flat(call())
        with monkeypatch.context() as patch:
            record = Recorder(patch, current=1)
            got = flat(call())
        torch.cuda.synchronize()
        assert record.made == [0, None], name
        for a, b in zip(got, want):
            assert torch.equal(a, b), name
