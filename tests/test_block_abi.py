"""The block operators' C entry points and binding on the CPU: exports,
constants, and every refusal before any HIP call."""
import re

import pytest
import torch

import structured_sparse_state_amd as pk

FAKE = 1 << 20      # an aligned, never-dereferenced address


@pytest.fixture(scope="module")
def lib():
    return pk.library()


def test_exports_every_declared_function(lib):
    names = pk.header_functions(pk.BLOCK_HEADER)
    assert set(names) == {"pdssm_linear_fwd", "pdssm_linear_workspace_bytes", "pdssm_linear_bwd",
                          "pdssm_linear_bwd_workspace_bytes", "pdssm_linear_step", "pdssm_layer_norm_fwd",
                          "pdssm_layer_norm_bwd", "pdssm_layer_norm_bwd_workspace_bytes", "pdssm_dropout"}
    for n in names:
        assert hasattr(lib, n) and hasattr(pk, n), n


def test_constants_match_binding():
    defs = dict(re.findall(r"#define\s+(PDSSM_[A-Z0-9_]+)\s+(0x[0-9A-Fa-f]+)u", open(pk.BLOCK_HEADER).read()))
    assert len(defs) == 2
    for name, val in defs.items():
        assert getattr(pk, name) == int(val, 16), name


SIZES = dict(B=2, Hk=2, Hv=4, L=100, Dk=64, Dv=32)
BAD_SIZES = [dict(B=-1), dict(Hk=-1), dict(Hv=-4), dict(L=-1), dict(L=(1 << 30) + 1), dict(Dk=0), dict(Dk=129),
             dict(Dv=0), dict(Dv=129), dict(Hk=0), dict(Hk=3), dict(B=1 << 40), dict(B=1 << 27, L=1 << 20)]


def _fwd(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, s0=None, o=FAKE, s_final=None, **SIZES, flags=1, strides=None, ws=FAKE,
             ws_bytes=1 << 40)
    a.update(kw)
    return pk.pdssm_linear_fwd(a["q"], a["k"], a["v"], a["g"], a["s0"], a["o"], a["s_final"], a["B"], a["Hk"], a["Hv"],
                               a["L"], a["Dk"], a["Dv"], 1.0, a["flags"], a["strides"], a["ws"], a["ws_bytes"], 0)


def _bwd(**kw):
    names = ("q", "k", "v", "g", "s0", "d_o", "ds_final", "dq", "dk", "dv", "dg", "ds0")
    a = dict({n: FAKE for n in names}, s0=None, ds_final=None, ds0=None, **SIZES, flags=1, strides=None, ws=FAKE,
             ws_bytes=1 << 40)
    a.update(kw)
    return pk.pdssm_linear_bwd(*(a[n] for n in names), a["B"], a["Hk"], a["Hv"], a["L"], a["Dk"], a["Dv"], 1.0,
                               a["flags"], a["strides"], a["ws"], a["ws_bytes"], 0)


def _step(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, s=FAKE, o=FAKE, s_out=FAKE, B=2, Hk=2, Hv=4, Dk=64, Dv=32, flags=1)
    a.update(kw)
    return pk.pdssm_linear_step(a["q"], a["k"], a["v"], a["g"], a["s"], a["o"], a["s_out"], a["B"], a["Hk"], a["Hv"],
                                a["Dk"], a["Dv"], 1.0, a["flags"], None, 0)


def test_linear_refusals(lib):
    for call in (_fwd, _bwd):
        for bad in BAD_SIZES:
            assert call(**bad) == pk.PDSSM_ERR_DIM, bad
        assert call(flags=8) == pk.PDSSM_ERR_FLAGS
        for name in ("q", "k", "v", "ws"):
            assert call(**{name: None}) == pk.PDSSM_ERR_NULL, name
            assert call(**{name: FAKE + 1}) == pk.PDSSM_ERR_ALIGN, name
        assert call(s0=FAKE + 4) == pk.PDSSM_ERR_ALIGN
        assert call(ws=FAKE + 8) == pk.PDSSM_ERR_ALIGN
        assert call(g=FAKE + 2) == pk.PDSSM_ERR_ALIGN
    assert _fwd(flags=3) == pk.PDSSM_ERR_FLAGS
    assert _bwd(flags=pk.PDSSM_NO_DG | pk.PDSSM_DG_HEADS) == pk.PDSSM_ERR_FLAGS
    assert _fwd(o=None) == pk.PDSSM_ERR_NULL
    assert _fwd(s_final=FAKE + 4) == pk.PDSSM_ERR_ALIGN
    for name in ("d_o", "dq", "dk", "dv", "dg"):
        assert _bwd(**{name: None}) == pk.PDSSM_ERR_NULL, name
        assert _bwd(**{name: FAKE + 1}) == pk.PDSSM_ERR_ALIGN, name
    for name in ("ds0", "ds_final"):
        assert _bwd(**{name: FAKE + 4}) == pk.PDSSM_ERR_ALIGN, name
    s = list(SIZES.values())
    assert _fwd(ws_bytes=pk.pdssm_linear_workspace_bytes(*s, 1) - 1) == pk.PDSSM_ERR_WORKSPACE
    for flags in (1, 1 | pk.PDSSM_NO_DG, 1 | pk.PDSSM_DG_HEADS):
        assert _bwd(flags=flags, ws_bytes=pk.pdssm_linear_bwd_workspace_bytes(*s, flags) - 1) == pk.PDSSM_ERR_WORKSPACE
    row = (1000, 100, 10)
    for bad in ((1000, 100, -1), (1000, 100, 1 << 23)):
        for n in range(5):
            assert _fwd(strides=[row] * n + [bad] + [row] * (4 - n)) == pk.PDSSM_ERR_DIM, n
        for n in range(9):
            assert _bwd(strides=[row] * n + [bad] + [row] * (8 - n)) == pk.PDSSM_ERR_DIM, n
    for bad in BAD_SIZES:
        sizes = list({**SIZES, **bad}.values())
        assert pk.pdssm_linear_workspace_bytes(*sizes, 1) == 0 and pk.pdssm_linear_bwd_workspace_bytes(*sizes, 1) == 0
    assert pk.pdssm_linear_workspace_bytes(*s, 2) == 0 and pk.pdssm_linear_bwd_workspace_bytes(*s, 6) == 0


def test_step_refusals(lib):
    for name in ("q", "k", "v", "s", "o", "s_out"):
        assert _step(**{name: None}) == pk.PDSSM_ERR_NULL, name
        assert _step(**{name: FAKE + 1}) == pk.PDSSM_ERR_ALIGN, name
    for bad in (dict(B=-1), dict(Hk=3), dict(Dk=129), dict(Dv=0)):
        assert _step(**bad) == pk.PDSSM_ERR_DIM, bad
    assert _step(flags=2) == pk.PDSSM_ERR_FLAGS
    assert _step(s=FAKE + 4) == pk.PDSSM_ERR_ALIGN and _step(g=FAKE + 2) == pk.PDSSM_ERR_ALIGN


def test_empty_linear_calls_read_nothing(lib):
    none = dict.fromkeys(("q", "k", "v", "g", "ws"))
    grads = dict.fromkeys(("d_o", "dq", "dk", "dv", "dg"))
    for empty in (dict(B=0), dict(Hv=0), dict(Hk=0, Hv=0)):
        assert _fwd(**none, o=None, **empty) == pk.PDSSM_OK
        assert _bwd(**none, **grads, **empty) == pk.PDSSM_OK
    assert _fwd(**none, o=None, L=0) == pk.PDSSM_OK
    assert _bwd(**none, **grads, L=0) == pk.PDSSM_OK
    assert _fwd(**none, o=None, L=0, s_final=FAKE, s0=FAKE) == pk.PDSSM_OK      # in place: nothing to do
    # a gradient [Hv] is written (with zeros) whenever there are heads
    for empty in (dict(B=0), dict(L=0)):
        assert _bwd(**none, **grads, flags=1 | pk.PDSSM_DG_HEADS, **empty) == pk.PDSSM_ERR_NULL
        assert _bwd(**none, **{**grads, "dg": FAKE + 2}, flags=1 | pk.PDSSM_DG_HEADS, **empty) == pk.PDSSM_ERR_ALIGN
    assert _step(q=None, s=None, B=0) == pk.PDSSM_OK


def test_workspaces_grow_with_what_they_hold(lib):
    fwd = lambda L, B=64: pk.pdssm_linear_workspace_bytes(B, 8, 16, L, 128, 128, 1)  # noqa: E731
    assert fwd(1 << 20) == 256                      # enough heads: nothing is kept
    assert fwd(4096, B=1) == fwd(1 << 20, B=1)      # a state for each segment, whatever the length
    bwd = lambda L, flags: pk.pdssm_linear_bwd_workspace_bytes(4, 16, 16, L, 128, 128, flags)  # noqa: E731
    assert bwd(4096, 1 | pk.PDSSM_NO_DG) == bwd(8192, 1 | pk.PDSSM_NO_DG)
    assert bwd(16384, 1) - bwd(8192, 1) == 2 * (bwd(8192, 1) - bwd(4096, 1)) > 0     # the states before the chunks


NORM = dict(B=2, H=3, L=10, D=64, p=0.1, rng=None, flags=1, eps=1e-5, strides=None)


def _norm(**kw):
    a = {**NORM, "x": FAKE, "residual": FAKE, "w": FAKE, "b": FAKE, "y": FAKE, "h": FAKE, **kw}
    return pk.pdssm_layer_norm_fwd(a["x"], a["residual"], a["w"], a["b"], a["y"], a["h"], a["B"], a["H"], a["L"], a["D"],
                                   a["eps"], a["p"], 1, 2, a["rng"], a["flags"], a["strides"], 0)


def _norm_bwd(**kw):
    names = ("h", "dy", "dh", "w", "dr", "dx", "dw", "db")
    a = {**NORM, **{n: FAKE for n in names}, "ws": FAKE, "ws_bytes": 1 << 40, **kw}
    return pk.pdssm_layer_norm_bwd(*(a[n] for n in names), a["B"], a["H"], a["L"], a["D"], a["eps"], a["p"], 1, 2,
                                   a["rng"], a["flags"], a["strides"], a["ws"], a["ws_bytes"], 0)


def _drop(**kw):
    a = {**NORM, "x": FAKE, "residual": FAKE, "y": FAKE, **kw}
    return pk.pdssm_dropout(a["x"], a["residual"], a["y"], a["B"], a["H"], a["L"], a["D"], a["p"], 1, 2, a["rng"],
                            a["flags"], a["strides"], 0)


def test_norm_and_dropout_refusals(lib):
    for call in (_norm, _norm_bwd, _drop):
        for bad in (dict(B=-1), dict(H=-1), dict(L=-1), dict(D=0), dict(D=16385), dict(B=1 << 20, L=1 << 20),
                    dict(B=1 << 31, L=0), dict(p=-0.1), dict(p=1.0), dict(p=float("nan"))):
            assert call(**bad) == pk.PDSSM_ERR_DIM, bad
        assert call(flags=2) == pk.PDSSM_ERR_FLAGS
        assert call(rng=FAKE + 4) == pk.PDSSM_ERR_ALIGN
    for call, names in ((_norm, ("x", "y")), (_norm_bwd, ("h", "dy", "ws")), (_drop, ("x", "y"))):
        for name in names:
            assert call(**{name: None}) == pk.PDSSM_ERR_NULL, name
            assert call(**{name: FAKE + 1}) == pk.PDSSM_ERR_ALIGN, name
    for call, names in ((_norm, ("residual", "h", "w", "b")), (_norm_bwd, ("dh", "dr", "dx", "w", "dw", "db")), (_drop, ("residual",))):
        for name in names:
            assert call(**{name: FAKE + 1}) == pk.PDSSM_ERR_ALIGN, name
    need = pk.pdssm_layer_norm_bwd_workspace_bytes(2, 3, 10, 64)
    assert need > 0 and _norm_bwd(ws_bytes=need - 1) == pk.PDSSM_ERR_WORKSPACE
    assert _norm_bwd(ws=FAKE + 4) == pk.PDSSM_ERR_ALIGN
    assert pk.pdssm_layer_norm_bwd_workspace_bytes(2, 3, 10, 0) == 0
    # the largest workspace stays at its rows of sums
    assert pk.pdssm_layer_norm_bwd_workspace_bytes(8, 128, 65536, 2048) <= 512 * 2 * 2048 * 4
    for empty in (dict(B=0), dict(H=0), dict(L=0)):
        assert _norm(x=None, y=None, **empty) == pk.PDSSM_OK
        assert _drop(x=None, y=None, **empty) == pk.PDSSM_OK
        assert _norm_bwd(h=None, dy=None, ws=None, dw=None, db=None, **empty) == pk.PDSSM_OK


def test_binding_refusals(lib):
    """What the binding checks itself, on CPU tensors (the call is never made)."""
    q, v = torch.zeros(2, 2, 5, 8), torch.zeros(2, 4, 5, 6)
    g = torch.zeros(2, 4, 5)
    for kw in (dict(k=torch.zeros(2, 2, 5, 7)), dict(v=v.bfloat16()), dict(g=g.double()), dict(g=g[:, :2]),
               dict(g=torch.zeros(3)), dict(g=torch.zeros(2, 4)), dict(q=q.double(), k=q.double(), v=v.double()),
               dict(s0=torch.zeros(2, 4, 8, 5)), dict(s0=torch.zeros(2, 4, 6, 8).transpose(2, 3)),
               dict(o=torch.zeros(2, 4, 5, 7)), dict(q=torch.zeros(2, 2, 8, 5).transpose(2, 3)), dict(v=v[0])):
        with pytest.raises(ValueError):
            pk.linear_attention(**{**dict(q=q, k=q, v=v, g=g), **kw})
    with pytest.raises(pk.PdssmError):
        pk.linear_attention(q[:, :1].expand(2, 3, 5, 8), q[:, :1].expand(2, 3, 5, 8), v, g)     # 4 heads over 3
    with pytest.raises(ValueError):
        pk.linear_attention_bwd(q, q, v, g, v[:, :2])
    with pytest.raises(ValueError, match="dg without g"):
        pk.linear_attention_bwd(q, q, v, None, v, out=(q, q, v, g, None))
    with pytest.raises(ValueError):
        pk.linear_attention_bwd(q, q, v, g, v, out=(q, q, v, torch.zeros(4), None))
    with pytest.raises(ValueError):
        pk.linear_attention_step(q[:, :, 0], q[:, :, 0], v[:, :, 0], g[:, :, 0], torch.zeros(2, 4, 6, 8))
    x, w = torch.zeros(2, 5, 8), torch.zeros(8)
    for kw in (dict(w=torch.zeros(7)), dict(b=w.double()), dict(residual=x.bfloat16()), dict(residual=x[:, :4]),
               dict(x=x.double()), dict(x=torch.zeros(())), dict(x=torch.zeros(1, 1, 1, 5, 8)), dict(w=torch.zeros(16)[::2]),
               dict(x=torch.zeros(2, 8, 5).transpose(1, 2)), dict(out=x[:1]), dict(h=x.bfloat16()),
               dict(seed=torch.zeros(2)), dict(seed=torch.zeros(3, dtype=torch.int64)),
               dict(seed=torch.zeros(2, dtype=torch.int64), offset=1)):
        with pytest.raises((ValueError, IndexError)):
            pk.layer_norm(**{**dict(x=x), **kw})
    for kw in (dict(dy=x[:1]), dict(dh=x.bfloat16()), dict(w=torch.zeros(7)), dict(out=(x, x), p=0.5), dict(out=(x[:1], None))):
        with pytest.raises(ValueError):
            pk.layer_norm_bwd(**{**dict(h=x, dy=x), **kw})
    for kw in (dict(residual=x[:1]), dict(out=x.bfloat16()), dict(seed=torch.zeros(2))):
        with pytest.raises(ValueError):
            pk.dropout(**{**dict(x=x, p=0.5, seed=1), **kw})
