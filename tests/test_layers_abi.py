"""The layer operators' C entry points and binding on the CPU: exports,
constants, and every refusal before any HIP call."""
import ctypes
import re

import pytest
import torch

import structured_sparse_state_amd as pk

FAKE = 1 << 20      # an aligned, never-dereferenced address


@pytest.fixture(scope="module")
def lib():
    return pk.library()


def test_exports_every_declared_function(lib):
    names = pk.header_functions(pk.LAYERS_HEADER)
    assert set(names) == {"pdssm_delta_fwd", "pdssm_delta_workspace_bytes", "pdssm_delta_bwd",
                          "pdssm_delta_bwd_workspace_bytes", "pdssm_delta_step", "pdssm_qk_norm_rope_fwd",
                          "pdssm_qk_norm_rope_bwd", "pdssm_qk_norm_rope_bwd_workspace_bytes"}
    for n in names:
        assert hasattr(lib, n) and hasattr(pk, n), n


def test_constants_match_binding():
    text = open(pk.LAYERS_HEADER).read()
    defs = dict(re.findall(r"#define\s+(PDSSM_[A-Z0-9_]+)\s+(0x[0-9A-Fa-f]+)u", text))
    assert len(defs) == 3
    for name, val in defs.items():
        assert getattr(pk, name) == int(val, 16), name


DELTA_SIZES = dict(B=2, Hk=2, Hv=4, L=100, Dk=64, Dv=32)
BAD_SIZES = [dict(B=-1), dict(Hk=-1), dict(Hv=-4), dict(L=-1), dict(L=(1 << 30) + 1), dict(Dk=0), dict(Dk=129),
             dict(Dv=0), dict(Dv=129), dict(Hk=0), dict(Hk=3), dict(B=1 << 40), dict(B=1 << 27, L=1 << 20)]


def _fwd(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, beta=FAKE, s0=None, o=FAKE, s_final=None, **DELTA_SIZES, scale=1.0,
             flags=1, strides=None, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    return pk.pdssm_delta_fwd(a["q"], a["k"], a["v"], a["g"], a["beta"], a["s0"], a["o"], a["s_final"], a["B"],
                              a["Hk"], a["Hv"], a["L"], a["Dk"], a["Dv"], a["scale"], a["flags"], a["strides"],
                              a["ws"], a["ws_bytes"], 0)


def _bwd(**kw):
    names = ("q", "k", "v", "g", "beta", "s0", "d_o", "ds_final", "dq", "dk", "dv", "dg", "dbeta", "ds0")
    a = dict({n: FAKE for n in names}, s0=None, ds_final=None, ds0=None, **DELTA_SIZES, flags=1, strides=None,
             ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    return pk.pdssm_delta_bwd(*(a[n] for n in names), a["B"], a["Hk"], a["Hv"], a["L"], a["Dk"], a["Dv"], 1.0,
                              a["flags"], a["strides"], a["ws"], a["ws_bytes"], 0)


def _step(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, beta=FAKE, s=FAKE, o=FAKE, s_out=FAKE, B=2, Hk=2, Hv=4, Dk=64, Dv=32,
             flags=1)
    a.update(kw)
    return pk.pdssm_delta_step(a["q"], a["k"], a["v"], a["g"], a["beta"], a["s"], a["o"], a["s_out"], a["B"], a["Hk"],
                               a["Hv"], a["Dk"], a["Dv"], 1.0, a["flags"], None, 0)


def test_delta_refusals(lib):
    for call in (_fwd, _bwd):
        for bad in BAD_SIZES:
            assert call(**bad) == pk.PDSSM_ERR_DIM, bad
        assert call(flags=2) == pk.PDSSM_ERR_FLAGS
        for name in ("q", "k", "v", "g", "beta", "ws"):
            assert call(**{name: None}) == pk.PDSSM_ERR_NULL, name
            assert call(**{name: FAKE + 1}) == pk.PDSSM_ERR_ALIGN, name
        assert call(s0=FAKE + 4) == pk.PDSSM_ERR_ALIGN
        assert call(ws=FAKE + 8) == pk.PDSSM_ERR_ALIGN
        assert call(g=FAKE + 2) == pk.PDSSM_ERR_ALIGN
    assert _fwd(o=None) == pk.PDSSM_ERR_NULL
    assert _fwd(s_final=FAKE + 4) == pk.PDSSM_ERR_ALIGN
    for name in ("d_o", "dq", "dk", "dv", "dg", "dbeta"):
        assert _bwd(**{name: None}) == pk.PDSSM_ERR_NULL, name
        assert _bwd(**{name: FAKE + 1}) == pk.PDSSM_ERR_ALIGN, name
    for name in ("ds0", "ds_final"):
        assert _bwd(**{name: FAKE + 4}) == pk.PDSSM_ERR_ALIGN, name
    s = list(DELTA_SIZES.values())
    assert _fwd(ws_bytes=pk.pdssm_delta_workspace_bytes(*s, 1) - 1) == pk.PDSSM_ERR_WORKSPACE
    assert _bwd(ws_bytes=pk.pdssm_delta_bwd_workspace_bytes(*s, 1) - 1) == pk.PDSSM_ERR_WORKSPACE
    row = (1000, 100, 10)
    for bad in ((1000, 100, -1), (1000, 100, 1 << 23)):
        assert _fwd(strides=[row] * 5 + [bad]) == pk.PDSSM_ERR_DIM
        assert _bwd(strides=[row] * 3 + [bad] + [row] * 7) == pk.PDSSM_ERR_DIM
    for bad in BAD_SIZES:
        sizes = list({**DELTA_SIZES, **bad}.values())
        assert pk.pdssm_delta_workspace_bytes(*sizes, 1) == 0 and pk.pdssm_delta_bwd_workspace_bytes(*sizes, 1) == 0
    assert pk.pdssm_delta_workspace_bytes(*s, 2) == 0


def test_step_refusals(lib):
    for name in ("q", "k", "v", "g", "beta", "s", "o", "s_out"):
        assert _step(**{name: None}) == pk.PDSSM_ERR_NULL, name
        assert _step(**{name: FAKE + 1}) == pk.PDSSM_ERR_ALIGN, name
    for bad in (dict(B=-1), dict(Hk=3), dict(Dk=129), dict(Dv=0)):
        assert _step(**bad) == pk.PDSSM_ERR_DIM, bad
    assert _step(flags=4) == pk.PDSSM_ERR_FLAGS
    assert _step(s=FAKE + 4) == pk.PDSSM_ERR_ALIGN


def test_empty_delta_calls_read_nothing(lib):
    none = dict.fromkeys(("q", "k", "v", "g", "beta", "ws"))
    for empty in (dict(B=0), dict(Hv=0), dict(Hk=0, Hv=0)):
        assert _fwd(**none, o=None, **empty) == pk.PDSSM_OK
        assert _bwd(**none, d_o=None, dq=None, dk=None, dv=None, dg=None, dbeta=None, **empty) == pk.PDSSM_OK
    assert _fwd(**none, o=None, L=0) == pk.PDSSM_OK
    assert _bwd(**none, d_o=None, L=0) == pk.PDSSM_OK
    assert _fwd(**none, o=None, L=0, s_final=FAKE, s0=FAKE) == pk.PDSSM_OK      # in place: nothing to do
    assert _step(q=None, s=None, B=0) == pk.PDSSM_OK


def test_delta_workspace_is_linear_in_length(lib):
    f = lambda L: pk.pdssm_delta_workspace_bytes(4, 8, 16, L, 128, 128, 1)  # noqa: E731
    assert f(8192) == 2 * f(4096)
    b = lambda L: pk.pdssm_delta_bwd_workspace_bytes(4, 8, 16, L, 128, 128, 1)  # noqa: E731
    assert b(8192) == 2 * b(4096)


NORM = dict(q=FAKE, k=FAKE, wq=FAKE, wk=FAKE, cos=FAKE, sin=FAKE, pos=None, B=2, Hq=4, Hk=2, L=10, D=64, R=32, P=10,
            flags=1)


def _norm(**kw):
    a = {**NORM, "q_out": FAKE, "k_out": FAKE, **kw}
    return pk.pdssm_qk_norm_rope_fwd(a["q"], a["k"], a["wq"], a["wk"], a["cos"], a["sin"], a["pos"], a["q_out"],
                                     a["k_out"], a["B"], a["Hq"], a["Hk"], a["L"], a["D"], a["R"], a["P"], 1e-6,
                                     a["flags"], None, 0)


def _norm_bwd(**kw):
    a = {**NORM, "dq_out": FAKE, "dk_out": FAKE, "dq": FAKE, "dk": FAKE, "dwq": FAKE, "dwk": FAKE, "ws": FAKE,
         "ws_bytes": 1 << 40, **kw}
    return pk.pdssm_qk_norm_rope_bwd(a["q"], a["k"], a["wq"], a["wk"], a["cos"], a["sin"], a["pos"], a["dq_out"],
                                     a["dk_out"], a["dq"], a["dk"], a["dwq"], a["dwk"], a["B"], a["Hq"], a["Hk"],
                                     a["L"], a["D"], a["R"], a["P"], 1e-6, a["flags"], None, a["ws"], a["ws_bytes"], 0)


def test_norm_refusals(lib):
    for call in (_norm, _norm_bwd):
        for bad in (dict(B=-1), dict(Hq=-1), dict(Hk=40000), dict(L=-1), dict(D=0), dict(D=257), dict(R=31),
                    dict(R=66), dict(R=-2), dict(P=0), dict(B=1 << 20, L=1 << 20)):
            assert call(**bad) == pk.PDSSM_ERR_DIM, bad
        assert call(flags=8) == pk.PDSSM_ERR_FLAGS
        for name in ("q", "k", "cos", "sin"):
            assert call(**{name: None}) == pk.PDSSM_ERR_NULL, name
        for name in ("q", "k", "cos", "sin", "wq", "wk"):
            assert call(**{name: FAKE + 1}) == pk.PDSSM_ERR_ALIGN, name
        assert call(pos=FAKE + 2) == pk.PDSSM_ERR_ALIGN
        assert call(cos=FAKE + 4) == pk.PDSSM_ERR_ALIGN
    for name in ("q_out", "k_out"):
        assert _norm(**{name: None}) == pk.PDSSM_ERR_NULL
    for name in ("dq_out", "dk_out", "dq", "dk", "ws"):
        assert _norm_bwd(**{name: None}) == pk.PDSSM_ERR_NULL, name
    need = pk.pdssm_qk_norm_rope_bwd_workspace_bytes(2, 4, 2, 10, 64)
    assert need > 0 and _norm_bwd(ws_bytes=need - 1) == pk.PDSSM_ERR_WORKSPACE
    assert _norm_bwd(ws=FAKE + 4) == pk.PDSSM_ERR_ALIGN
    # nothing to read or write
    for empty in (dict(B=0), dict(L=0), dict(Hq=0, Hk=0)):
        assert _norm(q=None, k=None, q_out=None, k_out=None, cos=None, sin=None, **empty) == pk.PDSSM_OK
    # the largest workspace a call can ask for stays a few MB
    assert pk.pdssm_qk_norm_rope_bwd_workspace_bytes(8, 128, 128, 65536, 256) < 8 << 20


def test_binding_refusals(lib):
    """What the binding checks itself, on CPU tensors (the call is never made)."""
    q, v = torch.zeros(2, 2, 5, 8), torch.zeros(2, 4, 5, 6)
    g = torch.zeros(2, 4, 5)
    for kw in (dict(k=torch.zeros(2, 2, 5, 7)), dict(v=v.bfloat16()), dict(g=g.double()), dict(beta=g[:, :2]),
               dict(q=q.double(), k=q.double(), v=v.double()), dict(s0=torch.zeros(2, 4, 8, 5)),
               dict(s0=torch.zeros(2, 4, 6, 8).transpose(2, 3)), dict(o=torch.zeros(2, 4, 5, 7)),
               dict(q=torch.zeros(2, 2, 8, 5).transpose(2, 3)), dict(v=v[0])):
        with pytest.raises(ValueError):
            pk.delta_rule(**{**dict(q=q, k=q, v=v, g=g, beta=g), **kw})
    with pytest.raises(pk.PdssmError):
        pk.delta_rule(q[:, :1].expand(2, 3, 5, 8), q[:, :1].expand(2, 3, 5, 8), v, g, g)     # 4 heads over 3
    with pytest.raises(ValueError):
        pk.delta_rule_bwd(q, q, v, g, g, v[:, :2])
    with pytest.raises(ValueError):
        pk.delta_step(q[:, :, 0], q[:, :, 0], v[:, :, 0], g[:, :, 0], g[:, :, 0], torch.zeros(2, 4, 6, 8))
    x = torch.zeros(2, 3, 5, 8)
    table = torch.zeros(5, 2)
    for kw in (dict(wq=torch.zeros(7)), dict(cos=table), dict(cos=table, sin=torch.zeros(5, 3)), dict(k=x[..., :6]),
               dict(pos=torch.zeros(2, 5, dtype=torch.int64)), dict(out=(x, x[:, :2])), dict(wq=torch.zeros(16)[::2])):
        with pytest.raises(ValueError):
            pk.qk_norm_rope(**{**dict(q=x, k=x), **kw})
    with pytest.raises(KeyError):
        pk.qk_norm_rope(x, x, kind="max")


def test_stride_struct_layout():
    assert ctypes.sizeof(pk._Strides) == 24
