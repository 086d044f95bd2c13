"""The serving operators' C ABI without a GPU: every declared symbol is exported, and bad arguments are
refused before any CUDA call (the addresses are never dereferenced)."""
import ctypes
import os
import re

import pytest

from gdn_chunkwise_ut_gb300 import _lib, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.lib()


def header():
    return open(os.path.join(ROOT, "include", "gdn_layer.h")).read()


def test_exports_every_declared_symbol(lib):
    names = set(re.findall(r"\bint (\w+)\s*\(", re.sub(r"/\*.*?\*/", "", header(), flags=re.S)))
    assert names == {"gdn_recurrent_fwd", "gdn_prep_fwd", "add_rms_norm_fwd", "gated_rms_norm_fwd", "gdn_state_copy"}
    for n in names:
        assert hasattr(lib, n) and n in _lib.SIGNATURES
    args = re.findall(r"int (\w+)\s*\((.*?)\);", re.sub(r"/\*.*?\*/", "", header(), flags=re.S), flags=re.S)
    for name, text in args:
        assert len(text.split(",")) == len(_lib.SIGNATURES[name][1]), name


def test_constants_match_the_header():
    text = header()
    for n in ("GDN_OUT_BF16", "GDN_OUT_F32", "GDN_OUT_E4M3"):
        assert int(re.search(rf"{n} = (\d+)", text).group(1)) == getattr(_lib, n)
    assert int(re.search(r"#define GDN_COPY_MAX_TENSORS (\d+)", text).group(1)) == _lib.GDN_COPY_MAX_TENSORS


def test_status_string(lib):
    assert lib.kkt_status_string(_lib.KKT_ERR_INDEX).decode() == "slot index out of range"


def test_recurrent_argument_errors(lib):
    def call(**kw):
        a = dict(q=0x1000, k=0x2000, v=0x3000, beta=0x4000, g=None, cu=None, N=2, T=1, Hk=2, Hv=4, dk=128, dv=128, io=0,
                 state=0x5000, st=1, P=8, slots=0x6000, out=None, o=0x7000)
        a.update(kw)
        return lib.gdn_recurrent_fwd(a["q"], a["k"], a["v"], a["beta"], a["g"], a["cu"], a["N"], a["T"], a["Hk"],
                                     a["Hv"], a["dk"], a["dv"], 1.0, a["io"], a["state"], a["st"], a["P"], a["slots"],
                                     a["out"], a["o"], None)
    for bad in (dict(q=None), dict(beta=None), dict(o=None), dict(state=None), dict(N=0), dict(T=-1), dict(Hk=0),
                dict(Hv=0), dict(Hk=3), dict(Hv=70000, Hk=1), dict(io=2), dict(st=7), dict(P=-1),
                dict(slots=None, N=9), dict(T=1 << 30, N=4)):
        assert call(**bad) == _lib.KKT_ERR_ARG, bad
    for bad in (dict(dk=96), dict(dv=256)):
        assert call(**bad) == _lib.KKT_ERR_UNSUPPORTED
    for bad in (dict(q=0x1008), dict(state=0x5008), dict(o=0x7004), dict(beta=0x4002), dict(g=0x8001),
                dict(slots=0x6002), dict(out=0x6002), dict(cu=0x9001)):
        assert call(**bad) == _lib.KKT_ERR_ALIGN, bad
    assert call(T=0, q=None, k=None, v=None, beta=None, o=None) == _lib.KKT_OK


def test_prep_argument_errors(lib):
    def call(**kw):
        a = dict(x=0x1000, w=0x2000, bias=None, a=0x3000, b=0x4000, A=0x5000, dt=0x6000, cu=None, N=2, T=1, Hk=2, Hv=4,
                 dk=128, dv=128, taps=4, expand=0, io=0, state=0x7000, P=8, slots=0x8000, q=0x9000, k=0xa000, v=0xb000,
                 g=0xc000, beta=0xd000, xs=1024, as_=4, bs=4)
        a.update(kw)
        return lib.gdn_prep_fwd(a["x"], a["xs"], a["w"], a["bias"], a["a"], a["as_"], a["b"], a["bs"], a["A"],
                                a["dt"], a["cu"], a["N"], a["T"], a["Hk"], a["Hv"], a["dk"], a["dv"], a["taps"], 1e-6, a["expand"], a["io"], a["state"],
                                a["P"], a["slots"], a["q"], a["k"], a["v"], a["g"], a["beta"], None)
    for bad in (dict(x=None), dict(w=None), dict(a=None), dict(A=None), dict(dt=None), dict(q=None), dict(beta=None),
                dict(state=None), dict(N=0), dict(T=-1), dict(Hk=3), dict(io=5), dict(slots=None, N=9), dict(P=-2),
                dict(xs=1016), dict(xs=0), dict(xs=1 << 40), dict(as_=3), dict(bs=-4), dict(bs=1 << 40)):
        assert call(**bad) == _lib.KKT_ERR_ARG, bad
    for bad in (dict(dk=96, dv=96), dict(dv=64), dict(taps=1), dict(taps=5)):
        assert call(**bad) == _lib.KKT_ERR_UNSUPPORTED, bad
    for bad in (dict(x=0x1008), dict(state=0x7004), dict(q=0x9008), dict(w=0x2001), dict(a=0x3001), dict(g=0xc002),
                dict(slots=0x8002), dict(xs=1028)):
        assert call(**bad) == _lib.KKT_ERR_ALIGN, bad
    assert call(T=0, x=None, a=None, b=None, q=None, k=None, v=None, g=None, beta=None) == _lib.KKT_OK


def test_norm_argument_errors(lib):
    def add(**kw):
        a = dict(x=0x1000, r=None, w=0x2000, rows=2, dim=256, io=0, out=0, group=128, y=0x3000, s=None, ro=None)
        a.update(kw)
        return lib.add_rms_norm_fwd(a["x"], a["r"], a["w"], a["rows"], a["dim"], 1e-6, a["io"], a["out"], a["group"],
                                    a["y"], a["s"], a["ro"], None)
    for bad in (dict(x=None), dict(w=None), dict(y=None), dict(dim=0), dict(rows=1 << 31), dict(rows=1 << 63),
                dict(io=2), dict(out=3), dict(out=2)):
        assert add(**bad) == _lib.KKT_ERR_ARG, bad
    assert add(dim=16385) == _lib.KKT_ERR_UNSUPPORTED and add(group=64) == _lib.KKT_ERR_UNSUPPORTED
    for bad in (dict(x=0x1002), dict(r=0x4008), dict(ro=0x4008), dict(out=2, s=0x5002)):
        assert add(**bad) == _lib.KKT_ERR_ALIGN, bad
    assert add(rows=0, x=None, y=None) == _lib.KKT_OK

    def gated(**kw):
        a = dict(x=0x1000, z=0x2000, w=0x3000, rows=2, dim=128, io=0, out=0, y=0x4000, s=None, zr=0, zs=0)
        a.update(kw)
        return lib.gated_rms_norm_fwd(a["x"], a["z"], a["zr"], a["zs"], a["w"], a["rows"], a["dim"], 1e-6,
                                      a["io"], a["out"], a["y"], a["s"], None)
    for bad in (dict(x=None), dict(z=None), dict(w=None), dict(y=None), dict(io=2), dict(out=-1), dict(out=2),
                dict(rows=1 << 62), dict(zr=-1, zs=128), dict(zr=2, zs=255), dict(zr=2, zs=1 << 40), dict(zr=3, zs=512)):
        assert gated(**bad) == _lib.KKT_ERR_ARG, bad
    assert gated(dim=96) == _lib.KKT_ERR_UNSUPPORTED
    assert gated(zr=2, zs=260) == _lib.KKT_ERR_ALIGN
    assert gated(z=0x2004) == _lib.KKT_ERR_ALIGN and gated(out=2, s=0x5001) == _lib.KKT_ERR_ALIGN
    assert gated(rows=0, x=None, z=None, y=None) == _lib.KKT_OK


def test_copy_argument_errors(lib):
    def arr(t, *v):
        return (t * len(v))(*v)

    def call(**kw):
        a = dict(dst=(0x1000, 0x2000), src=(0x3000, 0x4000), size=(64, 48), ds=(64, 48), ss=(128, 48), n=2,
                 dslots=0x5000, sslots=0x6000, m=3, dP=4, sP=4)
        a.update(kw)
        ptrs = [None if v is None else arr(t, *v) for v, t in ((a["dst"], ctypes.c_void_p), (a["src"], ctypes.c_void_p),
                (a["size"], ctypes.c_size_t), (a["ds"], ctypes.c_size_t), (a["ss"], ctypes.c_size_t))]
        return lib.gdn_state_copy(*[None if p is None else ctypes.addressof(p) for p in ptrs], a["n"], a["dslots"],
                                  a["sslots"], a["m"], a["dP"], a["sP"], None)
    for bad in (dict(n=0), dict(n=65), dict(m=-1), dict(dP=-1), dict(dst=None), dict(size=None), dict(ds=None),
                dict(ss=None), dict(dslots=None), dict(sslots=None), dict(dst=(0x1000, None)), dict(src=(None, 0x4000)),
                dict(size=(0, 48)), dict(ds=(32, 48)), dict(ss=(64, 32))):
        assert call(**bad) == _lib.KKT_ERR_ARG, bad
    assert call(dslots=0x5002) == _lib.KKT_ERR_ALIGN and call(sslots=0x6001) == _lib.KKT_ERR_ALIGN
    assert call(m=0) == _lib.KKT_OK


def test_binding_refuses_host_tensors(lib):
    """The native binding's checks, without a GPU: ValueError, nothing launched."""
    import torch

    from gdn_chunkwise_ut_gb300 import (add_rms_norm_fwd, gated_rms_norm_fwd, gdn_prep_fwd, gdn_recurrent_fwd,
                                        gdn_state_copy)
    x = torch.zeros((1, 1, 2, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        gdn_recurrent_fwd(x, x, x, torch.zeros((1, 1, 2)), torch.zeros((1, 2, 128, 128)))
    with pytest.raises(ValueError, match="expected"):
        gdn_recurrent_fwd(x[0], x, x, torch.zeros((1, 1, 2)), torch.zeros((1, 2, 128, 128)))
    with pytest.raises(ValueError, match="channels"):
        gdn_prep_fwd(x[0], x[0, 0], x[0], x[0], x[0, 0, 0], x[0, 0, 0], x[0], Hk=1, Hv=1, dk=64, dv=64)
    with pytest.raises(ValueError, match="integer"):
        gdn_prep_fwd(x[0], x[0, 0], x[0], x[0], x[0, 0, 0], x[0, 0, 0], x[0], Hk=1.5, Hv=1, dk=64, dv=64)
    with pytest.raises(ValueError, match="CUDA"):
        add_rms_norm_fwd(x, x[0, 0, 0])
    with pytest.raises(ValueError, match="CUDA"):
        gated_rms_norm_fwd(x, None, x[0, 0, 0])
    with pytest.raises(ValueError, match="CUDA"):
        gdn_state_copy([x], torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="list of tensors"):
        gdn_state_copy(3, torch.zeros(1, dtype=torch.int32))


def test_missing_binding_fails_loudly(lib, monkeypatch, tmp_path):
    import torch

    from gdn_chunkwise_ut_gb300 import add_rms_norm_fwd
    monkeypatch.setattr(_lib, "LIB_PATH", tmp_path / "libkkt.so")
    monkeypatch.setattr(_lib, "_binding", None)
    with pytest.raises(RuntimeError, match="binding is not built"):
        add_rms_norm_fwd(torch.zeros((1, 8)), torch.zeros(8))
