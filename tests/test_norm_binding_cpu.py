"""The norm with the residual's addition where no GPU is needed: refusals of the C entry
points and of the binding."""
import pytest
import torch

import activation_sparse_ffn_amd as sffn
from activation_sparse_ffn_amd import norm as nm

FAKE = 0x10000      # aligned addresses, never dereferenced: every call here is refused first


@pytest.fixture(scope="module")
def lib():
    return sffn.load_library()


def rows(address=FAKE, stride=64):
    return nm._Rows(address, stride)


def cfg(**kw):
    base = dict(d=64, dtype=1, out=0, eps=1e-6)
    base.update(kw)
    return nm._NormConfig(**base)


def refused(lib, status, want=sffn.SFFN_ERR_INVALID_ARG, says=""):
    assert status == want, (status, lib.sparse_ffn_last_error())
    assert says.encode() in lib.sparse_ffn_last_error(), lib.sparse_ffn_last_error()


@pytest.mark.parametrize("bad,says", [
    (dict(d=0), "d must"), (dict(d=(1 << 20) + 1), "d must"), (dict(d=-5), "d must"), (dict(dtype=2), "dtype"),
    (dict(out=3), "output"), (dict(out=-1), "output"), (dict(eps=0.0), "eps"), (dict(eps=float("nan")), "eps"),
    (dict(eps=float("inf")), "eps"), (dict(eps=-1e-6), "eps"),
])
def test_configs(lib, bad, says):
    r, c = rows(), cfg(**bad)
    refused(lib, lib.add_rms_norm(c, 4, r, None, None, r, None, None, None), says=says)
    refused(lib, lib.add_rms_norm_backward(c, 4, r, r, None, None, r, None, None, 0, None), says=says)
    assert lib.add_rms_norm_backward_workspace_size(c, 4) == 0


def test_forward_arguments(lib):
    r, o = rows(), rows(FAKE + 4096)

    def call(c=None, T=4, x=r, res=r, w=FAKE, y=o, scale=None, h=r):
        return lib.add_rms_norm(c or cfg(), T, x, res, w, y, scale, h, None)

    refused(lib, lib.add_rms_norm(None, 4, r, r, None, o, None, r, None), says="config")
    refused(lib, call(T=-1), says="T must")
    refused(lib, call(T=(1 << 30) + 1), sffn.SFFN_ERR_UNSUPPORTED, says="too large")
    refused(lib, call(x=None), says="x is null")
    refused(lib, call(x=rows(None)), says="x is null")
    refused(lib, call(x=rows(FAKE + 1)), says="x is not aligned")
    refused(lib, call(res=rows(FAKE, -1)), says="residual")
    refused(lib, call(x=rows(FAKE, 1 << 40)), says="stride")
    refused(lib, call(w=FAKE + 1), says="weight")
    refused(lib, call(y=None), says="y is null")
    refused(lib, call(y=rows(FAKE + 4096, 63)), says="y overlaps")
    refused(lib, call(h=rows(FAKE, 10)), says="h overlaps")
    refused(lib, call(res=None), says="h is the sum")
    refused(lib, call(h=o), says="the same")
    refused(lib, call(c=cfg(out=1)), says="scale is null")
    refused(lib, call(c=cfg(out=2), scale=FAKE + 2), says="scale")
    refused(lib, call(c=cfg(dtype=0), x=rows(FAKE + 2)), says="x is not aligned")
    assert lib.add_rms_norm(cfg(), 0, None, None, None, None, None, None, None) == sffn.SFFN_OK


def test_backward_arguments(lib):
    r = rows()

    def call(c=None, T=4, h=r, g=r, gh=r, w=FAKE, gx=r, gw=FAKE, ws=FAKE, n=1 << 30):
        return lib.add_rms_norm_backward(c or cfg(), T, h, g, gh, w, gx, gw, ws, n, None)

    refused(lib, call(h=None), says="h is null")
    refused(lib, call(g=None), says="g_y is null")
    refused(lib, call(gh=rows(FAKE + 1)), says="g_h")
    refused(lib, call(gx=rows(FAKE, 3)), says="g_x overlaps")
    refused(lib, call(gw=FAKE + 2), says="g_weight")
    refused(lib, call(ws=None), says="workspace is null")
    refused(lib, call(ws=FAKE + 16), says="256-byte")
    need = lib.add_rms_norm_backward_workspace_size(cfg(), 4)
    assert 0 < need <= 4 * 64 * 4
    refused(lib, call(n=need - 1), sffn.SFFN_ERR_WORKSPACE, says="needed")
    assert lib.add_rms_norm_backward(cfg(), 0, None, None, None, None, None, None, None, 0, None) == sffn.SFFN_OK
    # whatever the call, a row for each of the chip's compute units
    assert lib.add_rms_norm_backward_workspace_size(cfg(d=1 << 20), 1 << 30) <= 256 * (4 << 20)


def test_binding_refuses_what_it_cannot_pass_on():
    x = torch.zeros(3, 8)
    with pytest.raises(ValueError, match="GPU"):
        sffn.add_rms_norm(x)
    with pytest.raises(ValueError, match="GPU"):
        sffn.add_rms_norm_backward(x, x)
    with pytest.raises(TypeError):
        sffn.add_rms_norm([1.0])
    with pytest.raises(ValueError, match="shape"):
        sffn.add_rms_norm(torch.zeros(8))
    with pytest.raises(ValueError, match="float32"):
        sffn.add_rms_norm(x.half())
