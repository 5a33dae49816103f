"""Outputs of the norm that lie where its inputs do: taken where every row is written over
itself, refused where a row would be written over another one that is still to be read.
Without a GPU: refused calls enqueue nothing, and T = 1 stands for no other row."""
import pytest

import activation_sparse_ffn_amd as sffn
from tests.test_norm_binding_cpu import FAKE, cfg, refused, rows

A, B = FAKE, FAKE + (1 << 20)


@pytest.fixture(scope="module")
def lib():
    return sffn.load_library()


def forward(lib, x, r, y, h, out=0, T=4):
    return lib.add_rms_norm(cfg(out=out), T, x, r, FAKE, y, None if out == 0 else FAKE + 64, h, None)


@pytest.mark.parametrize("out", [1, 2])
def test_eight_bits_are_not_written_over_the_inputs(lib, out):
    """Their rows are shorter: with the same stride row 1 lies in what was row 0."""
    for T in (1, 4):
        refused(lib, forward(lib, rows(A), rows(B), rows(A), None, out, T), says="y lies where x does")
        refused(lib, forward(lib, rows(A), rows(B), rows(B), None, out, T), says="y lies where residual does")
        refused(lib, forward(lib, rows(A, 64), rows(B), rows(A, 128), None, out, T), says="y lies where x does")


def test_outputs_in_place_have_the_inputs_stride(lib):
    for stride in (0, 65, 128):
        refused(lib, forward(lib, rows(A, stride), rows(B), rows(A), None), says="y lies where x does")
        refused(lib, forward(lib, rows(A), rows(B, stride), rows(B), None), says="y lies where residual does")
        refused(lib, forward(lib, rows(A, stride), rows(B), rows(B), rows(A)), says="h lies where x does")
        refused(lib, forward(lib, rows(A), rows(B, stride), rows(A), rows(B)), says="h lies where residual does")
        refused(lib, forward(lib, rows(A, stride), rows(B), rows(B + 4096), rows(A), out=1), says="h lies where x does")


def test_gradients_in_place_have_the_inputs_stride(lib):
    a, b, c = rows(A), rows(B), rows(B + (1 << 16))

    def call(h=a, g=b, gh=c, gx=a):
        return lib.add_rms_norm_backward(cfg(), 4, h, g, gh, FAKE, gx, None, None, 0, None)

    for stride in (0, 65, 128):
        refused(lib, call(h=rows(A, stride), gx=rows(A)), says="g_x lies where h does")
        refused(lib, call(g=rows(B, stride), gx=rows(B)), says="g_x lies where g_y does")
        refused(lib, call(gh=rows(B + (1 << 16), stride), gx=c), says="g_x lies where g_h does")
