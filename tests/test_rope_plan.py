"""How exact a rotary plan's frequencies are, against 60-digit decimals, and the frequencies that it refuses because nothing
of them would be exact. No GPU needed."""
import decimal

import pytest

import gemm_q4_q8_gb300 as qg
from gemm_q4_q8_gb300 import build as qbuild

D = decimal.Decimal
PI = D("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    qbuild.build()


def turns(rot, base, i):
    """Turns a position of pair i, of the base that a C double holds."""
    with decimal.localcontext() as c:
        c.prec = 60
        return (D(base).ln() * D(-2 * i) / D(rot)).exp() / (2 * PI)


@pytest.mark.parametrize("rot,base", [(64, 1e4), (128, 5e5), (128, 1e6), (64, 1e7), (256, 1e6), (20, 500.25), (8, 1e-4),
                                      (16, 1.0), (128, 1e-7)])
def test_frequencies(rot, base):
    """The documented bound: theta_i 2^-51 rad a position, so turns 2^-51 turns a position, and the fixed point's 2^-64."""
    plan = qg.qrope_plan(rot, base=base)
    for i in range(rot // 2):
        want = turns(rot, base, i)
        with decimal.localcontext() as c:
            c.prec = 60
            off = abs(D(int(plan.step[i])) / 2 ** 64 - want % 1)
            off = min(off, 1 - off)  # just below a whole turn, and just above
            assert off <= want * D(2) ** -51 + D(2) ** -64, (i, float(off))


@pytest.mark.parametrize("kw", [dict(base=1e-30), dict(base=1e-300), dict(factor=1e-9), dict(base=1e-10, rot_dim=128, interleaved=True),
                                dict(base=1e-6, factor=1e-5, orig_ctx=1, low_turns=1e12, high_turns=2e12)])
def test_frequencies_of_whole_turns_only_are_refused(kw):
    """From 2^26 turns a position on, the fraction would be known to fewer bits than the f32 angle that comes of it; far above,
    to none."""
    with pytest.raises(qg.QGError) as e:
        qg.qrope_plan(kw.pop("rot_dim", 64), **kw)
    assert e.value.status == qg.QG_ERR_SHAPE


def test_largest_frequencies_that_are_taken():
    """Next to the border on both sides: pair 1 of 4 dimensions turns by base^(-1/2) a position."""
    near = float(2 ** 26 * 2 * PI) ** -2
    qg.qrope_plan(4, base=near * 1.001)
    with pytest.raises(qg.QGError):
        qg.qrope_plan(4, base=near * 0.999)
