"""Refusals of the adapter calls that fill the rows their list leaves out, without a GPU:
those of the plain calls, and a list that is missing or shorter than the output."""
import pytest

import mixture_experts_layer_06_amd as moe
from test_abi_block import LORA_SHAPES, P, misaligned, nulls

SHAPES = LORA_SHAPES + [(dict(T=17), moe.ERR_BAD_SHAPE), (dict(T=17, M=0), moe.ERR_BAD_SHAPE)]


def filled(x=P, base=P, dt=moe.BF16, T=16, a=P, b=P, sc=P, off=P, rows=P, e=4, M=16, H=64, N=64, R=16, out=P, u=P, ws=P,
           n=1 << 30):
    return moe.lib().moe_lora_filled(x, base, dt, T, a, b, sc, off, rows, e, M, H, N, R, out, u, ws, n, None)


@pytest.mark.parametrize("kw,status", SHAPES + nulls("x", "a", "b", "off", "rows", "out", "ws")
                         + misaligned("x", "base", "a", "b", "sc", "off", "rows", "out", "u", "ws")
                         + [(dict(n=moe.lora_workspace_size(moe.BF16, 4, 16, 64, 64, 16) - 1),
                             moe.ERR_WORKSPACE_TOO_SMALL)])
def test_forward(kw, status):
    assert filled(**kw) == status


def bwd_filled(d=P, x=P, u=P, dt=moe.BF16, T=16, a=P, b=P, sc=P, off=P, rows=P, e=4, M=16, H=64, N=64, R=16, base=P,
               dx=P, da=P, db=P, dwdt=moe.BF16, ws=P, n=1 << 30):
    return moe.lib().moe_lora_bwd_filled(d, x, u, dt, T, a, b, sc, off, rows, e, M, H, N, R, base, dx, da, db, dwdt, ws,
                                         n, None)


@pytest.mark.parametrize("kw,status", SHAPES + nulls("d", "x", "u", "a", "b", "off", "rows", "ws")
                         + misaligned("d", "x", "u", "a", "b", "sc", "off", "rows", "base", "dx", "da", "db", "ws")
                         + [(dict(dx=None, da=None, db=None), moe.ERR_NULL_POINTER),
                            (dict(dt=moe.F32, dwdt=moe.BF16), moe.ERR_BAD_DTYPE),
                            (dict(n=moe.lora_bwd_workspace_size(moe.BF16, 4, 16, 64, 64, 16) - 1),
                             moe.ERR_WORKSPACE_TOO_SMALL)])
def test_backward(kw, status):
    assert bwd_filled(**kw) == status


def test_no_rows_is_noop():
    assert filled(T=0, M=0, x=None, a=None, b=None, off=None, rows=None, out=None, u=None, ws=None, n=0) == moe.OK
