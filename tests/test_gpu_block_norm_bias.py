"""Gradients of layer norms that have a bias and no weight, and of wide rows."""
import pytest
import torch

import mixture_experts_layer_06_amd as moe
from test_gpu_block_norm import Case

pytestmark = pytest.mark.gpu


def bare(T, N, dt, res, gate, seed, post=True, pre=True):
    """Layer norms whose weights are left out: ones to the formulas."""
    c = Case(T, N, dt, res, "layer", gate, post, pre, "f32", seed)
    c.w["w_post"] = c.w["w_pre"] = None
    return c


@pytest.mark.parametrize("T,N,dt,res,gate", [(5, 70, "f32", "f32", "none"), (300, 1501, "bf16", "f32", "channel"),
                                             (129, 512, "bf16", "bf16", "token"), (40, 4096, "bf16", "f32", "none")])
def test_biases_without_weights(T, N, dt, res, gate):
    c = bare(T, N, dt, res, gate, T + N)
    c.check_forward()
    dh, dro, z, r, b_post, g, b_pre = c.dev("dh", "dro", "z", "r", "b_post", "gate", "b_pre")
    one = torch.ones(N, device="cuda")
    want = moe.block_norm_bwd(dh, dro, z, r, one, b_post, g, one, **c.how)
    got = moe.block_norm_bwd(dh, dro, z, r, None, b_post, g, None, b_pre=b_pre, **c.how)
    assert set(got) == {k for k in want if not k.startswith("dw_")}
    for k, v in got.items():
        assert torch.equal(v, want[k]), k
    # each bias alone
    got = moe.block_norm_bwd(dh, dro, z, r, None, None, None, None, b_pre=b_pre, **c.how)
    assert set(got) == {"dr", "dz", "db_pre"} and torch.equal(got["db_pre"], want["db_pre"])
    got = moe.block_norm_bwd(dh, dro, z, r, None, b_post, g, None, **c.how)
    assert set(got) == {"dr", "dz", "db_post"} | ({"dgate"} if g is not None else set())
    assert torch.equal(got["db_post"], want["db_post"])
    # left out with the others
    assert set(moe.block_norm_bwd(dh, dro, z, r, None, b_post, g, None, b_pre=b_pre, need_dw=False, **c.how)) == {"dr", "dz"}


def test_bias_of_a_norm_alone():
    c = bare(45, 333, "f32", "f32", "none", 3, post=False)
    r, dh, b = c.dev("r", "dh", "b_pre")
    one = torch.ones(333, device="cuda")
    want = moe.block_norm_bwd(dh, None, None, r, w_pre=one, kind=moe.NORM_LAYER)
    got = moe.block_norm_bwd(dh, None, None, r, b_pre=b, kind=moe.NORM_LAYER)
    assert set(got) == {"dr", "db_pre"}
    assert torch.equal(got["db_pre"], want["db_pre"]) and torch.equal(got["dr"], want["dr"])
    assert got["db_pre"].dtype == torch.float32


def test_no_rows_and_refusals():
    z = torch.empty((0, 64), device="cuda")
    w = torch.ones(64, device="cuda")
    got = moe.block_norm_bwd(z, z, z, z, None, w, post=True, b_pre=w, kind=moe.NORM_LAYER)
    assert got["db_post"].tolist() == got["db_pre"].tolist() == [0.0] * 64
    z = torch.zeros((4, 64), device="cuda")
    with pytest.raises(ValueError):
        moe.block_norm_bwd(z, z, z, z, w, b_pre=w[:32], kind=moe.NORM_LAYER)
    with pytest.raises(ValueError):
        moe.block_norm_bwd(z, z, z, z, w, b_pre=w.bfloat16(), kind=moe.NORM_LAYER)
    with pytest.raises(moe.MoeError):
        moe.block_norm_bwd(z, z, z, z, w, w_pre=w, b_pre=w)  # an RMS norm has no bias
    with pytest.raises(moe.MoeError):
        moe.block_norm_bwd(None, z, z, None, w, b_pre=w, kind=moe.NORM_LAYER)  # no norm after r_out


@pytest.mark.parametrize("T,N,dt,res,kind", [(30, 16384, "f32", "f32", "layer"), (520, 9001, "f32", "f32", "layer"),
                                             (300, 12000, "bf16", "bf16", "layer"), (270, 8200, "f32", "f32", "rms"),
                                             (9, 16383, "bf16", "f32", "layer"), (1030, 8191, "f32", "f32", "layer")])
def test_wide_rows(T, N, dt, res, kind):
    """Rows of 8192 to 16384 values, and just below, in every type and kind."""
    Case(T, N, dt, res, kind, "channel", True, True, "f32", N).check_backward()
