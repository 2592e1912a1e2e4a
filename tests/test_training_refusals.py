"""What the training-step operators refuse, before they touch a device (CPU):
every refusal is vrInvalidArgument from the library or ValueError from the
torch layer."""
import ctypes

import pytest
import torch

from ring_allreduce_virtual_gb300 import training

A = 1 << 20  # an address that is never used: the arguments are refused first
FAR = 1 << 30
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def vr():
    from ring_allreduce_virtual_gb300 import build
    build.build()
    import ring_allreduce_virtual_gb300 as m
    return m


def refused(vr, f, *args):
    with pytest.raises(vr.VrError) as e:
        f(*args)
    assert e.value.code == vr.vrInvalidArgument


FWD = dict(x=A, weight=2 * A, bias=3 * A, y=FAR, mean=4 * A, rstd=5 * A, rows=2, cols=8, xStride=8,
           yStride=8, eps=1e-5, dtype="bfloat16", weightType="float32")


@pytest.mark.parametrize("bad", [
    {"x": 0}, {"y": 0}, {"x": A + 1}, {"y": FAR + 1}, {"weight": 2 * A + 2}, {"bias": 3 * A + 1},
    {"mean": 4 * A + 2}, {"rstd": 5 * A + 2}, {"cols": 0}, {"xStride": 7}, {"yStride": 7},
    {"eps": -1e-5}, {"eps": NAN}, {"eps": INF}, {"dtype": "int32"}, {"dtype": "float64"},
    {"dtype": "float8_e4m3"}, {"weightType": "float16"}, {"weightType": "float64"},
    {"dtype": 99}, {"weightType": -1},
    {"y": A + 16}, {"y": A, "yStride": 16},  # y over x other than in place
])
def test_layer_norm_forward_refuses(vr, bad):
    refused(vr, vr.vrLayerNormForward, *{**FWD, **bad}.values())


def test_layer_norm_forward_of_no_rows_launches_nothing(vr):
    vr.vrLayerNormForward(*{**FWD, "rows": 0, "x": 0, "y": 0}.values())


BWD = dict(dy=A, x=2 * A, weight=3 * A, mean=4 * A, rstd=5 * A, dx=FAR, dweight=6 * A, dbias=7 * A,
           rows=2, cols=8, dyStride=8, xStride=8, dxStride=8, dtype="float16", weightType="float16",
           workspace=8 * A, workspaceBytes=1 << 24)


@pytest.mark.parametrize("bad", [
    {"dy": 0}, {"x": 0}, {"mean": 0}, {"rstd": 0}, {"dy": A + 1}, {"x": 2 * A + 1},
    {"dx": FAR + 1}, {"weight": 3 * A + 1}, {"mean": 4 * A + 2}, {"rstd": 5 * A + 1},
    {"dweight": 6 * A + 1}, {"dbias": 7 * A + 1}, {"cols": 0}, {"dyStride": 7}, {"xStride": 7},
    {"dxStride": 7}, {"dtype": "float64"}, {"weightType": "bfloat16"}, {"workspace": 0},
    {"workspace": 8 * A + 8}, {"workspaceBytes": 63}, {"dx": A}, {"dx": 2 * A}, {"dx": A + 32 - 2},
])
def test_layer_norm_backward_refuses(vr, bad):
    refused(vr, vr.vrLayerNormBackward, *{**BWD, **bad}.values())


def test_layer_norm_workspace(vr):
    assert vr.vrLayerNormBackwardWorkspace(2, 8, "float16") >= 64
    assert vr.vrLayerNormBackwardWorkspace(0, 8, "float32") >= 0
    refused(vr, vr.vrLayerNormBackwardWorkspace, 2, 0, "float16")
    refused(vr, vr.vrLayerNormBackwardWorkspace, 2, 8, "int8")


def norm_args(vr, ptrs=(A, 2 * A), counts=(8, 8), types=("float32", "bfloat16"), scale=1.0,
              norm=4 * A, norms=5 * A, ws=6 * A, nbytes=1 << 20):
    return vr.tensor_arrays(ptrs, counts, types), scale, norm, norms, ws, nbytes


@pytest.mark.parametrize("bad", [
    {"ptrs": (0, A)}, {"ptrs": (A + 2, A)}, {"ptrs": (A, A + 1)}, {"types": ("float32", "int32")},
    {"types": ("float32", "float8_e5m2")}, {"types": ("float32", 77)}, {"scale": INF},
    {"scale": NAN}, {"norm": 0, "norms": 0}, {"norm": A + 2}, {"norms": A + 1}, {"ws": 0},
    {"ws": 6 * A + 8}, {"nbytes": 64}, {"ptrs": (), "counts": (), "types": ()},
    {"counts": (8, 1 << 60)},
])
def test_grad_norm_refuses(vr, bad):
    refused(vr, vr.vrGradNorm, *norm_args(vr, **bad))


@pytest.mark.parametrize("outs,scale,most", [
    ((0, FAR), 1.0, 1.0), ((FAR + 2, FAR), 1.0, 1.0), ((FAR, FAR + 1), 1.0, 1.0),
    ((A + 4, FAR), 1.0, 1.0),  # over its own gradient, other than in place
    ((FAR, FAR + 64), NAN, 1.0), ((FAR, FAR + 64), 1.0, -1.0), ((FAR, FAR + 64), 1.0, NAN),
])
def test_clip_refuses(vr, outs, scale, most):
    arrays = norm_args(vr)[0]
    refused(vr, vr.vrClipGradNorm, arrays, (ctypes.c_void_p * 2)(*outs), scale, most, 4 * A, 6 * A,
            1 << 20)


def test_bindings_check_the_lengths_of_lists(vr):
    with pytest.raises(ValueError):
        vr.tensor_arrays([A], [8, 8], ["float32"])
    with pytest.raises(ValueError):
        vr.vrClipGradNorm(vr.tensor_arrays([A], [8], ["float32"]), (ctypes.c_void_p * 2)(A, A),
                          1.0, 1.0, A, A, 1 << 20)


def test_grad_norm_workspace(vr):
    assert vr.vrGradNormWorkspace(1) > 0
    assert vr.vrGradNormWorkspace(5000) > vr.vrGradNormWorkspace(1)
    refused(vr, vr.vrGradNormWorkspace, 0)


def test_torch_layer_refuses_host_tensors():
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError):
        training.layer_norm_forward(x)
    with pytest.raises(ValueError):
        training.TensorList([x])
    with pytest.raises(ValueError):
        training.TensorList([])


def test_rows_of_strided_tensors():
    t = torch.zeros(4, 6, 8)
    assert training._rows(t, "t") == (24, 8)
    assert training._rows(t[:, :, :5], "t") == (24, 8)
    assert training._rows(t[:, :1, :5], "t") == (4, 48)
    assert training._rows(t[1:3, 2], "t") == (2, 48)
    assert training._rows(t[0, 0], "t") == (1, 8)
    assert training._rows(torch.zeros(0, 8), "t") == (0, 8)
    assert training._rows(torch.zeros(3, 5)[:, :1], "t") == (3, 5)
    for bad in (t.transpose(1, 2), t[:, :3], t[:, :, ::2], torch.zeros(8).expand(4, 8),
                torch.zeros(1, 1).expand(4, 8)):
        with pytest.raises(ValueError):
            training._rows(bad, "t")
