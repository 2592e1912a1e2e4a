"""What the training-step operators refuse, before they touch a device (CPU):
every refusal is vrInvalidArgument from the library or ValueError from the
torch layer."""
import ctypes
import random

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


@pytest.mark.parametrize("bad", [
    {"y": 2 * A}, {"y": 3 * A + 16}, {"y": 4 * A}, {"y": 5 * A - 16},  # y over the parameters or the statistics
    {"mean": A}, {"mean": 2 * A + 28}, {"rstd": 3 * A}, {"rstd": FAR + 28}, {"mean": 5 * A + 4},
    {"y": A + 6, "cols": 4},  # side by side, but a byte too near
    {"y": A + 6, "xStride": 16, "yStride": 16}, {"y": A + 18, "xStride": 16, "yStride": 16},
    {"y": A + 16, "xStride": 16, "yStride": 24},  # strides that differ may not interleave
    {"mean": A + 12, "xStride": 16}, {"mean": A + 28, "xStride": 16},
])
def test_layer_norm_forward_refuses_overlaps(vr, bad):
    refused(vr, vr.vrLayerNormForward, *{**FWD, **bad}.values())


@pytest.mark.parametrize("bad", [
    {"dx": 3 * A}, {"dx": 4 * A}, {"dx": 5 * A}, {"dx": 6 * A}, {"dx": 7 * A + 14}, {"dx": 8 * A + 32},
    {"dweight": 7 * A}, {"dbias": 6 * A + 14}, {"dweight": A}, {"dbias": 2 * A}, {"dweight": 3 * A},
    {"dbias": 3 * A + 14}, {"dweight": 4 * A}, {"dbias": 5 * A + 4}, {"workspace": A}, {"workspace": 3 * A},
    {"workspace": 6 * A}, {"workspace": 7 * A}, {"workspace": 4 * A}, {"workspace": 5 * A},
    {"workspace": FAR}, {"workspace": 2 * A - 16},
])
def test_layer_norm_backward_refuses_overlaps(vr, bad):
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


@pytest.mark.parametrize("bad", [{"norm": A}, {"norm": 2 * A + 12}, {"norms": A + 28}, {"norms": 4 * A - 4},
                                 {"ws": A}, {"ws": 4 * A}, {"ws": 5 * A - 16}, {"ws": A - 4096}])
def test_grad_norm_refuses_overlaps(vr, bad):
    refused(vr, vr.vrGradNorm, *norm_args(vr, **bad))


B = 4096  # bytes of a tensor of these lists, and their distance
LISTS = {
    "the same tensor twice": ([A, A + B, A], None),
    "parts of each other": ([A, A + B, A + B + 64], None),
    "swapped": ([A, A + B, A + 2 * B], [A + B, A, FAR]),
    "shifted by one tensor": ([A, A + B, A + 2 * B], [A + B, A + 2 * B, A + 3 * B]),
    "shifted by less": ([A, A + B, A + 2 * B], [A + 64, A + B + 64, A + 2 * B + 64]),
    "one output twice": ([A, A + B, A + 2 * B], [FAR, FAR + B, FAR]),
    "outputs over each other": ([A, A + B, A + 2 * B], [FAR, FAR + B - 64, FAR + 4 * B]),
    "one in place, over another's": ([A, A + B, A + B + 128], [FAR, A + B, FAR + B]),
}


def clip_args(vr, ins, outs, types, n=B // 4, **kw):
    k = {"norm": FAR - A, "ws": FAR + A, "nbytes": 1 << 20, **kw}
    arrays = vr.tensor_arrays(ins, [n if t == "float32" else 2 * n for t in types], types)
    return arrays, (ctypes.c_void_p * len(ins))(*(outs or ins)), 1.0, 1.0, k["norm"], k["ws"], k["nbytes"]


@pytest.mark.parametrize("types", [["float32"] * 3, ["float32", "bfloat16", "float16"]], ids=["one", "mixed"])
@pytest.mark.parametrize("name", LISTS)
def test_clip_refuses_overlaps(vr, name, types):
    refused(vr, vr.vrClipGradNorm, *clip_args(vr, *LISTS[name], types))


@pytest.mark.parametrize("bad", [{"norm": A + B}, {"ws": A + 2 * B - 16}, {"norm": FAR + A}, {"ws": FAR}])
def test_clip_refuses_norms_and_workspaces_over_tensors(vr, bad):
    refused(vr, vr.vrClipGradNorm, *clip_args(vr, [A, A + B], [FAR, FAR + B], ["float32"] * 2, **bad))


@pytest.mark.parametrize("seed", range(20))
def test_clip_finds_one_overlap_in_a_long_list(vr, seed):
    rng = random.Random(seed)
    n = rng.choice([5, 100, 3000])
    places = [A + 2 * i * B for i in range(2 * n)]
    rng.shuffle(places)
    ins, outs = places[:n], places[n:]
    i, j = rng.sample(range(n), 2)
    bad = rng.choice([ins, outs])[j] + rng.choice([0, 16, B - 16, 16 - B])
    refused(vr, vr.vrClipGradNorm, *clip_args(vr, ins, [*outs[:i], bad, *outs[i + 1:]], ["float32"] * n, nbytes=1 << 22))


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
