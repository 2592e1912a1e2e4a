"""What dropout, the norm and rotation of heads and the losses refuse, before they
touch a device (CPU)."""
import ctypes

import pytest
import torch

from ring_allreduce_virtual_gb300 import training

A = 1 << 20  # addresses that are never used: the arguments are refused first
FAR = 1 << 34
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


DROP = dict(x=A, residual=2 * A, y=FAR, rows=4, cols=8, xStride=8, residualStride=8, yStride=8, p=0.1, seed=1,
            seedDevice=3 * A, offset=0, dtype="bfloat16")


@pytest.mark.parametrize("bad", [
    {"x": 0}, {"y": 0}, {"x": A + 1}, {"y": FAR + 1}, {"residual": 2 * A + 1}, {"seedDevice": 3 * A + 4},
    {"xStride": 7}, {"yStride": 7}, {"residualStride": 7}, {"p": -0.1}, {"p": 1.5}, {"p": NAN}, {"dtype": "int32"},
    {"dtype": "float64"}, {"dtype": "float8_e4m3"}, {"dtype": 99}, {"rows": 1 << 47}, {"xStride": 1 << 47},
    {"y": A + 16}, {"y": A, "yStride": 16}, {"y": 2 * A - 16}, {"y": 2 * A, "residualStride": 9}, {"y": 3 * A - 8},
])
def test_dropout_refuses(vr, bad):
    refused(vr, vr.vrDropout, *{**DROP, **bad}.values())


def test_dropout_of_nothing_launches_nothing(vr):
    vr.vrDropout(*{**DROP, "rows": 0, "x": 0, "y": 0}.values())
    vr.vrDropout(*{**DROP, "cols": 0, "x": 0, "y": 0}.values())


S = (1024, 128, 16)  # 2 batches of 8 tokens of up to 8 heads of 16
QK = dict(q=A, qHeads=8, qStrides=S, k=2 * A, kHeads=2, kStrides=S, qWeight=3 * A, kWeight=4 * A, qOut=FAR, qOutStrides=S,
          kOut=FAR + A, kOutStrides=S, cosTable=5 * A, sinTable=6 * A, tableRows=100, positions=7 * A,
          positionType="int64", positionStride=8, batch=2, tokens=8, dim=16, rotaryDim=16, interleaved=0, eps=1e-6,
          dtype="bfloat16", weightType="float32")


@pytest.mark.parametrize("bad", [
    {"q": 0}, {"k": 0}, {"qOut": 0}, {"kOut": 0}, {"q": A + 1}, {"kOut": FAR + A + 1}, {"qWeight": 3 * A + 2},
    {"kWeight": 4 * A + 1}, {"qStrides": None}, {"kStrides": None}, {"qOutStrides": None}, {"kOutStrides": None},
    {"qHeads": 0}, {"qHeads": 65536}, {"kHeads": 65536}, {"dim": 0}, {"dim": 1025}, {"rotaryDim": 17},
    {"rotaryDim": 18}, {"rotaryDim": 3}, {"interleaved": 2}, {"eps": -1.0}, {"eps": NAN}, {"eps": INF},
    {"dtype": "float64"}, {"weightType": "float16"}, {"dtype": "int8"}, {"cosTable": 0}, {"sinTable": 0},
    {"cosTable": 5 * A + 2}, {"positions": 0}, {"positions": 7 * A + 4}, {"positionType": "float32"},
    {"positionType": "uint64"}, {"batch": 1 << 31}, {"tokens": 1 << 31}, {"batch": 1 << 16, "tokens": 1 << 16},
    {"qStrides": (1 << 48, 128, 16)}, {"qOutStrides": (1024, 0, 16)}, {"qOutStrides": (1024, 128, 8)},
    {"qOutStrides": (512, 128, 16)}, {"kOutStrides": (1024, 16, 16)},
])
def test_qk_forward_refuses(vr, bad):
    refused(vr, vr.vrQkNormRopeForward, *{**QK, **bad}.values())


@pytest.mark.parametrize("bad", [
    {"qOut": A + 32}, {"qOut": A, "qOutStrides": (2048, 128, 16)}, {"qOut": 2 * A}, {"kOut": A}, {"kOut": 2 * A + 32},
    {"kOut": FAR}, {"qOut": 3 * A}, {"qOut": 4 * A}, {"kOut": 5 * A}, {"kOut": 6 * A}, {"qOut": 7 * A},
    {"k": A + 7 * 32, "qOut": A},  # in place over queries among whose last are k's
])
def test_qk_forward_refuses_overlaps(vr, bad):
    refused(vr, vr.vrQkNormRopeForward, *{**QK, **bad}.values())


S9 = (9 * 16 * 16, 16 * 16, 16)  # 8 of 9 tokens of up to 16 heads


@pytest.mark.parametrize("k,q_out,k_out", [
    (A + 7 * 32, A, FAR), (A + 8 * 32, A, A + 7 * 32), (A + 8 * 32, A, A + 8 * 32 + 16), (A + 512 - 30, A, FAR),
    (A + 8 * 32, A + 512, FAR), (A + 8 * 32, A, A + 9 * 512 - 30), (A + 8 * 32, A, A + 9 * 512),
])
def test_qk_forward_refuses_overlaps_among_some_tokens(vr, k, q_out, k_out):
    # in place, or shifted, in one projection that has more tokens
    strides = {name: S9 for name in ("qStrides", "kStrides", "qOutStrides", "kOutStrides")}
    refused(vr, vr.vrQkNormRopeForward, *{**QK, **strides, "k": k, "qOut": q_out, "kOut": k_out}.values())


def test_qk_forward_of_nothing_launches_nothing(vr):
    vr.vrQkNormRopeForward(*{**QK, "batch": 0, "q": 0, "k": 0, "qOut": 0, "kOut": 0}.values())
    vr.vrQkNormRopeForward(*{**QK, "tokens": 0, "q": 0, "k": 0, "qOut": 0, "kOut": 0}.values())


QKB = dict(dq=8 * A, dqStrides=S, dk=9 * A, dkStrides=S, q=A, qHeads=8, qStrides=S, k=2 * A, kHeads=2, kStrides=S,
           qWeight=3 * A, kWeight=4 * A, dqIn=FAR, dqInStrides=S, dkIn=FAR + A, dkInStrides=S, dqWeight=10 * A,
           dkWeight=11 * A, cosTable=5 * A, sinTable=6 * A, tableRows=100, positions=7 * A, positionType="int32",
           positionStride=0, batch=2, tokens=8, dim=16, rotaryDim=8, interleaved=1, eps=1e-6, dtype="float16",
           weightType="float16", workspace=64 * A, workspaceBytes=1 << 20)


@pytest.mark.parametrize("bad", [
    {"dq": 0}, {"dk": 0}, {"q": 0}, {"dqIn": 0}, {"dkIn": 0}, {"dqStrides": None}, {"dkInStrides": None},
    {"dqWeight": 10 * A + 1}, {"dkWeight": 11 * A + 1}, {"workspace": 0}, {"workspace": 64 * A + 8},
    {"workspaceBytes": 64}, {"dq": 8 * A + 1}, {"dqInStrides": (1024, 128, 15)},
    {"dqIn": A}, {"dkIn": 2 * A}, {"dqIn": 9 * A}, {"dkIn": 8 * A}, {"dqIn": 8 * A + 32}, {"dqWeight": 3 * A},
    {"dkWeight": 10 * A + 30}, {"workspace": 8 * A}, {"workspace": A}, {"dqIn": 5 * A}, {"dkIn": 64 * A},
    {"dqWeight": 8 * A}, {"dkWeight": 64 * A + 16},
])
def test_qk_backward_refuses(vr, bad):
    refused(vr, vr.vrQkNormRopeBackward, *{**QKB, **bad}.values())


def test_qk_workspace(vr):
    assert vr.vrQkNormRopeBackwardWorkspace(128) >= 1024
    refused(vr, vr.vrQkNormRopeBackwardWorkspace, 0)
    refused(vr, vr.vrQkNormRopeBackwardWorkspace, 1025)


LOGP = dict(logits=A, targets=2 * A, logp=3 * A, lse=4 * A, rest=5 * A, rows=8, cols=100, stride=100, dtype="bfloat16")
GRAD = dict(dlogp=3 * A, gain=5 * A, logits=A, targets=2 * A, lse=4 * A, rest=6 * A, dlogits=FAR, rows=8, cols=100, stride=100,
            dStride=100, dtype="float16")


@pytest.mark.parametrize("bad", [
    {"logits": 0}, {"targets": 0}, {"logp": 0}, {"logits": A + 1}, {"targets": 2 * A + 4}, {"logp": 3 * A + 2},
    {"lse": 4 * A + 2}, {"cols": 0}, {"stride": 99}, {"dtype": "float64"}, {"dtype": "int64"}, {"rows": 1 << 47},
    {"logp": A}, {"lse": A + 1596}, {"logp": 2 * A}, {"lse": 3 * A + 28},
    {"rest": 4 * A + 16}, {"lse": 0}, {"rest": 5 * A + 2},
])
def test_logprobs_forward_refuses(vr, bad):
    refused(vr, vr.vrTokenLogProbsForward, *{**LOGP, **bad}.values())


@pytest.mark.parametrize("bad", [
    {"logits": 0}, {"targets": 0}, {"dlogp": 0}, {"lse": 0}, {"dlogits": 0}, {"dlogits": FAR + 1}, {"gain": 5 * A + 2},
    {"stride": 99}, {"dStride": 99}, {"dtype": "int8"}, {"dlogits": A + 16}, {"dlogits": A, "dStride": 104},
    {"dlogits": 2 * A}, {"dlogits": 3 * A}, {"dlogits": 4 * A - 16}, {"dlogits": 5 * A - 1598},
    {"dlogits": 6 * A}, {"rest": 6 * A + 1},
])
def test_logprobs_backward_refuses(vr, bad):
    refused(vr, vr.vrTokenLogProbsBackward, *{**GRAD, **bad}.values())


def test_logprobs_of_no_rows_launch_nothing(vr):
    vr.vrTokenLogProbsForward(*{**LOGP, "rows": 0, "logits": 0}.values())
    vr.vrTokenLogProbsBackward(*{**GRAD, "rows": 0, "logits": 0, "dlogits": 0}.values())


POLICY = dict(logits=A, targets=2 * A, oldLogp=3 * A, advantages=4 * A, weights=5 * A, refLogp=6 * A, loss=7 * A,
              logp=8 * A, lse=9 * A, rest=12 * A, dlogp=10 * A, dlogits=FAR, rows=8, cols=100, stride=100, dStride=100, clipLow=0.2,
              clipHigh=0.2, klCoef=0.1, scale=1.0, dtype="bfloat16", workspace=11 * A, workspaceBytes=1 << 10)


@pytest.mark.parametrize("bad", [
    {"logits": 0}, {"targets": 0}, {"oldLogp": 0}, {"advantages": 0}, {"loss": 0}, {"logp": 0}, {"lse": 0},
    {"dlogp": 0}, {"workspace": 0}, {"workspaceBytes": 31}, {"workspace": 11 * A + 8}, {"loss": 7 * A + 2},
    {"weights": 5 * A + 1}, {"refLogp": 6 * A + 2}, {"clipLow": -0.1}, {"clipHigh": -0.1}, {"clipLow": NAN},
    {"klCoef": NAN}, {"klCoef": INF}, {"scale": NAN}, {"scale": INF}, {"cols": 0}, {"stride": 99}, {"dStride": 99},
    {"dtype": "float64"}, {"loss": 8 * A}, {"loss": A}, {"logp": 3 * A}, {"lse": 4 * A}, {"dlogp": 5 * A},
    {"dlogits": 6 * A}, {"dlogits": A + 16}, {"dlogits": A, "dStride": 101}, {"workspace": 10 * A + 16},
    {"workspace": A}, {"dlogits": 11 * A}, {"dlogp": 9 * A + 28}, {"logp": 2 * A + 60},
    {"rest": 0}, {"rest": 9 * A}, {"rest": A},
])
def test_policy_loss_refuses(vr, bad):
    refused(vr, vr.vrPolicyLoss, *{**POLICY, **bad}.values())


PREF = dict(logits=A, targets=2 * A, refLogps=3 * A, starts=4 * A, loss=5 * A, logps=6 * A, logp=7 * A, lse=8 * A,
            rest=11 * A, dlogp=9 * A, dlogits=FAR, pairs=2, rows=8, cols=100, stride=100, dStride=100, beta=0.1, labelSmoothing=0.1,
            scale=1.0, dtype="float32", workspace=10 * A, workspaceBytes=1 << 10)


@pytest.mark.parametrize("bad", [
    {"logits": 0}, {"targets": 0}, {"loss": 0}, {"logps": 0}, {"logp": 0}, {"lse": 0}, {"dlogp": 0}, {"workspace": 0},
    {"workspaceBytes": 31}, {"workspace": 10 * A + 8}, {"pairs": 0}, {"starts": 0, "rows": 6}, {"starts": 4 * A + 4},
    {"refLogps": 3 * A + 2}, {"beta": NAN}, {"beta": INF}, {"labelSmoothing": -0.1}, {"labelSmoothing": 1.1},
    {"labelSmoothing": NAN}, {"scale": INF}, {"cols": 0}, {"stride": 99}, {"dStride": 99}, {"dtype": "int32"},
    {"logps": 6 * A + 2}, {"loss": 6 * A}, {"logps": 3 * A + 12}, {"logps": 4 * A + 36}, {"logp": 2 * A + 60},
    {"dlogits": A + 16}, {"dlogits": 10 * A}, {"workspace": 9 * A + 16}, {"loss": A + 3196}, {"lse": 7 * A + 28},
    {"rest": 0}, {"rest": 8 * A + 4},
])
def test_preference_loss_refuses(vr, bad):
    refused(vr, vr.vrPreferenceLoss, *{**PREF, **bad}.values())


def test_loss_workspaces(vr):
    assert vr.vrPolicyLossWorkspace(100) >= 400 and vr.vrPolicyLossWorkspace(0) >= 0
    assert vr.vrPreferenceLossWorkspace(3) >= 48
    refused(vr, vr.vrPreferenceLossWorkspace, 0)


def test_strides_are_kept(vr):
    assert vr.strides3(4, 5, 6) is vr.strides3(4, 5, 6)
    assert list(vr.strides3(4, 5, 6)) == [4, 5, 6]
    assert isinstance(vr.strides3(1, 2, 3), ctypes.Array)


def test_torch_layer_refuses_host_tensors():
    x, t = torch.zeros(2, 8), torch.zeros(2, dtype=torch.int64)
    q = torch.zeros(2, 3, 8)
    for call in (lambda: training.dropout_forward(x, 0.1, 1), lambda: training.dropout_backward(x, 0.1, 1),
                 lambda: training.qk_norm_rope_forward(q, q), lambda: training.qk_norm_rope_backward(q, q, q, q),
                 lambda: training.token_logprobs_forward(x, t),
                 lambda: training.token_logprobs_backward(t.float(), x, t, t.float()),
                 lambda: training.policy_loss_forward(x, t, t.float(), t.float()),
                 lambda: training.preference_loss_forward(x, t, starts=torch.zeros(3, dtype=torch.int64))):
        with pytest.raises(ValueError):
            call()


def test_launches_on_the_tensors_device_and_stream(monkeypatch):
    # tensors that say they are on a second device, a library that records where it is called
    import contextlib
    import types

    class OnSecond(torch.Tensor):
        is_cuda = True
        device = torch.device("cpu")  # where the allocations of this test go

        def get_device(self):
            return 1

    state, seen = {"device": 0, "stream": None}, []

    class Library:
        def __getattr__(self, name):
            return lambda *a: (None if "Workspace" in name else seen.append((name, state["device"], a[-1]))) or 0

    @contextlib.contextmanager
    def device(index):
        was, state["device"] = state["device"], index
        yield
        state["device"] = was

    @contextlib.contextmanager
    def stream(s):
        was = dict(state)
        state.update(device=s.device_index, stream=s)
        yield
        state.update(was)

    monkeypatch.setattr(training.vr, "lib", lambda: Library())
    monkeypatch.setattr(training, "_raw_stream", lambda i: state["stream"].handle if state["stream"] else 100 + i)
    monkeypatch.setattr(training, "_current_device", lambda: state["device"])
    monkeypatch.setattr(training, "_qk_workspace", lambda dim: 1024)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "stream", stream)

    def on(t):
        return t.as_subclass(OnSecond)
    x, v, t = on(torch.zeros(4, 8)), on(torch.zeros(4)), on(torch.zeros(4, dtype=torch.int64))
    q, starts = on(torch.zeros(3, 2, 8)), on(torch.tensor([0, 2, 4]))

    def calls(**kw):
        yield "vrDropout", lambda: training.dropout_forward(x, 0.1, 1, **kw)
        yield "vrDropout", lambda: training.dropout_backward(x, 0.1, 1, **kw)
        yield "vrQkNormRopeForward", lambda: training.qk_norm_rope_forward(q, q, **kw)
        yield "vrQkNormRopeBackward", lambda: training.qk_norm_rope_backward(q, q, q, q, **kw)
        yield "vrTokenLogProbsForward", lambda: training.token_logprobs_forward(x, t, **kw)
        yield "vrTokenLogProbsBackward", lambda: training.token_logprobs_backward(v, x, t, v, **kw)
        yield "vrPolicyLoss", lambda: training.policy_loss_forward(x, t, v, v, **kw)
        yield "vrPolicyLoss", lambda: training.policy_loss_gradient(x, t, v, v, **kw)
        yield "vrPreferenceLoss", lambda: training.preference_loss_forward(x, t, starts=starts, **kw)
        yield "vrPreferenceLoss", lambda: training.preference_loss_gradient(x, t, starts=starts, **kw)
    for name, call in calls():
        call()
        assert seen[-1] == (name, 1, 101) and state["device"] == 0
    for name, call in calls(stream=types.SimpleNamespace(device_index=1, handle=77)):
        call()
        assert seen[-1] == (name, 1, 77) and state["device"] == 0
    count = len(seen)
    for _, call in calls(stream=types.SimpleNamespace(device_index=0, handle=77)):
        with pytest.raises(ValueError, match="stream"):
            call()
    assert len(seen) == count
