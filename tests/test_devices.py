"""Operands of one call lie on one GPU, the current one: the library launches, allocates and takes its
stream there.  Host logic, shown without a GPU: stand-ins for tensors, which only say where they lie."""
import pytest
import torch

import submanifold_sparse_convolution_gb300 as sc

BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


class On:
    """What the argument checks read of a dense tensor on a GPU."""
    is_cuda = True

    def __init__(self, gpu, shape, dtype=BF):
        self.gpu, self.shape, self.dtype = gpu, torch.Size(shape), dtype
        self.device = torch.device("cuda", gpu)

    def get_device(self):
        return self.gpu

    def dim(self):
        return len(self.shape)

    def stride(self):
        return tuple(self.shape[1:]) + (1,)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20


@pytest.fixture(autouse=True)
def no_calls(monkeypatch):
    def refuse(*_a, **_k):
        raise AssertionError("the call went past the checks")
    monkeypatch.setattr(sc, "_lib", refuse)
    monkeypatch.setattr(sc, "library", refuse)
    monkeypatch.setattr(torch, "empty", refuse)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(sc, "_current_device", lambda: 0, raising=False)


N, C, H = 6, 32, 48
# entry, operands (name: shape, type), options
ROWS = [
    (sc.rms_norm, dict(x=((N, C), BF), weight=((C,), F32), residual=((N, C), BF), sum_out=((N, C), BF))),
    (sc.rms_norm_backward, dict(dy=((N, C), BF), x=((N, C), BF), weight=((C,), F32), dres=((N, C), BF))),
    (sc.linear, dict(x=((N, C), BF), weight=((C, H), BF), bias=((H,), F32), residual=((N, H), BF), out=((N, H), BF))),
    (sc.linear, dict(x=((N, C), E4M3), weight=((H, C), E4M3), x_scale=((N,), F32), w_scale=((H,), F32))),
    (sc.linear_backward, dict(dy=((N, H), BF), x=((N, C), BF), weight=((C, H), BF), bias=((H,), F32))),
    (sc.gated_ffn, dict(x=((N, C), BF), w_gate=((C, H), BF), w_up=((C, H), BF), out=((N, H), BF))),
    (sc.gated_ffn, dict(x=((N, C), E4M3), w_gate=((H, C), E4M3), w_up=((H, C), E4M3), x_scale=((N,), F32),
                        gate_scale=((H,), F32), up_scale=((H,), F32))),
    (sc.gated_ffn_backward, dict(dh=((N, H), BF), x=((N, C), BF), w_gate=((C, H), BF), w_up=((C, H), BF))),
    (sc.quantize_weight, dict(weight=((C, H), BF))),
]


def make(operands, there=()):
    return {k: On(1 if k in there else 0, *v) for k, v in operands.items()}


@pytest.mark.parametrize("entry,operands", ROWS)
def test_row_operators_refuse_another_gpu(entry, operands):
    with pytest.raises(AssertionError, match="past the checks"):   # the stand-ins themselves are taken
        entry(**make(operands))
    with pytest.raises(ValueError, match="current"):               # all on a GPU that is not the current one
        entry(**make(operands, operands))
    for name in operands:                                          # one of them on another
        with pytest.raises(ValueError):
            entry(**make(operands, [name]))


# ---- the convolution's entries ---------------------------------------------------
class Stream:
    cuda_stream = 0

    def __init__(self, gpu):
        self.device = torch.device("cuda", gpu)


def conv_map(gpu):
    return sc.Map(None, N, On(gpu, (N, 4), torch.int32))


def pack(gpu):
    return sc.WPack(None, C, H, BF, On(gpu, (27, C, H)))


def square(gpu):
    return sc.WPack(None, C, C, BF, On(gpu, (27, C, C)))


FEATS, OUT, WEIGHTS = ((N, C), BF), ((N, H), BF), ((27, C, H), BF)
CONV = [
    ("build_map", dict(coords=((N, 4), torch.int32)), {}),
    ("build_map_strided", dict(coords=((N, 4), torch.int32)), {}),
    ("wpack_create", dict(weights=WEIGHTS), {}),
    ("subm_forward", dict(feats=FEATS, weights=WEIGHTS, out=OUT, scale=((H,), F32), bias=((H,), F32), residual=OUT),
     dict(m=conv_map)),
    ("subm_forward_packed", dict(feats=FEATS, out=OUT, scale=((H,), F32), bias=((H,), F32), residual=OUT),
     dict(m=conv_map, wp=pack)),
    ("subm_forward_layers", dict(feats=FEATS), dict(m=conv_map, wps=lambda gpu: [square(gpu)])),
    ("map_export", {}, dict(m=conv_map)),
    ("map_out_coords", {}, dict(m=conv_map)),
]


@pytest.mark.parametrize("name,tensors,handles", CONV)
def test_convolution_entries_refuse_another_gpu(monkeypatch, name, tensors, handles):
    class Lib:   # stands for the library; no function of it may be called
        def __getattr__(self, fn):
            raise AssertionError("the call went past the checks")
    monkeypatch.setattr(sc, "library", Lib)
    entry = getattr(sc, name)

    def call(there=(), stream=0):
        kw = {k: h(1 if k in there else 0) for k, h in handles.items()}
        return entry(**kw, **make(tensors, there), stream=Stream(stream))
    for there in [[k] for k in (*tensors, *handles)]:
        with pytest.raises(ValueError, match="current"):
            call(there)
    with pytest.raises(ValueError, match="current"):
        call(stream=1)
