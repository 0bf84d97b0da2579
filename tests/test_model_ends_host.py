"""Refusals of the embedding's, dropout's and cross entropy's entry points (no GPU: the pointers are fake, nothing is launched)."""
import ctypes
import math

import pytest
import torch

import fully_sharded_gb300 as fs

A, B, C, D, E, F, G, H = (0x10000000 * (i + 1) for i in range(8))  # far apart
lib = fs._lib
I32, I64 = fs.FSDP_DTYPE_I32, fs.FSDP_DTYPE_I64
BAD_SCALES = [math.nan, math.inf, 1e60]


def embedding(pointers=None, **over):
    a = dict(rows=4, cols=100, vocab=30, table_stride=100, addend_stride=100, out_stride=100, dtype=1, token_dtype=I64, scale=1.0)
    a.update(over)
    p = dict(tokens=A, table=B, addend=None, out=C)
    p.update(pointers or {})
    return lib.fsdp_embedding(ctypes.byref(fs.EmbeddingArgs(**a)), p["tokens"], p["table"], p["addend"], p["out"], None)


def test_embedding_refuses():
    for over in (dict(rows=-1), dict(cols=0), dict(vocab=0), dict(rows=(1 << 30) + 1), dict(cols=(1 << 30) + 1),
                 dict(vocab=(1 << 30) + 1), dict(table_stride=99), dict(out_stride=0), dict(dtype=2), dict(dtype=I32),
                 dict(token_dtype=1), dict(token_dtype=0), *(dict(scale=s) for s in BAD_SCALES)):
        assert embedding(**over) == fs.FSDP_EINVAL, over
    for p in (dict(tokens=None), dict(table=None), dict(out=None), dict(tokens=A + 4), dict(table=B + 1), dict(out=C + 1),
              dict(addend=D + 1)):
        assert embedding(p) == fs.FSDP_EINVAL, p
    assert embedding(dict(addend=D), addend_stride=50) == fs.FSDP_EINVAL
    for p in (dict(out=B + 200), dict(out=A), dict(addend=D, out=D + 2), dict(addend=C + 100)):
        assert embedding(p) == fs.FSDP_EALIAS, p
    assert embedding(dict(tokens=None, table=None, out=None), rows=0) == fs.FSDP_OK
    assert lib.fsdp_embedding(None, A, B, None, C, None) == fs.FSDP_EINVAL


def embedding_backward(pointers=None, ws_bytes=1 << 30, **over):
    a = dict(rows=4, cols=100, vocab=30, dout_stride=100, dtable_stride=100, dtype=1, table_dtype=1, token_dtype=I64,
             accumulate=1, scale=1.0)
    a.update(over)
    p = dict(tokens=A, dout=B, dtable=C, ws=D)
    p.update(pointers or {})
    return lib.fsdp_embedding_backward(ctypes.byref(fs.EmbeddingBackwardArgs(**a)), p["tokens"], p["dout"], p["dtable"],
                                       p["ws"], ws_bytes, None)


def test_embedding_backward_refuses():
    for over in (dict(rows=-1), dict(cols=0), dict(vocab=0), dict(rows=(1 << 30) + 1), dict(cols=(1 << 30) + 1),
                 dict(vocab=(1 << 30) + 1), dict(dout_stride=99), dict(dtable_stride=0), dict(dtype=2), dict(table_dtype=I64),
                 dict(token_dtype=1), *(dict(scale=s) for s in BAD_SCALES)):
        assert embedding_backward(**over) == fs.FSDP_EINVAL, over
    for p in (dict(tokens=None), dict(dout=None), dict(dtable=None), dict(ws=None), dict(tokens=A + 4), dict(dtable=C + 1)):
        assert embedding_backward(p) == fs.FSDP_EINVAL, p
    assert embedding_backward(ws_bytes=fs.fsdp_embedding_backward_workspace(4, 100, 30) - 1) == fs.FSDP_EWORKSPACE
    for p in (dict(dtable=B + 10), dict(dtable=A), dict(ws=A), dict(ws=B), dict(ws=C + 100)):
        assert embedding_backward(p) == fs.FSDP_EALIAS, p
    for sizes in ((-1, 1, 1), (1, 0, 1), (1, 1, 0)):
        with pytest.raises(fs.FsdpError):
            fs.fsdp_embedding_backward_workspace(*sizes)


def dropout(pointers=None, **over):
    a = dict(rows=4, cols=100, x_stride=100, residual_stride=100, out_stride=100, seed=1, offset=2, dtype=1, p=0.5)
    a.update(over)
    p = dict(x=A, residual=None, counter=None, out=B)
    p.update(pointers or {})
    return lib.fsdp_dropout(ctypes.byref(fs.DropoutArgs(**a)), p["x"], p["residual"], p["counter"], p["out"], None)


def test_dropout_refuses():
    for over in (dict(rows=-1), dict(cols=0), dict(rows=(1 << 40) + 1), dict(rows=1 << 30, cols=1 << 31, x_stride=1 << 31),
                 dict(x_stride=99), dict(out_stride=3), dict(dtype=2), dict(dtype=I64), dict(p=-0.1), dict(p=1.0),
                 dict(p=math.nan), dict(p=1 - 2.0 ** -18), dict(p=math.inf)):
        assert dropout(**over) == fs.FSDP_EINVAL, over
    for p in (dict(x=None), dict(out=None), dict(x=A + 1), dict(out=B + 1), dict(residual=C + 1), dict(counter=D + 4)):
        assert dropout(p) == fs.FSDP_EINVAL, p
    for p in (dict(out=A + 2), dict(residual=C, out=C + 2), dict(counter=B + 8)):
        assert dropout(p) == fs.FSDP_EALIAS, p
    assert dropout(dict(x=None, out=None), rows=0) == fs.FSDP_OK


def cross_entropy(pointers=None, ws_bytes=1 << 40, **over):
    a = dict(rows=40, cols=100, vocab=300, hidden_stride=100, weight_stride=100, dhidden_stride=100, dweight_stride=100,
             piece=0, target_dtype=I64, scale=1.0)
    a.update(over)
    p = dict(hidden=A, weight=B, targets=C, dloss=None, loss=D, lse=None, dhidden=E, dweight=F, ws=G)
    p.update(pointers or {})
    return lib.fsdp_cross_entropy(ctypes.byref(fs.CrossEntropyArgs(**a)), p["hidden"], p["weight"], p["targets"], p["dloss"],
                                  p["loss"], p["lse"], p["dhidden"], p["dweight"], p["ws"], ws_bytes, None)


def test_cross_entropy_refuses():
    for over in (dict(rows=-1), dict(cols=0), dict(vocab=0), dict(rows=(1 << 40) + 1), dict(cols=(1 << 24) + 1),
                 dict(vocab=(1 << 30) + 1), dict(piece=-1), dict(hidden_stride=99), dict(weight_stride=9),
                 dict(dhidden_stride=0), dict(dweight_stride=99), dict(target_dtype=1), dict(target_dtype=0),
                 *(dict(scale=s) for s in BAD_SCALES)):
        assert cross_entropy(**over) == fs.FSDP_EINVAL, over
    for p in (dict(hidden=None), dict(weight=None), dict(targets=None), dict(loss=None), dict(ws=None), dict(dhidden=None),
              dict(dweight=None), dict(hidden=A + 1), dict(weight=B + 1), dict(targets=C + 4), dict(loss=D + 2),
              dict(lse=H + 2), dict(dloss=H + 2), dict(dhidden=E + 1), dict(dweight=F + 1),
              dict(dhidden=None, dweight=None, dloss=H)):
        assert cross_entropy(p) == fs.FSDP_EINVAL, p
    need = fs.fsdp_cross_entropy_workspace(40, 100, 300)
    assert cross_entropy(ws_bytes=need - 1) == fs.FSDP_EWORKSPACE
    for p in (dict(dhidden=A + 2), dict(dweight=B), dict(dhidden=B), dict(loss=A), dict(loss=C), dict(lse=D + 4), dict(dloss=D),
              dict(ws=A), dict(ws=B), dict(ws=F + 200), dict(dweight=E + 100)):
        assert cross_entropy(p) == fs.FSDP_EALIAS, p
    for sizes in ((-1, 1, 1), (1, 0, 1), (1, 1, 0), (1, 1, 1, True, -1)):
        with pytest.raises(fs.FsdpError):
            fs.fsdp_cross_entropy_workspace(*sizes)


def test_workspace_is_bounded_by_the_piece():
    """The logits of many rows are never held: beyond one piece the workspace does not grow."""
    base = fs.fsdp_cross_entropy_workspace(40000, 768, 50257)
    assert fs.fsdp_cross_entropy_workspace(4000000, 768, 50257) == base
    assert base < 2 << 30
    assert fs.fsdp_cross_entropy_workspace(40000, 768, 50257, piece=1024) < base / 2
    assert fs.fsdp_cross_entropy_workspace(8192, 768, 50257, gradients=False) < 160 << 20


# ----------------------------------------------------------------- the binding

BF16, F32 = torch.bfloat16, torch.float32


class On:
    """A CPU tensor that says it lies on a CUDA device."""

    is_cuda = True

    def __init__(self, index, *shape, dtype=BF16, of=None):
        self._t, self._index = torch.zeros(*shape, dtype=dtype) if of is None else of, index

    def get_device(self):
        return self._index

    @property
    def device(self):
        return torch.device("cuda", self._index)

    def __getattr__(self, name):
        return getattr(self._t, name)


NAMES = ("fsdp_embedding", "fsdp_embedding_backward", "fsdp_dropout", "fsdp_cross_entropy")


@pytest.fixture
def first_device(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)

    def reached(*args):
        raise AssertionError("the library was reached")

    for name in NAMES:
        monkeypatch.setattr(fs._lib, name, reached)


def tensors(call, **other):
    """The call's tensors, each on device 0 but those given."""
    def on(name, *shape, dtype=BF16):
        return other.get(name) or On(0, *shape, dtype=dtype)

    if call == "embedding":
        fs.fsdp_embedding(on("tokens", 4, dtype=torch.int64), on("table", 9, 8), on("out", 4, 8), addend=on("addend", 4, 8), stream=0)
    elif call == "embedding_backward":
        fs.fsdp_embedding_backward(on("tokens", 4, dtype=torch.int32), on("dout", 4, 8), on("dtable", 9, 8, dtype=F32),
                                   on("workspace", 1 << 16, dtype=torch.uint8), stream=0)
    elif call == "dropout":
        fs.fsdp_dropout(on("x", 4, 8), on("out", 4, 8), 0.5, other.get("seed", 1), other.get("offset", 0), residual=on("residual", 4, 8),
                        counter=on("counter", 1, dtype=torch.int64), stream=0)
    else:
        fs.fsdp_cross_entropy(on("hidden", 4, 8), on("weight", 9, 8), on("targets", 4, dtype=torch.int64), on("loss", 4, dtype=F32),
                              on("workspace", 1 << 20, dtype=torch.uint8), lse=on("lse", 4, dtype=F32), dhidden=on("dhidden", 4, 8),
                              dweight=on("dweight", 9, 8), dloss=on("dloss", 4, dtype=F32), stream=0)


SHAPES = {"embedding": dict(tokens=((4,), torch.int64), table=((9, 8), BF16), out=((4, 8), BF16), addend=((4, 8), BF16)),
          "embedding_backward": dict(tokens=((4,), torch.int32), dout=((4, 8), BF16), dtable=((9, 8), F32),
                                     workspace=((1 << 16,), torch.uint8)),
          "dropout": dict(x=((4, 8), BF16), out=((4, 8), BF16), residual=((4, 8), BF16), counter=((1,), torch.int64)),
          "cross_entropy": dict(hidden=((4, 8), BF16), weight=((9, 8), BF16), targets=((4,), torch.int64), loss=((4,), F32),
                                workspace=((1 << 20,), torch.uint8), lse=((4,), F32), dhidden=((4, 8), BF16),
                                dweight=((9, 8), BF16), dloss=((4,), F32))}


@pytest.mark.parametrize("call,name", [(c, n) for c, names in SHAPES.items() for n in names])
def test_the_binding_refuses(first_device, call, name):
    shape, dtype = SHAPES[call][name]
    with pytest.raises(AssertionError, match="reached"):
        tensors(call)
    with pytest.raises(ValueError, match="cuda:1"):
        tensors(call, **{name: On(1, *shape, dtype=dtype)})
    if name == "workspace":
        return
    with pytest.raises(ValueError):
        tensors(call, **{name: On(0, *shape, dtype=torch.float16)})
    with pytest.raises(ValueError):
        tensors(call, **{name: On(0, *(s + 1 for s in shape), dtype=dtype)})
    apart = torch.zeros(*shape[:-1], 2 * max(shape[-1], 2), dtype=dtype)[..., ::2][..., :max(shape[-1], 2)]
    with pytest.raises(ValueError):
        tensors(call, **{name: On(0, of=apart)})


def test_the_binding_refuses_all_on_another_device(first_device):
    for call, shapes in SHAPES.items():
        with pytest.raises(ValueError, match="cuda:1"):
            tensors(call, **{n: On(1, *s, dtype=d) for n, (s, d) in shapes.items()})


@pytest.mark.parametrize("bad", [-1, 1 << 64])
@pytest.mark.parametrize("name", ["seed", "offset"])
def test_seeds_are_64_bits(first_device, bad, name):
    with pytest.raises(ValueError, match="64-bit"):
        tensors("dropout", **{name: bad})


def test_one_gradient_without_the_other(first_device):
    with pytest.raises(ValueError, match="both or neither"):
        fs.fsdp_cross_entropy(On(0, 4, 8), On(0, 9, 8), On(0, 4, dtype=torch.int64), On(0, 4, dtype=F32), None, dweight=On(0, 9, 8))
