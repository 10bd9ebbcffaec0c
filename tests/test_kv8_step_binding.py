"""What Megakernel.decode_step_kv8 refuses before anything reaches the library: tensors on the
host, of another type, or too small.  The library is a fake that records its calls, so no device
is needed and none of the refused addresses is ever read."""
import contextlib
import types

import pytest
import torch

import persistent_runtime_b200 as prb

BATCH, VOCAB = 3, 40


class FakeTensor:
    """A tensor of the device with the given index (-1: the host)."""

    def __init__(self, shape, dtype=torch.int32, index=0, contiguous=True):
        self.shape, self.dtype, self.index, self.contiguous = shape, dtype, index, contiguous

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for x in self.shape:
            n *= x
        return n

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return self.contiguous

    def data_ptr(self):
        return 1 << 20


@pytest.fixture
def step(monkeypatch):
    calls = []
    fake = types.SimpleNamespace(mk_decode_step_kv8_workspace=lambda *a: 0,
                                 mk_decode_step_kv8=lambda *a: calls.append(a) or 0)
    monkeypatch.setattr(prb, "lib", lambda: fake)
    cache = object.__new__(prb.KV8Cache)
    cache.device, cache._index, cache._i32, cache._ref = torch.device("cpu"), 0, torch.int32, 1 << 20
    cache._given = lambda stream: contextlib.nullcontext()
    mk = object.__new__(prb.Megakernel)
    mk._h, mk.w = None, types.SimpleNamespace(batch=BATCH, vocab=VOCAB)

    def run(**kw):
        a = dict(tokens_in=FakeTensor((BATCH,)), tokens_out=FakeTensor((BATCH,)), kv_len=FakeTensor((BATCH,)),
                 page_table=FakeTensor((BATCH, 4)), logits=None)
        a.update(kw)
        before = len(calls)
        try:
            mk.decode_step_kv8(a["tokens_in"], a["tokens_out"], a["kv_len"], cache, a["page_table"], a["logits"],
                               stream=types.SimpleNamespace(cuda_stream=0))
        finally:
            run.reached = len(calls) > before
        return run.reached
    return run


def refused(step, **kw):
    with pytest.raises(prb.MkError) as e:
        step(**kw)
    assert e.value.status == prb.MK_ERR_ARG and not step.reached, kw


@pytest.mark.parametrize("name", ["tokens_in", "tokens_out", "kv_len", "page_table"])
def test_wrong_integers_are_refused(step, name):
    shape = (BATCH, 4) if name == "page_table" else (BATCH,)
    refused(step, **{name: FakeTensor(shape, index=-1)})        # on the host
    refused(step, **{name: FakeTensor(shape, index=1)})         # on another device
    refused(step, **{name: FakeTensor(shape, torch.int64)})
    refused(step, **{name: FakeTensor(shape, contiguous=False)})
    refused(step, **{name: FakeTensor((BATCH - 1,) + shape[1:])})


def test_wrong_logits_are_refused(step):
    for bad in (dict(index=-1), dict(index=1), dict(dtype=torch.bfloat16), dict(contiguous=False),
                dict(shape=(BATCH, VOCAB - 1))):
        refused(step, logits=FakeTensor(**dict(dict(shape=(BATCH, VOCAB), dtype=torch.float32), **bad)))


def test_right_calls_reach_the_library(step):
    assert step()
    assert step(logits=FakeTensor((BATCH, VOCAB), torch.float32))
    # a row of a longer buffer of tokens, and other shapes of as many entries
    assert step(tokens_in=FakeTensor((BATCH, 1)), tokens_out=FakeTensor((2 * BATCH,)))
