"""The 8-bit cache's measured passes follow the stream they are run on, and
states of equal shape do not share working memory."""
import os
import sys

import pytest
import torch

from bit_kv_cache_int2_gb300 import build as B

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(__file__), "..", "perf"))

CASES = [{"op": "append", "T": 3, "track": True}, {"op": "decode", "track": True}, {"op": "evict", "budget": 300}]


@pytest.fixture(scope="module")
def ops():
    B.build()
    import operators

    operators.own = True
    yield operators
    operators.own = False


def case(**kw):
    return {"type": "int8", "B": 2, "Hkv": 2, "G": 4, "lo": 900, "hi": 2000, **kw}


def snapshot(x):
    return {k: v.clone() for k, v in x.items() if v is not None}


@pytest.mark.parametrize("kw", CASES)
def test_a_pass_is_captured_on_the_stream_it_is_run_on(ops, kw):
    c = case(**kw)
    want = snapshot(ops.run(ops.prepare(c, 1)))
    s = ops.prepare(c, 1)
    before = snapshot(s["cache"])
    ops.run(ops.prepare(c, 2))  # another state of the same shape, on the default stream
    torch.cuda.synchronize()
    g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=st):
        got = ops.run(s)
    torch.cuda.synchronize()
    for k in before:  # capturing ran nothing
        assert torch.equal(s["cache"][k].view(torch.uint8), before[k].view(torch.uint8)), k
    g.replay()
    torch.cuda.synchronize()
    for k in want:
        assert torch.equal(got[k].contiguous().view(torch.uint8), want[k].contiguous().view(torch.uint8)), k


def test_two_states_on_two_streams(ops):
    c = case(op="decode", track=True, B=8, lo=9000, hi=30000)
    want = [snapshot(ops.run(ops.prepare(c, i))) for i in (1, 2)]
    states = [ops.prepare(c, i) for i in (1, 2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for s, st in zip(states, streams):
        with torch.cuda.stream(st):
            got.append(ops.run(s))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for k in b:
            assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)), k
