"""What the serving loop's device timings enclose, with a fake device: events and calls in their order."""
import pytest

from bit_kv_cache_int2_gb300 import oscar

torch = pytest.importorskip("torch")


class FakeEvent:
    """Elapsed time: the calls between two events."""

    log = []

    def __init__(self, enable_timing):
        assert enable_timing

    def record(self):
        self.at = sum(x != "event" for x in FakeEvent.log)
        FakeEvent.log.append("event")

    def elapsed_time(self, other):
        return 1e3 * (other.at - self.at)


@pytest.fixture
def log(monkeypatch):
    FakeEvent.log = []
    monkeypatch.setattr(torch.cuda, "Event", FakeEvent)
    for name, x in (("oscar_rope", "turn"), ("oscar_prefill_kv8", "attend"), ("oscar_append_kv8", "append"),
                    ("oscar_import_tokens", "import"), ("oscar_import_bf16_history", "import")):
        monkeypatch.setattr(oscar, name, lambda *a, _x=x, **k: FakeEvent.log.append(_x))
    monkeypatch.setattr(oscar, "alloc_scratch", lambda *a, **k: torch.zeros(1))
    monkeypatch.setattr(oscar, "alloc_scratch_kv8", lambda *a, **k: torch.zeros(1))
    for name in ("bind_step_kv8", "bind_step_any_batch"):
        monkeypatch.setattr(oscar, name, lambda *a, **k: lambda k, v, q, n: FakeEvent.log.append("step"))
    return FakeEvent.log


def backend(fmt, timed, draw, **kw):
    from bit_kv_cache_int2_gb300 import serving

    cfg = oscar.make_config(1, 4, 2, max_batch=2, max_pages_per_req=4, num_pages=8)
    cache = dict(page_table=torch.zeros(2, 4, dtype=torch.int32), seq_lens=torch.zeros(2, dtype=torch.int32),
                 hist_lens=torch.zeros(2, dtype=torch.int32), **{x: torch.zeros(2, 1) for x in ("sink_k", "sink_v", "ring_k", "ring_v")})
    return serving.DeviceBackend(fmt, None, cfg, cache, draw, time_steps=timed, **kw)


def rows(req):
    return torch.zeros(req.prefix + req.gen, 8, 128).bfloat16()


@pytest.mark.parametrize("timed", [True, False])
def test_projections_are_timed_with_their_positions_and_without_callbacks(log, timed):
    from bit_kv_cache_int2_gb300 import serving

    be = backend("int8", timed, rows, rope=dict(table=None), prompt_chunk=8, on_prompt=lambda *a: log.append("seen"),
                 on_step=lambda *a: log.append("stepped"))
    req = serving.Request(rid=0, prefix=13, gen=3, pages=[1])
    be.admit(0, req)
    be.step([req])
    ev = ["event"] if timed else []
    chunk = ev + ["turn", "attend"] + ev + ["seen"] + ev + ["append"] + ev
    assert log == 2 * chunk + ev + ["turn", "step"] + ev + ["stepped"]
    if timed:
        assert serving.import_seconds(be) == 2 * 3 and serving.step_seconds(be) == 2


@pytest.mark.parametrize("fmt,call", [("int8", "append"), ("int2", "import"), ("bf16", "import")])
def test_prefixes_and_steps_are_timed_as_before(log, fmt, call):
    from bit_kv_cache_int2_gb300 import serving

    def draw(req):
        K = torch.zeros(2, req.prefix + req.gen, 128).bfloat16()
        return K, K, torch.zeros(req.gen, 4, 128).bfloat16()

    be = backend(fmt, True, draw)
    req = serving.Request(rid=0, prefix=13, gen=3, pages=[1])
    be.admit(0, req)
    be.step([req])
    assert log == ["event", call, "event", "event", "step", "event"]
    assert serving.import_seconds(be) == 1 and serving.step_seconds(be) == 1
    be.admit(1, serving.Request(rid=1, prefix=0, gen=3, pages=[2]))  # no prefix: nothing to time
    assert len(be.import_events) == 1
