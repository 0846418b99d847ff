"""CPU: the order of a DeltaStack's calls, recorded by stand-ins of the entry points: a sparse layer takes the settled
entry only right behind another layer's kernel, never behind the append (or rotation) of its own group of layers."""
import contextlib

import pytest
import torch

import long_context_layer_b200.stack as S

NAMES = ["rope", "kv_append_layers", "kv_append_layers_q8", "full_attn", "full_attn_q8", "window_attn", "window_attn_q8",
         "select_attn", "select_attn_q8", "sparse_attn", "sparse_attn_q8", "sparse_attn_settled", "sparse_attn_settled_q8"]


class Stream:
    cuda_stream = 0

    def __init__(self, *a):
        pass

    def wait_stream(self, other):
        pass

    wait_event = wait_stream


class Event:
    def record(self, stream):
        pass


@pytest.fixture
def calls(monkeypatch):
    log = []
    for name in NAMES:
        monkeypatch.setattr(S.N, name, lambda *a, _n=name, **kw: log.append(_n) or 0)
    monkeypatch.setattr(S.N, "workspace_init", lambda *a: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream())
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "Event", Event)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    return log


def run(kinds, cache, host, rotary=False, **kw):
    L = len(kinds)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    stack = S.DeltaStack(kinds, 4, 2, 64, torch.bfloat16, i32(0, 1), i32(0), i32(9), 1, 1, 4, window_tokens=8, cache=cache,
                         rotary=S.Rotary(64, device="cpu") if rotary else None)
    new = lambda h: torch.zeros(L, 1, h, 64, dtype=torch.bfloat16)  # noqa: E731
    if cache is None:
        pools = [[torch.zeros(1, 2, 16, 64, dtype=torch.bfloat16) for _ in kinds] for _ in "kv"]
    else:
        pools = [[S.Q8Pools(1, 2, 64, cache, device="cpu") for _ in kinds], None]
    if host:
        stack.step_host(new(4), new(2), new(2), *pools, new(4), new(4), new(2), new(2), new(4), **kw)
    else:
        stack.step(new(4), new(2), new(2), *pools, new(4), **kw)


ORDERS = [(["delta", "window", "sparse"], 2), (["full", "full", "delta", "sparse", "sparse"], 4), (["delta", "sparse", "sparse"], 2),
          (["delta", "sparse", "sparse", "window", "sparse", "sparse"], 5), (["delta", "window", "sparse", "sparse"], 3),
          (["full", "delta", "sparse", "sparse"], 9)]


@pytest.mark.parametrize("rotary", [False, True])
@pytest.mark.parametrize("cache", [None, "e4m3", "int8"])
@pytest.mark.parametrize("kinds,early", ORDERS)
def test_settled_layers_stand_behind_a_layer(calls, kinds, early, cache, rotary):
    for host in (False, True):
        calls.clear()
        run(kinds, cache, host, rotary, **(dict(early_layers=early) if host else {}))
        attention = [c for c in calls if "attn" in c]
        assert len(attention) == len(kinds)
        group = min(early, len(kinds)) if host else len(kinds)
        assert sum("append" in c for c in calls) == (1 if group == len(kinds) else 2)
        for before, c in zip(calls, calls[1:]):
            if "settled" in c:
                assert "window" in before or "sparse" in before, calls
        # elsewhere the settled entry is still taken
        for l in range(1, len(kinds)):
            if kinds[l] == "sparse":
                assert ("settled" in attention[l]) == (kinds[l - 1] in ("sparse", "window") and l != group), (l, calls)


def test_nothing_between_the_layers_keeps_the_settled_entry(calls):
    # without an append and without rotary positions the second group's first layer stands behind a layer too
    run(["delta", "sparse", "sparse", "sparse"], None, True, append=False, early_layers=2)
    assert calls == ["select_attn", "sparse_attn", "sparse_attn_settled", "sparse_attn_settled"]


@pytest.mark.parametrize("how", ["step", "step without append", "host", "host without append", "calibration"])
@pytest.mark.parametrize("bad", [dict(format="e4m3"), dict(num_phys_pages=2), dict(num_kv_heads=3), dict(head_dim=128), None])
def test_pools_of_another_format_or_shape_are_refused(calls, how, bad):
    # (a pool of fewer pages than the stack's descriptor names would be read past its end)
    kinds = ["full", "delta", "sparse"]
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    stack = S.DeltaStack(kinds, 4, 2, 64, torch.bfloat16, i32(0, 1), i32(0), i32(9), 1, 3, 4, cache="int8")
    new = lambda h: torch.zeros(3, 1, h, 64, dtype=torch.bfloat16)  # noqa: E731
    good = dict(num_phys_pages=3, num_kv_heads=2, head_dim=64, format="int8", device="cpu")
    pools = [S.Q8Pools(**good) for _ in kinds]
    pools[1] = "text" if bad is None else S.Q8Pools(**{**good, **bad})
    with pytest.raises(ValueError):
        if how == "calibration":
            stack.calibration_shifts(new(4), pools, None, new(4))
        elif how.startswith("host"):
            stack.step_host(new(4), new(2), new(2), pools, None, new(4), new(4), new(2), new(2), new(4),
                            append="without" not in how)
        else:
            stack.step(new(4), new(2), new(2), pools, None, new(4), append="without" not in how)
    assert calls == []                  # before anything is launched
