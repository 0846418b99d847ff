"""GPU: one workspace serves calls of several shapes, cache kinds and scoring modes in turn."""
import pytest
import torch

from tests.operator_helpers import DT, PAGE, Paged, Pool8, desc, flags, lib, stream, workspace

pytestmark = pytest.mark.gpu


class Shape:
    """One shape with a bf16 or fp32 cache and an 8-bit one, and every attention call over them."""

    def __init__(self, hq, hkv, d, dtype, lens, room=None, seed=0):
        L = lib()
        self.L, self.batch = L, len(lens)
        self.paged = Paged(lens, seed=seed, room=room)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(DT[dtype])  # noqa: E731
        self.k, self.v = (rand(self.paged.pages, hkv, PAGE, d) for _ in "kv")
        self.pool = Pool8(self.paged.pages, hkv, d, "int8").fill(gen)
        self.q = rand(self.batch, hq, d)
        self.desc, self.pt = desc(hq, hkv, d, dtype, self.paged.pages), self.paged.table()
        self.sel = {r: L.DeltaSelectParams(6, 16, 64, r) for r in (L.DELTA_HEAD_SUM, L.DELTA_HEAD_MAX)}

    def size(self):
        L, a = self.L, (self.desc, self.batch, self.paged.longest)
        return max(f(*a, r) for f in (L.workspace_size_reduce, L.workspace_size_q8) for r in self.sel)

    def calls(self):
        L = self.L
        return [(kind, r) for kind in ("plain", "q8") for r in ("full", "window", *self.sel)]

    def run(self, kind, what, ws, nb):
        L, o = self.L, torch.empty_like(self.q)
        a = (self.desc, self.pt)
        store = (self.k, self.v) if kind == "plain" else (self.pool.cache,)
        end = (o, ws, nb, stream())
        if what == "full":
            (L.full_attn if kind == "plain" else L.full_attn_q8)(*a, self.q, *store, *end)
            return [o]
        if what == "window":
            (L.window_attn if kind == "plain" else L.window_attn_q8)(*a, 100, 20, self.q, *store, *end)
            return [o]
        sp = self.sel[what]
        stride = L.sel_capacity(sp)
        cnt = torch.full((self.batch,), -1, dtype=torch.int32, device="cuda")
        pages = torch.full((self.batch, stride), -1, dtype=torch.int32, device="cuda")
        scores = torch.zeros(self.batch, self.paged.longest, device="cuda")
        fn = L.select_attn if kind == "plain" else L.select_attn_q8
        fn(*a, sp, self.q, *store, o, cnt, pages, stride, scores, ws, nb, stream())
        return [o, cnt, pages, scores]


def test_shapes_in_turn_give_what_each_gives_alone():
    shapes = [Shape(32, 8, 128, "bf16", [9000, 700], seed=1), Shape(7, 1, 64, "bf16", [100 * i for i in range(40)], seed=2),
              Shape(4, 4, 64, "f32", [3000], seed=3), Shape(40, 8, 128, "bf16", [500] * 5, room=20000, seed=4),
              Shape(8, 1, 128, "bf16", [20000, 3], seed=5)]
    nb = max(s.size() for s in shapes)
    todo = [(i, *c) for i, s in enumerate(shapes) for c in s.calls()]
    alone = {}
    for i, kind, what in todo:
        ws = workspace(nb)
        alone[i, kind, what] = shapes[i].run(kind, what, ws, nb)
        assert flags(ws) == 0
    shared = workspace(nb)
    gen = torch.Generator().manual_seed(0)
    for _ in range(6):
        for x in torch.randperm(len(todo), generator=gen).tolist():
            i, kind, what = todo[x]
            for got, want in zip(shapes[i].run(kind, what, shared, nb), alone[todo[x]]):
                assert torch.equal(got, want), todo[x]
    assert flags(shared) == 0
