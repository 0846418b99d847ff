"""CPU: the operators' entry points refuse bad arguments before anything is launched."""
import math

import pytest

FAKE = 1 << 40   # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import long_context_layer_b200 as lib
    return lib


def desc(L, **kw):
    d = dict(num_q_heads=28, num_kv_heads=4, head_dim=128, page_size=16, dtype=L.DELTA_BF16, sm_scale=0.0,
             num_phys_pages=512)
    d.update(kw)
    return L.DeltaDesc(**d)


def pt(L, batch=1, maxp=512):
    return L.DeltaPageTable(FAKE, FAKE, FAKE, batch, maxp)


def cache(L, **kw):
    c = dict(k_pool=FAKE, v_pool=FAKE, k_scale=FAKE, v_scale=FAKE, format=L.DELTA_E4M3)
    c.update(kw)
    return L.DeltaQ8Cache(**c)


BAD_CACHES = [dict(k_pool=None), dict(v_pool=None), dict(k_scale=None), dict(v_scale=None), dict(k_pool=FAKE + 8),
              dict(v_pool=FAKE + 1), dict(k_scale=FAKE + 2), dict(format=2), dict(format=-1)]


def calls_on(L, d, p, c):
    ws = 1 << 30
    sp = L.DeltaSelectParams(8, 16, 64, L.DELTA_HEAD_SUM)
    return [
        L.kv_append_q8(d, p, FAKE, FAKE, c, check=False),
        L.kv_append_layers_q8(d, p, [FAKE], [FAKE], [c], check=False),
        L.kv_write_q8(d, p, FAKE, 5, FAKE, FAKE, c, check=False),
        L.kv_read_q8(d, p, FAKE, 5, None, c, FAKE, FAKE, check=False),
        L.full_attn_q8(d, p, FAKE, c, FAKE, FAKE, ws, check=False),
        L.select_attn_q8(d, p, sp, FAKE, c, FAKE, FAKE, FAKE, 64, None, FAKE, ws, check=False),
        L.sparse_attn_q8(d, p, FAKE, FAKE, 4, FAKE, c, FAKE, FAKE, ws, check=False),
        L.sparse_attn_settled_q8(d, p, FAKE, FAKE, 4, FAKE, c, FAKE, FAKE, ws, check=False),
        L.window_attn_q8(d, p, 16, 4, FAKE, c, FAKE, FAKE, ws, check=False),
    ]


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_bad_cache_refused_everywhere(L, bad):
    assert set(calls_on(L, desc(L), pt(L), cache(L, **bad))) == {1}


@pytest.mark.parametrize("bad,status", [(dict(head_dim=96), 2), (dict(num_q_heads=27), 1), (dict(page_size=8), 2),
                                        (dict(dtype=5), 1), (dict(num_q_heads=36), 2), (dict(sm_scale=-1.0), 1)])
def test_bad_descriptor_refused_everywhere(L, bad, status):
    d = desc(L, **bad)
    assert set(calls_on(L, d, pt(L), cache(L))) == {status}
    assert L.window_attn(d, pt(L), 16, 4, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 30, check=False) == status
    plan = L.DeltaRope(FAKE, 64, 0, 1.0, FAKE, 1, 0)
    assert L.rope(d, plan, 1, FAKE, FAKE, FAKE, FAKE, check=False) == status


def test_empty_batch_is_a_no_op(L):
    d, p, c = desc(L), L.DeltaPageTable(None, None, None, 0, 0), cache(L)
    assert set(calls_on(L, d, p, c)) == {0}
    assert L.window_attn(d, p, 16, 4, None, None, None, None, None, 0, check=False) == 0


def test_window_arguments(L):
    d, p, ws = desc(L), pt(L), 1 << 30
    assert L.window_attn(d, p, -1, 4, FAKE, FAKE, FAKE, FAKE, FAKE, ws, check=False) == 1
    assert L.window_attn(d, p, 16, -1, FAKE, FAKE, FAKE, FAKE, FAKE, ws, check=False) == 1
    assert L.window_attn(d, p, 16, 4, None, FAKE, FAKE, FAKE, FAKE, ws, check=False) == 1
    assert L.window_attn(d, p, 16, 4, FAKE, None, FAKE, FAKE, FAKE, ws, check=False) == 1
    assert L.window_attn(d, p, 16, 4, FAKE, FAKE, FAKE + 4, FAKE, FAKE, ws, check=False) == 1
    assert L.window_attn(d, p, 16, 4, FAKE, FAKE, FAKE, FAKE, FAKE + 8, ws, check=False) == 3
    assert L.window_attn(d, p, 16, 4, FAKE, FAKE, FAKE, FAKE, FAKE, L.workspace_size(d, 1, 512) - 1, check=False) == 3
    assert L.window_attn_q8(d, p, -1, 4, FAKE, cache(L), FAKE, FAKE, ws, check=False) == 1
    assert L.window_attn_q8(d, p, 16, -1, FAKE, cache(L), FAKE, FAKE, ws, check=False) == 1


def test_q8_attention_arguments(L):
    d, p, c = desc(L), pt(L), cache(L)
    need = L.workspace_size_q8(d, 1, 512)
    assert need > 0 and L.workspace_size_q8(d, 1, 512, 7) == 0 and L.workspace_size_q8(desc(L, head_dim=80), 1, 512) == 0
    assert L.workspace_size_q8(d, -1, 512) == 0 and L.workspace_size_q8(d, 1, -1) == 0
    assert L.workspace_size_q8(d, 1, 512, L.DELTA_HEAD_MAX) == need + 28 * 512 * 16 * 4
    assert L.full_attn_q8(d, p, FAKE, c, FAKE, FAKE, need - 1, check=False) == 3
    assert L.full_attn_q8(d, p, FAKE, c, FAKE, None, need, check=False) == 3
    assert L.full_attn_q8(d, p, FAKE + 2, c, FAKE, FAKE, need, check=False) == 1
    assert L.full_attn_q8(d, p, FAKE, c, None, FAKE, need, check=False) == 1
    sp = L.DeltaSelectParams(64, 16, 256, L.DELTA_HEAD_SUM)
    cap = L.sel_capacity(sp)
    assert L.select_attn_q8(d, p, sp, FAKE, c, FAKE, FAKE, FAKE, cap - 1, None, FAKE, need, check=False) == 1
    assert L.select_attn_q8(d, p, sp, FAKE, c, FAKE, None, FAKE, cap, None, FAKE, need, check=False) == 1
    sp_max = L.DeltaSelectParams(64, 16, 256, L.DELTA_HEAD_MAX)
    assert L.select_attn_q8(d, p, sp_max, FAKE, c, FAKE, FAKE, FAKE, cap, None, FAKE, need, check=False) == 3
    big = L.workspace_size_q8(d, 1, 40000)
    assert L.select_attn_q8(d, pt(L, maxp=40000), sp, FAKE, c, FAKE, FAKE, FAKE, cap, None, FAKE, big, check=False) == 2
    assert L.sparse_attn_q8(d, p, None, FAKE, 4, FAKE, c, FAKE, FAKE, need, check=False) == 1
    assert L.sparse_attn_q8(d, p, FAKE, FAKE, 0, FAKE, c, FAKE, FAKE, need, check=False) == 1
    assert L.sparse_attn_settled_q8(d, p, FAKE, None, 4, FAKE, c, FAKE, FAKE, need, check=False) == 1


def test_cache_write_and_read_arguments(L):
    d, p, c = desc(L), pt(L), cache(L)
    assert L.kv_append_q8(d, p, None, FAKE, c, check=False) == 1
    assert L.kv_append_q8(d, p, FAKE, FAKE + 8, c, check=False) == 1
    assert L.kv_append_layers_q8(d, p, [FAKE] * 65, [FAKE] * 65, [c] * 65, check=False) == 2
    other = cache(L, format=L.DELTA_INT8)
    assert L.kv_append_layers_q8(d, p, [FAKE] * 2, [FAKE] * 2, [c, other], check=False) == 1
    assert L.kv_append_layers_q8(d, p, [FAKE, None], [FAKE] * 2, [c, c], check=False) == 1
    assert L.kv_write_q8(d, p, None, 5, FAKE, FAKE, c, check=False) == 1
    assert L.kv_write_q8(d, p, FAKE, -1, FAKE, FAKE, c, check=False) == 1
    assert L.kv_write_q8(d, p, FAKE, 5, None, FAKE, c, check=False) == 1
    assert L.kv_write_q8(d, p, FAKE, 5, FAKE, FAKE + 8, c, check=False) == 1
    assert L.kv_write_q8(d, p, FAKE, 5, FAKE, FAKE, c, row_stride=4 * 128 - 8, check=False) == 1
    assert L.kv_write_q8(d, p, FAKE, 5, FAKE, FAKE, c, row_stride=4 * 128 + 4, check=False) == 1
    assert L.kv_write_q8(d, p, None, 0, None, None, c, check=False) == 0
    assert L.kv_read_q8(d, p, None, 5, None, c, FAKE, FAKE, check=False) == 1
    assert L.kv_read_q8(d, p, FAKE, 5, None, c, None, FAKE, check=False) == 1
    assert L.kv_read_q8(d, p, FAKE, 5, None, c, FAKE, FAKE + 4, check=False) == 1
    assert L.kv_read_q8(d, p, FAKE, -5, None, c, FAKE, FAKE, check=False) == 1


@pytest.mark.parametrize("bad", [dict(rotary_dim=0), dict(rotary_dim=3), dict(rotary_dim=130), dict(layout=2),
                                 dict(magnitude=math.inf), dict(magnitude=math.nan), dict(turns=None), dict(turns=FAKE + 4),
                                 dict(positions=None), dict(num_positions=0)])
def test_rope_plan_refusals(L, bad):
    kw = dict(turns=FAKE, rotary_dim=64, layout=L.DELTA_ROPE_HALF, magnitude=1.0, positions=FAKE, num_positions=1, offset=0)
    kw.update(bad)
    assert L.rope(desc(L), L.DeltaRope(*kw.values()), 1, FAKE, FAKE, FAKE, FAKE, check=False) == 1


def test_rope_arguments(L):
    d, plan = desc(L), L.DeltaRope(FAKE, 64, 0, 1.0, FAKE, 1, 0)
    row = 28 * 128
    for kw in (dict(rows=-1), dict(q=None), dict(k_out=None), dict(q=FAKE + 8), dict(k_out=FAKE + 2), dict(q_stride=row - 8),
               dict(q_stride=row + 4), dict(k_out_stride=4 * 128 + 1), dict(q_out=FAKE, q_stride=row, q_out_stride=row + 8)):
        a = dict(rows=1, q=FAKE, q_out=FAKE, k=FAKE, k_out=FAKE)
        a.update(kw)
        assert L.rope(d, plan, check=False, **a) == 1, kw
    assert L.rope(d, plan, 0, FAKE, FAKE, FAKE, FAKE, check=False) == 0
    assert L.rope(d, plan, 3, None, None, None, None, check=False) == 0
