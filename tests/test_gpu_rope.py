"""GPU: rotary positions against the fp64 definition."""
import numpy as np
import pytest
import torch

from oracle import operators as R
from tests.operator_helpers import DT, HALF_STEP, assert_within, desc, host, lib, stream

pytestmark = pytest.mark.gpu


def tolerance(x, ref, turns, layout, magnitude, dtype):
    """|a| + |b| per rotated value times the error of cos and sin (float rounding of at most half a turn: 2 pi
    2^-26; sincospi 2^-22; their magnitude and the product and sum: four more roundings), and the output's."""
    half = len(turns)
    mag = np.abs(x).copy()
    for j in range(half):
        a, b = (j, j + half) if layout == "half" else (2 * j, 2 * j + 1)
        mag[..., a] = mag[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    mag[..., 2 * half:] = 0.0
    err = mag * abs(magnitude) * (2.0 ** -23 + 2.0 ** -22 + 4 * 2.0 ** -24)
    return err * (1 + HALF_STEP[dtype]) + np.abs(ref) * HALF_STEP[dtype] * (np.arange(x.shape[-1]) < 2 * half)


CASES = [
    # dtype, layout, hq, hkv, D, rotary_dim, rows, positions, offset, magnitude
    ("bf16", "half", 28, 4, 128, 128, 1, [8191], 0, 1.0),
    ("bf16", "interleaved", 8, 8, 128, 64, 5, [0, 1, 2, 3, 4], 0, 1.0),
    ("bf16", "half", 6, 2, 64, 50, 3, [7, 1000003, 12], -1, 1.25),      # odd rotary width: scalar items
    ("bf16", "interleaved", 3, 3, 128, 2, 2, [5, 6], 0, 1.0),
    ("f32", "half", 8, 1, 64, 64, 7, [3, 70], -1, 0.75),                # rows share positions in turn
    ("f32", "interleaved", 2, 1, 64, 62, 4, [0, 16777215, 1048576, 2], 0, 1.0),
    ("f32", "half", 5, 1, 128, 96, 1, [0], -1, 1.0),                    # an empty sequence's position, -1
    ("f32", "half", 1, 1, 128, 126, 2, [2147483647, 11], 0, 1.0),
]


def make(rows, heads, d, dtype, seed, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.randn(rows, heads * d + pad, generator=g, device="cuda").to(DT[dtype])
    return buf


def plan(L, turns, rd, layout, magnitude, pos, offset):
    return L.DeltaRope(turns.data_ptr(), rd, L.DELTA_ROPE_HALF if layout == "half" else L.DELTA_ROPE_INTERLEAVED, magnitude,
                       pos.data_ptr(), pos.numel(), offset)


@pytest.mark.parametrize("how", ["apart", "in place", "strided"])
@pytest.mark.parametrize("dtype,layout,hq,hkv,d,rd,rows,positions,offset,magnitude", CASES)
def test_rope(how, dtype, layout, hq, hkv, d, rd, rows, positions, offset, magnitude):
    L = lib()
    turns_h = R.rope_turns(rd, "bands", factor=4.0, original_len=4096.0, low=1.0, high=32.0)
    turns = torch.from_numpy(turns_h).cuda()
    pos = torch.tensor(positions, dtype=torch.int32, device="cuda")
    pad = 16 if how == "strided" else 0
    q, k = make(rows, hq, d, dtype, 1, pad), make(rows, hkv, d, dtype, 2, 2 * pad)
    q0, k0 = q.clone(), k.clone()
    qo, ko = (q, k) if how == "in place" else (torch.full_like(q, 77.0), torch.full_like(k, 77.0))
    strides = (dict(q_stride=q.stride(0), q_out_stride=qo.stride(0), k_stride=k.stride(0), k_out_stride=ko.stride(0))
               if how == "strided" else {})
    L.rope(desc(hq, hkv, d, dtype, 0), plan(L, turns, rd, layout, magnitude, pos, offset), rows, q, qo, k, ko,
           stream=stream(), **strides)
    at = [positions[r % len(positions)] + offset for r in range(rows)]
    for x0, out, heads in ((q0, qo, hq), (k0, ko, hkv)):
        x = host(x0)[:, :heads * d].reshape(rows, heads, d)
        ref = R.rope(x, at, turns_h, layout, magnitude)
        got = host(out)
        assert_within(got[:, :heads * d].reshape(rows, heads, d), ref, tolerance(x, ref, turns_h, layout, magnitude, dtype), how)
        if how == "strided":     # what lies between the rows stays
            assert np.all(got[:, heads * d:] == 77.0)


def test_rope_of_one_side_only():
    L = lib()
    turns = torch.from_numpy(R.rope_turns(64)).cuda()
    pos = torch.tensor([9], dtype=torch.int32, device="cuda")
    q, k = make(2, 4, 64, "bf16", 3), make(2, 2, 64, "bf16", 4)
    both_q, both_k, only_q, only_k = (torch.empty_like(x) for x in (q, k, q, k))
    p, d = plan(L, turns, 64, "half", 1.0, pos, 0), desc(4, 2, 64, "bf16", 0)
    L.rope(d, p, 2, q, both_q, k, both_k, stream=stream())
    L.rope(d, p, 2, q, only_q, None, None, stream=stream())
    L.rope(d, p, 2, None, None, k, only_k, stream=stream())
    assert torch.equal(both_q, only_q) and torch.equal(both_k, only_k)


def test_rope_of_many_rows_matches_row_by_row():
    # the launch for many rows gives a block several of them (the last block fewer)
    L = lib()
    rows = 148 * 8 * 4 + 3
    turns = torch.from_numpy(R.rope_turns(128)).cuda()
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    q, k = make(rows, 2, 128, "bf16", 5), make(rows, 1, 128, "bf16", 6)
    qo, ko, q1, k1 = (torch.empty_like(x) for x in (q, k, q, k))
    d = desc(2, 1, 128, "bf16", 0)
    L.rope(d, plan(L, turns, 128, "half", 1.0, pos, 0), rows, q, qo, k, ko, stream=stream())
    for r in list(range(0, rows, 997)) + [rows - 3, rows - 2, rows - 1]:
        L.rope(d, plan(L, turns, 128, "half", 1.0, pos[r:r + 1], 0), 1, q[r], q1[r], k[r], k1[r], stream=stream())
        assert torch.equal(qo[r], q1[r]) and torch.equal(ko[r], k1[r])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype,rd", [("bf16", 50), ("bf16", 6), ("f32", 62), ("bf16", 64)])
def test_other_dimensions_pass_through_whatever_they_hold(dtype, rd, layout):
    L = lib()
    x = make(3, 4, 128, dtype, 7).view(3, 4, 128)
    odd = torch.tensor([float("inf"), -float("inf"), -0.0, 0.0, float("nan")], device="cuda").to(x.dtype)
    x[..., rd:] = odd.repeat(26)[: 128 - rd]
    turns = torch.from_numpy(R.rope_turns(rd)).cuda()
    pos = torch.tensor([5, 90, 7], dtype=torch.int32, device="cuda")
    out = torch.full_like(x, 3.0)
    L.rope(desc(4, 4, 128, dtype, 0), plan(L, turns, rd, layout, 1.0, pos, 0), 3, x, out, None, None, stream=stream())
    a, b = out[..., rd:], x[..., rd:]
    assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(9.0), b.nan_to_num(9.0))
    assert torch.equal(torch.signbit(a) & ~a.isnan(), torch.signbit(b) & ~b.isnan())
    assert bool(out[..., :rd].isfinite().all())


@pytest.mark.parametrize("rows", [2, 600, 1300, 2600, 5000])
def test_every_split_of_rows_over_warps(rows):
    L = lib()
    turns_h = R.rope_turns(30)
    turns = torch.from_numpy(turns_h).cuda()
    pos = torch.arange(rows, dtype=torch.int32, device="cuda") * 3
    q, k = make(rows, 5, 64, "f32", 8), make(rows, 5, 64, "f32", 9)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    L.rope(desc(5, 5, 64, "f32", 0), plan(L, turns, 30, "half", 1.0, pos, 0), rows, q, qo, k, ko, stream=stream())
    pick = sorted({0, 1, rows // 3, rows - 2, rows - 1})
    for x0, out in ((q, qo), (k, ko)):
        x = host(x0)[pick].reshape(len(pick), 5, 64)
        ref = R.rope(x, [3 * r for r in pick], turns_h, "half")
        assert_within(host(out)[pick].reshape(len(pick), 5, 64), ref, tolerance(x, ref, turns_h, "half", 1.0, "f32"))
