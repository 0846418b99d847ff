"""CPU: workspace sizes grow with the shape and hold their two areas."""
import subprocess
import sys

import pytest

import long_context_layer_b200 as L


def desc(hq, hkv, d, dtype=L.DELTA_BF16):
    return L.DeltaDesc(hq, hkv, d, 16, dtype, 0.0, 16)


@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 64), (28, 4, 128), (64, 64, 128), (8, 1, 64)])
@pytest.mark.parametrize("size", [lambda *a: L.workspace_size_reduce(*a, 0), lambda *a: L.workspace_size_reduce(*a, 1),
                                  lambda *a: L.workspace_size_q8(*a, 0), lambda *a: L.workspace_size_q8(*a, 1)])
def test_sizes_hold_both_areas(size, hq, hkv, d):
    for batch in (1, 3, 64):
        for pages in (1, 17, 4096, 32768):
            nb = size(desc(hq, hkv, d), batch, pages)
            lead = nb // 32 // 256 * 256
            # 8 bytes a page and 4 bytes a unit and sequence, each rounded up to 256, lie before the lead
            assert nb % 256 == 0 and lead >= 256 + sum(-(-x // 256) * 256 for x in (4 * batch * hkv, 4 * batch, 8 * batch * pages))
            # a float per (query head, page) and a key per page behind it
            assert nb - lead >= 4 * batch * hq * pages + 4 * batch * pages


@pytest.mark.parametrize("size", [L.workspace_size_reduce, L.workspace_size_q8])
def test_the_logits_add_their_own_bytes(size):
    for hq, batch, pages in ((28, 1, 512), (1, 1, 4), (40, 16, 1100), (8, 3, 32768)):
        d = desc(hq, 1 if hq < 9 else 4, 64) if hq != 40 else desc(40, 8, 128)
        a, b = size(d, batch, pages, L.DELTA_HEAD_SUM), size(d, batch, pages, L.DELTA_HEAD_MAX)
        assert b - a == -(-64 * batch * hq * pages // 256) * 256
        lead = b // 32 // 256 * 256
        assert b - lead >= 68 * batch * hq * pages + 4 * batch * pages


def test_the_largest_batches_are_answered():
    # in a process of its own: a product of batch and heads that came out as 0 in 32 bits ended it
    code = ("import long_context_layer_b200 as L\n"
            "for hkv in (64, 16, 4, 1):\n"
            "    d = L.DeltaDesc(hkv, hkv, 128, 16, L.DELTA_BF16, 0.0, 16)\n"
            "    sizes = [[f(d, b, 4, r) for b in (1 << 16, 1 << 26, 1 << 27, 1 << 28, 1 << 30, 2 ** 31 - 1)]\n"
            "             for f in (L.workspace_size_reduce, L.workspace_size_q8) for r in (0, 1)]\n"
            "    assert all(s == sorted(s) and s[0] > 0 for s in sizes), sizes\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=L.__path__[0] + "/..")
    assert r.returncode == 0, r.stderr[-500:]
