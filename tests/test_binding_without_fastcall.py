"""CPU: the package imports and calls without the call module, which is built for one interpreter and named for it."""
import glob
import os
import subprocess
import sys
import sysconfig

import long_context_layer_b200 as L
from long_context_layer_b200 import _native as N

PACKAGE = os.path.dirname(N.__file__)

WITHOUT = """
import sys
sys.modules["long_context_layer_b200._fastcall"] = None          # as if it were not built
import long_context_layer_b200 as L
from long_context_layer_b200 import _native as N
assert N._bind is None
import pytest
FAKE = 1 << 40
d = L.DeltaDesc(28, 4, 128, 16, L.DELTA_BF16, 0.0, 512)
p = L.DeltaPageTable(FAKE, FAKE, FAKE, 1, 512)
c = L.DeltaQ8Cache(FAKE, FAKE, FAKE, FAKE, L.DELTA_E4M3)
ws = 1 << 30
calls = [
    lambda d, c: L.window_attn(d, p, 16, -1, FAKE, FAKE, FAKE, FAKE, FAKE, ws, check=False),
    lambda d, c: L.kv_append_q8(d, p, None, FAKE, c, check=False),
    lambda d, c: L.kv_append_layers_q8(d, p, [FAKE], [FAKE + 4], [c], check=False),
    lambda d, c: L.kv_write_q8(d, p, None, 5, FAKE, FAKE, c, check=False),
    lambda d, c: L.kv_read_q8(d, p, FAKE, -5, None, c, FAKE, FAKE, check=False),
    lambda d, c: L.full_attn_q8(d, p, FAKE + 8, c, FAKE, FAKE, ws, check=False),
    lambda d, c: L.select_attn_q8(d, p, L.DeltaSelectParams(8, -1, 64, 0), FAKE, c, FAKE, FAKE, FAKE, 64, None, FAKE, ws, check=False),
    lambda d, c: L.sparse_attn_q8(d, p, FAKE, FAKE, 0, FAKE, c, FAKE, FAKE, ws, check=False),
    lambda d, c: L.sparse_attn_settled_q8(d, p, None, FAKE, 4, FAKE, c, FAKE, FAKE, ws, check=False),
    lambda d, c: L.window_attn_q8(d, p, 16, 4, FAKE, c, None, FAKE, ws, check=False),
    lambda d, c: L.rope(d, L.DeltaRope(FAKE, 3, 0, 1.0, FAKE, 1, 0), 1, FAKE, FAKE, None, None, check=False),
]
for f in calls:
    assert f(d, c) == 1
    for wrong in ((p, c), (d, p)) if f is not calls[0] and f is not calls[-1] else ((p, c),):
        if f is calls[2] and wrong[1] is p:
            continue                         # an array of caches is made there
        with pytest.raises(TypeError):
            f(*wrong)
for bad, error in ((dict(window_tokens=2 ** 31), OverflowError), (dict(window_tokens=1.5), TypeError), (dict(q=-1), OverflowError),
                   (dict(q=2 ** 64), OverflowError), (dict(q="text"), AttributeError)):
    a = dict(window_tokens=16, q=FAKE, **{})
    a.update(bad)
    with pytest.raises(error):
        L.window_attn(d, p, a["window_tokens"], 4, a["q"], FAKE, FAKE, FAKE, FAKE, ws, check=False)
with pytest.raises(TypeError):
    N._window_attn(d, p)
assert L.workspace_size(d, 1, 512) > 0                            # the calls that never went through it
print("ok")
"""


def test_the_package_works_without_the_call_module():
    r = subprocess.run([sys.executable, "-c", WITHOUT], capture_output=True, text=True, cwd=os.path.dirname(PACKAGE))
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr[-800:]


def test_the_call_module_is_named_for_this_interpreter():
    built = [os.path.basename(x) for x in glob.glob(os.path.join(PACKAGE, "_fastcall*"))]
    assert "_fastcall" + sysconfig.get_config_var("EXT_SUFFIX") in built
    assert "_fastcall.so" not in built          # no file that every interpreter would load
    assert N._bind is not None and L.window_attn is N.window_attn
