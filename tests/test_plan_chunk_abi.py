"""The balanced chunk of a ragged batch for every shape that attention takes: a multiple of 64 in [64, 8192], also where the query
rows of one kv head take more CTAs than the GPU holds. Needs no GPU (the rule then counts 148 SMs)."""
import json
import os
import subprocess
import sys

import pytest

from sub_byte_quantized_gb300 import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CASES = [("int8_b64", 256, 8, 1, 512), ("e4m3_b64", 256, 16, 2, 300), ("int8_b64", 128, 8, 1, 4096), ("e4m3_b64", 128, 8, 8, 65000),
         ("q6_0", 256, 8, 1, 512), ("q6_0", 256, 32, 2, 4096), ("q6_0", 128, 8, 1, 8192), ("q4_0", 128, 8, 1, 8192), ("q8_0", 128, 64, 1, 4096),
         ("asym4_g32", 128, 8, 1, 8192), ("had_int4", 128, 8, 1, 16384), ("had_int2", 128, 8, 1, 65536), ("had_int2+had_int4", 128, 8, 1, 8192),
         ("q4_0", 256, 8, 1, 512), ("int8_b64", 256, 1, 1, 1), ("q6_0", 256, 1, 1, 5)]
CALL = """
import ctypes as C, json, sys
from sub_byte_quantized_gb300 import _lib
P = 1 << 20
lens, cases = json.loads(sys.argv[1])
n = (C.c_int32 * len(lens))(*lens)
for layout, D, hq, hkv, nq in cases:
    k, _, v = layout.partition("+")
    ids = _lib.LAYOUT_IDS
    c = _lib.KvqPagedCache(layout=_lib.mixed(ids[k], ids[v]) if v else ids[k], batch=len(lens), n_kv_heads=hkv, head_dim=D,
                           n_pages=64, page_size=64, max_pages_per_seq=1 << 14)
    for f, t in c._fields_:
        if t is C.c_void_p and f not in ("k_recent", "v_recent"):
            setattr(c, f, P)
    print(json.dumps([_lib.lib().kvq_paged_attend_plan_chunk(C.byref(c), hq, nq, dt, C.cast(n, C.c_void_p)) for dt in (0, 1, 2)]), flush=True)
"""


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__ as g
    try:
        _lib.lib()
    except RuntimeError:
        g.build()


@pytest.mark.parametrize("lens", [(0, 0, 0), (1, 0, 700), (5000, 64, 1 << 20)])
def test_every_shape_has_a_chunk(lens):
    """In a process of its own: an arithmetic fault there would end this one."""
    r = subprocess.run([sys.executable, "-c", CALL, json.dumps([lens, CASES])], capture_output=True, text=True, cwd=ROOT, timeout=300)
    got = [json.loads(x) for x in r.stdout.splitlines()]
    assert r.returncode == 0, (r.returncode, CASES[len(got)], r.stderr[-500:])
    assert len(got) == len(CASES)
    for case, chunks in zip(CASES, got):
        assert all(64 <= x <= 8192 and x % 64 == 0 for x in chunks), (case, chunks)
