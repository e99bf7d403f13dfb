"""GPU: the BGTQ_DEBUG_BOUNDS build on the 4-bit cache: a page entry outside the
pool, a length past the bound and an append past the capacity set
BGTQ_STATUS_BOUNDS beside the bits that the default build sets, and clean calls
give the same bytes and outputs.  Each bad index is one that the default build
catches before any access, so neither build leaves the cache's memory.  One
child process a build, which chooses it by its environment."""

import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

APPEND_CAPACITY, SEQLEN_CAPACITY, PAGE_RANGE, BOUNDS = 1, 2, 4, 16

CHILD = r'''
import hashlib, json
import torch
import rope_aware_quantized_gb300 as bg

H, G, T = 8, 4, 8192  # 4096 groups: the append of many groups
i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
torch.manual_seed(0)
k, v = (torch.randn((1, H, T, 128), device="cuda").half() for _ in range(2))
q = torch.randn((1, H * G, 33, 128), device="cuda").half()
res = {"lib": bg._native.library_path()}
digest = hashlib.sha256()

def append(cache, n, at):
    st = i32(0)
    bg.bgtq_fp4_append(k[:, :, :n], v[:, :, :n], i32(at), cache, status=st)
    return int(st.item())

def attend(cache, n, t, note=False):
    ws = torch.zeros(bg.bgtq_fp4_attn_workspace(H, G, 1, t, T), dtype=torch.uint8, device="cuda")
    out, st = torch.zeros((1, H * G, t, 128), device="cuda"), i32(0)
    bg.bgtq_fp4_attn(q[:, :, :t], cache, i32(n), T, out, ws, status=st)
    if note:
        digest.update(out.cpu().numpy().tobytes())
    return int(st.item())

cache = bg.Fp4Cache(H, 1, T, page_tokens=32)
res["clean"] = [append(cache, T, 0), append(cache, 5, 77), attend(cache, T, 1, True), attend(cache, T - 3, 33, True)]
digest.update(cache.groups.cpu().numpy().tobytes())
res["digest"] = digest.hexdigest()
res["bad_seq"] = [attend(cache, T + 100, 1), attend(cache, T + 100, 33)]
res["bad_append"] = [append(cache, 2, T - 1), append(cache, T, 1)]
cache.page_table[0, 3] = cache.n_pages + 5
res["bad_page"] = [attend(cache, T, 1), attend(cache, T, 33), append(cache, 40, 70), append(cache, T, 0)]
print(json.dumps(res))
'''


def run_child(debug):
    env = dict(os.environ, BGTQ_DEBUG_BOUNDS="1" if debug else "0", PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", CHILD], env=env, cwd=ROOT, capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, r.stderr[-4000:]
    return json.loads(r.stdout.strip().splitlines()[-1])


def test_bad_indices_are_flagged_in_the_debug_build_only():
    d, n = run_child(True), run_child(False)
    assert d["lib"].endswith("libbgtq_debug_bounds.so") and n["lib"].endswith("libbgtq.so")
    for r, extra in ((d, BOUNDS), (n, 0)):
        assert r["clean"] == [0] * 4
        assert r["bad_seq"] == [SEQLEN_CAPACITY | extra] * 2
        assert r["bad_append"] == [APPEND_CAPACITY | extra] * 2
        assert r["bad_page"] == [PAGE_RANGE | extra] * 4
    assert d["digest"] == n["digest"]
