"""The bounds-guard build libsq_debug.so guards the 4-bit and paged-cache kernels: with every buffer taken
for a little shorter than it is, each entry point's accesses near the end are skipped and reported;
with the true sizes no guard fires, in these calls and in the suites of far, tiny and non-finite
inputs. In child processes (the binding loads one library per process)."""
import os
import subprocess
import sys

import pytest

from w8a8_quantized_gemm_b200 import build as _b
from w8a8_quantized_gemm_b200 import sq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SUITES = ["tests/test_gpu_int4_tokens.py", "tests/test_gpu_int4_scales.py", "tests/test_gpu_int4_nonfinite.py",
          "tests/test_gpu_kv_scales.py", "tests/test_gpu_kv_queries.py", "tests/test_gpu_kv_far.py"]

SCRIPT = r"""
import torch
from w8a8_quantized_gemm_b200 import sq

bf16 = torch.bfloat16
cuda = dict(device="cuda")


def quant(asym):
    N, K = 40, 144
    W = torch.randn(N, K, **cuda).to(bf16)
    Wp = torch.zeros(sq.sq_int4_weight_bytes(N, K), dtype=torch.uint8, **cuda)
    e = torch.zeros(3, N, dtype=bf16, **cuda)
    z = torch.zeros(3, N, dtype=torch.uint8, **cuda) if asym else None
    return lambda: sq.sq_quant_weight_int4(W, None, 64, Wp, e, z), Wp, (W, Wp, e, z)


def dequant():
    call, _, (W, Wp, e, z) = quant(True)
    call()
    out = torch.zeros_like(W)
    return lambda: sq.sq_dequant_weight_int4(Wp, e, z, 64, out), out


def linear(M, N):
    K = 144
    Wp = torch.randint(0, 256, (sq.sq_int4_weight_bytes(N, K),), dtype=torch.uint8, **cuda)
    e = torch.ones(3, N, dtype=bf16, **cuda)
    z = torch.full((3, N), 7, dtype=torch.uint8, **cuda)
    X = torch.randn(M, K, **cuda).to(bf16)
    Y = torch.zeros(M, N, dtype=bf16, **cuda)
    return lambda: sq.sq_int4_linear(X, Wp, e, z, 64, None, Y), Y


def cache(int8, P):
    k = torch.ones(2, 3, 1, P, 64, dtype=torch.int8 if int8 else bf16, **cuda)
    s = torch.ones(2, 3, 1, P, **cuda)
    return sq.KvCache(k[0].clone(), k[1].clone(), s[0].clone(), s[1].clone()) if int8 else sq.KvCache(k[0].clone(), k[1].clone())


def append(int8):
    c = cache(int8, 8)
    x = torch.full((2, 1, 64), 3.0, dtype=bf16, **cuda)
    slots = torch.tensor([0, 23], dtype=torch.int32, **cuda)  # the last one of the cache
    return lambda: sq.sq_rope_kv_append(None, x, x, None, None, None, slots, c, None), c.tensors[0]


def attend(int8, P, n):
    c = cache(int8, P)
    q = torch.ones(1, 2, 64, dtype=bf16, **cuda)
    out = torch.zeros(1, 2, 64, dtype=bf16, **cuda)
    ws = sq.workspace(sq.SQ_OP_PAGED_ATTENTION, 1, 2, 64)
    table, lens = torch.arange(3, dtype=torch.int32, **cuda)[None], torch.tensor([n], dtype=torch.int32, **cuda)
    return lambda: sq.sq_paged_attention(q, c, table, lens, 0.125, out, ws=ws), out


calls = {"quant": quant(False), "quant with zero points": quant(True), "dequant": dequant(), "linear 1": linear(1, 2856),
         "linear 4": linear(4, 9480), "linear 4, few rows": linear(4, 40), "linear 16": linear(16, 40), "linear 17": linear(17, 40),
         "linear 64": linear(64, 40), "append": append(False), "append int8": append(True)}
for P, n in ((8, 24), (32, 96)):  # tiles row by row, and whole
    calls["attention %d" % P], calls["attention int8 %d" % P] = attend(False, P, n), attend(True, P, n)
for name, (call, out, *_) in calls.items():
    sq.sq_debug_guard_margin(0)
    call()
    sq.sq_sync_status()
    want = out.clone()
    out.zero_()
    sq.sq_debug_guard_margin(1)
    call()
    try:
        sq.sq_sync_status()
        print("SILENT", name)
    except sq.SqError as e:
        assert e.status == sq.SQ_ERR_BOUNDS and "guard" in str(e), e
    if not name.startswith("attention"):  # the end of the output is as it was
        assert int(out.reshape(-1)[-1:].view(torch.uint8).max()) == 0, name
    sq.sq_debug_guard_margin(0)
    call()
    sq.sq_sync_status()
    if "append" not in name:  # (what it leaves alone in the cache was cleared)
        assert torch.equal(out, want), name
print("GUARDED")
"""


def _child(*args):
    return subprocess.run([sys.executable, *args], cwd=ROOT, env=dict(os.environ, SQ_LIB_PATH=_b.LIB_DEBUG),
                          capture_output=True, text=True, timeout=1800)


def test_the_product_library_has_no_guards():
    with pytest.raises(sq.SqError) as ei:
        sq.sq_debug_guard_margin(0)
    assert ei.value.status == sq.SQ_ERR_UNSUPPORTED


@pytest.mark.gpu
def test_guards_fire():
    r = _child("-c", SCRIPT)
    assert r.returncode == 0 and "SILENT" not in r.stdout and "GUARDED" in r.stdout, r.stdout[-4000:] + r.stderr[-2000:]


@pytest.mark.gpu
def test_far_tiny_and_nonfinite_suites_on_the_guarded_build():
    r = _child("-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", *SUITES)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert " passed" in r.stdout
