"""The latent cache and its attention through the debug-bounds build (see
``test_gpu_debug_bounds.py``), in a fresh process: both formats, every block count,
odd splits, sizes and heads, rows split over blocks and empty ones, pages, slots and
indices out of range. No index check records a fault code. And the attention's
bounded waits, which run out where nothing arrives. Needs a GB300."""

import os
import subprocess
import sys
import textwrap

import pytest

from partial_inverse_rope_gb300.build import build

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = textwrap.dedent("""
    import torch
    import partial_inverse_rope_gb300 as ir

    gen = torch.Generator(device="cuda").manual_seed(1)
    BF16, E4M3 = ir.KV_LATENT_BF16, ir.KV_LATENT_E4M3

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=gen, device="cuda", dtype=torch.int32)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").to(torch.bfloat16)

    splits = [(448, 64), (480, 32), (96, 32), (48, 16), (16, 0), (16, 8), (512, 0), (112, 8), (272, 56), (16, 496)]
    lengths = [[1], [0, 64, 65, 0], [5, 640, 64, 1, 0, 320, 191], [9000, 17, 0, 4096], [0] * 3 + [70] * 300]
    done = 0
    for fmt in (BF16, E4M3):
        for nope, pe in splits + ([(0, 8), (6, 2), (450, 62), (200, 56)] if fmt == BF16 else []):
            for page, nh in ((64, 64), (7, 5), (16, 128)):
                pages = 9000 // page + 2
                cache = ir.kv_latent_empty(pages, page, nope, pe, fmt)
                n = pages * page
                slots = torch.randperm(n, generator=gen, device="cuda").to(torch.int32)
                ir.kv_latent_write(cache, normal(n, nope + pe), slots, nope, pe)
                some = ints(-5, n + 5, 777)
                ir.kv_latent_write(cache, normal(3, nope + pe), ints(-2**31, 0, 3), nope, pe)
                ir.kv_latent_read(cache, some, nope, pe)
                lens = lengths[done % len(lengths)]
                table = ints(-1, pages + 1, len(lens), -(-max(lens) // page) + 1)
                ir.latent_attn_decode(normal(len(lens), nh, nope + pe), cache, table,
                                      torch.tensor(lens, dtype=torch.int32, device="cuda"), nope, pe)
                rows, topk = [(1, 1), (3, 0), (5, 2048), (300, 130), (40, 65)][done % 5]
                ir.latent_attn_sparse(normal(rows, nh, nope + pe), cache, ints(-3, n + 3, rows, topk), nope, pe)
                done += 1
    code = ir.invrope_take_device_fault()
    print(done, "latent cases, fault code", hex(code))
    assert code == 0, hex(code)
""")


def test_latent_operators_through_the_debug_bounds_build():
    lib = build(debug_bounds=True)
    env = dict(os.environ, INVROPE_LIBRARY=lib)
    r = subprocess.run([sys.executable, "-c", SCRIPT], env=env, cwd=ROOT, capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "72 latent cases, fault code 0x0" in r.stdout


WAITS = textwrap.dedent("""
    import ctypes, time
    import torch
    import partial_inverse_rope_gb300 as ir

    hook = ir.lib().latent_debug_wait
    hook.argtypes, hook.restype = [ctypes.c_int, ctypes.POINTER(ctypes.c_int)], ctypes.c_int

    cache = ir.kv_latent_empty(40, 64, 448, 64, ir.KV_LATENT_E4M3)
    x = torch.randn(2560, 512, device="cuda").to(torch.bfloat16)
    ir.kv_latent_write(cache, x, torch.arange(2560, dtype=torch.int32, device="cuda"), 448, 64)
    q = torch.randn(2, 64, 512, device="cuda").to(torch.bfloat16)
    table = torch.arange(40, dtype=torch.int32, device="cuda").view(2, 20).contiguous()
    lens = torch.tensor([1280, 77], dtype=torch.int32, device="cuda")
    before = ir.latent_attn_decode(q, cache, table, lens, 448, 64)
    assert ir.invrope_take_device_fault() == 0
    for which, code, said in ((0, 0xA01, 2), (1, 0xB01, 2), (2, 0, 0)):
        done = (ctypes.c_int * 2)()
        t0 = time.monotonic()
        assert hook(which, done) == 0
        took = time.monotonic() - t0
        assert list(done) == [2, said], (which, list(done))
        assert 1.5 < took < 4.0, (which, took)  # one wait of 2 s; the second sees the flag
        assert ir.invrope_take_device_fault() == code, which
        assert ir.invrope_take_device_fault() == 0
        after = ir.latent_attn_decode(q, cache, table, lens, 448, 64)
        assert torch.equal(after[0], before[0]) and torch.equal(after[1], before[1])
    assert ir.invrope_take_device_fault() == 0
    print("waits ran out, context usable")
""")


def test_waits_that_run_out_report_and_leave_the_context_usable():
    lib = build(debug_bounds=True)
    env = dict(os.environ, INVROPE_LIBRARY=lib)
    r = subprocess.run([sys.executable, "-c", WAITS], env=env, cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "waits ran out, context usable" in r.stdout
