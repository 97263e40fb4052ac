"""Slots with the page table in shared memory through the debug-bounds build (see
``test_gpu_debug_bounds.py``), in a fresh process. No index check records a fault code.
Needs a GB300."""

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

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=gen, device="cuda", dtype=torch.int32)

    done = 0
    vectors = 16 * 1024 * torch.cuda.get_device_properties(0).multi_processor_count  # of a sequence
    for topk, seqs, gone, width, page in [(2052, 3, 0, 8192, 1), (2048, 2, 0, 100, 64), (2052, 3, 1, 50, 48), (641, 2, 0, 8192, 3),
                                          (641, 3, 1, 20, 64), (65537, 2, 0, 100, 16), (3, 2, 0, 7, 5)]:
        sq = -(-vectors // (topk // 4 if topk % 4 == 0 else topk)) + 1
        table, lens = ints(-2, seqs * width + 2, seqs - gone, width), ints(-3, width * page + 9, seqs - gone)
        idx = ints(-5, width * page + 30, seqs * sq - 2, topk)
        got = ir.kv_idx_local_to_slots(idx, table, lens, page, seqs * width, sq)
        assert torch.equal(got, ir.kv_idx_local_to_slots(idx, table, lens, page, seqs * width, sq, out=idx))
        done += 1
    code = ir.invrope_take_device_fault()
    print(done, "cases, fault code", hex(code))
    assert code == 0, hex(code)
""")


def test_through_the_debug_bounds_build():
    lib = build(debug_bounds=True)
    env = dict(os.environ, INVROPE_LIBRARY=lib)
    r = subprocess.run([sys.executable, "-c", SCRIPT], env=env, cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "7 cases, fault code 0x0" in r.stdout, r.stdout
