"""Rows of 8-bit caches that another program wrote: every code under every scale
byte has the same value in ``kv_latent_read`` and in the attention. Needs a GB300."""

import numpy as np
import pytest
import torch

import partial_inverse_rope_gb300 as ir
from gpu_helpers import ensure_built
from oracle import latent_oracle as L

pytestmark = pytest.mark.gpu

E4M3 = ir.KV_LATENT_E4M3


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()
    yield
    assert ir.invrope_take_device_fault() == 0


def _rows_of(codes, nope):
    """Under each of the 256 scale bytes, a row for each of ``codes``, all of whose
    channels hold it; and the channels' value, as bf16, [rows]."""
    byte, code = (t.flatten() for t in torch.meshgrid(torch.arange(256), codes.long(), indexing="ij"))
    rows = torch.zeros(len(byte), 1, ir.kv_latent_row_bytes(nope, 0, E4M3), dtype=torch.uint8)
    rows[:, 0, :nope] = code[:, None].to(torch.uint8)
    rows[:, 0, nope:nope + -(-nope // 64)] = byte[:, None].to(torch.uint8)
    scale = torch.where(byte == 255, torch.nan, torch.exp2((byte - 127).double()))
    value = torch.from_numpy(L.e4m3_value(code.numpy())) * scale
    return rows.cuda(), value.float().to(torch.bfloat16)  # fp32 holds it exactly, or an infinity


def _read_and_attended(codes, nope):
    """What each row reads as, and the attention's output over that row alone with a
    query of zeros: its weight is 1, and what is not finite makes the output NaN."""
    cache, value = _rows_of(codes, nope)
    slots = torch.arange(len(value), dtype=torch.int32, device="cuda")
    read = ir.kv_latent_read(cache, slots, nope, 0).cpu()
    q = torch.zeros(len(value), 1, nope, dtype=torch.bfloat16, device="cuda")
    O, _ = ir.latent_attn_sparse(q, cache, slots[:, None].contiguous(), nope, 0)
    return value[:, None].expand(-1, nope), read, O[:, 0].cpu()


def _bits(t):
    """bf16 bits, every NaN alike."""
    return torch.where(torch.isnan(t), torch.nan, t.float()).to(torch.bfloat16).contiguous().view(torch.int16)


def _same(want, read, attended):
    assert torch.equal(_bits(read), _bits(want))
    want = torch.where(torch.isfinite(want), want, torch.nan)
    assert torch.equal(torch.isnan(attended), torch.isnan(want))
    # a tensor core may drop fp32 subnormals, of 2^-126 at most
    off = (attended.double() - want.double()).abs().nan_to_num(0.0)
    assert (off <= 2.0 ** -126).all()
    normal = want.abs() >= 2.0 ** -126
    assert torch.equal(attended[normal], want[normal])


@pytest.mark.parametrize("nope", [64, 128, 400])
def test_every_scale_byte_reads_alike(nope):
    """Blocks of 128 channels with and without zeros behind the codes."""
    codes = torch.arange(256)[(torch.arange(256) & 127) != 127]
    _same(*_read_and_attended(codes, nope))


def test_the_least_scale_is_not_zero():
    cache, value = _rows_of(torch.tensor([0x38, 0x7E]), 64)  # 1 and 448
    got = ir.kv_latent_read(cache, torch.arange(2, dtype=torch.int32, device="cuda"), 64, 0).cpu()
    assert got[:, 0].tolist() == [2.0 ** -127, 448 * 2.0 ** -127] == value[:2].tolist()


@pytest.mark.parametrize("nope", [64, 128, 400])
def test_codes_of_all_bits_are_the_numbers_after_the_largest(nope):
    """0x7F and 0xFF are no NaN in a row: +-480 times the scale, read and attended to."""
    want, read, attended = _read_and_attended(torch.tensor([0x7F, 0xFF]), nope)
    byte = torch.arange(256).repeat_interleave(2)
    want = torch.tensor([480.0, -480.0]).double().repeat(256) * torch.exp2((byte - 127).double())
    want = torch.where(byte == 255, torch.nan, want).float().to(torch.bfloat16)
    _same(want[:, None].expand(-1, nope), read, attended)
