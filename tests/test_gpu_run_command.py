"""The command ``run_decode --pool``: prompts and tokens that find no page are said. Needs a GB300."""

import re

import pytest

import partial_inverse_rope_gb300 as ir
from gpu_helpers import ensure_built
from partial_inverse_rope_gb300 import run_decode

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()
    yield
    assert ir.invrope_take_device_fault() == 0


def _run(capsys, *args):
    status = run_decode.main(["--pool", "--chunk", "3", "--topk", "40", "--nh", "16", *args])
    out = capsys.readouterr().out
    return status, out, [int(n) for n in re.search(r"no page for (\d+) prompts and (\d+) of (\d+) tokens", out).groups()]


@pytest.mark.parametrize("graph", [[], ["--graph"]])
@pytest.mark.parametrize("args", [["--rows", "5", "--prompt", "300", "--steps", "6"], ["--rows", "1", "--prompt", "1", "--steps", "2"],
                                  ["--rows", "9", "--prompt", "65", "--steps", "0", "--page", "64"]])
def test_every_prompt_is_taken(capsys, args, graph):
    """5 prompts of 150 to 300 tokens take 20 pages of 64, three quarters of what they could fill are 19."""
    status, out, (prompts, tokens, of) = _run(capsys, *args, *graph)
    assert status == 0 and prompts == 0 and tokens == 0 and of == int(args[1]) * int(args[5])
    assert "outputs finite: True; watchdog fault code 0" in out


@pytest.mark.parametrize("graph", [[], ["--graph"]])
def test_tokens_without_a_page_are_counted(capsys, graph):
    """8 sequences of 300 + 400 tokens: at most 704 each, and pages for three quarters."""
    status, out, (prompts, tokens, of) = _run(capsys, "--rows", "8", "--prompt", "300", "--steps", "400", "--page", "16", *graph)
    assert status == 0 and prompts == 0 and of == 3200
    assert 0 < tokens < of


def test_a_refused_prompt_is_a_failure(capsys, monkeypatch):
    monkeypatch.setattr(run_decode, "pool_pages", lambda lens, most, page: 19)
    status, out, (prompts, tokens, of) = _run(capsys, "--rows", "5", "--prompt", "300", "--steps", "6")
    assert status == 1 and prompts > 0
