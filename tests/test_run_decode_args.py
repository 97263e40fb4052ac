"""Arguments that ``run_decode`` refuses. Needs no GPU."""

import pytest

from partial_inverse_rope_gb300 import run_decode


@pytest.mark.parametrize("prompt", ["0", "-5"])
def test_a_prompt_without_tokens_is_refused(prompt, capsys):
    """Its selected tokens would be rows that nothing has written."""
    with pytest.raises(SystemExit) as e:
        run_decode.main(["--prompt", prompt])
    assert e.value.code == 2 and "--prompt must be at least 1" in capsys.readouterr().err
