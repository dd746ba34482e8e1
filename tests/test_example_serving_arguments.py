"""The serving arguments of examples/decode_step.py."""
import pytest


@pytest.mark.parametrize("argv,cache,serve", [([], "e4m3", False), (["--cache", "int4"], "int4", False),
                                              (["--serve", "--cache", "bf16"], "bf16", True)])
def test_taken(argv, cache, serve):
    from examples import decode_step as ex
    args = ex.arguments(argv)
    assert (args.cache, args.serve) == (cache, serve)


def test_refused(capsys):
    from examples import decode_step as ex
    with pytest.raises(SystemExit):
        ex.arguments(["--cache", "int3"])
    assert "int3" in capsys.readouterr().err
