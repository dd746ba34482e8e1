"""examples/decode_step.py refuses arguments with which its steps would attend to nothing."""
import pytest


@pytest.mark.parametrize("argv", [["--context", "32"], ["--context", "58"], ["--context", "100", "--steps", "92"],
                                  ["--context", "0", "--steps", "1"], ["--steps", "0"], ["--batch", "0"], ["--layers", "0"]])
def test_refused(argv, capsys):
    from examples import decode_step as ex
    with pytest.raises(SystemExit):
        ex.arguments(argv)
    assert "must be" in capsys.readouterr().err


@pytest.mark.parametrize("argv,context,steps", [([], 4096, 50), (["--context", "59"], 59, 50),
                                                (["--context", "20", "--steps", "11"], 20, 11)])
def test_taken(argv, context, steps):
    from examples import decode_step as ex
    args = ex.arguments(argv)
    assert (args.context, args.steps) == (context, steps)
    assert args.context - args.steps - ex.SPARE > 0  # the first timed position
