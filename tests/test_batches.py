"""The order in which the attention's joint starts copies and waits for them (csrc/batches.cuh), on the host
against a model of its barrier: nothing is started after a wait that gave up, whichever threads saw it."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    out = tmp_path_factory.mktemp("batches")

    def compiled(name, *flags):
        exe = str(out / name)
        subprocess.run(["g++", "-std=c++20", "-O1", "-pthread", *flags, os.path.join(HERE, "batches_model.cpp"), "-o", exe],
                       check=True)

        def run(*args):
            r = subprocess.run([exe, *map(str, args)], check=True, capture_output=True, text=True, timeout=120)
            v = [int(x) for x in r.stdout.split()]
            return v[0], v[1:5], v[5:9]

        return run

    return compiled("model"), compiled("planted", "-DPLANTED")


@pytest.mark.parametrize("n,batch", [(1, 1), (2, 2), (38, 38), (38, 10), (9, 3), (152, 16)])
@pytest.mark.parametrize("joints", [1, 2])
def test_all_slices_are_used_once(model, n, batch, joints):
    assert model[0](n, batch, joints, -1, 0) == (0, [joints * -(-n // batch)] * 4, [1] * 4)


@pytest.mark.parametrize("who", [1, 2, 8, 6, 15])
@pytest.mark.parametrize("n,batch,joints,at", [(38, 10, 1, 0), (38, 10, 1, 2), (38, 10, 1, 3), (38, 38, 2, 0), (20, 10, 2, 1),
                                               (20, 10, 2, 2)])
def test_nothing_is_started_after_a_wait_that_gave_up(model, n, batch, joints, at, who):
    violations, used, ok = model[0](n, batch, joints, at, who)
    assert violations == 0
    assert used == [at if who >> w & 1 else at + 1 for w in range(4)]
    last = at + 1 == joints * -(-n // batch)
    assert all(not r for w, r in enumerate(ok) if who >> w & 1 or not last)


def test_the_model_sees_a_joint_that_goes_on(model):
    assert model[1](38, 10, 1, -1, 0) == (0, [4] * 4, [1] * 4)
    for n, batch, joints, at in ((38, 10, 1, 0), (38, 38, 2, 0)):
        assert model[1](n, batch, joints, at, 15)[0] > 0
