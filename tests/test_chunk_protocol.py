"""The chunk kernel's barriers on a CPU model (chunk_protocol.py): every form of
the kernel, whole runs and runs in which a wait gives up; and that the model sees
protocols that are wrong."""
import itertools

import pytest

from chunk_protocol import Run, Wrong, constants

STAGES, AHEAD, SCALES = constants()
FORMS = [(k8, D, two) for (k8, D), two in itertools.product(STAGES, (True, False))]
IDLE = [(), ((0, 2), (0, 3), (1, 2), (1, 3)), ((1, 1), (1, 2), (1, 3))]


def run(form, nt, seed, **kw):
    k8, D, two = form
    return Run(nt, two, k8, kw.pop("stages", STAGES[k8, D]), kw.pop("ahead", AHEAD), kw.pop("scales", SCALES),
               seed, **kw).go()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("nt", range(20))
def test_whole_runs(form, nt):
    for seed, idle in itertools.product(range(8), IDLE):
        assert run(form, nt, seed, idle=idle) == "done"


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("nt", [1, 2, 3, 5, 8, 13])
def test_a_load_that_is_never_reported(form, nt):
    """Every load in turn: the CTA ends, with nothing on its way, and says so."""
    for lost in range(2 * nt):
        for seed in range(6):
            assert run(form, nt, seed, lost=lost, idle=IDLE[seed % 3]) == "failed"


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("nt", [1, 2, 4, 9])
def test_waits_that_give_up_anywhere(form, nt):
    ends = {run(form, nt, seed, spurious=p, idle=IDLE[seed % 3]) for seed in range(60) for p in (0.01, 0.05)}
    assert "failed" in ends


def found(forms=FORMS, nts=range(1, 20), seeds=6, **kw):
    """What the model holds against a protocol."""
    what = set()
    for form, nt, seed in itertools.product(forms, nts, range(seeds)):
        try:
            run(form, nt, seed, **kw)
        except Wrong as e:
            what.add(str(e))
    return what


@pytest.mark.parametrize("change,what", [
    (dict(mutant="a phase too far"), "a wait passed by an earlier phase"),
    (dict(mutant="half of P"), "P of another tile"),
    (dict(mutant="K freed early"), "a product over a stage that holds something else"),
    (dict(mutant="a stage taken early"), "a stage written under a product"),
    (dict(scales=2), "scales of another tile"),
    (dict(mutant="arrivals held back", ahead=1), "every role waits"),
    (dict(stages=1), "every role waits"),
    (dict(mutant="products go on", spurious=0.02), "a product over a stage that holds something else"),
    (dict(mutant="P without S", spurious=0.02), "P of another tile"),
    (dict(mutant="load goes on", spurious=0.02), "a stage written under a product"),
    (dict(mutant="not drained", spurious=0.02), "TMEM freed under a product"),
    (dict(mutant="drained by the product warp's waits alone", spurious=0.02), "TMEM freed under a product"),
])
def test_wrong_protocols_are_seen(change, what):
    assert what in found(**change)
