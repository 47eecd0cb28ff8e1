"""The binding of the operators before the step, first used by two host threads
at once (no GPU: a stand-in for the library that says who goes on when)."""
import threading

from mixed_precision_sharded_amd import binding, training

NAMES = [*training._SIGNATURES, *training._SIZES]


class Library:
    """Entry points by name.  The thread "one" stops at its last lookup until the
    thread "two" has come to its first, and that one until `one` has returned."""

    def __init__(self):
        self.functions = {}
        self.two_may_start, self.two_is_inside, self.one_is_done = (threading.Event() for _ in range(3))

    def __getattr__(self, name):
        if threading.current_thread().name == "one" and name == NAMES[-1]:
            self.two_may_start.set()
            assert self.two_is_inside.wait(60)
        if threading.current_thread().name == "two":
            self.two_is_inside.set()
            assert self.one_is_done.wait(60)
        return self.functions.setdefault(name, lambda *args: 7)


def test_two_threads_at_first_use_both_find_the_entry_points(monkeypatch):
    library = Library()
    monkeypatch.setattr(binding, "_lib", library)
    got = {}

    def work():
        me = threading.current_thread().name
        if me == "two":
            assert library.two_may_start.wait(60)
        try:
            got[me] = training._function(NAMES[0])
        except Exception as e:  # noqa: BLE001 - the test says what it was
            got[me] = e
        if me == "one":
            library.one_is_done.set()

    threads = [threading.Thread(target=work, name=name, daemon=True) for name in ("one", "two")]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert got == {"one": library.functions[NAMES[0]], "two": library.functions[NAMES[0]]}
    for names in (training._SIGNATURES, training._SIZES):
        for n, argtypes in names.items():
            assert library.functions[n].argtypes == argtypes and library.functions[n].restype is not None


def test_another_library_is_bound_anew(monkeypatch):
    for _ in range(2):
        library = Library()
        monkeypatch.setattr(binding, "_lib", library)
        assert training._function(NAMES[0]) is library.functions[NAMES[0]]
        assert training.policy_loss_workspace_bytes(3, 100) == 7
