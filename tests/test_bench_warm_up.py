"""bench.py's warm-up: the interpreter's full collection of what the imports left comes
before it, so that none falls due in the timed passes."""
import gc

import bench


def test_order(monkeypatch):
    log = []
    monkeypatch.setattr(gc, "collect", lambda *a: log.append("collect"))
    bench.warm_up(lambda: log.append("run"), 3, lambda: log.append("wait"))
    assert log == ["collect", "run", "run", "run", "wait"]


def test_no_full_collection_after_it():
    """With as many new objects as make one due otherwise."""
    full = []
    note = lambda phase, info: full.append(phase) if info["generation"] == 2 else None
    kept = []
    limits = gc.get_threshold()

    def passes(n):  # 30 objects a pass stay, many collections of the young ones
        for _ in range(n):
            kept.extend([] for _ in range(30))

    def due():  # new objects that the young generations have handed on, a full collection next
        gc.disable()
        gc.collect()
        kept.extend([] for _ in range(len(gc.get_objects())))
        gc.set_threshold(20, 2, 2)
        gc.collect(1)
        gc.enable()

    gc.callbacks.append(note)
    try:
        due()
        full.clear()
        passes(25)
        assert full, "the state of the test makes none due"
        due()
        bench.warm_up(lambda: None, 3, lambda: None)
        full.clear()
        passes(25)
        assert not full
    finally:
        gc.enable()
        gc.set_threshold(*limits)
        gc.callbacks.remove(note)
