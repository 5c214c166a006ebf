"""First calls of two threads at once: the binding's table of entry points is either empty, and the thread
fills it, or whole."""
from __future__ import annotations

import torch  # noqa: F401  before the library, which takes the HIP runtime that torch has loaded


def test_entry_points_appear_together(monkeypatch):
    """A library whose entry points are asked for one by one, and another thread's look at the table each time."""
    from weight_only_bit_rtn_amd import adapters

    seen = []

    class Entry:
        argtypes = restype = None

    class Library:
        def __getattr__(self, name):  # each time: nothing is kept on the object
            seen.append(set(adapters._entry))
            if name.startswith("lowbit_lora_plan_"):  # the plan takes no workspace
                raise AttributeError(name)
            return Entry()

    library = Library()
    monkeypatch.setattr(adapters, "_load_library", lambda: library)
    monkeypatch.setattr(adapters, "_declared", None)
    monkeypatch.setattr(adapters, "_entry", {})
    assert adapters._lib() is library
    whole = {"lowbit_lora_plan", "lowbit_lora", "lowbit_lora_grad"}
    assert set(adapters._entry) == whole and seen
    assert all(names in (set(), whole) for names in seen)
