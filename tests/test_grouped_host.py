"""CPU checks of what the grouped products do on the host."""
import ctypes

import torch

INVALID = 1


def test_the_unread_workspace_is_the_librarys(moelib, monkeypatch):
    """A call without a workspace writes to memory that no allocator hands out: a
    block of the caching allocator may have an earlier owner whose work on the
    stream it was freed on is still to come, and these calls run on any stream."""
    import moe_expert_layer_08_b200 as m
    asked = []

    class Library:
        @staticmethod
        def moe_grouped_unread_workspace(device, where):
            asked.append(device)
            where._obj.value = 0x70000 + 0x1000 * device
            return 0

    def no_allocator(*args, **kwargs):
        raise AssertionError("memory of the allocator")

    monkeypatch.setattr(m, "_unread", {})
    monkeypatch.setattr(m, "load", lambda: Library)
    for name in ("empty", "zeros", "full"):
        monkeypatch.setattr(torch, name, no_allocator)
    for device in (0, 1, 0):
        at, size = m._grouped_workspace(None, torch.device("cuda", device))
        assert at == 0x70000 + 0x1000 * device and size == m._GROUPED_WORKSPACE
    assert asked == [0, 1]


def test_unread_workspace_refusals(moelib):
    p = ctypes.c_void_p()
    assert moelib.moe_grouped_unread_workspace(-1, ctypes.byref(p)) == INVALID
    assert moelib.moe_grouped_unread_workspace(0, None) == INVALID
    assert p.value is None
