"""Workspace sizes that are kept: one for each device."""


def test_backward_sizes_of_two_devices(lib, monkeypatch):
    # a fake of the size query, whose answer goes by the current device
    F, here = lib.functional, [0]
    monkeypatch.setattr(F.C, "qkv_prologue_bwd_workspace_size_ex", lambda L, V, T: 1000 + here[0] + (V is not None) * 50)
    F._backward_workspace.cache_clear()
    try:
        for device in (0, 1, 0, 2):
            here[0] = device
            assert F._backward_workspace("interleaved", 8, 2, 64, 100, False, device) == 1000 + device
            assert F._backward_workspace("interleaved", 8, 2, 64, 100, True, device) == 1050 + device
    finally:
        F._backward_workspace.cache_clear()
